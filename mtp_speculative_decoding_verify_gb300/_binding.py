"""ctypes binding of libmtpverify.so (include/mtp_verify.h).

Argument marshalling only: tensors are checked for device, dtype, shape and
contiguity, their raw pointers go into the C argument structs, and every step
of the verify path runs in the library's CUDA kernels. There is no CPU
fallback: if the library is missing, loading it raises.
"""
import ctypes
import operator
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_build", "libmtpverify.so")

MTP_OK, MTP_INVALID_ARG, MTP_UNSUPPORTED, MTP_CUDA_ERROR, MTP_DEVICE_ERROR = range(5)
ABI_VERSION = 5   # MTP_ABI_VERSION of the header the structs below mirror
MTP_F32, MTP_BF16 = 0, 1
MAX_DRAFTS = 15
BLOCK_SIZE = 64

_P = ctypes.c_void_p
_I = ctypes.c_int32


class AttnArgs(ctypes.Structure):
    _fields_ = [("q", _P), ("k_new", _P), ("v_new", _P), ("k_cache", _P), ("v_cache", _P),
                ("block_table", _P), ("ctx_lens", _P), ("out", _P),
                ("B", _I), ("D", _I), ("Hq", _I), ("Hkv", _I), ("d_qk", _I), ("d_v", _I),
                ("block_size", _I), ("max_blocks", _I), ("num_blocks", _I), ("is_mla", _I),
                ("sm_scale", ctypes.c_float), ("dtype", _I), ("parents", _P), ("workspace", _P),
                ("workspace_bytes", ctypes.c_size_t), ("timing_events", _P * 2)]


class LmArgs(ctypes.Structure):
    _fields_ = [("hidden", _P), ("lm_head", _P), ("tokens", _P), ("mode", _P), ("temperature", _P),
                ("q_draft", _P), ("seed", ctypes.c_uint64), ("out_tokens", _P), ("num_accepted", _P),
                ("tie_flags", _P), ("lse_out", _P), ("argmax_out", _P), ("logits_debug", _P),
                ("B", _I), ("D", _I), ("H", _I), ("V", _I), ("dtype", _I), ("any_sampling", _I),
                ("relaxed_topk", _I), ("relaxed_delta", ctypes.c_float), ("parents", _P), ("accepted_nodes", _P),
                ("workspace", _P), ("workspace_bytes", ctypes.c_size_t), ("timing_events", _P * 2),
                ("q_ready_event", _P)]


class DraftArgs(ctypes.Structure):
    _fields_ = [("hidden", _P), ("lm_head", _P), ("out_tokens", _P), ("lse_out", _P), ("B", _I), ("H", _I),
                ("V", _I), ("dtype", _I), ("workspace", _P), ("workspace_bytes", ctypes.c_size_t),
                ("timing_events", _P * 2)]


class KvCompactArgs(ctypes.Structure):
    _fields_ = [("k_cache", _P), ("v_cache", _P), ("block_table", _P), ("ctx_lens", _P), ("accepted_nodes", _P),
                ("num_accepted", _P), ("B", _I), ("D", _I), ("Hkv", _I), ("d_qk", _I), ("d_v", _I),
                ("block_size", _I), ("max_blocks", _I), ("num_blocks", _I), ("is_mla", _I), ("dtype", _I)]


class RollbackArgs(ctypes.Structure):
    _fields_ = [("block_table", _P), ("seq_lens", _P), ("num_accepted", _P), ("free_list", _P),
                ("free_count", _P), ("B", _I), ("D", _I), ("block_size", _I), ("max_blocks", _I),
                ("free_capacity", _I)]


class Kv8AppendArgs(ctypes.Structure):
    _fields_ = [("k_new", _P), ("v_new", _P), ("starts", _P), ("k_cache", _P), ("v_cache", _P), ("k_scale", _P),
                ("v_scale", _P), ("block_table", _P), ("ctx_lens", _P), ("T", _I), ("B", _I), ("Hkv", _I), ("d", _I),
                ("block_size", _I), ("max_blocks", _I), ("num_blocks", _I), ("dtype", _I)]


class WindowAttnArgs(ctypes.Structure):
    _fields_ = [("q", _P), ("k_new", _P), ("v_new", _P), ("k_cache", _P), ("v_cache", _P), ("k_scale", _P),
                ("v_scale", _P), ("block_table", _P), ("ctx_lens", _P), ("out", _P), ("B", _I), ("D", _I), ("Hq", _I),
                ("Hkv", _I), ("d", _I), ("block_size", _I), ("max_blocks", _I), ("num_blocks", _I), ("window", _I),
                ("sinks", _I), ("sm_scale", ctypes.c_float), ("dtype", _I), ("workspace", _P),
                ("workspace_bytes", ctypes.c_size_t), ("timing_events", _P * 2)]


class WindowReleaseArgs(ctypes.Structure):
    _fields_ = [("block_table", _P), ("seq_lens", _P), ("free_list", _P), ("free_count", _P), ("B", _I),
                ("block_size", _I), ("max_blocks", _I), ("free_capacity", _I), ("window", _I), ("sinks", _I),
                ("workspace", _P), ("workspace_bytes", ctypes.c_size_t)]


class BlockAssignArgs(ctypes.Structure):
    _fields_ = [("block_table", _P), ("seq_lens", _P), ("starts", _P), ("free_list", _P), ("free_count", _P),
                ("slot_map", _P), ("taken", _P), ("B", _I), ("T", _I), ("block_size", _I), ("max_blocks", _I),
                ("free_capacity", _I), ("workspace", _P), ("workspace_bytes", ctypes.c_size_t)]


class KvAppendArgs(ctypes.Structure):
    _fields_ = [("k_new", _P), ("v_new", _P), ("slot_map", _P), ("k_cache", _P), ("v_cache", _P),
                ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64), ("T", _I), ("Hkv", _I), ("d_qk", _I),
                ("d_v", _I), ("block_size", _I), ("num_blocks", _I), ("is_mla", _I), ("dtype", _I)]


class PrefixAttnArgs(ctypes.Structure):
    _fields_ = [("q", _P), ("k_new", _P), ("v_new", _P), ("k_cache", _P), ("v_cache", _P), ("block_table", _P),
                ("ctx_lens", _P), ("group_starts", _P), ("prefix_blocks", _P), ("out", _P), ("B", _I), ("D", _I),
                ("G", _I), ("Hq", _I), ("Hkv", _I), ("d", _I), ("block_size", _I), ("max_blocks", _I),
                ("num_blocks", _I), ("sm_scale", ctypes.c_float), ("dtype", _I), ("parents", _P), ("workspace", _P),
                ("workspace_bytes", ctypes.c_size_t), ("timing_events", _P * 2)]


class MtpError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__("mtp status %d: %s" % (code, msg))
        self.code = code


_lib = None


def lib():
    """Load libmtpverify.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libmtpverify.so is not built (run __graft_entry__.build() or "
                               "python -m mtp_speculative_decoding_verify_gb300.build)")
        L = ctypes.CDLL(LIB_PATH)
        L.mtp_verify_attention.argtypes = [ctypes.POINTER(AttnArgs), _P]
        L.mtp_verify_attention.restype = ctypes.c_int
        L.mtp_attention_workspace_size.argtypes = [ctypes.POINTER(AttnArgs)]
        L.mtp_attention_workspace_size.restype = ctypes.c_size_t
        L.mtp_verify_logits_accept.argtypes = [ctypes.POINTER(LmArgs), _P]
        L.mtp_verify_logits_accept.restype = ctypes.c_int
        L.mtp_lmhead_workspace_size.argtypes = [ctypes.POINTER(LmArgs)]
        L.mtp_lmhead_workspace_size.restype = ctypes.c_size_t
        L.kv_rollback.argtypes = [ctypes.POINTER(RollbackArgs), _P]
        L.kv_rollback.restype = ctypes.c_int
        L.mtp_last_error.argtypes = []
        L.mtp_last_error.restype = ctypes.c_char_p
        L.mtp_sync_status.argtypes = [_P]
        L.mtp_sync_status.restype = ctypes.c_int
        L.mtp_rng_debug.argtypes = [ctypes.c_uint64, ctypes.c_uint32, ctypes.c_uint32, ctypes.c_uint32,
                                    ctypes.c_uint32, ctypes.c_int32, _P, _P, _P, _P]
        L.mtp_rng_debug.restype = ctypes.c_int
        L.mtp_wait_selftest.argtypes = [ctypes.c_uint64, _P]
        L.mtp_wait_selftest.restype = ctypes.c_int
        L.mtp_verify_logits_accept_noalloc.argtypes = [ctypes.POINTER(LmArgs), _P]
        L.mtp_verify_logits_accept_noalloc.restype = ctypes.c_int
        L.mtp_noalloc_scratch_bytes.argtypes = []
        L.mtp_noalloc_scratch_bytes.restype = ctypes.c_size_t
        L.mtp_last_launch_count.argtypes = []
        L.mtp_last_launch_count.restype = ctypes.c_int
        L.mtp_draft_workspace_size.argtypes = [ctypes.POINTER(DraftArgs)]
        L.mtp_draft_workspace_size.restype = ctypes.c_size_t
        L.mtp_draft_argmax.argtypes = [ctypes.POINTER(DraftArgs), _P]
        L.mtp_draft_argmax.restype = ctypes.c_int
        L.mtp_tree_kv_compact.argtypes = [ctypes.POINTER(KvCompactArgs), _P]
        L.mtp_tree_kv_compact.restype = ctypes.c_int
        L.mtp_kv8_append.argtypes = [ctypes.POINTER(Kv8AppendArgs), _P]
        L.mtp_kv8_append.restype = ctypes.c_int
        for name in ("kv8", "window"):
            size, call = getattr(L, "mtp_attention_%s_workspace_size" % name), getattr(L, "mtp_verify_attention_" + name)
            size.argtypes = [ctypes.POINTER(WindowAttnArgs)]
            size.restype = ctypes.c_size_t
            call.argtypes = [ctypes.POINTER(WindowAttnArgs), _P]
            call.restype = ctypes.c_int
        L.mtp_window_release_workspace_size.argtypes = [ctypes.c_int32]
        L.mtp_window_release_workspace_size.restype = ctypes.c_size_t
        L.kv_window_release.argtypes = [ctypes.POINTER(WindowReleaseArgs), _P]
        L.kv_window_release.restype = ctypes.c_int
        L.mtp_block_assign_workspace_size.argtypes = [ctypes.c_int32, ctypes.c_int32]
        L.mtp_block_assign_workspace_size.restype = ctypes.c_size_t
        L.kv_block_assign.argtypes = [ctypes.POINTER(BlockAssignArgs), _P]
        L.kv_block_assign.restype = ctypes.c_int
        L.mtp_kv_append.argtypes = [ctypes.POINTER(KvAppendArgs), _P]
        L.mtp_kv_append.restype = ctypes.c_int
        L.mtp_attention_prefix_workspace_size.argtypes = [ctypes.POINTER(PrefixAttnArgs)]
        L.mtp_attention_prefix_workspace_size.restype = ctypes.c_size_t
        L.mtp_verify_attention_prefix.argtypes = [ctypes.POINTER(PrefixAttnArgs), _P]
        L.mtp_verify_attention_prefix.restype = ctypes.c_int
        L.mtp_hbm_read_probe.argtypes = [_P, ctypes.c_size_t, _P, ctypes.c_int32, ctypes.c_int32, _P]
        L.mtp_hbm_read_probe.restype = ctypes.c_int
        L.mtp_abi_version.argtypes = []
        L.mtp_abi_version.restype = ctypes.c_int
        L.mtp_abi_struct_size.argtypes = [ctypes.c_int]
        L.mtp_abi_struct_size.restype = ctypes.c_size_t
        if L.mtp_abi_version() != ABI_VERSION:
            raise RuntimeError("library ABI version %d, binding expects %d" % (L.mtp_abi_version(), ABI_VERSION))
        for which, st in enumerate((AttnArgs, LmArgs, RollbackArgs, DraftArgs, KvCompactArgs, Kv8AppendArgs,
                                    WindowAttnArgs, WindowReleaseArgs, BlockAssignArgs, KvAppendArgs,
                                    PrefixAttnArgs)):
            if L.mtp_abi_struct_size(which) != ctypes.sizeof(st):
                raise RuntimeError("ABI mismatch for %s" % st.__name__)
        _lib = L
    return _lib


def _check(rc):
    if rc != MTP_OK:
        raise MtpError(rc, lib().mtp_last_error().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dev(t, name, dtype=None, shape=None):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def _dtype_code(t):
    if t.dtype == torch.float32:
        return MTP_F32
    if t.dtype == torch.bfloat16:
        return MTP_BF16
    raise ValueError("tensors must be float32 or bfloat16, got %s" % t.dtype)


def _stream_handle(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


_ws_cache = {}


def _workspace(nbytes, device, key):
    """A cached device buffer of at least nbytes (torch allocator), 256-byte aligned."""
    buf = _ws_cache.get((device, key))
    if buf is None or buf.numel() < nbytes:
        buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
        _ws_cache[(device, key)] = buf
    return buf


def attn_args(q, k_new, v_new, k_cache, v_cache, block_table, ctx_lens, out, *, sm_scale=None, workspace=None,
              parents=None):
    """Fill AttnArgs from tensors (see mtp_verify_attention for shapes)."""
    is_mla = v_cache is None
    B, R, Hq, d_qk = q.shape
    D = R - 1
    dt = q.dtype
    if is_mla:
        num_blocks, bs, Hkv, dk = k_cache.shape
        d_v = out.shape[-1]
        _dev(k_new, "k_new", dt, (B, R, d_qk))
    else:
        num_blocks, bs, Hkv, dk = k_cache.shape
        d_v = v_cache.shape[-1]
        _dev(k_new, "k_new", dt, (B, R, Hkv, d_qk))
        _dev(v_new, "v_new", dt, (B, R, Hkv, d_v))
        _dev(v_cache, "v_cache", dt, (num_blocks, bs, Hkv, d_v))
    _dev(q, "q", dt)
    _dev(k_cache, "k_cache", dt)
    _dev(out, "out", dt, (B, R, Hq, d_v))
    _dev(block_table, "block_table", torch.int32)
    _dev(ctx_lens, "ctx_lens", torch.int32, (B,))
    _dev(parents, "parents", torch.int32, (B, R))
    if dk != d_qk:
        raise ValueError("k_cache head dim %d != q head dim %d" % (dk, d_qk))
    a = AttnArgs(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                 _ptr(ctx_lens), _ptr(out), B, D, Hq, Hkv, d_qk, d_v, bs, block_table.shape[1], num_blocks,
                 int(is_mla), float(sm_scale if sm_scale is not None else d_qk ** -0.5), _dtype_code(q),
                 _ptr(parents), None, 0)
    n = lib().mtp_attention_workspace_size(ctypes.byref(a))
    if n == 0:
        _check(MTP_INVALID_ARG)
    if workspace is None:
        workspace = _workspace(n, q.device, "attn")
    a.workspace = _ptr(workspace)
    a.workspace_bytes = workspace.numel() * workspace.element_size()
    return a


def mtp_verify_attention(q, k_new, v_new, k_cache, v_cache, block_table, ctx_lens, out, *, sm_scale=None,
                         workspace=None, stream=None, parents=None):
    """Append the verify tokens' K/V to the paged cache and run verify attention into `out`.

    q [B, R, Hq, d_qk]; GQA/MHA: k_new [B, R, Hkv, d], v_new [B, R, Hkv, d], caches [blocks, 64, Hkv, d];
    absorbed MLA: k_new [B, R, 576], v_new = v_cache = None, k_cache [blocks, 64, 1, 576];
    block_table [B, max_blocks] int32, ctx_lens [B] int32, out [B, R, Hq, d_v];
    parents [B, R] int32 (tree drafts) or None (chains).
    """
    a = attn_args(q, k_new, v_new, k_cache, v_cache, block_table, ctx_lens, out, sm_scale=sm_scale,
                  workspace=workspace, parents=parents)
    _check(lib().mtp_verify_attention(ctypes.byref(a), _stream_handle(stream)))


def lm_args(hidden, lm_head, tokens, mode, temperature, q_draft, seed, out_tokens, num_accepted, tie_flags,
            lse_out=None, argmax_out=None, logits_debug=None, workspace=None, relaxed_topk=0, relaxed_delta=0.0,
            parents=None, accepted_nodes=None):
    """Fill LmArgs from tensors (see mtp_verify_logits_accept for shapes)."""
    B, R = tokens.shape
    D = R - 1
    V, H = lm_head.shape
    dt = lm_head.dtype
    any_sampling = q_draft is not None
    _dev(hidden, "hidden", dt, (B * R, H))
    _dev(lm_head, "lm_head", dt)
    _dev(tokens, "tokens", torch.int32)
    _dev(mode, "mode", torch.uint8, (B,))
    _dev(temperature, "temperature", torch.float32, (B,))
    _dev(q_draft, "q_draft", torch.float32, (B, D, V))
    _dev(out_tokens, "out_tokens", torch.int32, (B, R))
    _dev(num_accepted, "num_accepted", torch.int32, (B,))
    _dev(tie_flags, "tie_flags", torch.uint8, (B,))
    _dev(lse_out, "lse_out", torch.float32, (B, R))
    _dev(argmax_out, "argmax_out", torch.int32, (B, R))
    _dev(logits_debug, "logits_debug", torch.float32, (B * R, V))
    _dev(parents, "parents", torch.int32, (B, R))
    _dev(accepted_nodes, "accepted_nodes", torch.int32, (B, R))
    a = LmArgs(_ptr(hidden), _ptr(lm_head), _ptr(tokens), _ptr(mode), _ptr(temperature), _ptr(q_draft),
               int(seed) & 0xFFFFFFFFFFFFFFFF, _ptr(out_tokens), _ptr(num_accepted), _ptr(tie_flags), _ptr(lse_out),
               _ptr(argmax_out), _ptr(logits_debug), B, D, H, V, _dtype_code(lm_head), int(any_sampling),
               int(relaxed_topk), float(relaxed_delta), _ptr(parents), _ptr(accepted_nodes), None, 0)
    n = lib().mtp_lmhead_workspace_size(ctypes.byref(a))
    if n == 0:
        _check(MTP_INVALID_ARG)
    if workspace is None:
        workspace = _workspace(n, hidden.device, "lm")
    a.workspace = _ptr(workspace)
    a.workspace_bytes = workspace.numel() * workspace.element_size()
    return a


def mtp_verify_logits_accept(hidden, lm_head, tokens, mode, temperature, q_draft, seed, out_tokens, num_accepted,
                             tie_flags, lse_out=None, argmax_out=None, logits_debug=None, workspace=None,
                             stream=None, relaxed_topk=0, relaxed_delta=0.0, parents=None, accepted_nodes=None,
                             q_ready_event=None):
    """LM head + streaming softmax statistics + greedy / rejection-sampling / relaxed acceptance.

    hidden [B*R, H], lm_head [V, H] (float32 or bfloat16), tokens [B, R] int32, mode [B] uint8,
    temperature [B] float32 or None, q_draft [B, D, V] float32 or None (None: every request greedy),
    outputs out_tokens [B, R] int32, num_accepted [B] int32, tie_flags [B] uint8, optional lse_out / argmax_out
    [B, R] and logits_debug [B*R, V]. relaxed_topk / relaxed_delta: the relaxed rule of mode-2 requests.
    parents [B, R] int32: tree drafts (greedy); accepted_nodes [B, R] int32: optional output, the accepted path.
    q_ready_event: optional torch.cuda.Event recorded after q_draft's copy; the stream waits for it only
    after the LM-head GEMM has been launched, so the copy may overlap the GEMM.
    """
    a = lm_args(hidden, lm_head, tokens, mode, temperature, q_draft, seed, out_tokens, num_accepted, tie_flags,
                lse_out, argmax_out, logits_debug, workspace, relaxed_topk, relaxed_delta, parents, accepted_nodes)
    a.q_ready_event = None if q_ready_event is None else q_ready_event.cuda_event
    _check(lib().mtp_verify_logits_accept(ctypes.byref(a), _stream_handle(stream)))


def draft_args(hidden, lm_head, out_tokens, lse_out=None, workspace=None):
    """Fill DraftArgs from tensors (see mtp_draft_argmax for shapes)."""
    B, H = hidden.shape
    V = lm_head.shape[0]
    dt = lm_head.dtype
    _dev(hidden, "hidden", dt, (B, H))
    _dev(lm_head, "lm_head", dt, (V, H))
    _dev(out_tokens, "out_tokens", torch.int32, (B,))
    _dev(lse_out, "lse_out", torch.float32, (B,))
    a = DraftArgs(_ptr(hidden), _ptr(lm_head), _ptr(out_tokens), _ptr(lse_out), B, H, V, _dtype_code(lm_head),
                  None, 0)
    n = lib().mtp_draft_workspace_size(ctypes.byref(a))
    if n == 0:
        _check(MTP_INVALID_ARG)
    if workspace is None:
        workspace = _workspace(n, hidden.device, "draft")
    a.workspace = _ptr(workspace)
    a.workspace_bytes = workspace.numel() * workspace.element_size()
    return a


def mtp_draft_argmax(hidden, lm_head, out_tokens, lse_out=None, workspace=None, stream=None):
    """One greedy draft step over the shared LM head: out_tokens[b] = argmax_v hidden[b] . lm_head[v]
    (lowest id on ties); hidden [B, H], lm_head [V, H] (float32 or bfloat16), out_tokens [B] int32,
    optional lse_out [B] float32."""
    a = draft_args(hidden, lm_head, out_tokens, lse_out, workspace)
    _check(lib().mtp_draft_argmax(ctypes.byref(a), _stream_handle(stream)))


def mtp_verify_logits_accept_noalloc(hidden, lm_head, tokens, mode, temperature, q_draft, seed, out_tokens,
                                     num_accepted, tie_flags, lse_out=None, argmax_out=None, logits_debug=None,
                                     stream=None, relaxed_topk=0, relaxed_delta=0.0, parents=None,
                                     accepted_nodes=None):
    """mtp_verify_logits_accept for callers that cannot allocate device memory:
    the scratch lives in a fixed array owned by the library (no workspace is
    allocated or passed). Raises MtpError if the batch needs more scratch
    than that array holds. Calls must not overlap on the GPU."""
    a = LmArgs(_ptr(hidden), _ptr(lm_head), _ptr(tokens), _ptr(mode), _ptr(temperature), _ptr(q_draft),
               int(seed) & 0xFFFFFFFFFFFFFFFF, _ptr(out_tokens), _ptr(num_accepted), _ptr(tie_flags), _ptr(lse_out),
               _ptr(argmax_out), _ptr(logits_debug), tokens.shape[0], tokens.shape[1] - 1, lm_head.shape[1],
               lm_head.shape[0], _dtype_code(lm_head), int(q_draft is not None), int(relaxed_topk),
               float(relaxed_delta), _ptr(parents), _ptr(accepted_nodes), None, 0)
    for t, n in ((hidden, "hidden"), (lm_head, "lm_head"), (tokens, "tokens"), (mode, "mode"),
                 (temperature, "temperature"), (q_draft, "q_draft"), (out_tokens, "out_tokens"),
                 (num_accepted, "num_accepted"), (tie_flags, "tie_flags"), (lse_out, "lse_out"),
                 (argmax_out, "argmax_out"), (logits_debug, "logits_debug"), (parents, "parents"),
                 (accepted_nodes, "accepted_nodes")):
        _dev(t, n)
    _check(lib().mtp_verify_logits_accept_noalloc(ctypes.byref(a), _stream_handle(stream)))


def compact_args(k_cache, v_cache, block_table, ctx_lens, accepted_nodes, num_accepted):
    """Fill KvCompactArgs from tensors (see mtp_tree_kv_compact)."""
    B, R = accepted_nodes.shape
    is_mla = v_cache is None
    num_blocks, bs, Hkv, d_qk = k_cache.shape
    d_v = d_qk if is_mla else v_cache.shape[-1]
    dt = k_cache.dtype
    _dev(k_cache, "k_cache", dt)
    _dev(v_cache, "v_cache", dt, (num_blocks, bs, Hkv, d_v))
    _dev(block_table, "block_table", torch.int32)
    _dev(ctx_lens, "ctx_lens", torch.int32, (B,))
    _dev(accepted_nodes, "accepted_nodes", torch.int32, (B, R))
    _dev(num_accepted, "num_accepted", torch.int32, (B,))
    return KvCompactArgs(_ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(ctx_lens), _ptr(accepted_nodes),
                         _ptr(num_accepted), B, R - 1, Hkv, d_qk, d_v, bs, block_table.shape[1], num_blocks,
                         int(is_mla), _dtype_code(k_cache))


def mtp_tree_kv_compact(k_cache, v_cache, block_table, ctx_lens, accepted_nodes, num_accepted, stream=None):
    """Move each request's accepted tree path K/V (accepted_nodes [B, R], num_accepted [B]) to slots
    ctx+1 .. ctx+n of the paged cache (ctx_lens = context lengths before the step); v_cache None for MLA."""
    a = compact_args(k_cache, v_cache, block_table, ctx_lens, accepted_nodes, num_accepted)
    _check(lib().mtp_tree_kv_compact(ctypes.byref(a), _stream_handle(stream)))


def rollback_args(block_table, seq_lens, num_accepted, free_list, free_count, *, D):
    B, max_blocks = block_table.shape
    _dev(block_table, "block_table", torch.int32)
    _dev(seq_lens, "seq_lens", torch.int32, (B,))
    _dev(num_accepted, "num_accepted", torch.int32, (B,))
    _dev(free_list, "free_list", torch.int32)
    _dev(free_count, "free_count", torch.int32, (1,))
    return RollbackArgs(_ptr(block_table), _ptr(seq_lens), _ptr(num_accepted), _ptr(free_list), _ptr(free_count),
                        B, D, BLOCK_SIZE, max_blocks, free_list.numel())


def kv_rollback(block_table, seq_lens, num_accepted, free_list, free_count, *, D, stream=None):
    """Truncate each request to ctx + n + 1 slots and release blocks holding only rejected drafts."""
    a = rollback_args(block_table, seq_lens, num_accepted, free_list, free_count, D=D)
    _check(lib().kv_rollback(ctypes.byref(a), _stream_handle(stream)))


def _refuse(t, name, index, dtype, shape):
    """Say what is wrong with one tensor argument of a call."""
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.get_device() != index:
        raise ValueError("%s is on cuda:%d, the call's first tensor on cuda:%d" % (name, t.get_device(), index))
    _dev(t, name, dtype, shape)


def _check_all(index, args):
    """Each (tensor, name, dtype, shape): on that device, of that type and shape, contiguous. (These checks are a large
    part of a small call's time on the host, so the tests that pass are made in place.)"""
    for t, name, dtype, shape in args:
        if t.get_device() != index or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
            _refuse(t, name, index, dtype, shape)


def _cuda_index(t, name):
    index = t.get_device()
    if index < 0:
        raise ValueError("%s must be a CUDA tensor" % name)
    return index


def _on(index, stream, call):
    """_check(call(stream handle)) with device `index` current, on `stream` or that device's current one."""
    if stream is None and torch.cuda.current_device() == index:
        _check(call(_raw_stream(index)))
        return
    if stream is not None and stream.device.index != index:
        raise ValueError("stream is on cuda:%d, the tensors on cuda:%d" % (stream.device.index, index))
    with torch.cuda.device(index):
        if stream is None:
            _check(call(_raw_stream(index)))
        else:
            with torch.cuda.stream(stream):
                _check(call(stream.cuda_stream))


def _raw_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


# torch's own quick form of the same, where this build of it has one
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)


def _int32(x):
    """x in the range of the argument; what is beyond it is as good as its end (a window past every slot, or refused)."""
    return max(-2 ** 31, min(int(x), 2 ** 31 - 1))


# torch's caching allocator without a tensor around the block (4 us less of a call's 20 on the host)
_raw_alloc = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_alloc",
                     lambda n, s: torch.cuda.caching_allocator_alloc(n, stream=s))
_raw_free = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_delete", torch.cuda.caching_allocator_delete)


def _scratch(a, workspace, index, n, s, call):
    """call() with the caller's workspace in `a`, or with n bytes that torch's allocator holds for stream s. Given back
    after the launch, as a tensor would be, they go to later work of that stream only (in a capture: of that graph)."""
    if workspace is not None:
        if workspace.get_device() != index or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on cuda:%d" % index)
        a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
        return call()
    p = _raw_alloc(n, s)
    try:
        a.workspace, a.workspace_bytes = p, n
        return call()
    finally:
        _raw_free(p)


def mtp_kv8_append(k_new, v_new, starts, k_cache, v_cache, k_scale, v_scale, block_table, ctx_lens, *, stream=None):
    """Quantise a ragged batch of new K/V into the 8-bit paged cache.

    k_new, v_new [T, Hkv, d] (float32 or bfloat16, d 64 or 128); starts [B+1] int32: request b appends tokens
    starts[b] .. starts[b+1]-1 at slots ctx_lens[b] and up; k_cache, v_cache [blocks, 64, Hkv, d] float8_e4m3fn;
    k_scale, v_scale [blocks, Hkv] float32 (both updated); block_table [B, max_blocks] int32, ctx_lens [B] int32.
    """
    T, Hkv, d = k_new.shape
    B, max_blocks = block_table.shape
    dt, nb = k_new.dtype, k_cache.shape[0]
    index = _cuda_index(k_new, "k_new")
    new, cache, scale, i32, f8 = (T, Hkv, d), (nb, BLOCK_SIZE, Hkv, d), (nb, Hkv), torch.int32, torch.float8_e4m3fn
    _check_all(index, ((k_new, "k_new", dt, new), (v_new, "v_new", dt, new), (starts, "starts", i32, (B + 1,)),
                       (k_cache, "k_cache", f8, cache), (v_cache, "v_cache", f8, cache),
                       (k_scale, "k_scale", torch.float32, scale), (v_scale, "v_scale", torch.float32, scale),
                       (block_table, "block_table", i32, (B, max_blocks)), (ctx_lens, "ctx_lens", i32, (B,))))
    a = Kv8AppendArgs(k_new.data_ptr(), v_new.data_ptr(), starts.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                      k_scale.data_ptr(), v_scale.data_ptr(), block_table.data_ptr(), ctx_lens.data_ptr(), T, B, Hkv,
                      d, BLOCK_SIZE, max_blocks, nb, _dtype_code(k_new))
    _on(index, stream, lambda s: lib().mtp_kv8_append(ctypes.byref(a), s))


def _window_attention(size, attend, q, k_new, v_new, k_cache, v_cache, k_scale, v_scale, block_table, ctx_lens, out,
                      window, sinks, sm_scale, workspace, stream):
    B, R, Hq, d = q.shape
    nb, _, Hkv, _ = k_cache.shape
    max_blocks = block_table.shape[-1]
    dt, i32 = q.dtype, torch.int32
    index = _cuda_index(q, "q")
    new, cache = (B, R, Hkv, d), (nb, BLOCK_SIZE, Hkv, d)
    ct = dt
    if k_scale is not None:
        ct, scale = torch.float8_e4m3fn, (nb, Hkv)
        _check_all(index, ((k_scale, "k_scale", torch.float32, scale), (v_scale, "v_scale", torch.float32, scale)))
    _check_all(index, ((q, "q", dt, (B, R, Hq, d)), (k_new, "k_new", dt, new), (v_new, "v_new", dt, new),
                       (k_cache, "k_cache", ct, cache), (v_cache, "v_cache", ct, cache),
                       (block_table, "block_table", i32, (B, max_blocks)), (ctx_lens, "ctx_lens", i32, (B,)),
                       (out, "out", dt, (B, R, Hq, d))))
    a = WindowAttnArgs(q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                       None if k_scale is None else k_scale.data_ptr(), None if v_scale is None else v_scale.data_ptr(),
                       block_table.data_ptr(), ctx_lens.data_ptr(), out.data_ptr(), B, R - 1, Hq, Hkv, d, BLOCK_SIZE,
                       max_blocks, nb, _int32(window), _int32(sinks),
                       d ** -0.5 if sm_scale is None else float(sm_scale), _dtype_code(q))
    ref = ctypes.byref(a)

    def call(s):
        n = 0
        if workspace is None:
            n = size(ref)
            if n == 0:
                _check(MTP_INVALID_ARG)
        return _scratch(a, workspace, index, n, s, lambda: attend(ref, s))

    _on(index, stream, call)


def mtp_verify_attention_kv8(q, k_new, v_new, k_cache, v_cache, k_scale, v_scale, block_table, ctx_lens, out, *,
                             window=0, sinks=0, sm_scale=None, workspace=None, stream=None):
    """Quantise the verify tokens' K/V into the 8-bit paged cache and run verify attention over it into `out`.

    q, out [B, R, Hq, d], k_new, v_new [B, R, Hkv, d] (float32 or bfloat16, d 64 or 128); k_cache, v_cache
    [blocks, 64, Hkv, d] float8_e4m3fn, k_scale, v_scale [blocks, Hkv] float32 (as mtp_kv8_append keeps them);
    block_table [B, max_blocks] int32, ctx_lens [B] int32. window > 0: a row sees the last `window` positions and the
    first `sinks` tokens; window = 0: all. Chains of drafts only.
    """
    L = lib()
    _window_attention(L.mtp_attention_kv8_workspace_size, L.mtp_verify_attention_kv8, q, k_new, v_new, k_cache, v_cache,
                      k_scale, v_scale, block_table, ctx_lens, out, window, sinks, sm_scale, workspace, stream)


def mtp_verify_attention_window(q, k_new, v_new, k_cache, v_cache, block_table, ctx_lens, out, *, window, sinks=0,
                                sm_scale=None, workspace=None, stream=None):
    """mtp_verify_attention for chains in which a row sees the last `window` >= 1 positions, its own among them, and
    the first `sinks` tokens (GQA/MHA caches [blocks, 64, Hkv, d] of q's type, d 64 or 128). Blocks that no row sees
    are not read; their table entries may be -1."""
    L = lib()
    _window_attention(L.mtp_attention_window_workspace_size, L.mtp_verify_attention_window, q, k_new, v_new, k_cache,
                      v_cache, None, None, block_table, ctx_lens, out, window, sinks, sm_scale, workspace, stream)


def kv_window_release(block_table, seq_lens, free_list, free_count, *, window, sinks=0, workspace=None, stream=None):
    """Return the blocks that no row at a position >= seq_lens sees behind `window` and `sinks` to the free list."""
    B, max_blocks = block_table.shape
    index, i32 = _cuda_index(block_table, "block_table"), torch.int32
    n_free = free_list.numel()
    _check_all(index, ((block_table, "block_table", i32, (B, max_blocks)), (seq_lens, "seq_lens", i32, (B,)),
                       (free_list, "free_list", i32, (n_free,)), (free_count, "free_count", i32, (1,))))
    L = lib()
    a = WindowReleaseArgs(block_table.data_ptr(), seq_lens.data_ptr(), free_list.data_ptr(), free_count.data_ptr(), B,
                          BLOCK_SIZE, max_blocks, n_free, _int32(window), _int32(sinks))

    n = L.mtp_window_release_workspace_size(B) if workspace is None else 0
    _on(index, stream, lambda s: _scratch(a, workspace, index, n, s, lambda: L.kv_window_release(ctypes.byref(a), s)))


_SHAPE, _DTYPE, _DATA = operator.attrgetter("shape"), operator.attrgetter("dtype"), torch.Tensor.data_ptr
_DEVICE, _DENSE = torch.Tensor.get_device, torch.Tensor.is_contiguous


def _pointers(index, names, tensors, dtypes, shapes):
    """The tensors' addresses, if all are on that device, of those types and shapes, and contiguous. (In a few passes that
    run in C: such a call's checks are a third of its time on the host.)"""
    if tuple(map(_SHAPE, tensors)) != shapes or tuple(map(_DTYPE, tensors)) != dtypes or not all(map(_DENSE, tensors)) or \
            tuple(map(_DEVICE, tensors)) != (index,) * len(tensors):
        _check_all(index, zip(tensors, names, dtypes, shapes))
    return map(_DATA, tensors)


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _run(index, stream, workspace, a, size, call):
    """call(a, stream handle) on device `index`, with the caller's workspace or size(a) bytes that torch holds for the
    stream (as _on and _scratch, without the steps that the usual call does not need)."""
    ref = ctypes.byref(a)

    def bytes_needed():
        n = size(ref)
        if n == 0:
            _check(MTP_INVALID_ARG)
        return n

    if workspace is not None or stream is not None or _current_device() != index:
        _on(index, stream, lambda s: _scratch(a, workspace, index, bytes_needed() if workspace is None else 0, s, lambda: call(ref, s)))
        return
    s, n = _raw_stream(index), bytes_needed()
    a.workspace_bytes = n
    a.workspace = p = _raw_alloc(n, s)
    try:
        rc = call(ref, s)
    finally:
        _raw_free(p)
    if rc != MTP_OK:
        _check(rc)


_ASSIGN_NAMES = ("block_table", "seq_lens", "starts", "free_list", "free_count", "slot_map", "taken")
_ASSIGN_TYPES = (torch.int32, torch.int32, torch.int32, torch.int32, torch.int32, torch.int64, torch.int32)


def kv_block_assign(block_table, seq_lens, starts, free_list, free_count, slot_map, taken, *, workspace=None, stream=None):
    """Take blocks for the tokens about to be appended from the free list, and map those tokens to cache slots.

    Request b holds seq_lens[b] tokens and appends tokens starts[b] .. starts[b+1]-1 of a ragged batch (starts [B+1]
    int32). Table entries < 0 that they need take blocks from the end of free_list[:free_count] (block_table [B,
    max_blocks], free_count [1] int32, updated). slot_map [T] int64: each token's slot, block * 64 + offset. taken [B]
    int32: blocks taken, or -1 for a request that the list has too few blocks for (its slots are -1, its table row as it
    was, and later requests do not overtake it).
    """
    B, max_blocks = block_table.shape
    n_free, T, index = free_list.numel(), slot_map.numel(), _cuda_index(block_table, "block_table")
    ptrs = _pointers(index, _ASSIGN_NAMES, (block_table, seq_lens, starts, free_list, free_count, slot_map, taken), _ASSIGN_TYPES,
                     ((B, max_blocks), (B,), (B + 1,), (n_free,), (1,), (T,), (B,)))
    L = lib()
    a = BlockAssignArgs(*ptrs, B, T, BLOCK_SIZE, max_blocks, n_free)
    _run(index, stream, workspace, a, lambda _: max(256, L.mtp_block_assign_workspace_size(B, T)), L.kv_block_assign)


def _token_rows(t, name, index, dtype, shape):
    """Elements from a token to the next of a [T, Hkv, d] tensor whose tokens may lie apart."""
    if t.get_device() != index or t.dtype is not dtype or t.shape != shape:
        _refuse(t, name, index, dtype, shape)
    apart, head, one = t.stride()
    T, Hkv, d = shape
    if (one != 1 and d > 1) or (head != d and Hkv > 1):
        raise ValueError("%s: a token's values must be contiguous" % name)
    return apart if T > 1 else Hkv * d


def mtp_kv_append(k_new, v_new, slot_map, k_cache, v_cache, *, stream=None):
    """Copy the K/V of new tokens to the slots of the paged cache that slot_map [T] int64 gives (< 0: skipped).

    k_new, v_new [T, Hkv, d] (float32 or bfloat16; views with tokens apart will do, a token's values contiguous), caches
    [blocks, 64, Hkv, d] of the same type. Absorbed MLA: k_new [T, 576] or [T, 1, 576], v_new = v_cache = None.
    """
    if v_new is None and k_new.dim() == 2:
        k_new = k_new.unsqueeze(1)
    T, Hkv, d = shape = k_new.shape
    nb, dt, index = k_cache.shape[0], k_new.dtype, _cuda_index(k_new, "k_new")
    if T > 2 ** 31 - 1:              # (the struct's field would take it modulo 2^32, and rows would be left out unsaid)
        raise ValueError("k_new: more than 2^31 - 1 tokens")
    k_stride = _token_rows(k_new, "k_new", index, dt, shape)
    if v_new is not None and v_cache is not None:
        d_v = v_new.shape[-1]
        v_stride = _token_rows(v_new, "v_new", index, dt, (T, Hkv, d_v))
        slots, k_at, v_at = _pointers(index, ("slot_map", "k_cache", "v_cache"), (slot_map, k_cache, v_cache), (torch.int64, dt, dt),
                                      ((T,), (nb, BLOCK_SIZE, Hkv, d), (nb, BLOCK_SIZE, Hkv, d_v)))
        v = v_new.data_ptr()
    elif v_new is None and v_cache is None:
        v = v_at = None
        d_v = v_stride = 0
        slots, k_at = _pointers(index, ("slot_map", "k_cache"), (slot_map, k_cache), (torch.int64, dt), ((T,), (nb, BLOCK_SIZE, Hkv, d)))
    else:
        raise ValueError("v_new and v_cache go together")
    a = KvAppendArgs(k_new.data_ptr(), v, slots, k_at, v_at, k_stride, v_stride, T, Hkv, d, d_v, BLOCK_SIZE, nb, v is None,
                     _dtype_code(k_new))
    if stream is None and _current_device() == index:
        _check(lib().mtp_kv_append(ctypes.byref(a), _raw_stream(index)))
    else:
        _on(index, stream, lambda s: lib().mtp_kv_append(ctypes.byref(a), s))


_PREFIX_NAMES = ("q", "k_new", "v_new", "k_cache", "v_cache", "block_table", "ctx_lens", "group_starts", "prefix_blocks", "out")


def mtp_verify_attention_prefix(q, k_new, v_new, k_cache, v_cache, block_table, ctx_lens, group_starts, prefix_blocks, out,
                                *, sm_scale=None, parents=None, workspace=None, stream=None):
    """mtp_verify_attention (GQA/MHA) of groups of requests whose tables begin with the same blocks, which are read once.

    q, out [B, R, Hq, d], k_new, v_new [B, R, Hkv, d], caches [blocks, 64, Hkv, d] (float32 or bfloat16, d 64 or 128),
    block_table [B, max_blocks] int32, ctx_lens [B] int32 (prefix included); group_starts [G+1] int32: group g is requests
    group_starts[g] .. group_starts[g+1]-1; prefix_blocks [G] int32: full blocks that they share, those of the row of the
    group's first request. parents [B, R] int32 (tree drafts) or None (chains).
    """
    B, R, Hq, d = rows = q.shape
    nb, _, Hkv, _ = k_cache.shape
    max_blocks, G = block_table.shape[-1], prefix_blocks.shape[0]
    dt, i32, index = q.dtype, torch.int32, _cuda_index(q, "q")
    new, cache = (B, R, Hkv, d), (nb, BLOCK_SIZE, Hkv, d)
    ptrs = _pointers(index, _PREFIX_NAMES,
                     (q, k_new, v_new, k_cache, v_cache, block_table, ctx_lens, group_starts, prefix_blocks, out),
                     (dt, dt, dt, dt, dt, i32, i32, i32, i32, dt),
                     (rows, new, new, cache, cache, (B, max_blocks), (B,), (G + 1,), (G,), rows))
    if parents is not None:
        parents, = _pointers(index, ("parents",), (parents,), (i32,), ((B, R),))
    L = lib()
    a = PrefixAttnArgs(*ptrs, B, R - 1, G, Hq, Hkv, d, BLOCK_SIZE, max_blocks, nb, d ** -0.5 if sm_scale is None else float(sm_scale),
                       _dtype_code(q), parents)
    _run(index, stream, workspace, a, L.mtp_attention_prefix_workspace_size, L.mtp_verify_attention_prefix)


def sync_status(stream=None):
    """Synchronise the stream and raise MtpError if a device-side range check tripped."""
    _check(lib().mtp_sync_status(_stream_handle(stream)))


def rng_debug(seed, b, j, tag, v0, n, device="cuda", stream=None):
    """Philox stream check: (word0 uint32 as int64, race exponential, accept uniform) for v = v0 .. v0+n-1."""
    w = torch.empty(n, dtype=torch.int32, device=device)
    e = torch.empty(n, dtype=torch.float32, device=device)
    u = torch.empty(n, dtype=torch.float32, device=device)
    _check(lib().mtp_rng_debug(int(seed), b, j, tag, v0, n, _ptr(w), _ptr(e), _ptr(u), _stream_handle(stream)))
    return w.cpu().numpy().view("uint32"), e.cpu().numpy(), u.cpu().numpy()


def wait_selftest(timeout_ns, stream=None):
    """Run the kernels' bounded mbarrier wait on a barrier nothing arrives on
    (it must give up after timeout_ns and flag a timeout)."""
    _check(lib().mtp_wait_selftest(int(timeout_ns), _stream_handle(stream)))


def hbm_read_probe(buf, sink, ctas_per_sm=2, bulk=False, stream=None):
    """Stream the bytes of device tensor `buf` once (read-bandwidth probe), by
    16-byte loads or (bulk=True) bulk copies into shared memory; `sink` is a
    1-element int32 device tensor that receives an XOR of the data."""
    _check(lib().mtp_hbm_read_probe(_ptr(buf), buf.numel() * buf.element_size(), _ptr(sink), int(ctas_per_sm),
                                    int(bool(bulk)), _stream_handle(stream)))
