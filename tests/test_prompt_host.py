"""The calls for requests that share a prompt, on the host: struct layouts, refused arguments, empty calls (no kernel is
launched), and pins of the plain implementations that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import prompt_ref


@pytest.fixture(scope="module")
def mtplib():
    from mtp_speculative_decoding_verify_gb300 import build
    build.build()
    from mtp_speculative_decoding_verify_gb300 import _binding
    return _binding


def test_struct_layouts(mtplib):
    L = mtplib.lib()
    for which, st in ((8, mtplib.BlockAssignArgs), (9, mtplib.KvAppendArgs), (10, mtplib.PrefixAttnArgs)):
        assert L.mtp_abi_struct_size(which) == ctypes.sizeof(st)


def _assign(m, **kw):
    a = m.BlockAssignArgs()
    for n in ("block_table", "seq_lens", "starts", "free_list", "free_count", "slot_map", "taken"):
        setattr(a, n, 16)
    a.B, a.T, a.block_size, a.max_blocks, a.free_capacity, a.workspace, a.workspace_bytes = 3, 100, 64, 8, 50, 256, 1 << 20
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), 1), (dict(T=-1), 1), (dict(block_size=32), 1), (dict(max_blocks=0), 1), (dict(max_blocks=(1 << 24) + 1), 1),
    (dict(free_capacity=-1), 1), (dict(B=(1 << 20) + 1), 2), (dict(block_table=None), 1), (dict(seq_lens=None), 1),
    (dict(starts=None), 1), (dict(free_list=None), 1), (dict(free_count=None), 1), (dict(slot_map=None), 1),
    (dict(taken=None), 1), (dict(workspace=None), 1), (dict(workspace=128), 1), (dict(workspace_bytes=8), 1),
])
def test_assign_refuses(mtplib, kw, code):
    L = mtplib.lib()
    assert L.kv_block_assign(ctypes.byref(_assign(mtplib, **kw)), None) == code
    assert L.mtp_last_error()


def _append(m, **kw):
    a = m.KvAppendArgs()
    for n in ("k_new", "v_new", "slot_map", "k_cache", "v_cache"):
        setattr(a, n, 16)
    a.k_stride = a.v_stride = 4 * 128
    a.T, a.Hkv, a.d_qk, a.d_v, a.block_size, a.num_blocks, a.is_mla, a.dtype = 10, 4, 128, 128, 64, 16, 0, 1
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(block_size=128), 1), (dict(num_blocks=0), 1), (dict(dtype=2), 1), (dict(Hkv=0), 1),
    (dict(Hkv=1 << 17), 1), (dict(d_qk=0), 1), (dict(d_v=8192), 1), (dict(Hkv=1, d_qk=12), 2), (dict(Hkv=3, d_v=4), 2),
    (dict(k_new=None), 1), (dict(v_new=None), 1), (dict(v_cache=None), 1), (dict(slot_map=None), 1), (dict(is_mla=1), 1),
    (dict(is_mla=1, Hkv=1), 1), (dict(k_stride=511), 1), (dict(v_stride=256), 1), (dict(k_stride=-512), 1),
    (dict(k_stride=1 << 41), 1), (dict(k_new=8), 1), (dict(v_cache=24), 1), (dict(k_stride=516), 1),
])
def test_append_refuses(mtplib, kw, code):
    L = mtplib.lib()
    assert L.mtp_kv_append(ctypes.byref(_append(mtplib, **kw)), None) == code
    assert L.mtp_last_error()


def _attn(m, **kw):
    a = m.PrefixAttnArgs()
    for n in ("q", "k_new", "v_new", "k_cache", "v_cache", "block_table", "ctx_lens", "group_starts", "prefix_blocks", "out"):
        setattr(a, n, 16)
    a.B, a.D, a.G, a.Hq, a.Hkv, a.d, a.block_size, a.max_blocks, a.num_blocks = 4, 3, 2, 8, 2, 128, 64, 8, 16
    a.sm_scale, a.dtype = 0.088, 1
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), 1), (dict(G=-1), 1), (dict(D=16), 1), (dict(D=-1), 1), (dict(block_size=32), 1), (dict(max_blocks=0), 1),
    (dict(max_blocks=(1 << 24) + 1), 1), (dict(num_blocks=-1), 1), (dict(Hkv=3), 1), (dict(Hq=0), 1), (dict(dtype=7), 1),
    (dict(sm_scale=0.0), 1), (dict(sm_scale=float("nan")), 1), (dict(sm_scale=float("inf")), 1), (dict(d=96), 2),
    (dict(d=576), 2), (dict(q=None), 1), (dict(out=None), 1), (dict(ctx_lens=None), 1), (dict(group_starts=None), 1),
    (dict(prefix_blocks=None), 1), (dict(q=8), 1), (dict(v_cache=24), 1), (dict(B=1 << 25), 2), (dict(G=(1 << 20) + 1), 2),
    (dict(B=1 << 10, max_blocks=1 << 21), 2),
])
def test_attention_refuses(mtplib, kw, code):
    L = mtplib.lib()
    a = _attn(mtplib, **kw)
    assert L.mtp_verify_attention_prefix(ctypes.byref(a), None) == code
    assert L.mtp_last_error()
    assert L.mtp_attention_prefix_workspace_size(ctypes.byref(a)) == 0


def test_empty_calls_do_nothing(mtplib):
    L = mtplib.lib()
    assert L.mtp_verify_attention_prefix(ctypes.byref(_attn(mtplib, B=0, q=None)), None) == 0
    assert L.kv_block_assign(ctypes.byref(_assign(mtplib, B=0, workspace=None)), None) == 0
    assert L.mtp_kv_append(ctypes.byref(_append(mtplib, T=0, k_new=None)), None) == 0
    assert L.mtp_block_assign_workspace_size(-1, 4) == 0 and L.mtp_block_assign_workspace_size(4, -1) == 0
    assert L.mtp_block_assign_workspace_size(4, 10000) >= 4 * (1 + 8 + 4)


def test_binding_refuses_host_tensors(mtplib):
    z, i32 = torch.zeros, dict(dtype=torch.int32)
    with pytest.raises(ValueError):
        mtplib.kv_block_assign(z(1, 4, **i32), z(1, **i32), z(2, **i32), z(4, **i32), z(1, **i32),
                               z(3, dtype=torch.int64), z(1, **i32))
    with pytest.raises(ValueError):
        mtplib.mtp_kv_append(z(3, 2, 64), z(3, 2, 64), z(3, dtype=torch.int64), z(4, 64, 2, 64), z(4, 64, 2, 64))


def test_plain_assign_by_hand():
    table = np.array([[7, -1, -1], [8, 9, -1], [-1, -1, -1], [-1, -1, -1]], np.int32)
    slots = np.full(9, 99, np.int64)
    taken, left = prompt_ref.assign(table, [62, 100, 0, 0], [0, 4, 7, 9, 9], np.array([1, 2, 3], np.int32), 3, slots)
    assert taken.tolist() == [1, 0, 1, 0] and left == 1
    assert table.tolist() == [[7, 3, -1], [8, 9, -1], [2, -1, -1], [-1, -1, -1]]
    assert slots.tolist() == [7 * 64 + 62, 7 * 64 + 63, 3 * 64, 3 * 64 + 1, 9 * 64 + 36, 9 * 64 + 37, 9 * 64 + 38, 128, 129]


def test_plain_attention_of_a_tree_is_that_of_its_paths():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((4, 2, 8)), rng.standard_normal((9, 1, 8)), rng.standard_normal((9, 1, 8))
    out, _, _ = prompt_ref.attention(q, k, v, 5, 0.3, parents=[-1, 0, 0, 2])
    keep = [0, 1, 2, 3, 4, 5, 7, 8]                        # the path 0, 2, 3 as a chain
    chain, _, _ = prompt_ref.attention(q[[0, 2, 3]], k[keep], v[keep], 5, 0.3)
    assert np.allclose(out[[0, 2, 3]], chain, rtol=1e-12)
