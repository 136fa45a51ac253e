"""The 8-bit cache and window entries on the host: struct layouts, refused arguments, empty calls (no kernel is
launched), and the pins of the plain implementation that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import kv8_ref


@pytest.fixture(scope="module")
def mtplib():
    from mtp_speculative_decoding_verify_gb300 import build
    build.build()
    from mtp_speculative_decoding_verify_gb300 import _binding
    return _binding


def test_struct_layouts(mtplib):
    L = mtplib.lib()
    for which, st in ((5, mtplib.Kv8AppendArgs), (6, mtplib.WindowAttnArgs), (7, mtplib.WindowReleaseArgs)):
        assert L.mtp_abi_struct_size(which) == ctypes.sizeof(st)


def _append(m, **kw):
    a = m.Kv8AppendArgs()
    for n in ("k_new", "v_new", "starts", "k_cache", "v_cache", "k_scale", "v_scale", "block_table", "ctx_lens"):
        setattr(a, n, 16)
    a.T, a.B, a.Hkv, a.d, a.block_size, a.max_blocks, a.num_blocks, a.dtype = 10, 2, 4, 128, 64, 8, 16, 1
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(B=-1), 1), (dict(block_size=128), 1), (dict(max_blocks=0), 1), (dict(num_blocks=0), 1),
    (dict(max_blocks=(1 << 24) + 1), 1), (dict(Hkv=0), 1), (dict(dtype=2), 1), (dict(d=96), 2), (dict(k_new=None), 1),
    (dict(starts=None), 1), (dict(v_scale=None), 1), (dict(k_new=8), 1), (dict(v_cache=4), 1),
    (dict(B=1 << 28, Hkv=4), 2),
])
def test_append_refuses(mtplib, kw, code):
    L = mtplib.lib()
    assert L.mtp_kv8_append(ctypes.byref(_append(mtplib, **kw)), None) == code
    assert L.mtp_last_error()


def _attn(m, kv8, **kw):
    a = m.WindowAttnArgs()
    for n in ("q", "k_new", "v_new", "k_cache", "v_cache", "block_table", "ctx_lens", "out"):
        setattr(a, n, 16)
    if kv8:
        a.k_scale = a.v_scale = 16
    a.B, a.D, a.Hq, a.Hkv, a.d, a.block_size, a.max_blocks, a.num_blocks = 2, 3, 8, 2, 128, 64, 8, 16
    a.window, a.sinks, a.sm_scale, a.dtype = 100, 4, 0.088, 1
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kv8", [True, False])
@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), 1), (dict(D=16), 1), (dict(D=-1), 1), (dict(block_size=32), 1), (dict(max_blocks=0), 1),
    (dict(num_blocks=-1), 1), (dict(Hkv=3), 1), (dict(Hq=0), 1), (dict(dtype=7), 1), (dict(sm_scale=0.0), 1),
    (dict(sm_scale=float("nan")), 1), (dict(sm_scale=float("inf")), 1), (dict(window=-1), 1), (dict(sinks=-1), 1),
    (dict(window=0, sinks=4), 1), (dict(d=96), 2), (dict(q=None), 1), (dict(out=None), 1), (dict(ctx_lens=None), 1),
    (dict(q=8), 1), (dict(k_cache=24), 1), (dict(B=1 << 25), 2),
])
def test_attention_refuses(mtplib, kv8, kw, code):
    L = mtplib.lib()
    a = _attn(mtplib, kv8, **kw)
    name = "kv8" if kv8 else "window"
    assert getattr(L, "mtp_verify_attention_" + name)(ctypes.byref(a), None) == code
    assert L.mtp_last_error()
    assert getattr(L, "mtp_attention_%s_workspace_size" % name)(ctypes.byref(a)) == 0


def test_attention_scales_belong_to_the_8_bit_cache(mtplib):
    L = mtplib.lib()
    assert L.mtp_verify_attention_kv8(ctypes.byref(_attn(mtplib, False)), None) == 1
    assert L.mtp_verify_attention_window(ctypes.byref(_attn(mtplib, True)), None) == 1
    assert L.mtp_verify_attention_window(ctypes.byref(_attn(mtplib, False, window=0, sinks=0)), None) == 1


def _release(m, **kw):
    a = m.WindowReleaseArgs(16, 16, 16, 16, 2, 64, 8, 100, 64, 4, 256, 256)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw", [
    dict(B=-1), dict(block_size=32), dict(max_blocks=0), dict(free_capacity=-1), dict(window=0), dict(sinks=-1),
    dict(block_table=None), dict(free_count=None), dict(workspace=None), dict(workspace=128), dict(workspace_bytes=8),
])
def test_release_refuses(mtplib, kw):
    L = mtplib.lib()
    assert L.kv_window_release(ctypes.byref(_release(mtplib, **kw)), None) == 1
    assert L.mtp_last_error()
    assert L.mtp_window_release_workspace_size(-1) == 0 and L.mtp_window_release_workspace_size(300) >= 301 * 4


def test_empty_calls_do_nothing(mtplib):
    L = mtplib.lib()
    assert L.mtp_kv8_append(ctypes.byref(_append(mtplib, B=0)), None) == 0
    assert L.mtp_kv8_append(ctypes.byref(_append(mtplib, T=0, k_new=None)), None) == 0
    assert L.mtp_verify_attention_kv8(ctypes.byref(_attn(mtplib, True, B=0, q=None)), None) == 0
    assert L.mtp_verify_attention_window(ctypes.byref(_attn(mtplib, False, B=0)), None) == 0
    assert L.kv_window_release(ctypes.byref(_release(mtplib, B=0, workspace=None)), None) == 0


def test_binding_refuses_host_tensors(mtplib):
    z = torch.zeros
    with pytest.raises(ValueError):
        mtplib.mtp_kv8_append(z(3, 2, 64), z(3, 2, 64), z(2, dtype=torch.int32), z(1), z(1), z(1), z(1),
                              z(1, 4, dtype=torch.int32), z(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        mtplib.kv_window_release(z(1, 4, dtype=torch.int32), z(1, dtype=torch.int32), z(4, dtype=torch.int32),
                                 z(1, dtype=torch.int32), window=64)


def test_plain_e4m3_is_the_type():
    """Every byte's value and the rounding of a dense range agree with torch's own e4m3 type."""
    bits = torch.arange(256, dtype=torch.uint8)
    want = bits.view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(kv8_ref.VALUES.astype(np.float32), want, equal_nan=True)
    x = np.concatenate([np.linspace(-448, 448, 20001), np.linspace(-0.05, 0.05, 20001)]).astype(np.float32)
    got = kv8_ref.VALUES[kv8_ref.to_e4m3(x)]
    assert np.array_equal(got, torch.from_numpy(x).to(torch.float8_e4m3fn).float().numpy())
    assert np.isnan(kv8_ref.VALUES[kv8_ref.to_e4m3([np.nan, np.inf, -np.inf])]).all()


def test_plain_scale_is_the_smallest_that_holds():
    a = np.array([0.0, 1e-35, 1.0, 448.0, 448.0001, 3e38])
    s, _ = kv8_ref.block_scale(np.ones(6, np.float32), True, a)
    assert s[0] == s[1] == np.float32(2.0 ** -100)
    assert (448.0 * s.astype(np.float64) >= np.float32(a)).all()
    assert (448.0 * s[2:].astype(np.float64) / 2 < a[2:]).all()
    s, k = kv8_ref.block_scale(np.full(2, 0.3, np.float32), False, np.array([100.0, 1000.0]))
    assert s[0] == np.float32(0.3) and k[0] == 0 and k[1] == 3 and s[1] == np.float32(0.3) * 8


def test_plain_release_keeps_what_a_row_sees():
    table = np.arange(40, dtype=np.int32).reshape(4, 10)
    free = np.full(40, -1, np.int32)
    lens, w, sinks = [640, 65, 300, 0], 100, 70
    n = kv8_ref.release(table, lens, free, 0, w, sinks)
    for b, L in enumerate(lens):
        for i in range(10):
            t = np.arange(i * 64, i * 64 + 64)
            seen = any(kv8_ref.visible(t, p, w, sinks).any() for p in range(L, 641))   # now or by a later row
            assert (table[b, i] == -1) == (not seen), (b, i)
    assert n == (table == -1).sum() and (free[n:] == -1).all()
