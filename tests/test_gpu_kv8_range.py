"""The ends of what windowed and 8-bit verify attention take: scales far apart and at their limits, rows of Q with
outliers, sinks whose value is nothing, values that are not finite behind a vanishing weight, more rows than a CTA's,
ragged batches however their pages are cut into shares, shared prefixes, a workspace used again."""
import ctypes
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import kv8_ref
import mtp_speculative_decoding_verify_gb300 as mv
from mtp_speculative_decoding_verify_gb300 import _binding
from test_gpu_kv8_window import DEV, Case, bound, dev, host, TYPES

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_error_left():
    mv.sync_status()
    yield
    mv.sync_status()


def check_rows(c, g, requests=None, heads=None, hidden=None, q_eps=None, tokens=None):
    """Outputs of some requests, query heads and verify tokens, after c.append(). hidden: {(request, KV head): block of the table that
    takes no part}. As in `bound`, with two things more. Its last term is of p 2^(V's scale), which is what the 8-bit
    kernel splits, so V's scales weight the neighbours here. And q_eps(q, k) is what Q's own representation may add to
    a score; every p moves by that, and numerator and denominator with it."""
    got = g["out"].double().cpu().numpy()
    R, Hq, Hkv = c.R, c.q.shape[2], c.k.shape[2]
    for b in range(len(c.ctx)) if requests is None else requests:
        t = np.arange(c.ctx[b] + R)
        t = t[kv8_ref.visible(t, c.ctx[b], c.window, c.sinks) | (t > c.ctx[b])]
        ks, vs = c.rows(0, b)(t), c.rows(1, b)(t)
        scale = c.scale[1][c.table[b, t // 64]].astype(np.float64) if c.kv8 else np.ones((len(t), Hkv))
        for j in range(R) if tokens is None else tokens:
            for h in range(Hq) if heads is None else heads:
                kv = h // (Hq // Hkv)
                see = kv8_ref.visible(t, c.ctx[b] + j, c.window, c.sinks)
                if hidden and (b, kv) in hidden:
                    see &= t // 64 != hidden[b, kv]
                k, v, s, q = ks[see, kv], vs[see, kv], scale[see, kv], c.q[b, j, h].astype(np.float64)
                x = k @ q * c.d ** -0.5
                w = np.exp(x - x.max())
                w /= w.sum()
                ref, absolute = w @ v, w @ np.abs(v)
                near = (np.lib.stride_tricks.sliding_window_view(np.pad(w * s, 767), 1535).max(axis=1) / s) @ np.abs(v)
                lim = bound(c.t, c.kv8, c.d, c.ctx[b] + R, ref, absolute, (np.abs(k) @ np.abs(q)).max() * c.d ** -0.5, near)
                if q_eps is not None:
                    lim = lim + 2 * q_eps(q, k) * c.d ** -0.5 * absolute
                far = np.abs(got[b, j, h] - ref) - lim
                assert far.max() <= 0, (b, j, h, far.max(), np.abs(ref).max())


@pytest.mark.parametrize("ctx", [[1000, 70], [9000], [500, 600, 64] * 20], ids=["two", "long", "many"])
@pytest.mark.parametrize("kind,t", [("huge", "bf16"), ("tiny", "bf16"), ("tiny", "f32"), ("mixed", "bf16"), ("mixed", "f32")])
def test_scales_of_v(kind, t, ctx):
    """huge: V up to 2^126, of which no sum of two stays finite; tiny: the least scale; mixed: 2^-30 to 2^30 by block."""
    c = Case(True, t, len(ctx), 3, 4, 1, 64, ctx, 0, 0, seed=len(ctx))
    rng = np.random.default_rng(3)
    if kind == "huge":
        c.scale[1] = 2.0 ** 118
    elif kind == "tiny":
        c.scale[1] = 2.0 ** -100
        c.v *= np.float32(2.0 ** -96)
    else:
        c.scale[1] = 2.0 ** rng.integers(-30, 31, c.scale[1].shape)
    g = c.to_gpu()
    c.call(g)
    mv.sync_status()
    c.append()
    check_rows(c, g, range(min(3, len(ctx))))


@pytest.mark.parametrize("d,Hq", [(128, 2), (64, 12)])
def test_outliers_in_q(d, Hq):
    """Rows with a few values hundreds of times the others, next to requests without. Q is held as two e4m3 terms, and
    in a request with such a row as three. What is left out of a score: without the third at most 2^-19 sum|q| max|k|
    (more brings the third in); with it, of values below 2^-10 of the row's largest, half a step of e5m2 of a rest of at
    most 2^-18 of that largest value: 2^-21 max|q| sum|k|."""
    c = Case(True, "bf16", 4, 4, Hq, 1, d, [300, 900, 64, 5], 0, 0, seed=6)
    c.q[::2, :, :, 5] *= 400.0
    c.q[0, 1, 0, :40] *= 3000.0
    c.q = host(torch.from_numpy(c.q).to(torch.bfloat16))
    g = c.to_gpu()
    c.call(g)
    mv.sync_status()
    c.append()
    check_rows(c, g, q_eps=lambda q, k: 2.0 ** -19 * np.abs(q).sum() * np.abs(k).max() + 2.0 ** -21 * np.abs(q).max() * np.abs(k).sum(1).max())


def to_first_token(c, b, slot, amp):
    """q of request b near amp u for one u of each KV head, and the key at `slot` along u."""
    rng = np.random.default_rng(8)
    Hkv = c.k.shape[2]
    u = np.sign(rng.standard_normal((Hkv, c.d)))
    group = c.q.shape[2] // Hkv
    c.q[b] = host(torch.from_numpy(amp * np.repeat(u, group, axis=0)[None] + 0.3 * c.q[b]).to(TYPES[c.t]))
    blk = c.table[b, slot // 64]
    if c.kv8:
        c.scale[0][blk] = 2.0 ** -8
        c.byte[0][blk, slot % 64] = kv8_ref.to_e4m3(448.0 * u)
    else:
        c.cache[0][blk, slot % 64] = 1.75 * u


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("R,Hq,Hkv", [(2, 19, 19), (6, 152, 19)])
def test_first_token_takes_the_weight_and_has_no_value(t, R, Hq, Hkv):
    """The first token's score is some 20 octaves above the others' and V is zero in the first 13 blocks: what remains
    must be as exact as among scores of one size."""
    c = Case(True, t, 8, R, Hq, Hkv, 64, [1500] * 8, 0, 0, seed=2, stale=False)
    for b in range(8):
        to_first_token(c, b, 0, 1.0)
        c.byte[1][c.table[b, :13]] = 0
    g = c.to_gpu()
    c.call(g)
    mv.sync_status()
    c.append()
    check_rows(c, g, (0, 3, 7), (0, Hq // 2, Hq - 1))


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("kv8", [True, False], ids=["kv8", "window"])
@pytest.mark.parametrize("first,nan", [(0, 200), (200, 10), (650, 20)])
def test_a_nan_reaches_its_rows_whatever_its_weight(kv8, t, first, nan):
    """Formula and formats agree on 0 x NaN: a key whose weight underflows still hands its NaN on."""
    c = Case(kv8, t, 2, 2, 4, 2, 64, [700, 700], 0 if kv8 else 5000, 0, seed=5)
    for b in range(2):
        to_first_token(c, b, first, 30.0)
    if kv8:
        c.byte[1][c.table[0, nan // 64], nan % 64, 1, 9] = 127
    else:
        c.cache[1][c.table[0, nan // 64], nan % 64, 1, 9] = np.nan
    g = c.to_gpu()
    c.call(g)
    mv.sync_status()
    want = np.zeros((2, 2, 4, 64), bool)
    want[0, :, 2:, 9] = True
    assert np.array_equal(np.isnan(host(g["out"])), want)


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("which", [0, 1], ids=["k", "v"])
@pytest.mark.parametrize("bad", [0.0, -1.0, np.inf, np.nan, 2.0 ** 121, 2.0 ** -101])
def test_a_scale_out_of_range_is_reported_and_its_block_takes_no_part(t, which, bad):
    c = Case(True, t, 3, 4, 8, 2, 64, [500, 77, 300], 0, 0, seed=7)
    good = c.scale[which][c.table[0, 3], 1]
    c.scale[which][c.table[0, 3], 1] = bad
    g = c.to_gpu()
    c.call(g)
    with pytest.raises(mv.MtpError, match="scale"):
        mv.sync_status()
    c.scale[which][c.table[0, 3], 1] = good
    c.append()
    check_rows(c, g, hidden={(0, 1): 3})


@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 3)])
@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("kv8", [True, False], ids=["kv8", "window"])
@pytest.mark.parametrize("shape", [(2, 16, 32, 32, 64, [70, 300]), (2, 16, 12, 1, 64, [0, 400]), (1, 15, 16, 2, 128, [500]),
                                   (3, 9, 8, 1, 128, [64, 63, 900])], ids=lambda s: "R%d_%d/%dx%d" % s[1:5])
def test_heads_and_rows(kv8, t, shape, window, sinks):
    """A KV head for each head; 192, 120 and 72 rows a KV head, where CTAs take 64 (8-bit) or 112 (window) of them."""
    c = Case(kv8, t, *shape, window if kv8 or window else 10 ** 6, sinks, seed=1)
    g = c.to_gpu()
    c.call(g)
    mv.sync_status()
    c.check(g)


@pytest.mark.parametrize("seed", range(8))
@pytest.mark.parametrize("kv8", [True, False], ids=["kv8", "window"])
def test_ragged_batches_however_they_are_cut(kv8, seed):
    rng = np.random.default_rng(100 + seed)
    Hkv = int(rng.choice([1, 2, 4]))
    B = int(rng.choice([1, 2, 7, 18, 40, 90]))
    top = int(rng.choice([60, 700, 1500]))
    ctx = [int(x) for x in (rng.integers(0, top, B) if seed % 2 else top - rng.integers(0, min(top, 200), B))]
    window = int(rng.choice([0, 50, 400])) if kv8 else int(rng.choice([50, 400, 10 ** 5]))
    c = Case(kv8, "bf16", B, int(rng.choice([1, 3, 5])), 2 * Hkv, Hkv, 64, ctx, window, int(rng.choice([0, 70])) if window else 0, seed=seed)
    g = c.to_gpu()
    c.call(g)
    mv.sync_status()
    c.append()
    check_rows(c, g, heads={0, 2 * Hkv - 1}, tokens={0, c.R - 1})


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("kv8", [True, False], ids=["kv8", "window"])
def test_requests_may_share_full_blocks(kv8, t):
    c = Case(kv8, t, 4, 2, 4, 2, 64, [400, 300, 450, 400], 0 if kv8 else 350, 0, seed=4, drop=False)
    for b in range(1, 4):
        n = c.ctx[b] // 64 - 1
        c.table[b, :min(n, 5)] = c.table[0, :min(n, 5)]
    g = c.to_gpu()
    c.call(g)
    mv.sync_status()
    c.check(g)


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("kv8", [True, False], ids=["kv8", "window"])
def test_a_workspace_is_used_again_and_launches_are_counted(kv8, t):
    """Calls of other shapes leave anything in it; results are those of a workspace of the call's own."""
    L = _binding.lib()
    cs = [Case(kv8, t, len(x), R, Hq, 2, 64, x, 0 if kv8 else 900, 0, seed=i)
          for i, (x, R, Hq) in enumerate((([5000, 70, 0], 4, 4), ([64] * 50, 1, 8), ([1, 2000], 16, 12)))]
    gs, want = [c.to_gpu() for c in cs], []
    for c, g in zip(cs, gs):
        c.call(g)
        want.append(g["out"].clone())
        assert L.mtp_last_launch_count() in ((2,) if t == "bf16" else (2, 3))   # append, attention, fp32: a merge
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device=DEV)
    for _ in range(2):
        for c, g in zip(cs, gs):
            g["out"].zero_()
            c.call(g, workspace=ws)
        for g, w in zip(gs, want):
            assert torch.equal(g["out"], w)


def test_no_requests_and_no_tokens():
    L = _binding.lib()
    c = Case(True, "bf16", 1, 2, 4, 2, 64, [70], 0, 0)
    g = c.to_gpu()
    e = {n: g[n][:0] for n in ("q", "k_new", "v_new", "out")}
    mv.mtp_verify_attention_kv8(e["q"], e["k_new"], e["v_new"], g["kc"], g["vc"], g["ks"], g["vs"], g["table"][:0], g["ctx"][:0], e["out"])
    assert L.mtp_last_launch_count() == 0
    mv.mtp_kv8_append(e["k_new"].view(0, 2, 64), e["v_new"].view(0, 2, 64), dev(np.zeros(2, np.int32)), g["kc"], g["vc"], g["ks"], g["vs"],
                      g["table"], g["ctx"])
    assert L.mtp_last_launch_count() == 0
    mv.kv_window_release(g["table"][:0], g["ctx"][:0], g["ctx"][:0], dev(np.zeros(1, np.int32)), window=5)
    assert L.mtp_last_launch_count() == 0


def test_workspaces_and_windows_that_are_refused():
    """A workspace on the host, with gaps, off its alignment or too small; a window far below zero."""
    c = Case(True, "bf16", 1, 2, 4, 2, 64, [70], 0, 0)
    g = c.to_gpu()
    big = torch.zeros(8 << 20, dtype=torch.uint8, device=DEV)
    for ws in (torch.zeros(8 << 20, dtype=torch.uint8), big[::2]):
        with pytest.raises(ValueError, match="workspace"):
            c.call(g, workspace=ws)
        with pytest.raises(ValueError, match="workspace"):
            mv.kv_window_release(g["table"], g["ctx"], g["ctx"], g["ctx"], window=5, workspace=ws)
    for ws, word in ((big[16:], "aligned"), (big[:1024], "workspace")):
        with pytest.raises(mv.MtpError, match=word):
            c.call(g, workspace=ws)
    with pytest.raises(mv.MtpError, match="workspace"):
        mv.kv_window_release(g["table"], g["ctx"], g["ctx"], g["ctx"], window=5, workspace=big[:4])
    elsewhere = SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)
    with pytest.raises(ValueError, match="stream"):
        c.call(g, stream=elsewhere)
    c.window = -2 ** 40
    with pytest.raises(mv.MtpError, match="window"):
        c.call(g)
    with pytest.raises(mv.MtpError, match="window"):
        mv.kv_window_release(g["table"], g["ctx"], g["ctx"], g["ctx"], window=-2 ** 40)
    assert (g["out"] == 7.0).all()


@pytest.mark.parametrize("field,value", [("max_blocks", 2 ** 24 + 1), ("Hq", 2 ** 30), ("Hkv", 2 ** 17), ("B", 2 ** 27), ("d", 96), ("D", 16),
                                         ("block_size", 32), ("window", -1), ("sm_scale", float("inf"))])
def test_sizes_beyond_the_limits_are_refused(field, value):
    """By the C entry itself: nothing is launched, and a workspace size of 0 says so beforehand."""
    L = _binding.lib()
    a = _binding.WindowAttnArgs(*([16] * 10), 1, 3, 8, 2, 64, 64, 16, 4, 0, 0, 0.1, 1)
    assert L.mtp_attention_kv8_workspace_size(ctypes.byref(a)) > 0
    setattr(a, field, value)
    if field in ("Hq", "Hkv"):
        a.Hq, a.Hkv = (value, 2) if field == "Hq" else (value, value)
    assert L.mtp_attention_kv8_workspace_size(ctypes.byref(a)) == 0
    assert L.mtp_verify_attention_kv8(ctypes.byref(a), None) != 0


@pytest.mark.parametrize("t,d", [("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("kv8", [True, False], ids=["kv8", "window"])
def test_blocks_whose_offsets_pass_32_bits(kv8, t, d):
    """The same call with every block moved to the end of a cache of more than 2^32 elements."""
    c = Case(kv8, t, 2, 3, 16, 8, d, [300, 70], 0 if kv8 else 200, 0, seed=2, drop=False)
    g, far = c.to_gpu(), c.to_gpu()
    n = 2 ** 32 // (64 * 8 * d) + c.nb + 1
    names = ("kc", "vc") + (("ks", "vs") if kv8 else ())
    for name in names:
        far[name] = torch.empty((n,) + g[name].shape[1:], dtype=g[name].dtype, device=DEV)
        as_bytes = (lambda x: x.view(torch.uint8)) if name[1] == "c" and kv8 else (lambda x: x)
        as_bytes(far[name])[n - c.nb:] = as_bytes(g[name]).flip(0)
    far["table"] = torch.where(g["table"] < 0, g["table"], n - 1 - g["table"]).int()
    c.call(g)
    c.call(far)
    mv.sync_status()
    assert torch.equal(far["out"], g["out"])
    for name in names:
        x, y = far[name][n - c.nb:], g[name]
        if name[1] == "c":
            x, y = x.view(torch.uint8), y.view(torch.uint8)
        assert torch.equal(x.flip(0), y)
    c.check(g)
    if kv8:     # and the append of many tokens
        m = 130
        new = [torch.randn(m, 8, d, device=DEV).to(TYPES[t]) for _ in "kv"]
        starts, ctx = dev(np.array([0, m, m], np.int32)), dev(np.zeros(2, np.int32))
        for s in (g, far):
            mv.mtp_kv8_append(new[0], new[1], starts, s["kc"], s["vc"], s["ks"], s["vs"], s["table"], ctx)
        mv.sync_status()
        for name in names:
            x, y = far[name][n - c.nb:], g[name]
            if name[1] == "c":
                x, y = x.view(torch.uint8), y.view(torch.uint8)
            assert torch.equal(x.flip(0), y)
