"""The 8-bit cache append, verify attention over it and behind a window, and the window release, against the plain
float64 implementation (kv8_ref): bytes, scales, tables and free lists to the bit, attention within a bound made of
the roundings that the kernels make."""
import numpy as np
import pytest
import torch

import kv8_ref
import mtp_speculative_decoding_verify_gb300 as mv

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}     # half a step of the output type, relative


@pytest.fixture(autouse=True)
def _no_error_left():
    mv.sync_status()
    yield
    mv.sync_status()


def host(t):
    return t.detach().cpu().float().numpy()


def raw(t):
    return t.detach().cpu().view(torch.uint8).numpy()


def same_bytes(a, b):
    nan = (a & 127) == 127
    return np.array_equal(nan, (b & 127) == 127) and np.array_equal(a[~nan], b[~nan])


def tables(rng, ctx, n, spare=3, extra=0):
    need = [(c + k + 63) // 64 for c, k in zip(ctx, n)]
    nb = sum(need) + spare
    perm = rng.permutation(nb).astype(np.int32)
    t = np.full((len(ctx), max(need + [1]) + extra), -1, np.int32)
    at = 0
    for b, m in enumerate(need):
        t[b, :m] = perm[at:at + m]
        at += m
    return t, nb


def cache8(rng, nb, Hkv, d, pow2=True):
    """Random bytes, no NaN among them, and scales around 2^-6."""
    byte = rng.integers(0, 127, (2, nb, 64, Hkv, d)).astype(np.uint8) | (rng.integers(0, 2, (2, nb, 64, Hkv, d)) << 7).astype(np.uint8)
    scale = 2.0 ** rng.integers(-8, -4, (2, nb, Hkv)) if pow2 else rng.uniform(0.003, 0.05, (2, nb, Hkv))
    return byte, scale.astype(np.float32)


def dev8(byte):
    return torch.from_numpy(byte.copy()).to(DEV).view(torch.float8_e4m3fn)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


# ---------------------------------------------------------------------------------------------------------- append
APPENDS = {
    "verify sized": ([0, 1, 63, 64, 200], [4, 4, 4, 4, 4]),
    "none, one and many": ([0, 5, 64, 127, 130, 3], [0, 1, 64, 65, 129, 0]),
    "long": ([0, 77], [700, 1]),
    "one token": ([63], [1]),
    "starts a block": ([64, 128], [64, 1]),
    "many requests": (list(range(0, 400, 5)), [(7 * i) % 23 for i in range(80)]),
}


@pytest.mark.parametrize("name", list(APPENDS))
@pytest.mark.parametrize("t,d,Hkv,pow2", [("bf16", 128, 8, True), ("f32", 64, 3, False), ("bf16", 64, 1, False), ("f32", 128, 2, True)])
def test_append_to_the_bit(name, t, d, Hkv, pow2):
    ctx, n = APPENDS[name]
    rng = np.random.default_rng(5)
    table, nb = tables(rng, ctx, n)
    byte, scale = cache8(rng, nb, Hkv, d, pow2)
    starts = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    x = rng.standard_normal((2, starts[-1], Hkv, d)) * 2.0 ** rng.integers(-6, 7, (2, starts[-1], Hkv, 1))
    xt = [torch.from_numpy(a).to(TYPES[t]).to(DEV) for a in x]
    k, v, ks, vs = dev8(byte[0]), dev8(byte[1]), dev(scale[0]), dev(scale[1])
    mv.mtp_kv8_append(xt[0], xt[1], dev(starts), k, v, ks, vs, dev(table), dev(np.array(ctx, np.int32)))
    mv.sync_status()
    for i, (c, s) in enumerate(((k, ks), (v, vs))):
        kv8_ref.append(byte[i], scale[i], host(xt[i]), starts, ctx, table)
        assert np.array_equal(host(s), scale[i])
        assert same_bytes(raw(c), byte[i])


def test_append_special_values():
    """Zeros, what is not finite, values that underflow, the largest floats, and a scale that grows far."""
    rng = np.random.default_rng(1)
    ctx, n = [0, 10, 20, 64, 30], [3, 2, 2, 2, 2]
    table, nb = tables(rng, ctx, n)
    byte, scale = cache8(rng, nb, 2, 64)
    starts = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    x = np.zeros((11, 2, 64), np.float32)
    x[3] = rng.standard_normal((2, 64))
    x[3, 0, :4] = [np.inf, -np.inf, np.nan, 1e-30]
    x[4, 1, 5] = np.nan
    x[5:7] = 3e38
    x[7, :, 1] = 1e-36
    x[9:11] = 1e9
    k, v, ks, vs = dev8(byte[0]), dev8(byte[1]), dev(scale[0]), dev(scale[1])
    mv.mtp_kv8_append(dev(x), dev(-x), dev(starts), k, v, ks, vs, dev(table), dev(np.array(ctx, np.int32)))
    mv.sync_status()
    for i, (c, s, y) in enumerate(((k, ks, x), (v, vs, -x))):
        kv8_ref.append(byte[i], scale[i], y, starts, ctx, table)
        assert np.array_equal(host(s), scale[i])
        assert same_bytes(raw(c), byte[i])
        assert np.isnan(kv8_ref.VALUES[byte[i][table[1, 0], 10, 0, :3]]).all()


@pytest.mark.parametrize("fault,word", [("starts", "length"), ("ctx", "length"), ("long", "length"), ("block", "block-id"),
                                        ("block high", "block-id"), ("scale", "scale")])
def test_append_skips_and_reports_a_bad_request(fault, word):
    rng = np.random.default_rng(2)
    ctx, n = [5, 70, 8], [30, 3, 6]
    table, nb = tables(rng, ctx, n)
    byte, scale = cache8(rng, nb, 2, 128)
    starts = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    x = rng.standard_normal((2, starts[-1], 2, 128)).astype(np.float32)
    bad = dict(starts=starts.copy(), ctx=np.array(ctx, np.int32), table=table.copy())
    if fault == "starts":
        bad["starts"][3] = 1000
    elif fault == "ctx":
        bad["ctx"][2] = -1
    elif fault == "long":
        bad["ctx"][2] = 2 ** 31 - 3
    elif fault == "block":
        bad["table"][2, 0] = -1
    elif fault == "block high":
        bad["table"][2, 0] = nb
    else:
        scale[:, table[2, 0]] = [0.0, np.inf]
    k, v, ks, vs = dev8(byte[0]), dev8(byte[1]), dev(scale[0]), dev(scale[1])
    mv.mtp_kv8_append(dev(x[0]), dev(x[1]), dev(bad["starts"]), k, v, ks, vs, dev(bad["table"]), dev(bad["ctx"]))
    with pytest.raises(mv.MtpError, match=word):
        mv.sync_status()
    for i, (c, s) in enumerate(((k, ks), (v, vs))):
        kv8_ref.append(byte[i], scale[i], x[i], starts[:3], ctx[:2], table)   # the other two requests
        assert np.array_equal(host(s), scale[i]) and same_bytes(raw(c), byte[i])


# ------------------------------------------------------------------------------------------------------- attention
def bound(t, kv8, d, n, ref, absolute, score, near):
    """What the kernels' roundings can move an output by. The output's own: EPS |ref|. A score: d products and sums,
    the scale and the exponent's argument in fp32, at most (d + 8) 2^-23 score, which moves every p, and so numerator
    and denominator, by that factor. Sums over n keys in fp32: n 2^-23 each, numerator and denominator. (2^-23: a
    tensor-core sum may cut off instead of rounding.) And a probability's own, of its share of sum p|v|:
      fp32 rows 0; bf16 cache 2^-8 (bf16);
      8-bit cache 2^-8 + 2^-11: p = hi + lo / 16 with e4m3 hi and lo, each off by at most 2^-4 of what it rounds (2^-4
      2^-4), after a rounding to f16 (2^-11). Below e4m3's normal numbers lo is off by half a step of 2^-9, over 16:
      2^-14, where the largest p of a row's keys in a tile of 128 is 2^-4 or more at least in each fifth tile: 2^-10 of
      the largest one within 767 visible slots of the key."""
    p_eps = 0.0 if t == "f32" else 2.0 ** -8 + 2.0 ** -11 if kv8 else 2.0 ** -8
    floor = 2.0 ** -10 * near if kv8 and t == "bf16" else 0.0
    # |ref| <= absolute, so every relative change of p counts at most twice
    return EPS[t] * np.abs(ref) * 1.01 + (p_eps + 2 * (d + 8) * 2.0 ** -23 * np.maximum(score, 1.0) + 2 * n * 2.0 ** -23) * absolute + floor


class Case:
    def __init__(self, kv8, t, B, R, Hq, Hkv, d, ctx, window, sinks, seed=0, drop=True, pow2=True, stale=True, amp=1.0):
        rng = np.random.default_rng(seed)
        self.kv8, self.t, self.window, self.sinks, self.ctx = kv8, t, window, sinks, list(ctx)
        self.table, nb = tables(rng, ctx, [R] * B, extra=1)
        self.d, self.R, self.nb = d, R, nb
        bf = TYPES[t]
        if kv8:
            self.byte, self.scale = cache8(rng, nb, Hkv, d, pow2)
            small = rng.standard_normal((2, nb, 64, Hkv, d)) * 60
            self.byte = kv8_ref.to_e4m3(small)
        else:
            self.cache = rng.standard_normal((2, nb, 64, Hkv, d))
        if stale:   # slots behind the last verify token, and whole unused blocks, hold NaN
            live = np.zeros((nb, 64), bool)
            for b, c in enumerate(ctx):
                for s in range(c):
                    live[self.table[b, s // 64], s % 64] = True
            if kv8:
                self.byte[:, ~live] = 127
            else:
                self.cache[:, ~live] = np.nan
        if not kv8:
            self.cache = host(torch.from_numpy(self.cache).to(bf))
        if drop and window:   # blocks that no row sees are gone
            for b, c in enumerate(ctx):
                for i in range(self.table.shape[1]):
                    if i * 64 >= sinks and i * 64 + 63 <= c - window:
                        self.table[b, i] = -1
        self.q, self.k, self.v = (host(torch.from_numpy(rng.standard_normal(s) * amp).to(bf))
                                  for s in ((B, R, Hq, d), (B, R, Hkv, d), (B, R, Hkv, d)))

    def to_gpu(self):
        bf = TYPES[self.t]
        g = dict(q=dev(self.q).to(bf), k_new=dev(self.k).to(bf), v_new=dev(self.v).to(bf), table=dev(self.table),
                 ctx=dev(np.array(self.ctx, np.int32)))
        g["out"] = torch.full(g["q"].shape, 7.0, dtype=bf, device=DEV)
        if self.kv8:
            g.update(kc=dev8(self.byte[0]), vc=dev8(self.byte[1]), ks=dev(self.scale[0]), vs=dev(self.scale[1]))
        else:
            g.update(kc=dev(self.cache[0]).to(bf), vc=dev(self.cache[1]).to(bf))
        return g

    def call(self, g, **kw):
        kw = dict(window=self.window, sinks=self.sinks, **kw)
        if self.kv8:
            mv.mtp_verify_attention_kv8(g["q"], g["k_new"], g["v_new"], g["kc"], g["vc"], g["ks"], g["vs"], g["table"], g["ctx"], g["out"], **kw)
        else:
            mv.mtp_verify_attention_window(g["q"], g["k_new"], g["v_new"], g["kc"], g["vc"], g["table"], g["ctx"], g["out"], **kw)

    def append(self, skip=()):
        B, R = self.q.shape[:2]
        for i, x in enumerate((self.k, self.v)):
            for b in range(B):
                if b in skip:
                    continue
                if self.kv8:
                    kv8_ref.append(self.byte[i], self.scale[i], x[b], [0, R], [self.ctx[b]], self.table[b:b + 1])
                else:
                    for j in range(R):
                        p = self.ctx[b] + j
                        self.cache[i][self.table[b, p // 64], p % 64] = x[b, j]

    def rows(self, i, b):
        def get(t):
            blk = self.table[b, t // 64]
            if self.kv8:
                return kv8_ref.VALUES[self.byte[i][blk, t % 64]] * self.scale[i][blk].astype(np.float64)[:, :, None]
            return self.cache[i][blk, t % 64].astype(np.float64)
        return get

    def check(self, g, skip=()):
        """Caches to the bit; the outputs of the requests not in `skip`."""
        self.append(skip)
        for i, (c, s) in enumerate((("kc", "ks"), ("vc", "vs"))):
            if self.kv8:
                assert np.array_equal(host(g[s]), self.scale[i]) and same_bytes(raw(g[c]), self.byte[i])
            else:
                assert np.array_equal(host(g[c]), self.cache[i], equal_nan=True)
        got = g["out"].double().cpu().numpy()
        for b in range(len(self.ctx)):
            if b in skip:
                assert (got[b] == 7.0).all()
                continue
            ref, absolute, score, near = kv8_ref.attention(self.q[b], self.rows(0, b), self.rows(1, b), self.ctx[b],
                                                     self.d ** -0.5, self.window, self.sinks)
            lim = bound(self.t, self.kv8, self.d, self.ctx[b] + self.R, ref, absolute, score, near)
            assert np.isfinite(got[b]).all()
            far = np.abs(got[b] - ref) - lim
            assert far.max() <= 0, (b, far.max(), np.abs(got[b] - ref).max())


SHAPES = [  # B, R, Hq, Hkv, d, contexts
    (1, 1, 8, 8, 128, [0]),
    (1, 2, 32, 8, 128, [997]),
    (5, 4, 8, 2, 128, [0, 1, 63, 64, 300]),
    (3, 16, 4, 1, 64, [48, 49, 1000]),
    (2, 6, 16, 2, 128, [511, 130]),             # 48 rows a KV head
    (4, 3, 6, 2, 64, [5, 60, 62, 700]),
    (2, 16, 8, 1, 128, [100, 1600]),            # 128 rows: more than a CTA's
    (3, 7, 7, 1, 64, [64, 65, 127]),
    (9, 1, 3, 3, 64, [0, 1, 2, 63, 64, 65, 127, 128, 129]),
]
WINDOWS = [(0, 0), (1, 0), (17, 3), (64, 64), (333, 100), (100000, 5)]


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "B%d_R%d_%d/%dx%d" % s[:5])
@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("kv8", [True, False], ids=["kv8", "window"])
def test_attention(kv8, t, shape, window, sinks):
    if not kv8 and window == 0:
        window = 2 ** 31 - 1        # the widest there is
    c = Case(kv8, t, *shape, window, sinks, seed=len(shape[5]) + window % 97)
    g = c.to_gpu()
    c.call(g)
    mv.sync_status()
    c.check(g)


@pytest.mark.parametrize("kv8", [True, False], ids=["kv8", "window"])
def test_attention_long_context_is_split_and_joined(kv8):
    """One request over many CTAs, next to short ones; a scale that is no power of two; peaked rows."""
    c = Case(kv8, "bf16", 3, 4, 8, 2, 128, [9000, 3, 4097], 0 if kv8 else 8000, 0 if kv8 else 9, seed=4, pow2=False, amp=3.0)
    g = c.to_gpu()
    c.call(g)
    mv.sync_status()
    c.check(g)


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("kv8", [True, False], ids=["kv8", "window"])
def test_attention_many_requests(kv8, t):
    ctx = [(37 * i) % 301 for i in range(150)]
    c = Case(kv8, t, 150, 4, 4, 2, 64, ctx, 90, 2, seed=9)
    g = c.to_gpu()
    c.call(g)
    mv.sync_status()
    c.check(g)


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("kv8", [True, False], ids=["kv8", "window"])
@pytest.mark.parametrize("what", ["k", "v"])
def test_not_finite_reaches_the_rows_that_see_it_only(kv8, t, what):
    """Verify token 2 holds a NaN and slot 70 of the context another, which rows 0 and 1 still have in their window."""
    c = Case(kv8, t, 1, 4, 4, 2, 64, [100], 32, 0, seed=3)
    getattr(c, what)[0, 2, 1, 5] = np.nan
    i = "kv".index(what)
    if kv8:
        c.byte[i, c.table[0, 1], 70 - 64, 0, 9] = 127
    else:
        c.cache[i][c.table[0, 1], 70 - 64, 0, 9] = np.nan
    g = c.to_gpu()
    c.call(g)
    mv.sync_status()
    got = g["out"].float().cpu().numpy()[0]     # [R, Hq, d]; heads 0, 1 read KV head 0, heads 2, 3 KV head 1
    want = np.zeros((4, 4, 64), bool)
    if what == "v":
        want[:2, :2, 9] = True
        want[2:, 2:, 5] = True
    else:
        want[:2, :2] = True
        want[2:, 2:] = True
    assert np.array_equal(np.isnan(got), want)


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("kv8", [True, False], ids=["kv8", "window"])
@pytest.mark.parametrize("bad", [-1, 10 ** 6, 2 ** 31 - 2])
def test_attention_skips_a_request_of_bad_length(kv8, t, bad):
    c = Case(kv8, t, 3, 4, 8, 2, 128, [200, 77, 300], 100, 4, seed=6)
    g = c.to_gpu()
    g["ctx"][1] = bad
    c.call(g)
    with pytest.raises(mv.MtpError, match="length"):
        mv.sync_status()
    got = g["out"]
    assert (got[1] == 7.0).all()
    c.check(g, skip=(1,))


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("kv8", [True, False], ids=["kv8", "window"])
@pytest.mark.parametrize("bad", [-1, 10 ** 6])
def test_attention_reports_a_bad_block_and_serves_the_rest(kv8, t, bad):
    c = Case(kv8, t, 3, 4, 8, 2, 64, [500, 77, 300], 0 if kv8 else 1000, 0, seed=7)
    g = c.to_gpu()
    g["table"][0, 3] = bad
    c.call(g)
    with pytest.raises(mv.MtpError, match="block-id"):
        mv.sync_status()
    assert torch.isfinite(g["out"][0]).all()
    # the other requests as ever; request 0 as if its block 3 held nothing
    c.append()
    for b in range(3):
        def without(i):
            get = c.rows(i, b)
            return lambda t_: get(t_[(t_ // 64 != 3) | (b != 0)])
        t_all = np.arange(c.ctx[b] + 4)
        keep = (t_all // 64 != 3) | (b != 0)
        q = c.q[b]
        for j in range(4):
            seen = keep & kv8_ref.visible(t_all, c.ctx[b] + j, c.window, 0)
            k, v = c.rows(0, b)(t_all[seen]), c.rows(1, b)(t_all[seen])
            for h in range(8):
                x = k[:, h // 4] @ q[j, h].astype(np.float64) * 64 ** -0.5
                w = np.exp(x - x.max())
                w /= w.sum()
                ref, absolute = w @ v[:, h // 4], w @ np.abs(v[:, h // 4])
                score = (np.abs(k[:, h // 4]) @ np.abs(q[j, h])).max() / 8
                lim = bound(t, kv8, 64, 600, ref, absolute, score, w.max() * np.abs(v[:, h // 4]).sum(0))
                assert (np.abs(g["out"][b, j, h].double().cpu().numpy() - ref) <= lim).all()


def test_every_block_bad_gives_zeros():
    c = Case(False, "bf16", 1, 2, 4, 2, 64, [100], 1000, 0, seed=7)
    g = c.to_gpu()
    g["table"].fill_(-1)
    c.call(g)
    with pytest.raises(mv.MtpError, match="block-id"):
        mv.sync_status()
    assert (g["out"] == 0).all()


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("kv8", [True, False], ids=["kv8", "window"])
def test_same_bits_every_time_and_in_graphs(kv8, t):
    """Repeated calls, two graphs replayed at once on two streams, a call on a stream of its own: one result."""
    mk = lambda s: Case(kv8, t, 6, 4, 16, 2, 128, [3000, 70, 0, 900, 64, 1], 0 if kv8 else 2000, 0, seed=s)  # noqa: E731
    cs = [mk(11), mk(12)]
    gs = [c.to_gpu() for c in cs]
    want = []
    for c, g in zip(cs, gs):
        c.call(g)
        want.append(g["out"].clone())
    graphs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for c, g in zip(cs, gs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            c.call(g)
        graphs.append(graph)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for g in gs:
            g["out"].zero_()
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for g, w in zip(gs, want):
            assert torch.equal(g["out"], w)
    for c, g, s in zip(cs, gs, streams):     # eager calls at once, each on a stream given by name
        g["out"].zero_()
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for c, g, s in zip(cs, gs, streams):
            c.call(g, stream=s)
    torch.cuda.synchronize()
    for g, w in zip(gs, want):
        assert torch.equal(g["out"], w)
    mv.sync_status()
    cs[0].check(gs[0])


def test_arguments_are_refused():
    c = Case(True, "bf16", 2, 4, 8, 2, 128, [10, 20], 0, 0)
    g = c.to_gpu()
    ok = dict(q=g["q"], k_new=g["k_new"], v_new=g["v_new"], k_cache=g["kc"], v_cache=g["vc"], k_scale=g["ks"], v_scale=g["vs"],
              block_table=g["table"], ctx_lens=g["ctx"], out=g["out"])
    for kw in (dict(q=g["q"].float()), dict(q=g["q"].half()), dict(k_cache=g["kc"].view(torch.uint8)), dict(k_new=g["k_new"][:, :2]),
               dict(out=g["out"].transpose(1, 2)), dict(ctx_lens=g["ctx"].long()), dict(block_table=g["table"][:1]),
               dict(k_scale=g["ks"][:, :1]), dict(v_scale=g["vs"].double()), dict(ctx_lens=g["ctx"].cpu())):
        with pytest.raises(ValueError):
            mv.mtp_verify_attention_kv8(**{**ok, **kw})
    for kw in (dict(window=-1), dict(sinks=1), dict(sm_scale=0.0), dict(workspace=torch.empty(8, dtype=torch.uint8, device=DEV)[:0])):
        with pytest.raises(mv.MtpError):
            mv.mtp_verify_attention_kv8(**ok, **kw)
    off = torch.empty(g["q"].numel() + 1, dtype=torch.bfloat16, device=DEV)[1:].view(g["q"].shape)
    with pytest.raises(mv.MtpError, match="aligned"):
        mv.mtp_verify_attention_kv8(**{**ok, "q": off})
    with pytest.raises(mv.MtpError, match="window"):
        mv.mtp_verify_attention_window(g["q"], g["k_new"], g["v_new"], g["k_new"].new_zeros(c.nb, 64, 2, 128),
                                       g["k_new"].new_zeros(c.nb, 64, 2, 128), g["table"], g["ctx"], g["out"], window=0)
    assert (g["out"] == 7.0).all()


# --------------------------------------------------------------------------------------------------------- release
@pytest.mark.parametrize("B,top,window,sinks,capacity", [
    (1, 10, 1, 0, 100), (5, 700, 64, 0, 1000), (5, 700, 100, 70, 1000), (300, 2000, 333, 4, 100000), (3, 100000, 4096, 100, 10 ** 6),
    (40, 3000, 10, 0, 300), (7, 500, 10 ** 9, 0, 10), (7, 500, 1, 10 ** 9, 10), (1030, 200, 17, 65, 10 ** 6)])
def test_release(B, top, window, sinks, capacity):
    rng = np.random.default_rng(B)
    lens = rng.integers(0, top + 1, B).astype(np.int32)
    table, nb = tables(rng, list(lens), [4] * B, extra=2)
    table[rng.random(table.shape) < 0.2] = -1          # some went before
    free = np.full(capacity, -1, np.int32)
    t, f, n = dev(table), dev(free), torch.full((1,), 3, dtype=torch.int32, device=DEV)
    mv.kv_window_release(t, dev(lens), f, n, window=window, sinks=sinks)
    count = kv8_ref.release(table, lens, free, 3, window, sinks)
    try:
        mv.sync_status()
        fits = True
    except mv.MtpError as e:
        fits = False
        assert "free-list" in str(e)
    assert int(n) == count and np.array_equal(t.cpu().numpy(), table) and np.array_equal(f.cpu().numpy(), free)
    gone = sum(int((table[b, -(-sinks // 64):max(0, (lens[b] - window + 1) // 64)] >= 0).sum()) for b in range(B)
               if (lens[b] - window + 1) // 64 > -(-sinks // 64))
    assert fits == (gone == 0)                          # what is left over did not fit


def test_release_skips_bad_lengths_and_refuses_bad_arguments():
    rng = np.random.default_rng(0)
    lens = np.array([500, -5, 10 ** 6, 400], np.int32)
    table, _ = tables(rng, [500, 500, 500, 400], [4] * 4)
    free = np.full(100, -1, np.int32)
    t, f, n = dev(table), dev(free), torch.zeros(1, dtype=torch.int32, device=DEV)
    mv.kv_window_release(t, dev(lens), f, n, window=64)
    with pytest.raises(mv.MtpError, match="length"):
        mv.sync_status()
    count = kv8_ref.release(table, lens, free, 0, 64, 0)
    assert int(n) == count and np.array_equal(t.cpu().numpy(), table) and np.array_equal(f.cpu().numpy(), free)
    with pytest.raises(mv.MtpError):
        mv.kv_window_release(t, dev(lens), f, n, window=0)
    with pytest.raises(ValueError):
        mv.kv_window_release(t, dev(lens[:2]), f, n, window=64)
    with pytest.raises(ValueError):
        mv.kv_window_release(t, dev(lens), f.long(), n, window=64)


# ------------------------------------------------------------------------------------------------- used together
def test_a_serving_loop_on_the_8_bit_cache():
    """Prefill chunks appended, then steps of verify attention, rollback and window release, on one captured graph;
    tables, lengths, bytes and scales to the bit and outputs within their bound at every step."""
    rng = np.random.default_rng(21)
    B, R, Hq, Hkv, d, window, sinks, steps = 3, 4, 8, 2, 64, 100, 5, 9
    first = [190, 64, 0]
    table, nb = tables(rng, first, [steps * R] * B, extra=1)
    c = Case(True, "bf16", B, R, Hq, Hkv, d, first, window, sinks, seed=2, drop=False)
    c.table, c.nb = table, nb
    c.byte, c.scale = cache8(rng, nb, Hkv, d)
    c.byte[:] = 127
    g = c.to_gpu()
    ctx = dev(np.zeros(B, np.int32))
    lens = np.zeros(B, int)
    for part in (0.5, 1.0):                           # two chunks each
        n = [int(x * part) - int(y) for x, y in zip(first, lens)]
        starts = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        x = [torch.from_numpy(rng.standard_normal((starts[-1], Hkv, d))).to(torch.bfloat16) for _ in "kv"]
        mv.mtp_kv8_append(x[0].to(DEV), x[1].to(DEV), dev(starts), g["kc"], g["vc"], g["ks"], g["vs"], g["table"], ctx)
        for i in range(2):
            kv8_ref.append(c.byte[i], c.scale[i], host(x[i]), starts, lens, table)
        lens += n
        ctx.copy_(dev(lens.astype(np.int32)))
    g["ctx"].copy_(ctx)
    free = np.full(60, -1, np.int32)
    f, count = dev(free), torch.zeros(1, dtype=torch.int32, device=DEV)
    accepted = torch.zeros(B, dtype=torch.int32, device=DEV)

    def step():
        c.call(g)
        mv.kv_rollback(g["table"], g["ctx"], accepted, f, count, D=R - 1)
        mv.kv_window_release(g["table"], g["ctx"], f, count, window=window, sinks=sinks)

    torch.cuda.synchronize()
    graph, at = None, 0
    for i in range(steps):
        c.q, c.k, c.v = (host(torch.from_numpy(rng.standard_normal(s.shape)).to(torch.bfloat16)) for s in (c.q, c.k, c.v))
        for n, x in (("q", c.q), ("k_new", c.k), ("v_new", c.v)):
            g[n].copy_(dev(x))
        n = rng.integers(0, R, B)
        accepted.copy_(dev(n.astype(np.int32)))
        # tables: the block a rollback took is given back before the next step needs it
        blocks = table.copy()
        g["table"].copy_(dev(table))
        c.ctx = [int(x) for x in lens]
        if i == 0:
            step()
        else:
            if graph is None:
                keep = [x.clone() for x in (g["table"], g["ctx"], f, count)]
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    step()
                for x, y in zip((g["table"], g["ctx"], f, count), keep):
                    x.copy_(y)
            graph.replay()
        torch.cuda.synchronize()
        mv.sync_status()
        c.check(g)
        lens = lens + n + 1
        assert np.array_equal(g["ctx"].cpu().numpy(), lens)
        for b in range(B):                            # rollback, as its own tests pin it: by request, then block
            for y in range((lens[b] + 63) // 64, (c.ctx[b] + R - 1) // 64 + 1):
                free[at], table[b, y], at = table[b, y], -1, at + 1
        at = kv8_ref.release(table, lens, free, at, window, sinks)
        assert int(count) == at and np.array_equal(f.cpu().numpy(), free)
        assert np.array_equal(g["table"].cpu().numpy(), table)
        back = (table < 0) & (blocks >= 0) & (np.arange(table.shape[1]) >= (lens[:, None] // 64))
        table[back] = blocks[back]                    # (this loop's allocator hands the same block out again)
