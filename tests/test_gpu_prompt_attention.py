"""Verify attention of requests that share a prefix, against the plain float64 implementation (prompt_ref), within a bound
made of the roundings that the kernels make; and the calls around it together, as a server uses them."""
import numpy as np
import pytest
import torch

import mtp_speculative_decoding_verify_gb300 as mv
import prompt_ref

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


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def bound(t, d, n, ref, absolute, score):
    """What the kernels' roundings can move an output by. The output's own: EPS |ref|. A score: d products and sums, the
    scale and the exponent's argument in fp32, at most (d + 8) 2^-23 score, which moves every p, and so numerator and
    denominator, by that factor. Sums over n keys in fp32, 64 more for the joins of partial results: (n + 64) 2^-23 each.
    (2^-23: a tensor-core sum may cut off instead of rounding.) A bf16 row's probability is rounded to bf16: 2^-8 of its
    share of sum p|v|. |ref| <= absolute, so every relative change of p counts at most twice."""
    p_eps = 0.0 if t == "f32" else 2.0 ** -8
    return (EPS[t] * np.abs(ref) * 1.01 +
            (p_eps + 2 * (d + 8) * 2.0 ** -23 * np.maximum(score, 1.0) + 2 * (n + 64) * 2.0 ** -23) * absolute)


class Case:
    """groups: (blocks of the prefix, the own tokens of each request) in order; `before` and `after`: contexts of requests
    in no group. Unused slots and blocks hold NaN."""

    def __init__(self, t, R, Hq, Hkv, d, groups, before=(), after=(), tree=False, seed=0, amp=1.0, rows=True):
        rng = np.random.default_rng(seed)
        self.t, self.d, self.R = t, d, R
        self.blocks = [0] * len(before) + [p for p, own in groups for _ in own] + [0] * len(after)
        tails = list(before) + [x for _, own in groups for x in own] + list(after)
        self.ctx = [64 * p + x for p, x in zip(self.blocks, tails)]
        B = len(tails)
        self.starts = np.cumsum([len(before)] + [len(own) for _, own in groups]).astype(np.int32)
        self.prefix = np.array([p for p, _ in groups], np.int32)
        need = [-(-(c + R) // 64) for c in self.ctx]
        self.nb = sum(n - p for n, p in zip(need, self.blocks)) + int(self.prefix.sum()) + 3
        perm = list(rng.permutation(self.nb).astype(np.int32))
        self.table = np.full((B, max(need) + 1), -1, np.int32)
        live, b = np.zeros((self.nb, 64), bool), len(before)
        for p, own in groups:
            ids = [perm.pop() for _ in range(p)]
            live[ids] = True
            for i in range(len(own)):
                if rows or i == 0:
                    self.table[b + i, :p] = ids
            b += len(own)
        for b in range(B):
            for i in range(self.blocks[b], need[b]):
                self.table[b, i] = perm.pop()
            for s in range(64 * self.blocks[b], self.ctx[b]):
                live[self.table[b, s // 64], s % 64] = True
        bf = TYPES[t]
        cache = rng.standard_normal((2, self.nb, 64, Hkv, d))
        cache[:, ~live] = np.nan
        self.cache = host(torch.from_numpy(cache).to(bf))
        self.q, self.k, self.v = (host(torch.from_numpy(rng.standard_normal(s) * amp).to(bf))
                                  for s in ((B, R, Hq, d), (B, R, Hkv, d), (B, R, Hkv, d)))
        self.parents = None
        if tree:
            self.parents = np.array([[-1] + [int(rng.integers(0, k)) for k in range(1, R)] for _ in range(B)], np.int32)

    def to_gpu(self):
        bf = TYPES[self.t]
        g = dict(q=dev(self.q).to(bf), k_new=dev(self.k).to(bf), v_new=dev(self.v).to(bf), table=dev(self.table),
                 ctx=dev(np.array(self.ctx, np.int32)), k=dev(self.cache[0]).to(bf), v=dev(self.cache[1]).to(bf),
                 starts=dev(self.starts), prefix=dev(self.prefix), parents=None if self.parents is None else dev(self.parents))
        g["out"] = torch.full_like(g["q"], 7.0)
        return g

    def call(self, g, **kw):
        mv.mtp_verify_attention_prefix(g["q"], g["k_new"], g["v_new"], g["k"], g["v"], g["table"], g["ctx"], g["starts"],
                                       g["prefix"], g["out"], parents=g["parents"], **kw)

    def rows_of(self, b, i):
        """K (0) or V (1) of request b's slots, its verify tokens' last."""
        first = next((int(self.starts[g]) for g in range(len(self.prefix)) if self.starts[g] <= b < self.starts[g + 1]), b)
        t = np.arange(self.ctx[b])
        owner = np.where(t // 64 < self.blocks[b], first, b)
        return np.concatenate([self.cache[i][self.table[owner, t // 64], t % 64], (self.k, self.v)[i][b]])

    def reference(self, b, scale):
        par = None if self.parents is None else self.parents[b]
        return prompt_ref.attention(self.q[b], self.rows_of(b, 0), self.rows_of(b, 1), self.ctx[b], scale, par)

    def check(self, g, skip=(), scale=None):
        scale = self.d ** -0.5 if scale is None else scale
        got = host(g["out"]).astype(np.float64)
        for b in range(len(self.ctx)):
            if b in skip:
                assert (got[b] == 7.0).all()
                continue
            ref, absolute, score = self.reference(b, scale)
            room = bound(self.t, self.d, self.ctx[b] + self.R, ref, absolute, score)
            bad = ~(np.abs(got[b] - ref) <= room)
            bad &= ~((np.isnan(ref) & np.isnan(got[b])) | (np.isinf(ref) & (ref == got[b])))
            assert not bad.any(), (b, int(bad.sum()), float(np.nanmax(np.abs(got[b] - ref))), float(np.nanmin(room)))
        kc, vc = host(g["k"]), host(g["v"])      # the verify tokens' K/V, and nothing else
        want = self.cache.copy()
        for b in range(len(self.ctx)):
            for j in range(self.R if b not in skip else 0):
                s = self.ctx[b] + j
                want[0][self.table[b, s // 64], s % 64] = self.k[b, j]
                want[1][self.table[b, s // 64], s % 64] = self.v[b, j]
        assert np.array_equal(kc, want[0], equal_nan=True) and np.array_equal(vc, want[1], equal_nan=True)


GROUPS = {
    "one request": dict(groups=[(1, [0])]),
    "four samples": dict(groups=[(5, [0, 3, 64, 130])]),
    "no groups": dict(groups=[], before=[0, 5, 64, 200]),
    "of all kinds": dict(groups=[(3, [0, 70, 1, 64, 5]), (0, [10, 100]), (17, [9]), (2, []), (6, [3 * i for i in range(30)])],
                         before=[5, 130], after=[0, 64, 700]),
    "long and short": dict(groups=[(70, [1, 2, 3]), (1, [63, 64, 65, 66, 0, 1, 2])]),
    "own pages long": dict(groups=[(2, [3000, 10, 1500])]),
}
HEADS = [(32, 8, 128), (12, 4, 64), (7, 1, 128), (8, 8, 64), (16, 2, 64)]


@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("Hq,Hkv,d", HEADS)
@pytest.mark.parametrize("t,R,tree", [("bf16", 4, False), ("f32", 2, False), ("bf16", 1, False), ("bf16", 16, True), ("f32", 5, True)])
def test_attention(name, Hq, Hkv, d, t, R, tree):
    c = Case(t, R, Hq, Hkv, d, tree=tree, seed=R + d, **GROUPS[name])
    g = c.to_gpu()
    c.call(g)
    mv.sync_status()
    c.check(g)


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,d", [(160, 1, 64), (256, 2, 128), (300, 1, 64), (65, 1, 128)])
def test_many_heads_a_kv_head(t, Hq, Hkv, d):
    c = Case(t, 2, Hq, Hkv, d, groups=[(3, [0, 5, 70]), (4, [1])], after=[9])
    g = c.to_gpu()
    c.call(g)
    mv.sync_status()
    c.check(g)


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("P,n", [(33, 64), (128, 9), (2, 200), (300, 2)])
def test_many_rows_and_long_prefixes(t, P, n):
    c = Case(t, 4, 8, 2, 128 if t == "bf16" else 64, groups=[(P, [(13 * i) % 90 for i in range(n)])])
    g = c.to_gpu()
    c.call(g)
    mv.sync_status()
    c.check(g)


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("n_groups", [0, 3, 1300])
def test_many_requests_and_many_groups(t, n_groups):
    """More of both than the schedule keeps in shared memory."""
    rng = np.random.default_rng(n_groups)
    if n_groups == 1300:
        groups = [(int(rng.integers(0, 3)), [int(x) for x in rng.integers(0, 40, int(rng.integers(0, 3)))]) for _ in range(1300)]
    else:
        groups = [(2 + i, [int(x) for x in rng.integers(0, 150, 400)]) for i in range(n_groups)]
    c = Case(t, 1, 2, 1, 64, groups=groups, before=[5, 70], after=[int(x) for x in rng.integers(0, 150, 30 if n_groups else 1400)])
    g = c.to_gpu()
    c.call(g)
    mv.sync_status()
    c.check(g)


def test_the_same_as_verify_attention():
    """Over the same tables, up to the order of the sums; and the others' entries of the prefix are not looked at. (In
    slots behind the last token mtp_verify_attention wants finite values.)"""
    c = Case("bf16", 4, 32, 8, 128, groups=[(9, [0, 100, 7, 64] * 4)])
    c.cache = np.nan_to_num(c.cache)
    g = c.to_gpu()
    c.call(g)
    other = torch.empty_like(g["out"])
    mv.mtp_verify_attention(g["q"], g["k_new"], g["v_new"], g["k"], g["v"], g["table"], g["ctx"], other)
    most = float((g["out"].float() - other.float()).abs().max())
    assert most <= 2.0 ** -5   # two roundings of P and of outputs below 1 apart
    out = g["out"].clone()
    g["table"][1:, :9] = -1
    c.call(g)
    mv.sync_status()
    assert torch.equal(out, g["out"])


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_results_do_not_change(t):
    c = Case(t, 3, 16, 4, 64, groups=[(40, [10 * i for i in range(20)]), (3, [900, 3])], tree=True)
    g = c.to_gpu()
    c.call(g)
    first = g["out"].clone()
    for _ in range(5):
        g["out"].fill_(0.0)
        c.call(g)
        assert torch.equal(first, g["out"])
    mv.sync_status()


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1.0, 30.0, 1e-4])
def test_scales_of_scores(t, scale):
    c = Case(t, 2, 8, 2, 64, groups=[(6, [0, 30, 64, 100])], amp=2.0)
    g = c.to_gpu()
    c.call(g, sm_scale=scale)
    mv.sync_status()
    c.check(g, scale=scale)


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_infinities_and_nan(t):
    """Of K and V in the prefix, in own slots, and in verify keys off a row's path, act as in the formula."""
    c = Case(t, 4, 8, 2, 64, groups=[(5, [3, 64, 10]), (2, [0, 1])], tree=True, seed=4)
    first = c.table[0]
    c.cache[1][first[1], 7, 0, 3] = np.nan           # V of a shared slot: that dim of every row of the head
    c.cache[1][first[2], 9, 1, 5] = np.inf
    c.cache[0][first[4], 0, 1, :] = np.where(c.q[1, 0, 4] > 0, -np.inf, np.inf)   # scores of -inf for one row, others NaN or so
    c.v[3, 2, 0, 0] = np.nan                         # a verify key's: only rows below it
    c.k[4, 3, 1, 2] = np.nan
    g = c.to_gpu()
    c.call(g)
    mv.sync_status()
    c.check(g)


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_scores_of_minus_infinity_only(t):
    """A row all of whose scores are -inf is NaN, and one with a prefix of them is its own slots' result."""
    c = Case(t, 1, 2, 1, 64, groups=[(2, [0, 5])])
    c.q[:] = np.abs(c.q) + 1.0
    c.cache[0][c.table[0, :2]] = -np.inf
    c.k[0] = -np.inf
    g = c.to_gpu()
    c.call(g)
    mv.sync_status()
    c.check(g)
    assert np.isnan(host(g["out"])[0]).all() and np.isfinite(host(g["out"])[1]).all()


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("fault", ["negative", "beyond the table", "shorter than the prefix", "far too long"])
def test_a_bad_length_is_skipped_and_reported(t, fault):
    c = Case(t, 2, 8, 2, 64, groups=[(3, [0, 70, 9]), (2, [5])], after=[30])
    right = c.ctx[1]
    c.ctx[1] = {"negative": -1, "beyond the table": c.table.shape[1] * 64 - 1, "shorter than the prefix": 191,
                "far too long": 2 ** 31 - 1}[fault]
    g = c.to_gpu()
    c.call(g)
    with pytest.raises(mv.MtpError, match="length"):
        mv.sync_status()
    c.ctx[1] = right
    c.check(g, skip=(1,))


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("P", [-1, 1 << 20, 2 ** 31 - 1])
def test_a_bad_prefix_is_skipped_and_reported(t, P):
    c = Case(t, 2, 8, 2, 64, groups=[(3, [0, 70, 9]), (2, [5, 6])], after=[30])
    g = c.to_gpu()
    g["prefix"][1] = P
    c.call(g)
    with pytest.raises(mv.MtpError, match="length"):
        mv.sync_status()
    c.check(g, skip=(3, 4))


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("starts", [[0, 4, 3, 6], [-1, 3, 3, 6], [0, 3, 3, 7], [0, 2 ** 31 - 1, 3, 6]])
def test_with_bad_starts_requests_attend_by_themselves(t, starts):
    c = Case(t, 2, 8, 2, 64, groups=[(3, [0, 70, 9]), (2, []), (4, [6, 7, 70])])
    g = c.to_gpu()
    g["starts"].copy_(dev(np.array(starts, np.int32)))
    c.call(g)
    with pytest.raises(mv.MtpError, match="length"):
        mv.sync_status()
    c.check(g)


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [-1, 10 ** 6])
def test_a_bad_block_takes_no_part(t, bad):
    c = Case(t, 2, 8, 2, 64, groups=[(5, [0, 70, 9]), (1, [64]), (1, [0])])
    g = c.to_gpu()
    drop = [(0, 2), (0, 3), (3, 0)]                   # pages 2 and 3 of the first group, all of the second's prefix
    for b, i in drop:
        g["table"][b, i] = bad
    g["table"][1, 5] = bad                            # and a request's own
    c.call(g)
    with pytest.raises(mv.MtpError, match="block-id"):
        mv.sync_status()
    gone = {0: [2, 3], 1: [2, 3, 5], 2: [2, 3], 3: [0], 4: []}
    got = host(g["out"]).astype(np.float64)
    for b in range(5):
        at = np.arange(c.ctx[b] + 2)
        keep = ~np.isin(at // 64, gone[b]) | (at >= c.ctx[b])
        ref, absolute, score = prompt_ref.attention(c.q[b], c.rows_of(b, 0)[keep], c.rows_of(b, 1)[keep], int(keep.sum()) - 2,
                                                    64 ** -0.5)
        assert (np.abs(got[b] - ref) <= bound(t, 64, len(at), ref, absolute, score)).all(), b


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_a_call_that_serves_nobody_and_one_right_behind_it(t):
    """With the same workspace: the second begins only when the first is done."""
    c = Case(t, 2, 8, 2, 64, groups=[(40, [0, 70, 9] * 9), (0, [6, 7, 70])])
    g, ws = c.to_gpu(), torch.empty(1 << 28, dtype=torch.uint8, device=DEV)
    none = dict(g, ctx=torch.full_like(g["ctx"], -1))
    for _ in range(3):
        c.call(none, workspace=ws)
        assert (g["out"] == 7.0).all()
    for _ in range(3):
        c.call(none, workspace=ws)
        c.call(g, workspace=ws)
    with pytest.raises(mv.MtpError, match="length"):
        mv.sync_status()
    c.check(g)


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_a_malformed_tree_is_taken_as_a_chain_and_reported(t):
    c = Case(t, 4, 8, 2, 64, groups=[(2, [0, 70, 9]), (1, [62])], tree=True)
    g = c.to_gpu()
    for b, k, par in ((0, 0, 0), (1, 2, 2), (3, 3, -1)):
        g["parents"][b, k] = par
        c.parents[b] = np.arange(-1, 3)
    c.call(g)
    with pytest.raises(mv.MtpError, match="tree"):
        mv.sync_status()
    c.check(g)


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_blocks_beyond_32_bits(t):
    """Blocks at both ends of a cache of more than 2^32 values."""
    c = Case(t, 3, 16, 8, 128, groups=[(6, [0, 70, 9])], after=[100])
    g = c.to_gpu()
    nb = (1 << 32) // (64 * 8 * 128) + c.nb + 1
    far = torch.arange(c.nb, device=DEV)
    far[c.nb // 2:] += nb - c.nb
    for n in "kv":
        cache = torch.zeros(nb, 64, 8, 128, dtype=g[n].dtype, device=DEV)
        cache[far] = g[n]
        g[n] = cache
    g["table"] = torch.where(g["table"] >= 0, far[g["table"].long().clamp(min=0)].int(), -1)
    c.call(g)
    mv.sync_status()
    for n in "kv":
        g[n] = g[n][far]
    c.check(g)


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_two_graphs_with_one_workspace(t):
    """One after the other, with other sizes and from other streams."""
    cases = [Case(t, 3, 16, 4, 64, groups=[(9, [5 * i for i in range(n)])], before=[40], seed=n) for n in (2, 31)]
    ws = torch.empty(1 << 28, dtype=torch.uint8, device=DEV)
    graphs = []
    for c in cases:
        g = c.to_gpu()
        c.call(g, workspace=ws)
        torch.cuda.synchronize()
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=side):
            c.call(g, workspace=ws)
        graphs.append((graph, g))
    for _ in range(3):
        for graph, g in graphs:
            g["out"].fill_(7.0)
            graph.replay()
    torch.cuda.synchronize()
    mv.sync_status()
    for c, (_, g) in zip(cases, graphs):
        c.check(g)


def test_in_a_graph_on_its_own_stream():
    c = Case("bf16", 4, 32, 8, 128, groups=[(20, [10 * i for i in range(9)]), (3, [900, 3])])
    g = c.to_gpu()
    c.call(g)                                         # the first call on a device stays outside a capture
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        c.call(g)
    for seed in (1, 2):                               # other inputs, and other lengths, in the same tensors
        other = Case("bf16", 4, 32, 8, 128, groups=[(20, [10 * i for i in range(9)]), (3, [900, 3])], seed=seed)
        h = other.to_gpu()
        for n in ("q", "k_new", "v_new", "k", "v", "table", "ctx", "starts", "prefix"):
            g[n].copy_(h[n])
        g["out"].fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        mv.sync_status(side)
        other.check(g)


def test_two_calls_at_once():
    """On two streams, each with its own workspace (the default)."""
    cases = [Case("bf16", 4, 32, 8, 128, groups=[(30, [5 * i for i in range(12)])], seed=s) for s in (0, 1)]
    gs = [c.to_gpu() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        for c, g, s in zip(cases, gs, streams):
            c.call(g, stream=s)
    torch.cuda.synchronize()
    mv.sync_status()
    for c, g in zip(cases, gs):
        c.check(g)


def test_refusals_of_the_binding():
    c = Case("bf16", 2, 8, 2, 64, groups=[(2, [0, 5])])
    g = c.to_gpu()
    with pytest.raises(ValueError, match="k_cache"):
        c.call(dict(g, k=g["k"].float()))
    with pytest.raises(ValueError, match="group_starts"):
        c.call(dict(g, starts=g["starts"][:1]))
    with pytest.raises(ValueError, match="prefix_blocks"):
        c.call(dict(g, prefix=g["prefix"].long()))
    with pytest.raises(ValueError, match="parents"):
        c.call(dict(g, parents=g["table"]))
    with pytest.raises(mv.MtpError, match="workspace"):
        c.call(g, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    assert (g["out"] == 7.0).all()


def test_a_server_of_samples_of_one_prompt():
    """The prompt's blocks and slots, its K/V by slot, then steps of four samples that share it: blocks for the step's
    tokens, attention, rollback; against attention over the sequences themselves."""
    rng = np.random.default_rng(0)
    n, P, R, Hq, Hkv, d, nb = 4, 150, 3, 8, 2, 64, 40
    new = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(torch.bfloat16).to(DEV)
    kc, vc = new(nb, 64, Hkv, d), new(nb, 64, Hkv, d)
    table = torch.full((n, 8), -1, dtype=torch.int32, device=DEV)
    free = torch.arange(nb, dtype=torch.int32, device=DEV)
    count = torch.full((1,), nb, dtype=torch.int32, device=DEV)
    lens = torch.zeros(n, dtype=torch.int32, device=DEV)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)

    def assign(starts, T):
        slots, taken = torch.empty(T, dtype=torch.int64, device=DEV), torch.empty(n, dtype=torch.int32, device=DEV)
        mv.kv_block_assign(table, lens, starts, free, count, slots, taken)
        return slots, taken

    # the prompt's two full blocks belong to the first sample; its last 22 tokens are every sample's own
    k, v = new(P, Hkv, d), new(P, Hkv, d)
    slots, taken = assign(i32(0, 128, 128, 128, 128), 128)
    assert taken.tolist() == [2, 0, 0, 0]
    mv.mtp_kv_append(k[:128], v[:128], slots, kc, vc)
    table[1:, :2] = table[0, :2]
    lens += 128
    slots, taken = assign(i32(0, 22, 44, 66, 88), 88)
    assert taken.tolist() == [1, 1, 1, 1] and int(count) == nb - 6
    mv.mtp_kv_append(k[128:].repeat(n, 1, 1), v[128:].repeat(n, 1, 1), slots, kc, vc)
    lens += 22
    seqs = [[list(host(k)), list(host(v))] for _ in range(n)]
    starts, out = torch.arange(0, n * R + 1, R, dtype=torch.int32, device=DEV), new(n, R, Hq, d)
    for step in range(40):
        slots, taken = assign(starts, n * R)
        assert (taken >= 0).all()
        q, kn, vn = new(n, R, Hq, d), new(n, R, Hkv, d), new(n, R, Hkv, d)
        mv.mtp_verify_attention_prefix(q, kn, vn, kc, vc, table, lens, i32(0, n), i32(2), out)
        accepted = torch.from_numpy(rng.integers(0, R, n).astype(np.int32)).to(DEV)
        ctx = lens.tolist()
        for b in range(n):
            keys, values = (np.array(x + list(host(y[b]))) for x, y in zip(seqs[b], (kn, vn)))
            if step % 13 == 0:
                ref, absolute, score = prompt_ref.attention(host(q[b]), keys, values, ctx[b], d ** -0.5)
                assert (np.abs(host(out[b]) - ref) <= bound("bf16", d, len(keys), ref, absolute, score)).all()
            for x, y in zip(seqs[b], (keys, values)):
                x[:] = list(y[:ctx[b] + 1 + int(accepted[b])])
        mv.kv_rollback(table, lens, accepted, free, count, D=R - 1)
        mv.sync_status()
        assert lens.tolist() == [len(s[0]) for s in seqs]
    held = sorted(set(table[table >= 0].tolist()))
    assert sorted(held + free[:int(count)].tolist()) == list(range(nb))
