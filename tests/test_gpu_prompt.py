"""Blocks and slots from request lengths and the append by slot, against the plain implementations: tables, slots, counts
and bytes have to agree to the last."""
import numpy as np
import pytest
import torch

import mtp_speculative_decoding_verify_gb300 as mv
import prompt_ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def _no_error_left():
    mv.sync_status()
    yield
    mv.sync_status()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


class Pool:
    """Tables whose requests hold `lens` tokens, and a free list with `free` blocks (default: as many as asked for)."""

    def __init__(self, lens, n, free=None, room=2, seed=0, head=0, tail=0):
        rng = np.random.default_rng(seed)
        lens, n = np.array(lens, np.int64), np.array(n, np.int64)
        held, need = -(-lens // 64), -(-(lens + n) // 64)
        want = int(np.maximum(need - held, 0).sum())
        free = want if free is None else free
        ids = rng.permutation(int(held.sum()) + free).astype(np.int32)
        self.table = np.full((len(lens), int(max(need.max(), held.max())) + room), -1, np.int32)
        at = free
        for b, m in enumerate(held):
            self.table[b, :m] = ids[at:at + m]
            at += m
        self.free = np.concatenate([ids[:free], np.full(5, -1, np.int32)])
        self.count, self.lens = free, lens.astype(np.int32)
        self.starts = (head + np.concatenate([[0], np.cumsum(n)])).astype(np.int32)
        self.T = int(self.starts[-1]) + tail

    def call(self, **kw):
        g = dict(table=dev(self.table), count=dev(np.array([self.count], np.int32)),
                 slots=torch.full((self.T,), 77, dtype=torch.int64, device=DEV),
                 taken=torch.full((len(self.lens),), 55, dtype=torch.int32, device=DEV))
        mv.kv_block_assign(g["table"], dev(self.lens), dev(self.starts), dev(self.free), g["count"], g["slots"], g["taken"], **kw)
        return g

    def check(self, g):
        slots = np.full(self.T, 77, np.int64)
        table = self.table.copy()
        taken, left = prompt_ref.assign(table, self.lens, self.starts, self.free, self.count, slots)
        assert np.array_equal(g["taken"].cpu().numpy(), taken)
        assert np.array_equal(g["table"].cpu().numpy(), table)
        assert np.array_equal(g["slots"].cpu().numpy(), slots)
        assert int(g["count"]) == left


SIZES = {
    "step": (list(range(0, 300, 7)), [4] * 43),
    "one token": ([63], [1]),
    "one request, one block more": ([64], [1]),
    "nothing to append": ([0, 5, 64], [0, 0, 0]),
    "none, one and many": ([0, 5, 64, 127, 130, 3, 2048], [0, 1, 64, 65, 129, 0, 2048]),
    "a chunk among steps": ([100 + 3 * b for b in range(200)], [4] * 120 + [1900] + [3] * 79),
    "long": ([0, 77, 2047, 2048, 2049], [70000, 1, 2048, 4097, 2047]),
    "many requests": ([(37 * b) % 500 for b in range(2500)], [b % 5 for b in range(2500)]),
    "many chunks": ([(37 * b) % 5000 for b in range(300)], [(91 * b) % 4500 for b in range(300)]),
}


@pytest.mark.parametrize("name", list(SIZES))
@pytest.mark.parametrize("share", [1.0, 2.0, 0.6, 0.0])
def test_assign_to_the_last_entry(name, share):
    lens, n = SIZES[name]
    want = sum(max(0, -(-(a + m) // 64) - -(-a // 64)) for a, m in zip(lens, n))
    pool = Pool(lens, n, free=int(want * share), head=3, tail=4)
    pool.check(pool.call())


@pytest.mark.parametrize("n", [[3, 8, 0, 21], [40, 0, 9, 300]])
@pytest.mark.parametrize("share", [1.0, 0.6])
def test_assign_for_more_requests_than_a_batch_has(n, share):
    """Steps of many requests by one CTA, and longer appends by more pieces than are summed one by one."""
    B = 9001
    lens, n = [(37 * b) % 500 for b in range(B)], [n[b % 4] for b in range(B)]
    want = sum(max(0, -(-(a + m) // 64) - -(-a // 64)) for a, m in zip(lens, n))
    pool = Pool(lens, n, free=int(want * share), head=1)
    pool.check(pool.call())


@pytest.mark.parametrize("n", [[3, 10, 2, 16], [300, 10, 4000, 129]])
def test_assign_keeps_blocks_that_are_there(n):
    """Blocks handed out before, gaps among them, and a refused request asked again."""
    pool = Pool([60, 0, 640, 64], n, free=80)
    rng = np.random.default_rng(3)
    for b in range(4):
        last = (int(pool.lens[b]) + n[b] - 1) // 64
        for i in range(-(-int(pool.lens[b]) // 64), last + 1):
            if rng.random() < 0.4:
                pool.table[b, i] = 1000 + 100 * b + i
    pool.check(pool.call())
    pool.count = 1
    g = pool.call()
    pool.check(g)
    pool.table, pool.count = g["table"].cpu().numpy(), 70      # the second time the rest is served
    g = pool.call()
    pool.check(g)
    assert (g["taken"].cpu().numpy() >= 0).all()


@pytest.mark.parametrize("big", [False, True])
@pytest.mark.parametrize("fault,word", [("negative length", "length"), ("too long", "length"), ("far too long", "length"),
                                        ("no block for its tokens", "block-id"), ("bad id in the list", "block-id"),
                                        ("count below 0", "free-list"), ("count beyond the list", "free-list")])
def test_assign_refuses_and_reports_a_bad_request(big, fault, word):
    n = [4, 6, 5, 7] if not big else [400, 6000, 5, 70]
    pool = Pool([10, 70, 128, 3], n, free=400)
    if fault == "negative length":
        pool.lens[1] = -1
    elif fault == "too long":
        pool.lens[1] = pool.table.shape[1] * 64 - n[1] + 1
    elif fault == "far too long":
        pool.lens[1] = 2 ** 31 - 1
    elif fault == "no block for its tokens":
        pool.table[1, 1] = -1
    elif fault == "bad id in the list":
        pool.free[pool.count - 1] = -3
        pool.lens[0] = 64
        pool.table[0] = -1
        pool.table[0, 0] = 399
    elif fault == "count below 0":
        pool.count = -2
    else:
        pool.count = len(pool.free) + 1
    g = pool.call()
    with pytest.raises(mv.MtpError, match=word):
        mv.sync_status()
    if "count" in fault:
        given, pool.count = pool.count, 0
        g["count"] += -given
    pool.check(g)


@pytest.mark.parametrize("big", [False, True])
@pytest.mark.parametrize("starts", [[0, 5, 4, 9, 12], [-1, 2, 4, 9, 12], [0, 3, 6, 9, 1 << 20], [0, 1 << 30, 6, 9, 12]])
def test_assign_does_nothing_with_bad_starts(big, starts):
    pool = Pool([10, 70, 128, 3], [4, 3, 3, 3] if not big else [4, 3, 3, 3000])
    pool.starts = np.array(starts, np.int32)
    g = pool.call()
    with pytest.raises(mv.MtpError, match="length"):
        mv.sync_status()
    assert (g["taken"] == -1).all() and (g["slots"] == 77).all() and int(g["count"]) == pool.count
    assert np.array_equal(g["table"].cpu().numpy(), pool.table)


def test_assign_in_a_graph_on_its_own_stream():
    lens, n = SIZES["many chunks"]
    pool = Pool(lens, n, free=5000)
    g = pool.call()
    table, count = dev(pool.table), dev(np.array([pool.count], np.int32))
    lens_d, starts, free = dev(pool.lens), dev(pool.starts), dev(pool.free)
    slots, taken = torch.full_like(g["slots"], 77), torch.full_like(g["taken"], 55)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        mv.kv_block_assign(table, lens_d, starts, free, count, slots, taken)
    for _ in range(2):
        table.copy_(dev(pool.table))
        count.fill_(pool.count)
        slots.fill_(77)
        graph.replay()
        torch.cuda.synchronize()
        pool.check(dict(table=table, count=count, slots=slots, taken=taken))


# ---------------------------------------------------------------------------------------------------------- append
@pytest.mark.parametrize("T", [0, 1, 7, 1000])
@pytest.mark.parametrize("t", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("Hkv,d,d_v,apart", [(8, 128, 128, 0), (1, 64, 64, 0), (3, 64, 128, 16), (1, 576, None, 0), (1, 576, None, 64), (2, 128, 128, 4 * 128)])
def test_append_puts_rows_at_their_slots(T, t, Hkv, d, d_v, apart):
    gen = torch.Generator(device=DEV).manual_seed(T + Hkv)
    nb = T // 64 + 5
    row = Hkv * (d + (d_v or 0)) + apart
    rows = torch.randn(max(T, 1), row, generator=gen, device=DEV).to(t)[:T]
    k = rows[:, :Hkv * d].unflatten(1, (Hkv, d))
    v = None if d_v is None else rows[:, Hkv * d:Hkv * (d + d_v)].unflatten(1, (Hkv, d_v))
    kc = torch.randn(nb, 64, Hkv, d, generator=gen, device=DEV).to(t)
    vc = None if d_v is None else torch.randn(nb, 64, Hkv, d_v, generator=gen, device=DEV).to(t)
    slots = torch.randperm(nb * 64, generator=gen, device=DEV)[:T]
    slots[::5] = -1 - slots[::5]
    want_k, want_v = kc.clone(), None if vc is None else vc.clone()
    live = slots >= 0
    want_k.view(-1, Hkv, d)[slots[live]] = k[live]
    if v is not None:
        want_v.view(-1, Hkv, d_v)[slots[live]] = v[live]
    mv.mtp_kv_append(k if d_v is not None or T % 2 else k.flatten(1), v, slots, kc, vc)
    mv.sync_status()
    assert torch.equal(kc, want_k)
    assert vc is None or torch.equal(vc, want_v)


def test_append_reports_a_slot_beyond_the_cache():
    k = torch.ones(4, 2, 64, device=DEV)
    kc, vc = torch.zeros(3, 64, 2, 64, device=DEV), torch.zeros(3, 64, 2, 64, device=DEV)
    mv.mtp_kv_append(k, 2 * k, torch.tensor([5, 3 * 64, 2 ** 40, 191], device=DEV), kc, vc)
    with pytest.raises(mv.MtpError, match="block-id"):
        mv.sync_status()
    at = torch.zeros(3 * 64, device=DEV)
    at[[5, 191]] = 1.0
    assert torch.equal(kc.view(192, 128), at[:, None].expand(-1, 128)) and torch.equal(vc.view(192, 128), 2 * at[:, None].expand(-1, 128))


def test_append_beyond_32_bits():
    """A cache of more than 2^32 values: slots far apart."""
    nb = (1 << 32) // (64 * 8 * 128) + 3
    kc = torch.zeros(nb, 64, 8, 128, dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    slots = torch.tensor([nb * 64 - 1, 0, nb * 32], device=DEV)
    k = torch.arange(1, 4, device=DEV, dtype=torch.bfloat16)[:, None, None].expand(3, 8, 128).contiguous()
    mv.mtp_kv_append(k, -k, slots, kc, vc)
    mv.sync_status()
    for c, sign in ((kc, 1), (vc, -1)):
        rows = c.view(-1, 1024)
        assert torch.equal(rows[slots], sign * k.view(3, -1))
        assert int(torch.count_nonzero(rows[:, 0])) == 3


def test_append_refuses_scattered_values():
    k = torch.zeros(4, 64, 2, device=DEV).transpose(1, 2)
    c = torch.zeros(3, 64, 2, 64, device=DEV)
    slots = torch.zeros(4, dtype=torch.int64, device=DEV)
    with pytest.raises(ValueError, match="contiguous"):
        mv.mtp_kv_append(k, k, slots, c, c.clone())
    with pytest.raises(ValueError):
        mv.mtp_kv_append(k.contiguous(), None, slots, c, c)
    with pytest.raises(ValueError):
        mv.mtp_kv_append(k.contiguous(), k.contiguous(), slots.int(), c, c.clone())
