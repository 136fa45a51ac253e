"""Verify attention over the 8-bit cache where V's scales in one request lie as far apart as they may: blocks of zeros
(whose scale the append makes 2^-100) next to blocks of large values. The weight of a zero block counts in the softmax
whatever its scale."""
import numpy as np
import pytest
import torch

import kv8_ref
import mtp_speculative_decoding_verify_gb300 as mv
from test_gpu_kv8_range import check_rows
from test_gpu_kv8_window import Case, host

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_error_left():
    mv.sync_status()
    yield
    mv.sync_status()


ORDERS = {  # which of n blocks hold zeros
    "behind": lambda n: np.arange(n) >= 2,
    "before": lambda n: np.arange(n) < n - 2,
    "between": lambda n: np.arange(n) % 2 == 1,
    "middle": lambda n: (np.arange(n) >= 3) & (np.arange(n) < n - 2),
}
SCORES = {  # octaves of a block's scores over the first one's
    "equal": lambda n: np.zeros(n),
    "rising": lambda n: np.linspace(0, 12, n),
    "falling": lambda n: np.linspace(12, 0, n),
    "jump": lambda n: 19.5 * (np.arange(n) >= 2),
}


def far_apart(order, scores, e, R, Hq, ctx, d=64, window=0, sinks=0, t="bf16"):
    """Requests whose V is zero in some blocks and of size 2^(e + 4) in the others, with scores by block."""
    c = Case(True, t, len(ctx), R, Hq, 1, d, ctx, window, sinks, seed=len(ctx) + e, drop=False)
    rng = np.random.default_rng(e)
    u = np.sign(rng.standard_normal(d))
    c.q = host(torch.from_numpy(np.broadcast_to(u, c.q.shape) + 0.01 * rng.standard_normal(c.q.shape)).to(torch.bfloat16))
    # scores: q.k d^-0.5 log2(e) octaves, of u.u = d
    per = d ** 0.5 * np.log2(np.e)
    c.v = host(torch.from_numpy(rng.standard_normal(c.v.shape) * 2.0 ** (e + 4)).to(torch.bfloat16))
    for b, n in enumerate(ctx):
        pages = (n + R + 63) // 64
        zero, octaves = ORDERS[order](pages), SCORES[scores](pages)
        for i in range(pages):
            blk = c.table[b, i]
            c.scale[0, blk], c.scale[1, blk] = 2.0 ** -6, 2.0 ** -100 if zero[i] else 2.0 ** e
            c.byte[0, blk] = kv8_ref.to_e4m3(64 * (octaves[i] / per * u + 0.02 * rng.standard_normal(c.byte[0, blk].shape)))
            c.byte[1, blk] = 0 if zero[i] else kv8_ref.to_e4m3(16 * rng.standard_normal(c.byte[1, blk].shape))
        c.k[b] = octaves[-1] / per * u
        if zero[-1]:
            c.v[b] = 0
    c.k = host(torch.from_numpy(c.k).to(torch.bfloat16))
    return c


def run(c, requests=None):
    g = c.to_gpu()
    c.call(g)
    mv.sync_status()
    c.append()
    check_rows(c, g, requests)


@pytest.mark.parametrize("e", [14, 28, 60, 120])
@pytest.mark.parametrize("scores", list(SCORES))
@pytest.mark.parametrize("order", list(ORDERS))
@pytest.mark.parametrize("R,Hq", [(2, 2), (3, 8), (6, 8)], ids=["4 rows", "24 rows", "48 rows"])
def test_zero_blocks_among_large_ones(order, scores, e, R, Hq):
    run(far_apart(order, scores, e, R, Hq, [560, 130]))


@pytest.mark.parametrize("e", [28, 60, 120])
@pytest.mark.parametrize("d,Hq", [(64, 4), (128, 16)])
@pytest.mark.parametrize("order", list(ORDERS))
def test_zero_blocks_of_a_request_that_ctas_share(order, e, d, Hq):
    run(far_apart(order, "rising", e, 3, Hq, [4000, 700], d=d))


@pytest.mark.parametrize("order", list(ORDERS))
@pytest.mark.parametrize("window,sinks", [(150, 0), (64, 70), (300, 1)])
@pytest.mark.parametrize("R,Hq", [(16, 1), (15, 4)], ids=["16 rows", "60 rows"])
def test_zero_blocks_that_some_rows_do_not_see(order, window, sinks, R, Hq):
    """Pages at the window's edge leave some rows' tiles empty, with a scale of V far from what the row has met."""
    run(far_apart(order, "equal", 60, R, Hq, [570, 700, 64 * 9 - 7], window=window, sinks=sinks))


@pytest.mark.parametrize("scores", list(SCORES))
@pytest.mark.parametrize("R,Hq", [(2, 2), (6, 8)])
def test_every_value_zero(scores, R, Hq):
    c = far_apart("behind", scores, 0, R, Hq, [560, 2100])
    c.byte[1], c.scale[1], c.v[:] = 0, 2.0 ** -100, 0
    g = c.to_gpu()
    c.call(g)
    assert (g["out"] == 0).all()
