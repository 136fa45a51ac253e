"""Verify attention of requests that share a prefix where bad blocks leave a row little to see, or nothing: such a row is 0,
whatever Q holds, and of the cache only what has a place is written."""
import numpy as np
import pytest
import torch

import mtp_speculative_decoding_verify_gb300 as mv
import prompt_ref
from test_gpu_prompt_attention import Case, bound, host

pytestmark = pytest.mark.gpu
HEADS = [("bf16", 8, 2, 64), ("bf16", 48, 4, 128), ("bf16", 160, 1, 64), ("f32", 8, 2, 64), ("f32", 6, 1, 128)]


@pytest.fixture(autouse=True)
def _no_error_left():
    mv.sync_status()
    yield
    mv.sync_status()


def call_with_bad_blocks(c, drop, bad):
    """Drop the table's entries `drop` ((request, block), a prefix's by the row of its group's first request), call, and
    compare outputs and caches with attention over what is left."""
    g = c.to_gpu()
    for b, i in drop:
        g["table"][b, i] = bad
    c.call(g)
    with pytest.raises(mv.MtpError, match="block-id"):
        mv.sync_status()
    got, want, R = host(g["out"]).astype(np.float64), c.cache.copy(), c.R
    for b, ctx in enumerate(c.ctx):
        first = next((int(c.starts[k]) for k in range(len(c.prefix)) if c.starts[k] <= b < c.starts[k + 1]), b)
        gone = {i for r, i in drop if r == (first if i < c.blocks[b] else b)}
        see = prompt_ref.path_rows(None if c.parents is None else c.parents[b], R)
        k, v = c.rows_of(b, 0), c.rows_of(b, 1)
        for j in range(R):
            if (ctx + j) // 64 not in gone:
                at = c.table[b, (ctx + j) // 64], (ctx + j) % 64
                want[0][at], want[1][at] = c.k[b, j], c.v[b, j]
            t = np.array([x for x in range(ctx + R) if x // 64 not in gone and (x < ctx or see[j, x - ctx])], int)
            if len(t) == 0:
                assert (got[b, j] == 0.0).all(), (b, j)
                continue
            # (row j alone, of which the last key that is left is its "verify token")
            ref, absolute, score = prompt_ref.attention(c.q[b, j:j + 1], k[t], v[t], len(t) - 1, c.d ** -0.5)
            assert (np.abs(got[b, j:j + 1] - ref) <= bound(c.t, c.d, len(t), ref, absolute, score)).all(), (b, j)
    assert np.array_equal(host(g["k"]), want[0], equal_nan=True) and np.array_equal(host(g["v"]), want[1], equal_nan=True)


@pytest.mark.parametrize("t,Hq,Hkv,d", HEADS)
@pytest.mark.parametrize("bad", [-1, 10 ** 6])
@pytest.mark.parametrize("tree", [False, True])
def test_rows_that_see_nothing_are_0(t, Hq, Hkv, d, bad, tree):
    """All blocks of requests in no group, of a request and its group's prefix, and of all of a group."""
    c = Case(t, 4, Hq, Hkv, d, before=[0, 100], groups=[(5, [10, 70, 0]), (2, [3, 64]), (0, [40, 200])], after=[300], tree=tree)
    drop = [(b, i) for b in (0, 1, 3, 6, 8, 9) for i in range(c.table.shape[1]) if i >= c.blocks[b]]
    drop += [(2, i) for i in range(5)] + [(5, i) for i in range(2)]
    c.q[3, 1, 0, 5], c.q[9, 0, 1, 7] = np.nan, np.inf
    call_with_bad_blocks(c, drop, bad)


@pytest.mark.parametrize("t,Hq,Hkv,d", HEADS)
def test_verify_tokens_without_a_block(t, Hq, Hkv, d):
    """The block of all verify tokens, and the second of two that they lie in."""
    c = Case(t, 4, Hq, Hkv, d, before=[64, 126], groups=[(3, [0, 62, 5]), (1, [0])], after=[63])
    call_with_bad_blocks(c, [(0, 1), (1, 2), (2, 3), (3, 4), (5, 1), (6, 1)], -1)


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_a_long_prefix_of_bad_blocks_only(t):
    """Shares of it whose every tile is empty."""
    c = Case(t, 2, 8, 2, 64, groups=[(150, [9, 0, 70]), (150, [5])])
    call_with_bad_blocks(c, [(0, i) for i in range(150)] + [(3, i) for i in range(149)] + [(3, 150)], -1)
