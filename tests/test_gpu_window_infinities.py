"""Infinities and NaN that a row of windowed or 8-bit verify attention sees act as in softmax(q k) v: a score of -inf
has no weight, 0 x inf and 0 x NaN are NaN, and a row all of whose scores are -inf is NaN. Only a row that sees no slot
at all (bad blocks) is 0."""
import numpy as np
import pytest
import torch

import kv8_ref
import mtp_speculative_decoding_verify_gb300 as mv
from test_gpu_kv8_window import Case, bound, host, TYPES

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_error_left():
    mv.sync_status()
    yield
    mv.sync_status()


def check(c, g):
    """Against the formula in float64, infinities and NaN in place; finite outputs within `bound` of the keys whose
    score is finite."""
    c.append()
    got = g["out"].double().cpu().numpy()
    group = c.q.shape[2] // c.k.shape[2]
    kinds = set()
    for b in range(len(c.ctx)):
        t = np.arange(c.ctx[b] + c.R)
        t = t[kv8_ref.visible(t, c.ctx[b], c.window, c.sinks) | (t > c.ctx[b])]
        ks, vs = c.rows(0, b)(t), c.rows(1, b)(t)
        for j in range(c.R):
            see = kv8_ref.visible(t, c.ctx[b] + j, c.window, c.sinks)
            for h in range(c.q.shape[2]):
                k, v, q = ks[see, h // group], vs[see, h // group], c.q[b, j, h].astype(np.float64)
                with np.errstate(invalid="ignore"):
                    x = (k * q).sum(1) * c.d ** -0.5
                    w = np.exp(x - x.max())
                    w /= w.sum()
                    ref = (w[:, None] * v).sum(0)
                    x = got[b, j, h]
                where = (b, j, h)
                assert np.array_equal(np.isnan(x), np.isnan(ref)), where
                assert np.array_equal(x[np.isinf(x)], ref[np.isinf(x)]) and np.array_equal(np.isinf(x), np.isinf(ref)), where
                kinds |= {"nan"} if np.isnan(ref).any() else {"inf"} if np.isinf(ref).any() else {"finite"}
                f = np.isfinite(ref)
                if f.any():
                    on = w > 0
                    absolute, score = w[on] @ np.abs(v[on][:, f]), (np.abs(k[on]) @ np.abs(q)).max() * c.d ** -0.5
                    lim = bound(c.t, c.kv8, c.d, c.ctx[b] + c.R, ref[f], absolute, score, w.max() * np.abs(v[on][:, f]).sum(0))
                    assert (np.abs(x[f] - ref[f]) <= lim).all(), where
    return kinds


def windowed(t, ctx, window, sinks=0, R=3, Hq=4, seed=0, **kw):
    c = Case(False, t, len(ctx), R, Hq, 2, 64, ctx, window, sinks, seed=seed, drop=False, **kw)
    c.q[:, :, :, 5] = np.abs(c.q[:, :, :, 5]) + 0.5
    c.q = host(torch.from_numpy(c.q).to(TYPES[t]))
    return c


def put(c, which, b, slots, kvh, dim, value):
    """One dim of K (0) or V (1) of some slots of request b, verify tokens' among them."""
    for s in slots:
        if s >= c.ctx[b]:
            (c.k, c.v)[which][b, s - c.ctx[b], kvh, dim] = value
        else:
            c.cache[which][c.table[b, s // 64], s % 64, kvh, dim] = value


def run(c):
    g = c.to_gpu()
    c.call(g)
    mv.sync_status()
    return check(c, g)


CASES = [([0, 100, 64], 1, 0), ([10, 200, 130], 1000, 0), ([300, 90], 70, 3), ([2500], 5000, 0), ([2500, 70], 2000, 65),
         ([400] * 40, 10 ** 6, 0)]


@pytest.mark.parametrize("ctx,window,sinks", CASES)
@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_every_score_minus_infinity(t, ctx, window, sinks):
    c = windowed(t, ctx, window, sinks)
    put(c, 0, 0, range(ctx[0] + c.R), 1, 5, -np.inf)
    assert run(c) == {"nan", "finite"}


@pytest.mark.parametrize("ctx,window,sinks", CASES)
@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_some_scores_minus_infinity(t, ctx, window, sinks):
    """The first part of a request and its second verify token: row 1 of window 1 sees nothing else."""
    c = windowed(t, ctx, window, sinks)
    for b in range(0, len(ctx), 2):
        put(c, 0, b, list(range(ctx[b] * 2 // 3)) + [ctx[b] + 1], 0, 5, -np.inf)
    run(c)


@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("at", [3, 290, 1200, 2490, 2501])
@pytest.mark.parametrize("window,sinks", [(5000, 0), (2300, 10)])
@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_a_value_behind_a_score_of_minus_infinity(t, window, sinks, at, value):
    """0 x inf: NaN in that dim of the rows that see the slot, in whole pages and in masked ones."""
    c = windowed(t, [2500, 130], window, sinks, seed=at)
    put(c, 0, 0, [at], 1, 5, -np.inf)
    put(c, 1, 0, [at], 1, 9, value)
    put(c, 1, 0, [at], 0, 11, value)         # head 0's score is finite
    assert "nan" in run(c) or at < 2500 - window


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_a_split_of_minus_infinities_hands_its_nan_on(t):
    """A long part of the request without weight, a NaN of V in it."""
    c = windowed(t, [2500], 5000)
    put(c, 0, 0, range(1000), 1, 5, -np.inf)
    put(c, 1, 0, [100], 1, 9, np.nan)
    assert run(c) == {"nan", "finite"}


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("ctx", [[0, 70], [700, 70], [4000, 70]])
def test_infinite_queries_over_the_8_bit_cache(t, sign, ctx):
    """q = sign inf against keys below zero in that dim: scores of -inf (or inf), softmax of which is NaN either way."""
    c = Case(True, t, 2, 2, 4, 2, 64, ctx, 0, 0, seed=1)
    c.byte[0, :, :, :, 5] |= 128
    c.byte[0, :, :, :, 5] = np.where(c.byte[0, :, :, :, 5] == 128, 129, c.byte[0, :, :, :, 5])     # (not -0)
    c.k[:, :, :, 5] = -1.0
    c.q[0, 1, 2, 5] = sign * np.inf
    assert run(c) == {"nan", "finite"}


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("kv8", [True, False], ids=["kv8", "window"])
@pytest.mark.parametrize("ctx", [100, 3000])
def test_rows_that_see_no_slot_are_zero(t, kv8, ctx):
    """Request 1's blocks are all bad; request 0 sees scores of -inf only; request 2 is an ordinary one."""
    c = Case(kv8, t, 3, 3, 4, 2, 64, [ctx, ctx, ctx], 0 if kv8 else 10 ** 5, 0, seed=3)
    if not kv8:
        c.q[:, :, :, 5] = 1.0
        put(c, 0, 0, range(ctx + 3), 0, 5, -np.inf)
    g = c.to_gpu()
    g["table"][1] = -1
    c.call(g)
    with pytest.raises(mv.MtpError, match="block-id"):
        mv.sync_status()
    out = host(g["out"])
    assert (out[1] == 0).all() and np.isfinite(out[2]).all()
    assert np.isnan(out[0, :, :2]).all() != kv8 and np.isfinite(out[0, :, 2:]).all()
