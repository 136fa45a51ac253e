"""How exact windowed and 8-bit verify attention of bf16 rows is on the whole, where a bound for each output by itself
says little: long rows of flat weights, so that a page left out or a probability of half its bits shows."""
import numpy as np
import pytest

import kv8_ref
import mtp_speculative_decoding_verify_gb300 as mv
from test_gpu_kv8_window import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_error_left():
    mv.sync_status()
    yield
    mv.sync_status()


SHAPES = [  # R, Hq, Hkv, d, contexts
    (4, 8, 2, 128, [2900, 640]),            # 16 rows a KV head
    (2, 4, 4, 64, [3100, 2000, 64]),        # 2
    (6, 8, 1, 128, [2900, 1000]),           # 48
    (5, 6, 1, 64, [3000]),                  # 30
    (9, 16, 2, 64, [1500, 2500]),           # 72
    (4, 8, 2, 128, [9000, 3, 4097]),
]


def errors(c, got):
    """(root mean square error, its limit, and the errors of outputs without slots 64 .. 127 and of probabilities of 4
    bits) of each request, all over the outputs' root mean square.

    An output's error is the sum over its keys of w e v, with w the weight, plus what rounds the output:
      e, of a probability: at most 2^-8 (bf16), or 2^-8 + 2^-11 (two e4m3 terms behind a rounding to f16), roundings to
        nearest, so without a sign of their own from key to key. And e4m3's steps below its normal numbers: 2^-10 of
        the largest probability near (see `bound` of the per-output test; scores here lie within a few octaves). As a
        sum of independent terms, the square is at most e^2 sum (w v)^2; twice the root of that is allowed.
      fp32 sums: 2^-23 of what is summed, at each of n steps, in numerator and denominator. Partial sums of V's signs
        stay within four times root sum (w v)^2.
      the output in bf16: 2^-8 of it."""
    eps = 2.0 ** -8 + (2.0 ** -11 if c.kv8 else 0.0)
    floor = 2.0 ** -10 if c.kv8 else 0.0
    group = c.q.shape[2] // c.k.shape[2]
    for b in range(len(c.ctx)):
        t = np.arange(c.ctx[b] + c.R)
        t = t[kv8_ref.visible(t, c.ctx[b], c.window, c.sinks) | (t > c.ctx[b])]
        ks, vs = c.rows(0, b)(t), c.rows(1, b)(t)
        far = lim = lost = coarse = size = 0.0
        for j in range(c.R):
            see = kv8_ref.visible(t, c.ctx[b] + j, c.window, c.sinks)
            for h in range(c.q.shape[2]):
                k, v, q = ks[see, h // group], vs[see, h // group], c.q[b, j, h].astype(np.float64)
                x = k @ q * c.d ** -0.5
                w = np.exp(x - x.max())
                w /= w.sum()
                ref, noise = w @ v, (w * w) @ (v * v)
                most = (eps * eps) * noise + (floor * w.max()) ** 2 * (v * v).sum(0)
                sums = 2 * len(w) * 2.0 ** -23 * (np.abs(ref) + 4 * np.sqrt(noise))
                lim += ((2.0 ** -8 * ref) ** 2 + 4 * most + sums ** 2).sum()
                far += ((got[b, j, h] - ref) ** 2).sum()
                size += (ref ** 2).sum()
                gone = (t[see] >= 64) & (t[see] < 128)
                other = w[~gone] @ v[~gone] / max(w[~gone].sum(), 1e-30)
                lost += ((other - ref) ** 2).sum()
                m, e = np.frexp(w)
                coarse += ((np.ldexp(np.round(m * 16) / 16, e) @ v - ref) ** 2).sum()
        yield tuple(np.sqrt(x / size) for x in (far, lim, lost, coarse))


@pytest.mark.parametrize("window", [0, 700, 10 ** 5])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "R%d_%d/%dx%d_%d" % (*s[:4], s[4][0]))
@pytest.mark.parametrize("kv8", [True, False], ids=["kv8", "window"])
def test_error_over_all_outputs(kv8, shape, window):
    if window == 0 and not kv8:
        window = 2 ** 31 - 1
    R, Hq, Hkv, d, ctx = shape
    c = Case(kv8, "bf16", len(ctx), R, Hq, Hkv, d, ctx, window, 3 if window else 0, seed=R)
    c.q *= np.float32(0.25)                  # (a power of two: still bf16)
    g = c.to_gpu()
    c.call(g)
    mv.sync_status()
    c.append()
    for b, (far, lim, lost, coarse) in enumerate(errors(c, g["out"].double().cpu().numpy())):
        print("request %d: %.2e of %.2e; without a page %.2e, with 4 bits %.2e" % (b, far, lim, lost, coarse))
        assert far <= lim
        if c.ctx[b] > 200:
            assert coarse > 1.4 * lim
            assert window == 700 or lost > 4 * lim
