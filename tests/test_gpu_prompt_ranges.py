"""Block assignment on each of its launch plans, up to their borders, and batches in which long appends stand among steps;
mtp_last_launch_count says that a case runs the plan that it is there for (1: one CTA, 2: counts and pieces)."""
import pytest

import mtp_speculative_decoding_verify_gb300 as mv
from test_gpu_prompt import Pool

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_error_left():
    mv.sync_status()
    yield
    mv.sync_status()


def run(n, share, launches):
    lens = [(37 * b) % 500 for b in range(len(n))]
    want = sum(max(0, -(-(a + m) // 64) - -(-a // 64)) for a, m in zip(lens, n))
    pool = Pool(lens, n, free=int(want * share), head=1, tail=2)
    g = pool.call()
    assert mv.lib().mtp_last_launch_count() == launches
    pool.check(g)


def spread(B, T):
    """T tokens over B requests, unevenly: some append none, some more than 16."""
    n = [(0, 5, 9, 18)[b % 4] * T // (8 * B) for b in range(B)]
    for b in range(B):
        if sum(n) >= T:
            break
        n[b] += 1
    n[-1] += T - sum(n)
    return n


# T counts the entry before starts[0] and the two from starts[B] on, too
@pytest.mark.parametrize("B,T,launches", [(8000, 64000, 1), (2500, 20000, 1), (8192, 65536, 1), (8193, 65537, 2), (9000, 17000, 1),
                                          (1024, 16384, 1), (1024, 16385, 2), (3000, 24000, 1), (3000, 24001, 2), (100, 1600, 1),
                                          (100, 1601, 2)])
@pytest.mark.parametrize("share", [1.0, 0.6])
def test_at_the_borders_of_the_plans(B, T, launches, share):
    run(spread(B, T - 3), share, launches)


@pytest.mark.parametrize("B,T", [(8176, 65540), (8176, 68000)])
@pytest.mark.parametrize("share", [1.0, 0.6])
def test_at_the_border_of_counts_by_groups(B, T, share):
    """T / 2048 + 2 B pieces: 16384, the most that are summed one by one, and 16385."""
    run(spread(B, T - 3), share, 2)


@pytest.mark.parametrize("B,long,launches", [
    (1500, {1300: 9000}, 1), (1500, {1024: 5000, 1055: 1, 1030: 4000, 1499: 700}, 1), (4000, {0: 6000, 2047: 6000, 2048: 8000}, 1),
    (8192, {5000: 30000, 5001: 200}, 1), (1500, {1300: 30000}, 2), (9000, {b: 300 for b in range(100, 9000, 40)}, 2),
])
@pytest.mark.parametrize("share", [1.0, 0.9, 0.4])
def test_prompts_among_the_steps_of_many_requests(B, long, launches, share):
    """Of the second and later thousand requests too, which one CTA does after the first."""
    run([long.get(b, 1 + b % 4) for b in range(B)], share, launches)
