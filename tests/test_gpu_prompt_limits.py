"""The calls for requests that share a prompt where a batch's tokens come near the end of 31 bits, and pass it."""
import pytest
import torch

import mtp_speculative_decoding_verify_gb300 as mv

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_error_left():
    mv.sync_status()
    yield
    mv.sync_status()
    torch.cuda.empty_cache()      # (tens of GB)


def needs(n_bytes):
    if torch.cuda.mem_get_info()[0] < n_bytes + (1 << 30):
        pytest.skip("%d GB" % (n_bytes >> 30))


@pytest.mark.parametrize("T", [2 ** 31, 2 ** 32, 2 ** 32 + 3])
def test_append_refuses_more_tokens_than_31_bits_count(T):
    """Not a part of them: 2^32 + 3 are not 3. (Tokens all at one address, so that the slots are all that takes room.)"""
    needs(8 * T)
    slots = torch.empty(T, dtype=torch.int64, device="cuda")
    k = torch.ones(1, 1, 8, dtype=torch.bfloat16, device="cuda").expand(T, 1, 8)
    cache = torch.zeros(2, 64, 1, 8, dtype=torch.bfloat16, device="cuda")
    slots[:4] = torch.arange(4)
    with pytest.raises(ValueError, match="2\\^31"):
        mv.mtp_kv_append(k, k, slots, cache, cache.clone())
    assert not cache.any()


@pytest.mark.parametrize("T", [2 ** 31 - 1, 2 ** 31 - 2048, 2 ** 31 - 2049])
def test_assign_clears_the_slots_of_a_refused_request_of_any_length(T):
    """One of almost all of the batch's tokens, which no table is wide enough for, before one that is served."""
    needs(8 * T)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    table, count = torch.full((2, 4), -1, dtype=torch.int32, device="cuda"), i32(3)
    slots, taken = torch.full((T,), 77, dtype=torch.int64, device="cuda"), i32(55, 55)
    mv.kv_block_assign(table, i32(0, 0), i32(0, T - 5, T), i32(8, 7, 6), count, slots, taken)
    with pytest.raises(mv.MtpError, match="length"):
        mv.sync_status()
    assert taken.tolist() == [-1, 1] and int(count) == 2 and table.tolist() == [[-1] * 4, [6, -1, -1, -1]]
    assert int(slots[:T - 5].max()) == -1 and int(slots[:T - 5].min()) == -1
    assert slots[T - 5:].tolist() == [6 * 64 + x for x in range(5)]
