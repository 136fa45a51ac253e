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
