"""Context lengths at the end of 32 bits, where adding a step's rows wraps around: every call reports them as too long
and serves the other requests as ever."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU hosts too; the marker keeps them out of -m "not gpu"
    pytest.skip("needs a CUDA device", allow_module_level=True)

import mtp_speculative_decoding_verify_gb300 as mv  # noqa: E402
from mtp_speculative_decoding_verify_gb300 import synth  # noqa: E402
from test_gpu_gqa_tc import CASES as GQA_TC  # noqa: E402
from test_gpu_parity import SMALL  # noqa: E402

DEV = torch.device("cuda:0")
WORKLOADS = {
    "fp32": SMALL["cfg0"].with_(B=3),
    "bf16 GQA": SMALL["cfg3_small_mixed"],
    "bf16 GQA, 64 rows": GQA_TC["rows64_chain"],
    "MLA": synth.CFG1.with_(name="MLA, lengths", B=3, D=2, Hq=16, ctx=(60, 300), H=64, V=777),
    "MLA pairs": synth.CFG1.with_(name="MLA pairs, lengths", B=3, D=7, Hq=16, ctx=(60, 700), H=64, V=777),
}


def _length_error():
    with pytest.raises(mv.MtpError) as ei:
        mv.sync_status()
    assert ei.value.code == 4 and "length" in str(ei.value)


@pytest.mark.parametrize("back", [0, 1, "D", "R"])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("name", list(WORKLOADS))
def test_attention(name, back, tree):
    w = WORKLOADS[name]
    parents = None
    if tree:
        parents = torch.arange(-1, w.R - 1, dtype=torch.int32, device=DEV).repeat(w.B, 1).contiguous()

    def run(bad):
        att = synth.make_attention_inputs(w, DEV)
        out = torch.full((w.B, w.R, w.Hq, w.d_v), 7.0, dtype=w.torch_dtype, device=DEV)
        if bad:
            att["ctx_lens"][1] = 2 ** 31 - 1 - {"D": w.D, "R": w.R}.get(back, back)
        mv.mtp_verify_attention(att["q"], att["k_new"], att["v_new"], att["k_cache"], att["v_cache"], att["block_table"],
                                att["ctx_lens"], out, sm_scale=w.sm_scale, parents=parents)
        return out

    want = run(False)
    mv.sync_status()
    got = run(True)
    _length_error()
    others = [b for b in range(w.B) if b != 1]
    assert (got[1] == 7.0).all()
    assert torch.equal(got[others], want[others])


@pytest.mark.parametrize("back", [0, 1, 3, 4])
def test_rollback_and_compaction(back):
    D, length = 3, 2 ** 31 - 1 - back
    table = torch.arange(6, dtype=torch.int32, device=DEV).view(2, 3)
    lens = torch.tensor([length, 126], dtype=torch.int32, device=DEV)
    n = torch.tensor([1, 0], dtype=torch.int32, device=DEV)
    free, count = torch.full((8,), -1, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    mv.kv_rollback(table, lens, n, free, count, D=D)
    _length_error()
    assert table.tolist() == [[0, 1, 2], [3, 4, -1]] and lens.tolist() == [length, 127]
    assert free.tolist() == [5] + [-1] * 7 and int(count) == 1

    cache = [torch.randn(6, 64, 2, 64, device=DEV) for _ in "kv"]
    want = [c.clone() for c in cache]
    for c in want:
        c[4, 1] = c[4, 2]
    nodes = torch.tensor([[0, 2, -1, -1], [0, 2, -1, -1]], dtype=torch.int32, device=DEV)
    table = torch.arange(6, dtype=torch.int32, device=DEV).view(2, 3)
    lens = torch.tensor([length, 64], dtype=torch.int32, device=DEV)
    mv.mtp_tree_kv_compact(cache[0], cache[1], table, lens, nodes, torch.ones(2, dtype=torch.int32, device=DEV))
    _length_error()
    assert all(torch.equal(a, b) for a, b in zip(cache, want))
