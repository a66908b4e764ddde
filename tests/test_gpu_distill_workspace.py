"""Statistics of many rows without a workspace, through the C call and the
binding: the same bits as with one."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a HIP GPU"),
]

import vocab_sharded_embedding_amd as vpe  # noqa: E402


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,v", [(256, 151936), (300, 1001), (256, 3)])
def test_null_workspace(m, v, dtype):
    g = torch.Generator(device="cuda").manual_seed(m + v)
    z = torch.randn(m, v, generator=g, device="cuda").to(dtype)
    k = 3
    ids = torch.randint(0, v, (m, k), generator=g, device="cuda")
    t = torch.randn(m, k, generator=g, device="cuda")
    ws = torch.empty(max(16, vpe.vpe_distill_workspace(m, v)), dtype=torch.uint8, device="cuda")
    lse, dot = vpe.vpe_distill_shard(z, ids, t, 0, v, workspace=ws)
    got = [torch.full((m,), float("nan"), device="cuda") for _ in range(2)]
    rs = vpe.load_library().vpe_distill_shard(
        z.data_ptr(), v, 0, m, v, vpe.VPE_F32 if dtype == torch.float32 else vpe.VPE_BF16, 0, v,
        1.0, ids.data_ptr(), vpe.VPE_I64, t.data_ptr(), vpe.VPE_F32, k, None, got[0].data_ptr(),
        got[1].data_ptr(), None, 0, torch.cuda.current_stream().cuda_stream)
    assert rs == vpe.VPE_OK
    assert torch.equal(got[0], lse) and torch.equal(got[1], dot)
    again = vpe.vpe_distill_shard(z, ids, t, 0, v)
    assert torch.equal(again[0], lse) and torch.equal(again[1], dot)
