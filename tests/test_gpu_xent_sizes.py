"""Sizes at which one launch would need more work-items than a grid holds, or which are
too large for a test against all of a 64-bit result: parts of it are compared."""
import pytest
import torch

import vocab_sharded_embedding_amd as vpe
from _loss import HALF, U, assert_within

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_sums_of_more_values_than_a_grid_of_the_join(dtype):
    """17000 x 4100 values of grad_x, and rows without a target among the last ones."""
    m, vocab, dim = 17000, 70, 4100
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(m, dim, generator=g, device="cuda").to(dtype)
    w = (0.02 * torch.randn(vocab, dim, generator=g, device="cuda")).to(dtype)
    t = torch.randint(0, vocab, (m,), generator=g, device="cuda")
    t[torch.arange(m, device="cuda") % 1000 > 990] = -100
    z = x.double() @ w.double().T
    live = t >= 0
    lse = torch.where(live, torch.logsumexp(z, 1), 0.0).float()
    gl = torch.ones(m, device="cuda")
    gx, none = vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, vocab, with_weight=False)
    assert none is None and (gx[~live] == 0).all()
    p = torch.exp(z - lse.double()[:, None])
    d = p.clone()
    d[live, t[live]] -= 1
    d = torch.where(live[:, None], d, 0.0)
    size = (x.double().abs() @ w.double().abs().T).max(1).values[:, None]
    # logits: dim terms; exponential, subtraction and factor: a few U of p
    err = p * U * ((dim + 2) * size + 3 * (z - lse.double()[:, None]).abs() + 8)
    err = err + (HALF[dtype] + 4 * U) * (d.abs() + err)
    want = d @ w.double()
    bound = err @ w.double().abs() + (vocab + 64) * U * ((d.abs() + err) @ w.double().abs())
    bound = bound + (HALF[dtype] + 2 * U) * (want.abs() + bound) + 1e-37
    assert_within(gx[live], want[live], bound[live], "grad_x")
    zl = torch.randn(m, vocab, generator=g, device="cuda").to(dtype)
    gx, none = vpe.vpe_lmhead_grad(zl, x, w, with_weight=False)
    want, mag = zl.double() @ w.double(), zl.double().abs() @ w.double().abs()
    bound = (vocab + 64) * U * mag
    bound = bound + (HALF[dtype] + 2 * U) * (want.abs() + bound) + 1e-37
    assert_within(gx, want, bound, "grad_x of given logits' gradient")
