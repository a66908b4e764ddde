"""Sizes at which one launch would need more work-items than a grid holds, or which are
too large for a test against all of a 64-bit result: parts of it are compared."""
import pytest
import torch

import vocab_sharded_embedding_amd as vpe
from _loss import HALF, U, assert_within

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
MOST = (1 << 31) - 1


def test_the_largest_table_is_cleared():
    """2^31 - 1 rows of one value: 2^24 tiles of 128 rows."""
    w = torch.zeros(MOST, 1, device="cuda", dtype=BF16)
    gw = torch.full_like(w, 7.0)
    x = torch.empty(0, 1, device="cuda", dtype=BF16)
    none = torch.empty(0, device="cuda")
    ids = torch.empty(0, device="cuda", dtype=torch.int64)
    vpe.vpe_lmhead_xent_grad(x, w, ids, none, none, 0, MOST, grad_weight=gw)
    assert not gw.any()


def test_the_loss_of_the_largest_table():
    """In pieces, whose last one is ragged.  A tile's sum and 2^14 pairs joined one after
    another: (64 + 2^14 4) U at most."""
    w = torch.empty(MOST, 1, device="cuda", dtype=BF16)
    for c in w.split(1 << 28):
        c.copy_(torch.randn(c.shape, device="cuda"))
    x = torch.tensor([[1.0], [-0.5]], device="cuda", dtype=BF16)
    w[MOST - 1], w[12345] = 9.0, 11.0
    t = torch.tensor([MOST - 1, 12345], device="cuda")
    lse, at = vpe.vpe_lmhead_xent(x, w, t, 0, MOST)
    want = torch.zeros(2, dtype=torch.float64, device="cuda")
    for c in w.split(1 << 26):
        want += torch.exp(x.double() * c.double().T).sum(1)
    assert (lse.double() - want.log()).abs().max() <= (64 + 4 * 2 ** 14) * U
    assert at.tolist() == [9.0, -5.5]


@pytest.mark.parametrize("dtype,vocab,dim", [(F32, 16500, 8), (BF16, 16500, 8)],
                         ids=["f32", "bf16"])
def test_the_most_rows(dtype, vocab, dim):
    """2^21 rows against 16500: 2^35 logits, in three pieces of the table."""
    m = 1 << 21
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(m, dim, generator=g, device="cuda").to(dtype)
    w = torch.randn(vocab, dim, generator=g, device="cuda").to(dtype)
    t = torch.randint(0, vocab, (m,), generator=g, device="cuda", dtype=torch.int32)
    t[::17] = -1
    a, b = vpe.vpe_lmhead_xent(x, w, t, 0, vocab)
    loss, lse = vpe.vpe_xent_loss([a], [b], t, vocab)
    assert (loss[::17] == 0).all() and (lse[::17] == 0).all()
    pick = torch.cat([torch.arange(300, device="cuda"), torch.arange(m - 300, m, device="cuda"),
                      torch.randint(0, m, (3000,), generator=g, device="cuda")])
    pick = pick[t[pick] >= 0]
    z = x[pick].double() @ w.double().T
    size = (x[pick].double().abs() @ w.double().abs().T).max(1).values
    want = torch.logsumexp(z, 1)
    bound = (dim + 2) * U * size + 400 * U + 4 * U * want.abs()
    assert_within(lse[pick], want, bound, "lse")
    zt = torch.gather(z, 1, t[pick].long()[:, None])[:, 0]
    assert_within(loss[pick], want - zt, 2 * bound + 4 * U * zt.abs(), "loss")


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
