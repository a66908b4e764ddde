"""The gradient of a lookup in which one token holds most positions, with values
of one sign that fp32 sums do not hold exactly, against the sum in 64 bits.

Bound, u = 2^-24.  A piece of at most 32 sorted rows is summed in turn: at most
31 additions, each off by at most u of a partial sum that, all values having one
sign, is no larger than the whole.  The pieces of a run are joined in 64 bits
(at most 2^26 of them: 2^-27 of the sum, less than u / 8) and rounded to fp32
once; a run of fewer than 17 pieces may also be joined in fp32.  The factor and
the output's rounding follow.  So
  |error| <= (31 + 16 + 1 + 1) u |scale| sum |dy|  +  eps/2 |result|
however many positions the token has (with accumulate one addition more).
"""
import pytest

torch = pytest.importorskip("torch")

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a HIP GPU"),
]

import vocab_sharded_embedding_amd as vpe  # noqa: E402

F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24


@pytest.mark.parametrize("gdt", [F32, BF16])
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("n,dim,vary", [
    (500, 24, True), (4000, 24, True), (8192, 36, False), (12345, 260, True), (65536, 8, False),
    (131072, 64, True), (131072, 5, False), (2 ** 21 + 77, 8, False), (2 ** 21, 4, True),
])
def test_one_sign_sums_of_long_runs(n, dim, vary, dt, gdt):
    g = torch.Generator(device="cuda").manual_seed(n + dim)
    rows, token, scale = 9, 4, 1.3
    ids = torch.full((n,), token, device="cuda")
    ids[torch.randint(0, n, (5,), generator=g, device="cuda")] = 7
    dy = torch.full((n, dim), 0.7, device="cuda")
    if vary:
        dy = dy + 0.5 * torch.rand(n, dim, generator=g, device="cuda")
    dy = dy.to(dt)
    total = torch.zeros(rows, dim, dtype=torch.float64, device="cuda")
    for t in (token, 7):
        total[t] = dy[ids == t].double().sum(0)
    scale32 = float(torch.tensor(scale, dtype=F32))
    ref = scale32 * total
    got = vpe.vpe_embed_grad(ids, dy, 0, rows, scale, dtype=gdt)
    half = torch.finfo(gdt).eps / 2
    bound = 49 * U * ref.abs()
    bound = bound + half * (ref.abs() + bound)
    err = (got.double() - ref).abs()
    assert bool((err <= bound).all()), float((err / ref.abs().clamp(min=1e-9)).max())
    before = (torch.rand(rows, dim, generator=g, device="cuda") * n).to(gdt)
    acc = before.clone()
    vpe.vpe_embed_grad(ids, dy, 0, rows, scale, grad_weight=acc, accumulate=True)
    ref = ref + before.double()
    bound = 50 * U * ref.abs()
    bound = bound + half * (ref.abs() + bound)
    err = (acc.double() - ref).abs()
    assert bool((err <= bound).all()), float((err / ref.abs().clamp(min=1e-9)).max())
