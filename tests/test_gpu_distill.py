"""Distillation from a teacher's top logits, through the public calls, against
the definition in 64 bits.

Bounds, u = 2^-24 (the half step of fp32).  A power of two is taken at an
argument that carries at most 3 roundings of its parts (the factor
log2(e) / T, the product's fma, the stored offset), so its relative error is at
most 3 u |argument| + 4 u.  With A the largest |z / T|:
  lse   u |lse| + (6 A + cols / 256 + 64) u   (sums: one thread's share, then joins)
  p_e   rp = (8 max |t / T| + 8 max |teacher_lse| + k / 64 + 32) u, relative
  loss  (rp + (k / 64 + 40) u) (sum p |z / T| + sum p |log p| + P |lse|) + P d(lse)
  grad  |g| / T (P q (6 (|z / T| + |lse|) + 16) u + sum p (rp + 8 u)), and the output
        type's half step of the result (2^-126 below which fp32 powers vanish)
"""
import pytest

torch = pytest.importorskip("torch")

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a HIP GPU"),
]

import vocab_sharded_embedding_amd as vpe  # noqa: E402
from _gpu import dev  # noqa: E402

F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24
INF = float("inf")


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _definition(z, ids, t, temp, tail=None, lse=None):
    """(loss, lse, dloss/dz, and the sizes the bounds need) in 64 bits; z: the whole rows."""
    m, v = z.shape
    z = z.double() / temp
    valid = (ids >= 0) & (ids < v)
    t = torch.where(valid, t.double() / temp, -INF)
    norm = torch.logsumexp(t, 1, keepdim=True) if tail is None else tail.double()[:, None]
    p = torch.where(torch.isneginf(t), 0.0, torch.exp(t - norm))
    lse = torch.logsumexp(z, 1) if lse is None else lse.double()
    at = torch.where(valid, ids.long(), 0)
    zk = torch.gather(z, 1, at)
    on = p != 0
    logp = torch.where(on, t - norm, 0.0)
    loss = torch.where(on, p * (logp - zk + lse[:, None]), 0.0).sum(1)
    mass = p.sum(1)
    q = mass[:, None] * torch.exp(z - lse[:, None])
    ps = torch.zeros_like(z).scatter_add_(1, at, p)
    grad = (q - ps) / temp
    empty = ~on.any(1)
    loss[empty] = 0
    grad[empty] = 0
    size = torch.where(on, p * (zk.abs() + logp.abs()), 0.0).sum(1) + mass * lse.abs()
    t_most = torch.where(torch.isfinite(t), t.abs(), 0.0).max()
    return loss, lse, grad, dict(q=q, ps=ps, z=z, mass=mass, size=size, t_most=t_most)


def _case(seed, m, v, k, dtype, tdt, itype, tail=False, ragged=True):
    g = _gen(seed)
    z = 3.0 * torch.randn(m, v, generator=g, device="cuda")
    base = torch.randint(0, v, (m, 1), generator=g, device="cuda")
    step = torch.randint(1, max(2, v // max(k, 1)), (m, 1), generator=g, device="cuda")
    ids = (base + step * torch.arange(k, device="cuda")) % v
    t = 4.0 + 2.0 * torch.randn(m, k, generator=g, device="cuda")
    z.scatter_(1, ids, t + torch.randn(m, k, generator=g, device="cuda")) if k <= v else None
    if ragged:
        count = torch.randint(0, k + 1, (m,), generator=g, device="cuda")
        count[0] = k
        pad = torch.tensor([-1, v, 2 ** 31 - 1, -2 ** 31], device="cuda")[
            torch.randint(0, 4, (m, k), generator=g, device="cuda")]
        ids = torch.where(torch.arange(k, device="cuda") < count[:, None], ids, pad)
    t = t.to(tdt)
    tl = None
    if tail:
        kept = torch.where((ids >= 0) & (ids < v), t.float(), -INF)
        tl = torch.logsumexp(kept, 1) + 0.25
    return z.to(dtype), ids.to(itype), t, tl, g


def _shards(z, ids, t, tl, temp, tp):
    m, v = z.shape
    rows = v // tp
    return [vpe.vpe_distill_shard(z, ids, t, r * rows, v, temperature=temp, teacher_lse=tl,
                                  shard_rows=rows, col_offset=r * rows) for r in range(tp)]


def _check(z, ids, t, tl, temp, tp, g, k):
    m, v = z.shape
    rows = v // tp
    parts = _shards(z, ids, t, tl, temp, tp)
    loss, lse = vpe.vpe_distill_loss([a for a, _ in parts], [b for _, b in parts], ids, t, v,
                                     temperature=temp, teacher_lse=tl)
    rloss, rlse, rgrad, s = _definition(z, ids, t, temp, tl)
    big = s["z"].abs().amax(1)
    d_lse = U * rlse.abs() * (1 + tp) + (6 * big + rows / 256 + 64 + 8 * tp) * U
    assert bool(((lse.double() - rlse).abs() <= d_lse).all())
    # a row without entries has a log-sum-exp of -inf, and no p_e
    tl_most = 0 if tl is None else torch.where(torch.isfinite(tl), tl.abs(), 0.0).max()
    rp = (8 * s["t_most"] + 8 * tl_most + k / 64 + 32) * U
    d_loss = (rp + (k / 64 + 40) * U) * s["size"] + s["mass"] * d_lse
    err = (loss.double() - rloss).abs()
    assert bool((err <= d_loss).all()), float((err / d_loss.clamp(min=1e-300)).max())

    go = torch.randn(m, generator=g, device="cuda")
    if m > 2:
        go[1] = 0.0
    out = torch.full_like(z, float("nan"))
    for r in range(tp):
        vpe.vpe_distill_grad(z, lse, go, ids, t, r * rows, v, temperature=temp, teacher_lse=tl,
                             shard_rows=rows, col_offset=r * rows, grad_logits=out)
    _, _, rgrad, s = _definition(z, ids, t, temp, tl, lse=lse)
    ref = rgrad * go.double()[:, None]
    bound = (go.double().abs() / temp)[:, None] * (
        s["q"] * (6 * (s["z"].abs() + rlse.abs()[:, None]) + 16) * U + (s["q"] + s["ps"]) * rp
        + s["ps"] * 8 * U)
    bound = bound + torch.finfo(z.dtype).eps / 2 * (ref.abs() + bound) + 2.0 ** -126
    err = (out.double() - ref).abs()
    assert bool((err <= bound).all()), float((err / bound).max())
    # in place, and a shard alone in its own buffer, give the same bits
    again = z.clone()
    for r in range(tp):
        vpe.vpe_distill_grad(again, lse, go, ids, t, r * rows, v, temperature=temp, teacher_lse=tl,
                             shard_rows=rows, col_offset=r * rows, grad_logits=again)
    view = torch.int16 if z.dtype == BF16 else torch.int32
    assert torch.equal(again.view(view), out.view(view))
    last = z[:, (tp - 1) * rows:].contiguous()
    alone = vpe.vpe_distill_grad(last, lse, go, ids, t, (tp - 1) * rows, v, temperature=temp,
                                 teacher_lse=tl)
    assert torch.equal(alone.view(view), out[:, (tp - 1) * rows:].contiguous().view(view))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,v,k,tp,temp,tail", [
    (1, 1, 1, 1, 1.0, False), (1, 7, 3, 1, 2.0, False), (3, 40, 40, 1, 0.5, True),
    (5, 257, 17, 1, 1.0, True), (4, 2048, 64, 2, 2.0, False), (2, 8195, 20, 1, 1.0, False),
    (9, 30003, 100, 3, 3.0, False), (33, 4100, 255, 4, 1.5, True), (2, 151936, 1024, 1, 1.0, False),
    (1, 151936, 50, 2, 2.0, True), (300, 1001, 5, 1, 1.0, False), (2100, 260, 257, 2, 0.7, False),
])
def test_loss_and_gradient(m, v, k, tp, temp, tail, dtype):
    tdt = BF16 if (m + k) % 2 else F32
    itype = torch.int32 if (v + k) % 2 else torch.int64
    z, ids, t, tl, g = _case(m + v + k, m, v, k, dtype, tdt, itype, tail)
    _check(z, ids, t, tl, temp, tp, g, k)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,v,k,tp", [(256, 50001, 33, 1), (257, 9001, 7, 1), (3, 70003, 9, 1),
                                      (3, 140006, 9, 2), (40, 120001, 65, 1), (1, 41000, 2, 1),
                                      (1, 82000, 2, 1)])
def test_few_and_many_rows_of_many_slices(m, v, k, tp, dtype):
    # the statistics take a workgroup per row, or cut few long rows over the chip
    z, ids, t, tl, g = _case(m + v, m, v, k, dtype, F32, torch.int32, tail=bool(k % 2))
    _check(z, ids, t, tl, 1.5, tp, g, k)


@pytest.mark.parametrize("col,extra", [(0, 5), (1, 0), (3, 2), (8, 8), (13, 1)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strided_rows_and_untouched_columns(col, extra, dtype):
    m, rows, k = 6, 1003, 11
    z, ids, t, _, g = _case(77, m, rows, k, dtype, F32, torch.int64)
    ld = col + rows + extra
    wide = torch.full((m, ld), float("nan"), dtype=dtype, device="cuda")
    wide[:, col:col + rows] = z
    ref = vpe.vpe_distill_shard(z, ids, t, 0, rows)
    got = vpe.vpe_distill_shard(wide, ids, t, 0, rows, shard_rows=rows, col_offset=col)
    # slices and vectors fall alike, so the bits do
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    go = torch.ones(m, device="cuda")
    out = torch.full((m, ld + 3), 7.0, dtype=dtype, device="cuda")
    vpe.vpe_distill_grad(wide, ref[0], go, ids, t, 0, rows, shard_rows=rows, col_offset=col,
                         grad_logits=out, grad_col_offset=col + 2)
    alone = vpe.vpe_distill_grad(z, ref[0], go, ids, t, 0, rows)
    assert torch.equal(out[:, col + 2:col + 2 + rows], alone)
    assert bool((out[:, :col + 2] == 7).all()) and bool((out[:, col + 2 + rows:] == 7).all())


@pytest.mark.parametrize("k", [2, 3, 64, 300, 1024])
def test_ids_that_occur_more_than_once(k):
    m, v = 8, 500
    g = _gen(k)
    z = torch.randn(m, v, generator=g, device="cuda")
    ids = torch.randint(0, 40, (m, k), generator=g, device="cuda") * 9
    ids[0] = 123  # one id, k times
    t = torch.randn(m, k, generator=g, device="cuda")
    _check(z, ids, t, None, 1.0, 1, g, k)
    _check(z.to(BF16), ids, t, None, 1.0, 2, g, k)
    # columns that collide in a table of 8192 entries, far apart
    z = torch.randn(m, 30000, generator=g, device="cuda")
    ids = torch.randint(0, 3, (m, k), generator=g, device="cuda") * 8192 + 5
    _check(z, ids, t, None, 1.0, 1, g, k)


def test_rows_without_entries_whatever_they_hold():
    m, v, k = 5, 3000, 4
    z = torch.randn(m, v, device="cuda")
    z[1] = float("nan")
    z[2] = -INF
    z[3] = INF
    ids = torch.tensor([[-1, v, -7, 2 ** 31 - 1]] * m, device="cuda")
    ids[0] = torch.tensor([3, 5, -1, 9], device="cuda")
    t = torch.randn(m, k, device="cuda")
    t[1] = float("nan")  # padding's logits are not looked at
    ids[4] = torch.tensor([1, 2, 3, 4], device="cuda")
    t[4] = -INF          # entries of no probability
    for tl in (None, torch.tensor([1.0, -INF, 0.0, INF, 2.0], device="cuda")):
        lse, dot = vpe.vpe_distill_shard(z, ids, t, 0, v, teacher_lse=tl)
        loss, _ = vpe.vpe_distill_loss([lse], [dot], ids, t, v, teacher_lse=tl)
        assert bool((loss[1:] == 0).all()) and bool((dot[1:] == 0).all()) and float(loss[0]) != 0
        grad = vpe.vpe_distill_grad(z, lse, torch.ones(m, device="cuda"), ids, t, 0, v,
                                    teacher_lse=tl)
        assert not bool(grad[1:].view(torch.int32).any())
        assert bool(torch.isfinite(grad[0]).all())
    # a gradient of 0 for the row's loss: zeros, the logits are not read
    grad = vpe.vpe_distill_grad(z, lse, torch.zeros(m, device="cuda"), ids, t, 0, v)
    assert not bool(grad.view(torch.int32).any())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("low", [-INF, "lowest"])
def test_masked_columns(low, dtype):
    m, v, k = 4, 20000, 30
    z, ids, t, _, g = _case(3, m, v, k, dtype, F32, torch.int64, ragged=False)
    low = torch.finfo(dtype).min if low == "lowest" else low
    masked = torch.rand(m, v, generator=g, device="cuda") < 0.7
    masked[2] = True
    masked.scatter_(1, ids, False)  # the teacher's own tokens stay
    z[masked] = low
    z[3, :8192] = low  # whole slices of a row
    ids[3] = 8192 + torch.arange(k, device="cuda") * 30
    z[3, ids[3]] = 1.0
    lse, dot = vpe.vpe_distill_shard(z, ids, t, 0, v)
    loss, full = vpe.vpe_distill_loss([lse], [dot], ids, t, v)
    rloss, rlse, rgrad, s = _definition(z, ids, t, 1.0)
    # the masked columns add nothing; the bounds of the finite ones hold
    assert bool(((full.double() - rlse).abs() <= U * rlse.abs() + (6 * 20 + v / 256 + 64) * U).all())
    assert bool(((loss.double() - rloss).abs() <= 2e-5 * (1 + s["size"])).all())
    grad = vpe.vpe_distill_grad(z, full, torch.ones(m, device="cuda"), ids, t, 0, v)
    rest = masked & (z == low)
    assert not bool(grad[rest].any())
    assert bool(torch.isfinite(grad).all())


def test_infinite_and_nan_values_follow_the_formulas():
    v, k = 9000, 3
    z = torch.randn(4, v, device="cuda")
    ids = torch.tensor([[1, 2, 3]] * 4, device="cuda")
    t = torch.zeros(4, k, device="cuda")
    z[0, 2] = -INF      # the teacher wants a token that the student excludes
    z[1, 8999] = float("nan")
    z[2] = -INF         # nothing left: log 0 / 0
    lse, dot = vpe.vpe_distill_shard(z, ids, t, 0, v)
    loss, full = vpe.vpe_distill_loss([lse], [dot], ids, t, v)
    assert float(loss[0]) == INF and bool(torch.isnan(loss[1])) and bool(torch.isnan(loss[2]))
    assert bool(torch.isfinite(loss[3]))
    assert float(full[2]) == -INF and bool(torch.isnan(full[1]))
    grad = vpe.vpe_distill_grad(z, full, torch.ones(4, device="cuda"), ids, t, 0, v)
    assert bool(torch.isfinite(grad[0]).all()) and abs(float(grad[0, 2]) + 1 / 3) < 1e-6
    assert bool(torch.isnan(grad[1]).all()) and bool(torch.isfinite(grad[3]).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("temp", [1.0, 2.0])
def test_shards_that_hold_the_lowest_value_only(temp, dtype):
    # row 0: all of one shard of two; row 1: everything, where 64 bits give a
    # log-sum-exp whose nearest fp32 value is lowest / T, and exp(z / T - that) = 1
    m, v, k = 3, 6000, 4
    low = torch.finfo(dtype).min
    z = torch.randn(m, v, generator=_gen(9), device="cuda").to(dtype)
    z[0, v // 2:] = low
    z[1] = low
    ids = torch.tensor([[5, 17, 100, 1000]] * m, device="cuda")
    t = torch.zeros(m, k, device="cuda")
    parts = _shards(z, ids, t, None, temp, 2)
    loss, full = vpe.vpe_distill_loss([a for a, _ in parts], [b for _, b in parts], ids, t, v,
                                      temperature=temp)
    assert float(parts[1][0][0]) == low / temp and float(parts[0][0][1]) == low / temp
    _, rlse, rgrad, _ = _definition(z, ids, t, temp, lse=full)
    assert float(full[1]) == low / temp and bool(torch.isfinite(loss).all())
    grad = vpe.vpe_distill_grad(z, full, torch.ones(m, device="cuda"), ids, t, 0, v,
                                temperature=temp)
    # q and p are at most 1 here; |z / T| and |lse| at most 16 where they enter the bound
    bound = (6 * 32 + 16 + 32 + 8) * U + torch.finfo(dtype).eps / 2 * rgrad.abs()
    assert bool(((grad.double() - rgrad).abs() <= bound).all())
    assert bool((grad[0, v // 2:] == 0).all())


def test_rows_that_hold_plus_infinity():
    m, v, k = 3, 9000, 2
    z = torch.randn(m, v, generator=_gen(10), device="cuda")
    z[0, 8998] = INF    # not the teacher's: excluded by the student for good
    z[1, [7, 6000]] = INF
    ids = torch.tensor([[1, 7]] * m, device="cuda")
    t = torch.zeros(m, k, device="cuda")
    for tp in (1, 2):
        parts = _shards(z, ids, t, None, 1.5, tp)
        loss, full = vpe.vpe_distill_loss([a for a, _ in parts], [b for _, b in parts], ids, t, v,
                                          temperature=1.5)
        assert full.tolist()[:2] == [INF, INF] and bool(torch.isfinite(full[2]))
        assert float(loss[0]) == INF and bool(torch.isnan(loss[1]))  # inf - inf
        grad = vpe.vpe_distill_grad(z, full, torch.ones(m, device="cuda"), ids, t, 0, v,
                                    temperature=1.5)
        nan = torch.zeros_like(z, dtype=torch.bool)
        nan[0, 8998] = nan[1, 7] = nan[1, 6000] = True
        assert torch.equal(torch.isnan(grad), nan)
        p = (grad[0] * 1.5)[[1, 7]] + 0.5
        assert bool((p.abs() <= 8 * U).all())


def test_shard_lse_of_the_lm_head_can_be_used():
    g = _gen(21)
    m, v, d, k, tp = 17, 512, 64, 9, 2
    rows = v // tp
    x = torch.randn(m, d, generator=g, device="cuda").to(BF16)
    w = torch.randn(v, d, generator=g, device="cuda").to(BF16) * 0.2
    ids = torch.randint(0, v, (m, k), generator=g, device="cuda")
    t = torch.randn(m, k, generator=g, device="cuda")
    logits = torch.empty(m, v, dtype=BF16, device="cuda")
    a, b = [], []
    for r in range(tp):
        _, lse = vpe.vpe_lmhead_logsumexp(x, w[r * rows:(r + 1) * rows], logits,
                                          col_offset=r * rows)
        none, dot = vpe.vpe_distill_shard(logits, ids, t, r * rows, v, shard_rows=rows,
                                          col_offset=r * rows, with_lse=False)
        assert none is None
        a.append(lse)
        b.append(dot)
    loss, lse = vpe.vpe_distill_loss(a, b, ids, t, v)
    parts = _shards(logits, ids, t, None, 1.0, tp)
    other, _ = vpe.vpe_distill_loss([p for p, _ in parts], [q for _, q in parts], ids, t, v)
    for (_, q), mine in zip(parts, b):
        assert torch.equal(q, mine)
    assert bool(((loss - other).abs() <= 1e-4).all())


def test_gradient_matches_differences_of_the_loss():
    # central differences of the 64-bit loss: error h^2 |f'''| / 6, |f'''| <= 1
    g = _gen(31)
    m, v, k, temp, h = 3, 50, 6, 1.5, 1e-3
    z = torch.randn(m, v, generator=g, device="cuda")
    ids = torch.randint(0, v, (m, k), generator=g, device="cuda")
    t = torch.randn(m, k, generator=g, device="cuda")
    lse, dot = vpe.vpe_distill_shard(z, ids, t, 0, v, temperature=temp)
    _, full = vpe.vpe_distill_loss([lse], [dot], ids, t, v, temperature=temp)
    grad = vpe.vpe_distill_grad(z, full, torch.ones(m, device="cuda"), ids, t, 0, v,
                                temperature=temp)
    for j in list(range(0, v, 7)) + ids[0].tolist():
        up, down = z.double().clone(), z.double().clone()
        up[:, j] += h
        down[:, j] -= h
        diff = (_definition(up, ids, t, temp)[0] - _definition(down, ids, t, temp)[0]) / (2 * h)
        assert bool(((grad[:, j].double() - diff).abs() <= h * h + 2e-6).all())


def test_rows_past_two_gib():
    # rows of 2.4 GB, so row 2 begins past byte 2^32
    m, rows, ld = 3, 5000, 1_200_000_000
    wide = torch.empty(m * ld, dtype=BF16, device="cuda").view(m, ld)
    g = _gen(41)
    z = torch.randn(m, rows, generator=g, device="cuda").to(BF16)
    wide[:, ld - rows:] = z
    ids = torch.randint(0, rows, (m, 8), generator=g, device="cuda")
    t = torch.randn(m, 8, generator=g, device="cuda")
    a = vpe.vpe_distill_shard(wide, ids, t, 0, rows, shard_rows=rows, col_offset=ld - rows)
    b = vpe.vpe_distill_shard(z, ids, t, 0, rows)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    go = torch.ones(m, device="cuda")
    vpe.vpe_distill_grad(wide, a[0], go, ids, t, 0, rows, shard_rows=rows, col_offset=ld - rows,
                         grad_logits=wide)
    assert torch.equal(wide[:, ld - rows:], vpe.vpe_distill_grad(z, a[0], go, ids, t, 0, rows))


def test_no_rows():
    z = torch.empty(0, 100, device="cuda")
    ids, t = torch.empty(0, 4, dtype=torch.int64, device="cuda"), torch.empty(0, 4, device="cuda")
    lse, dot = vpe.vpe_distill_shard(z, ids, t, 0, 100)
    loss, full = vpe.vpe_distill_loss([lse], [dot], ids, t, 100)
    grad = vpe.vpe_distill_grad(z, full, loss, ids, t, 0, 100)
    assert loss.numel() == 0 and grad.shape == (0, 100)


def test_training_step_captured_and_replayed():
    """Lookup, LM head, loss, gradients of the logits and of the tied table: as one
    captured step, replayed against the eager step."""
    g = _gen(51)
    V, D, tp, n, k = 640, 64, 2, 48, 8
    rows, scale, temp = V // tp, 8.0, 2.0
    table = [(torch.randn(rows, D, generator=g, device="cuda") * 0.1).to(BF16) for _ in range(tp)]
    ids = torch.randint(0, V, (n,), generator=g, device="cuda")
    t_ids = torch.randint(-1, V, (n, k), generator=g, device="cuda")
    t = torch.randn(n, k, generator=g, device="cuda")
    go = torch.full((n,), temp * temp / n, device="cuda")

    def step():
        x = vpe.vpe_sum_partials([vpe.vpe_embed_scaled(ids, table[r], r * rows, scale)
                                  for r in range(tp)])
        logits = torch.empty(n, V, dtype=BF16, device="cuda")
        for r in range(tp):
            vpe.vpe_lmhead(x, table[r], logits, col_offset=r * rows)
        parts = _shards(logits, t_ids, t, None, temp, tp)
        loss, lse = vpe.vpe_distill_loss([a for a, _ in parts], [b for _, b in parts], t_ids, t,
                                         V, temperature=temp)
        dz = [vpe.vpe_distill_grad(logits, lse, go, t_ids, t, r * rows, V, temperature=temp,
                                   shard_rows=rows, col_offset=r * rows) for r in range(tp)]
        dx = sum(dz[r].float() @ table[r].float() for r in range(tp)).to(BF16)
        dw = []
        for r in range(tp):
            d = (dz[r].float().t().contiguous() @ x.float()).contiguous()  # the LM head's part
            dw.append(vpe.vpe_embed_grad(ids, dx, r * rows, rows, scale, grad_weight=d,
                                         accumulate=True))
        return loss, dx, dw

    # the table's gradient against autograd over the whole table in 64 bits
    w = torch.cat(table).double().requires_grad_()
    x = (w[ids] * scale)
    x = x + (x.to(BF16).double() - x).detach()
    z = x @ w.t()
    z = z + (z.to(BF16).double() - z).detach()
    valid = t_ids >= 0
    p = torch.softmax(torch.where(valid, t.double() / temp, -INF), 1)
    logq = torch.log_softmax(z / temp, 1)
    per_row = torch.where(p > 0, p * (torch.log(p.clamp(min=1e-300))
                                      - torch.gather(logq, 1, t_ids.clamp(min=0))), 0.0).sum(1)
    (per_row * go.double()).sum().backward()
    loss, dx, dw = step()
    assert bool(((loss.double() - per_row.detach()).abs() <= 1e-2).all())
    got, ref = torch.cat(dw).double(), w.grad
    # bf16 logits gradients and bf16 dx: each term is off by at most 2^-8 of its size
    assert float((got - ref).abs().max()) <= 2.0 ** -6 * float(ref.abs().max())

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for rep in range(3):
        ids.copy_(torch.randint(0, V, (n,), generator=g, device="cuda"))
        t.copy_(torch.randn(n, k, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        eager = step()
        assert torch.equal(held[0], eager[0]) and torch.equal(held[1], eager[1])
        for a, b in zip(held[2], eager[2]):
            assert torch.equal(a, b)


def test_layer_distillation():
    V, D, tp, m, k = 512, 64, 2, 9, 5
    g = _gen(61)
    heads = [vpe.ParallelLMHead(V, D, tp, r, device=dev()) for r in range(tp)]
    for h in heads:
        h.weight.data.copy_((torch.randn(V // tp, D, generator=g, device="cuda") * 0.1).to(BF16))
    x = torch.randn(m, D, generator=g, device="cuda").to(BF16)
    ids = torch.randint(0, V, (m, k), generator=g, device="cuda")
    t = torch.randn(m, k, generator=g, device="cuda")
    full = torch.empty(m, V, dtype=BF16, device="cuda")
    own = [h(x) for h in heads]
    for h in heads:
        h(x, logits=full)
    one = [h.distill_shard(z, ids, t, temperature=2.0) for h, z in zip(heads, own)]
    two = [h.distill_shard(full, ids, t, temperature=2.0) for h in heads]
    for a, b in zip(one, two):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    loss, lse = heads[0].distill_loss([a for a, _ in one], [b for _, b in one], ids, t,
                                      temperature=2.0)
    ref = vpe.vpe_distill_loss([a for a, _ in one], [b for _, b in one], ids, t, V,
                               temperature=2.0)
    assert torch.equal(loss, ref[0]) and torch.equal(lse, ref[1])
    go = torch.rand(m, generator=g, device="cuda")
    for h, z in zip(heads, own):
        a = h.distill_grad(z, lse, go, ids, t, temperature=2.0)
        s = h.vocab_start_idx
        b = h.distill_grad(full, lse, go, ids, t, temperature=2.0)
        assert torch.equal(a, b) and a.shape == (m, V // tp)
        assert torch.equal(a, vpe.vpe_distill_grad(z, lse, go, ids, t, s, V, temperature=2.0))
        with pytest.raises(ValueError):
            h.distill_grad(z[:, :-1].contiguous(), lse, go, ids, t)


def test_the_most_rows():
    m, v, k = 2 ** 21, 3, 2
    z, ids, t, tl, g = _case(61, m, v, k, F32, F32, torch.int32)
    _check(z, ids, t, tl, 1.0, 1, g, k)


def test_two_streams_at_once():
    v, k = 5000, 12
    work = [_case(70 + i, m, v, k, BF16, F32, torch.int64)[:3]
            for i, m in enumerate((3, 300, 40, 257))]

    def step(z, ids, t):
        lse, dot = vpe.vpe_distill_shard(z, ids, t, 0, v)
        loss, lse = vpe.vpe_distill_loss([lse], [dot], ids, t, v)
        return loss, vpe.vpe_distill_grad(z, lse, torch.ones_like(loss), ids, t, 0, v)

    ref = [step(*w) for w in work]
    streams = [torch.cuda.Stream() for _ in work]
    torch.cuda.synchronize()
    got = []
    for st, w in zip(streams, work):
        with torch.cuda.stream(st):
            got.append(step(*w))
    torch.cuda.synchronize()
    for a, b in zip(got, ref):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
