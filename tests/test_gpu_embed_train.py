"""The scaled lookup and the gradient of the lookup, through the public calls,
against their definitions in 64 bits.

Bounds.  The scaled lookup is one fp32 product and one rounding, repeated here
bit for bit.  A gradient row is a sum of c rows in fp32, times the factor,
rounded once: pieces of at most 32 rows are summed in turn and joined, so a
value goes through at most 31 + ceil(c / 32) additions, and
  |error| <= (32 + c / 32 + 3) 2^-24 |scale| sum |dy|  +  eps/2 |result|,
eps/2 the output type's half step.  Integer gradients below 2^24 are exact.
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


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ids(g, n, vocab, kind, itype):
    if kind == "uniform":
        ids = torch.randint(-3, vocab + 3, (n,), generator=g, device="cuda")
    elif kind == "one":
        ids = torch.full((n,), vocab // 2, device="cuda")
    elif kind == "none":
        ids = torch.full((n,), -1, device="cuda")
    elif kind == "runs":  # runs of every length from 1 up
        c = torch.arange(1, 400, device="cuda")
        ids = torch.repeat_interleave(c * 7 % vocab, c)[:n]
        ids = torch.cat([ids, torch.zeros(n - ids.numel(), dtype=ids.dtype, device="cuda")])
        ids = ids[torch.randperm(n, generator=g, device="cuda")]
    else:  # a few tokens take most of the positions
        ids = (torch.rand(n, generator=g, device="cuda") ** 8 * vocab).long()
    return ids.to(itype)


def _lookup(ids, weight, start, scale):
    local = ids.long() - start
    own = (local >= 0) & (local < weight.shape[0])
    y = weight[torch.where(own, local, 0)].float() * torch.tensor(scale, dtype=F32, device="cuda")
    return torch.where(own[:, None], y, 0.0).to(weight.dtype)


def _bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == BF16 else torch.int32)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("itype", [torch.int32, torch.int64])
@pytest.mark.parametrize("n,rows,dim,start", [
    (0, 10, 8, 0), (1, 1, 1, 0), (1, 7, 3, 2), (16, 100, 1024, 50), (255, 301, 64, 0),
    (33, 50, 1001, 7), (9, 20, 130, 1), (1000, 333, 2048, 100), (70, 40, 4096, 3),
    (5, 9, 10001, 0), (40, 30, 514, 12), (4100, 600, 12, 4),
])
def test_scaled_lookup(n, rows, dim, start, itype, dtype):
    g = _gen(n + rows + dim)
    weight = torch.randn(rows, dim, generator=g, device="cuda").to(dtype)
    ids = torch.randint(start - 5, start + rows + 5, (n,), generator=g, device="cuda").to(itype)
    for scale in (1.0, 32.0, 0.3, -2.75):
        got = vpe.vpe_embed_scaled(ids, weight, start, scale)
        assert torch.equal(_bits(got), _bits(_lookup(ids, weight, start, scale))), scale


def test_scaled_lookup_special_values_and_shapes():
    weight = torch.tensor([[float("inf"), -0.0, 1e38, float("nan")]], device="cuda")
    ids = torch.tensor([[0, 5], [-1, 0]], device="cuda")
    got = vpe.vpe_embed_scaled(ids, weight, 0, -10.0)
    assert got.shape == (2, 2, 4)
    assert got[0, 0, 0] == -float("inf") and got[0, 0, 2] == -float("inf")
    assert bool(torch.isnan(got[0, 0, 3])) and got[0, 0, 1] == 0
    assert torch.equal(_bits(got[0, 1]), torch.zeros(4, dtype=torch.int32, device="cuda"))
    assert torch.equal(_bits(got[1, 0]), torch.zeros(4, dtype=torch.int32, device="cuda"))


def test_scaled_lookup_unaligned_rows():
    # views that begin off a 16-byte boundary take narrower vectors
    base = torch.randn(40 * 24 + 8, device="cuda").to(BF16)
    ids = torch.arange(40, device="cuda")
    for shift in range(8):
        weight = base[shift:shift + 40 * 24].view(40, 24)
        out = torch.empty(40 * 24 + 8, dtype=BF16, device="cuda")[shift:shift + 40 * 24]
        got = vpe.vpe_embed_scaled(ids, weight, 0, 3.0, out=out.view(40, 24))
        assert torch.equal(_bits(got), _bits(_lookup(ids, weight, 0, 3.0)))


def test_scaled_lookup_past_two_gib():
    rows, dim = 1_100_000, 1024  # 2.25 GB of bf16
    weight = torch.empty(rows, dim, dtype=BF16, device="cuda")
    weight[:] = (torch.arange(rows, device="cuda") % 251)[:, None].to(BF16)
    ids = torch.tensor([0, rows - 1, 1_048_575, 1_048_576, 1_048_577], device="cuda")
    got = vpe.vpe_embed_scaled(ids, weight, 0, 2.0)
    assert torch.equal(got[:, 17].long(), ids % 251 * 2)


# ---------------------------------------------------------------------------
# gradient
# ---------------------------------------------------------------------------
def _grad_reference(ids, dy, start, rows):
    """(sum of the rows, sum of their absolute values, rows per token) in 64 bits."""
    local = ids.long().reshape(-1) - start
    own = (local >= 0) & (local < rows)
    at = local[own]
    x = dy.reshape(-1, dy.shape[-1])[own].double()
    total = torch.zeros(rows, x.shape[1], dtype=torch.float64, device="cuda")
    total.index_add_(0, at, x)
    size = torch.zeros_like(total).index_add_(0, at, x.abs())
    count = torch.zeros(rows, dtype=torch.float64, device="cuda").index_add_(
        0, at, torch.ones_like(at, dtype=torch.float64))
    return total, size, count


def _check_grad(got, ids, dy, start, rows, scale, before=None):
    total, size, count = _grad_reference(ids, dy, start, rows)
    ref = scale * total
    bound = (35 + count / 32)[:, None] * 2.0 ** -24 * abs(scale) * size
    if before is not None:
        ref = ref + before.double()
        bound = bound + 2.0 ** -23 * (before.double().abs() + abs(scale) * size)
    bound = bound + torch.finfo(got.dtype).eps / 2 * (ref.abs() + bound) + 1e-40
    err = (got.double() - ref).abs()
    assert bool((err <= bound).all()), float((err / bound).max())
    if before is None:
        empty = _bits(got)[count == 0]
        assert not bool(empty.any()), "rows without an id must be +0.0"
    else:
        assert torch.equal(_bits(got)[count == 0], _bits(before)[count == 0])


TYPES = [(F32, F32), (BF16, BF16), (BF16, F32), (F32, BF16)]


@pytest.mark.parametrize("dt,gdt", TYPES)
@pytest.mark.parametrize("n,rows,dim,kind", [
    (1, 1, 1, "uniform"), (1, 50, 8, "uniform"), (2, 3, 5, "one"), (31, 100, 64, "uniform"),
    (32, 9, 16, "one"), (33, 9, 16, "one"), (64, 9, 16, "one"), (65, 9, 24, "one"),
    (257, 2048, 64, "uniform"), (1000, 40, 1001, "few"), (1024, 513, 130, "uniform"),
    (1025, 600, 8, "few"), (3000, 700, 1024, "runs"), (8192, 300, 48, "runs"),
    (8193, 300, 48, "runs"), (8192, 5, 36, "one"), (12345, 75968, 12, "uniform"),
    (20000, 512, 40, "few"), (9000, 262145, 4, "uniform"), (30000, 3, 2050, "one"),
    (500, 64, 16, "none"), (10000, 64, 16, "none"), (40000, 100000, 24, "runs"),
])
def test_gradient(n, rows, dim, kind, dt, gdt):
    g = _gen(n + 3 * rows + dim)
    start = 11
    ids = _ids(g, n, rows, kind, torch.int32 if n % 2 else torch.int64)
    if kind != "none":
        ids = ids + start
    dy = torch.randn(n, dim, generator=g, device="cuda").to(dt)
    got = vpe.vpe_embed_grad(ids, dy, start, rows, 1.75, dtype=gdt)
    assert got.dtype == gdt
    _check_grad(got, ids, dy, start, rows, 1.75)
    # the same bits again, whatever the workspace held
    need = vpe.vpe_embed_grad_workspace(n, rows, dim)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    out = torch.full((rows, dim), float("nan"), dtype=gdt, device="cuda")
    vpe.vpe_embed_grad(ids, dy, start, rows, 1.75, grad_weight=out, workspace=ws)
    assert torch.equal(_bits(out), _bits(got))
    # added to what is there
    before = torch.randn(rows, dim, generator=g, device="cuda").to(gdt)
    acc = before.clone()
    vpe.vpe_embed_grad(ids, dy, start, rows, 1.75, grad_weight=acc, accumulate=True)
    _check_grad(acc, ids, dy, start, rows, 1.75, before=before)


@pytest.mark.parametrize("n", [7000, 50000, 300000])
def test_gradient_exact_on_integers(n):
    g = _gen(n)
    rows, dim = 1000, 16
    ids = _ids(g, n, rows, "few", torch.int64)
    dy = torch.randint(-8, 9, (n, dim), generator=g, device="cuda").to(BF16)
    total, _, _ = _grad_reference(ids, dy, 0, rows)
    got = vpe.vpe_embed_grad(ids, dy, 0, rows, dtype=F32)
    assert torch.equal(got.double(), total)


def test_gradient_ignores_rows_of_other_shards():
    g = _gen(1)
    n, rows, dim = 600, 64, 48
    ids = torch.randint(0, 4 * rows, (n,), generator=g, device="cuda")
    dy = torch.randn(n, dim, generator=g, device="cuda")
    ref = vpe.vpe_embed_grad(ids, dy, rows, rows)
    hurt = dy.clone()
    hurt[(ids < rows) | (ids >= 2 * rows)] = float("nan")
    assert torch.equal(_bits(vpe.vpe_embed_grad(ids, hurt, rows, rows)), _bits(ref))
    # an infinity stays in its own row
    hurt = dy.clone()
    hurt[(ids == rows).nonzero()[0, 0], 3] = float("inf")
    got = vpe.vpe_embed_grad(ids, hurt, rows, rows)
    assert got[0, 3] == float("inf")
    got[0, 3] = ref[0, 3]
    assert torch.equal(_bits(got), _bits(ref))


def test_gradient_of_nothing():
    ids = torch.empty(0, dtype=torch.int64, device="cuda")
    dy = torch.empty(0, 24, device="cuda")
    got = vpe.vpe_embed_grad(ids, dy, 0, 77)
    assert got.shape == (77, 24) and not bool(_bits(got).any())
    kept = torch.full((77, 24), 5.0, device="cuda")
    vpe.vpe_embed_grad(ids, dy, 0, 77, grad_weight=kept, accumulate=True)
    assert bool((kept == 5.0).all())


def test_gradient_unaligned_buffers():
    n, rows, dim = 300, 40, 24
    ids = torch.randint(0, rows, (n,), device="cuda")
    flat = torch.randn(n * dim + 8, device="cuda").to(BF16)
    for shift in range(0, 8, 3):
        dy = flat[shift:shift + n * dim].view(n, dim)
        for gdt in (BF16, F32):
            out = torch.empty(rows * dim + 8, dtype=gdt, device="cuda")
            out.fill_(9.0)
            dw = out[shift:shift + rows * dim].view(rows, dim)
            vpe.vpe_embed_grad(ids, dy, 0, rows, grad_weight=dw)
            _check_grad(dw, ids, dy, 0, rows, 1.0)
            assert bool((out[:shift] == 9).all()) and bool((out[shift + rows * dim:] == 9).all())


def test_gradient_matches_differences_of_the_lookup():
    # the lookup is linear in the table, so a difference is exact up to rounding
    g = _gen(5)
    n, rows, dim, start, scale = 40, 12, 6, 3, 2.5
    ids = torch.randint(0, 20, (n,), generator=g, device="cuda")
    weight = torch.randint(-4, 5, (rows, dim), generator=g, device="cuda").float()
    dy = torch.randint(-4, 5, (n, dim), generator=g, device="cuda").float()
    grad = vpe.vpe_embed_grad(ids, dy, start, rows, scale)
    base = (vpe.vpe_embed_scaled(ids, weight, start, scale) * dy).sum()
    for j, c in [(0, 0), (5, 3), (11, 5), (2, 4)]:
        moved = weight.clone()
        moved[j, c] += 1
        diff = (vpe.vpe_embed_scaled(ids, moved, start, scale) * dy).sum() - base
        assert float(diff) == float(grad[j, c])


def test_gradient_past_two_gib():
    # grad_out past byte 2^32 and a table shard past 2^31
    n, dim = 1_100_000, 2048
    dy = torch.zeros(n, dim, dtype=BF16, device="cuda")
    rows = 600_000
    ids = torch.full((n,), -1, dtype=torch.int64, device="cuda")
    ids[-1], ids[0], ids[n // 2] = rows - 1, rows - 1, 77
    dy[-1], dy[0], dy[n // 2] = 3.0, 5.0, 7.0
    got = vpe.vpe_embed_grad(ids, dy, 0, rows)
    assert bool((got[rows - 1] == 8).all()) and bool((got[77] == 7).all())
    got[rows - 1] = 0
    got[77] = 0
    assert not bool(got.any())


def test_gradient_captured_and_replayed():
    g = _gen(9)
    rows, dim = 500, 64
    for n in (400, 9000):
        ids = torch.randint(0, rows, (n,), generator=g, device="cuda")
        dy = torch.randn(n, dim, generator=g, device="cuda")
        out = torch.empty(rows, dim, device="cuda")
        ws = torch.empty(vpe.vpe_embed_grad_workspace(n, rows, dim), dtype=torch.uint8,
                         device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            vpe.vpe_embed_grad(ids, dy, 0, rows, 0.5, grad_weight=out, workspace=ws)
        for rep in range(3):
            ids.copy_(torch.randint(0, rows, (n,), generator=g, device="cuda"))
            dy.copy_(torch.randn(n, dim, generator=g, device="cuda"))
            out.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(_bits(out), _bits(vpe.vpe_embed_grad(ids, dy, 0, rows, 0.5)))


def test_two_streams_at_once():
    g = _gen(12)
    rows, dim, n = 3000, 256, 9000
    work = [(torch.randint(0, rows, (n,), generator=g, device="cuda"),
             torch.randn(n, dim, generator=g, device="cuda")) for _ in range(4)]
    ref = [vpe.vpe_embed_grad(i, d, 0, rows) for i, d in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    got = []
    for st, (i, d) in zip(streams, work):
        with torch.cuda.stream(st):
            got.append(vpe.vpe_embed_grad(i, d, 0, rows))
    torch.cuda.synchronize()
    for a, b in zip(got, ref):
        assert torch.equal(_bits(a), _bits(b))


def test_layer_weight_grad():
    emb = vpe.VocabParallelEmbedding(96, 32, tp_size=2, tp_rank=1, dtype=F32, device=dev())
    emb.weight.data.normal_()
    ids = torch.randint(0, 96, (4, 9), device="cuda")
    assert torch.equal(emb(ids, scale=2.0), vpe.vpe_embed_scaled(ids, emb.weight, 48, 2.0))
    assert torch.equal(emb(ids), vpe.vpe_embed(ids, emb.weight, 48))
    dy = torch.randn(4, 9, 32, device="cuda")
    got = emb.weight_grad(ids, dy, scale=2.0)
    assert torch.equal(got, vpe.vpe_embed_grad(ids, dy, 48, 48, 2.0))
    twice = emb.weight_grad(ids, dy, scale=2.0, grad_weight=got.clone(), accumulate=True)
    _check_grad(twice, ids, dy, 48, 48, 2.0, before=got)


def test_more_rows_than_one_launch_takes():
    n = 2 ** 24 + 5  # of the lookup; then runs of 13107 chunks, 70 GB of rows
    weight = torch.arange(7, device="cuda", dtype=F32)[:, None].contiguous()
    ids = torch.arange(n, device="cuda") % 9
    got = vpe.vpe_embed_scaled(ids, weight, 0, 3.0)
    assert torch.equal(got[:, 0], torch.where(ids < 7, ids * 3.0, 0.0))
    n, dim, rows = 2 ** 21, 16640, 4
    if torch.cuda.mem_get_info()[0] < 110e9:
        pytest.skip("needs 110 GB of device memory")
    ids = torch.arange(n, device="cuda") * (rows + 1) // n  # 5 long runs, the last one's unowned
    dy = torch.ones(n, dim, dtype=BF16, device="cuda")
    dy[0], dy[-1] = 3.0, float("nan")
    got = vpe.vpe_embed_grad(ids, dy, 0, rows, 0.5, dtype=F32)
    count = torch.bincount(ids, minlength=rows + 1)[:rows].float()  # exact sums below 2^24
    count[0] += 2
    assert torch.equal(got, (0.5 * count)[:, None].expand(rows, dim))


@pytest.mark.parametrize("n,rows,dim", [(300, 2 ** 28 + 3, 1), (9001, 2 ** 28 + 3, 1),
                                        (70, 6, 2 ** 20), (9000, 700, 2 ** 15 + 1)])
def test_gradient_of_many_rows_and_of_wide_ones(n, rows, dim):
    g = _gen(n)
    ids = torch.randint(0, rows, (n,), generator=g, device="cuda")
    ids[:3] = rows - 1
    dy = torch.randint(-8, 9, (n, dim), generator=g, device="cuda").to(BF16)
    got = vpe.vpe_embed_grad(ids, dy, 0, rows, 0.5, dtype=F32)
    ref = torch.zeros(rows, dim, device="cuda").index_add_(0, ids, dy.float() * 0.5)  # exact
    assert torch.equal(got, ref)
    vpe.vpe_embed_grad(ids, dy, 0, rows, 0.5, grad_weight=got, accumulate=True)
    assert torch.equal(got, 2 * ref)
