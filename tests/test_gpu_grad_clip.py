"""Global gradient norm and clipping on the GPU against the formulas in 64 bits.

sumsq: products and sums in fp64, a rounding per element at most, u = 2^-53: over
n elements n u of the sum.  norm: its root, and one rounding to fp32.  The factor
carries the roundings of the sum, the root, the sum with 1e-6, the quotient and
the one to fp32; the product one in fp32 and one to the tensor's type."""
import math

import pytest
import torch

import vocab_sharded_embedding_amd as vpe
from _loss import HALF, U

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def _grads(sizes, seed, scale=1e-2, types=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * scale).to(
        types[i] if types else (BF16 if i % 3 else F32)) for i, n in enumerate(sizes)]


def _sumsq(tensors):
    return math.fsum(float((t.double() ** 2).sum()) for t in tensors)


def _check(tensors, got, sums, max_norm, norm):
    n = sum(t.numel() for t in tensors)
    want = math.sqrt(math.fsum(sums))
    assert abs(norm.item() - want) <= want * (U * 1.001 + n * 2.0 ** -53) + 1e-45
    f = min(1.0, max_norm / (want + 1e-6))
    for t, o in zip(tensors, got):
        ref = t.double() * f
        bound = ref.abs() * (HALF[t.dtype] + 2 * U + (n + 8) * 2.0 ** -53) * 1.01 + 2.0 ** -133
        assert o.dtype == t.dtype and bool(((o.double() - ref).abs() <= bound).all())


SIZES = [[1], [5], [255, 256, 257], [1, 0, 2, 3], [16384], [16385, 7], [100003, 1, 33, 4096],
         [2048 * 9 + 1] * 7, [3] * 97, [11 * (i % 13) + 1 for i in range(400)],
         [5_000_001, 12, 70_000_003]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("clips", [True, False])
def test_norm_and_clip(sizes, clips):
    grads = _grads(sizes, len(sizes) + sum(sizes))
    sums = vpe.vpe_grad_sumsq(grads)
    want = _sumsq(grads)
    assert sums.dtype == torch.float64
    assert abs(sums.item() - want) <= want * sum(sizes) * 2.0 ** -53
    assert torch.equal(sums, vpe.vpe_grad_sumsq(grads))
    max_norm = math.sqrt(want) * (0.3 if clips else 1.5)
    out = [torch.full_like(t, float("nan")) for t in grads]
    norm = vpe.vpe_grad_clip(grads, [sums], max_norm, out=out)
    assert norm.dtype == F32 and norm.shape == (1,)
    _check(grads, out, [want], max_norm, norm)
    if not clips:
        assert all(torch.equal(o, t) for o, t in zip(out, grads))
    # in place: the same bits
    same = [t.clone() for t in grads]
    assert torch.equal(vpe.vpe_grad_clip(same, [sums], max_norm), norm)
    assert all(torch.equal(o, t) for o, t in zip(out, same))


def test_ranks_share_one_norm():
    ranks = [_grads([100, 31], 1), _grads([4097], 2), _grads([1, 2, 3], 3)]
    sums = [vpe.vpe_grad_sumsq(g) for g in ranks]
    want = [_sumsq(g) for g in ranks]
    for g in ranks:
        out = [torch.empty_like(t) for t in g]
        norm = vpe.vpe_grad_clip(g, sums, 0.05, out=out)
        _check(g, out, want, 0.05, norm)


def test_unaligned_tensors():
    flat = _grads([50_000], 5, types=[BF16])[0]
    dst = torch.zeros_like(flat)
    cuts = [(1, 700), (703, 16390), (20001, 20002), (30005, 49999)]
    grads = [flat[a:b] for a, b in cuts]
    out = [dst[a + 1:b + 1] for a, b in cuts]
    sums = vpe.vpe_grad_sumsq(grads)
    norm = vpe.vpe_grad_clip(grads, [sums], 0.1, out=out)
    _check(grads, out, [_sumsq(grads)], 0.1, norm)
    touched = torch.zeros_like(flat, dtype=torch.bool)
    for a, b in cuts:
        touched[a + 1:b + 1] = True
    assert (dst[~touched] == 0).all()


def test_values_past_fp32_squares():
    # squares past fp32's largest value, and below its smallest
    for scale, dtype in ((1e30, F32), (1e30, BF16), (1e-30, F32), (1e-30, BF16)):
        grads = _grads([3000, 17], 9, scale=scale, types=[dtype, dtype])
        sums = vpe.vpe_grad_sumsq(grads)
        want = _sumsq(grads)
        assert abs(sums.item() - want) <= want * 4000 * 2.0 ** -53
        out = [torch.empty_like(t) for t in grads]
        norm = vpe.vpe_grad_clip(grads, [sums], 1.0, out=out)
        _check(grads, out, [want], 1.0, norm)


def test_zeros_infinities_and_nan():
    z = [torch.zeros(100, device="cuda")]
    norm = vpe.vpe_grad_clip(z, [vpe.vpe_grad_sumsq(z)], 1.0)
    assert norm.item() == 0 and (z[0] == 0).all()
    g = _grads([1000], 3, types=[F32])
    g[0][7] = float("inf")
    out = [torch.empty_like(t) for t in g]
    norm = vpe.vpe_grad_clip(g, [vpe.vpe_grad_sumsq(g)], 1.0, out=out)
    assert norm.item() == float("inf")
    assert torch.isnan(out[0][7]) and (torch.cat([out[0][:7], out[0][8:]]) == 0).all()
    g[0][7] = float("nan")
    norm = vpe.vpe_grad_clip(g, [vpe.vpe_grad_sumsq(g)], 1.0, out=out)
    assert torch.isnan(norm).all() and torch.isnan(out[0]).all()
    g = _grads([1000], 3, types=[F32])
    norm = vpe.vpe_grad_clip(g, [vpe.vpe_grad_sumsq(g)], 0.0)
    assert norm.item() > 0 and (g[0] == 0).all()


def test_no_elements():
    g = [torch.empty(0, device="cuda"), torch.empty(0, device="cuda", dtype=BF16)]
    s = vpe.vpe_grad_sumsq(g)
    assert s.item() == 0
    assert vpe.vpe_grad_clip(g, [s], 1.0).item() == 0


def test_refusals():
    a, b = torch.zeros(8, device="cuda"), torch.zeros(8, device="cuda")
    s = vpe.vpe_grad_sumsq([a])
    for bad in (lambda: vpe.vpe_grad_sumsq([]), lambda: vpe.vpe_grad_clip([], [s], 1.0),
                lambda: vpe.vpe_grad_clip([a], [], 1.0),
                lambda: vpe.vpe_grad_sumsq([a, b.cpu()]),
                lambda: vpe.vpe_grad_sumsq([torch.zeros(4, 4, device="cuda").t()[:, :3]]),
                lambda: vpe.vpe_grad_clip([a], [s.float()], 1.0),
                lambda: vpe.vpe_grad_clip([a, a], [s], 1.0),
                lambda: vpe.vpe_grad_clip([a[:6], a[4:]], [s], 1.0),
                lambda: vpe.vpe_grad_clip([a, b], [s], 1.0, out=[b, a]),
                lambda: vpe.vpe_grad_clip([a, b], [s], 1.0, out=[a]),
                lambda: vpe.vpe_grad_clip([a], [s], 1.0, out=[b.bfloat16()]),
                lambda: vpe.vpe_grad_clip([a[:4]], [s], 1.0, out=[a[2:6]]),
                lambda: vpe.vpe_grad_clip([a], [s], 1.0, norm=a[:1]),
                lambda: vpe.vpe_grad_clip([a], [s], 1.0, norm=s)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        vpe.vpe_grad_sumsq([a.half()])
    for bad in (-1.0, float("inf"), float("nan")):
        with pytest.raises(vpe.VpeError):
            vpe.vpe_grad_clip([a], [s], bad)
    # the same gradient twice counts twice in the sum
    assert vpe.vpe_grad_sumsq([b + 2, a + 1]).item() == 40
    c = b + 1
    assert vpe.vpe_grad_sumsq([c, c]).item() == 16


def test_captured_and_replayed():
    """The table of tensors belongs to the captured launches."""
    grads = _grads([70_001, 5, 300_000], 11)
    out = [torch.empty_like(t) for t in grads]
    sums, norm = torch.empty(1, dtype=torch.float64, device="cuda"), torch.empty(1, device="cuda")
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        vpe.vpe_grad_sumsq(grads, sumsq=sums, workspace=ws)
        vpe.vpe_grad_clip(grads, [sums], 0.5, out=out, norm=norm)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vpe.vpe_grad_sumsq(grads, sumsq=sums, workspace=ws)
        vpe.vpe_grad_clip(grads, [sums], 0.5, out=out, norm=norm)
    for step in range(3):
        fresh = _grads([70_001, 5, 300_000], 20 + step, scale=1e-3 * (step + 1))
        for t, f in zip(grads, fresh):
            t.copy_(f)
        graph.replay()
        torch.cuda.synchronize()
        want = vpe.vpe_grad_sumsq(fresh)
        eager = [torch.empty_like(t) for t in fresh]
        eager_norm = vpe.vpe_grad_clip(fresh, [want], 0.5, out=eager)
        assert torch.equal(sums, want) and torch.equal(norm, eager_norm)
        assert all(torch.equal(a, b) for a, b in zip(out, eager))
