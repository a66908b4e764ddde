"""The loss calls at their documented limits: the widest rows, the most ranks, the most
tensors of one call."""
import math

import pytest
import torch

import vocab_sharded_embedding_amd as vpe
from _loss import HALF, U, Reference, assert_within, products

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("m,vocab,less", [(3, 300, 0), (70, 515, 1), (300, 2000, 0),
                                          (520, 700, 9)])
def test_the_widest_rows(m, vocab, less, dtype):
    dim = vpe.VPE_MAX_LOSS_DIM - less
    g = torch.Generator(device="cuda").manual_seed(m)
    x = torch.randn(m, dim, generator=g, device="cuda").to(dtype)
    w = (torch.randn(vocab, dim, generator=g, device="cuda") / 64).to(dtype)
    t = torch.randint(0, vocab, (m,), generator=g, device="cuda")
    t[::6] = vocab
    gl = torch.rand(m, generator=g, device="cuda") + 0.5
    ref = Reference(x, w, t, vocab, gl)
    a, b = vpe.vpe_lmhead_xent(x, w, t, 0, vocab)
    loss, lse = vpe.vpe_xent_loss([a], [b], t, vocab)
    assert_within(loss, ref.loss, ref.loss_err, "loss")
    gx, gw = vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, vocab)
    rx, ex, rw, ew = ref.grads(slice(0, vocab), dtype, dtype)
    assert_within(gx, rx, ex, "grad_x")
    assert_within(gw, rw, ew, "grad_weight")
    d = torch.randn(m, vocab, generator=g, device="cuda").to(dtype)
    gx, gw = vpe.vpe_lmhead_grad(d, x, w)
    rx, ex, rw, ew = products(d.double(), torch.zeros_like(d.double()), x.double(), w.double(),
                              dtype, dtype)
    assert_within(gx, rx, ex, "grad_x")
    assert_within(gw, rw, ew, "grad_weight")


@pytest.mark.parametrize("m", [5, 300])
def test_the_most_ranks(m):
    """64 shards, some of which hold nothing but -inf for a row; and 64 sums of squares."""
    tp, rows, dim = 64, 40, 48
    vocab = tp * rows
    g = torch.Generator(device="cuda").manual_seed(m)
    x = torch.randn(m, dim, generator=g, device="cuda")
    w = 0.3 * torch.randn(vocab, dim, generator=g, device="cuda")
    t = torch.randint(0, vocab, (m,), generator=g, device="cuda", dtype=torch.int32)
    ref = Reference(x, w, t, vocab)
    parts = [vpe.vpe_lmhead_xent(x, w[r * rows:(r + 1) * rows], t, r * rows, vocab)
             for r in range(tp)]
    loss, lse = vpe.vpe_xent_loss([a for a, _ in parts], [b for _, b in parts], t, vocab)
    # the joins of 63 pairs: an exponential, a product and a sum each
    assert_within(lse, ref.lse, ref.lse_err + 63 * 5 * U, "lse")
    assert_within(loss, ref.loss, ref.loss_err + 63 * 5 * U, "loss")
    none = torch.full((m,), -math.inf, device="cuda")
    zero = torch.zeros(m, device="cuda")
    last, at = [none] * 63 + [parts[0][0]], [zero] * 64
    assert torch.equal(vpe.vpe_xent_loss(last, at, t, vocab)[1], parts[0][0])
    assert torch.equal(vpe.vpe_xent_loss(last[::-1], at, t, vocab)[1], parts[0][0])
    assert (vpe.vpe_xent_loss([none] * 64, at, t, vocab)[1] == -math.inf).all()
    sums = [vpe.vpe_grad_sumsq([w[r * rows:(r + 1) * rows]]) for r in range(tp)]
    norm = vpe.vpe_grad_clip([w], sums, 1e9)
    want = torch.linalg.vector_norm(w.double()).item()
    assert abs(norm.item() - want) <= want * (U * 1.001 + 1e-12)
    for bad in (lambda: vpe.vpe_xent_loss([none] * 65, [zero] * 65, t, vocab),
                lambda: vpe.vpe_grad_clip([w], sums + sums[:1], 1.0)):
        with pytest.raises(vpe.VpeError):
            bad()


def test_the_most_tensors():
    n = vpe.VPE_MAX_GRAD_TENSORS
    g = torch.Generator(device="cuda").manual_seed(4)
    counts = [i % 7 for i in range(n)]
    flat = {t: (torch.randn(4 * n, generator=g, device="cuda") * 1e-2).to(t) for t in (F32, BF16)}
    used = dict.fromkeys(flat, 0)
    grads = []
    for i, c in enumerate(counts):
        dtype = BF16 if i % 3 else F32
        grads.append(flat[dtype].narrow(0, used[dtype], c))
        used[dtype] += c
    keep = {t: f.clone() for t, f in flat.items()}
    sums = vpe.vpe_grad_sumsq(grads)
    want = sum(float((f[:used[t]].double() ** 2).sum()) for t, f in flat.items())
    assert abs(sums.item() - want) <= want * 4 * n * 2.0 ** -52
    norm = vpe.vpe_grad_clip(grads, [sums], 0.25 * math.sqrt(want))
    assert abs(norm.item() - math.sqrt(want)) <= math.sqrt(want) * (U * 1.001 + 1e-9)
    for t, f in flat.items():
        part = keep[t][:used[t]].double() * 0.25
        # (1e-6 beside a norm of a few: up to 2e-6 of the factor)
        assert ((f[:used[t]].double() - part).abs() <= (HALF[t] + 2 * U + 2e-6) * part.abs()).all()
        assert torch.equal(f[used[t]:], keep[t][used[t]:])
    with pytest.raises(vpe.VpeError):
        vpe.vpe_grad_sumsq(grads + grads[1:2])
