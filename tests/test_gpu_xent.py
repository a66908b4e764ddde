"""Cross entropy from the head's shards, its gradients and the head's backward on
the GPU, against 64-bit references with bounds derived from the roundings."""
import pytest
import torch

import vocab_sharded_embedding_amd as vpe
from _loss import Reference, assert_within, products

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def _inputs(m, vocab, dim, dtype, seed, itype=torch.int64, padded=True, lean=6.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = (torch.randn(vocab, dim, generator=g, device="cuda") * 0.05).to(dtype)
    t = torch.randint(0, vocab, (m,), generator=g, device="cuda")
    x = torch.randn(m, dim, generator=g, device="cuda")
    x = x + lean * torch.rand(m, 1, generator=g, device="cuda") * w[t].float() / (0.0025 * dim)
    if padded and m > 2:
        t[::5] = -100
        t[1::7] = vocab
    gl = torch.rand(m, generator=g, device="cuda") + 0.5
    if m > 8:
        gl[3] = 0.0
        gl[6] = -0.75
    return x.to(dtype), w, t.to(itype), gl


def _shards(vocab, tp):
    r = vocab // tp
    return [slice(i * r, (i + 1) * r) for i in range(tp)]


def _loss(x, w, t, vocab, tp):
    parts = [vpe.vpe_lmhead_xent(x, w[s], t, s.start, vocab) for s in _shards(vocab, tp)]
    return vpe.vpe_xent_loss([a for a, _ in parts], [b for _, b in parts], t, vocab), parts


SIZES = [
    # rows, vocabulary, width, ranks
    (1, 7, 1, 1), (1, 1000, 64, 1), (2, 256, 8, 2), (3, 130, 33, 1), (31, 999, 100, 3),
    (32, 512, 128, 2), (33, 1024, 72, 4), (64, 777, 64, 1), (65, 1536, 200, 3),
    (127, 640, 320, 5), (128, 2048, 64, 2), (129, 515, 257, 1), (256, 4096, 64, 2),
    (257, 1000, 136, 1), (300, 5031, 40, 3), (513, 2500, 96, 1), (1100, 1300, 64, 2),
]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("m,vocab,dim,tp", SIZES)
def test_loss(m, vocab, dim, tp, dtype):
    x, w, t, _ = _inputs(m, vocab, dim, dtype, m * 31 + vocab,
                         itype=torch.int32 if m % 2 else torch.int64)
    ref = Reference(x, w, t, vocab)
    (loss, lse), parts = _loss(x, w, t, vocab, tp)
    assert_within(lse, ref.lse, ref.lse_err, "lse")
    assert_within(loss, ref.loss, ref.loss_err, "loss")
    assert (loss[~ref.live] == 0).all() and (lse[~ref.live] == 0).all()
    for a, b in parts:
        assert (a[~ref.live] == 0).all() and (b[~ref.live] == 0).all()
    again, _ = _loss(x, w, t, vocab, tp)
    assert torch.equal(loss, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("m,vocab,dim,tp", SIZES)
def test_gradients(m, vocab, dim, tp, dtype):
    x, w, t, gl = _inputs(m, vocab, dim, dtype, m * 17 + vocab)
    ref = Reference(x, w, t, vocab, gl)
    (_, lse), _ = _loss(x, w, t, vocab, tp)
    for s in _shards(vocab, tp):
        for xd, wd in ((dtype, dtype), (F32, F32), (BF16, F32)):
            gx, gw = vpe.vpe_lmhead_xent_grad(x, w[s], t, lse, gl, s.start, vocab, x_dtype=xd,
                                              weight_dtype=wd)
            rx, ex, rw, ew = ref.grads(s, xd, wd)
            assert gx.dtype == xd and gw.dtype == wd
            assert_within(gx, rx, ex, f"grad_x {xd} of {s}")
            assert_within(gw, rw, ew, f"grad_weight {wd} of {s}")
            assert (gx[~ref.used] == 0).all()
        again = vpe.vpe_lmhead_xent_grad(x, w[s], t, lse, gl, s.start, vocab, x_dtype=xd,
                                         weight_dtype=wd)
        assert torch.equal(gx, again[0]) and torch.equal(gw, again[1])


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("m,vocab,dim,tp", SIZES)
def test_head_backward(m, vocab, dim, tp, dtype):
    x, w, _, _ = _inputs(m, vocab, dim, dtype, m * 13 + vocab)
    g = torch.Generator(device="cuda").manual_seed(m)
    d = (torch.randn(m, vocab, generator=g, device="cuda") * 0.1).to(dtype)
    for s in _shards(vocab, tp):
        for xd, wd in ((dtype, dtype), (F32, BF16)):
            gx, gw = vpe.vpe_lmhead_grad(d, x, w[s], col_offset=s.start, x_dtype=xd,
                                         weight_dtype=wd)
            dd = d[:, s].double()
            rx, ex, rw, ew = products(dd, torch.zeros_like(dd), x.double(), w[s].double(), xd, wd)
            assert_within(gx, rx, ex, f"grad_x {xd} of {s}")
            assert_within(gw, rw, ew, f"grad_weight {wd} of {s}")


@pytest.mark.parametrize("m,vocab,dim,dtype", [
    # several pieces of the vocabulary: 128 MB of bf16 (of fp32) each
    (2047, 75001, 64, BF16), (1200, 130000, 72, BF16), (4100, 40000, 40, BF16),
    (700, 100007, 33, F32),
])
def test_pieces(m, vocab, dim, dtype):
    x, w, t, gl = _inputs(m, vocab, dim, dtype, m)
    ref = Reference(x, w, t, vocab, gl)
    (loss, lse), _ = _loss(x, w, t, vocab, 1)
    assert_within(loss, ref.loss, ref.loss_err, "loss")
    rx, ex, rw, ew = ref.grads(slice(0, vocab), dtype, dtype)
    gx, gw = vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, vocab)
    assert_within(gx, rx, ex, "grad_x")
    assert_within(gw, rw, ew, "grad_weight")
    # one gradient alone: the same bits where the same tiles take it
    only_x, none = vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, vocab, with_weight=False)
    assert none is None
    assert_within(only_x, rx, ex, "grad_x alone")
    none, only_w = vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, vocab, with_x=False)
    assert none is None
    assert_within(only_w, rw, ew, "grad_weight alone")
    del rx, ex, rw, ew
    base = (0.1 * torch.randn(vocab, dim, device="cuda")).to(dtype)
    acc = base.clone()
    vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, vocab, grad_weight=acc, accumulate=True)
    rx, ex, rw, ew = ref.grads(slice(0, vocab), dtype, dtype, base)
    assert_within(acc, rw, ew, "grad_weight added")


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_rows_longer_than_a_tile_may_stride(dtype):
    """Vocabularies past 2^22 ids: logits' gradients in pieces and copies."""
    m, vocab, dim = 3, (1 << 22) + 77, 8
    x, w, t, gl = _inputs(m, vocab, dim, dtype, 5, padded=False)
    t[1] = vocab - 1
    ref = Reference(x, w, t, vocab, gl)
    (loss, lse), _ = _loss(x, w, t, vocab, 1)
    assert_within(loss, ref.loss, ref.loss_err, "loss")
    rx, ex, rw, ew = ref.grads(slice(0, vocab), dtype, dtype)
    gx, gw = vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, vocab)
    assert_within(gx, rx, ex, "grad_x")
    assert_within(gw, rw, ew, "grad_weight")
    d = ref.d.to(dtype)
    gx, gw = vpe.vpe_lmhead_grad(d, x, w)
    dd = d.double()
    rx, ex, rw, ew = products(dd, torch.zeros_like(dd), x.double(), w.double(), dtype, dtype)
    assert_within(gx, rx, ex, "grad_x")
    assert_within(gw, rw, ew, "grad_weight")
