"""bf16 gradients whose products go in tiles of 256 x 256, with the logits of the next
piece beside them, against 64-bit references with bounds derived from the roundings."""
import pytest
import torch

import vocab_sharded_embedding_amd as vpe
from _loss import Reference, assert_within, products
from _loss_large import BACKWARD, COPIED, LIVE, ONE_PIECE, PIECES, SMALLER

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def _case(m, vocab, dim, seed, live=None):
    """Hidden rows that lean towards their target's row, `live` of them with a target;
    the others hold NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = (0.1 * torch.randn(vocab, dim, generator=g, device="cuda")).to(BF16)
    t = torch.randint(0, vocab, (m,), generator=g, device="cuda")
    x = torch.randn(m, dim, generator=g, device="cuda")
    x = x + 12 * torch.rand(m, 1, generator=g, device="cuda") * w[t].float() / (0.01 * dim)
    x = x.to(BF16)
    gl = torch.rand(m, generator=g, device="cuda") + 0.5
    gl[m // 2] *= -1
    if live is not None:
        dead = torch.randperm(m, generator=g, device="cuda")[live:]
        t[dead] = -100
        x[dead] = float("nan")
    return x, w, t, gl


def _loss(x, w, t, vocab):
    a, b = vpe.vpe_lmhead_xent(x, w, t, 0, vocab)
    return vpe.vpe_xent_loss([a], [b], t, vocab)


def _reference(x, w, t, vocab, gl):
    return Reference(torch.where(t[:, None] >= 0, x, 0.0), w, t, vocab, gl)


def _check(x, w, t, gl, vocab, types=((BF16, BF16), (F32, F32))):
    ref = _reference(x, w, t, vocab, gl)
    loss, lse = _loss(x, w, t, vocab)
    assert_within(loss, ref.loss, ref.loss_err, "loss")
    for xd, wd in types:
        rx, ex, rw, ew = ref.grads(slice(0, vocab), xd, wd)
        gx, gw = vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, vocab, x_dtype=xd, weight_dtype=wd)
        assert_within(gx, rx, ex, f"grad_x {xd}")
        assert_within(gw, rw, ew, f"grad_weight {wd}")
        assert (gx[t < 0] == 0).all()
        again = vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, vocab, x_dtype=xd, weight_dtype=wd)
        assert torch.equal(gx, again[0]) and torch.equal(gw, again[1])
    return ref, lse, (rx, ex, rw, ew), (gx, gw)


@pytest.mark.parametrize("m,vocab,dim", ONE_PIECE + COPIED + PIECES)
def test_gradients(m, vocab, dim):
    _check(*_case(m, vocab, dim, m), vocab)


@pytest.mark.parametrize("live", LIVE)
def test_pieces_of_live_rows(live):
    m, vocab, dim = PIECES[0]
    x, w, t, gl = _case(m, vocab, dim, live, live)
    _check(x, w, t, gl, vocab, types=((BF16, F32),))


@pytest.mark.parametrize("m,vocab,dim", [PIECES[0], PIECES[2], ONE_PIECE[1], COPIED[1]])
def test_one_gradient_alone_and_added(m, vocab, dim):
    x, w, t, gl = _case(m, vocab, dim, m + 1, m - 99)
    ref, lse, (rx, ex, rw, ew), _ = _check(x, w, t, gl, vocab, types=((F32, BF16),))
    gx, none = vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, vocab, x_dtype=F32, with_weight=False)
    assert none is None
    assert_within(gx, rx, ex, "grad_x alone")
    none, gw = vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, vocab, with_x=False)
    assert none is None
    assert_within(gw, rw, ew, "grad_weight alone")
    del rx, ex, rw, ew, gx, gw
    for dtype in (BF16, F32):
        base = (0.1 * torch.randn(vocab, dim, device="cuda")).to(dtype)
        for with_x in (True, False):
            acc = base.clone()
            vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, vocab, grad_weight=acc, accumulate=True,
                                     with_x=with_x)
            _, _, rw, ew = ref.grads(slice(0, vocab), BF16, dtype, base)
            assert_within(acc, rw, ew, f"grad_weight added in {dtype}")


@pytest.mark.parametrize("tp", [2, 3])
def test_shards_of_one_loss(tp):
    """Every rank's gradients in several pieces; a target lies in one shard alone."""
    m, rows, dim = 1030, 70016, 136
    vocab = tp * rows
    x, w, t, gl = _case(m, vocab, dim, tp, 1000)
    ref = _reference(x, w, t, vocab, gl)
    cut = [slice(r * rows, (r + 1) * rows) for r in range(tp)]
    parts = [vpe.vpe_lmhead_xent(x, w[s], t, s.start, vocab) for s in cut]
    loss, lse = vpe.vpe_xent_loss([a for a, _ in parts], [b for _, b in parts], t, vocab)
    assert_within(loss, ref.loss, ref.loss_err, "loss")
    for s in cut:
        rx, ex, rw, ew = ref.grads(s, F32, BF16)
        gx, gw = vpe.vpe_lmhead_xent_grad(x, w[s], t, lse, gl, s.start, vocab, x_dtype=F32)
        assert_within(gx, rx, ex, f"grad_x of {s}")
        assert_within(gw, rw, ew, f"grad_weight of {s}")


@pytest.mark.parametrize("around", [0, 29])
@pytest.mark.parametrize("m,rows,dim", BACKWARD + SMALLER)
def test_head_backward(m, rows, dim, around):
    """The shard's columns alone, or between others that hold NaN."""
    x, w, _, _ = _case(m, rows, dim, m)
    g = torch.Generator(device="cuda").manual_seed(rows)
    col = 8 if around else 0
    d = torch.full((m, rows + around), float("nan"), device="cuda", dtype=BF16)
    d[:, col:col + rows] = (torch.randn(m, rows, generator=g, device="cuda") * 0.1).to(BF16)
    dd = d[:, col:col + rows].double()
    zero = torch.zeros_like(dd)
    for xd, wd in ((BF16, F32), (F32, BF16)):
        rx, ex, rw, ew = products(dd, zero, x.double(), w.double(), xd, wd)
        kw = dict(col_offset=col, x_dtype=xd, weight_dtype=wd)
        gx, gw = vpe.vpe_lmhead_grad(d, x, w, **kw)
        assert_within(gx, rx, ex, f"grad_x {xd}")
        assert_within(gw, rw, ew, f"grad_weight {wd}")
        again = vpe.vpe_lmhead_grad(d, x, w, **kw)
        assert torch.equal(gx, again[0]) and torch.equal(gw, again[1])
        gx, none = vpe.vpe_lmhead_grad(d, x, w, col_offset=col, x_dtype=xd, with_weight=False)
        assert none is None
        assert_within(gx, rx, ex, f"grad_x {xd} alone")
        none, gw = vpe.vpe_lmhead_grad(d, x, w, col_offset=col, weight_dtype=wd, with_x=False)
        assert none is None
        assert_within(gw, rw, ew, f"grad_weight {wd} alone")
        base = torch.randn(rows, dim, generator=g, device="cuda").to(wd)
        acc = base.clone()
        vpe.vpe_lmhead_grad(d, x, w, col_offset=col, grad_weight=acc, accumulate=True)
        _, _, rw, ew = products(dd, zero, x.double(), w.double(), xd, wd, base)
        assert_within(acc, rw, ew, f"grad_weight {wd} added")


def test_pieces_captured_and_replayed():
    """The pieces' two buffers belong to the workspace of the captured call."""
    m, vocab, dim = PIECES[0]
    x, w, t, gl = _case(m, vocab, dim, 1)
    lse = _loss(x, w, t, vocab)[1].clone()
    d = torch.empty(200, 9001, device="cuda", dtype=BF16)

    def buffers():
        return (torch.empty_like(x), torch.empty_like(w), torch.empty(200, dim, device="cuda"),
                torch.empty(9001, dim, device="cuda"))

    def calls(x, w, t, lse, gl, d, out, ws):
        vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, vocab, grad_x=out[0], grad_weight=out[1],
                                 workspace=ws)
        vpe.vpe_lmhead_grad(d, x[:200], w[:9001], grad_x=out[2], grad_weight=out[3], workspace=ws)

    need = max(vpe.vpe_lmhead_xent_grad_workspace(m, dim, vocab, vpe.VPE_BF16),
               vpe.vpe_lmhead_grad_workspace(200, dim, 9001, vpe.VPE_BF16))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    out = buffers()
    d.zero_()
    calls(x, w, t, lse, gl, d, out, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(x, w, t, lse, gl, d, out, ws)
    for turn in range(4):
        fresh = _case(m, vocab, dim, turn + 2, None if turn == 0 else 1000 - 300 * turn)
        fresh[0][:200].nan_to_num_(0.0)
        new_lse = _loss(*fresh[:3], vocab)[1]
        new_d = torch.randn(200, 9001, device="cuda").to(BF16)
        for a, b in zip((x, w, t, gl, lse, d), (*fresh, new_lse, new_d)):
            a.copy_(b)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        eager = buffers()
        calls(*fresh[:3], new_lse, fresh[3], new_d, eager, torch.empty_like(ws))
        for i, (a, b) in enumerate(zip(out, eager)):
            assert torch.equal(a, b), (turn, i)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shift", ["width", "table", "rows"])
@pytest.mark.parametrize("m", [20, 60, 128, 200, 300])
def test_one_gradient_of_unaligned_rows(m, shift, dtype):
    """The operand that a lone gradient does not read may lie at any element."""
    rows, dim = 2000, 129 if shift == "width" else 136
    g = torch.Generator(device="cuda").manual_seed(m)

    def at(first, *shape):
        n = shape[0] * shape[1]
        whole = torch.full((n + 16,), float("nan"), device="cuda", dtype=dtype)
        whole[first:first + n] = torch.randn(n, generator=g, device="cuda").to(dtype)
        return whole[first:first + n].view(shape)

    d = at(0, m, rows)
    w, x = at(1 if shift == "table" else 0, rows, dim), at(3 if shift == "rows" else 0, m, dim)
    dd = d.double()
    rx, ex, rw, ew = products(dd, torch.zeros_like(dd), x.double(), w.double(), dtype, dtype)
    gx, _ = vpe.vpe_lmhead_grad(d, x, w, with_weight=False)
    assert_within(gx, rx, ex, "grad_x alone")
    _, gw = vpe.vpe_lmhead_grad(d, x, w, with_x=False)
    assert_within(gw, rw, ew, "grad_weight alone")
    # an operand that is not read takes no part, whatever it holds and wherever it lies
    same, _ = vpe.vpe_lmhead_grad(d, torch.full_like(x, float("nan")), w, with_weight=False)
    assert torch.equal(same, gx)
    _, same = vpe.vpe_lmhead_grad(d, x, torch.full_like(w, float("nan")), with_x=False)
    assert torch.equal(same, gw)
