"""Edges of the cross entropy, its gradients and the head's backward on the GPU: what
masked rows and foreign columns hold, empty batches, workspaces, streams, captured
launches, refusals, and the calls together as a training step makes them."""
import pytest
import torch

import vocab_sharded_embedding_amd as vpe
from _loss import HALF, U, Reference, assert_within, products

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
INF, NAN = float("inf"), float("nan")


def _case(m, vocab, dim, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(m, dim, generator=g, device="cuda").to(dtype)
    w = (0.1 * torch.randn(vocab, dim, generator=g, device="cuda")).to(dtype)
    t = torch.randint(0, vocab, (m,), generator=g, device="cuda")
    return x, w, t, torch.rand(m, generator=g, device="cuda") + 0.5


def _loss(x, w, t, vocab, **kw):
    a, b = vpe.vpe_lmhead_xent(x, w, t, 0, vocab, **kw)
    return vpe.vpe_xent_loss([a], [b], t, vocab)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("m", [5, 40, 200, 700, 1300])
def test_masked_rows_may_hold_anything(m, dtype):
    vocab, dim = 777, 72
    x, w, t, gl = _case(m, vocab, dim, dtype, m)
    dead = torch.arange(m, device="cuda") % 4 == 1
    t[dead] = -100
    zero = torch.arange(m, device="cuda") % 7 == 3
    gl[zero] = 0.0
    ref = Reference(x, w, t, vocab, gl)
    bad = x.clone()
    bad[dead] = torch.tensor([NAN, INF, -INF], device="cuda").to(dtype).repeat(dim // 3)
    loss, lse = _loss(bad, w, t, vocab)
    assert_within(loss, ref.loss, ref.loss_err, "loss")
    assert (loss[dead] == 0).all() and (lse[dead] == 0).all()
    # a row without a factor takes no part in the gradients either
    bad[zero] = NAN
    lse_bad = torch.where(dead | zero, NAN, lse)
    gl_bad = torch.where(dead, NAN, gl)
    gx, gw = vpe.vpe_lmhead_xent_grad(bad, w, t, lse_bad, gl_bad, 0, vocab)
    rx, ex, rw, ew = ref.grads(slice(0, vocab), dtype, dtype)
    assert_within(gx, rx, ex, "grad_x")
    assert_within(gw, rw, ew, "grad_weight")
    assert (gx[dead | zero] == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("m", [3, 300])
def test_no_live_rows(m, dtype):
    x, w, t, gl = _case(m, 300, 40, dtype)
    t[:] = torch.arange(m, device="cuda") % 2 * 1000 - 5   # -5 and 995
    loss, lse = _loss(x, w, t, 300)
    assert (loss == 0).all() and (lse == 0).all()
    gx, gw = vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, 300)
    assert (gx == 0).all() and (gw == 0).all()
    keep = torch.randn(300, 40, device="cuda").to(dtype)
    acc = keep.clone()
    vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, 300, grad_weight=acc, accumulate=True)
    assert torch.equal(acc, keep)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_empty_batch(dtype):
    x, w, t, gl = _case(0, 50, 24, dtype)
    a, b = vpe.vpe_lmhead_xent(x, w, t, 0, 50)
    loss, lse = vpe.vpe_xent_loss([a], [b], t, 50)
    assert loss.numel() == 0 and lse.numel() == 0
    gx, gw = vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, 50)
    assert gx.shape == (0, 24) and (gw == 0).all()
    gx, gw = vpe.vpe_lmhead_grad(torch.empty(0, 50, device="cuda", dtype=dtype), x, w)
    assert gx.shape == (0, 24) and (gw == 0).all()
    keep = torch.randn(50, 24, device="cuda").to(dtype)
    acc = keep.clone()
    vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, 50, grad_weight=acc, accumulate=True)
    vpe.vpe_lmhead_grad(torch.empty(0, 50, device="cuda", dtype=dtype), x, w, grad_weight=acc,
                        accumulate=True)
    assert torch.equal(acc, keep)


@pytest.mark.parametrize("m", [4, 300])
def test_infinities_and_nan_stay_in_their_row(m):
    x, w, t, _ = _case(m, 900, 64, F32)
    ref = Reference(x, w, t, 900)
    x[1, 5], x[2, 7] = NAN, INF
    loss, lse = _loss(x, w, t, 900)
    assert torch.isnan(loss[1]) and torch.isnan(loss[2])
    keep = torch.ones(m, dtype=torch.bool, device="cuda")
    keep[1:3] = False
    assert_within(loss[keep], ref.loss[keep], ref.loss_err[keep], "loss")


def test_large_logits():
    """Logits far apart: the softmax is one-hot, the loss their difference."""
    x = torch.full((40, 64), 100.0, device="cuda")
    w = torch.zeros(500, 64, device="cuda")
    w[7] = 50.0       # logit 320000, all others 0
    t = torch.full((40,), 7, device="cuda")
    t[20:] = 3
    loss, lse = _loss(x, w, t, 500)
    assert (loss[:20] == 0).all() and (loss[20:] == 320000).all()
    gl = torch.ones(40, device="cuda")
    gx, gw = vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, 500)
    assert (gx[:20] == 0).all() and (gx[20:] == 50).all()
    assert (gw[7] == 2000).all() and (gw[3] == -2000).all()
    assert (gw[:3] == 0).all() and (gw[8:] == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_shard_far_up_a_vocabulary(dtype):
    """Ids past 2^32, and a vocabulary larger than the ranks at hand."""
    start, vocab, rows, m = (1 << 33) + 5, 1 << 40, 1000, 70
    x, w, t, gl = _case(m, rows, 48, dtype)
    ids = t + start
    ids[3], ids[4], ids[5], ids[6] = start - 1, start + rows, vocab, -1
    mine = (ids >= start) & (ids < start + rows)
    a, b = vpe.vpe_lmhead_xent(x, w, ids, start, vocab)
    z = x.double() @ w.double().T
    ref = Reference(x, w, torch.where(mine, t, 0), rows, gl)
    live = (ids >= 0) & (ids < vocab)
    assert_within(a[live], torch.logsumexp(z, 1)[live], ref.lse_err[live], "shard_lse")
    assert (a[~live] == 0).all() and (b[~mine] == 0).all()
    zt = torch.gather(z, 1, t[:, None])[:, 0]
    assert_within(b[mine], zt[mine], ref.zerr[mine], "target_logit")
    # the gradient of a row whose target is another rank's: the softmax alone
    lse = torch.logsumexp(z, 1).float()
    gx, gw = vpe.vpe_lmhead_xent_grad(x, w, ids, lse, gl, start, vocab, x_dtype=F32,
                                      weight_dtype=F32)
    p = torch.exp(z - lse.double()[:, None])
    one = torch.zeros_like(p).scatter_(1, t[:, None], mine.double()[:, None])
    used = live.double()[:, None] * gl.double()[:, None]
    d = used * (p - one)
    err = used * p * (ref.arg + ref.lse_err + 8 * U)[:, None] * 1.01
    err = err + (4 * U + HALF[dtype]) * (d.abs() + err) + 2 * U * used
    rx, ex, rw, ew = products(d, err, x.double(), w.double(), F32, F32)
    assert_within(gx, rx, ex, "grad_x")
    assert_within(gw, rw, ew, "grad_weight")


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,col", [(64, 8), (100, 3), (77, 16), (256, 40)])
def test_head_backward_reads_its_columns_only(rows, col, dtype):
    m, dim = 150, 56
    x, w, _, _ = _case(m, rows, dim, dtype)
    d = torch.full((m, rows + col + 29), NAN, device="cuda", dtype=dtype)
    d[:, col:col + rows] = torch.randn(m, rows, device="cuda").to(dtype)
    gx, gw = vpe.vpe_lmhead_grad(d, x, w, col_offset=col)
    dd = d[:, col:col + rows].double()
    rx, ex, rw, ew = products(dd, torch.zeros_like(dd), x.double(), w.double(), dtype, dtype)
    assert_within(gx, rx, ex, "grad_x")
    assert_within(gw, rw, ew, "grad_weight")


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("gdtype", [F32, BF16], ids=["to_f32", "to_bf16"])
@pytest.mark.parametrize("m,vocab,dim", [(20, 300, 33), (180, 515, 64), (1100, 700, 40)])
def test_added_gradients(m, vocab, dim, dtype, gdtype):
    x, w, t, gl = _case(m, vocab, dim, dtype, m)
    ref = Reference(x, w, t, vocab, gl)
    _, lse = _loss(x, w, t, vocab)
    base = torch.randn(vocab, dim, device="cuda").to(gdtype)
    acc = base.clone()
    gx, gw = vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, vocab, grad_weight=acc, accumulate=True)
    assert gw is acc
    _, _, rw, ew = ref.grads(slice(0, vocab), dtype, gdtype, base)
    assert_within(acc, rw, ew, "grad_weight added")
    d = torch.randn(m, vocab, device="cuda").to(dtype)
    acc = base.clone()
    vpe.vpe_lmhead_grad(d, x, w, grad_weight=acc, accumulate=True, with_x=False)
    dd = d.double()
    _, _, rw, ew = products(dd, torch.zeros_like(dd), x.double(), w.double(), dtype, gdtype, base)
    assert_within(acc, rw, ew, "grad_weight added")


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_unaligned_tensors_and_what_lies_around_them(dtype):
    """Odd widths put every row at another alignment; nothing beside the outputs is
    written."""
    m, vocab, dim = 90, 333, 37
    x, w, t, gl = _case(m, vocab, dim, dtype)
    pad = 5
    wide = torch.full((m * dim + vocab * dim + 3 * pad,), 7.0, device="cuda", dtype=dtype)
    gx = wide[pad:pad + m * dim].view(m, dim)
    gw = wide[2 * pad + m * dim:2 * pad + m * dim + vocab * dim].view(vocab, dim)
    shift = torch.cat([x.new_zeros(1), x.reshape(-1)])[1:].view(m, dim)
    ref = Reference(x, w, t, vocab, gl)
    _, lse = _loss(shift, w, t, vocab)
    vpe.vpe_lmhead_xent_grad(shift, w, t, lse, gl, 0, vocab, grad_x=gx, grad_weight=gw)
    rx, ex, rw, ew = ref.grads(slice(0, vocab), dtype, dtype)
    assert_within(gx, rx, ex, "grad_x")
    assert_within(gw, rw, ew, "grad_weight")
    rest = torch.cat([wide[:pad], wide[pad + m * dim:2 * pad + m * dim],
                      wide[2 * pad + m * dim + vocab * dim:]])
    assert (rest == 7.0).all()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("m,vocab,dim", [(20, 33001, 37), (60, 34007, 129), (128, 33001, 100),
                                         (300, 40003, 65), (520, 33001, 63)])
def test_rows_at_any_element(m, vocab, dim, dtype):
    """Rows that begin at any element, with what must not count right before the first
    and right behind the last one."""
    g = torch.Generator(device="cuda").manual_seed(m)

    def between(n, scale):
        whole = torch.full((n + 2,), NAN, device="cuda", dtype=dtype)
        whole[1:-1] = (scale * torch.randn(n, generator=g, device="cuda")).to(dtype)
        return whole[1:-1]

    x, w = between(m * dim, 1.0).view(m, dim), between(vocab * dim, 0.1).view(vocab, dim)
    t = torch.randint(0, vocab, (m,), generator=g, device="cuda")
    t[::9] = -1
    gl = torch.rand(m, generator=g, device="cuda") + 0.5
    ref = Reference(x, w, t, vocab, gl)
    loss, lse = _loss(x, w, t, vocab)
    assert_within(loss, ref.loss, ref.loss_err, "loss")
    gx, gw = vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, vocab)
    rx, ex, rw, ew = ref.grads(slice(0, vocab), dtype, dtype)
    assert_within(gx, rx, ex, "grad_x")
    assert_within(gw, rw, ew, "grad_weight")
    d = between(m * vocab, 1.0).view(m, vocab)
    gx, gw = vpe.vpe_lmhead_grad(d, x, w)
    dd = d.double()
    rx, ex, rw, ew = products(dd, torch.zeros_like(dd), x.double(), w.double(), dtype, dtype)
    assert_within(gx, rx, ex, "grad_x")
    assert_within(gw, rw, ew, "grad_weight")


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_a_small_last_piece_of_a_copied_table(dtype):
    """32768 (65536) table rows are copied at a time; the last 300 hold the logits that
    matter."""
    m, dim, vocab = 640, 1021, (32768 if dtype == F32 else 65536) + 300
    x, w, t, gl = _case(m, vocab, dim, dtype)
    w[-300:] *= 4
    t[::3] = vocab - 1 - torch.arange(t[::3].numel(), device="cuda")
    ref = Reference(x, w, t, vocab, gl)
    loss, lse = _loss(x, w, t, vocab)
    assert_within(loss, ref.loss, ref.loss_err, "loss")
    assert_within(lse, ref.lse, ref.lse_err, "lse")


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("live", [1, 63, 64, 65, 127, 128, 129, 255, 256, 257, 383, 385])
def test_live_rows_around_a_tile(live, dtype):
    """The last tile of live rows full, half full and beyond."""
    m, vocab, dim = 520, 34000, 136
    x, w, t, gl = _case(m, vocab, dim, dtype, live)
    order = torch.randperm(m, device="cuda")
    t[order[live:]] = -100
    ref = Reference(x, w, t, vocab, gl)
    loss, lse = _loss(x, w, t, vocab)
    assert_within(loss, ref.loss, ref.loss_err, "loss")
    gx, gw = vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, vocab)
    rx, ex, rw, ew = ref.grads(slice(0, vocab), dtype, dtype)
    assert_within(gx, rx, ex, "grad_x")
    assert_within(gw, rw, ew, "grad_weight")


@pytest.mark.parametrize("live", [0, 1, 128, 129, 256, 300, 384, 385, 642, 700, 768, 769, 900,
                                  1024, 1025, 1030])
def test_live_rows_in_large_tiles(live):
    """As above where the bf16 logits take 256 x 256 tiles, by workgroups that go from
    tile to tile: whole, half and divided ones."""
    m, vocab, dim = 1030, 44000, 72
    x, w, t, gl = _case(m, vocab, dim, BF16, live)
    order = torch.randperm(m, device="cuda")
    t[order[live:]] = -100
    x[order[live:]] = NAN
    clean = torch.where(t[:, None] < 0, 0.0, x)
    ref = Reference(clean, w, t, vocab, gl)
    loss, lse = _loss(x, w, t, vocab)
    assert_within(loss, ref.loss, ref.loss_err, "loss")
    gx, gw = vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, vocab)
    rx, ex, rw, ew = ref.grads(slice(0, vocab), BF16, BF16)
    assert_within(gx, rx, ex, "grad_x")
    assert_within(gw, rw, ew, "grad_weight")


def test_large_tiles_captured():
    m, vocab, dim = 1100, 70000, 64
    x, w, t, gl = _case(m, vocab, dim, BF16)
    buf = _buffers(m, vocab, dim, BF16)
    _step(x, w, t, gl, vocab, *buf)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _step(x, w, t, gl, vocab, *buf)
    for turn in range(4):
        fresh = _case(m, vocab, dim, BF16, turn + 1)
        fresh[2][turn::3] = -100
        for a, b in zip((x, w, t, gl), fresh):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        eager = _buffers(m, vocab, dim, BF16)
        _step(*fresh, vocab, *eager)
        for name, i in (("loss", 0), ("lse", 1), ("grad_x", 4), ("grad_weight", 5), ("norm", 9)):
            assert torch.equal(buf[i], eager[i]), (turn, name)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_hidden_rows_alone_at_any_element(dtype):
    m, vocab, dim = 150, 640, 64
    x, w, _, _ = _case(m, vocab, dim, dtype)
    odd = torch.cat([x.new_zeros(1), x.reshape(-1)])[1:].view(m, dim)
    d = torch.randn(m, vocab, device="cuda").to(dtype)
    for a, b in zip(vpe.vpe_lmhead_grad(d, odd, w), vpe.vpe_lmhead_grad(d, x, w)):
        assert torch.equal(a, b)


def _bytes(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_a_workspace_for_more_rows_serves_fewer(dtype):
    vocab, dim, code = 5000, 64, 1 if dtype == BF16 else 0
    most = 600
    ws = _bytes(max(vpe.vpe_lmhead_xent_workspace(most, dim, vocab, code),
                    vpe.vpe_lmhead_xent_grad_workspace(most, dim, vocab, code),
                    vpe.vpe_lmhead_grad_workspace(most, dim, vocab, code)))
    for m in (600, 1, 33, 300, 65, 129):
        ws.fill_(255)
        x, w, t, gl = _case(m, vocab, dim, dtype, m)
        ref = Reference(x, w, t, vocab, gl)
        loss, lse = _loss(x, w, t, vocab, workspace=ws)
        assert_within(loss, ref.loss, ref.loss_err, "loss")
        gx, gw = vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, vocab, workspace=ws)
        rx, ex, rw, ew = ref.grads(slice(0, vocab), dtype, dtype)
        assert_within(gx, rx, ex, "grad_x")
        assert_within(gw, rw, ew, "grad_weight")
        with pytest.raises(vpe.VpeError):
            vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, vocab, workspace=_bytes(1 << 12))


def test_gradients_against_differences():
    """Central differences of the summed loss in 64 bits, in random directions."""
    m, vocab, dim = 60, 400, 48
    x, w, t, gl = _case(m, vocab, dim, F32)
    t[::6] = -1
    _, lse = _loss(x, w, t, vocab)
    gx, gw = vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, vocab)

    def total(xx, ww):
        z = xx @ ww.T
        live = t >= 0
        at = torch.where(live, t, 0)[:, None]
        loss = torch.logsumexp(z, 1) - torch.gather(z, 1, at)[:, 0]
        return (torch.where(live, loss, 0.0) * gl.double()).sum()

    g = torch.Generator(device="cuda").manual_seed(1)
    h = 1e-5
    for _ in range(4):
        dx = torch.randn(m, dim, generator=g, device="cuda", dtype=torch.float64)
        dw = torch.randn(vocab, dim, generator=g, device="cuda", dtype=torch.float64)
        xd, wd = x.double(), w.double()
        slope = (total(xd + h * dx, wd + h * dw) - total(xd - h * dx, wd - h * dw)) / (2 * h)
        got = (gx.double() * dx).sum() + (gw.double() * dw).sum()
        # the third derivative's part of the difference is below 1e-4 of |dx|, |dw|
        # of order 1 times h^2; fp32 gradients are within 1e-4 of their size
        size = (gx.double() * dx).abs().sum() + (gw.double() * dw).abs().sum()
        assert abs(got - slope) <= 1e-4 * size


def _step(x, w, t, gl, vocab, loss, lse, a, b, gx, gw, ws, sums, cws, norm):
    vpe.vpe_lmhead_xent(x, w, t, 0, vocab, shard_lse=a, target_logit=b, workspace=ws)
    vpe.vpe_xent_loss([a], [b], t, vocab, loss=loss, lse=lse)
    vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, vocab, grad_x=gx, grad_weight=gw, workspace=ws)
    vpe.vpe_grad_sumsq([gx, gw], sumsq=sums, workspace=cws)
    vpe.vpe_grad_clip([gx, gw], [sums], 0.05, norm=norm)


def _buffers(m, vocab, dim, dtype):
    code = 1 if dtype == BF16 else 0
    f = [torch.empty(m, device="cuda") for _ in range(4)]
    need = max(vpe.vpe_lmhead_xent_workspace(m, dim, vocab, code),
               vpe.vpe_lmhead_xent_grad_workspace(m, dim, vocab, code))
    return (*f, torch.empty(m, dim, device="cuda", dtype=dtype),
            torch.empty(vocab, dim, device="cuda", dtype=dtype), _bytes(need),
            torch.empty(1, dtype=torch.float64, device="cuda"),
            _bytes(vpe.vpe_grad_sumsq_workspace([m * dim, vocab * dim])),
            torch.empty(1, device="cuda"))


@pytest.mark.parametrize("m,dtype", [(30, BF16), (300, BF16), (1200, BF16), (200, F32)])
def test_captured_steps_replayed(m, dtype):
    """Two captured steps with workspaces of their own, replayed in turn, with eager
    work between: every replay equals the eager result on the same inputs."""
    vocab, dim = 3000, 64
    graphs, held = [], []
    for k in range(2):
        x, w, t, gl = _case(m, vocab, dim, dtype, k)
        buf = _buffers(m, vocab, dim, dtype)
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            _step(x, w, t, gl, vocab, *buf)
        torch.cuda.current_stream().wait_stream(stream)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            _step(x, w, t, gl, vocab, *buf)
        graphs.append(graph)
        held.append((x, w, t, gl, buf))
    for turn in range(4):
        for k in range(2):
            x, w, t, gl, buf = held[k]
            fresh = _case(m, vocab, dim, dtype, 10 + 3 * turn + k)
            fresh[2][turn::5] = -100
            for a, b in zip((x, w, t, gl), fresh):
                a.copy_(b)
            graphs[k].replay()
            torch.cuda.synchronize()
            eager = _buffers(m, vocab, dim, dtype)
            _step(*fresh, vocab, *eager)
            for name, i in (("loss", 0), ("lse", 1), ("grad_x", 4), ("grad_weight", 5),
                            ("sumsq", 7), ("norm", 9)):
                assert torch.equal(buf[i], eager[i]), (turn, k, name)


def test_calls_on_two_streams_at_once():
    vocab, dim, m = 20000, 128, 400
    cases = [_case(m, vocab, dim, BF16, k) for k in range(2)]
    want = []
    for x, w, t, gl in cases:
        loss, lse = _loss(x, w, t, vocab)
        want.append((loss, *vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, vocab)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for (x, w, t, gl), st in zip(cases, streams):
            with torch.cuda.stream(st):
                loss, lse = _loss(x, w, t, vocab)
                got.append((loss, *vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, vocab)))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_refusals():
    x, w, t, gl = _case(8, 100, 32, BF16)
    loss, lse = _loss(x, w, t, 100)
    d = torch.zeros(8, 100, device="cuda", dtype=BF16)
    own = torch.zeros(8, 32, device="cuda", dtype=BF16)
    value = [
        lambda: vpe.vpe_lmhead_xent(x[:, :16], w, t, 0, 100),
        lambda: vpe.vpe_lmhead_xent(x, w, t[:7], 0, 100),
        lambda: vpe.vpe_lmhead_xent(x.t().contiguous().t(), w, t, 0, 100),
        lambda: vpe.vpe_lmhead_xent(x, w.cpu(), t, 0, 100),
        lambda: vpe.vpe_lmhead_xent(x, w, t, 0, 100, shard_lse=torch.empty(7, device="cuda")),
        lambda: vpe.vpe_lmhead_xent(x, w, t, 0, 100, shard_lse=loss, target_logit=loss),
        lambda: vpe.vpe_xent_loss([], [], t, 100),
        lambda: vpe.vpe_xent_loss([lse], [], t, 100),
        lambda: vpe.vpe_xent_loss([lse], [loss], t, 100, loss=gl, lse=gl),
        lambda: vpe.vpe_xent_loss([lse[:7]], [loss], t, 100),
        lambda: vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl[:7], 0, 100),
        lambda: vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl.double(), 0, 100),
        lambda: vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, 100, with_x=False,
                                         with_weight=False),
        lambda: vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, 100, grad_x=x),
        lambda: vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, 100, grad_weight=w),
        lambda: vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, 100, grad_x=own[:7]),
        lambda: vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, 100, grad_x=own, x_dtype=F32),
        lambda: vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, 100, grad_x=own, with_x=False),
        lambda: vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, 100, accumulate=True),
        lambda: vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, 100, accumulate=True,
                                         with_weight=False),
        lambda: vpe.vpe_lmhead_grad(d[:7], x, w),
        lambda: vpe.vpe_lmhead_grad(d.float(), x, w),
        lambda: vpe.vpe_lmhead_grad(d, x, w, grad_weight=w),
    ]
    for i, bad in enumerate(value):
        with pytest.raises(ValueError):
            bad()
            pytest.fail(f"case {i} was taken")
    for bad in (lambda: vpe.vpe_lmhead_xent(x, w.float(), t, 0, 100),
                lambda: vpe.vpe_lmhead_xent(x.half(), w.half(), t, 0, 100),
                lambda: vpe.vpe_lmhead_xent(x, w, t.short(), 0, 100),
                lambda: vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, 100,
                                                 x_dtype=torch.float16)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: vpe.vpe_lmhead_xent(x, w, t, 1, 100),
                lambda: vpe.vpe_lmhead_xent(x, w, t, -1, 200),
                lambda: vpe.vpe_lmhead_grad(d, x, w, col_offset=1)):
        with pytest.raises(vpe.VpeError):
            bad()


def test_no_autograd_graph():
    x, w, t, gl = _case(8, 100, 32, F32)
    x.requires_grad_(), w.requires_grad_()
    loss, lse = _loss(x, w, t, 100)
    gx, gw = vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, 100)
    assert not any(o.requires_grad for o in (loss, lse, gx, gw))


@pytest.mark.parametrize("tp,dtype", [(1, F32), (2, F32), (2, BF16), (4, BF16)])
def test_a_training_step_over_tied_shards(tp, dtype):
    """Lookup, head, loss, gradients of both uses of the tied table, clipping and an
    update, through the layers, against the same step in 64 bits."""
    vocab, dim, m, lr, most = 1200, 48, 90, 0.5, 0.7
    g = torch.Generator(device="cuda").manual_seed(3)
    table = (0.3 * torch.randn(vocab, dim, generator=g, device="cuda")).to(dtype)
    ids = torch.randint(0, vocab, (m,), generator=g, device="cuda")
    targets = torch.randint(0, vocab, (m,), generator=g, device="cuda")
    targets[::8] = -100
    embeds, heads = [], []
    for r in range(tp):
        e = vpe.VocabParallelEmbedding(vocab, dim, tp_size=tp, tp_rank=r, dtype=dtype,
                                       device="cuda")
        e.weight_loader(e.weight, table)
        embeds.append(e)
        heads.append(vpe.ParallelLMHead(vocab, dim, tp_size=tp, tp_rank=r, dtype=dtype,
                                        device="cuda").tie_to(e))
    x = embeds[0].sum_partials([e(ids) for e in embeds])
    assert torch.equal(x, table[ids])
    parts = [h.xent_shard(x, targets) for h in heads]
    loss, lse = heads[0].xent_loss([a for a, _ in parts], [b for _, b in parts], targets)
    live = targets >= 0
    gl = torch.where(live, 1.0 / live.sum(), 0.0)
    pieces = [h.xent_grad(x, targets, lse, gl, x_dtype=F32, weight_dtype=F32) for h in heads]
    gx = heads[0].sum_partials([p for p, _ in pieces])
    grads = []
    for e, (_, gw) in zip(embeds, pieces):
        grads.append(e.weight_grad(ids, gx, grad_weight=gw, accumulate=True))
    sums = [vpe.vpe_grad_sumsq([gw]) for gw in grads]
    norms = [vpe.vpe_grad_clip([gw], sums, most) for gw in grads]
    assert all(torch.equal(n, norms[0]) for n in norms)

    t64 = table.double().requires_grad_()
    h = t64[ids]
    want = torch.nn.functional.cross_entropy(h @ t64.T, targets, reduction="none",
                                             ignore_index=-100)
    ((want * gl.double()).sum()).backward()
    # a bf16 table's d is held in bf16: 2^-8 of each entry; fp32 roundings are far below
    rel = 2 * HALF[dtype] + 1e-5
    assert (loss.double() - want.detach()).abs().max() <= 1e-5 * (1 + want.abs().max())
    norm64 = torch.linalg.vector_norm(t64.grad)
    assert abs(norms[0].double() - norm64) <= rel * norm64
    clipped = t64.grad * min(1.0, most / (norm64.item() + 1e-6))
    got = torch.cat(grads).double()
    assert torch.linalg.vector_norm(got - clipped) <= 2 * rel * torch.linalg.vector_norm(clipped)
    updated = table.double() - lr * got
    assert torch.linalg.vector_norm(updated - (table.double() - lr * clipped)) <= \
        2 * rel * lr * torch.linalg.vector_norm(clipped)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_head_backward_after_distillation(dtype):
    """distill_grad's result straight into the head's backward, over two ranks."""
    vocab, dim, m, tp, k = 640, 64, 50, 2, 8
    x, w, _, gl = _case(m, vocab, dim, dtype)
    heads, logits = [], torch.empty(m, vocab, device="cuda", dtype=dtype)
    for r in range(tp):
        h = vpe.ParallelLMHead(vocab, dim, tp_size=tp, tp_rank=r, dtype=dtype, device="cuda")
        h.weight_loader(h.weight, w)
        h(x, logits=logits)
        heads.append(h)
    ids = torch.randint(0, vocab, (m, k), device="cuda")
    teacher = torch.randn(m, k, device="cuda")
    parts = [h.distill_shard(logits, ids, teacher) for h in heads]
    _, lse = heads[0].distill_loss([a for a, _ in parts], [b for _, b in parts], ids, teacher)
    for h in heads:
        h.distill_grad(logits, lse, gl, ids, teacher, grad_logits=logits)
    d = logits.double()
    out = [h.grad(logits, x, x_dtype=F32, weight_dtype=F32) for h in heads]
    for r, (gx, gw) in enumerate(out):
        s = slice(r * vocab // tp, (r + 1) * vocab // tp)
        rx, ex, rw, ew = products(d[:, s], torch.zeros_like(d[:, s]), x.double(), w[s].double(),
                                  F32, F32)
        assert_within(gx, rx, ex, "grad_x")
        assert_within(gw, rw, ew, "grad_weight")
