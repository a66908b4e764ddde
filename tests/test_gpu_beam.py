"""Beam search through the public calls, against a plain selection over whole
rows.  A candidate's score is two fp32 operations, repeated here one by one, so
scores, parents and tokens are compared bit for bit, ties included.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a HIP GPU"),
]

import vocab_sharded_embedding_amd as vpe  # noqa: E402
from _gpu import dev  # noqa: E402

F32, BF16 = torch.float32, torch.bfloat16
INF = float("inf")


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _plain(logits, lse, scores, beams, picks):
    """Stable descending order of ((z - lse) + score), NaN last, on the host in numpy."""
    z = logits.float().cpu().numpy()
    with np.errstate(invalid="ignore"):
        c = (z - lse.cpu().numpy()[:, None]) + scores.cpu().numpy()[:, None]
    assert c.dtype == np.float32
    v = z.shape[1]
    c = c.reshape(-1, beams * v)
    out = []
    for row in c:
        # -c ascends as c descends; a stable sort keeps the lower place first
        rank = np.where(np.isnan(row), np.float32(INF), -row)
        order = np.lexsort((np.arange(row.size), np.isnan(row), rank))[:picks]
        out.append((row[order], order // v, order % v))
    s, p, t = (np.stack(x) for x in zip(*out))
    return s, p, t


def _check(logits, lse, scores, beams, picks, tp=1):
    m, v = logits.shape
    rows = v // tp
    keys = [vpe.vpe_beam_select(logits, lse, scores, beams, picks, r * rows, v, shard_rows=rows,
                                col_offset=r * rows) for r in range(tp)]
    got = vpe.vpe_beam_merge(keys, v)
    back = vpe.vpe_beam_merge(keys[::-1], v)
    s, p, t = _plain(logits, lse, scores, beams, picks)
    n = s.shape[1]  # fewer candidates than picks: the rest is empty
    assert np.array_equal(got[0][:, :n].cpu().numpy(), s, equal_nan=True)
    assert np.array_equal(got[1][:, :n].cpu().numpy(), p)
    assert np.array_equal(got[2][:, :n].cpu().numpy(), t)
    assert bool((got[0][:, n:] == -INF).all())
    assert bool((got[1][:, n:] == -1).all()) and bool((got[2][:, n:] == -1).all())
    for a, b in zip(got, back):
        assert torch.equal(a.nan_to_num(9e9), b.nan_to_num(9e9))
    return keys


def _case(seed, n, beams, v, dtype):
    g = _gen(seed)
    logits = (3 * torch.randn(n * beams, v, generator=g, device="cuda")).to(dtype)
    lse = torch.logsumexp(logits.float(), 1)
    scores = -10 * torch.rand(n * beams, generator=g, device="cuda")
    return logits, lse, scores, g


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,beams,picks,v,tp", [
    (1, 1, 1, 1, 1), (1, 1, 5, 3, 1), (1, 3, 64, 7, 1), (2, 1, 2, 1000, 1), (1, 4, 8, 151936, 1),
    (3, 5, 10, 8193, 1), (2, 8, 16, 75968, 2), (5, 32, 64, 5001, 3), (1, 64, 64, 8200, 1),
    (40, 2, 4, 513, 1), (1, 7, 13, 300001, 1), (2, 2, 64, 60000, 4), (1, 1, 64, 16384, 1),
    (9, 3, 6, 24999, 3), (1, 33, 33, 40, 1),
])
def test_selection(n, beams, picks, v, tp, dtype):
    logits, lse, scores, _ = _case(n + beams + v, n, beams, v, dtype)
    _check(logits, lse, scores, beams, picks, tp)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_ties_go_to_the_lower_place(dtype):
    n, beams, v = 2, 4, 20000
    logits = torch.zeros(n * beams, v, device="cuda").to(dtype)
    lse = torch.zeros(n * beams, device="cuda")
    scores = torch.zeros(n * beams, device="cuda")
    for picks in (1, 8, 64):
        _check(logits, lse, scores, beams, picks)
    # a few values over and over, and beams of equal scores
    g = _gen(5)
    logits = torch.randint(-2, 3, (n * beams, v), generator=g, device="cuda").to(dtype)
    _check(logits, lse, scores, beams, 64, 4)
    # scores that differ by less than the sum keeps: equal after rounding
    logits = (torch.rand(n * beams, v, generator=g, device="cuda") * 1e-6).to(dtype)
    _check(logits, lse + 12.0, scores - 30.0, beams, 64, 2)
    # -0 and +0 are equal
    logits = torch.where(torch.rand(n * beams, v, generator=g, device="cuda") < 0.5, 0.0, -0.0)
    scores = torch.where(torch.arange(n * beams, device="cuda") % 2 == 0, 0.0, -0.0)
    _check(logits.to(dtype), lse, scores, beams, 20)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("order", ["up", "down", "front", "one_thread"])
def test_sorted_and_clustered_rows(order, dtype):
    n, beams, v = 1, 3, 50000
    logits, lse, scores, g = _case(8, n, beams, v, dtype)
    logits = logits.float().sort(1).values
    if order == "down":
        logits = logits.flip(1).contiguous()
    elif order == "front":  # the best of the row lie side by side
        logits = torch.cat([logits[:, -300:], logits[:, :-300]], 1).contiguous()
    elif order == "one_thread":  # the best 8 of every 2048
        logits = torch.full((n * beams, v), -5.0, device="cuda")
        at = torch.arange(v, device="cuda") % 2048 < 8
        logits[:, at] = torch.randn(n * beams, int(at.sum()), generator=g, device="cuda")
    for picks in (3, 64):
        _check(logits.to(dtype), lse, scores, beams, picks)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_masked_infinite_and_nan(dtype):
    n, beams, v = 3, 4, 9000
    logits, lse, scores, g = _case(11, n, beams, v, dtype)
    logits[torch.rand(n * beams, v, generator=g, device="cuda") < 0.99] = -INF
    scores[1] = -INF                     # a beam that does not exist
    logits[5] = -INF                     # a row that the mask leaves empty
    lse[5] = -INF                        # its log-sum-exp: NaN scores
    logits[6] = torch.finfo(dtype).min   # the type's lowest value
    logits[7, 17] = float("nan")
    scores[8:12] = -INF                  # a sequence with nothing left
    for picks in (1, 8, 64):
        _check(logits, lse, scores, beams, picks)
    logits[:] = float("nan")
    _check(logits, lse, scores, beams, 8, 2)
    logits[:] = -INF
    lse[:] = 0.0
    scores[:] = 0.0
    _check(logits, lse, scores, beams, 64, 3)
    logits[2, 100] = INF
    _check(logits, lse, scores, beams, 3)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_infinite_logits_of_rows_that_end_at_minus_infinity(dtype):
    # +inf - inf and +inf + -inf are NaN, the row's other scores are -inf
    n, beams, v = 1, 3, 20000
    logits, lse, scores, g = _case(12, n, beams, v, dtype)
    logits[:, ::7] = INF
    lse[0] = INF
    scores[1] = -INF
    scores[2] = -INF
    lse[2] = INF
    for picks in (1, 10, 64):
        _check(logits, lse, scores, beams, picks, 2)
    logits[:] = INF
    _check(logits, lse, scores, beams, 20)


@pytest.mark.parametrize("col,extra", [(0, 0), (1, 0), (5, 3), (8, 1)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strided_rows(col, extra, dtype):
    n, beams, v = 2, 3, 10007
    logits, lse, scores, _ = _case(col, n, beams, v, dtype)
    wide = torch.full((n * beams, col + v + extra), INF, dtype=dtype, device="cuda")
    wide[:, col:col + v] = logits
    a = vpe.vpe_beam_select(wide, lse, scores, beams, 9, 0, v, shard_rows=v, col_offset=col)
    b = vpe.vpe_beam_select(logits, lse, scores, beams, 9, 0, v)
    assert torch.equal(a, b)


def test_rows_past_two_gib():
    beams, v, ld = 3, 5000, 1_200_000_000
    logits, lse, scores, _ = _case(3, 1, beams, v, BF16)
    wide = torch.empty(beams * ld, dtype=BF16, device="cuda").view(beams, ld)
    wide[:, ld - v:] = logits
    a = vpe.vpe_beam_select(wide, lse, scores, beams, 6, 0, v, shard_rows=v, col_offset=ld - v)
    assert torch.equal(a, vpe.vpe_beam_select(logits, lse, scores, beams, 6, 0, v))


def test_places_use_32_bits():
    # beam 1 of a vocabulary of 2^31 - 1: places end just under 2^32
    beams, vocab, rows = 2, 2 ** 31 - 1, 4000
    logits, lse, scores, _ = _case(4, 1, beams, rows, F32)
    start = vocab - rows
    keys = vpe.vpe_beam_select(logits, lse, scores, beams, 12, start, vocab)
    s, p, t = vpe.vpe_beam_merge([keys], vocab)
    rs, rp, rt = _plain(logits, lse, scores, beams, 12)
    assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(p.cpu().numpy(), rp)
    assert np.array_equal(t.cpu().numpy(), rt + start)


def test_the_same_shard_twice_counts_twice():
    logits, lse, scores, _ = _case(6, 2, 2, 700, F32)
    keys = vpe.vpe_beam_select(logits, lse, scores, 2, 4, 0, 700)
    one = vpe.vpe_beam_merge([keys], 700)
    two = vpe.vpe_beam_merge([keys, keys], 700)
    assert torch.equal(two[2][:, ::2], one[2][:, :2]) and torch.equal(two[2][:, 1::2], one[2][:, :2])


def test_no_sequences():
    z = torch.empty(0, 50, device="cuda")
    e = torch.empty(0, device="cuda")
    keys = vpe.vpe_beam_select(z, e, e, 4, 8, 0, 50)
    s, p, t = vpe.vpe_beam_merge([keys], 50)
    assert s.shape == p.shape == t.shape == (0, 8)
    assert vpe.vpe_beam_reorder(torch.empty(0, 3, device="cuda"), p[:, :4], 4).shape == (0, 3)


# ---------------------------------------------------------------------------
# reordering
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [torch.uint8, BF16, F32, torch.int64])
@pytest.mark.parametrize("outer,n,b_in,b_out,row", [
    (1, 1, 1, 1, 1), (1, 1, 1, 4, 7), (2, 3, 4, 4, 33), (1, 5, 2, 3, 256), (3, 2, 8, 8, 1000),
    (1, 2, 3, 3, 20000), (28, 4, 4, 4, 64), (1, 1000, 3, 2, 5), (2, 1, 64, 64, 257),
])
def test_reorder(outer, n, b_in, b_out, row, dtype):
    g = _gen(outer + n + row)
    state = torch.randint(0, 100, (outer, n * b_in, row), generator=g, device="cuda").to(dtype)
    parents = torch.randint(-1, b_in + 1, (n, b_out + 3), generator=g, device="cuda")[:, :b_out]
    got = vpe.vpe_beam_reorder(state, parents, b_in, dim=1)
    src = parents + b_in * torch.arange(n, device="cuda")[:, None]
    ok = ((parents >= 0) & (parents < b_in)).reshape(-1)
    ref = state[:, torch.where(ok, src.reshape(-1), 0)] * ok[None, :, None].to(dtype)
    assert torch.equal(got, ref)


def test_reorder_unaligned_and_long_rows():
    flat = torch.randint(0, 255, (3 * 1001 * 2 + 16,), device="cuda").to(torch.uint8)
    parents = torch.tensor([[1, 0, 0]], device="cuda")
    for shift in range(0, 9, 2):
        state = flat[shift:shift + 2 * 3003].view(2, 3003)
        got = vpe.vpe_beam_reorder(state, parents, 2)
        assert torch.equal(got, state[parents[0]])
    # rows past byte 2^32
    state = torch.zeros(3, 1_500_000_000, dtype=torch.uint8, device="cuda")
    state[2, -5:] = 7
    got = vpe.vpe_beam_reorder(state, torch.tensor([[2, 1, 2]], device="cuda"), 3)
    assert bool((got[0, -5:] == 7).all()) and bool((got[2, -5:] == 7).all())
    assert not bool(got[1].any()) and not bool(got[0, :-5].any())


def test_beam_search_as_it_is_used():
    """Whole searches over the sharded LM head: lookup, logits with their log-sum-exp,
    selection, reordering, as a captured step replayed, against plain torch."""
    g = _gen(71)
    V, D, tp, n, beams, steps = 600, 64, 2, 3, 4, 5
    rows = V // tp
    table = [(torch.randn(rows, D, generator=g, device="cuda") * 0.5).to(BF16) for _ in range(tp)]
    mix = (torch.randn(D, D, generator=g, device="cuda") * 0.1)
    m = n * beams
    state = torch.zeros(m, D, device="cuda")
    history = torch.zeros(m, steps, dtype=torch.int64, device="cuda")
    scores = torch.full((n, beams), -INF, device="cuda")
    tokens = torch.zeros(m, dtype=torch.int64, device="cuda")
    at = torch.zeros((), dtype=torch.int64, device="cuda")

    def begin():
        state.zero_(), history.zero_(), tokens.zero_(), at.zero_()
        scores.fill_(-INF)
        scores[:, 0] = 0.0
        tokens.view(n, beams).copy_(torch.arange(1, n + 1, device="cuda")[:, None].expand(n, beams))

    def step():
        x = vpe.vpe_sum_partials([vpe.vpe_embed_scaled(tokens, table[r], r * rows, 2.0)
                                  for r in range(tp)])
        state.copy_(torch.tanh(state @ mix + x.float()))
        logits = torch.empty(m, V, dtype=BF16, device="cuda")
        lse = vpe.vpe_logsumexp_combine([
            vpe.vpe_lmhead_logsumexp(state.to(BF16), table[r], logits, col_offset=r * rows)[1]
            for r in range(tp)])
        keys = [vpe.vpe_beam_select(logits, lse, scores.view(-1), beams, 2 * beams, r * rows, V,
                                    shard_rows=rows, col_offset=r * rows) for r in range(tp)]
        s, p, t = vpe.vpe_beam_merge(keys, V)
        ref = _plain_device(logits, lse, scores, n, beams)
        scores.copy_(s[:, :beams])
        tokens.copy_(t[:, :beams].reshape(-1))
        state.copy_(vpe.vpe_beam_reorder(state, p[:, :beams], beams))
        history.copy_(vpe.vpe_beam_reorder(history, p[:, :beams], beams))
        history.scatter_(1, at.expand(m, 1), tokens[:, None])
        at.add_(1)
        return s, p, t, ref

    def _plain_device(logits, lse, scores, n, beams):
        c = (logits.float() - lse[:, None]) + scores.view(-1, 1)
        return c.view(n, beams * V)

    def run(call):
        begin()
        seen = []
        for _ in range(steps):
            s, p, t, cand = call()
            torch.cuda.synchronize()
            top = torch.sort(cand, dim=1, descending=True, stable=True)
            assert torch.equal(s, top.values[:, :2 * beams])
            assert torch.equal(p * V + t, top.indices[:, :2 * beams])
            seen.append((s.clone(), p.clone(), t.clone()))
        return seen, history.clone(), scores.clone()

    eager = run(step)
    # histories hold each survivor's own tokens
    seen, hist, _ = eager
    lines = [[[]] * beams for _ in range(n)]
    for s, p, t in seen:
        lines = [[lines[i][int(p[i, b])] + [int(t[i, b])] for b in range(beams)] for i in range(n)]
    assert hist.view(n, beams, steps).tolist() == lines
    begin()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()

    def replay():
        graph.replay()
        return held

    for _ in range(2):
        again = run(replay)
        assert torch.equal(again[1], eager[1]) and torch.equal(again[2], eager[2])


def test_layer_beam_calls():
    V, D, tp, n, beams = 512, 64, 2, 2, 3
    g = _gen(81)
    heads = [vpe.ParallelLMHead(V, D, tp, r, device=dev()) for r in range(tp)]
    for h in heads:
        h.weight.data.copy_((torch.randn(V // tp, D, generator=g, device="cuda") * 0.1).to(BF16))
    x = torch.randn(n * beams, D, generator=g, device="cuda").to(BF16)
    full = torch.empty(n * beams, V, dtype=BF16, device="cuda")
    lse = vpe.ParallelLMHead.combine_logsumexp([h.logsumexp(x, full)[1] for h in heads])
    scores = -torch.rand(n * beams, generator=g, device="cuda")
    a = [h.beam_select(full, lse, scores, beams, 6) for h in heads]
    b = [h.beam_select(h(x), lse, scores, beams, 6) for h in heads]
    for p, q in zip(a, b):
        assert torch.equal(p, q)
    s, p, t = heads[0].merge_beams(a)
    rs, rp, rt = _plain(full, lse, scores, beams, 6)
    assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(t.cpu().numpy(), rt)
    state = torch.randn(2, n * beams, 5, device="cuda")
    got = heads[0].reorder_beams(state, p[:, :beams], beams, dim=1)
    assert torch.equal(got, vpe.vpe_beam_reorder(state, p[:, :beams], beams, dim=1))


def test_the_most_sequences():
    n, v = 2 ** 21, 3
    logits, lse, scores, _ = _case(81, n, 1, v, F32)
    got = vpe.vpe_beam_merge([vpe.vpe_beam_select(logits, lse, scores, 1, 2, 0, v)], v)
    c = (logits - lse[:, None]) + scores[:, None]
    ref, at = torch.sort(c, dim=1, descending=True, stable=True)
    assert torch.equal(got[0], ref[:, :2]) and torch.equal(got[2], at[:, :2])
    assert not bool(got[1].any())


def test_two_streams_at_once():
    work = [(_case(90 + i, n, beams, v, BF16), beams, v)
            for i, (n, beams, v) in enumerate(((2, 4, 30000), (9, 1, 7000), (1, 16, 50001)))]

    def step(case, beams, v):
        logits, lse, scores, _ = case
        out = vpe.vpe_beam_merge([vpe.vpe_beam_select(logits, lse, scores, beams, 16, 0, v)], v)
        return (*out, vpe.vpe_beam_reorder(logits, out[1], beams))

    ref = [step(*w) for w in work]
    streams = [torch.cuda.Stream() for _ in work]
    torch.cuda.synchronize()
    got = []
    for st, w in zip(streams, work):
        with torch.cuda.stream(st):
            got.append(step(*w))
    torch.cuda.synchronize()
    for a, b in zip(got, ref):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_more_rows_than_one_launch_takes():
    n, v = 32768 + 40, 17001
    logits = torch.randn(n, v, generator=_gen(99), device="cuda", dtype=F32).to(BF16)
    lse, scores = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    got = vpe.vpe_beam_merge([vpe.vpe_beam_select(logits, lse, scores, 1, 5, 0, v)], v)
    for rows in (slice(0, 40), slice(32760, n)):
        ref, at = torch.sort(logits[rows].float(), dim=1, descending=True, stable=True)
        assert torch.equal(got[0][rows], ref[:, :5]) and torch.equal(got[2][rows], at[:, :5])
