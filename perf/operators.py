"""Training and beam-search operators of the vocabulary-sharded layers: the
cases they are timed on, their plain forms, and their values in 64 bits.

Operators:
  embed       lookup in one rank's table shard, times a factor
  embed_grad  gradient of that lookup with respect to the shard
  distill     loss against a teacher's top logits, from the logits' shards, and
              its gradient with respect to them: a training step's part
  distill_grad  the gradient alone, on one rank's shard
  beam        one step of beam search: selection over beams and vocabulary
              from the logits' shards, then the reordering of the states

With `own` false `run` uses elementary torch operations in fp32; with `own`
true it calls the library.  `rank` -1 stands for all tp ranks held on one
device, their logits side by side in one [rows, vocab] buffer.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "i32": torch.int32, "i64": torch.int64}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a decode step's lookup for 16 running sequences: latency
        dict(name="embed_decode_16", op="embed", n=16, vocab=151936, tp=2, rank=0, dim=1024,
             dtype="bf16", itype="i32", dist="uniform"),
        # a training batch on one of four ranks, hidden 4096: bandwidth
        dict(name="embed_train_131072", op="embed", n=131072, vocab=151936, tp=4, rank=2,
             dim=4096, dtype="bf16", itype="i32", dist="uniform"),
        # the tiny fp32 configuration: latency of the whole gradient
        dict(name="embed_grad_tiny_f32", op="embed_grad", n=257, vocab=4096, tp=2, rank=1, dim=64,
             dtype="f32", gdtype="f32", itype="i64", dist="uniform"),
        # one micro-batch on a rank of two: most rows of the shard get zeros
        dict(name="embed_grad_8192", op="embed_grad", n=8192, vocab=151936, tp=2, rank=0,
             dim=1024, dtype="bf16", gdtype="bf16", itype="i32", dist="uniform"),
        # natural text (Zipf): a few tokens hold thousands of positions; fp32 gradient
        dict(name="embed_grad_zipf_65536", op="embed_grad", n=65536, vocab=151936, tp=1, rank=0,
             dim=1024, dtype="bf16", gdtype="f32", itype="i32", dist="zipf"),
        # a few short sequences against the whole vocabulary on one rank
        dict(name="distill_8x151936_f32", op="distill", rows=8, vocab=151936, tp=1, rank=-1, k=20,
             dtype="f32", tdtype="f32", itype="i64", temperature=2.0, tail=False),
        # both ranks of two on one device, teacher's mass beyond its top logits left out
        dict(name="distill_1024_tp2", op="distill", rows=1024, vocab=151936, tp=2, rank=-1, k=64,
             dtype="bf16", tdtype="bf16", itype="i32", temperature=1.0, tail=True),
        # one rank's logits gradient, an odd number of rows and entries
        dict(name="distill_grad_251", op="distill_grad", rows=251, vocab=151936, tp=2, rank=1,
             k=51, dtype="bf16", tdtype="f32", itype="i64", temperature=1.5, tail=False),
        # a training batch on one of four ranks
        dict(name="distill_grad_4096", op="distill_grad", rows=4096, vocab=151936, tp=4, rank=2,
             k=128, dtype="bf16", tdtype="bf16", itype="i32", temperature=2.0, tail=True),
        # one request, first step (only beam 0 lives), whole vocabulary on one rank: latency
        dict(name="beam_first_1x4", op="beam", seqs=1, beams=4, picks=8, vocab=151936, tp=1,
             dtype="bf16", layers=4, width=1024, table=64, first=True),
        # a serving batch, logits of two ranks
        dict(name="beam_32x8_tp2", op="beam", seqs=32, beams=8, picks=16, vocab=151936, tp=2,
             dtype="bf16", layers=28, width=2048, table=257, first=False),
        # wide beams with fp32 logits
        dict(name="beam_5x32_f32", op="beam", seqs=5, beams=32, picks=64, vocab=50257, tp=1,
             dtype="f32", layers=3, width=1001, table=33, first=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "distill", "distill_grad", "beam"])
    tp = rng.choice([1, 2, 3, 4])
    vocab = rng.choice([_log_int(rng, 4096 // tp, 151936 // tp) * tp, 151936 // tp * tp])
    dt = rng.choice(["bf16", "bf16", "f32"])
    it = rng.choice(["i32", "i64"])
    if op in ("embed", "embed_grad"):
        dim = rng.choice([64, 256, 1024, 2048, 4096, _log_int(rng, 8, 4096)])
        dim = min(dim, 155_600_000 // (vocab // tp))
        n = _log_int(rng, 1, min(131072, (131072 * 1024) // dim))
        case = dict(op=op, n=n, vocab=vocab, tp=tp, rank=rng.randrange(tp), dim=dim, dtype=dt,
                    itype=it, dist=rng.choice(["uniform", "zipf"]))
        if op == "embed_grad":
            case["gdtype"] = rng.choice([dt, "f32"])
        return case
    if op in ("distill", "distill_grad"):
        rank = rng.randrange(tp) if op == "distill_grad" else -1
        width = vocab if rank < 0 else vocab // tp
        rows = _log_int(rng, 1, max(2, min(4096, 60_000_000 // width)))
        return dict(op=op, rows=rows, vocab=vocab, tp=tp, rank=rank, k=_log_int(rng, 1, 256),
                    dtype=dt, tdtype=rng.choice(["f32", "bf16"]), itype=it,
                    temperature=rng.choice([1.0, 2.0, round(rng.uniform(0.5, 4.0), 2)]),
                    tail=rng.random() < 0.5)
    beams = _log_int(rng, 1, 32)
    seqs = _log_int(rng, 1, max(1, min(64, 35_000_000 // (vocab * beams))))
    return dict(op="beam", seqs=seqs, beams=beams, picks=2 * beams, vocab=vocab, tp=tp, dtype=dt,
                layers=rng.choice([1, 4, 28]), width=_log_int(rng, 16, 2048),
                table=_log_int(rng, 1, 512), first=rng.random() < 0.2)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _token_ids(case, g):
    """Ids of the whole vocabulary: uniform, or Zipf (s = 1.1) over a fixed shuffle of the ids."""
    n, v = case["n"], case["vocab"]
    if case["dist"] == "uniform":
        ids = torch.randint(0, v, (n,), generator=g, device="cuda")
    else:
        w = torch.arange(1, v + 1, device="cuda", dtype=torch.float64) ** -1.1
        cdf = torch.cumsum(w, 0)
        u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64) * cdf[-1]
        rank = torch.searchsorted(cdf, u).clamp_(max=v - 1)
        ids = torch.randperm(v, generator=g, device="cuda")[rank]
    return ids.to(DTYPES[case["itype"]])


def _prepare_embed(case, g):
    rows, dim = case["vocab"] // case["tp"], case["dim"]
    s = dict(case=case, ids=_token_ids(case, g), start=case["rank"] * rows, rows=rows,
             scale=math.sqrt(dim))
    if case["op"] == "embed":
        s["weight"] = (_randn(g, rows, dim) * 0.02).to(DTYPES[case["dtype"]])
    else:
        s["grad_out"] = (_randn(g, case["n"], dim) * 1e-2).to(DTYPES[case["dtype"]])
    return s


def _prepare_distill(case, g):
    m, v, k, tp, rank = case["rows"], case["vocab"], case["k"], case["tp"], case["rank"]
    rows = v // tp
    start, width = (0, v) if rank < 0 else (rank * rows, rows)
    # the teacher's ids are distinct within a row; its logits fall with their rank
    base = torch.randint(0, v, (m, 1), generator=g, device="cuda")
    step = torch.randint(1, max(2, v // k), (m, 1), generator=g, device="cuda")
    ids = (base + step * torch.arange(k, device="cuda")) % v
    t = 9.0 + 2.0 * _randn(g, m, k)
    t = torch.sort(t, dim=1, descending=True).values
    # the student agrees with the teacher up to noise on the teacher's ids
    z = 2.0 * _randn(g, m, width)
    local = ids - start
    near = t + _randn(g, m, k)
    spare = torch.cat([z, z.new_zeros(m, 1)], 1)
    spare.scatter_(1, torch.where((local >= 0) & (local < width), local, width), near)
    logits = spare[:, :width].to(DTYPES[case["dtype"]]).contiguous()
    del spare, z
    # some rows have fewer entries, and the last ones (padding of the batch) none
    count = torch.where(torch.rand(m, generator=g, device="cuda") < 0.1,
                        torch.randint(1, k + 1, (m,), generator=g, device="cuda"),
                        torch.full((m,), k, device="cuda"))
    count[m - m // 16:] = 0
    ids = torch.where(torch.arange(k, device="cuda") < count[:, None], ids, -1)
    teacher = t.to(DTYPES[case["tdtype"]])
    temp = case["temperature"]
    tail = None
    if case["tail"]:
        kept = torch.where(ids >= 0, teacher.float() / temp, float("-inf"))
        tail = torch.logsumexp(kept, 1).clamp_(min=-1e4)
        tail = (tail + 0.3 * torch.rand(m, generator=g, device="cuda")).contiguous()
    s = dict(case=case, logits=logits, ids=ids.to(DTYPES[case["itype"]]).contiguous(),
             teacher=teacher, tail=tail, start=start, rows=rows)
    s["grad_loss"] = torch.full((m,), temp * temp / m, device="cuda")
    if case["op"] == "distill_grad":
        lse = torch.cat([torch.logsumexp(c.float() / temp, 1) for c in logits.split(256)])
        s["lse"] = lse + math.log(tp)  # the other ranks' columns are like this one's
    return s


def _prepare_beam(case, g):
    b, v = case["beams"], case["vocab"]
    m = case["seqs"] * b
    z = 2.5 * _randn(g, m, v)
    z[:, torch.randint(0, v, (v // 100 + 1,), generator=g, device="cuda")] = float("-inf")
    logits = z.to(DTYPES[case["dtype"]])
    del z
    lse = torch.cat([torch.logsumexp(c.float(), 1) for c in logits.split(256)])
    scores = -20.0 * torch.rand(case["seqs"], b, generator=g, device="cuda")
    scores = torch.sort(scores, dim=1, descending=True).values
    if case["first"]:
        scores[:, 1:] = float("-inf")
    return dict(case=case, logits=logits, lse=lse, scores=scores.reshape(-1).contiguous(),
                rows=v // case["tp"],
                state=_randn(g, case["layers"], m, case["width"]).to(torch.bfloat16),
                table=torch.randint(0, 1 << 20, (m, case["table"]), generator=g, device="cuda",
                                    dtype=torch.int32))


def prepare(case, seed):
    g = _gen(seed)
    if case["op"].startswith("embed"):
        return _prepare_embed(case, g)
    if case["op"].startswith("distill"):
        return _prepare_distill(case, g)
    return _prepare_beam(case, g)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _plain_embed(s):
    local = s["ids"].long() - s["start"]
    owned = (local >= 0) & (local < s["rows"])
    y = s["weight"][torch.where(owned, local, 0)].float() * s["scale"]
    return torch.where(owned[:, None], y, 0.0).to(s["weight"].dtype)


def _plain_embed_grad(s):
    local = s["ids"].long() - s["start"]
    owned = (local >= 0) & (local < s["rows"])
    spare = torch.where(owned, local, s["rows"])
    dw = torch.zeros(s["rows"] + 1, s["grad_out"].shape[1], device="cuda")
    dw.index_add_(0, spare, s["grad_out"].float())
    return (dw[:s["rows"]] * s["scale"]).to(DTYPES[s["case"]["gdtype"]])


def _plain_teacher(s):
    """Entries that count, their probabilities and their logarithms (0 where none)."""
    ids = s["ids"].long()
    valid = (ids >= 0) & (ids < s["case"]["vocab"])
    t = torch.where(valid, s["teacher"].float() / s["case"]["temperature"], float("-inf"))
    if s["tail"] is None:
        top = torch.clamp(t.max(1, keepdim=True).values, min=-3e38)
        norm = top + torch.log(torch.exp(t - top).sum(1, keepdim=True))
    else:
        norm = s["tail"][:, None]
    logp = torch.where(valid, t - norm, float("-inf"))
    p = torch.exp(logp)
    return ids, p, torch.where(p > 0, logp, 0.0)


def _plain_distill(s):
    ids, p, logp = _plain_teacher(s)
    t = s["case"]["temperature"]
    z = s["logits"].float() / t
    top = z.max(1, keepdim=True).values
    lse = top + torch.log(torch.exp(z - top).sum(1, keepdim=True))
    zk = torch.gather(z, 1, torch.where(p > 0, ids, 0))
    loss = torch.where(p > 0, p * (logp - (zk - lse)), 0.0).sum(1)
    return loss, lse[:, 0], _plain_logits_grad(s, z, lse, ids, p)


def _plain_distill_grad(s):
    ids, p, _ = _plain_teacher(s)
    z = s["logits"].float() / s["case"]["temperature"]
    return _plain_logits_grad(s, z, s["lse"][:, None], ids, p)


def _plain_logits_grad(s, z, lse, ids, p):
    q = torch.exp(z - lse) * p.sum(1, keepdim=True)
    local = ids - s["start"]
    here = (local >= 0) & (local < z.shape[1])
    q.scatter_add_(1, torch.where(here, local, 0), torch.where(here, -p, 0.0))
    return (q * (s["grad_loss"] / s["case"]["temperature"])[:, None]).to(s["logits"].dtype)


def _plain_beam(s):
    c = s["case"]
    n, b, v = c["seqs"], c["beams"], c["vocab"]
    cand = (s["logits"].float() - s["lse"][:, None]) + s["scores"][:, None] + 0.0
    cand = cand.reshape(n, b * v)
    # one key per candidate: ordered by score, then by the lower place; NaN last
    bits = cand.view(torch.int32).long()
    order = torch.where(bits < 0, -(bits & 0x7FFFFFFF) - 1, bits)
    order = torch.where(torch.isnan(cand), -(1 << 31), order)
    key = (order << 32) + (0xFFFFFFFF - torch.arange(b * v, device="cuda"))
    place = torch.topk(key, c["picks"], dim=1).indices
    scores = torch.gather(cand, 1, place)
    parent, token = place // v, place % v
    src = (parent[:, :b] + b * torch.arange(n, device="cuda")[:, None]).reshape(-1)
    return scores, parent, token, s["state"][:, src], s["table"][src]


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _own(s):
    import vocab_sharded_embedding_amd as vpe
    c = s["case"]
    if c["op"] == "embed":
        return vpe.vpe_embed_scaled(s["ids"], s["weight"], s["start"], s["scale"])
    if c["op"] == "embed_grad":
        return vpe.vpe_embed_grad(s["ids"], s["grad_out"], s["start"], s["rows"], s["scale"],
                                  dtype=DTYPES[c["gdtype"]])
    if c["op"] == "distill":
        t, v, ranks = c["temperature"], c["vocab"], range(c["tp"])
        shards = [vpe.vpe_distill_shard(s["logits"], s["ids"], s["teacher"], r * s["rows"], v,
                                        temperature=t, teacher_lse=s["tail"],
                                        shard_rows=s["rows"], col_offset=r * s["rows"])
                  for r in ranks]
        loss, lse = vpe.vpe_distill_loss([a for a, _ in shards], [b for _, b in shards], s["ids"],
                                         s["teacher"], v, temperature=t, teacher_lse=s["tail"])
        grad = torch.empty_like(s["logits"])
        for r in ranks:
            vpe.vpe_distill_grad(s["logits"], lse, s["grad_loss"], s["ids"], s["teacher"],
                                 r * s["rows"], v, temperature=t, teacher_lse=s["tail"],
                                 shard_rows=s["rows"], col_offset=r * s["rows"],
                                 grad_logits=grad)
        return loss, lse, grad
    if c["op"] == "distill_grad":
        return vpe.vpe_distill_grad(s["logits"], s["lse"], s["grad_loss"], s["ids"], s["teacher"],
                                    s["start"], c["vocab"], temperature=c["temperature"],
                                    teacher_lse=s["tail"])
    keys = [vpe.vpe_beam_select(s["logits"], s["lse"], s["scores"], c["beams"], c["picks"],
                                r * s["rows"], c["vocab"], shard_rows=s["rows"],
                                col_offset=r * s["rows"]) for r in range(c["tp"])]
    scores, parent, token = vpe.vpe_beam_merge(keys, c["vocab"])
    # the first `beams` picks live on
    state = vpe.vpe_beam_reorder(s["state"], parent[:, :c["beams"]], c["beams"], dim=1)
    table = vpe.vpe_beam_reorder(s["table"], parent[:, :c["beams"]], c["beams"])
    return scores, parent, token, state, table


PLAIN = dict(embed=_plain_embed, embed_grad=_plain_embed_grad, distill=_plain_distill,
             distill_grad=_plain_distill_grad, beam=_plain_beam)


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _owned(case):
    """Expected owned ids, and expected distinct ones among them."""
    n, v, tp = case["n"], case["vocab"], case["tp"]
    p = np.full(v, 1.0 / v)
    if case["dist"] == "zipf":
        p = np.arange(1, v + 1, dtype=np.float64) ** -1.1
        p /= p.sum()
    return n / tp, float((-np.expm1(n * np.log1p(-p))).sum()) / tp


def work(case):
    size = {"f32": 4, "bf16": 2, "i32": 4, "i64": 8}
    op, e = case["op"], size[case["dtype"]]
    if op.startswith("embed"):
        owned, distinct = _owned(case)
        ids, row = case["n"] * size[case["itype"]], case["dim"] * e
        if op == "embed":
            return dict(bytes=ids + distinct * row + case["n"] * row, flops=owned * case["dim"])
        dw = case["vocab"] // case["tp"] * case["dim"] * size[case["gdtype"]]
        return dict(bytes=ids + owned * row + dw, flops=2 * owned * case["dim"])
    if op.startswith("distill"):
        m = case["rows"]
        width = case["vocab"] // (1 if case["rank"] < 0 else case["tp"])
        teacher = m * case["k"] * (size[case["itype"]] + size[case["tdtype"]])
        live = m - m // 16  # rows without entries need no logits for their gradient
        reads, flops = live * width, 5 * live * width
        if op == "distill":  # the log-sum-exp of every row is an output
            reads, flops = m * width, flops + 4 * m * width
        return dict(bytes=(reads + m * width) * e + teacher + 12 * m, flops=flops)
    m = case["seqs"] * case["beams"]
    moved = 2 * m * (case["layers"] * case["width"] * 2 + case["table"] * 4)
    return dict(bytes=m * case["vocab"] * e + 8 * m + 20 * case["seqs"] * case["picks"] + moved,
                flops=3 * m * case["vocab"])


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_teacher(s):
    ids = s["ids"].long()
    counts = (ids > -1) & (ids < s["case"]["vocab"])
    t = s["teacher"].double() / s["case"]["temperature"]
    w = torch.where(counts, torch.exp(t), 0.0)
    total = w.sum(1, keepdim=True) if s["tail"] is None else torch.exp(s["tail"].double())[:, None]
    return ids, torch.where(w > 0, w / total, 0.0)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "embed":
        lo, hi = s["start"], s["start"] + s["rows"]
        mine = ((s["ids"] >= lo) & (s["ids"] < hi)).nonzero()[:, 0]
        out = torch.zeros(case["n"], case["dim"], dtype=torch.float64, device="cuda")
        out[mine] = s["weight"].double()[s["ids"][mine].long() - lo] * s["scale"]
        return out
    if op == "embed_grad":
        # rows sorted by token, running sums, differences at the tokens' ends
        lo, hi = s["start"], s["start"] + s["rows"]
        mine = ((s["ids"] >= lo) & (s["ids"] < hi)).nonzero()[:, 0]
        row, by = torch.sort(s["ids"][mine].long() - lo)
        out = torch.zeros(s["rows"], case["dim"], dtype=torch.float64, device="cuda")
        if mine.numel():
            which, count = torch.unique_consecutive(row, return_counts=True)
            end = torch.cumsum(count, 0)
            for c in range(0, case["dim"], 256):
                run_sum = torch.cumsum(s["grad_out"][mine[by], c:c + 256].double(), 0)[end - 1]
                run_sum[1:] = run_sum[1:] - run_sum[:-1].clone()
                out[which, c:c + 256] = run_sum * s["scale"]
        return out
    if op.startswith("distill"):
        ids, p = _exact_teacher(s)
        temp, lo, width = case["temperature"], s["start"], s["logits"].shape[1]
        here = (ids >= lo) & (ids < lo + width)
        at = torch.where(here, ids - lo, 0)
        outs = []
        for i in range(0, case["rows"], 256):
            j = slice(i, i + 256)
            z = s["logits"][j].double() / temp
            pk = torch.where(here[j], p[j], 0.0)
            lse = torch.logsumexp(z, 1) if op == "distill" else s["lse"][j].double()
            d = p[j].sum(1, keepdim=True) * torch.exp(z - lse[:, None])
            d.scatter_add_(1, at[j], -pk)
            d = d * s["grad_loss"][j].double()[:, None] / temp
            loss = torch.xlogy(pk, pk) - pk * (torch.gather(z, 1, at[j]) - lse[:, None])
            outs.append((loss.sum(1), lse, d))
        whole = tuple(torch.cat(o) for o in zip(*outs))
        return whole[2] if op == "distill_grad" else whole
    v = case["vocab"]
    best = []
    for i in range(case["seqs"]):
        j = slice(i * case["beams"], (i + 1) * case["beams"])
        cand = s["logits"][j].double() + (s["scores"][j].double() - s["lse"][j].double())[:, None]
        best.append(torch.sort(cand.reshape(-1), descending=True).values[:case["picks"]])
    return torch.stack(best), None, None, None, None
