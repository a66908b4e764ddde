"""Roundings of the softmax in the loss and its gradients, seen one entry at a time: the
hidden rows are rows of the identity, so that z[i, j] = W[j, i] and the gradient of the
table holds d[i, j] = g_i (exp(z[i, j] - lse_i) - [j = t_i]) itself."""
import pytest
import torch

import vocab_sharded_embedding_amd as vpe
from _loss import HALF, U, assert_within

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
INF = float("inf")
# rows, vocabulary: every width of tiles in bf16 (32, 64, 128, 256) and in fp32
SIZES = [(1, 300), (30, 500), (50, 1000), (120, 2000), (300, 1500), (600, 70000)]


def _identity(m, dtype):
    return torch.eye(m, (m + 63) // 64 * 64, device="cuda").to(dtype)


def _logits(m, vocab, dtype, level, seed):
    """W [vocab, width]: logits around `level`, the target's 8 to 20 above the rest."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.zeros(vocab, (m + 63) // 64 * 64, device="cuda")
    w[:, :m] = level + 2 * torch.randn(vocab, m, generator=g, device="cuda")
    t = torch.randint(0, vocab, (m,), generator=g, device="cuda")
    w[t, torch.arange(m, device="cuda")] = level + 16 + 12 * torch.rand(m, generator=g,
                                                                      device="cuda")
    w = w.to(dtype)
    return w, t, w[:, :m].T.double().contiguous()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("level", [0.0, 20.0, -330.0, 344.0, 5000.0])
@pytest.mark.parametrize("m,vocab", SIZES)
def test_entries_of_the_gradient(m, vocab, level, dtype):
    """An entry's error goes with the distance of its logit from the log-sum-exp, and not
    with their size.

    The difference t = z - lse is rounded (U |t|), its product with log2(e) too (U |t|,
    and 0.25 U |t| for the constant), the exponential is within 2 U of its value more;
    subtracting 1 and the factor round d itself (2 U), and so does `dtype`."""
    w, t, z = _logits(m, vocab, dtype, level, m)
    lse = torch.logsumexp(z, 1).float()
    diff = z - lse.double()[:, None]
    p = torch.exp(diff)
    d = p.clone()
    d[torch.arange(m, device="cuda"), t] -= 1
    # (exponentials below 2^-126 may be flushed)
    err = p * U * (3 * diff.abs() + 4) + 2.0 ** -126
    err = err + (HALF[dtype] + 4 * U) * (d.abs() + err)
    _, gw = vpe.vpe_lmhead_xent_grad(_identity(m, dtype), w, t, lse, torch.ones(m, device="cuda"),
                                     0, vocab, weight_dtype=F32)
    assert_within(gw[:, :m].T, d, err, "d")


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("level", [0.0, -355.9, 355.9, 711.0, 5000.0])
@pytest.mark.parametrize("m,vocab", SIZES)
def test_sums_of_the_loss(m, vocab, level, dtype):
    """The log-sum-exp is its row's maximum, exact, and a logarithm added to it with one
    rounding.  The logarithm's argument is a sum of exponentials of differences: each
    off by U (3 |z - max| + 4) of itself, which is at most 4 U on the sum (x exp(-x) <=
    0.37), n terms added with at most 64 + 16 roundings one behind another in a tile and
    log2(n) + 24 in the joins, each of them with a factor's 4 U."""
    w, t, z = _logits(m, vocab, dtype, level, m)
    want = torch.logsumexp(z, 1)
    got, at = vpe.vpe_lmhead_xent(_identity(m, dtype), w, t, 0, vocab)
    assert torch.equal(at.double(), z[torch.arange(m, device="cuda"), t])
    bound = U * want.abs() + 200 * U + 2 * U * (want - z.max(1).values)
    assert_within(got, want, bound, "shard_lse")


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("m,vocab", SIZES)
def test_logits_next_to_the_largest_float(m, vocab, dtype):
    """Finite logits whose product with log2(e) is not: 3e38, and all of a row's at
    -3e38 but one."""
    w, t, _ = _logits(m, vocab, dtype, 0.0, m)
    row = torch.arange(m, device="cuda")
    big = torch.tensor(3e38, device="cuda").to(dtype).float()
    w[t[::2], row[::2]] = big.to(dtype)
    if m > 1:
        w[:, 1] = -big.to(dtype)
    z = w[:, :m].T.double().contiguous()
    x = _identity(m, dtype)
    a, b = vpe.vpe_lmhead_xent(x, w, t, 0, vocab)
    loss, lse = vpe.vpe_xent_loss([a], [b], t, vocab)
    assert (lse[::2] == big).all() and (loss[::2] == 0).all()
    if m > 1:  # (log of vocab is far below a rounding)
        assert lse[1] == -big and loss[1] == 0
    rest = torch.arange(m, device="cuda")[3::2]
    want = torch.logsumexp(z[rest], 1)
    assert ((lse[rest].double() - want).abs() <= U * want.abs() + 200 * U).all()
    gl = torch.ones(m, device="cuda")
    _, gw = vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, vocab, weight_dtype=F32)
    d = gw[:, :m].T
    assert (d[::2] == 0).all()
    if m > 1:  # every difference is 0
        one = torch.zeros(vocab, device="cuda")
        one[t[1]] = 1
        assert torch.equal(d[1], 1 - one)
    p = torch.exp(z[rest] - lse[rest].double()[:, None])
    p[torch.arange(rest.numel(), device="cuda"), t[rest]] -= 1
    assert ((d[rest].double() - p).abs() <= (HALF[dtype] + 100 * U) * p.abs() + 100 * U).all()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_infinite_sums_follow_the_formula(dtype):
    """A log-sum-exp of +inf leaves exponentials of 0, one of -inf those of +inf, and
    neither touches another row."""
    m, vocab = 40, 900
    w, t, z = _logits(m, vocab, dtype, 3.0, 1)
    x, gl = _identity(m, dtype), torch.ones(m, device="cuda")
    lse = torch.logsumexp(z, 1).float()
    _, want = vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, vocab, weight_dtype=F32)
    lse[5], lse[11] = INF, -INF
    gx, _ = vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, vocab, x_dtype=F32, with_weight=False)
    assert torch.equal(gx[5], -w[t[5]].float())
    assert not torch.isfinite(gx[11]).any()
    lse[11] = INF
    _, got = vpe.vpe_lmhead_xent_grad(x, w, t, lse, gl, 0, vocab, weight_dtype=F32)
    keep = [i for i in range(m) if i not in (5, 11)]
    assert torch.equal(got[:, keep], want[:, keep])
    for i in (5, 11):
        assert got[t[i], i] == -1 and (got[:, i] != 0).sum() == 1
