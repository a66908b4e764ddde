"""The head's cross entropy and its gradients in 64 bits, with bounds on what the
library's roundings may do, for the GPU tests."""
import torch

# half a step, relative to the value
HALF = {t: torch.finfo(t).eps / 2 for t in (torch.float32, torch.bfloat16)}
U = 2.0 ** -24


class Reference:
    """x, weight, targets, grad_loss on any device; everything in float64.

    A product of two bf16 or fp32 values summed in fp32 over n terms is off by at
    most n half-steps of the sum of the terms' magnitudes (plus the fp32 products'
    own); `zerr` is that for the logits.  The exponentials' arguments carry that,
    the rounding of the multiplication by log2(e) and of the subtraction of the
    maximum or the log-sum-exp (a few half-steps of their size), v_exp_f32 and
    logf two more, and a sum of n non-negative terms n half-steps at most."""

    def __init__(self, x, weight, targets, vocab, grad_loss=None):
        self.dtype = x.dtype
        self.x, self.w = x.double(), weight.double()
        t = targets.long()
        m, n = self.x.shape[0], self.w.shape[0]
        self.live = (t >= 0) & (t < vocab)
        if grad_loss is not None:
            self.used = self.live & (grad_loss != 0)
        else:
            self.used = self.live
        self.x = torch.where(self.live[:, None], self.x, 0.0)
        z = self.x @ self.w.T
        mag = self.x.abs() @ self.w.abs().T
        self.zerr = (self.x.shape[1] + 2) * U * mag.max(1).values
        self.lse = torch.logsumexp(z, 1)
        at = torch.where(self.live, t, 0)[:, None]
        self.zt = torch.gather(z, 1, at)[:, 0]
        size = z.abs().max(1).values + self.lse.abs()
        # terms below 2^-126 may be flushed: no more than n 2^-126 of a sum >= 1
        self.arg = self.zerr + 8 * U * (size + 1)
        self.lse_err = self.arg + (n + 16) * U + 4 * U * self.lse.abs()
        self.loss = torch.where(self.live, self.lse - self.zt, 0.0)
        self.loss_err = torch.where(
            self.live, self.lse_err + self.zerr + 4 * U * (self.lse.abs() + self.zt.abs()), 0.0)
        self.lse = torch.where(self.live, self.lse, 0.0)
        if grad_loss is None:
            return
        g = torch.where(self.used, grad_loss.double(), 0.0)[:, None]
        p = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
        e = p * (self.arg + self.lse_err)[:, None] * 1.01 + 8 * U * p
        one = torch.zeros_like(p)
        one.scatter_(1, at, self.live.double()[:, None])
        self.d = g * (p - one)
        # the kept entry: factor over the largest one, product, (bf16) rounding
        self.derr = g.abs() * e + (4 * U + HALF[self.dtype]) * (self.d.abs() + g.abs() * e)
        self.derr = self.derr + g.abs() * one * 2 * U

    def grads(self, rows, x_dtype, w_dtype, base=None):
        """(grad_x, its bound, grad_weight, its bound) of the shard `rows`."""
        return products(self.d[:, rows], self.derr[:, rows], self.x, self.w[rows], x_dtype,
                        w_dtype, base)


def products(d, derr, x, w, x_dtype, w_dtype, base=None):
    """(d W, bound, d^T x, bound), sums in fp32 and one rounding; `base` is added
    to the second before it."""
    gx, gw = d @ w, d.T.contiguous() @ x
    n, m = d.shape[1], d.shape[0]
    # every sum of partial sums adds its own half-steps: 64 covers the joins
    xerr = derr @ w.abs() + (n + 64) * U * ((d.abs() + derr) @ w.abs())
    werr = derr.T.contiguous() @ x.abs()
    werr = werr + (m + 64) * U * ((d.abs() + derr).T.contiguous() @ x.abs())
    if base is not None:
        gw = gw + base.double()
        werr = werr + 2 * U * gw.abs()
    tiny = 1e-37  # results below fp32's normal range
    xerr = xerr + (HALF[x_dtype] + 2 * U) * (gx.abs() + xerr) + tiny
    werr = werr + (HALF[w_dtype] + 2 * U) * (gw.abs() + werr) + tiny
    return gx, xerr, gw, werr


def assert_within(got, want, bound, what):
    over = (got.double() - want).abs() - bound
    assert not torch.isnan(over).any(), f"{what}: NaN"
    worst = over.max().item() if over.numel() else 0.0
    assert worst <= 0, (f"{what}: {int((over > 0).sum())} of {over.numel()} past the bound, by "
                        f"{worst:.3g}")
