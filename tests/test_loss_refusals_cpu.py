"""Calls of the loss boundary that documentation refuses, each by itself, without a GPU
(the calls never reach a kernel launch)."""
import pytest

torch = pytest.importorskip("torch")

import vocab_sharded_embedding_amd as vpe  # noqa: E402


@pytest.fixture
def calls(monkeypatch):
    """Calls that the library would get, from tensors in host memory."""
    got = []
    monkeypatch.setattr(vpe.loss, "placed", lambda names, *tensors: 0)
    monkeypatch.setattr(vpe.loss, "enqueue", lambda name, *args: got.append(name))
    return got


@pytest.mark.parametrize("apart", [True, False], ids=["into_others", "in_place"])
def test_norm_inside_a_gradient(calls, apart):
    """The norm is written while gradients are read: it may lie in none of them, in
    place or not."""
    pool = torch.zeros(64)
    grads = [pool[8:24], pool[32:33], pool[40:40]]
    out = [torch.zeros(16), torch.zeros(1), torch.zeros(0)] if apart else None
    sumsq = [torch.zeros(1, dtype=torch.float64) for _ in range(2)]

    def clip(at):
        return vpe.vpe_grad_clip(grads, sumsq, 1.0, out=out, norm=pool[at:at + 1])

    for at in (8, 9, 23, 32):
        with pytest.raises(ValueError, match="overlap|apart"):
            clip(at)
    assert not calls
    for at in (7, 24, 31, 33, 40):  # neighbours, and where a tensor of no elements is
        assert clip(at).item() == 0
    assert calls == ["vpe_grad_clip"] * 5
    inside = sumsq[1].view(torch.float32)
    for norm in (inside[:1], inside[1:]):
        with pytest.raises(ValueError, match="overlap|apart"):
            vpe.vpe_grad_clip(grads, sumsq, 1.0, out=out, norm=norm)
    if apart:
        with pytest.raises(ValueError, match="overlap|apart"):
            vpe.vpe_grad_clip(grads, sumsq, 1.0, out=out, norm=out[0][3:4])
    # gradients may be read from one place twice, where nothing is written there
    if apart:
        vpe.vpe_grad_clip([grads[0], grads[0]], sumsq, 1.0, out=[out[0], torch.zeros(16)],
                          norm=torch.zeros(1))
