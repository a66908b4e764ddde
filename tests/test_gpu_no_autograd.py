"""The layers' calls build no autograd graph, whatever requires a gradient: the
gradients are calls of their own."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a HIP GPU"),
]

import vocab_sharded_embedding_amd as vpe  # noqa: E402


def test_outputs_do_not_require_gradients():
    emb = vpe.VocabParallelEmbedding(96, 32, dtype=torch.float32, device="cuda")
    emb.weight.data.normal_()
    emb.weight.requires_grad_(True)
    ids = torch.randint(0, 96, (7,), device="cuda")
    assert not emb(ids, scale=2.0).requires_grad and not emb(ids).requires_grad
    head = vpe.ParallelLMHead(96, 32, dtype=torch.float32, device="cuda")
    logits = torch.randn(7, 96, device="cuda", requires_grad=True)
    top = torch.randn(7, 3, device="cuda", requires_grad=True)
    top_ids = torch.randint(0, 96, (7, 3), device="cuda")
    lse, dot = head.distill_shard(logits, top_ids, top)
    loss, whole = head.distill_loss([lse], [dot], top_ids, top)
    assert not any(t.requires_grad for t in (lse, dot, loss, whole))
    grad = head.distill_grad(logits, whole, torch.ones(7, device="cuda"), top_ids, top)
    # what autograd gives for the same loss
    p = torch.softmax(top.detach(), 1)
    ref = torch.softmax(logits.detach(), 1).scatter_add(1, top_ids, -p)
    # fp32 probabilities of at most 1: 32 roundings of each side are plenty
    assert bool(((grad - ref).abs() <= 64 * 2.0 ** -24).all())
