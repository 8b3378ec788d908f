"""The training step of examples/train_step.py: it runs, and its gradients are those of the same step in
64 bits (torch's derivatives of the plain form).

Bound: fp32 sums in five operators in a row, each off by some 2^-24 times the terms' norm (sqrt(K) of
them at most, K <= 500), and the gradients' two ways through the block: 1e-4 of the norm holds all of it; bf16
rounds about ten times on the way, 2^-9 of the value in the mean each: 5e-2.
"""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def _plain_loss(w, x, tokens, k, topk_idx, entropy_share):
    """The block and its loss; the selected experts are given (their choice has no derivative)."""
    def norm(s, name):
        mean = s.mean(1, keepdim=True)
        return (s - mean) / torch.sqrt(((s - mean) ** 2).mean(1, keepdim=True) + 1e-5) * w[name + ".w"] + w[name + ".b"]

    def network(rows, w13, w2):
        a, b = (rows @ w13.T).chunk(2, -1)
        return (a * torch.sigmoid(a) * b) @ w2.T

    h = norm(x, "norm_in")
    scores = (h @ w["w_r"]).gather(1, topk_idx)
    gates = torch.softmax(scores, 1)
    y = sum(network(h, w["ws13"][i], w["ws2"][i]) for i in range(w["ws13"].shape[0]))
    for e in range(w["w13"].shape[0]):
        t, j = (topk_idx == e).nonzero(as_tuple=True)
        y = y.index_add(0, t, gates[t, j][:, None] * network(h[t], w["w13"][e], w["w2"][e]))
    logp = torch.log_softmax(norm(y + x, "norm_out") @ w["head"].T, 1)
    counts = (tokens >= 0).double()
    lp = logp.gather(1, tokens.clamp(min=0).long()[:, None])[:, 0]
    ent = -(logp.exp() * logp).sum(1)
    return -((lp + entropy_share * ent) * counts).sum() / counts.sum()


@pytest.mark.parametrize("dtype,bound", [(torch.float32, 1e-4), (torch.bfloat16, 5e-2)])
@pytest.mark.parametrize("T", [24, 129])
def test_gradients_of_a_step(T, dtype, bound):
    import train_step as ex
    d, vocab, k = 128, 500, 2
    block = ex.TrainBlock(T, d=d, E=5, k=k, f=64, S=2, vocab=vocab, dtype=dtype, seed=T)
    for n in (block.norm_in, block.norm_out):
        n.weight.add_(0.2 * torch.randn_like(n.weight))
        n.bias.add_(0.1 * torch.randn_like(n.bias))
    x, tokens = ex.inputs(T, d=d, vocab=vocab, dtype=dtype)
    out = block.forward(x, tokens)
    loss = -((out["logprob"] + ex.ENTROPY * out["entropy"]) * (tokens >= 0)).sum() / (tokens >= 0).sum()
    grads = block.backward(tokens)
    w = {n: t.detach().cpu().double().requires_grad_(True) for n, t in block.weights().items()}
    x64 = x.cpu().double().requires_grad_(True)
    want = _plain_loss(w, x64, tokens.cpu(), k, block.layer.saved["topk_idx"].cpu().long(), ex.ENTROPY)
    want.backward()
    want = float(want.detach())
    assert abs(float(loss) - want) <= bound * abs(want)
    for name, ref in {**{n: t.grad for n, t in w.items()}, "x": x64.grad}.items():
        got = grads[name].cpu().double()
        assert float((got - ref).norm()) <= bound * float(ref.norm()), name


def test_steps_with_clipping():
    """The clipped gradients have the limit's norm, the weights move by them, and every step's norm is that of
    the gradients then."""
    import train_step as ex
    T = 200
    block = ex.TrainBlock(T, d=128, f=64, vocab=700, dtype=torch.float32)
    x, tokens = ex.inputs(T, d=128, vocab=700, dtype=torch.float32)
    for _ in range(3):
        before = {n: t.clone() for n, t in block.weights().items()}
        loss, norm = block.step(x, tokens, rate=0.5, max_norm=0.25)
        assert bool(torch.isfinite(loss)) and float(norm) > 0.25
        moved = sum(float(((t - before[n]).double() ** 2).sum()) for n, t in block.weights().items()) ** 0.5
        # fp32 weights of size 1 keep 2^-24 of themselves: 3e5 of them lose 2^-25 sqrt(3e5) = 2e-5 of a step
        assert abs(moved - 0.5 * 0.25) <= 1e-3 * 0.125
