"""One training step of an MoE block and its head, on one GPU.

x -> layer norm -> MoE layer -> (+ x) layer norm -> head -> log probabilities of the next tokens; the loss is
their negative mean over the tokens that count, less a little of the entropy. All gradients are
clipped by their global norm and the weights take a step of plain descent.

    python examples/train_step.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from dropless_token_routing_gb300.api import GradClipper, LayerNorm, LayerParams, Linear, MoELayer, TokenLogprobs  # noqa: E402

ENTROPY = 0.01   # the loss's share of the entropy


class TrainBlock:
    def __init__(self, T, d=256, E=8, k=2, f=128, S=1, vocab=2000, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape, dt=dtype):
            return torch.randn(*shape, generator=g, device="cuda", dtype=dt) * shape[-1] ** -0.5

        ones, zeros = torch.ones(d, dtype=dtype, device="cuda"), torch.zeros(d, dtype=dtype, device="cuda")
        self.norm_in = LayerNorm(ones.clone(), zeros.clone(), max_rows=T)
        self.params = LayerParams(w13=weight(E, 2 * f, d), w2=weight(E, d, f), w_r=weight(d, E, dt=torch.float32),
                                  ws13=weight(S, 2 * f, d), ws2=weight(S, d, f))
        self.layer = MoELayer(self.params, T, d, E, k, f, S, f, dtype)
        self.norm_out = LayerNorm(ones.clone(), zeros.clone(), max_rows=T)
        self.head = Linear(weight(vocab, d), max_rows=T)
        self.logprobs = TokenLogprobs(T, vocab, dtype=dtype)
        self.clipper = None

    def forward(self, x, tokens):
        """x [T, d], tokens [T] (-1: none) -> dict of logprob and entropy [T]."""
        h = self.layer.forward(self.norm_in.forward(x, save=True))
        y, _ = self.norm_out.forward(h, residual=x, save=True)
        return self.logprobs.forward(self.head.forward(y, save=True), tokens, entropy=True, save=True)

    def backward(self, tokens):
        """Gradients of the loss by every weight, and by x."""
        counts = (tokens >= 0).float()
        share = counts / counts.sum()
        head = self.head.backward(self.logprobs.backward(-share, d_entropy=-ENTROPY * share))
        out = self.norm_out.backward(head["dx"])
        layer = self.layer.backward(out["dx"])
        first = self.norm_in.backward(layer["dx"])
        return {"head": head["dw"], "norm_out.w": out["dw"], "norm_out.b": out["db"], "norm_in.w": first["dw"],
                "norm_in.b": first["db"], **{n: layer["d" + n] for n in ("w13", "w2", "ws13", "ws2", "w_r")},
                "x": first["dx"] + out["dx"]}

    def weights(self):
        p = self.params
        return {"head": self.head.w, "norm_out.w": self.norm_out.weight, "norm_out.b": self.norm_out.bias,
                "norm_in.w": self.norm_in.weight, "norm_in.b": self.norm_in.bias, "w13": p.w13, "w2": p.w2,
                "ws13": p.ws13, "ws2": p.ws2, "w_r": p.w_r}

    def step(self, x, tokens, rate=0.1, max_norm=1.0):
        """-> (loss, norm of the gradients)"""
        out = self.forward(x, tokens)
        grads = self.backward(tokens)
        if self.clipper is None:     # the gradients lie in the operators' own buffers
            self.clipper = GradClipper([grads[n] for n in self.weights()])
        norm = self.clipper.clip(max_norm)
        for name, w in self.weights().items():
            w.sub_(grads[name], alpha=rate)
        counts = (tokens >= 0).float()
        return -((out["logprob"] + ENTROPY * out["entropy"]) * counts).sum() / counts.sum(), norm


def inputs(T, d=256, vocab=2000, dtype=torch.bfloat16, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    tokens = torch.randint(0, vocab, (T,), generator=g, device="cuda", dtype=torch.int32)
    tokens[-T // 8:] = -1            # padding
    return torch.randn(T, d, generator=g, device="cuda", dtype=dtype), tokens


def main():
    T = 512
    block = TrainBlock(T)
    x, tokens = inputs(T)
    for i in range(10):
        loss, norm = block.step(x, tokens)
        print(f"step {i}: loss {float(loss):.4f}, norm of the gradients {float(norm):.3f}")


if __name__ == "__main__":
    main()
