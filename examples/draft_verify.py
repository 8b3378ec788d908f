"""One verification step of drafted tokens through an MoE block, on one GPU.

Every user has a token and n drafted ones; their rows go together through the attention output
projection (with the residual), the MoE layer for a few tokens (with the residual) and the head;
the target's probabilities then decide which drafted tokens stay.

    python examples/draft_verify.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from dropless_token_routing_gb300.api import DraftVerifier, LayerParams, Linear, MoEDecodeLayer  # noqa: E402


class DraftBlock:
    """Projection + residual -> MoE layer + residual -> head -> verification."""

    def __init__(self, users, drafted, d=512, E=16, k=2, f=256, S=1, vocab=4000, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape, dt=dtype):
            return torch.randn(*shape, generator=g, device="cuda", dtype=dt) * shape[-1] ** -0.5

        rows = users * (drafted + 1)
        self.users, self.drafted, self.vocab = users, drafted, vocab
        self.project = Linear(weight(d, d), max_rows=rows)
        params = LayerParams(w13=weight(E, 2 * f, d), w2=weight(E, d, f), w_r=weight(d, E, dt=torch.float32),
                             ws13=weight(S, 2 * f, d), ws2=weight(S, d, f))
        self.layer = MoEDecodeLayer(params, rows, d, E, k, f, S, f, dtype)
        self.head = Linear(weight(vocab, d), max_rows=rows)
        self.verifier = DraftVerifier(users, drafted, vocab)

    def step(self, attended, x, draft_tokens, draft_probs, u_accept, u_sample):
        """attended, x [users * (drafted + 1), d] -> (tokens [users, drafted + 1], accepted [users])."""
        x = self.project.forward(attended, residual=x)
        x = self.layer.forward(x, residual=x)
        scores = self.head.forward(x).float()
        target = torch.softmax(scores, -1).view(self.users, self.drafted + 1, self.vocab)
        return self.verifier.verify(draft_tokens, draft_probs, target, u_accept, u_sample)


def inputs(block, d=512, dtype=torch.bfloat16, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    users, n, V = block.users, block.drafted, block.vocab
    rows = users * (n + 1)
    probs = torch.softmax(2 * torch.randn(users, n, V, generator=g, device="cuda"), -1)
    tokens = torch.multinomial(probs.view(users * n, V), 1, generator=g).view(users, n).to(torch.int32)
    return (torch.randn(rows, d, generator=g, device="cuda", dtype=dtype),
            torch.randn(rows, d, generator=g, device="cuda", dtype=dtype), tokens, probs,
            torch.rand(users, n, generator=g, device="cuda"), torch.rand(users, generator=g, device="cuda"))


def main():
    block = DraftBlock(users=6, drafted=4)
    tokens, accepted = block.step(*inputs(block))
    for user in range(block.users):
        print(f"user {user}: {int(accepted[user])} of {block.drafted} drafted tokens kept, tokens {tokens[user].tolist()}")


if __name__ == "__main__":
    main()
