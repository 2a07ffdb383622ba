"""A decode step of several requests at once, each with its own adapter and its own way of sampling: a shared ternary projection
with an adapter beside it, a layer of ternary experts, and the next tokens from a ternary output head.

Weights are random.  The same step is also done request by request; it gives the same hidden states up to the steps of the 8-bit
quantization.

    python examples/mixed_batch.py [--requests 12]
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import bit_quantized_matvec_amd as tq  # noqa: E402
import tq_inputs as TI  # noqa: E402

HIDDEN, VOCAB = 1024, 4000
EXPERTS, CHOSEN, INNER = 8, 2, 512
ADAPTERS, RANK = 5, 16


def ternary(g, rows, cols):
    return tq.repack(torch.from_numpy(TI.pq2_matrix(g, rows, cols).reshape(-1)).cuda(), "pq2_0", rows, cols)


def norm(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


class Model:
    def __init__(self, seed=0):
        g = np.random.default_rng(seed)
        normal = lambda *shape, std=1.0: torch.from_numpy(g.standard_normal(shape, dtype=np.float32) * std).cuda()  # noqa: E731
        self.mix = ternary(g, HIDDEN, HIDDEN)
        self.a = normal(ADAPTERS, RANK, HIDDEN, std=HIDDEN**-0.5).bfloat16()
        self.b = normal(ADAPTERS, HIDDEN, RANK, std=RANK**-0.5).bfloat16()
        self.ranks = torch.tensor([16, 8, 4, 16, 12], dtype=torch.int32, device="cuda")
        self.scale = torch.full((ADAPTERS,), 0.5, device="cuda")
        self.router = normal(EXPERTS, HIDDEN, std=HIDDEN**-0.5)
        self.bias = normal(EXPERTS, std=0.05)
        self.up = torch.stack([ternary(g, 2 * INNER, HIDDEN) for _ in range(EXPERTS)])
        self.down = torch.stack([ternary(g, HIDDEN, INNER) for _ in range(EXPERTS)])
        self.head = ternary(g, VOCAB, HIDDEN)

    def hidden(self, x, adapter):
        t = x.shape[0]
        # a shared projection, and each request's adapter beside it
        y = norm(x)
        z = tq.gemm("pq2_0", self.mix, HIDDEN, HIDDEN, *tq.quantize_q8k(y))
        ws = tq.adapter_workspace(t, ADAPTERS, RANK, HIDDEN)  # (a server keeps one per batch size)
        x = x + tq.adapter_add(z, y, self.a, self.b, adapter, ranks=self.ranks, scale=self.scale, ws=ws)
        # each token's experts
        y = norm(x)
        weights, experts = tq.route(y @ self.router.t(), CHOSEN, score="sigmoid", bias=self.bias)
        lists = tq.expert_lists(experts, EXPERTS)
        q, d, _ = tq.quantize_q8k(y)
        gate, up = tq.gemm_experts("pq2_0", self.up, 2 * INNER, HIDDEN, q, d, *lists).split(INNER, 1)
        q, d, _ = tq.quantize_q8k(torch.nn.functional.silu(gate) * up)
        z = tq.gemm_experts("pq2_0", self.down, HIDDEN, INNER, q, d, *lists)
        return x + (z.view(t, CHOSEN, HIDDEN) * weights[:, :, None]).sum(1)

    def step(self, x, adapter, u, temperature, top_k, top_p, min_p):
        """(hidden states, tokens, their log probabilities) of one token for each request."""
        h = self.hidden(x, adapter)
        logits = tq.gemm("pq2_0", self.head, VOCAB, HIDDEN, *tq.quantize_q8k(norm(h)))
        logprob = torch.empty(x.shape[0], device="cuda")
        tokens = tq.sample(logits, u, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p, logprob=logprob,
                           ws=tq.sample_workspace(x.shape[0], VOCAB))
        return h, tokens, logprob


def requests(n, seed=0):
    """Random requests: inputs, adapters (some none), random numbers and sampling parameters (some greedy)."""
    g = np.random.default_rng(seed + 1)
    cuda = lambda x, t: torch.from_numpy(np.asarray(x)).to("cuda", t)  # noqa: E731
    return (cuda(g.standard_normal((n, HIDDEN)), torch.float32), cuda(g.integers(-1, ADAPTERS, n), torch.int32), cuda(g.random(n), torch.float32),
            cuda(g.choice([0.0, 0.7, 1.0], n), torch.float32), cuda(g.choice([0, 20, 50], n), torch.int32), cuda(g.choice([1.0, 0.9], n), torch.float32),
            cuda(g.choice([0.0, 0.05], n), torch.float32))


def run(n, seed=0):
    """The step of n requests at once, and of each by itself."""
    model, batch = Model(seed), requests(n, seed)
    at_once = model.step(*batch)
    alone = [model.step(*(x[i : i + 1] for x in batch)) for i in range(n)]
    return at_once, tuple(torch.cat(x) for x in zip(*alone))


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    p.add_argument("--requests", type=int, default=12)
    a = p.parse_args()
    (h, tokens, logprob), (h1, tokens1, _) = run(a.requests)
    print(f"tokens {tokens.tolist()}\nlog probabilities {[round(x, 2) for x in logprob.tolist()]}")
    print(f"at once against one by one: {(h - h1).norm() / h1.norm():.2e} of the hidden states' norm, {(tokens != tokens1).sum().item()} other tokens")
