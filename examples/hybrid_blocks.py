"""Two blocks of a hybrid model, from a prompt to single tokens: softmax attention over a paged cache, then a gated delta rule.

Every projection is a packed-ternary product; between them run the per-head norm with rotary positions and the append to the
cache (rope_append), the attention over it (paged_attn) and the delta rule (gdn).  Weights are random.

    python examples/hybrid_blocks.py [--prompt 200] [--new 16]
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import bit_quantized_matvec_amd as tq  # noqa: E402
import tq_inputs as TI  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM, PAGE = 1024, 8, 2, 64, 16
K_HEADS, V_HEADS, DK, DV = 2, 4, 64, 64


class Linear:
    """A packed-ternary matrix; fp32 activations are quantized to q8_K on the way in."""

    def __init__(self, g, rows, cols):
        self.rows, self.cols = rows, cols
        canonical = torch.from_numpy(TI.pq2_matrix(g, rows, cols).reshape(-1)).cuda()
        self.w = tq.repack(canonical, "pq2_0", rows, cols)

    def __call__(self, x):
        if x.shape[0] == 1:
            return tq.gemv_f32("pq2_0", self.w, self.rows, self.cols, x)[None]
        return torch.cat([tq.gemm("pq2_0", self.w, self.rows, self.cols, *tq.quantize_q8k(y.contiguous())) for y in x.split(64)])


def norm(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


class Attention:
    def __init__(self, g, context):
        self.qkv = Linear(g, (HEADS + 2 * KV_HEADS) * DIM, HIDDEN)
        self.out = Linear(g, HIDDEN, HEADS * DIM)
        self.freq, self.rope_scale = tq.rope_frequencies(DIM // 2, 1e6, device="cuda")  # half of each head turns
        self.norms = [torch.from_numpy(1 + 0.1 * g.standard_normal(DIM, dtype=np.float32)).cuda() for _ in "qk"]
        pages = -(-context // PAGE)
        self.k, self.v = tq.kv_cache(pages, KV_HEADS, PAGE, DIM)
        self.table = torch.from_numpy(g.permutation(pages).astype(np.int32)).cuda()[None]

    def __call__(self, x, step):
        qkv = self.qkv(norm(x))
        q, k, v = (y.unflatten(1, (-1, DIM)) for y in qkv.split([HEADS * DIM, KV_HEADS * DIM, KV_HEADS * DIM], 1))
        at = step.positions.long()
        slots = self.table[0, at // PAGE].long() * PAGE + at % PAGE
        q = tq.rope_append(q, k, v, step.positions, slots, self.freq, self.k, self.v, q_norm=self.norms[0], k_norm=self.norms[1],
                           rope_scale=self.rope_scale)
        ws = tq.attn_workspace(x.shape[0], 1, HEADS, KV_HEADS, DIM)  # (a server keeps one per batch size)
        y = tq.paged_attn(q, self.k, self.v, self.table, step.kv_len, step.cu, max_len=x.shape[0], out_dtype=torch.float32, ws=ws)
        return x + self.out(y.flatten(1))


class DeltaRule:
    def __init__(self, g):
        self.qkv = Linear(g, 2 * K_HEADS * DK + V_HEADS * DV, HIDDEN)
        self.out = Linear(g, HIDDEN, V_HEADS * DV)
        self.gates = torch.from_numpy(g.standard_normal((2 * V_HEADS, HIDDEN), dtype=np.float32)).cuda() * HIDDEN**-0.5
        self.state = torch.zeros(1, V_HEADS, DK, DV, device="cuda")

    def __call__(self, x, step):
        y = norm(x)
        q, k, v = self.qkv(y).split([K_HEADS * DK, K_HEADS * DK, V_HEADS * DV], 1)
        a, b = (y @ self.gates.t()).split(V_HEADS, 1)
        g, beta = -torch.nn.functional.softplus(a - 2).contiguous(), torch.sigmoid(b).contiguous()
        ws = tq.gdn_workspace(x.shape[0], 1, V_HEADS, DK, DV, max_len=x.shape[0])
        o = tq.gdn(q.unflatten(1, (-1, DK)), k.unflatten(1, (-1, DK)), v.unflatten(1, (-1, DV)), g, beta, self.state, step.cu, l2norm=True,
                   max_len=x.shape[0], ws=ws)
        return x + self.out(o.flatten(1))


class Step:
    """Positions and lengths of one sequence's `n` new tokens behind `past` ones."""

    def __init__(self, past, n):
        self.positions = torch.arange(past, past + n, dtype=torch.int32, device="cuda")
        self.kv_len = torch.tensor([past + n], dtype=torch.int32, device="cuda")
        self.cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")


class Model:
    def __init__(self, context, seed=0):
        g = np.random.default_rng(seed)
        self.blocks = [Attention(g, context), DeltaRule(g)]
        self.past = 0

    def __call__(self, x):
        step = Step(self.past, x.shape[0])
        for block in self.blocks:
            x = block(x, step)
        self.past += x.shape[0]
        return x


def run(prompt, new, seed=0):
    """Outputs of `prompt` tokens at once and `new` ones one by one, and of all of them at once."""
    x = torch.from_numpy(np.random.default_rng(seed + 1).standard_normal((prompt + new, HIDDEN), dtype=np.float32)).cuda()
    model = Model(prompt + new, seed)
    steps = torch.cat([model(x[:prompt])] + [model(x[i : i + 1]) for i in range(prompt, prompt + new)])
    return steps, Model(prompt + new, seed)(x)


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    p.add_argument("--prompt", type=int, default=200)
    p.add_argument("--new", type=int, default=16)
    a = p.parse_args()
    steps, whole = run(a.prompt, a.new)
    off = (steps - whole).norm() / whole.norm()
    print(f"{a.prompt} + {a.new} tokens; one by one against all at once: {off:.2e} of the outputs' norm")
