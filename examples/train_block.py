"""Training steps of one Engram layer on synthetic data: the n-gram hash of token ids, trainable
embedding rows, the `wkv` projection and the gate forward, then their gradients, the global norm with
clipping and a plain gradient step.

    python examples/train_block.py [--steps 20] [--tokens 4096] [--dim 1024]

The table is fp32 and read as bf16 (the lookup rounds); only the rows that a step's tokens hash to
get a gradient, so its size does not depend on the table's. The projection's two gradients are plain
matrix products and run as torch matmuls.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gram_hash_embedding_gb300 as geng  # noqa: E402
import synth  # noqa: E402


class Block:
    """One Engram layer's parameters (a table of `rows` rows, wkv, the gate's weights) and their step."""

    def __init__(self, rows: int, n_cols: int, head_dim: int, hc: int, dim: int, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        K = n_cols * head_dim
        self.hc, self.dim = hc, dim
        self.table = torch.randn((rows, head_dim), generator=g, device="cuda")
        self.wkv = (torch.randn(((hc + 1) * dim, K), generator=g, device="cuda") * K ** -0.5).bfloat16()
        self.q = (0.5 + torch.rand((hc, dim), generator=g, device="cuda")).bfloat16()
        self.k = (0.5 + torch.rand((hc, dim), generator=g, device="cuda")).bfloat16()

    def forward(self, x, ids, mask):
        """x bf16 [T, hc, dim], ids int64 [T, C] row ids: the layer's output and what its gradient needs."""
        emb = geng.engram_embed(ids, self.table, out_dtype=torch.bfloat16).view(ids.shape[0], -1)
        kv = geng.engram_project(emb, self.wkv)
        return geng.engram_gate(x, kv, self.q, self.k, mask), emb, kv

    def gradients(self, x, ids, mask, emb, kv, dout):
        dx, dkv, dq, dk = geng.engram_gate_grad(x, kv, self.q, self.k, dout, mask)
        dwkv = dkv.t() @ emb
        rows, drows, count = geng.engram_embed_grad(ids, dkv @ self.wkv, self.table.shape[0])
        return dx, {"wkv": dwkv, "q": dq, "k": dk, "rows": drows}, rows, count

    def step(self, grads, rows, count, lr: float, max_norm: float):
        """Clip all gradients by their global norm, in place, and apply them; returns the norm."""
        names = ("wkv", "q", "k", "rows")
        norm = geng.engram_grad_clip([grads[n] for n in names], max_norm, counts=[None, None, None, count])
        self.wkv -= (lr * grads["wkv"]).to(self.wkv.dtype)
        self.q -= (lr * grads["q"]).to(self.q.dtype)
        self.k -= (lr * grads["k"]).to(self.k.dtype)
        n = int(count)
        self.table.index_add_(0, rows[:n], grads["rows"][:n], alpha=-lr)
        return norm


def train(steps: int = 20, tokens: int = 4096, dim: int = 1024, hc: int = 4, lr: float = 0.5, max_norm: float = 4.0,
          log=print):
    """Fit the layer's output to that of another layer with the same tokens; returns the losses."""
    wl = synth.make_workload(5)  # two layers, 24 columns of rows a token, small tables
    lay = wl.layout
    L = min(tokens, wl.L)
    B = max(1, min(wl.B, tokens // L))
    T = B * L
    hasher = geng.EngramHash(n_layers=lay.n_layers, max_ngram=lay.max_ngram, n_heads=lay.n_heads,
                             head_dim=lay.head_dim, block=lay.block, max_batch=B, max_seq_len=L,
                             token_map=lay.token_map, multipliers=lay.multipliers, primes=lay.primes,
                             offsets=lay.offsets, dead=lay.dead, pad_id=lay.pad_id)
    ids = hasher.hash(torch.from_numpy(wl.ids[:B, :L].copy()).cuda()).view(T, lay.n_layers, lay.n_cols)[:, 0]
    mask = torch.ones(T, dtype=torch.bool, device="cuda")
    mask[::10] = False
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((T, hc, dim), generator=g, device="cuda").bfloat16()
    student, teacher = (Block(lay.rows[0], lay.n_cols, lay.head_dim, hc, dim, seed) for seed in (2, 3))
    target = teacher.forward(x, ids, mask)[0].float()
    losses = []
    for step in range(steps):
        out, emb, kv = student.forward(x, ids, mask)
        diff = out.float() - target
        losses.append(float(diff.square().mean()))
        dout = (diff * (2 / dim)).bfloat16()  # of the squared error summed over tokens and copies
        _, grads, rows, count = student.gradients(x, ids, mask, emb, kv, dout)
        norm = student.step(grads, rows, count, lr, max_norm)
        log(f"step {step}: loss {losses[-1]:.5f}, gradient norm {float(norm):.3f}, {int(count)} rows")
    hasher.close()
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--dim", type=int, default=1024)
    a = ap.parse_args()
    synth.build()
    geng.build()
    train(a.steps, a.tokens, a.dim)
