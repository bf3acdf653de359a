"""The training operators together (GPU only): one layer's gradients through the library against torch's
own differentiation of the plain formulas in 64 bits, and the example's steps, whose loss has to fall.

Tolerance of the chain: the library keeps the rows, the keys and values, and dkv in bf16, so each stage's
inputs carry a rounding of 2^-8 relative that the 64-bit chain does not; over the four stages and the
projection's sums the relative error of a gradient tensor in its 2-norm stays below 4 * 2^-8 times a factor
for the gate's slope, whose relative change is up to 1/(2m) + 1/(2 sqrt m) times dot's. The inputs keep m of
order 1, so 2^-4 covers it.
"""
import numpy as np
import pytest
import torch

import gram_hash_embedding_gb300 as geng
from examples import train_block as ex
from tests import gpu_helpers as H

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    H.build_all()
    yield


def test_layer_gradients_against_autograd():
    T, C, head_dim, hc, dim, rows = 96, 6, 64, 2, 256, 500
    blk = ex.Block(rows, C, head_dim, hc, dim, seed=7)
    g = torch.Generator(device="cuda").manual_seed(8)
    ids = torch.randint(-1, rows, (T, C), generator=g, device="cuda")
    mask = torch.arange(T, device="cuda") % 7 != 3
    # residual copies aligned with the keys, so that |dot| is of order 1
    kv0 = geng.engram_project(geng.engram_embed(ids, blk.table, out_dtype=torch.bfloat16).view(T, -1), blk.wkv)
    x = (torch.randn((T, hc, dim), generator=g, device="cuda") + 0.3 * kv0.view(T, hc + 1, dim)[:, :hc].float()).bfloat16()
    out, emb, kv = blk.forward(x, ids, mask)
    dout = torch.randn((T, hc, dim), generator=g, device="cuda").bfloat16()
    dx, grads, grad_rows, count = blk.gradients(x, ids, mask, emb, kv, dout)

    leaf = lambda t: t.double().requires_grad_()
    table, wkv, q, k, x64 = (leaf(t) for t in (blk.table, blk.wkv, blk.q, blk.k, x))
    ok = ids >= 0
    e = (table[ids.clamp(min=0)] * ok[..., None]).reshape(T, -1)
    y = (e @ wkv.t()).view(T, hc + 1, dim)
    key, v = y[:, :hc], y[:, hc:]
    r = torch.rsqrt(x64.square().mean(-1) + 1e-20) * torch.rsqrt(key.square().mean(-1) + 1e-20)
    dot = (x64 * q * k * key).sum(-1) * r * dim ** -0.5
    gate = torch.sigmoid(dot.abs().clamp_min(1e-6).sqrt().copysign(dot))
    gate = torch.where(mask[:, None], gate, 0.0)
    (x64 + gate[..., None] * v).backward(dout.double())

    n = int(count)
    dense = torch.zeros_like(table).index_copy_(0, grad_rows[:n], grads["rows"][:n].double())
    for name, got, exp in (("x", dx, x64.grad), ("wkv", grads["wkv"], wkv.grad), ("q", grads["q"], q.grad),
                           ("k", grads["k"], k.grad), ("table", dense, table.grad)):
        off = float((got.double() - exp).norm() / exp.norm())
        assert off < 2.0 ** -4, (name, off)
    assert torch.equal(grad_rows[:n], torch.unique(ids[ok]))


def test_example_loss_falls():
    losses = ex.train(steps=8, tokens=512, dim=256, log=lambda s: None)
    assert np.isfinite(losses).all() and losses[-1] < 0.9 * losses[0], losses
    assert geng.engram_device_status() == 0
