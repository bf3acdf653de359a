"""The low-bit operators as they are used together (GPU only): the example's steps with 8-bit checkpoints, and a layer served
from a 4-bit table and 4-bit weights that were quantised from trained ones.

The gradients from checkpoints are those of the values that the checkpoints stand for: against the formula in 64 bits on
these values they are held to the bounds of engram_gate_grad's own tests. The served layer is held to the bf16 calls on the
same values: the products of both sum K = 1,536 terms in fp32 (each off by at most 2 K 2^-23 of sum|a w|) and round once
to bf16, 2^-8 each."""
import numpy as np
import pytest
import torch

import gram_hash_embedding_gb300 as geng
from examples import train_block as ex
from tests import gpu_helpers as H
from tests import test_gpu_gate_grad as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    H.build_all()
    yield
    assert geng.engram_device_status() == 0


def test_layer_gradients_from_checkpoints():
    T, C, head_dim, hc, dim, rows = 96, 6, 64, 2, 256, 500
    blk = ex.Block(rows, C, head_dim, hc, dim, seed=7)
    g = torch.Generator(device="cuda").manual_seed(8)
    ids = torch.randint(-1, rows, (T, C), generator=g, device="cuda")
    mask = torch.arange(T, device="cuda") % 7 != 3
    kv0 = geng.engram_project(geng.engram_embed(ids, blk.table, out_dtype=torch.bfloat16).view(T, -1), blk.wkv)
    x = (torch.randn((T, hc, dim), generator=g, device="cuda") + 0.3 * kv0.view(T, hc + 1, dim)[:, :hc].float()).bfloat16()
    out, emb, kv = blk.forward(x, ids, mask)
    dout = torch.randn((T, hc, dim), generator=g, device="cuda").bfloat16()
    saved = blk.checkpoint(x, kv)
    dx, grads, grad_rows, count = blk.gradients(None, ids, mask, emb, None, dout, saved)
    xb, kb = geng.engram_dequantize8(*saved[:2], 128), geng.engram_dequantize8(*saved[2:], 128).view(T, -1)
    dkv = geng.engram_gate_grad8(*saved, blk.q, blk.k, dout, mask=mask)[1]
    G._check([t.cpu() for t in (xb, kb, blk.q, blk.k, dout, mask)], [dx, dkv, grads["q"], grads["k"]], "checkpoints")
    # the rest of the chain runs on dkv as it does without checkpoints
    assert torch.equal(grads["wkv"], dkv.t() @ emb)
    exp = geng.engram_embed_grad(ids, dkv @ blk.wkv, rows)
    n = int(count)
    assert n == int(exp[2]) and torch.equal(grad_rows, exp[0]) and torch.equal(grads["rows"][:n], exp[1][:n])


def test_example_runs_with_checkpoints():
    losses = ex.train(steps=3, tokens=256, dim=256, log=lambda s: None, checkpoint8=True)
    assert len(losses) == 3 and np.isfinite(losses).all()


@pytest.mark.parametrize("block", [32, 16])
@pytest.mark.parametrize("T", [1, 100, 700])
def test_a_trained_layer_served_in_4_bits(block, T):
    """ids -> 4-bit rows as an operand -> 4-bit projection -> gate, all captured in one graph, against the bf16 calls on
    the values that codes and scales stand for."""
    C, head_dim, hc, dim, rows = 12, 128, 2, 512, 2000
    blk = ex.Block(rows, C, head_dim, hc, dim, seed=3)
    factor = 2.0 ** -10
    Q, S = geng.engram_quantize4(blk.table, block)
    wq, ws = geng.engram_quantize4(blk.wkv, block, scale=factor, tiled=True)
    g = torch.Generator(device="cuda").manual_seed(T)
    ids = torch.randint(-1, rows, (T, C), generator=g, device="cuda")
    mask = torch.rand(T, generator=g, device="cuda") < 0.8
    x = torch.randn((T, hc, dim), generator=g, device="cuda").bfloat16()
    out = torch.empty_like(x)

    def step():
        a, sa = geng.engram_lookup4_operand(ids, Q, S, block)
        kv = geng.engram_project4(a, sa, wq, ws, block, scale=factor)
        return geng.engram_gate(x, kv, blk.q, blk.k, mask, out=out), kv

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, kv = step()
    for seed in range(2):
        ids.copy_(torch.randint(-1, rows, (T, C), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda"))
        graph.replay()
        emb = geng.engram_lookup4(ids, Q, S, block).view(T, -1)
        w = geng.engram_dequantize4(wq, ws, block, scale=factor, tiled=True)  # exact in bf16
        want = geng.engram_project(emb, w)
        e = 2 * emb.shape[1] * 2.0 ** -23 * (emb.abs().double() @ w.abs().double().t())
        off = (kv.double() - want.double()).abs()
        assert (off <= 2 * 2.0 ** -8 * (want.double().abs() + e) + 2 * e + 2.0 ** -133).all()
        assert torch.equal(out, geng.engram_gate(x, kv, blk.q, blk.k, mask))
