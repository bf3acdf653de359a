"""The gate's gradient from 8-bit checkpoints (engram_gate_grad8) against the formula in 64 bits on the bf16 values that
the checkpoints stand for, within engram_gate_grad's bounds (GPU only). The two calls run the same arithmetic on those
values, but split a row's columns otherwise (a checkpoint's rows have to start on 16 bytes; with 4 copies and more a
thread has 4 columns), so their sums run in another order; where the split is the same the bits are equal."""
import numpy as np
import pytest
import torch

import gram_hash_embedding_gb300 as geng
from tests import gpu_helpers as H
from tests import test_gpu_gate_grad as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    H.build_all()
    yield
    assert geng.engram_device_status() == 0


def _checkpoints(args, block):
    """engram_quantize8's checkpoints of x and kv, and the same call's arguments with the values they stand for."""
    x, kv = args[0].cuda(), args[1].cuda()
    T, hc, dim = x.shape
    xq = geng.engram_quantize8(x, block)
    kq = geng.engram_quantize8(kv.view(T, hc + 1, dim), block)
    back = [geng.engram_dequantize8(*xq, block), geng.engram_dequantize8(*kq, block).view(T, -1)]
    return xq, kq, [t.cpu() for t in back] + list(args[2:])


def _run8(xq, kq, args, block, **kw):
    return geng.engram_gate_grad8(*xq, *kq, *[a.cuda() for a in args[2:5]], block=block, mask=args[5].cuda(), **kw)


@pytest.mark.parametrize("block", [32, 64, 128])
@pytest.mark.parametrize("T,hc,dim", [(1, 1, 16), (1, 4, 5120), (2, 8, 16384), (3, 2, 1040), (37, 4, 256),
                                      (200, 2, 272), (333, 1, 2064), (65, 8, 640), (500, 4, 1024), (1500, 1, 64),
                                      (9, 4, 16384), (700, 8, 96), (311, 4, 5120), (19, 1, 16368), (5, 2, 10256)])
def test_gradient_of_the_values(T, hc, dim, block):
    if block != 128 and T * hc * dim > 1 << 20:
        pytest.skip("one block length at the large sizes")
    args = G._inputs(np.random.default_rng(T * 3 + dim + block), T, hc, dim)
    xq, kq, back = _checkpoints(args, block)
    got = _run8(xq, kq, back, block)
    G._check(back, got, f"T={T} hc={hc} dim={dim} block={block}")
    again = _run8(xq, kq, back, block)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("T,hc,dim", [(1500, 1, 64), (200, 2, 272)])
def test_whole_rows_of_few_copies_give_the_bits_of_the_values_gradient(T, hc, dim):
    args = G._inputs(np.random.default_rng(T + dim), T, hc, dim)
    xq, kq, back = _checkpoints(args, 32)
    got, exp = _run8(xq, kq, back, 32), G._run(back)
    assert torch.equal(got[0].view(torch.int16), exp[0].view(torch.int16))
    assert torch.equal(got[1].view(torch.int16), exp[1].view(torch.int16))


def test_masked_tokens_and_nan():
    """A masked token passes dout through whatever its checkpoint holds; in an open one a NaN stays with its copy."""
    T, hc, dim = 40, 4, 512
    args = G._inputs(np.random.default_rng(1), T, hc, dim, masked=0.0)
    args[5][::3] = False
    clean_x, clean_k, back = _checkpoints(args, 128)
    exp = _run8(clean_x, clean_k, back, 128)
    off = ~args[5]
    args[0][off], args[1][off] = float("nan"), float("inf")
    xq, kq, _ = _checkpoints(args, 128)
    got = _run8(xq, kq, back, 128)
    assert all(torch.equal(a, b) for a, b in zip(got, exp))
    args[0][1, 2, 7] = float("nan")  # an open token's third copy
    xq, kq, nan_back = _checkpoints(args, 128)
    got = _run8(xq, kq, nan_back, 128)
    assert torch.isnan(got[0][1, 2]).all() and torch.equal(got[0][1, :2], exp[0][1, :2])
    assert torch.isnan(got[2][2]).all() and torch.equal(got[2][3], exp[2][3])


def test_outputs_in_place_streams_and_graphs():
    T, hc, dim = 64, 2, 1024
    args = G._inputs(np.random.default_rng(4), T, hc, dim)
    xq, kq, back = _checkpoints(args, 64)
    exp = _run8(xq, kq, back, 64)
    ws = torch.empty(geng.engram_gate_grad8_workspace(T, hc, dim), dtype=torch.uint8, device="cuda")
    dout = args[4].cuda()
    dev = [a.cuda() for a in args[2:4]]
    mask = args[5].cuda()
    got = geng.engram_gate_grad8(*xq, *kq, *dev, dout, block=64, mask=mask, dx=dout, workspace=ws)
    assert got[0] is dout and all(torch.equal(a, b) for a, b in zip(got, exp))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = geng.engram_gate_grad8(*xq, *kq, *dev, args[4].cuda(), block=64, mask=mask, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, exp))
    dout = args[4].cuda()
    outs = [torch.empty_like(t) for t in exp]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        geng.engram_gate_grad8(*xq, *kq, *dev, dout, block=64, mask=mask, dx=outs[0], dkv=outs[1], dq_weight=outs[2],
                               dk_weight=outs[3], workspace=ws)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(outs, exp))


def test_no_tokens():
    e = torch.empty((0, 2, 64), dtype=torch.uint8, device="cuda")
    w = torch.ones((2, 64), dtype=torch.bfloat16, device="cuda")
    got = geng.engram_gate_grad8(e, e[..., :1], torch.empty((0, 3, 64), dtype=torch.uint8, device="cuda"),
                                 torch.empty((0, 3, 1), dtype=torch.uint8, device="cuda"), w, w, e.bfloat16(), block=64)
    assert got[0].shape == (0, 2, 64) and got[1].shape == (0, 192) and (got[2] == 0).all() and (got[3] == 0).all()
