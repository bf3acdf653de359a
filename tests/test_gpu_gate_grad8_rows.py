"""The gate's gradient from 8-bit checkpoints of narrow rows, which the lanes of a warp hold (GPU only): against the formula in
64 bits within engram_gate_grad's bounds, at the widths where the number of lanes a token and of vectors a lane change."""
import numpy as np
import pytest
import torch

import gram_hash_embedding_gb300 as geng
from tests import gpu_helpers as H
from tests import test_gpu_gate_grad as G
from tests import test_gpu_gate_grad8 as E

pytestmark = pytest.mark.gpu

WIDTHS = [(1, 16), (1, 80), (1, 256), (1, 272), (1, 512), (1, 528), (1, 1024), (1, 1040), (2, 48), (2, 128), (2, 144), (2, 512),
          (2, 528), (4, 32), (4, 64), (4, 112), (4, 256), (4, 272), (8, 16), (8, 64), (8, 128), (8, 240), (8, 256), (8, 272)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    H.build_all()
    yield
    assert geng.engram_device_status() == 0


@pytest.mark.parametrize("block", [32, 64, 128])
@pytest.mark.parametrize("hc,dim", WIDTHS)
def test_widths(hc, dim, block):
    for T in (1, 3, 33, 700):
        args = G._inputs(np.random.default_rng(T + hc * dim + block), T, hc, dim)
        xq, kq, back = E._checkpoints(args, block)
        got = E._run8(xq, kq, back, block)
        G._check(back, got, f"T={T} hc={hc} dim={dim} block={block}")
        assert all(torch.equal(a, b) for a, b in zip(got, E._run8(xq, kq, back, block)))


@pytest.mark.parametrize("T,hc,dim", [(40000, 1, 64), (9000, 1, 256), (6000, 1, 528), (20000, 2, 96), (7000, 2, 400),
                                      (21000, 4, 64), (8000, 4, 240), (12000, 8, 32), (5000, 8, 256)])
def test_several_tokens_a_warp(T, hc, dim):
    E.test_many_tokens_a_cluster(T, hc, dim)


@pytest.mark.parametrize("T,hc,dim", [(500, 1, 512), (600, 2, 64), (400, 4, 128), (300, 4, 256), (4000, 8, 96)])
def test_small_dots(T, hc, dim):
    E.test_small_dots(T, hc, dim)


@pytest.mark.parametrize("hc,dim", [(1, 64), (2, 128), (4, 48), (4, 256), (8, 64), (1, 1024)])
def test_masked_neighbours_and_nan(hc, dim):
    """What a masked token's checkpoint holds does not reach the tokens of the same warp, nor a NaN another copy or token."""
    T = 64
    args = G._inputs(np.random.default_rng(dim), T, hc, dim, masked=0.0)
    args[5][1::2] = False
    xq, kq, back = E._checkpoints(args, 64)
    exp = E._run8(xq, kq, back, 64)
    off = ~args[5]
    args[0][off], args[1][off] = float("nan"), float("-inf")
    xq, kq, _ = E._checkpoints(args, 64)
    got = E._run8(xq, kq, back, 64)
    assert all(torch.equal(a, b) for a, b in zip(got, exp))
    for i in (0, hc - 1):
        bad = [a.clone() for a in args]
        bad[0][2, i, dim - 3] = float("nan")
        xq, kq, _ = E._checkpoints(bad, 64)
        got = E._run8(xq, kq, back, 64)
        assert torch.isnan(got[0][2, i]).all() and torch.isnan(got[2][i]).all()
        for j in range(hc):
            if j != i:
                assert torch.equal(got[0][:, j], exp[0][:, j]) and torch.equal(got[2][j], exp[2][j])
        keep = [t for t in range(T) if t != 2]
        assert torch.equal(got[0][keep], exp[0][keep]) and torch.equal(got[1][keep], exp[1][keep])


def test_all_masked():
    T, hc, dim, block = 100, 4, 64, 32
    args = G._inputs(np.random.default_rng(0), T, hc, dim)
    args[5][:] = False
    xq, kq, back = E._checkpoints(args, block)
    dx, dkv, dq, dk = E._run8(xq, kq, back, block)
    assert torch.equal(dx.cpu(), back[4]) and not dkv.any() and not dq.any() and not dk.any()


@pytest.mark.parametrize("T,hc,dim", [(3000, 1, 16), (2000, 2, 64), (1000, 4, 256), (500, 8, 128)])
def test_in_place_on_another_stream_and_in_a_graph(T, hc, dim):
    args = G._inputs(np.random.default_rng(T), T, hc, dim)
    xq, kq, back = E._checkpoints(args, 32)
    exp = E._run8(xq, kq, back, 32)
    dev, mask = [a.cuda() for a in args[2:4]], args[5].cuda()
    s = torch.cuda.Stream()
    dout = args[4].cuda()
    got = geng.engram_gate_grad8(*xq, *kq, *dev, dout, block=32, mask=mask, dx=dout, stream=s)
    s.synchronize()
    assert got[0] is dout and all(torch.equal(a, b) for a, b in zip(got, exp))
    dout = args[4].cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = geng.engram_gate_grad8(*xq, *kq, *dev, dout, block=32, mask=mask)
    for _ in range(2):
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, exp))
