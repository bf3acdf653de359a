"""The gate's gradient from 8-bit checkpoints (engram_gate_grad8) against the formula in 64 bits on the bf16 values that
the checkpoints stand for, within engram_gate_grad's bounds (GPU only): the same arithmetic on those values, its sums in an
order of their own."""
import ctypes

import numpy as np
import pytest
import torch

import gram_hash_embedding_gb300 as geng
from tests import gpu_helpers as H
from tests import test_gpu_gate_grad as G
from tests import train_ref as R

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


@pytest.mark.parametrize("T,hc,dim", [(4000, 4, 256), (3000, 8, 640), (2500, 2, 1040), (1200, 1, 5120), (900, 4, 5120),
                                      (400, 8, 5120)])
def test_many_tokens_a_cluster(T, hc, dim):
    """Rings and buffers go round several times, over runs of masked and of open tokens."""
    rng = np.random.default_rng(T + dim)
    args = G._inputs(rng, T, hc, dim)
    args[5] = torch.from_numpy(np.repeat(rng.random(-(-T // 50)) < 0.7, 50)[:T] ^ (rng.random(T) < 0.1))
    xq, kq, back = _checkpoints(args, 128)
    got = _run8(xq, kq, back, 128)
    G._check(back, got, f"T={T} hc={hc} dim={dim}")
    assert all(torch.equal(a, b) for a, b in zip(got, _run8(xq, kq, back, 128)))


@pytest.mark.parametrize("T,hc,dim", [(1500, 1, 64), (900, 2, 1040), (700, 1, 5120), (600, 2, 5120), (400, 4, 1024),
                                      (500, 8, 256)])
def test_small_dots(T, hc, dim):
    """Keys nearly orthogonal to h, where sum(h w key) is formed once more in twice the precision: dot is held to the
    error of the mean squares alone. Tokens with a copy of |dot| outside [1e-5, 0.03] are masked out."""
    rng = np.random.default_rng(T + dim)
    args = G._inputs(rng, T, hc, dim, masked=0.0)
    x, q, k = G._f64(args[0]), G._f64(args[2]), G._f64(args[3])
    kv = rng.standard_normal((T, hc + 1, dim))
    key = kv[:, :hc]
    key -= (x * q * k * key).sum(-1, keepdims=True) / (x * x * q * k * q * k).sum(-1, keepdims=True) * (x * q * k)
    args[1] = G._bf(kv.reshape(T, -1))
    xq, kq, back = _checkpoints(args, 128)
    dot = np.abs(R.gate_grad(G._f64(back[0]), G._f64(back[1]), q, k, G._f64(args[4]), np.ones(T, bool), G.EPS)[5][..., 0])
    back[5] = torch.from_numpy(((dot > 1e-5) & (dot < 0.03)).all(1))
    assert back[5].sum() >= 5
    got = _run8(xq, kq, back, 128)
    G._check(back, got, "small dots", small=True)
    assert all(torch.equal(a, b) for a, b in zip(got, _run8(xq, kq, back, 128)))


@pytest.mark.parametrize("T,hc,dim", [(300, 4, 5120), (300, 2, 256), (160, 8, 1024)])
def test_withheld_sums_time_out_and_the_next_call_is_right(T, hc, dim):
    args = G._inputs(np.random.default_rng(T), T, hc, dim, masked=0.0)
    xq, kq, back = _checkpoints(args, 128)
    L = geng._lib()
    P, I64, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    L.engram_gate_grad8_withhold.argtypes = [P, P, P, P, I32, P, P, P, P, I64, I32, I32, ctypes.c_float, P, P, P, P, P,
                                             ctypes.c_uint64, I64, P]
    L.engram_gate_grad8_withhold.restype = ctypes.c_int
    dev = [a.cuda() for a in back[2:5]]
    outs = [torch.empty((T, hc, dim), dtype=torch.bfloat16, device="cuda"),
            torch.empty((T, (hc + 1) * dim), dtype=torch.bfloat16, device="cuda"),
            torch.empty((hc, dim), device="cuda"), torch.empty((hc, dim), device="cuda")]
    ws = torch.empty(geng.engram_gate_grad8_workspace(T, hc, dim), dtype=torch.uint8, device="cuda")
    rc = L.engram_gate_grad8_withhold(*[t.data_ptr() for t in (*xq, *kq)], 128, *[t.data_ptr() for t in dev], None, T, hc,
                                      dim, G.EPS, *[t.data_ptr() for t in outs], ws.data_ptr(), ws.numel(), T // 2,
                                      torch.cuda.current_stream().cuda_stream)
    assert rc == geng.OK and geng.engram_device_status() == geng.STATUS_TIMEOUT
    G._check(back, _run8(xq, kq, back, 128), "after the timeout")
    assert geng.engram_device_status() == 0


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


def test_offsets_beyond_32_bits():
    """More than 2^32 codes: the last tokens' gradients, against the formula on these tokens alone (every other token masked)."""
    T, hc, dim, n = 1_100_000, 4, 1024, 24
    args = G._inputs(np.random.default_rng(3), n, hc, dim, masked=0.0)
    xq, kq, back = _checkpoints(args, 128)
    x = torch.zeros((T, hc, dim), dtype=torch.uint8, device="cuda")
    kv = torch.zeros((T, hc + 1, dim), dtype=torch.uint8, device="cuda")
    xs = torch.full((T, hc, dim // 128), 127, dtype=torch.uint8, device="cuda")
    ks = torch.full((T, hc + 1, dim // 128), 127, dtype=torch.uint8, device="cuda")
    x[-n:], kv[-n:] = xq[0], kq[0]
    xs[-n:], ks[-n:] = xq[1].view(torch.uint8), kq[1].view(torch.uint8)
    dout = torch.ones((T, hc, dim), dtype=torch.bfloat16, device="cuda")
    dout[-n:] = args[4].cuda()
    mask = torch.zeros(T, dtype=torch.bool, device="cuda")
    mask[-n:] = True
    got = geng.engram_gate_grad8(x, xs, kv, ks, args[2].cuda(), args[3].cuda(), dout, mask=mask, dx=dout)
    assert (got[0][: -n : 4099] == 1).all() and (got[1][: -n : 4099] == 0).all()
    G._check(back, [got[0][-n:], got[1][-n:], got[2], got[3]], "last tokens")


@pytest.mark.parametrize("block", [32, 64])
@pytest.mark.parametrize("T,hc,dim", [(900, 1, 5120), (700, 2, 5120), (600, 4, 2048), (400, 4, 5120), (200, 8, 5120)])
def test_scales_at_any_address(T, hc, dim, block):
    """Scales are read by words where they lie on 4-byte boundaries, else by bytes: the same bits."""
    args = G._inputs(np.random.default_rng(T + block), T, hc, dim)
    xq, kq, back = _checkpoints(args, block)
    want = _run8(xq, kq, back, block)
    G._check(back, want, f"T={T} hc={hc} dim={dim} block={block}")
    for off in (1, 2):
        moved = []
        for _, s in (xq, kq):
            room = torch.full((s.numel() + 8,), 255, dtype=torch.uint8, device="cuda")
            room[off:off + s.numel()] = s.view(torch.uint8).flatten()
            moved.append(room[off:off + s.numel()].view(s.shape))
        got = _run8((xq[0], moved[0]), (kq[0], moved[1]), back, block)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("T,hc,dim,block", [(3000, 4, 272, 32), (2600, 4, 512, 64), (1800, 4, 1040, 32), (1300, 4, 1280, 128),
                                            (1900, 2, 1040, 64), (1000, 2, 2304, 32), (1800, 2, 10240, 128)])
def test_scalars_and_copies_in_one_warp(T, hc, dim, block):
    rng = np.random.default_rng(T + dim)
    args = G._inputs(rng, T, hc, dim)
    args[5] = torch.from_numpy(np.repeat(rng.random(-(-T // 40)) < 0.8, 40)[:T] ^ (rng.random(T) < 0.1))
    xq, kq, back = _checkpoints(args, block)
    got = _run8(xq, kq, back, block)
    G._check(back, got, f"T={T} hc={hc} dim={dim}")
    assert all(torch.equal(a, b) for a, b in zip(got, _run8(xq, kq, back, block)))


@pytest.mark.parametrize("T,hc,dim", [(1800, 4, 1040), (1000, 2, 2304)])
def test_small_dots_with_one_warp(T, hc, dim):
    test_small_dots(T, hc, dim)


def test_withheld_sums_with_one_warp():
    test_withheld_sums_time_out_and_the_next_call_is_right(1800, 4, 1040)


@pytest.mark.parametrize("T,hc,dim", [(400, 4, 6144), (300, 4, 12288), (200, 8, 3584), (150, 8, 7168), (400, 2, 10240),
                                      (300, 1, 12288)])
def test_rows_of_three_and_six_ctas(T, hc, dim):
    args = G._inputs(np.random.default_rng(T + dim), T, hc, dim)
    xq, kq, back = _checkpoints(args, 64)
    got = _run8(xq, kq, back, 64)
    G._check(back, got, f"T={T} hc={hc} dim={dim}")
    assert all(torch.equal(a, b) for a, b in zip(got, _run8(xq, kq, back, 64)))
