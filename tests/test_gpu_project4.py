"""The projection of 4-bit operands on the tensor cores (engram_project4) against the product of their values in 64 bits
(GPU only).

Tolerance, from the arithmetic: a product of two values (code * scale each) is exact in fp32; the kernel adds the K
products in fp32 in some order (even with truncating adds each of the K - 1 additions errs by at most 2^-23 of the
running sum's magnitude, bounded by sum|a w|), multiplies by the factor (2^-24) and rounds once to bf16, by at most half
a step, 2^-8 relative: |got - exact| <= 2^-8 (|exact| + e) + e, e = (K + 1) 2^-23 sum|a w| |factor|.
Operands whose sums are whole numbers below 2^24 are exact up to that last rounding: there the bits have to be equal."""
import ctypes

import numpy as np
import pytest
import torch

import gram_hash_embedding_gb300 as geng
from tests import gpu_helpers as H
from tests import lowbit_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    H.build_all()
    yield
    assert geng.engram_device_status() == 0


def _operand(rng, rows, K, block, whole=False):
    """(codes, tiled scales, values in 64 bits): every code; scales over several powers of two, or 1 and 2."""
    codes = rng.integers(0, 16, (rows, K)).astype(np.uint8)
    n = K // block if K % block == 0 else -(-K // block)
    if whole:
        codes = np.where((codes & 7) % 2 == 1, codes & 14, codes).astype(np.uint8)  # 0, 1, 2, 4 and their negatives
        raw = rng.integers(127, 129, (rows, n)) if block == 32 else rng.choice([0x38, 0x40], (rows, n))
    else:
        raw = rng.integers(118, 126, (rows, n)) if block == 32 else rng.integers(0x10, 0x50, (rows, n))
    raw = raw.astype(np.uint8)
    v = R.values4(codes, raw, block)
    t = np.full((-(-rows // 128), -(-n // 4), 512), 0xFF if block == 32 else 0x7F, np.uint8)  # NaN where no row is
    full = np.zeros((rows, -(-n // 4) * 4), np.uint8)
    full[:, :n] = raw
    r, k = np.arange(rows)[:, None], np.arange(full.shape[1])[None, :]
    t[r // 128, k // 4, (r % 32) * 16 + (r // 32 % 4) * 4 + k % 4] = full
    return torch.from_numpy(R.pack(codes)).cuda(), torch.from_numpy(t).cuda(), torch.from_numpy(v).cuda()


def _check(got, a, w, scale, K, what):
    exact = a @ w.t() * scale
    e = (K + 1) * 2.0 ** -23 * (a.abs() @ w.abs().t()) * abs(scale)
    tol = 2.0 ** -8 * (exact.abs() + e) + e + 2.0 ** -133
    bad = ~((got.double() - exact).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first {bad.nonzero()[0].tolist()}"


SHAPES = [
    (128, 256, 128),    # whole tiles, one stage
    (1, 32, 8),         # the smallest
    (1, 6144, 520),     # one token
    (2, 96, 1000),      # K over one and a half MMAs
    (16, 2080, 3000),   # few tokens: K split over the CTAs of a cluster, in odd parts
    (17, 6144, 136),
    (33, 288, 264),     # K past one stage by half an MMA
    (64, 768, 25608),   # more row blocks of w than CTAs fit at once
    (65, 1120, 4000),
    (129, 512, 1000),
    (200, 2048, 9000),
    (200, 544, 20008),  # one wave of the widest tiles
    (300, 96, 12008),
    (300, 544, 520),    # ragged everywhere
    (257, 1024, 2056),
    (1000, 3 * 256, 1032),
    (2200, 96, 2056),   # more tiles than pairs of SMs: both accumulators in turn
    (5000, 512, 4104),  # and wide tiles
]


@pytest.mark.parametrize("block", [32, 16])
@pytest.mark.parametrize("T,K,N", SHAPES)
def test_project4(block, T, K, N):
    rng = np.random.default_rng(T + K + N)
    a, sa, va = _operand(rng, T, K, block)
    w, sw, vw = _operand(rng, N, K, block)
    out = torch.full((T * N + 256,), -7.0, dtype=torch.bfloat16, device="cuda")
    got = geng.engram_project4(a, sa, w, sw, block, scale=0.75, out=out[128:-128].view(T, N))
    _check(got, va, vw, 0.75, K, f"T={T} K={K} N={N} block={block}")
    assert (out[:128] == -7).all() and (out[-128:] == -7).all()
    again = geng.engram_project4(a, sa, w, sw, block, scale=0.75)
    assert torch.equal(got, again)


@pytest.mark.parametrize("block", [32, 16])
@pytest.mark.parametrize("T,K,N", [(1, 32, 8), (5, 160, 136), (130, 512, 264), (700, 320, 1000), (3000, 256, 4104)])
def test_whole_numbers_are_exact(block, T, K, N):
    rng = np.random.default_rng(T + K)
    a, sa, va = _operand(rng, T, K, block, whole=True)
    w, sw, vw = _operand(rng, N, K, block, whole=True)
    got = geng.engram_project4(a, sa, w, sw, block)
    assert torch.equal(got, (va @ vw.t()).to(torch.float32).to(torch.bfloat16))


@pytest.mark.parametrize("block", [32, 16])
def test_one_hot_columns(block):
    """A single code in each row of w picks one column of a with its own scale: the layouts of codes and scales."""
    T, K, N = 200, 640, 640
    rng = np.random.default_rng(3)
    a, sa, va = _operand(rng, T, K, block)
    codes = np.zeros((N, K), np.uint8)
    codes[np.arange(N), np.arange(N)] = 2  # 1.0
    raw = (rng.integers(120, 130, (N, K // block)) if block == 32 else rng.integers(0x20, 0x48, (N, K // block))).astype(np.uint8)
    w, sw = torch.from_numpy(R.pack(codes)).cuda(), torch.from_numpy(R.tile(raw)).cuda()
    vw = torch.from_numpy(R.values4(codes, raw, block)).cuda()
    got = geng.engram_project4(a, sa, w, sw, block)
    assert torch.equal(got, (va @ vw.t()).to(torch.float32).to(torch.bfloat16))


def test_chain_from_ids_and_from_values():
    """The 4-bit block as it is used: a table and weights quantised once, rows gathered as they stand or quantised from
    bf16, the projection, then the gate; a second call on another stream while the first is in flight."""
    g = torch.Generator(device="cuda").manual_seed(6)
    rows, C, dim, T, hc, width, block = 3000, 6, 64, 300, 2, 256, 32
    table = torch.randn((rows, dim), generator=g, device="cuda") * 0.1
    wkv = torch.randn(((hc + 1) * width, C * dim), generator=g, device="cuda") * (C * dim) ** -0.5
    Q, S = geng.engram_quantize4(table, block)
    wq, ws = geng.engram_quantize4(wkv, block, tiled=True)
    idx = torch.randint(-1, rows, (T, C), generator=g, device="cuda")
    a, sa = geng.engram_lookup4_operand(idx, Q, S, block)
    kv = geng.engram_project4(a, sa, wq, ws, block)
    va = geng.engram_lookup4(idx, Q, S, block).view(T, -1).double()
    vw = geng.engram_dequantize4(wq, ws, block, tiled=True, out_dtype=torch.float32).double()
    _check(kv, va, vw, 1.0, C * dim, "from ids")
    # values of a looked-up row are their own quantisation
    b, sb = geng.engram_quantize4(va.bfloat16(), block, tiled=True)
    assert torch.equal(geng.engram_project4(b, sb, wq, ws, block), kv)
    x = torch.randn((T, hc, width), generator=g, device="cuda").bfloat16()
    q = torch.ones((hc, width), dtype=torch.bfloat16, device="cuda")
    y = geng.engram_gate(x, kv, q, q)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    kv2 = geng.engram_project4(a, sa, wq, ws, block, stream=s)
    kv3 = geng.engram_project4(b, sb, wq, ws, block)
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(kv2, kv) and torch.equal(kv3, kv) and torch.isfinite(y).all()


@pytest.mark.parametrize("block", [32, 16])
@pytest.mark.parametrize("T", [20, 100, 300])
def test_a_nan_block_stays_in_its_row_and_column(block, T):
    """A NaN or an infinity among the values makes its block's scale NaN: that token's outputs are NaN, a weight's
    likewise its column, and every other output is as without it."""
    K, N = 320, 776
    g = torch.Generator(device="cuda").manual_seed(T)
    x, w = torch.randn((T, K), generator=g, device="cuda"), torch.randn((N, K), generator=g, device="cuda")
    run = lambda: geng.engram_project4(*geng.engram_quantize4(x, block, tiled=True),  # noqa: E731
                                       *geng.engram_quantize4(w, block, tiled=True), block)
    want = run()
    x[7, 100], x[T - 1, 319], w[300, 0] = float("nan"), float("-inf"), float("inf")
    got = run()
    nan = torch.zeros((T, N), dtype=torch.bool, device="cuda")
    nan[7], nan[T - 1], nan[:, 300] = True, True, True
    assert torch.equal(torch.isnan(got), nan) and torch.equal(got[~nan], want[~nan])


def test_outputs_beyond_32_bits():
    """More than 2^32 outputs: the last rows and columns are in place."""
    T, K, N, block = 170_000, 64, 25608, 32
    rng = np.random.default_rng(1)
    w, sw, vw = _operand(rng, N, K, block)
    x = torch.randn((T, K), device="cuda")
    a, sa = geng.engram_quantize4(x, block, tiled=True)
    got = geng.engram_project4(a, sa, w, sw, block)
    va = geng.engram_dequantize4(a, sa, block, tiled=True, out_dtype=torch.float32)
    for rows in (slice(0, 3), slice(T // 2, T // 2 + 3), slice(T - 300, T)):
        _check(got[rows], va[rows].double(), vw, 1.0, K, str(rows))


def test_calls_of_several_streams_at_once():
    """Few-token calls of different sizes and one of many tokens, in flight together."""
    rng = np.random.default_rng(5)
    block, K, N = 16, 1024, 6000
    w, sw, vw = _operand(rng, N, K, block)
    ops = [_operand(rng, T, K, block) for T in (1, 20, 50, 128, 700)]
    want = [geng.engram_project4(a, sa, w, sw, block) for a, sa, _ in ops]
    streams = [torch.cuda.Stream() for _ in ops]
    torch.cuda.synchronize()
    for _ in range(20):
        got = []
        for (a, sa, _), s in zip(ops, streams):
            got.append(geng.engram_project4(a, sa, w, sw, block, stream=s))
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_graph_replays_with_new_inputs():
    T, K, N, block = 70, 512, 776, 16
    rng = np.random.default_rng(9)
    a, sa, _ = _operand(rng, T, K, block)
    w, sw, vw = _operand(rng, N, K, block)
    out = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    geng.engram_project4(a, sa, w, sw, block, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        geng.engram_project4(a, sa, w, sw, block, out=out)
    for seed in range(2):
        b, sb, vb = _operand(np.random.default_rng(seed), T, K, block)
        a.copy_(b)
        sa.copy_(sb)
        graph.replay()
        _check(out, vb, vw, 1.0, K, "replay")


@pytest.mark.parametrize("T", [64, 2000])
def test_a_withheld_tile_times_out_and_the_next_call_is_right(T):
    L = geng._lib()
    P, I64, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    L.engram_project4_withhold.argtypes = [P, P, P, P, I64, I32, I32, I32, ctypes.c_float, P, I32, P]
    L.engram_project4_withhold.restype = ctypes.c_int
    K, N, block = 256, 1024, 32
    rng = np.random.default_rng(T)
    a, sa, va = _operand(rng, T, K, block)
    w, sw, vw = _operand(rng, N, K, block)
    out = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    rc = L.engram_project4_withhold(a.data_ptr(), sa.data_ptr(), w.data_ptr(), sw.data_ptr(), T, K, N, block, 1.0,
                                    out.data_ptr(), 0, torch.cuda.current_stream().cuda_stream)
    assert rc == geng.OK
    assert geng.engram_device_status() == geng.STATUS_TIMEOUT
    _check(geng.engram_project4(a, sa, w, sw, block), va, vw, 1.0, K, "after the timeout")
    assert geng.engram_device_status() == 0
