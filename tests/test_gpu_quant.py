"""Block-scaled quantisation and reading back (engram_quantize4 / 8, engram_dequantize4 / 8) against the formats'
definition in 64 bits (GPU only). Codes and scales have to be equal: the choice of a code is that of exact arithmetic.
Values read back are exact in fp32; in bf16 and fp16 they round once, as numpy's and torch's conversions do."""
import numpy as np
import pytest
import torch

import gram_hash_embedding_gb300 as geng
from tests import gpu_helpers as H
from tests import lowbit_ref as R

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    H.build_all()
    yield
    assert geng.engram_device_status() == 0


def _host(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def _values(rng, rows, cols, dtype):
    """Values of many sizes; zeros, blocks of zeros, exact borders between codes, values next to them, signed zeros."""
    x = rng.standard_normal((rows, cols)) * 2.0 ** rng.integers(-9, 9, (rows, 1))
    x *= np.where(rng.random((rows, cols)) < 0.1, 0.0, 1.0) * np.exp(rng.standard_normal((rows, cols)))
    border = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -2.5, -5.0], (rows, cols)) * \
        2.0 ** rng.integers(-3, 4, (rows, 1)) * (1 + rng.integers(0, 8, (rows, 1)) / 8)
    nudge = np.where(rng.random((rows, cols)) < 0.3, rng.integers(-2, 3, (rows, cols)) * 2.0 ** -23, 0.0)
    x = np.where(rng.random((rows, 1)) < 0.5, border * (1 + nudge), x)
    x[rng.random((rows, cols)) < 0.02] = -0.0
    x[:, : min(cols, 32)] *= (rng.random((rows, 1)) > 0.2)
    return torch.from_numpy(x.astype(np.float32)).to(TYPES[dtype])


@pytest.mark.parametrize("block", [32, 16])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (129, 160), (300, 1024), (5, 6144), (1000, 64), (257, 224)])
def test_quantize4(block, dtype, rows, cols):
    rng = np.random.default_rng(rows * 7 + cols + block)
    x = _values(rng, rows, cols, dtype)
    for factor in (1.0, 2.0 ** -5):
        want, raw = R.quantise(x.double().numpy(), block, 4, factor)
        codes, scales = geng.engram_quantize4(x.cuda(), block, scale=factor)
        assert codes.shape == (rows, cols // 2) and scales.shape == (rows, cols // block)
        assert np.array_equal(_host(scales), raw)
        assert np.array_equal(R.unpack(_host(codes)), want)
        tcodes, tiled = geng.engram_quantize4(x.cuda(), block, scale=factor, tiled=True)
        assert torch.equal(tcodes, codes) and tiled.numel() == geng.engram_tiled_scales(rows, cols, block)
        # the row's whole last group is written, zeros past its scales
        n = -(-cols // (4 * block)) * 4
        t = R.untile(_host(tiled), rows, n)
        assert np.array_equal(t[:, :raw.shape[1]], raw) and (t[:, raw.shape[1]:] == 0).all()
        v = R.values4(want, raw, block) * factor
        for out in (torch.float32, torch.bfloat16, torch.float16):
            got = geng.engram_dequantize4(codes, scales, block, scale=factor, out_dtype=out)
            exp = torch.from_numpy(v).to(torch.float32).to(out)
            assert torch.equal(got.cpu(), exp), out
            again = geng.engram_dequantize4(codes, tiled, block, scale=factor, tiled=True, out_dtype=out)
            assert torch.equal(again, got)


@pytest.mark.parametrize("block", [32, 64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols", [(1, 8), (3, 104), (129, 128), (77, 1040), (40, 5120), (1000, 24), (9, 1000)])
def test_quantize8(block, dtype, rows, cols):
    rng = np.random.default_rng(rows * 5 + cols + block)
    x = _values(rng, rows, cols, dtype)
    want, raw = R.quantise(x.double().numpy(), block, 8)
    v = R.values8(want, raw, block)
    for sdt, kind in ((geng.SCALE_E8M0, None), (geng.SCALE_F32, torch.float32), (geng.SCALE_BF16, torch.bfloat16)):
        codes, scales = geng.engram_quantize8(x.cuda(), block, sdt)
        assert np.array_equal(_host(codes), want)
        if kind is None:
            assert np.array_equal(_host(scales), raw)
        else:
            assert scales.dtype == kind and np.array_equal(scales.double().cpu().numpy(), 2.0 ** (raw - 127.0))
        for out in (torch.float32, torch.bfloat16, torch.float16):
            got = geng.engram_dequantize8(codes, scales, block, out_dtype=out)
            assert torch.equal(got.cpu(), torch.from_numpy(v).to(torch.float32).to(out)), (sdt, out)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_extremes(dtype):
    """The type's largest and smallest values, subnormal blocks, infinities and NaN: a block that holds one of these
    reads back as NaN, its neighbours are as without it."""
    t = TYPES[dtype]
    f = torch.finfo(t)
    x = torch.zeros((8, 128), dtype=t)
    x[0] = f.max
    x[1, ::3] = f.tiny
    x[2, 5] = -f.smallest_normal
    x[3] = f.eps
    x[4, 0::32] = f.max
    x[4, 1::32] = f.tiny
    x[5, 40] = float("nan")
    x[6, 100] = float("-inf")
    x[5, 0], x[6, 1] = 3.0, -5.0
    x[7, 64] = float("inf")
    if dtype != "f16":
        x[2] = torch.arange(128).to(torch.float32).mul(2.0 ** -133).to(t)  # subnormal
    for block in (32, 16):
        want, raw = R.quantise(x.double().numpy(), block, 4)
        codes, scales = geng.engram_quantize4(x.cuda(), block)
        assert np.array_equal(_host(scales), raw) and np.array_equal(R.unpack(_host(codes)), want)
        got = geng.engram_dequantize4(codes, scales, block, out_dtype=torch.float32).cpu()
        exp = torch.from_numpy(R.values4(want, raw, block)).float()
        assert torch.equal(torch.isnan(got), torch.isnan(exp)) and torch.isnan(got[5]).sum() == block
        assert torch.equal(got.nan_to_num(), exp.nan_to_num())
    for block in (32, 64, 128):
        want, raw = R.quantise(x.double().numpy(), block, 8)
        codes, scales = geng.engram_quantize8(x.cuda(), block)
        assert np.array_equal(_host(scales), raw) and np.array_equal(_host(codes), want)
        got = geng.engram_dequantize8(codes, scales, block, out_dtype=torch.float32).cpu()
        exp = torch.from_numpy(R.values8(want, raw, block)).float()
        assert torch.equal(torch.isnan(got), torch.isnan(exp)) and torch.isnan(got[5]).sum() == block
        assert torch.equal(got.nan_to_num(), exp.nan_to_num())


def test_strides_shapes_and_bounds():
    """Rows a stride apart, leading dimensions, outputs given by the caller, and nothing written past them."""
    g = torch.Generator(device="cuda").manual_seed(3)
    wide = torch.randn((50, 256), generator=g, device="cuda").bfloat16()
    x = wide[:, 64:160]
    a, b = geng.engram_quantize4(x, 32), geng.engram_quantize4(x.contiguous(), 32)
    assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(a, b))
    a, b = geng.engram_quantize8(x, 64), geng.engram_quantize8(x.contiguous(), 64)
    assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(a, b))
    deep = torch.randn((7, 3, 96), generator=g, device="cuda")
    codes, scales = geng.engram_quantize4(deep, 16)
    assert codes.shape == (7, 3, 48) and scales.shape == (7, 3, 6)
    assert geng.engram_dequantize4(codes, scales, 16).shape == deep.shape
    codes, scales = geng.engram_quantize8(deep, 64)
    assert codes.shape == deep.shape and scales.shape == (7, 3, 2)
    for quant, n_codes, n_scales in ((lambda c, s: geng.engram_quantize4(wide, 32, codes=c, scales=s), 50 * 128, 400),
                                     (lambda c, s: geng.engram_quantize8(wide, 128, codes=c, scales=s), 50 * 256, 100)):
        whole = torch.full((n_codes + n_scales + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        c, s = whole[128:128 + n_codes], whole[n_codes + 256:n_codes + 256 + n_scales]
        quant(c, s)
        assert (whole[:128] == 0xA5).all() and (whole[128 + n_codes:n_codes + 256] == 0xA5).all()
        assert (whole[n_codes + 256 + n_scales:] == 0xA5).all()
    # tiled scales: of the last 128 rows only the given ones are written
    tiled = torch.full((1, 2, 512), 0xA5, dtype=torch.uint8, device="cuda")
    geng.engram_quantize4(wide, 32, tiled=True, scales=tiled)
    raw = R.untile(tiled.cpu().numpy(), 128, 8)
    assert (raw[50:] == 0xA5).all() and (raw[:50] < 0xA5).all()
    for empty in (torch.empty((0, 64), device="cuda"), torch.empty((0, 3, 64), device="cuda")):
        codes, scales = geng.engram_quantize4(empty)
        assert codes.shape == (*empty.shape[:-1], 32) and scales.shape == (*empty.shape[:-1], 2)
        assert geng.engram_dequantize4(codes, scales, 32).shape == empty.shape
        codes, scales = geng.engram_quantize8(empty)
        assert geng.engram_dequantize8(codes, scales, 128).shape == empty.shape


def test_a_table_for_the_lookup():
    """Trained rows as a serving table: engram_quantize8's codes and scales are what engram_lookup takes."""
    g = torch.Generator(device="cuda").manual_seed(5)
    rows = torch.randn((500, 256), generator=g, device="cuda") * 0.02
    idx = torch.randint(-1, 501, (37, 6), generator=g, device="cuda")
    for sdt in (geng.SCALE_F32, geng.SCALE_BF16, geng.SCALE_E8M0):
        W, S = geng.engram_quantize8(rows, 128, sdt)
        got = geng.engram_lookup(idx, W, S, 128)
        ok = (idx >= 0) & (idx < 500)
        exp = torch.where(ok[..., None], geng.engram_dequantize8(W, S, 128)[idx.clamp(0, 499)], 0.0)
        assert torch.equal(got, exp.to(torch.bfloat16))


def test_other_stream_and_graph():
    x = torch.randn((300, 512), device="cuda").bfloat16()
    torch.cuda.synchronize()
    codes, scales = geng.engram_quantize4(x, 16)
    s = torch.cuda.Stream()
    c2, s2 = geng.engram_quantize4(x, 16, stream=s)
    v2 = geng.engram_dequantize4(c2, s2, 16, stream=s)
    s.synchronize()
    assert torch.equal(codes, c2) and torch.equal(v2, geng.engram_dequantize4(codes, scales, 16))
    q = torch.empty_like(codes)
    sc = torch.empty_like(scales)
    out = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        geng.engram_quantize4(x, 16, codes=q, scales=sc)
        geng.engram_dequantize4(q, sc, 16, out=out)
    for seed in range(2):
        x.copy_(torch.randn((300, 512), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda"))
        graph.replay()
        assert torch.equal(out, geng.engram_dequantize4(*geng.engram_quantize4(x, 16), 16))


def test_values_beyond_32_bits():
    """More than 2^32 values: the last rows, there and back."""
    rows, cols = 68_000_000, 64
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    tail = torch.randn((40, cols), device="cuda").bfloat16()
    x[-40:] = tail
    for block in (32, 16):
        for tiled in (False, True):
            codes, scales = geng.engram_quantize4(x, block, tiled=tiled)
            c, s = geng.engram_quantize4(tail, block)
            assert torch.equal(codes[-40:], c)
            back = geng.engram_dequantize4(codes, scales, block, tiled=tiled)
            assert torch.equal(back[-40:], geng.engram_dequantize4(c, s, block))
            del codes, scales, back
    codes, scales = geng.engram_quantize8(x, 32)
    c, s = geng.engram_quantize8(tail, 32)
    assert torch.equal(codes[-40:], c) and torch.equal(scales[-40:].view(torch.uint8), s.view(torch.uint8))
    assert torch.equal(geng.engram_dequantize8(codes, scales, 32)[-40:], geng.engram_dequantize8(c, s, 32))
