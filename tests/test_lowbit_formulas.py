"""The low-bit operators without a GPU: the formats' reference against torch's own conversions and brute force, and
what the entry points refuse."""
import ctypes
import itertools

import numpy as np
import pytest
import torch

import gram_hash_embedding_gb300 as geng
from tests import lowbit_ref as R

P, I64, I32, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    geng.build()
    return geng._lib()


def test_e4m3_grid_is_torchs():
    codes = torch.arange(127, dtype=torch.uint8)
    assert np.array_equal(codes.view(torch.float8_e4m3fn).double().numpy(), R.E4M3)
    v = np.abs(np.random.default_rng(0).standard_normal(20000).astype(np.float32)) * 100
    v = np.concatenate([v, (R.E4M3[1:] + R.E4M3[:-1]).astype(np.float32) / 2])
    v = v[v < 448]
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(R.nearest(v.astype(np.float64), R.E4M3), want)


def test_e2m1_by_brute_force():
    v = np.concatenate([np.linspace(0, 7, 1401), (R.E2M1[1:] + R.E2M1[:-1]) / 2])
    got = R.nearest(v, R.E2M1)
    for x, g in zip(v, got):
        d = np.abs(R.E2M1 - x)
        best = np.flatnonzero(d == d.min())
        assert g == (best[0] if best.size == 1 else best[best % 2 == 0][0])


@pytest.mark.parametrize("bits,block", [(4, 32), (4, 16), (8, 32), (8, 128)])
def test_quantise_never_leaves_a_nearer_code(bits, block):
    rng = np.random.default_rng(bits + block)
    x = rng.standard_normal((20, 256)) * 2.0 ** rng.integers(-20, 6, (20, 1))
    codes, raw = R.quantise(x, block, bits)
    v = R.values4(codes, raw, block) if bits == 4 else R.values8(codes, raw, block)
    s = np.repeat(R.scale_value(raw, not (bits == 4 and block == 16)), block, 1)
    grid = R.E2M1 if bits == 4 else R.E4M3
    best = np.abs(np.abs(x)[..., None] - s[..., None] * grid).min(-1)
    assert np.array_equal(np.abs(x - v), best)
    if not (bits == 4 and block == 16):  # a power of two that holds the block, and no smaller one does
        amax = np.abs(R.blocks(x, block)).max(-1)
        sv = R.scale_value(raw, True)
        assert (amax <= grid[-1] * sv).all() and (amax > grid[-1] * sv / 2).all()


def test_tiles_there_and_back():
    raw = np.random.default_rng(1).integers(0, 256, (300, 11)).astype(np.uint8)
    t = R.tile(raw)
    assert t.shape == (3, 3, 512) and np.array_equal(R.untile(t, 300, 11), raw)


def test_tiled_scale_bytes(lib):
    for rows, cols, block in itertools.product((1, 128, 129, 5000), (32, 64, 160, 6144), (16, 32)):
        assert lib.engram_tiled_scales(rows, cols, block) == R.tile(np.zeros((rows, cols // block), np.uint8)).size
    for bad in ((0, 32, 32), (-1, 32, 32), (4, 48, 16), (4, 32, 8), (4, 0, 32), (1 << 40, 6144, 32)):
        assert lib.engram_tiled_scales(*bad) == 0


# rejected before anything is launched: the pointers are never dereferenced
A = 1 << 20


def test_quantize_refusals(lib):
    def q4(x=A, rows=4, cols=64, stride=64, t=1, block=32, scale=1.0, tiled=0, codes=A, scales=A):
        return lib.engram_quantize4(x, rows, cols, stride, t, block, scale, tiled, codes, scales, None)

    for kw in ({"block": 8}, {"block": 64}, {"cols": 48}, {"cols": 0}, {"cols": 80, "block": 16, "tiled": 1, "stride": 80},
               {"rows": 1 << 40, "cols": 64}):
        assert q4(**kw) == geng.ERR_UNSUPPORTED, kw
    for kw in ({"x": None}, {"codes": None}, {"scales": None}, {"x": A + 8}, {"codes": A + 8}, {"scales": A + 8},
               {"rows": -1}, {"stride": 56}, {"stride": 68}, {"t": 3}, {"scale": 0.0}, {"scale": 3.0}, {"scale": -2.0},
               {"scale": float("inf")}, {"scale": float("nan")}, {"scale": 2.0 ** -130}):
        assert q4(**kw) == geng.ERR_INVALID, kw
    assert q4(rows=0, x=None, codes=None, scales=None) == geng.OK

    def q8(x=A, rows=4, cols=64, stride=64, t=1, block=32, sdt=geng.SCALE_E8M0, codes=A, scales=A):
        return lib.engram_quantize8(x, rows, cols, stride, t, block, sdt, codes, scales, None)

    for kw in ({"block": 16}, {"cols": 12}, {"sdt": geng.SCALE_E4M3}, {"sdt": 7}, {"rows": 1 << 41}):
        assert q8(**kw) == geng.ERR_UNSUPPORTED, kw
    for kw in ({"x": None}, {"codes": A + 4}, {"scales": A + 2, "sdt": geng.SCALE_F32}, {"scales": A + 1, "sdt": geng.SCALE_BF16},
               {"rows": -1}, {"stride": 63}, {"t": -1}):
        assert q8(**kw) == geng.ERR_INVALID, kw
    assert q8(rows=0, x=None, codes=None, scales=None) == geng.OK

    def d4(codes=A, scales=A, rows=4, cols=64, block=32, scale=1.0, tiled=0, out=A, t=1):
        return lib.engram_dequantize4(codes, scales, rows, cols, block, scale, tiled, out, t, None)

    assert d4(block=24) == d4(cols=40) == geng.ERR_UNSUPPORTED
    for kw in ({"codes": None}, {"out": A + 4}, {"scales": A + 1}, {"scale": float("nan")}, {"t": 9}, {"rows": -1}):
        assert d4(**kw) == geng.ERR_INVALID, kw
    assert d4(rows=0, codes=None, scales=None, out=None) == geng.OK

    def d8(codes=A, scales=A, rows=4, cols=64, block=32, sdt=geng.SCALE_BF16, out=A, t=1):
        return lib.engram_dequantize8(codes, scales, rows, cols, block, sdt, out, t, None)

    assert d8(block=48) == d8(cols=4) == d8(sdt=geng.SCALE_E4M3) == geng.ERR_UNSUPPORTED
    assert d8(codes=None) == d8(scales=A + 1) == d8(out=A + 8) == d8(t=5) == geng.ERR_INVALID


def test_lookup_refusals(lib):
    def l4(idx=A, stride=3, T=5, C=3, Q=A, S=A, rows=9, dim=64, block=32, scale=1.0, out=A):
        return lib.engram_lookup4(idx, stride, T, C, Q, S, rows, dim, block, scale, out, None)

    for kw in ({"block": 128}, {"dim": 48}, {"dim": 0}, {"dim": 1 << 17}, {"T": 1 << 30}):
        assert l4(**kw) == geng.ERR_UNSUPPORTED, kw
    for kw in ({"idx": None}, {"idx": A + 4}, {"stride": 2}, {"T": -1}, {"C": 0}, {"Q": None}, {"Q": A + 8}, {"S": None},
               {"rows": -1}, {"out": None}, {"out": A + 8}, {"scale": float("inf")}):
        assert l4(**kw) == geng.ERR_INVALID, kw
    assert l4(T=0, idx=None, Q=None, S=None, out=None) == geng.OK

    def lo(C=3, dim=64, block=32, codes=A, scales=A, T=5):
        return lib.engram_lookup4_operand(A, C, T, C, A, A, 9, dim, block, codes, scales, None)

    assert lo(C=1, dim=48, block=16) == geng.ERR_UNSUPPORTED  # K not a multiple of 32
    assert lo(codes=None) == lo(scales=A + 8) == lo(codes=A + 8) == geng.ERR_INVALID
    assert lo(T=0, codes=None) == geng.OK


def test_project_refusals(lib):
    def p4(a=A, sa=A, w=A, sw=A, T=5, K=64, N=16, block=32, scale=1.0, out=A):
        return lib.engram_project4(a, sa, w, sw, T, K, N, block, scale, out, None)

    for kw in ({"block": 64}, {"K": 48}, {"K": 0}, {"N": 12}, {"N": 0}, {"T": 1 << 31}, {"N": (1 << 31) - 8},
               {"T": (1 << 31) - 1, "K": 1 << 20}):
        assert p4(**kw) == geng.ERR_UNSUPPORTED, kw
    for kw in ({"a": None}, {"sa": None}, {"w": None}, {"sw": None}, {"out": None}, {"a": A + 8}, {"sa": A + 64},
               {"sw": A + 16}, {"out": A + 8}, {"T": -1}, {"scale": float("nan")}):
        assert p4(**kw) == geng.ERR_INVALID, kw
    assert p4(T=0, a=None, sa=None, w=None, sw=None, out=None) == geng.OK
    hook = lib.engram_project4_withhold
    hook.argtypes, hook.restype = [P, P, P, P, I64, I32, I32, I32, F, P, I32, P], ctypes.c_int
    assert hook(A, A, A, A, 5, 64, 16, 32, 1.0, A, -1, None) == geng.ERR_INVALID


def test_gate_grad8_refusals(lib):
    def g8(x=A, xs=A, kv=A, ks=A, block=128, q=A, T=4, hc=2, dim=64, ws=1 << 30, dout=A, space=A):
        return lib.engram_gate_grad8(x, xs, kv, ks, block, q, A, dout, None, T, hc, dim, 1e-20, A, A, A, A, space, ws, None)

    for kw in ({"block": 16}, {"block": 256}, {"dim": 72}, {"hc": 3}, {"dim": 0}, {"dim": 32768}, {"T": 1 << 31}):
        assert g8(**kw) == geng.ERR_UNSUPPORTED, kw
    for kw in ({"x": None}, {"xs": None}, {"ks": None}, {"kv": A + 8}, {"x": A + 8}, {"q": None}, {"dout": A + 8}, {"T": -1},
               {"ws": 0}, {"space": A + 16}):
        assert g8(**kw) == geng.ERR_INVALID, kw
    assert lib.engram_gate_grad8_workspace(0, 2, 64) == lib.engram_gate_grad8_workspace(4, 2, 72) == 0


def test_gate_grad8_workspace_never_falls(lib):
    for hc, dim in itertools.product((1, 2, 4, 8), (16, 96, 1040, 2064, 5120, 16384)):
        sizes = [lib.engram_gate_grad8_workspace(T, hc, dim) for T in (1, 2, 3, 9, 40, 76, 77, 152, 153, 400, 1000, 5000, 40000)]
        assert all(b >= a for a, b in zip(sizes, sizes[1:])), (hc, dim, sizes)


def test_binding_refuses_before_any_pointer():
    """Shapes and types are refused before a pointer is taken; CPU tensors get that far."""
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    for bad in (8, 64, 0):
        with pytest.raises(ValueError, match="block"):
            geng.engram_quantize4(torch.zeros((2, 64)), bad)
        with pytest.raises(ValueError, match="block"):
            geng.engram_quantize8(torch.zeros((2, 64)), 16)
    with pytest.raises(TypeError, match="CUDA"):
        geng.engram_quantize4(torch.zeros((2, 64)))
    with pytest.raises(ValueError, match="scale_dtype"):
        geng.engram_quantize8(torch.zeros((2, 64)), 64, geng.SCALE_E4M3)
    with pytest.raises(ValueError, match="multiple of 32"):
        geng.engram_dequantize4(u8(2, 8), u8(2, 1), 32)
    with pytest.raises(ValueError, match="whole blocks"):
        geng.engram_lookup4(torch.zeros(3, dtype=torch.int64), u8(5, 24), u8(5, 1), 32)
    with pytest.raises(ValueError, match="S has"):
        geng.engram_lookup4(torch.zeros(3, dtype=torch.int64), _fake(5, 32), _fake(5, 3), 32)
    with pytest.raises(ValueError, match="w must be"):
        geng.engram_project4(u8(2, 32), u8(1, 1, 512), u8(8, 16), u8(1, 1, 512), 32)
    with pytest.raises(ValueError, match="not a multiple of 32"):
        geng.engram_project4(u8(2, 8), u8(1, 1, 512), u8(8, 8), u8(1, 1, 512), 32)
    with pytest.raises(ValueError, match="a has|a_scales has"):
        geng.engram_project4(_fake(2, 32), _fake(1, 2, 512), _fake(8, 32), _fake(1, 1, 512), 32, out=torch.empty(2, 8))


class _OnDevice(torch.Tensor):
    is_cuda = True


def _fake(*shape, dtype=torch.uint8):
    return torch.zeros(shape, dtype=dtype).as_subclass(_OnDevice)


def test_gate_grad8_binding_sizes():
    x, k = _fake(3, 2, 64), _fake(3, 3, 64)
    w = torch.zeros((2, 64), dtype=torch.bfloat16)
    ok = dict(dx=_fake(3, 2, 64, dtype=torch.bfloat16), dkv=_fake(3, 192, dtype=torch.bfloat16),
              dq_weight=_fake(2, 64, dtype=torch.float32), dk_weight=_fake(2, 64, dtype=torch.float32))
    for args, what in (((x, _fake(3, 2, 2), k, _fake(3, 3, 1)), "x_scales has"), ((x, _fake(3, 2, 1), k, _fake(3, 3, 2)), "kv_scales has"),
                       ((x, _fake(3, 2, 1), _fake(3, 2, 64), _fake(3, 3, 1)), "kv has")):
        with pytest.raises(ValueError, match=what):
            geng.engram_gate_grad8(*args, w, w, x.to(torch.bfloat16), block=64, **ok)
    with pytest.raises(TypeError, match="x must be"):
        geng.engram_gate_grad8(x.to(torch.bfloat16), _fake(3, 2, 1), k, _fake(3, 3, 1), w, w, x, block=64, **ok)


def test_tensors_of_another_device_are_refused(monkeypatch):
    class On:
        def __init__(self, index):
            self.index, self.device = index, f"cuda:{index}"

        def get_device(self):
            return self.index

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(geng, "_raw_stream", lambda dev: 7)
    assert geng._stream_on((On(0), None), None, (On(0),)) == 7
    for inputs, temps in (((On(1),), ()), ((On(0), On(1)), ()), ((On(0),), (On(1),)), ((None, On(0)), (On(0), On(1)))):
        with pytest.raises(ValueError, match="cuda:1, the current device is cuda:0"):
            geng._stream_on(inputs, None, temps)
