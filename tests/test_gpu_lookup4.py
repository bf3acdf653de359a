"""Rows of 4-bit tables (engram_lookup4, engram_lookup4_operand) against the table's values in 64 bits (GPU only).
Every result is exact: a value has at most six significant bits."""
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


def _table(rng, rows, dim, block):
    """Codes and scales as a program holds them, and their values."""
    codes = rng.integers(0, 16, (rows, dim)).astype(np.uint8)
    raw = (rng.integers(110, 140, (rows, dim // block)) if block == 32 else rng.integers(0, 0x7F, (rows, dim // block))).astype(np.uint8)
    return torch.from_numpy(R.pack(codes)).cuda(), torch.from_numpy(raw).cuda(), codes, raw


@pytest.mark.parametrize("block", [32, 16])
@pytest.mark.parametrize("T,C,dim,rows", [(1, 1, 32, 5), (1, 24, 128, 1000), (37, 3, 96, 77), (130, 24, 256, 5000),
                                          (513, 2, 64, 300), (64, 5, 512, 100), (3, 1, 6144, 9), (700, 7, 160, 2000)])
def test_lookup4(block, T, C, dim, rows):
    rng = np.random.default_rng(T + dim)
    Q, S, codes, raw = _table(rng, rows, dim, block)
    idx = rng.integers(-3, rows + 3, (T, C))
    ok = (idx >= 0) & (idx < rows)
    at = np.where(ok, idx, 0)
    v = np.where(ok[..., None], R.values4(codes, raw, block)[at], 0.0)
    ids = torch.from_numpy(idx).cuda()
    for scale in (1.0, 0.125):
        exp = torch.from_numpy(v * scale).to(torch.float32).to(torch.bfloat16)
        got = geng.engram_lookup4(ids, Q, S, block, scale=scale)
        assert got.shape == (T, C, dim) and torch.equal(got.cpu(), exp)
    dtyped = S.view(torch.float8_e4m3fn) if block == 16 else S.view(torch.float8_e8m0fnu)
    assert torch.equal(geng.engram_lookup4(ids, Q, dtyped, block, scale=0.125), got)
    # one layer's slice of a wider tensor of ids; any contiguous shape
    wide = torch.full((T, 3, C), 10 ** 12, device="cuda", dtype=torch.int64)
    wide[:, 1] = ids
    assert torch.equal(geng.engram_lookup4(wide[:, 1], Q, S, block, scale=0.125), got)
    assert torch.equal(geng.engram_lookup4(ids.reshape(-1), Q, S, block, scale=0.125), got.view(-1, dim))
    if C * dim % 32 == 0:
        pad = torch.full((geng.engram_tiled_scales(T, C * dim, block) + 256,), 0xA5, dtype=torch.uint8, device="cuda")
        oc, os = geng.engram_lookup4_operand(wide[:, 1], Q, S, block, scales=pad[128:-128])
        want = np.where(ok[..., None], codes[at], 0).reshape(T, -1)
        assert np.array_equal(R.unpack(oc.cpu().numpy()), want)
        n = C * dim // block
        groups = -(-n // 4) * 4
        t = R.untile(os.cpu().numpy().reshape(-1, groups // 4, 512), -(-T // 128) * 128, groups)
        assert np.array_equal(t[:T, :n], np.where(ok[..., None], raw[at], 0).reshape(T, -1))
        assert (t[:T, n:] == 0).all() and (t[T:] == 0xA5).all()  # the last group in full, no row past the last
        assert (pad[:128] == 0xA5).all() and (pad[-128:] == 0xA5).all()
        vals = geng.engram_dequantize4(oc, os, block, tiled=True)
        assert torch.equal(vals.view(T, C, dim), geng.engram_lookup4(ids, Q, S, block))


def test_rows_of_16_values():
    """The narrowest rows: blocks of 16, two columns to a multiple of 32."""
    rng = np.random.default_rng(2)
    Q, S, codes, raw = _table(rng, 50, 48, 16)
    idx = torch.from_numpy(rng.integers(0, 50, (33, 2))).cuda()
    exp = torch.from_numpy(R.values4(codes, raw, 16)[idx.cpu().numpy()]).to(torch.float32).to(torch.bfloat16)
    assert torch.equal(geng.engram_lookup4(idx, Q, S, 16).cpu(), exp)
    oc, os = geng.engram_lookup4_operand(idx, Q, S, 16)
    assert torch.equal(geng.engram_dequantize4(oc, os, 16, tiled=True).view(33, 2, 48).cpu(), exp)


def test_empty_calls():
    Q, S = torch.zeros((4, 32), dtype=torch.uint8, device="cuda"), torch.zeros((4, 2), dtype=torch.uint8, device="cuda")
    assert geng.engram_lookup4(torch.empty((0, 3), dtype=torch.int64, device="cuda"), Q, S, 32).shape == (0, 3, 64)
    codes, scales = geng.engram_lookup4_operand(torch.empty((0, 3), dtype=torch.int64, device="cuda"), Q, S, 32)
    assert codes.shape == (0, 96) and scales.numel() == 0
    none = torch.empty((0, 32), dtype=torch.uint8, device="cuda")
    got = geng.engram_lookup4(torch.zeros((5, 3), dtype=torch.int64, device="cuda"), none, none[:, :2], 32)
    assert (got == 0).all()


def test_rows_beyond_32_bits():
    """A table of more than 2^32 bytes: rows at its far end."""
    rows, dim = 70_000_000, 128
    Q = torch.empty((rows, dim // 2), dtype=torch.uint8, device="cuda")
    S = torch.full((rows, dim // 16), 0x38, dtype=torch.uint8, device="cuda")  # E4M3 1.0
    Q[-3:] = torch.arange(3 * 64, device="cuda", dtype=torch.int64).view(3, 64).to(torch.uint8)
    S[-1] = 0x40  # 2.0
    idx = torch.tensor([[rows - 1, rows - 3], [rows, rows - 2]], device="cuda")
    got = geng.engram_lookup4(idx, Q, S, 16).cpu()
    v = torch.from_numpy(R.values4(R.unpack(Q[-3:].cpu().numpy()), S[-3:].cpu().numpy(), 16)).to(torch.bfloat16)
    assert torch.equal(got[0, 0], v[2]) and torch.equal(got[0, 1], v[0])
    assert (got[1, 0] == 0).all() and torch.equal(got[1, 1], v[1])
