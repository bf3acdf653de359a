"""Trainable embedding rows (engram_embed) and their gradient (engram_embed_grad, _dense) against plain
64-bit sums (GPU only).

Tolerances. The lookup is one fp32 multiply and one rounding, so it is compared bit for bit with the
same two steps in torch on the CPU. A gradient row of m terms: an fp32 sum of m values in any order is
within (m - 1) 2^-24 sum|x| (to first order; 2 covers the rest) of the exact sum, the factor adds one
fp32 rounding, adding to what was there another, and the store rounds once to the stored type (2^-24,
2^-8 or 2^-11 of the value; fp16 values below 2^-14 are 2^-24 apart).
"""
import numpy as np
import pytest
import torch

import gram_hash_embedding_gb300 as geng
from tests import gpu_helpers as H
from tests import train_ref as R

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ROUND = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def _built():
    H.build_all()
    yield


def _vals(rng, shape, dtype):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(DT[dtype])


def _f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def _ids(rng, T, C, rows, kind):
    if kind == "uniform":
        ids = rng.integers(0, max(rows, 1), (T, C))
    elif kind == "one":      # every id the same row
        ids = np.full((T, C), rows // 2)
    elif kind == "none":     # nothing inside the table
        ids = rng.choice([-1, rows, rows + 5, -(2 ** 40), 2 ** 40], (T, C))
    elif kind == "heavy":    # half of the ids are one row, the rest spread
        ids = np.where(rng.random((T, C)) < 0.5, rows - 1, rng.integers(0, rows, (T, C)))
    elif kind == "runs":     # rows of 1, 2, 3, ... occurrences: runs end everywhere in a tile
        flat = np.repeat(np.arange(T * C), np.arange(1, T * C + 1) % 37 + 1)[:T * C] % rows
        ids = rng.permutation(flat).reshape(T, C)
    elif kind == "distinct":
        ids = rng.permutation(rows)[:T * C].reshape(T, C)
    if kind in ("uniform", "heavy"):
        ids = np.where(rng.random((T, C)) < 0.1, rng.choice([-1, rows, -(2 ** 62), 2 ** 62], (T, C)), ids)
    return ids.astype(np.int64)


# ------------------------------------------------------------------------------------------ lookup
@pytest.mark.parametrize("wt,ot", [(a, b) for a in DT for b in DT])
@pytest.mark.parametrize("T,C,dim,rows", [(1, 1, 8, 1), (7, 3, 100, 50), (65, 24, 128, 999), (33, 1, 5120, 40),
                                          (5, 2, 1, 9), (200, 2, 24, 77)])
def test_embed_bits(wt, ot, T, C, dim, rows):
    rng = np.random.default_rng(T * 1000 + dim)
    W = _vals(rng, (rows, dim), wt)
    idx = torch.from_numpy(_ids(rng, T, C, rows, "uniform"))
    ok = (idx >= 0) & (idx < rows)
    exp = torch.where(ok[..., None], W[idx.clamp(0, rows - 1) * ok].float() * np.float32(11.25), 0.0).to(DT[ot])
    got = geng.engram_embed(idx.cuda(), W.cuda(), scale=11.25, out_dtype=DT[ot])
    assert got.shape == (T, C, dim) and got.dtype == DT[ot]
    assert torch.equal(got.cpu(), exp)
    assert not torch.signbit(got.cpu()[~ok]).any()  # +0, not -0


def test_embed_views_and_special_values():
    """A hash output's layer slice as ids, a table whose rows are a stride apart, misaligned tables,
    infinities and NaN, which stay where they are; an id outside the table reads nothing."""
    rng = np.random.default_rng(3)
    T, C, dim, rows = 37, 6, 64, 55
    big = _vals(rng, (rows, 3 * dim + 1), "bf16").cuda()
    h = torch.from_numpy(rng.integers(0, rows, (T, 2, C))).cuda()
    for off in (0, dim, 1):  # 1: rows on odd addresses, moved value by value
        W = big[:, off:off + dim]
        exp = (W.float() * 0.5)[h[:, 1]].to(torch.bfloat16)
        assert torch.equal(geng.engram_embed(h[:, 1], W, scale=0.5), exp)
    W = big[:, :dim].contiguous()
    W[3] = float("nan")
    W[4] = float("inf")
    W[5] = -0.0
    idx = torch.tensor([[3, 4, 5, -1, rows, 2]], device="cuda")
    got = geng.engram_embed(idx, W, scale=-1.0)
    assert torch.isnan(got[0, 0]).all() and (got[0, 1] == -float("inf")).all()
    assert (got[0, 2] == 0).all() and not torch.signbit(got[0, 2]).any()
    assert (got[0, 3:5].view(torch.int16) == 0).all()
    assert torch.equal(got[0, 5], -W[2])
    # other shapes of ids; an empty call; an empty table
    assert geng.engram_embed(idx[0], W).shape == (6, dim)
    assert geng.engram_embed(idx[0, 0], W).shape == (dim,)
    assert geng.engram_embed(torch.empty((0, 4), dtype=torch.int64, device="cuda"), W).shape == (0, 4, dim)
    assert (geng.engram_embed(idx, W[:0]) == 0).all()


# ---------------------------------------------------------------------------------------- gradient
def _check_rows(idx, dout, rows, scale, got, gt, what):
    grad_rows, grad, count = got
    ids, exp, mag, times = R.embed_grad(idx, _f64(dout), rows, scale)
    n = idx.size
    assert int(count) == ids.size, f"{what}: {int(count)} distinct rows, expected {ids.size}"
    assert np.array_equal(grad_rows.cpu().numpy(), np.concatenate([ids, np.full(n - ids.size, -1)])), what
    _close(_f64(grad)[:ids.size], exp, mag, times, gt, what)


def _close(g, exp, mag, times, gt, what, old=0.0):
    u = 2.0 ** -24
    tol = (times[:, None] + 2) * u * mag + u * np.abs(old) + ROUND[gt] * (np.abs(exp) + np.abs(old)) + (2.0 ** -24 if gt == "f16" else 0.0) + 1e-40
    bad = np.abs(g - exp) > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off; first {np.argwhere(bad)[0]}: " \
                          f"{g[bad][0]} for {exp[bad][0]} +- {tol[bad][0]}"


SHAPES = [(1, 1, 128, 1, "uniform"), (3, 1, 8, 2 ** 32 - 2, "uniform"), (1777, 3, 100, 5003, "uniform"), (256, 24, 128, 384_006_168, "uniform"),
          (300, 24, 32, 1000, "heavy"), (5000, 1, 16, 70_000, "one"), (2049, 1, 264, 9000, "distinct"),
          (40_000, 1, 128, 200, "uniform"), (9000, 2, 128, 1 << 20, "runs"), (31, 1, 5120, 60, "heavy"),
          (70_000, 1, 64, 129_280, "heavy"), (64, 2, 128, 100, "none"), (4096, 1, 128, 4096, "distinct"),
          (4097, 1, 7, 300, "uniform"), (100_000, 2, 8, 100_000, "one"), (513, 1, 1, 20, "runs")]


@pytest.mark.parametrize("T,C,dim,rows,kind", SHAPES)
@pytest.mark.parametrize("dt,gt", [("bf16", "f32"), ("f32", "f32"), ("f16", "bf16"), ("f32", "f16")])
def test_embed_grad_rows(T, C, dim, rows, kind, dt, gt):
    rng = np.random.default_rng(T + dim)
    idx = _ids(rng, T, C, rows, kind)
    dout = _vals(rng, (T, C, dim), dt)
    grad = torch.full((T * C, dim), 7.0, device="cuda", dtype=DT[gt])
    got = geng.engram_embed_grad(torch.from_numpy(idx).cuda(), dout.cuda(), rows, scale=0.75, grad=grad)
    _check_rows(idx, dout, rows, 0.75, got, gt, f"{kind} {T}x{C}x{dim}")
    assert (got[1][int(got[2]):] == 7.0).all()  # rows past the count are not written
    # the same call again: the same bits
    again = geng.engram_embed_grad(torch.from_numpy(idx).cuda(), dout.cuda(), rows, scale=0.75, grad_dtype=DT[gt])
    k = int(got[2])
    assert torch.equal(again[1][:k].view(torch.int8), got[1][:k].view(torch.int8))


# tables of few rows (digits of few bits), and calls on both sides of 32,768 ids, up to which the sums number the
# segments, and of 622,592, where the sort's tiles grow
@pytest.mark.parametrize("T,C,dim,rows,kind", [(8193, 1, 520, 3000, "heavy"), (20_000, 1, 264, 3000, "one"), (10_000, 1, 1032, 500, "none"),
                                               (32_768, 1, 8, 9000, "runs"), (32_769, 1, 8, 9000, "uniform"), (348_000, 1, 8, 2520, "uniform"), (622_592, 1, 4, 50, "runs"), (622_593, 1, 4, 1342, "uniform"),
                                               (30_000, 24, 8, 1, "uniform"), (207_600, 3, 4, 2_700_000, "heavy")])
def test_embed_grad_rows_many_ids(T, C, dim, rows, kind):
    test_embed_grad_rows(T, C, dim, rows, kind, "bf16", "f32")


@pytest.mark.parametrize("T,C,dim,rows,kind", [s for s in SHAPES if s[3] <= 200_000])
@pytest.mark.parametrize("dt,gt,acc", [("bf16", "f32", False), ("f32", "bf16", False), ("bf16", "f32", True),
                                       ("f16", "f16", True)])
def test_embed_grad_dense(T, C, dim, rows, kind, dt, gt, acc):
    rng = np.random.default_rng(T + dim + 1)
    idx = _ids(rng, T, C, rows, kind)
    dout = _vals(rng, (T, C, dim), dt)
    old = _vals(rng, (rows, dim), gt) if acc else torch.full((rows, dim), float("nan"), dtype=DT[gt])
    grad = old.clone().cuda()
    got = geng.engram_embed_grad_dense(torch.from_numpy(idx).cuda(), dout.cuda(), grad, scale=-2.5, accumulate=acc)
    assert got.data_ptr() == grad.data_ptr()
    ids, exp, mag, times = R.embed_grad(idx, _f64(dout), rows, -2.5)
    o = _f64(old)[ids] if acc else 0.0
    _close(_f64(got)[ids], exp + o, mag, times, gt, f"dense {kind}", old=o)
    rest = np.ones(rows, bool)
    rest[ids] = False
    if acc:
        assert torch.equal(got.cpu()[torch.from_numpy(rest)], old[torch.from_numpy(rest)])
    else:
        assert (got.cpu()[torch.from_numpy(rest)].float().view(torch.int32) == 0).all()


def test_embed_grad_views():
    """ids as a hash output's layer slice, gradients whose tokens are a stride apart, a gradient table
    inside a wider one (the columns beside it stay), and misaligned buffers."""
    rng = np.random.default_rng(11)
    T, C, dim, rows = 130, 6, 64, 40
    h = torch.from_numpy(rng.integers(-2, rows + 2, (T, 2, C))).cuda()
    wide = _vals(rng, (T, C * dim + 24), "bf16").cuda()
    for off in (0, 8, 1):
        dout = wide[:, off:off + C * dim]
        got = geng.engram_embed_grad(h[:, 1], dout, rows)
        _check_rows(h[:, 1].cpu().numpy(), dout.cpu().contiguous(), rows, 1.0, got, "f32", f"offset {off}")
        got3 = geng.engram_embed_grad(h[:, 1], dout.unflatten(1, (C, dim)), rows)
        assert all(torch.equal(a[:int(got[2])], b[:int(got[2])]) for a, b in zip(got, got3))
        table = torch.full((rows, dim + 16), 3.0, device="cuda")
        geng.engram_embed_grad_dense(h[:, 1], dout, table[:, off:off + dim])
        ids, exp, mag, times = R.embed_grad(h[:, 1].cpu().numpy(), _f64(dout), rows, 1.0)
        _close(_f64(table[:, off:off + dim])[ids], exp, mag, times, "f32", "strided table")
        assert (table[:, :off] == 3.0).all() and (table[:, off + dim:] == 3.0).all()


def test_embed_grad_padding_and_special_values():
    """What padding ids point at may hold anything; infinities and NaN reach only their own rows."""
    T, dim, rows = 96, 128, 10
    idx = torch.arange(T, device="cuda") % 12 - 1  # -1 and 10 are outside
    dout = torch.ones((T, dim), device="cuda", dtype=torch.bfloat16)
    dout[(idx < 0) | (idx >= rows)] = float("nan")
    dout[idx == 3, 5] = float("inf")
    grad_rows, grad, count = geng.engram_embed_grad(idx, dout, rows)
    assert int(count) == rows and torch.equal(grad_rows[:rows], torch.arange(rows, device="cuda"))
    exp = torch.full((rows, dim), 8.0, device="cuda")
    exp[3, 5] = float("inf")
    assert torch.equal(grad[:rows], exp)
    dense = geng.engram_embed_grad_dense(idx, dout, torch.empty((rows, dim), device="cuda"))
    assert torch.equal(dense, exp)


def test_embed_grad_empty():
    none = torch.empty((0, 3), dtype=torch.int64, device="cuda")
    d = torch.empty((0, 3, 16), device="cuda")
    rows, grad, count = geng.engram_embed_grad(none, d, 9)
    assert rows.shape == (0,) and grad.shape == (0, 16) and int(count) == 0
    g = torch.full((9, 16), 5.0, device="cuda")
    geng.engram_embed_grad_dense(none, d, g, accumulate=True)
    assert (g == 5.0).all()
    geng.engram_embed_grad_dense(none, d, g)
    assert (g == 0.0).all()
    # a table of no rows
    rows, grad, count = geng.engram_embed_grad(torch.zeros(4, dtype=torch.int64, device="cuda"),
                                               torch.ones((4, 16), device="cuda"), 0)
    assert int(count) == 0 and (rows == -1).all()


def test_embed_grad_offsets_beyond_32_bits():
    """More than 2^31 values of dout, of the sparse gradient and of a dense table: only the last few ids
    lie inside the table, so little is read, at offsets past 32 bits."""
    dim = 512
    n = (1 << 31) // dim + 700
    idx = torch.full((n,), -1, device="cuda")
    idx[-3:] = torch.tensor([n - 1, 4, n - 1], device="cuda")
    dout = torch.empty((n, dim), device="cuda", dtype=torch.bfloat16)
    dout[-3:] = torch.tensor([1.0, 2.0, 4.0], device="cuda")[:, None]
    grad_rows, grad, count = geng.engram_embed_grad(idx, dout, n, grad_dtype=torch.bfloat16)
    assert int(count) == 2 and grad_rows[:3].tolist() == [4, n - 1, -1]
    assert (grad[0] == 2.0).all() and (grad[1] == 5.0).all()
    table = dout  # the same memory as a dense table after its values have been used
    d3 = torch.full((3, dim), 2.0, device="cuda")
    geng.engram_embed_grad_dense(torch.tensor([n - 1, 0, n - 1], device="cuda"), d3, table)
    assert (table[-1] == 4.0).all() and (table[0] == 2.0).all() and (table[-2] == 0).all() and (table[1:9] == 0).all()
    got = geng.engram_embed(torch.tensor([n - 1, 1], device="cuda"), table, out_dtype=torch.float32)
    assert (got[0] == 4.0).all() and (got[1] == 0).all()


def test_embed_grad_on_another_stream():
    rng = np.random.default_rng(2)
    T, C, dim, rows = 600, 4, 64, 77
    idx = _ids(rng, T, C, rows, "heavy")
    dout = _vals(rng, (T, C, dim), "bf16")
    s = torch.cuda.Stream()
    di, dd = torch.from_numpy(idx).cuda(), dout.cuda()
    got = geng.engram_embed_grad(di, dd, rows, stream=s)
    out = geng.engram_embed(di, dd[:50, 0], stream=s)
    torch.cuda.current_stream().wait_stream(s)
    _check_rows(idx, dout, rows, 1.0, got, "f32", "side stream")
    assert torch.equal(out[1, 0], dd[:50, 0][idx[1, 0]] if 0 <= idx[1, 0] < 50 else torch.zeros_like(out[1, 0]))


def test_embed_grad_in_a_graph():
    """Captured once, replayed on new ids and gradients in the same buffers."""
    rng = np.random.default_rng(4)
    T, C, dim, rows = 500, 2, 128, 300
    di, dd = torch.zeros((T, C), dtype=torch.int64, device="cuda"), torch.zeros((T, C, dim), device="cuda")
    out = [torch.empty(T * C, dtype=torch.int64, device="cuda"), torch.empty((T * C, dim), device="cuda"),
           torch.empty(1, dtype=torch.int64, device="cuda")]
    ws = torch.empty(geng.engram_embed_grad_workspace(T * C, rows, dim), dtype=torch.uint8, device="cuda")
    call = lambda: geng.engram_embed_grad(di, dd, rows, grad_rows=out[0], grad=out[1], count=out[2], workspace=ws)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for kind in ("heavy", "uniform", "none"):
        idx, dout = _ids(rng, T, C, rows, kind), _vals(rng, (T, C, dim), "f32")
        di.copy_(torch.from_numpy(idx))
        dd.copy_(dout)
        g.replay()
        torch.cuda.synchronize()
        _check_rows(idx, dout, rows, 1.0, out, "f32", kind)


@pytest.mark.parametrize("n,dim,kind", [(40_000, 128, "heavy"), (40_000, 64, "one"), (9000, 264, "runs"), (700, 128, "heavy"),
                                        (12_000, 100, "heavy"), (700_000, 16, "one"), (3000, 2048, "one")])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_embed_grad_bits_do_not_depend_on_addresses(n, dim, kind, dt):
    """The same ids and gradients in aligned buffers, in views that allow only 4 or 1 values an access and in
    rows a stride apart: the same bits, in both forms, which agree with each other too."""
    rng = np.random.default_rng(n + dim)
    rows = 3000
    idx = torch.from_numpy(_ids(rng, n, 1, rows, kind)).cuda()
    dout = _vals(rng, (n, dim), dt).cuda()
    first = None
    for off, gap in ((0, 0), (4, 0), (1, 0), (0, 1), (8, 24)):
        d = torch.empty(n * (dim + gap) + 8, device="cuda", dtype=DT[dt])[off:off + n * (dim + gap)].view(n, dim + gap)[:, :dim]
        d.copy_(dout)
        grad = torch.empty(n * dim + 8, device="cuda")[off:off + n * dim].view(n, dim)
        grad_rows, grad, count = geng.engram_embed_grad(idx, d, rows, grad=grad)
        k = int(count)
        got = grad[:k].clone()
        table = torch.empty(rows * (dim + gap) + 8, device="cuda")[off:off + rows * (dim + gap)].view(rows, dim + gap)[:, :dim]
        geng.engram_embed_grad_dense(idx, d, table)
        assert torch.equal(table[grad_rows[:k]].view(torch.int32), got.view(torch.int32)), (off, gap)
        if first is None:
            first = got
            assert torch.isfinite(first).all() and k > 0
        assert torch.equal(got.view(torch.int32), first.view(torch.int32)), (off, gap)


def test_embed_grad_empty_flat():
    """An empty batch whose gradients are laid out [T, C * dim]."""
    none = torch.empty((0, 3), dtype=torch.int64, device="cuda")
    rows, grad, count = geng.engram_embed_grad(none, torch.empty((0, 48), device="cuda"), 9)
    assert rows.shape == (0,) and grad.shape == (0, 16) and int(count) == 0
    g = torch.full((9, 16), 5.0, device="cuda")
    geng.engram_embed_grad_dense(none, torch.empty((0, 48), device="cuda"), g, accumulate=True)
    assert (g == 5.0).all()
    geng.engram_embed_grad_dense(none, torch.empty((0, 48), device="cuda"), g)
    assert (g == 0.0).all()


# ------------------------------------------------------------- rows that are never written, NaN sums
# The comparison above (_close) takes a NaN for a hit. These cases compare so that a NaN misses.
def _close_strict(g, exp, mag, times, gt, what, old=0.0):
    u = 2.0 ** -24
    tol = (times[:, None] + 2) * u * mag + u * np.abs(old) + ROUND[gt] * (np.abs(exp) + np.abs(old)) + (2.0 ** -24 if gt == "f16" else 0.0) + 1e-40
    bad = ~(np.abs(g - exp) <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off; first {np.argwhere(bad)[0]}: {g[bad][0]} for {exp[bad][0]}"


STRICT = SHAPES + [(8193, 1, 520, 3000, "heavy"), (20_000, 1, 264, 3000, "one"), (32_768, 1, 8, 9000, "runs"), (32_769, 1, 8, 9000, "uniform"),
                   (622_593, 1, 4, 1342, "uniform"), (30_000, 24, 8, 1, "uniform"), (207_600, 3, 4, 2_700_000, "heavy")]


@pytest.mark.parametrize("T,C,dim,rows,kind", STRICT)
@pytest.mark.parametrize("dt,gt", [("bf16", "f32"), ("f32", "bf16"), ("f16", "f16")])
def test_embed_grad_writes_every_row(T, C, dim, rows, kind, dt, gt):
    """Both forms into buffers of NaN, and the dense form added to what a buffer holds."""
    rng = np.random.default_rng(T + dim + 2)
    idx = _ids(rng, T, C, rows, kind)
    dout = _vals(rng, (T, C, dim), dt)
    ids, exp, mag, times = R.embed_grad(idx, _f64(dout), rows, 0.75)
    di, dd = torch.from_numpy(idx).cuda(), dout.cuda()
    grad = torch.full((T * C, dim), float("nan"), device="cuda", dtype=DT[gt])
    grad_rows, grad, count = geng.engram_embed_grad(di, dd, rows, scale=0.75, grad=grad)
    k = int(count)
    assert k == ids.size and np.array_equal(grad_rows.cpu().numpy()[:k], ids)
    _close_strict(_f64(grad[:k]), exp, mag, times, gt, "sparse")
    assert torch.isnan(grad[k:]).all()
    if rows > 3_000_000:  # a dense table of those would be large
        return
    table = geng.engram_embed_grad_dense(di, dd, torch.full((rows, dim), float("nan"), device="cuda", dtype=DT[gt]), scale=0.75)
    _close_strict(_f64(table)[ids], exp, mag, times, gt, "dense")
    rest = np.ones(rows, bool)
    rest[ids] = False
    assert (table.cpu()[torch.from_numpy(rest)].float().view(torch.int32) == 0).all()
    old = _vals(rng, (rows, dim), gt)
    table = geng.engram_embed_grad_dense(di, dd, old.cuda(), scale=0.75, accumulate=True)
    o = _f64(old)[ids]
    _close_strict(_f64(table)[ids], exp + o, mag, times, gt, "added", old=o)
    assert torch.equal(table.cpu()[torch.from_numpy(rest)], old[torch.from_numpy(rest)])


def test_strict_comparison_sees_a_row_that_is_never_written():
    exp, times = np.ones((3, 4)), np.ones(3)
    _close_strict(exp.copy(), exp, exp, times, "f32", "")
    g = exp.copy()
    g[1] = np.nan
    with pytest.raises(AssertionError):
        _close_strict(g, exp, exp, times, "f32", "")
