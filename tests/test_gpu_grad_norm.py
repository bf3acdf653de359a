"""The global gradient norm and clipping (engram_grad_norm, engram_grad_clip) against 64-bit sums (GPU
only).

Tolerances. A thread adds at most 256 squares in fp32 before the sum is joined in 64 bits, and every
square and addition rounds once (2^-24), so the sum of squares is within 257 * 2^-24 of itself; the root
halves that and the result rounds once: 2^-16 relative covers it. A maximum is exact. Given the norm
that the call returned, a clipped value is one fp32 division, one fp32 product and one rounding to the
stored type, so it is compared bit for bit with the same steps on the CPU.
"""
import numpy as np
import pytest
import torch

import gram_hash_embedding_gb300 as geng
from tests import gpu_helpers as H

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    H.build_all()
    yield


def _grads(rng, sizes, kinds, scale=1.0):
    return [torch.from_numpy((rng.standard_normal(n) * scale).astype(np.float32)).to(DT[k])
            for n, k in zip(sizes, kinds)]


def _norm64(ts, kind=2):
    if kind == 2:
        return float(np.sqrt(sum((t.double() ** 2).sum().item() for t in ts)))
    return max([t.double().abs().max().item() for t in ts if t.numel()] + [0.0])


def _clipped(t, norm, max_norm, dtype=None):
    coef = np.float32(max_norm) / (np.float32(norm) + np.float32(1e-6))
    coef = np.float32(1.0) if coef > 1 else coef
    return (t.float() * torch.tensor(coef)).to(dtype or t.dtype)


CASES = [([1], ["f32"]), ([0, 5, 0], ["bf16", "f32", "f16"]), ([16384], ["bf16"]), ([16385, 1, 7], ["f16", "bf16", "f32"]),
         ([100_003] * 5, ["bf16", "f32", "f16", "bf16", "f32"]), (list(range(0, 700)), ["bf16", "f32", "f16"] * 233 + ["f32"]),
         ([3_000_001, 50], ["f32", "bf16"]), ([9] * 1300, ["f32"] * 1300), ([40_000_003], ["bf16"])]


@pytest.mark.parametrize("sizes,kinds", CASES, ids=[str(len(c[0])) + "x" + str(max(c[0])) for c in CASES])
def test_norm_and_clip(sizes, kinds):
    rng = np.random.default_rng(len(sizes))
    host = _grads(rng, sizes, kinds, 0.1)
    for kind in (2.0, float("inf")):
        dev = [t.cuda() for t in host]
        norm = geng.engram_grad_norm(dev, norm_type=kind)
        exp = _norm64(host, kind)
        assert norm.shape == () and abs(float(norm) - exp) <= (2.0 ** -16 * exp if kind == 2 else 0.0)
        again = geng.engram_grad_norm(dev, norm_type=kind)
        assert torch.equal(norm, again)
        for max_norm in (0.25 * exp, 4 * exp, 0.0):
            work = [t.clone() for t in dev]
            got = geng.engram_grad_clip(work, max_norm, norm_type=kind)
            assert abs(float(got) - exp) <= (2.0 ** -16 * exp if kind == 2 else 0.0)
            for w, t in zip(work, host):
                assert torch.equal(w.cpu(), _clipped(t, float(got), max_norm))
        outs = [torch.full(t.shape, 9.0, dtype=DT["f32" if i % 2 else "bf16"], device="cuda") for i, t in enumerate(host)]
        got = geng.engram_grad_clip(dev, 0.5 * exp, norm_type=kind, out=outs)
        for o, t, d in zip(outs, host, dev):
            assert torch.equal(o.cpu(), _clipped(t, float(got), 0.5 * exp, o.dtype))
            assert torch.equal(d.cpu(), t)  # the source stays


def test_misaligned_tensors_and_mixed_destinations():
    """Views at odd addresses, sources and destinations aligned differently, and some in place."""
    rng = np.random.default_rng(1)
    base = {k: torch.from_numpy(rng.standard_normal(200_000).astype(np.float32)).to(DT[k]).cuda() for k in DT}
    src = [base["bf16"][1:70_002], base["f32"][3:50_000], base["f16"][100_005:100_017], base["f16"][7:99_999], base["bf16"][80_000:80_003]]
    keep = [t.cpu().clone() for t in src]
    flat = torch.full((400_000,), 5.0, device="cuda")
    outs, at = [], 1
    for i, t in enumerate(src):
        outs.append(None if i == 3 else flat[at:at + t.numel()])
        at += t.numel() + 1
    norm = geng.engram_grad_clip(src, 1.0, out=outs)
    exp = _norm64(keep)
    assert abs(float(norm) - exp) <= 2.0 ** -16 * exp
    at = 1
    for i, t in enumerate(keep):
        got = src[i] if i == 3 else flat[at:at + t.numel()]
        assert torch.equal(got.cpu(), _clipped(t, float(norm), 1.0, got.dtype)), i
        if i != 3:
            assert torch.equal(src[i].cpu(), t) and flat[at - 1] == 5.0 and flat[at + t.numel()] == 5.0
        at += t.numel() + 1


@pytest.mark.parametrize("dim", [1, 100, 128])
def test_counts(dim):
    """Only the leading rows that a device-side count names are read and written; what is behind them may be
    anything; counts of 0, of all rows, beyond all rows and below 0."""
    rng = np.random.default_rng(dim)
    n = 3001
    for used in (0, 1, 1777, n, n + 50, -3):
        k = max(0, min(used, n))
        g = torch.from_numpy(rng.standard_normal((n, dim)).astype(np.float32))
        g[k:] = float("nan")
        other = torch.from_numpy(rng.standard_normal(777).astype(np.float32))
        dev = [other.cuda(), g.cuda()]
        counts = [None, torch.tensor([used], device="cuda")]
        norm = geng.engram_grad_norm(dev, counts=counts)
        exp = _norm64([other, g[:k]])
        assert abs(float(norm) - exp) <= 2.0 ** -16 * exp
        got = geng.engram_grad_clip(dev, 0.5, counts=counts)
        assert torch.equal(dev[1][:k].cpu(), _clipped(g[:k], float(got), 0.5)) and torch.isnan(dev[1][k:]).all()
        assert torch.equal(dev[0].cpu(), _clipped(other, float(got), 0.5))


def test_special_values():
    """NaN anywhere: the norm and every clipped value are NaN. An infinity: factor 0, itself NaN. Values
    whose squares underflow or overflow fp32."""
    for kind in (2.0, float("inf")):
        g = [torch.ones(100_000, device="cuda"), torch.ones(37, device="cuda", dtype=torch.bfloat16)]
        g[1][36] = float("nan")
        assert torch.isnan(geng.engram_grad_clip(g, 1.0, norm_type=kind))
        assert torch.isnan(g[0]).all() and torch.isnan(g[1]).all()
        g = [torch.ones(100_000, device="cuda"), torch.ones(37, device="cuda", dtype=torch.bfloat16)]
        g[0][5] = -float("inf")
        assert float(geng.engram_grad_clip(g, 1.0, norm_type=kind)) == float("inf")
        assert torch.isnan(g[0][5]) and (g[0][6:] == 0).all() and (g[1] == 0).all()
    big = torch.full((10,), 1e30, device="cuda")
    assert float(geng.engram_grad_norm([big])) == float("inf")
    assert float(geng.engram_grad_norm([big], norm_type=float("inf"))) == np.float32(1e30)
    zero = torch.zeros(5000, device="cuda")
    assert float(geng.engram_grad_clip([zero], 1.0)) == 0.0 and (zero == 0).all()


def test_no_tensors_streams_and_graphs():
    assert float(geng.engram_grad_norm([])) == 0.0
    assert float(geng.engram_grad_clip([], 1.0)) == 0.0
    rng = np.random.default_rng(3)
    host = _grads(rng, [70_001, 33, 500_000], ["bf16", "f32", "f32"])
    dev = [t.cuda() for t in host]
    s = torch.cuda.Stream()
    outs = [torch.empty(t.shape, device="cuda") for t in host]
    norm = geng.engram_grad_clip(dev, 1.0, out=outs, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for o, t in zip(outs, host):
        assert torch.equal(o.cpu(), _clipped(t, float(norm), 1.0, o.dtype))
    ws = torch.empty(geng.engram_grad_norm_workspace(3), dtype=torch.uint8, device="cuda")
    norm = torch.zeros((), device="cuda")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        geng.engram_grad_clip(dev, 2.0, out=outs, norm=norm, workspace=ws)
    for scale in (1.0, 3.0):
        for d, t in zip(dev, host):
            d.copy_(t.float() * scale)
        g.replay()
        torch.cuda.synchronize()
        exp = _norm64([d.cpu() for d in dev])
        assert abs(float(norm) - exp) <= 2.0 ** -16 * exp
        for o, d in zip(outs, dev):
            assert torch.equal(o.cpu(), _clipped(d.cpu(), float(norm), 2.0, o.dtype))


def test_prepared_call():
    """Marshalled once, called on refilled buffers and inside a graph: the same bits as the plain calls."""
    rng = np.random.default_rng(7)
    sizes = [5000, 1, 70_001, 33] * 15
    dev = [t.cuda() for t in _grads(rng, sizes, ["bf16", "f32", "f16", "f32"] * 15)]
    dev.append(torch.from_numpy(rng.standard_normal((400, 16)).astype(np.float32)).cuda())
    counts = [None] * len(sizes) + [torch.tensor([123], device="cuda")]
    outs = [torch.zeros(t.shape, device="cuda") for t in dev]
    exp = [torch.zeros(t.shape, device="cuda") for t in dev]
    clip = geng.PreparedGradClip(dev, 1.0, out=outs, counts=counts)
    norm = geng.PreparedGradClip(dev, norm_type=float("inf"), counts=counts)
    clip()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        clip()
    for scale, call in ((1.0, clip), (0.25, clip), (4.0, g.replay)):
        for t in dev:
            t.mul_(scale)
        call()
        want = geng.engram_grad_clip(dev, 1.0, out=exp, counts=counts)
        assert torch.equal(clip.norm, want) and all(torch.equal(a, b) for a, b in zip(outs, exp))
        assert torch.equal(norm(), geng.engram_grad_norm(dev, float("inf"), counts))
    with pytest.raises(ValueError, match="norm_type"):
        geng.PreparedGradClip(dev, 1.0, norm_type=1)
    with pytest.raises(geng.EngramError):
        geng.PreparedGradClip(dev, -1.0)()


def test_more_than_32_bits_of_values():
    n = (1 << 31) + 70_001
    t = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    t[-1], t[5], t[(1 << 31) + 3] = 2.0, 3.0, 6.0
    assert float(geng.engram_grad_norm([t])) == 7.0
    assert float(geng.engram_grad_norm([t], norm_type=float("inf"))) == 6.0
    geng.engram_grad_clip([t], 3.5)
    assert (t[-1], t[5], t[(1 << 31) + 3]) == (1.0, 1.5, 3.0) and int(t.count_nonzero()) == 3


def test_prepared_call_on_another_stream():
    """Built behind work of its stream that still writes into the memory it gets, called on another stream at
    once; and dropped while its call is still waiting there: its memory is not handed out before."""
    rng = np.random.default_rng(17)
    host = _grads(rng, [70_001, 33, 500_000], ["bf16", "f32", "f32"])
    for given in (False, True):
        dev = [t.cuda() for t in host]
        outs = [torch.empty(t.shape, device="cuda") for t in host]
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        before = [torch.empty((), device="cuda"), torch.empty(geng.engram_grad_norm_workspace(3), dtype=torch.uint8, device="cuda")]
        torch.cuda._sleep(100_000_000)
        for t in before:
            t.fill_(77)
        del before, t
        clip = geng.PreparedGradClip(dev, 1.0, out=outs, stream=side if given else None)
        with torch.cuda.stream(side):
            norm = clip()
        torch.cuda.synchronize()
        exp = _norm64(host)
        assert abs(float(norm) - exp) <= 2.0 ** -16 * exp
        for o, t in zip(outs, host):
            assert torch.equal(o.cpu(), _clipped(t, float(norm), 1.0, o.dtype))
        at = clip.norm.data_ptr()
        with torch.cuda.stream(side):
            torch.cuda._sleep(100_000_000)
            clip()
        del clip, norm
        other = [torch.empty((), device="cuda") for _ in range(64)]
        assert all(t.data_ptr() != at for t in other)
        torch.cuda.synchronize()


def test_empty_batch_through_the_chain():
    """An empty batch's sparse gradient with its count, clipped beside another tensor."""
    none = torch.empty((0, 3), dtype=torch.int64, device="cuda")
    _, grad, count = geng.engram_embed_grad(none, torch.empty((0, 3, 16), device="cuda"), 9)
    other = torch.full((100,), 2.0, device="cuda")
    exp = _clipped(other.cpu(), 20.0, 1.0)
    assert float(geng.engram_grad_norm([grad, other], counts=[count, None])) == 20.0
    assert float(geng.engram_grad_clip([grad, other], 1.0, counts=[count, None])) == 20.0
    assert torch.equal(other.cpu(), exp)
    assert float(geng.engram_grad_norm([grad], counts=[count])) == 0.0
