"""The training operators' 64-bit formulas against differences, and the refusals of their entry points
that need no GPU."""
import ctypes

import numpy as np
import pytest
import torch

import gram_hash_embedding_gb300 as geng
from tests import train_ref as R


@pytest.fixture(scope="module")
def lib():
    geng.build()
    return geng._lib()


@pytest.mark.parametrize("T,hc,dim", [(3, 2, 16), (2, 4, 8), (4, 1, 24)])
def test_gate_gradient_against_differences(T, hc, dim):
    """Central differences in 64 bits: a step of 1e-5 leaves about 1e-10 of truncation and 1e-11 of rounding
    per value of order 1; 1e-6 covers both where |dot| is of order 0.1 and more."""
    rng = np.random.default_rng(dim)
    x = rng.standard_normal((T, hc, dim))
    kv = rng.standard_normal((T, hc + 1, dim))
    kv[:, :hc] += np.where(rng.random((T, hc, 1)) < 0.5, -1, 1) * x
    kv = kv.reshape(T, -1)
    q, k = rng.uniform(0.5, 1.5, (hc, dim)), rng.uniform(0.5, 1.5, (hc, dim))
    dout = rng.standard_normal((T, hc, dim))
    mask = np.arange(T) != 1
    grads = R.gate_grad(x, kv, q, k, dout, mask, 1e-20)
    assert np.abs(grads[5]).min() > 0.05
    ins = [x, kv, q, k]
    loss = lambda a: (R.gate(*a, mask, 1e-20) * dout).sum()
    for j in range(4):
        flat = ins[j].reshape(-1)
        for i in rng.choice(flat.size, min(40, flat.size), replace=False):
            hi, lo = [a.copy() for a in ins], [a.copy() for a in ins]
            hi[j].reshape(-1)[i] += 1e-5
            lo[j].reshape(-1)[i] -= 1e-5
            assert abs((loss(hi) - loss(lo)) / 2e-5 - grads[j].reshape(-1)[i]) < 1e-6, (j, i)


def test_embed_gradient_against_differences():
    """The lookup is linear in the table: a difference is the gradient up to rounding."""
    rng = np.random.default_rng(1)
    W = rng.standard_normal((7, 5))
    idx = np.array([[3, 3, -1], [0, 9, 3]])
    dout = rng.standard_normal((2, 3, 5))
    ids, g, _, times = R.embed_grad(idx, dout, 7, 0.5)
    assert ids.tolist() == [0, 3] and times.tolist() == [1, 3]
    full = np.zeros_like(W)
    full[ids] = g
    for r in range(7):
        for c in range(5):
            hi = W.copy()
            hi[r, c] += 1.0
            d = ((R.embed(idx, hi, 0.5, 7) - R.embed(idx, W, 0.5, 7)) * dout).sum()
            assert abs(d - full[r, c]) < 1e-12


def test_embed_refusals(lib):
    P = ctypes.c_void_p
    a = P(4096)  # never dereferenced: every call is refused (or has nothing to do) before a launch
    ok = dict(idx=a, istride=3, T=4, C=3, W=a, rows=10, dim=8, wstride=8, wt=geng.TYPE_BF16, scale=1.0, out=a,
              ot=geng.TYPE_F32)

    def call(**kw):
        v = {**ok, **kw}
        return lib.engram_embed(v["idx"], v["istride"], v["T"], v["C"], v["W"], v["rows"], v["dim"], v["wstride"],
                                v["wt"], v["scale"], v["out"], v["ot"], None)
    assert call(T=0) == geng.OK and call(T=0, idx=None, out=None) == geng.OK
    for bad in (dict(T=-1), dict(C=0), dict(rows=-1), dict(dim=0), dict(istride=2), dict(wstride=7), dict(wt=3),
                dict(ot=-1), dict(scale=float("nan")), dict(scale=float("inf")), dict(idx=None), dict(idx=P(4100)),
                dict(W=None), dict(W=P(4097)), dict(out=None), dict(out=P(4098))):
        assert call(**bad) == geng.ERR_INVALID, bad
    for bad in (dict(dim=65537, wstride=65537), dict(T=(1 << 31) // 3 + 1), dict(rows=(1 << 32) - 1)):
        assert call(**bad) == geng.ERR_UNSUPPORTED, bad


def test_embed_grad_refusals(lib):
    P = ctypes.c_void_p
    a = P(4096)
    need = lib.engram_embed_grad_workspace(12, 10, 8)
    assert need > 0 and need % 256 == 0
    assert lib.engram_embed_grad_workspace(0, 10, 8) == 0
    ok = dict(idx=a, istride=3, T=4, C=3, dout=a, dstride=24, dt=geng.TYPE_BF16, rows=10, dim=8, scale=1.0, gr=a,
              grad=a, gstride=8, gt=geng.TYPE_F32, count=a, ws=a, nbytes=need)

    def sparse(**kw):
        v = {**ok, **kw}
        return lib.engram_embed_grad(v["idx"], v["istride"], v["T"], v["C"], v["dout"], v["dstride"], v["dt"],
                                     v["rows"], v["dim"], v["scale"], v["gr"], v["grad"], v["gt"], v["count"], v["ws"],
                                     v["nbytes"], None)

    def dense(**kw):
        v = {**ok, **kw}
        return lib.engram_embed_grad_dense(v["idx"], v["istride"], v["T"], v["C"], v["dout"], v["dstride"], v["dt"],
                                           v["rows"], v["dim"], v["scale"], v["grad"], v["gstride"], v["gt"], 1,
                                           v["ws"], v["nbytes"], None)
    assert dense(T=0) == geng.OK and dense(rows=0) == geng.OK
    both = (dict(T=-1), dict(C=0), dict(rows=-1), dict(dim=0), dict(istride=2), dict(dstride=23), dict(dt=3), dict(gt=7),
            dict(scale=float("nan")), dict(idx=None), dict(idx=P(4100)), dict(dout=None), dict(dout=P(4097)),
            dict(grad=None), dict(grad=P(4098)), dict(ws=None), dict(ws=P(4096 + 128)), dict(nbytes=need - 1))
    for f, more in ((sparse, (dict(gr=None), dict(gr=P(4100)), dict(count=None), dict(count=P(4100)))),
                    (dense, (dict(gstride=7),))):
        for bad in both + more:
            assert f(**bad) == geng.ERR_INVALID, (f.__name__, bad)
        for bad in (dict(dim=65537, dstride=3 * 65537, gstride=65537), dict(T=(1 << 31) // 3 + 1),
                    dict(rows=(1 << 32) - 1)):
            assert f(**bad) == geng.ERR_UNSUPPORTED, (f.__name__, bad)


def test_gate_grad_refusals(lib):
    P = ctypes.c_void_p
    a = P(4096)
    need = lib.engram_gate_grad_workspace(5, 4, 64)
    assert need > 0 and need % 256 == 0
    for T, hc, dim in ((0, 4, 64), (5, 3, 64), (5, 4, 60), (5, 4, 16392), (1 << 31, 4, 64)):
        assert lib.engram_gate_grad_workspace(T, hc, dim) == 0
    names = ["x", "kv", "q", "k", "dout", "dx", "dkv", "dq", "dk", "ws"]
    ok = {n: a for n in names} | dict(T=5, hc=4, dim=64, nbytes=need)

    def call(**kw):
        v = {**ok, **kw}
        return lib.engram_gate_grad(v["x"], v["kv"], v["q"], v["k"], v["dout"], None, v["T"], v["hc"], v["dim"], 1e-20,
                                    v["dx"], v["dkv"], v["dq"], v["dk"], v["ws"], v["nbytes"], None)
    for n in names:
        assert call(**{n: None}) == geng.ERR_INVALID, n
        assert call(**{n: P(4096 + 8)}) == geng.ERR_INVALID, n
    assert call(T=-1) == geng.ERR_INVALID and call(nbytes=need - 1) == geng.ERR_INVALID
    for bad in (dict(hc=3), dict(dim=0), dict(dim=12), dict(dim=16392), dict(T=1 << 31)):
        assert call(**bad) == geng.ERR_UNSUPPORTED, bad


def test_norm_refusals(lib):
    P = ctypes.c_void_p
    a = P(4096)
    need = lib.engram_grad_norm_workspace(2)
    assert need > 0 and lib.engram_grad_norm_workspace(0) == 0

    def call(t=None, n=2, kind=geng.NORM_L2, norm=a, ws=a, nbytes=need, max_norm=1.0, clip=True):
        arr = (geng._Tensor * 2)(geng._Tensor(4096, None, None, 10, 0, geng.TYPE_F32, 0),
                                 geng._Tensor(4096, None, None, 10, 0, geng.TYPE_BF16, 0))
        if t:
            for k, v in t.items():
                setattr(arr[1], k, v)
        if clip:
            return lib.engram_grad_clip(arr, n, kind, max_norm, norm, ws, nbytes, None)
        return lib.engram_grad_norm(arr, n, kind, norm, ws, nbytes, None)
    for clip in (True, False):
        for bad in (dict(n=-1), dict(kind=1), dict(norm=None), dict(norm=P(4098)), dict(ws=None), dict(ws=P(4097)),
                    dict(nbytes=need - 1), dict(t=dict(n=-1)), dict(t=dict(type=3)), dict(t=dict(data=None)),
                    dict(t=dict(data=4097)), dict(t=dict(rows_used=4096, row_len=0)),
                    dict(t=dict(rows_used=4096, row_len=3)), dict(t=dict(rows_used=4100, row_len=5))):
            assert call(clip=clip, **bad) == geng.ERR_INVALID, bad
        assert call(clip=clip, t=dict(n=(1 << 36) + 1)) == geng.ERR_UNSUPPORTED
    for bad in (dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(max_norm=float("inf")),
                dict(t=dict(out=4097, out_type=geng.TYPE_F32)), dict(t=dict(out=8192, out_type=5)),
                dict(t=dict(out=4096, out_type=geng.TYPE_F32))):
        assert call(**bad) == geng.ERR_INVALID, bad
    assert lib.engram_grad_norm(None, 2, geng.NORM_L2, a, a, need, None) == geng.ERR_INVALID


def test_binding_refuses_before_any_pointer():
    idx = torch.zeros((4, 3), dtype=torch.int64)
    W = torch.zeros((5, 8))
    with pytest.raises(TypeError, match="CUDA tensor"):
        geng.engram_embed(idx, W)
    with pytest.raises(TypeError, match="CUDA tensor"):
        geng.engram_embed_grad(idx, torch.zeros((4, 3, 8)), 5)
    with pytest.raises(TypeError, match="CUDA tensor"):
        geng.engram_embed_grad_dense(idx, torch.zeros((4, 3, 8)), W)
    with pytest.raises(TypeError, match="CUDA tensor"):
        geng.engram_grad_norm([W])
    with pytest.raises(ValueError, match="norm_type"):
        geng.engram_grad_norm([W], norm_type=3)
    with pytest.raises(ValueError, match="one entry per gradient"):
        geng.engram_grad_clip([W], 1.0, out=[])
    x = torch.zeros((3, 4, 64), dtype=torch.bfloat16)
    w = torch.zeros((4, 64), dtype=torch.bfloat16)
    kv = torch.zeros((3, 5 * 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="dout has"):
        geng.engram_gate_grad(x, kv, w, w, x[:2])
    with pytest.raises(ValueError, match="kv has"):
        geng.engram_gate_grad(x, kv[:, 64:], w, w, x)
    with pytest.raises(ValueError, match="mask has"):
        geng.engram_gate_grad(x, kv, w, w, x, mask=torch.ones(4, dtype=torch.bool))


def test_workspaces_never_shrink(lib):
    """A workspace made for the largest call serves every smaller one: its size never falls as the ids, tokens
    or tensors grow, across every change of tiles, units and clusters."""
    rng = np.random.default_rng(0)
    edges = [1, 100, 1216, 2432, 4864, 8192, 9728, 19456, 32768, 38912, 77824, 155648, 311296, 622592, 1245184, 1867776]
    ns = sorted({max(1, n + d) for n in edges for d in (-1, 0, 1, 2)} | set(range(1, 700)) |
                {int(n) for n in np.exp(rng.uniform(0, np.log(2 ** 31 - 1), 4000))} | set(range(50, 200_000, 61)))
    for dim in (1, 3, 4, 7, 8, 12, 16, 20, 36, 64, 100, 128, 256, 260, 264, 512, 1000, 1024, 1027, 2048, 5120, 20_000, 65536):
        sizes = [lib.engram_embed_grad_workspace(n, 10 ** 6, dim) for n in ns]
        fall = [(a, b) for a, b, x, y in zip(ns, ns[1:], sizes, sizes[1:]) if y < x]
        assert not fall, f"dim {dim}: smaller for {fall[0][1]} ids than for {fall[0][0]}"
    Ts = list(range(1, 700)) + list(range(700, 40_000, 37))
    for hc in (1, 2, 4, 8):
        for dim in (8, 64, 168, 464, 512, 1024, 1032, 2048, 2056, 3616, 3800, 5120, 10248, 12000, 16384):
            sizes = [lib.engram_gate_grad_workspace(T, hc, dim) for T in Ts]
            fall = [(a, b) for a, b, x, y in zip(Ts, Ts[1:], sizes, sizes[1:]) if y < x]
            assert not fall, f"{hc} x {dim}: smaller for {fall[0][1]} tokens than for {fall[0][0]}"
    sizes = [lib.engram_grad_norm_workspace(n) for n in range(3000)]
    assert sizes == sorted(sizes)
