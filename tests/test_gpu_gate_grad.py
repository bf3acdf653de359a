"""The gate's gradient (engram_gate_grad) against its formula in 64 bits (GPU only); the formula itself
is checked against differences in test_train_formulas.py.

Tolerances, from the arithmetic (u = 2^-24). An fp32 sum of dim terms in any order is within dim * u of
the sum of its terms' magnitudes, so with s = (dim + 8) u: the mean squares are within s of themselves,
sum(h w key) within s sum|h w key| and sum(dout value) within s sum|dout value|. Hence
  ddot_err = psi(dot) s sum|dout v| + |ddot| (dot_err (1 / (2m) + 1 / (2 sqrt m)) + 16 u),
  dot_err  = r s sum|h w key| + |dot| (s + 4 u)
where psi = gate (1 - gate) / (2 sqrt m), whose logarithm changes by at most 1/(2m) + 1/(2 sqrt m) per
unit of dot. A result's error follows term by term; bf16 results add one rounding (2^-8). First-order
bounds, so everything in fp32 is taken twice. Inputs keep |dot| away from the 1e-6 clamp by more than
dot_err (checked), except where dot is exactly 0.
"""
import numpy as np
import pytest
import torch

import gram_hash_embedding_gb300 as geng
from tests import gpu_helpers as H
from tests import train_ref as R

pytestmark = pytest.mark.gpu
EPS = 1e-20


@pytest.fixture(scope="module", autouse=True)
def _built():
    H.build_all()
    yield


def _bf(a):
    return torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16)


def _f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def _inputs(rng, T, hc, dim, masked=0.2):
    x = rng.standard_normal((T, hc, dim))
    kv = rng.standard_normal((T, hc + 1, dim))
    sign = np.where(rng.random((T, hc, 1)) < 0.3, -1.0, 1.0)
    # mostly aligned or opposed keys: |dot| = O(1), well away from the clamp
    kv[:, :hc] = 0.5 * kv[:, :hc] + sign * (0.3 + 1.5 * dim ** -0.5) * x
    q, k = rng.uniform(0.5, 1.5, (hc, dim)), rng.uniform(0.5, 1.5, (hc, dim))
    dout = rng.standard_normal((T, hc, dim))
    mask = rng.random(T) >= masked
    return [_bf(a) for a in (x, kv.reshape(T, -1), q, k, dout)] + [torch.from_numpy(mask)]


def _check(args, got, what, small=False):
    x, kv, q, k, dout = (_f64(a) for a in args[:5])
    mask = args[5].cpu().numpy()
    T, hc, dim = x.shape
    u, s = 2.0 ** -24, (dim + 8) * 2.0 ** -24
    dx, dkv, dq, dk, ddot, dot = R.gate_grad(x, kv, q, k, dout, mask, EPS)
    kv3 = kv.reshape(T, hc + 1, dim)
    key, v = kv3[:, :hc], kv3[:, hc:]
    A, B = (x * x).mean(-1, keepdims=True) + EPS, (key * key).mean(-1, keepdims=True) + EPS
    r, w, m = 1 / np.sqrt(A * B * dim), q * k, np.abs(dot)
    dot_err = r * s * np.abs(x * w * key).sum(-1, keepdims=True) + m * (s + 4 * u)
    if small:  # the sum in twice the precision: what is left is the mean squares' error and single roundings
        dot_err = m * (2 * s + 16 * u)
    clear = (np.abs(m - 1e-6) > 2 * dot_err) & ((m > 4 * dot_err) | (m == 0)) | ~mask[:, None, None]
    assert clear.all(), f"{what}: the test's own inputs are too near the clamp"
    root = np.sqrt(np.maximum(m, 1e-6))
    g = 1 / (1 + np.exp(-np.copysign(root, dot)))
    psi = np.where(m >= 1e-6, g * (1 - g) * 0.5 / root, 0.0)
    ddot_err = psi * s * np.abs(dout * v).sum(-1, keepdims=True) + \
        np.abs(ddot) * (dot_err * (0.5 / np.maximum(m, 1e-6) + 0.5 / root) + 16 * u)
    on = mask[:, None, None]

    def bound(a, b, A_):  # of ddot * (r w a - dot / (A dim) b)
        part = np.abs(r * w * a) + m / (A_ * dim) * np.abs(b)
        return 2 * on * (ddot_err * part + np.abs(ddot) * ((2 * s + 8 * u) * part + dot_err / (A_ * dim) * np.abs(b)))

    def close(t, exp, tol, name):
        t = _f64(t)
        bad = ~(np.abs(t - exp) <= tol)
        assert not bad.any(), f"{what}: {name}: {int(bad.sum())} of {bad.size} off; first {np.argwhere(bad)[0]}: " \
                              f"{t[bad][0]} for {exp[bad][0]} +- {np.broadcast_to(tol, exp.shape)[bad][0]}"

    f32 = bound(key, x, A)
    close(got[0], dx, f32 + 2 * u * np.abs(dout) + 2.0 ** -8 * (np.abs(dx) + f32) + 1e-40, "dx")
    gate_err = np.where(on, g * (1 - g) * dot_err * 0.5 / root + 4 * u, 0.0)
    fk = bound(x, key, B)
    fv = 2 * (gate_err * np.abs(dout)).sum(1, keepdims=True) + 2 * hc * u * np.abs(np.where(on, g * dout, 0)).sum(1, keepdims=True)
    fk = np.concatenate([fk, fv], 1).reshape(T, -1)
    close(got[1], dkv, fk + 2.0 ** -8 * (np.abs(dkv) + fk) + 1e-40, "dkv")
    term = 2 * (ddot_err * r + np.abs(ddot) * r * (s + (T + 16) * u)) * on * np.abs(x * key)
    tw = term.sum(0)
    close(got[2], dq, tw * np.abs(k) + 1e-40, "dq_weight")
    close(got[3], dk, tw * np.abs(q) + 1e-40, "dk_weight")
    off = ~args[5]
    assert torch.equal(got[0].cpu()[off].view(torch.int16), args[4][off].view(torch.int16)), what
    assert (got[1].cpu()[off].view(torch.int16) == 0).all(), what


def _run(args, **kw):
    return geng.engram_gate_grad(*[a.cuda() for a in args[:5]], mask=args[5].cuda(), **kw)


@pytest.mark.parametrize("T,hc,dim", [(1, 1, 8), (1, 4, 5120), (2, 8, 16384), (3, 2, 1032), (37, 4, 256), (200, 2, 264),
                                      (333, 1, 2056), (65, 8, 640), (500, 4, 1024), (1500, 1, 64), (9, 4, 16384),
                                      (700, 8, 96), (311, 4, 5120), (19, 1, 16376), (5, 2, 10248)])
def test_gate_grad(T, hc, dim):
    args = _inputs(np.random.default_rng(T * 7 + dim), T, hc, dim)
    got = _run(args)
    _check(args, got, f"T={T} hc={hc} dim={dim}")
    again = _run(args)
    assert all(torch.equal(a, b) for a, b in zip(got, again))  # the same bits


def test_gate_grad_masks():
    """Every token masked; none; no mask given; and masked tokens that hold infinities and NaN."""
    rng = np.random.default_rng(5)
    T, hc, dim = 70, 4, 512
    args = _inputs(rng, T, hc, dim)
    args[5][:] = False
    got = _run(args)
    _check(args, got, "all masked")
    assert (got[2] == 0).all() and (got[3] == 0).all()
    args[5][:] = True
    _check(args, _run(args), "none masked")
    free = geng.engram_gate_grad(*[a.cuda() for a in args[:5]])
    assert all(torch.equal(a, b) for a, b in zip(free, _run(args)))
    clean = [a.clone() for a in args]
    for a in (args, clean):
        a[5][::3] = False
    bad = ~args[5]
    args[0][bad] = float("nan")
    args[1][bad] = float("inf")
    args[4][bad, 0] = float("inf")
    args[4][bad, 1] = float("nan")
    got, exp = _run(args), _run(clean)
    assert torch.equal(got[0].cpu()[bad].view(torch.int16), args[4][bad].view(torch.int16))
    assert (got[1].cpu()[bad].view(torch.int16) == 0).all()
    for a, b in zip(got[:2], exp[:2]):
        assert torch.equal(a.cpu()[~bad], b.cpu()[~bad])
    assert torch.equal(got[2], exp[2]) and torch.equal(got[3], exp[3])


@pytest.mark.parametrize("T,hc,dim", [(600, 1, 64), (300, 4, 1024), (200, 2, 5120), (64, 8, 640), (90, 4, 5120)])
def test_gate_grad_small_dots(T, hc, dim):
    """Keys almost orthogonal to h: sum(h w key) cancels and 1 / sqrt(dot) magnifies what an fp32 sum of it
    would be off by. The kernel forms such sums in twice the precision, so dot is held to the error of the
    mean squares alone. Tokens with a copy of |dot| outside [1e-5, 0.03] are masked out."""
    rng = np.random.default_rng(T + dim)
    args = _inputs(rng, T, hc, dim, masked=0.0)
    x, q, k = _f64(args[0]), _f64(args[2]), _f64(args[3])
    kv = rng.standard_normal((T, hc + 1, dim))
    key = kv[:, :hc]
    key -= (x * q * k * key).sum(-1, keepdims=True) / (x * x * q * k * q * k).sum(-1, keepdims=True) * (x * q * k)
    kv[:, :hc] = key + rng.uniform(-1, 1, (T, hc, 1)) * 0.002 * dim ** -0.5 * x
    args[1] = _bf(kv.reshape(T, -1))
    dot = np.abs(R.gate_grad(x, _f64(args[1]), q, k, _f64(args[4]), np.ones(T, bool), EPS)[5][..., 0])
    args[5] = torch.from_numpy(((dot > 1e-5) & (dot < 0.03)).all(1))
    assert args[5].float().mean() > 0.5
    got = _run(args)
    _check(args, got, "small dots", small=True)
    assert all(torch.equal(a, b) for a, b in zip(got, _run(args)))


def test_gate_grad_clamped_and_zero_rows():
    """A key orthogonal to h (dot exactly 0) and an all-zero key, h or value: the gate's slope is 0 at the
    clamp, so dx = dout and the key's gradient is 0; nothing turns into NaN."""
    T, hc, dim = 6, 2, 64
    rng = np.random.default_rng(8)
    args = _inputs(rng, T, hc, dim, masked=0.0)
    kv = args[1].view(T, hc + 1, dim)
    args[2][:] = 1.0
    args[3][:] = 1.0
    args[0][0, 0, :] = 1.0
    kv[0, 0, :] = torch.tensor([1.0, -1.0] * (dim // 2))  # sum(h key) = 0 exactly
    kv[1, :hc] = 0.0
    args[0][2] = 0.0
    kv[3, hc] = 0.0
    got = _run(args)
    _check([a[3:] if a.shape[0] == T else a for a in args], [got[0][3:], got[1][3:], *_run([a[3:] if a.shape[0] == T else a for a in args])[2:]], "rest")
    dx, dkv = got[0].cpu(), got[1].cpu().view(T, hc + 1, dim)
    assert torch.equal(dx[0, 0], args[4][0, 0]) and (dkv[0, 0] == 0).all()
    assert torch.equal(dx[1], args[4][1]) and (dkv[1, :hc] == 0).all()
    assert torch.equal(dx[2], args[4][2]) and (dkv[2, :hc] == 0).all()
    assert all(torch.isfinite(t).all() for t in got)


def test_gate_grad_in_place_streams_and_empty():
    rng = np.random.default_rng(6)
    T, hc, dim = 90, 4, 1024
    args = _inputs(rng, T, hc, dim)
    exp = _run(args)
    dev = [a.cuda() for a in args[:5]]
    got = geng.engram_gate_grad(*dev, mask=args[5].cuda(), dx=dev[4])  # dx into dout
    assert all(torch.equal(a, b) for a, b in zip(got, exp))
    s = torch.cuda.Stream()
    dev = [a.cuda() for a in args[:5]]
    got = geng.engram_gate_grad(*dev, mask=args[5].cuda(), stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, exp))
    none = [a[:0].cuda() if a.shape[0] == T else a.cuda() for a in args[:5]]
    got = geng.engram_gate_grad(*none)
    assert got[0].shape == (0, hc, dim) and (got[2] == 0).all() and (got[3] == 0).all()


def test_gate_grad_matches_the_forward_by_differences():
    """Along a random direction, the change of a loss through engram_gate itself (its bf16 output widened)
    agrees with the gradient to the forward's own rounding: steps of whole bf16 ulps, many values."""
    rng = np.random.default_rng(12)
    T, hc, dim = 64, 2, 1024
    args = _inputs(rng, T, hc, dim, masked=0.1)
    x, kv, q, k, dout = (_f64(a) for a in args[:5])
    mask = args[5].numpy()
    dx, dkv, _, _ = (_f64(a) for a in _run(args))
    for which in ("x", "kv"):
        base = args[0] if which == "x" else args[1]
        step = _bf(rng.standard_normal(base.shape) * 2.0 ** -4)
        hi, lo = (base.float() + step.float()).to(torch.bfloat16), (base.float() - step.float()).to(torch.bfloat16)
        change = 0.5 * (_f64(hi) - _f64(lo))
        ins = lambda b: (_f64(b), kv) if which == "x" else (x, _f64(b))
        f = lambda b: (R.gate(*ins(b), q, k, mask, EPS) * dout).sum()
        diff = 0.5 * (f(hi) - f(lo))
        pred = (change * (dx if which == "x" else dkv)).sum()
        # third-order terms of a step of 1/16 of the inputs' size, and bf16 results: 2^-8 of each term
        tol = 2.0 ** -8 * np.abs(change * (dx if which == "x" else dkv)).sum() + 0.02 * abs(diff)
        assert abs(diff - pred) <= tol, (which, diff, pred, tol)


@pytest.mark.parametrize("T,hc,dim", [(4, 4, 5120), (400, 4, 5120)])
def test_gate_grad_withheld_sums_end_with_the_timeout_flag(T, hc, dim):
    """A token's sums that never arrive: the waits run out, the call ends within seconds with the flag
    raised, and the same context then computes a correct gradient."""
    import ctypes
    import time

    L = geng._lib()
    P, I32 = ctypes.c_void_p, ctypes.c_int32
    L.engram_gate_grad_withhold.argtypes = [P, P, P, P, P, P, ctypes.c_int64, I32, I32, ctypes.c_float, P, P, P, P, P,
                                            ctypes.c_uint64, ctypes.c_int64, P]
    args = _inputs(np.random.default_rng(3), T, hc, dim, masked=0.0)
    dev = [a.cuda() for a in args[:5]]
    out = [torch.empty_like(dev[0]), torch.empty_like(dev[1])] + [torch.empty((hc, dim), device="cuda") for _ in range(2)]
    ws = torch.empty(geng.engram_gate_grad_workspace(T, hc, dim), dtype=torch.uint8, device="cuda")
    assert geng.engram_device_status() == 0  # a clean start (reads and clears)
    call = lambda token: L.engram_gate_grad_withhold(*[a.data_ptr() for a in dev], None, T, hc, dim, EPS,
                                                     *[o.data_ptr() for o in out], ws.data_ptr(), ws.numel(), token,
                                                     torch.cuda.current_stream().cuda_stream)
    assert call(-1) == geng.ERR_INVALID
    t0 = time.time()
    assert call(1) == geng.OK
    torch.cuda.synchronize()
    assert time.time() - t0 < 30.0
    assert geng.engram_device_status() & geng.STATUS_TIMEOUT
    _check(args, _run(args), "after the timeout")
    assert geng.engram_device_status() == 0


# many CTAs to an SM (narrow rows), and rows cut in two where that brings more columns onto an SM
@pytest.mark.parametrize("T,hc,dim", [(9000, 1, 64), (5003, 1, 216), (6000, 4, 168), (4001, 2, 512), (2500, 8, 464),
                                      (400, 4, 1536), (333, 1, 3800), (170, 8, 1600), (310, 2, 3200), (157, 4, 3616)])
def test_gate_grad_many_tokens(T, hc, dim):
    args = _inputs(np.random.default_rng(T + hc * dim), T, hc, dim)
    got = _run(args)
    _check(args, got, f"T={T} hc={hc} dim={dim}")
    again = _run(args)
    assert all(torch.equal(a.view(torch.int8), b.view(torch.int8)) for a, b in zip(got, again))


def test_gate_grad_offsets_beyond_32_bits():
    """More than 2^31 values of x: all tokens masked but the last few, which have to come out right."""
    hc, dim = 4, 5120
    T, k = (1 << 31) // (hc * dim) + 50, 5
    args = _inputs(np.random.default_rng(4), k, hc, dim, masked=0.0)
    x, kv, dout = (torch.zeros((T, *a.shape[1:]), dtype=torch.bfloat16, device="cuda") for a in (args[0], args[1], args[4]))
    for big, a in ((x, args[0]), (kv, args[1]), (dout, args[4])):
        big[-k:] = a.cuda()
    dout[:-k, 1, 7] = 3.0
    mask = torch.zeros(T, dtype=torch.bool, device="cuda")
    mask[-k:] = True
    dx, dkv, dq, dk = geng.engram_gate_grad(x, kv, args[2].cuda(), args[3].cuda(), dout, mask)
    _check(args, (dx[-k:], dkv[-k:], dq, dk), "last tokens")
    assert torch.equal(dx[:-k], dout[:-k]) and not dkv[:-k].any()


@pytest.mark.parametrize("T,hc,dim", [(40, 4, 1024), (40, 8, 640), (30, 4, 5120), (33, 1, 64)])
def test_gate_grad_nan_and_infinity_in_open_tokens(T, hc, dim):
    """A NaN or an infinity in an open token's x, key, value or dout: NaN wherever the formula has it (a NaN dot
    makes the gate NaN, and with it the value's gradient), nothing of it in other tokens."""
    clean = _inputs(np.random.default_rng(T + dim), T, hc, dim, masked=0.0)
    args = [a.clone() for a in clean]
    kv = args[1].view(T, hc + 1, dim)
    i = hc - 1
    args[0][3, i, 5] = float("nan")
    kv[7, 0, dim - 1] = float("nan")
    args[0][11, 0, 9] = float("inf")
    kv[13, i, 0] = -float("inf")
    kv[17, hc, 6] = float("nan")
    args[4][19, i, 7] = float("nan")
    bad = [3, 7, 11, 13, 17, 19]
    got, exp = _run(args), _run(clean)
    with np.errstate(all="ignore"):
        want = R.gate_grad(*(_f64(a) for a in args[:5]), args[5].numpy(), EPS)
    for name, g, w in zip(("dx", "dkv", "dq_weight", "dk_weight"), got, want):
        assert np.array_equal(np.isnan(_f64(g)), np.isnan(w)), name
    assert all(torch.isnan(got[1].view(T, hc + 1, dim)[t, hc]).all() for t in (3, 7, 11, 13))  # the value's gradient
    good = np.setdiff1d(np.arange(T), bad)
    for g, e in zip(got[:2], exp[:2]):
        assert torch.equal(g[good], e[good])


@pytest.mark.parametrize("T,hc,dim", [(64, 2, 1024), (48, 4, 512), (24, 8, 640), (16, 4, 5120)])
def test_gate_grad_is_the_gradient_of_the_forward_kernel(T, hc, dim):
    """Central differences of sum(dout * engram_gate(...)) against engram_gate_grad, for x, the keys, the value and
    both weights, each along the signs of what its gradient adds through the gate, so that nothing cancels. dout
    leans on the value, which makes that part large. The bound: 8 standard deviations of the sum of the outputs'
    bf16 roundings (independent, uniform over an ulp), twice the difference's own truncation (the formula's
    difference less the formula's gradient, in 64 bits), and 2^-8 of every term for the gradient's rounding to
    bf16. All of it has to stay below a tenth of the part looked at, and a gradient without that part, or with its
    sign changed, has to be seen."""
    rng = np.random.default_rng(T + dim)
    x, kv = rng.standard_normal((T, hc, dim)), rng.standard_normal((T, hc + 1, dim))
    kv[:, :hc] += np.where(rng.random((T, hc, 1)) < 0.3, -1.0, 1.0) * 5 * dim ** -0.5 * x  # |dot| of about 5
    q, k = rng.uniform(0.5, 1.5, (hc, dim)), rng.uniform(0.5, 1.5, (hc, dim))
    dout = np.where(rng.random((T, hc, 1)) < 0.5, -1, 1) * kv[:, hc:] + 0.25 * rng.standard_normal((T, hc, dim))
    mask = rng.random(T) >= 0.1
    args = [_bf(a) for a in (x, kv.reshape(T, -1), q, k, dout)] + [torch.from_numpy(mask)]
    D = _f64(args[4])
    got, want = _run(args), R.gate_grad(*(_f64(a) for a in args[:5]), mask, EPS)
    key_part = np.zeros((T, hc + 1, dim))
    key_part[:, :hc] = 1.0
    key_part = key_part.reshape(T, -1)
    ulp = lambda o: 2.0 ** (np.floor(np.log2(np.abs(o) + 1e-30)) - 7)
    gpu = lambda ins: _f64(geng.engram_gate(*[a.cuda() for a in ins], mask=args[5].cuda(), eps=EPS))
    formula = lambda ins: R.gate(*[_f64(a) for a in ins], mask, EPS)
    for name, j, part, step in (("x", 0, want[0] - D, 2.0 ** -7), ("keys", 1, want[1] * key_part, 2.0 ** -7),
                                ("value", 1, want[1] * (1 - key_part), 2.0 ** -4), ("q_weight", 2, want[2], 2.0 ** -6),
                                ("k_weight", 3, want[3], 2.0 ** -6)):
        move = torch.from_numpy(np.sign(part) * step).float()
        hi, lo = list(args[:4]), list(args[:4])
        hi[j], lo[j] = (args[j].float() + move).to(torch.bfloat16), (args[j].float() - move).to(torch.bfloat16)
        change = 0.5 * (_f64(hi[j]) - _f64(lo[j]))
        diff = 0.5 * ((gpu(hi) - gpu(lo)) * D).sum()
        fhi, flo = formula(hi), formula(lo)
        trunc = abs(0.5 * ((fhi - flo) * D).sum() - (change * want[j]).sum())
        noise = np.sqrt(((0.5 * D) ** 2 * (ulp(fhi) ** 2 + ulp(flo) ** 2) / 12).sum())
        g = _f64(got[j])
        tol = 8 * noise + 2 * trunc + 2.0 ** -8 * np.abs(change * g).sum()
        pred, through = (change * g).sum(), (change * part).sum()
        assert tol < 0.1 * through, (name, tol, through)
        assert abs(diff - pred) <= tol, (name, diff, pred, tol)
        assert abs(diff - (pred - through)) > tol and abs(diff - (pred - 2 * through)) > tol, name
