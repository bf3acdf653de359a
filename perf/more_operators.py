"""The low-bit operators of the Engram block as measured cases: 4-bit microscaled values (quantised and
read back, rows of 4-bit tables, the `wkv` projection as a product of 4-bit operands), and activation
checkpoints in 8 bits (their quantisation, and the gate's gradient that reads them). Each operator in its
plain form (elementary torch operations in 32 bits, in 64 next to a rounding's border, rounded once at the
end) and, where `own` is true, through this package's entry points.

4-bit values are E2M1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), two to a byte, with one scale for
each block of a row: blocks of 32 with a power of two ("mx"), blocks of 16 with an E4M3 number ("nv"); a
power of two for the whole tensor goes with both. 8-bit values are E4M3 with a power of two for each block."""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BLOCK = {"mx": 32, "nv": 16}
W_FACTOR = 2.0 ** -12  # of the projection's "nv" weights, so that the E4M3 scales of values of order 0.01 are normal


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a decode batch's looked-up rows (24 columns of 256) to 4 bits and back: latency counts
        {"name": "pack4 256x6144 mx", "op": "pack4", "rows": 256, "dim": 6144, "dtype": "bf16", "fmt": "mx"},
        # the projection's weights at the released width, once when a model is loaded
        {"name": "pack4 25600x6144 nv", "op": "pack4", "rows": 25600, "dim": 6144, "dtype": "bf16", "fmt": "nv"},
        # one decode step of 256 sequences over a 4-bit table
        {"name": "rows4 256x24 mx", "op": "rows4", "T": 256, "C": 24, "dim": 128, "rows": 1_000_003, "fmt": "mx"},
        # the full-scale batch, 8 sequences of 8,192 tokens, over a table of 24 million rows
        {"name": "rows4 65536x24 nv", "op": "rows4", "T": 65536, "C": 24, "dim": 128, "rows": 24_000_000,
         "fmt": "nv"},
        # one token through the projection: the weights are all there is to read
        {"name": "project4 1 mx", "op": "project4", "T": 1, "C": 24, "dim": 256, "N": 25600, "fmt": "mx",
         "src": "operand"},
        # a decode batch from the bf16 rows of another lookup, quantised within the call
        {"name": "project4 256 nv", "op": "project4", "T": 256, "C": 24, "dim": 256, "N": 25600, "fmt": "nv",
         "src": "values"},
        # an odd prompt of a narrower layer
        {"name": "project4 777x1992 mx", "op": "project4", "T": 777, "C": 11, "dim": 96, "N": 1992, "fmt": "mx",
         "src": "values"},
        # a batch of prompts from the hash ids: the 4-bit rows are gathered as they stand, then multiplied
        {"name": "project4 16384 mx", "op": "project4", "T": 16384, "C": 24, "dim": 256, "N": 25600, "fmt": "mx",
         "src": "ids"},
        # the residual copies of an odd small batch, kept in 8 bits
        {"name": "pack8 333x2x1040", "op": "pack8", "rows": 666, "dim": 1040, "dtype": "bf16", "block": 128},
        # the keys and values of 16,384 tokens at the released width (5 rows of 5,120 a token)
        {"name": "pack8 16384x5x5120", "op": "pack8", "rows": 81920, "dim": 5120, "dtype": "bf16", "block": 128},
        # the gate's gradient from checkpoints of an odd small batch
        {"name": "grad8 333x2x1040", "op": "grad8", "T": 333, "hc": 2, "dim": 1040, "block": 128, "masked": 0.1},
        # the gate's gradient from checkpoints at the released width: 4 residual copies of 5,120
        {"name": "grad8 16384x4x5120", "op": "grad8", "T": 16384, "hc": 4, "dim": 5120, "block": 128, "masked": 0.1},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["pack4", "rows4", "project4", "pack8", "grad8"])
    fmt = rng.choice(["mx", "nv"])
    if op == "pack4":
        dim = 32 * _log_int(rng, 1, 320)
        dtype = rng.choice(["f32", "bf16", "f16"])
        return {"op": op, "rows": _log_int(rng, 1, max(1, 100_000_000 // dim)), "dim": dim, "dtype": dtype, "fmt": fmt}
    if op == "rows4":
        C, dim = rng.choice([1, 2, 3, 6, 24]), rng.choice([32, 64, 96, 128, 256, 512])
        return {"op": op, "T": _log_int(rng, 1, 65536 * 24 * 128 // (2 * C * dim)), "C": C, "dim": dim,
                "rows": _log_int(rng, 1000, 12_000_000 * 128 // dim), "fmt": fmt}
    if op == "project4":
        C, dim = rng.choice([1, 3, 7, 16, 24]), rng.choice([32, 64, 96, 160, 256])
        return {"op": op, "T": _log_int(rng, 1, 12_000), "C": C, "dim": dim, "N": 8 * _log_int(rng, 2, 2500),
                "fmt": fmt, "src": rng.choice(["operand", "values", "ids"])}
    block = rng.choice([32, 64, 128])
    if op == "pack8":
        dim = 8 * _log_int(rng, 1, 1024)
        return {"op": op, "rows": _log_int(rng, 1, 150_000_000 // dim), "dim": dim,
                "dtype": rng.choice(["f32", "bf16", "f16"]), "block": block}
    hc, dim = rng.choice([1, 2, 4, 8]), 16 * _log_int(rng, 4, 320)
    T = _log_int(rng, 1, max(1, min(40_000, 16384 * 4 * 5120 // (2 * hc * dim))))
    return {"op": op, "T": T, "hc": hc, "dim": dim, "block": block, "masked": rng.choice([0.0, 0.1, 0.5])}


# -------------------------------------------------------------- the formats, in elementary operations
def _pow2(e):
    """2^e in 64 bits, by its bits (a power function is off by a rounding here and there)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _pow2_scale(amax, most):
    """The smallest power of two (2^-127 at least) whose `most`-fold holds amax, and its exponent."""
    m, e = torch.frexp(amax.double())                 # amax = m 2^e, m in [0.5, 1)
    lm, le = math.frexp(most)
    e = torch.where(amax == 0, -127, e - le + (m > lm).to(torch.int64)).clamp(min=-127)
    return _pow2(e), e


def _round_to(v, bits, least, most):
    """v in 64 bits to the nearest number of `bits` bits after the leading one, steps of `least` at least,
    |v| at most `most`; ties to even."""
    e = torch.frexp(v)[1] - 1
    step = _pow2((e - bits).clamp(min=-1022)).clamp(min=least)
    return (torch.round(v / step) * step).clamp(-most, most)


def _quantise4(x, fmt, factor):
    """Codes' values [rows, dim] and scales' values [rows, dim / block], both fp32."""
    b = BLOCK[fmt]
    v = x.double().reshape(x.shape[0], -1, b) / factor
    amax = v.abs().amax(-1, keepdim=True)
    s = _pow2_scale(amax, 6.0)[0] if fmt == "mx" else _round_to(amax / torch.full_like(amax, 6.0), 3, 2.0 ** -9, 448.0)
    q = torch.where(s > 0, _round_to(v / torch.where(s > 0, s, 1.0), 1, 0.5, 6.0), 0.0)
    return q.reshape(x.shape).float(), s.reshape(x.shape[0], -1).float()


def _quantise8(x, block):
    """As _quantise4 for E4M3 codes in blocks of `block`, the last of a row maybe shorter."""
    rows, dim = x.shape
    n = -(-dim // block)
    v = torch.nn.functional.pad(x.double(), (0, n * block - dim)).reshape(rows, n, block)
    s = _pow2_scale(v.abs().amax(-1, keepdim=True), 448.0)[0]
    q = _round_to(v / s, 3, 2.0 ** -9, 448.0)
    return q.reshape(rows, -1)[:, :dim].float(), s.reshape(rows, n).float()


def _pack(q):
    """E2M1 values to bytes: the even place of a pair in the low four bits."""
    a = q.abs()
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code |= torch.where(q < 0, 8, 0).to(torch.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4)


def _unpack(codes):
    """Bytes to E2M1 values, fp32."""
    c = torch.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1)
    a = (c & 7).float()
    a = torch.where(a < 4, a / 2, torch.where(a < 6, a - 2, 2 * a - 8))
    return torch.where(c >= 8, -a, a)


def _stored(s, fmt):
    """Scales' values in their storage type: UE8M0 bytes (exponent + 127) or E4M3."""
    if fmt == "nv":
        return s.to(torch.float8_e4m3fn)
    return (torch.frexp(s)[1] + 126).to(torch.uint8).view(torch.float8_e8m0fnu)


def _tiles(S, rows):
    """Scales [rows, n] in the order the product reads them: 512 bytes for 128 rows and 4 scales of each,
    [row blocks, groups of 4 scales, row % 32, row / 32, 4]."""
    n = S.shape[1]
    rb, kb = -(-rows // 128), -(-n // 4)
    p = torch.zeros((rb * 128, kb * 4), device=S.device, dtype=torch.uint8)
    p[:rows, :n] = S.view(torch.uint8)
    return p.reshape(rb, 4, 32, kb, 4).permute(0, 3, 2, 1, 4).contiguous().view(S.dtype)


# ----------------------------------------------------------------------------------------- inputs
def _row_ids(gen, T, C, rows):
    """Row ids as text gives them: the rank of a token's n-gram is log-uniform (Zipf's law with
    exponent 1), spread over the column's own range of rows; one position in 50 is padding (-1)."""
    span = rows // C
    u = torch.rand((T, C), generator=gen, device="cuda", dtype=torch.float64)
    rank = (span ** u).to(torch.int64).clamp_(1, span)
    ids = (rank * 2_654_435_761) % span + torch.arange(C, device="cuda") * span
    return torch.where(torch.rand((T, C), generator=gen, device="cuda") < 0.02, -1, ids)


def _activations(gen, rows, dim, dtype):
    """Values of uneven size: a normal number times a size of its own for each 8 columns of a row."""
    x = torch.randn((rows, dim), generator=gen, device="cuda")
    size = torch.exp(torch.randn((rows, dim // 8, 1), generator=gen, device="cuda"))
    return (x.view(rows, dim // 8, 8) * size).view(rows, dim).to(dtype)


def _table4(gen, rows, dim, fmt):
    """A 4-bit table: codes of a bell shape, scales over two or three powers of two."""
    lut = torch.tensor([0, 0, 1, 1, 2, 2, 3, 4, 8, 9, 9, 10, 10, 11, 12, 5], device="cuda", dtype=torch.uint8)
    r = torch.randint(0, 256, (rows, dim // 2), generator=gen, device="cuda", dtype=torch.uint8)
    both = (lut.long()[:, None] | (lut.long()[None, :] << 4)).reshape(-1).to(torch.uint8)
    Q = torch.cat([both[part.long()] for part in r.split(4_000_000)])
    S = torch.randint(0, 24, (rows, dim // BLOCK[fmt]), generator=gen, device="cuda", dtype=torch.uint8)
    return Q, (S // 8 + 122).view(torch.float8_e8m0fnu) if fmt == "mx" else (S + 24).view(torch.float8_e4m3fn)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s, op = {"case": dict(case)}, case["op"]
    if op in ("pack4", "pack8"):
        s["x"] = _activations(gen, case["rows"], case["dim"], DTYPES[case["dtype"]])
        return s
    if op == "rows4":
        s["idx"] = _row_ids(gen, case["T"], case["C"], case["rows"])
        s["Q"], s["S"] = _table4(gen, case["rows"], case["dim"], case["fmt"])
        return s
    if op == "project4":
        T, K, N, fmt = case["T"], case["C"] * case["dim"], case["N"], case["fmt"]
        w = torch.randn((N, K), generator=gen, device="cuda") * K ** -0.5
        q, sc = _quantise4(w, fmt, W_FACTOR)
        # the weights as a program keeps them: codes, and their scales row by row and in the product's order
        s["wq"], s["ws"] = _pack(q), _stored(sc, fmt)
        s["wt"] = _tiles(s["ws"], N)
        if case["src"] == "ids":
            rows = 200_003
            s["idx"] = _row_ids(gen, T, case["C"], rows)
            s["Q"], s["S"] = _table4(gen, rows, case["dim"], fmt)
            return s
        x = _activations(gen, T, K, torch.bfloat16)
        if case["src"] == "values":
            s["x"] = x
            return s
        q, sc = _quantise4(x, fmt, 1.0)
        s["aq"], s["as"] = _pack(q), _stored(sc, fmt)
        s["at"] = _tiles(s["as"], T)
        return s
    T, hc, dim = case["T"], case["hc"], case["dim"]
    bf = torch.bfloat16
    x = torch.randn((T, hc, dim), generator=gen, device="cuda")
    kv = torch.empty((T, hc + 1, dim), device="cuda")
    kv[:, :hc] = 0.1 * x + torch.randn((T, hc, dim), generator=gen, device="cuda")
    kv[:, hc] = torch.randn((T, dim), generator=gen, device="cuda")
    for name, t in (("x", x), ("kv", kv)):  # the checkpoints as the forward pass left them
        q, sc = _quantise8(t.to(bf).view(-1, dim), case["block"])
        s[name + "q"] = q.to(torch.float8_e4m3fn).view(t.shape)
        s[name + "s"] = _stored(sc, "mx").view(t.shape[0], t.shape[1], -1)
    s["q"] = (0.5 + torch.rand((hc, dim), generator=gen, device="cuda")).to(bf)
    s["k"] = (0.5 + torch.rand((hc, dim), generator=gen, device="cuda")).to(bf)
    s["dout"] = (0.01 * torch.randn((T, hc, dim), generator=gen, device="cuda")).to(bf)
    s["mask"] = torch.rand((T,), generator=gen, device="cuda") >= case["masked"]
    return s


# -------------------------------------------------------------------------------------- one pass
def run(state):
    c = state["case"]
    if own:
        return _run_own(state, c)
    return {"pack4": _plain_pack4, "rows4": _plain_rows4, "project4": _plain_project4, "pack8": _plain_pack8,
            "grad8": _plain_grad8}[c["op"]](state, c)


def _run_own(s, c):
    import gram_hash_embedding_gb300 as geng

    op = c["op"]
    if op == "pack4":  # the values that the codes stand for
        b = BLOCK[c["fmt"]]
        codes, scales = geng.engram_quantize4(s["x"], b)
        return geng.engram_dequantize4(codes, scales, b)
    if op == "pack8":
        codes, scales = geng.engram_quantize8(s["x"], c["block"])
        return {"codes": codes.view(torch.float8_e4m3fn), "scales": scales}
    if op == "rows4":
        return geng.engram_lookup4(s["idx"], s["Q"], s["S"], BLOCK[c["fmt"]])
    if op == "project4":
        b = BLOCK[c["fmt"]]
        if c["src"] == "operand":
            a, at = s["aq"], s["at"]
        elif c["src"] == "values":
            a, at = geng.engram_quantize4(s["x"], b, tiled=True)
        else:
            a, at = geng.engram_lookup4_operand(s["idx"], s["Q"], s["S"], b)
        return geng.engram_project4(a, at, s["wq"], s["wt"], b, scale=W_FACTOR)
    dx, dkv, dq, dk = geng.engram_gate_grad8(s["xq"], s["xs"], s["kvq"], s["kvs"], s["q"], s["k"], s["dout"],
                                             c["block"], mask=s["mask"])
    return {"dx": dx, "dkv": dkv, "dq": dq, "dk": dk}


def _plain_pack4(s, c):
    q, sc = _quantise4(s["x"], c["fmt"], 1.0)
    return (q.reshape(q.shape[0], -1, BLOCK[c["fmt"]]) * sc[..., None]).reshape(q.shape).to(torch.bfloat16)


def _plain_pack8(s, c):
    q, sc = _quantise8(s["x"], c["block"])
    return {"codes": q.to(torch.float8_e4m3fn), "scales": _stored(sc, "mx")}


def _values4(codes, scales, block):
    v = _unpack(codes)
    return (v.reshape(v.shape[0], -1, block) * scales.float()[..., None]).reshape(v.shape)


def _gather4(s, c):
    idx = s["idx"].reshape(-1)
    ok = (idx >= 0) & (idx < s["Q"].shape[0])
    at = torch.where(ok, idx, 0)
    v = _values4(s["Q"][at], s["S"].view(torch.uint8)[at].view(s["S"].dtype), BLOCK[c["fmt"]])
    return torch.where(ok[:, None], v, 0.0)


def _plain_rows4(s, c):
    return _gather4(s, c).reshape(c["T"], c["C"], c["dim"]).to(torch.bfloat16)


def _plain_project4(s, c):
    b = BLOCK[c["fmt"]]
    if c["src"] == "operand":
        a = _values4(s["aq"], s["as"], b)
    elif c["src"] == "values":
        q, sc = _quantise4(s["x"], c["fmt"], 1.0)
        a = (q.reshape(q.shape[0], -1, b) * sc[..., None]).reshape(q.shape)
    else:
        a = _gather4(s, c).reshape(c["T"], -1)
    return (a @ _values4(s["wq"], s["ws"], b).t() * W_FACTOR).to(torch.bfloat16)


def _values8(codes, scales, block):
    T, n, dim = codes.shape
    return codes.float() * scales.float().repeat_interleave(block, -1)[..., :dim]


def _plain_grad8(s, c):
    hc, dim = c["hc"], c["dim"]
    h, u = _values8(s["xq"], s["xs"], c["block"]), s["dout"].float()
    kv = _values8(s["kvq"], s["kvs"], c["block"])
    k, v = kv[:, :hc], kv[:, hc:]
    q, w = s["q"].float(), s["k"].float()
    open_ = s["mask"][:, None, None]
    a = (h * h).mean(-1, keepdim=True) + 1e-20
    b = (k * k).mean(-1, keepdim=True) + 1e-20
    r = dim ** -0.5 / (a.sqrt() * b.sqrt())
    dot = (h * (q * w) * k).sum(-1, keepdim=True) * r
    m = dot.abs()
    z = torch.copysign(m.clamp(min=1e-6).sqrt(), dot)
    g = 1 / (1 + torch.exp(-z))
    dg = (u * v).sum(-1, keepdim=True)
    ddot = dg * g * (1 - g) * torch.where(m >= 1e-6, 0.5 / m.clamp(min=1e-6).sqrt(), 0.0)
    cc = ddot * r
    e = ddot * dot / dim
    dh = u + torch.where(open_, cc * (q * w) * k - e / a * h, 0.0)
    dkey = torch.where(open_, cc * (q * w) * h - e / b * k, 0.0)
    dv = torch.where(open_, g * u, 0.0).sum(1, keepdim=True)
    dw = torch.where(open_, cc * h * k, 0.0).sum(0)
    return {"dx": dh.to(torch.bfloat16), "dkv": torch.cat([dkey, dv], 1).reshape(c["T"], -1).to(torch.bfloat16),
            "dq": dw * w, "dk": dw * q}


# --------------------------------------------------------------------------------- work and truth
def _unique(n, span, C):
    """Distinct rows among n ids (n / C in each of C columns of `span` rows, log-uniform ranks)."""
    edges = np.unique(np.floor(np.exp(np.linspace(0, math.log(max(span, 2)), 4000))))
    lo, hi = edges[:-1], edges[1:]
    p = np.log(hi / lo) / math.log(max(span, 2)) / (hi - lo)
    return C * float(((hi - lo) * -np.expm1(-(0.98 * n / C) * p)).sum())


def work(case):
    op = case["op"]
    size = {"f32": 4, "bf16": 2, "f16": 2}
    if op == "pack4":  # there: the values read, codes and scales written; back: the reverse, into bf16
        n = case["rows"] * case["dim"]
        held = n / 2 + n / BLOCK[case["fmt"]]
        return {"bytes": n * (size[case["dtype"]] + 2) + 2 * held, "flops": 6 * n}
    if op == "pack8":
        n = case["rows"] * case["dim"]
        return {"bytes": n * (size[case["dtype"]] + 1) + case["rows"] * -(-case["dim"] // case["block"]), "flops": 4 * n}
    if op in ("rows4", "project4"):
        T, C, dim = case["T"], case["C"], case["dim"]
        held = dim / 2 + dim / BLOCK[case["fmt"]]  # a row's codes and scales
        rows = case.get("rows", 200_003)
        gather = 8 * T * C + min(_unique(T * C, rows // C, C), T * C) * held
        if op == "rows4":
            return {"bytes": gather + 2 * T * C * dim, "flops": T * C * dim}
        read = {"operand": T * C * held, "values": 2 * T * C * dim, "ids": gather}[case["src"]]
        return {"bytes": read + case["N"] * C * held + 2 * T * case["N"], "flops": 2 * T * C * dim * case["N"]}
    T, hc, dim = case["T"], case["hc"], case["dim"]
    scales = -(-dim // case["block"])
    # the checkpoints of x, the keys and the value; the output's gradient; dx and dkv; the weights and their gradients
    return {"bytes": T * (2 * hc + 1) * (dim + scales) + 2 * T * dim * hc + 2 * T * dim * (2 * hc + 1) + hc * dim * 12,
            "flops": 30 * T * hc * dim}


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _nearest(v, grid, most):
    """The index of the grid's number nearest to v >= 0 in 64 bits; ties to the even index; above `most`, the last."""
    g = torch.tensor(grid, device=v.device, dtype=torch.float64)
    mid = (g[1:] + g[:-1]) / 2
    up = torch.searchsorted(mid, v, right=False)      # midpoints below v
    tie = (up < mid.numel()) & (v == mid[up.clamp(max=mid.numel() - 1)])
    return torch.where(v > most, len(grid) - 1, up + (tie & (up % 2 == 1)).to(torch.int64))


E4M3 = tuple(m * 2.0 ** -9 for m in range(8)) + tuple((8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8))[:-1]


def _exact_blocks(x, block, grid, most, fmt, factor=1.0):
    """(values of codes, scales) of x [rows, dim] by the formats' definition: the grid's nearest number."""
    rows, dim = x.shape
    n = -(-dim // block)
    q, s = torch.zeros((rows, n * block), device="cuda", dtype=torch.float64), []
    g = torch.tensor(grid, device="cuda", dtype=torch.float64)
    e4m3 = torch.tensor(E4M3, device="cuda", dtype=torch.float64)
    powers = torch.tensor([2.0 ** e for e in range(-127, 128)], device="cuda", dtype=torch.float64)
    for at in range(0, rows, max(1, 20_000_000 // dim)):
        part = torch.zeros((min(rows - at, max(1, 20_000_000 // dim)), n * block), device="cuda", dtype=torch.float64)
        part[:, :dim] = x[at:at + part.shape[0]].double() / factor
        v = part.view(-1, n, block)
        amax = v.abs().amax(-1)
        if fmt == "nv":
            sc = e4m3[_nearest(amax / torch.full_like(amax, most), E4M3, 448.0)]
        else:
            sc = powers[torch.searchsorted(powers * most, amax)]
        code = _nearest(v.abs() / torch.where(sc > 0, sc, 1.0)[..., None], grid, most)
        val = torch.where(sc[..., None] > 0, g[code], 0.0) * torch.sign(v)
        q[at:at + part.shape[0]] = val.view(part.shape)
        s.append(sc)
    return q[:, :dim], torch.cat(s)


def _exact4(codes, scales, block):
    t = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda", dtype=torch.float64)
    v = torch.empty((codes.shape[0], 2 * codes.shape[1]), device="cuda", dtype=torch.float64)
    v[:, 0::2], v[:, 1::2] = t[(codes % 16).long()], t[(codes // 16).long()]
    raw = scales.view(torch.uint8).double()
    if scales.dtype == torch.float8_e4m3fn:  # below 8 the steps of 2^-9, above 8 steps to each power of two
        sc = torch.where(raw < 8, raw * 2.0 ** -9, (8 + raw % 8) * _pow2(torch.floor(raw / 8) - 10))
    else:
        sc = _pow2(raw - 127)
    return v * sc.repeat_interleave(block, 1)


def exact(case, seed):
    """The definitions in 64 bits, from the same inputs."""
    op = case["op"]
    if op == "project4" and case["T"] * case["N"] * case["C"] * case["dim"] > 1.2e13:
        return None
    s = prepare(case, seed)
    if op in ("pack4", "pack8"):
        if op == "pack8":
            q, sc = _exact_blocks(s["x"], case["block"], E4M3, 448.0, "mx")
            return {"codes": q, "scales": sc}
        b = BLOCK[case["fmt"]]
        q, sc = _exact_blocks(s["x"], b, E2M1, 6.0, case["fmt"])
        return q * sc.repeat_interleave(b, 1)
    if op in ("rows4", "project4"):
        b = BLOCK[case["fmt"]]
        if "idx" in s:
            idx = s["idx"].reshape(-1)
            inside = ((idx >= 0) & (idx < s["Q"].shape[0])).nonzero()[:, 0]
            a = torch.zeros((idx.numel(), case["dim"]), device="cuda", dtype=torch.float64)
            for at in inside.split(2_000_000):
                a[at] = _exact4(s["Q"][idx[at]], s["S"].view(torch.uint8)[idx[at]].view(s["S"].dtype), b)
            if op == "rows4":
                return a.view(case["T"], case["C"], case["dim"])
            a = a.view(case["T"], -1)
        elif "x" in s:
            q, sc = _exact_blocks(s["x"], b, E2M1, 6.0, case["fmt"])
            a = q * sc.repeat_interleave(b, 1)
        else:
            a = _exact4(s["aq"], s["as"], b)
        return a @ (_exact4(s["wq"], s["ws"], b) * W_FACTOR).t()
    # out_i = h_i + gate_i * value, differentiated by hand through u = h/|h| and y = key/|key|:
    # dot = sqrt(dim) * sum(u q k y), because mean squares are |.|^2 / dim (eps is far below them)
    T, hc, dim = case["T"], case["hc"], case["dim"]

    def value_of(name, i):
        raw = s[name + "s"][:, i].view(torch.uint8).double()
        return s[name + "q"][:, i].double() * _pow2(raw - 127).repeat_interleave(case["block"], 1)[:, :dim]

    value = value_of("kv", hc)
    live = s["mask"].double()[:, None]
    dx = torch.empty((T, hc, dim), device="cuda", dtype=torch.float64)
    dkv = torch.zeros((T, hc + 1, dim), device="cuda", dtype=torch.float64)
    dq = torch.empty((hc, dim), device="cuda", dtype=torch.float64)
    dk = torch.empty((hc, dim), device="cuda", dtype=torch.float64)
    for i in range(hc):
        h, key, up = value_of("x", i), value_of("kv", i), s["dout"][:, i].double()
        q, k = s["q"][i].double(), s["k"][i].double()
        nh, nk = h.norm(dim=1, keepdim=True), key.norm(dim=1, keepdim=True)
        u, y = h / nh, key / nk
        cos = (u * q * k * y).sum(1, keepdim=True)
        dot = math.sqrt(dim) * cos
        root = dot.abs().clamp(min=1e-6).sqrt()
        gate = torch.sigmoid(torch.where(dot < 0, -root, root))
        slope = gate * (1 - gate) * (dot.abs() >= 1e-6) / (2 * root)
        t = (up * value).sum(1, keepdim=True) * slope * math.sqrt(dim) * live  # d loss / d cos
        dx[:, i] = up + t / nh * (q * k * y - cos * u)
        dkv[:, i] = t / nk * (q * k * u - cos * y)
        dkv[:, hc] += gate * live * up
        dw = (t * u * y).sum(0)
        dq[i], dk[i] = dw * k, dw * q
    return {"dx": dx, "dkv": dkv.reshape(T, -1), "dq": dq, "dk": dk}
