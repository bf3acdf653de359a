"""The operators that train the Engram front end, as measured cases: the lookup of trainable
embedding rows and its gradient by sorted row ids, the gradient of the Engram gate, and the global
gradient norm with clipping. Each operator in its plain form (elementary torch operations in 32 bits,
rounded once at the end) and, where `own` is true, through this package's entry points."""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
FULL_ROWS = 384_006_168  # rows of a full-scale hash table: 24 columns of 16 million buckets and more
VOCAB = 129_280          # the tokenizer's ids
CLIP_EPS = 1e-6          # added to the norm before the division, as the common clipping formula has it


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of 256 sequences: 24 hash columns a token, a trainable bf16 table
        {"name": "embed decode 256x24", "op": "embed", "T": 256, "C": 24, "dim": 128, "rows": 1_000_003,
         "table": "bf16", "out": "bf16", "scale": 1.0},
        # the full-scale batch, 8 sequences of 8,192 tokens, over tables of 24 million rows
        {"name": "embed full 65536x24", "op": "embed", "T": 65536, "C": 24, "dim": 128, "rows": 24_000_000,
         "table": "bf16", "out": "bf16", "scale": 1.0},
        # gradient rows of a small step: few duplicates, latency counts
        {"name": "rows decode 256x24", "op": "rows", "T": 256, "C": 24, "dim": 128, "rows": FULL_ROWS,
         "dout": "bf16", "grad": "f32", "scale": 1.0},
        # gradient rows of the full-scale batch for one layer's table: half of the n-grams repeat
        {"name": "rows full 65536x24", "op": "rows", "T": 65536, "C": 24, "dim": 128, "rows": FULL_ROWS,
         "dout": "bf16", "grad": "f32", "scale": 1.0},
        # the token embedding of a model of width 5,120, scaled by the root of its width: a dense gradient
        {"name": "dense tokens 16384", "op": "dense", "T": 16384, "C": 1, "dim": 5120, "rows": VOCAB,
         "dout": "bf16", "grad": "f32", "scale": 71.55417528, "accumulate": False},
        # a small table of odd sizes whose gradient is added to what earlier micro-batches left
        {"name": "dense odd 1777x3", "op": "dense", "T": 1777, "C": 3, "dim": 100, "rows": 5003,
         "dout": "f32", "grad": "f32", "scale": 0.5, "accumulate": True},
        # the gate's gradient at an odd small width
        {"name": "gate odd 333", "op": "gate", "T": 333, "hc": 2, "dim": 1032, "masked": 0.1},
        # the gate's gradient for 16,384 tokens at the released width: 4 residual copies of 5,120
        {"name": "gate 16384", "op": "gate", "T": 16384, "hc": 4, "dim": 5120, "masked": 0.1},
        # the norm of a small model's gradients, for the log
        {"name": "norm small", "op": "norm", "tensors": 24, "values": 30_011, "dtype": "mix", "sparse": 0, "dim": 128},
        # the norm over a block's weights and the gradient rows of its table (1.57M rows, part of them in use)
        {"name": "norm large", "op": "norm", "tensors": 300, "values": 400_000_000, "dtype": "mix",
         "sparse": 1_572_864, "dim": 128},
        # clipping a small model's gradients into the optimizer's flat fp32 buffer
        {"name": "clip small", "op": "clip", "tensors": 12, "values": 200_003, "dtype": "mix", "sparse": 0, "dim": 128},
        # clipping a block's gradients: weights in bf16 and fp32, and the gradient rows of its table
        {"name": "clip large", "op": "clip", "tensors": 200, "values": 400_000_000, "dtype": "mix",
         "sparse": 1_572_864, "dim": 128},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed", "rows", "dense", "gate", "norm", "clip"])
    if op in ("embed", "rows"):
        C = rng.choice([1, 2, 3, 6, 24])
        dim = rng.choice([16, 32, 64, 100, 128, 256, 512])
        T = _log_int(rng, 1, max(1, min(65536 * 24 // C, 65536 * 24 * 128 // (C * dim))))
        rows = _log_int(rng, 1000, 12_000_000 * 128 // dim if op == "embed" else FULL_ROWS)
        case = {"op": op, "T": T, "C": C, "dim": dim, "rows": max(rows, 2 * C), "scale": rng.choice([1.0, 0.125, 11.3137085])}
        if op == "embed":
            case.update(table=rng.choice(["f32", "bf16", "f16"]), out=rng.choice(["f32", "bf16", "f16"]))
            if case["table"] == "f32" or case["out"] == "f32":
                case["T"] = max(1, T // 2)
        else:
            case.update(dout=rng.choice(["f32", "bf16", "f16"]), grad=rng.choice(["f32", "f32", "bf16"]))
            if case["dout"] == "f32":
                case["T"] = max(1, T // 2)
        return case
    if op == "dense":
        dim = rng.choice([64, 100, 257, 512, 1024, 2048, 5120])
        rows = _log_int(rng, 100, min(VOCAB, 129_280 * 5120 // (2 * dim)))
        return {"op": op, "T": _log_int(rng, 1, 12_000), "C": 1, "dim": dim, "rows": rows,
                "dout": rng.choice(["f32", "bf16", "f16"]), "grad": rng.choice(["f32", "f32", "bf16"]),
                "scale": round(math.sqrt(dim), 6), "accumulate": rng.random() < 0.3}
    if op == "gate":
        hc = rng.choice([1, 2, 4, 8])
        dim = 8 * _log_int(rng, 8, 640)
        return {"op": op, "T": _log_int(rng, 1, max(1, 16384 * 4 * 5120 // (hc * dim) // 2)) if hc * dim > 1024 else
                _log_int(rng, 1, 40_000), "hc": hc, "dim": dim, "masked": rng.choice([0.0, 0.1, 0.5])}
    tensors = _log_int(rng, 1, 400)
    return {"op": op, "tensors": tensors, "values": max(tensors, _log_int(rng, 1000, 300_000_000)),
            "dtype": rng.choice(["f32", "bf16", "f16", "mix"]), "sparse": rng.choice([0, 0, 1003, 100_000]),
            "dim": rng.choice([64, 100, 128])}


# ----------------------------------------------------------------------------------------- inputs
def _row_ids(gen, T, C, rows):
    """Row ids as text gives them: the rank of a token's n-gram is log-uniform (Zipf's law with
    exponent 1), spread over the column's own range of rows; one position in 50 is padding (-1)."""
    span = rows // C
    u = torch.rand((T, C), generator=gen, device="cuda", dtype=torch.float64)
    rank = (span ** u).to(torch.int64).clamp_(1, span)
    ids = (rank * 2_654_435_761) % span + torch.arange(C, device="cuda") * span
    return torch.where(torch.rand((T, C), generator=gen, device="cuda") < 0.02, -1, ids)


def _normal(gen, shape, dtype=torch.float32, scale=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype).mul_(scale)


def _sizes(case):
    """The sizes of the tensors of a gradient list: spread over three decades, mostly odd, in all
    about `values`; and whether each is fp32, bf16 or fp16."""
    k = case["tensors"]
    w = [math.exp(3 * math.log(10) * ((i * 37) % k) / k) for i in range(k)]
    sizes = [max(1, int(case["values"] * x / sum(w))) for x in w]
    kinds = [case["dtype"] if case["dtype"] != "mix" else ("bf16", "f32", "bf16", "f16")[i % 4] for i in range(k)]
    return sizes, kinds


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s, op = {"case": dict(case)}, case["op"]
    if op in ("embed", "rows", "dense"):
        T, C, dim, rows = case["T"], case["C"], case["dim"], case["rows"]
        s["idx"] = _row_ids(gen, T, C, rows)
        if op == "embed":
            s["W"] = _normal(gen, (rows, dim), DTYPES[case["table"]], 0.02)
            return s
        s["dout"] = _normal(gen, (T, C, dim), DTYPES[case["dout"]], 0.01)
        if op == "rows":
            # the buffers of a training loop: rows past the call's count are never written
            s["grad"] = torch.zeros((T * C, dim), device="cuda", dtype=DTYPES[case["grad"]])
        elif case["accumulate"]:
            s["grad"] = _normal(gen, (rows, dim), DTYPES[case["grad"]], 0.01)
        else:
            s["grad"] = torch.empty((rows, dim), device="cuda", dtype=DTYPES[case["grad"]])
        return s
    if op == "gate":
        T, hc, dim = case["T"], case["hc"], case["dim"]
        bf = torch.bfloat16
        s["x"] = _normal(gen, (T, hc, dim), bf)
        kv = torch.empty((T, hc + 1, dim), device="cuda", dtype=bf)
        kv[:, :hc] = (0.1 * s["x"].float() + torch.randn((T, hc, dim), generator=gen, device="cuda")).to(bf)
        kv[:, hc] = torch.randn((T, dim), generator=gen, device="cuda").to(bf)
        s["kv"] = kv.reshape(T, (hc + 1) * dim)
        s["q"] = (0.5 + torch.rand((hc, dim), generator=gen, device="cuda")).to(bf)
        s["k"] = (0.5 + torch.rand((hc, dim), generator=gen, device="cuda")).to(bf)
        s["dout"] = _normal(gen, (T, hc, dim), bf, 0.01)
        s["mask"] = torch.rand((T,), generator=gen, device="cuda") >= case["masked"]
        return s
    sizes, kinds = _sizes(case)
    s["grads"] = [_normal(gen, (n,), DTYPES[k], 0.01) for n, k in zip(sizes, kinds)]
    s["counts"] = [None] * len(sizes)
    if case["sparse"]:
        s["grads"].append(_normal(gen, (case["sparse"], case["dim"]), torch.float32, 0.01))
        s["counts"].append(torch.tensor([int(case["sparse"] * (0.55 + 0.001 * (seed % 100)))], device="cuda"))
    if op == "clip":
        # the optimizer's flat fp32 buffer, every tensor's part on a 32-byte boundary
        at = np.cumsum([0] + [(g.numel() + 7) // 8 * 8 for g in s["grads"]]).tolist()
        s["flat"] = torch.zeros(at[-1], device="cuda")
        s["outs"] = [s["flat"][a:a + g.numel()].view(g.shape) for a, g in zip(at, s["grads"])]
    return s


# -------------------------------------------------------------------------------------- one pass
def run(state):
    c = state["case"]
    if own:
        return _run_own(state, c)
    return {"embed": _plain_embed, "rows": _plain_rows, "dense": _plain_dense, "gate": _plain_gate,
            "norm": _plain_norm, "clip": _plain_clip}[c["op"]](state, c)


def _run_own(s, c):
    import gram_hash_embedding_gb300 as geng

    op = c["op"]
    if op == "embed":
        return geng.engram_embed(s["idx"], s["W"], scale=c["scale"], out_dtype=DTYPES[c["out"]])
    if op == "rows":
        rows, grad, count = geng.engram_embed_grad(s["idx"], s["dout"], c["rows"], scale=c["scale"], grad=s["grad"])
        return {"rows": rows, "grad": grad, "count": count}
    if op == "dense":
        return geng.engram_embed_grad_dense(s["idx"], s["dout"], s["grad"], scale=c["scale"],
                                            accumulate=c["accumulate"])
    if op == "gate":
        dx, dkv, dq, dk = geng.engram_gate_grad(s["x"], s["kv"], s["q"], s["k"], s["dout"], mask=s["mask"])
        return {"dx": dx, "dkv": dkv, "dq": dq, "dk": dk}
    if op == "norm":
        return geng.engram_grad_norm(s["grads"], counts=s["counts"])
    norm = geng.engram_grad_clip(s["grads"], 1.0, out=s["outs"], counts=s["counts"])
    return {"norm": norm, "grads": s["flat"]}


def _plain_embed(s, c):
    ok = (s["idx"] >= 0) & (s["idx"] < c["rows"])
    rows = s["W"][torch.where(ok, s["idx"], 0)].float() * c["scale"]
    return torch.where(ok[..., None], rows, 0.0).to(DTYPES[c["out"]])


def _plain_sorted(s, c):
    """Row ids in ascending order (those outside the table last, as `rows`) and their positions."""
    idx = s["idx"].reshape(-1)
    key = torch.where((idx >= 0) & (idx < c["rows"]), idx, c["rows"])
    return torch.sort(key, stable=True)


def _plain_rows(s, c):
    key, pos = _plain_sorted(s, c)
    n = key.numel()
    head = torch.ones_like(key, dtype=torch.bool)
    head[1:] = key[1:] != key[:-1]
    head &= key < c["rows"]
    slot = torch.where(key < c["rows"], torch.cumsum(head, 0) - 1, n)
    g = s["dout"].reshape(n, c["dim"])[pos].float()
    acc = torch.zeros((n + 1, c["dim"]), device="cuda").index_add_(0, slot, g)[:n]
    rows = torch.full((n + 1,), -1, device="cuda", dtype=torch.int64).scatter_(0, slot, key)[:n]
    return {"rows": rows, "grad": (acc * c["scale"]).to(DTYPES[c["grad"]]), "count": head.sum().reshape(1)}


def _plain_dense(s, c):
    key, pos = _plain_sorted(s, c)
    g = s["dout"].reshape(key.numel(), c["dim"])[pos].float()
    acc = torch.zeros((c["rows"] + 1, c["dim"]), device="cuda").index_add_(0, key, g)[:c["rows"]] * c["scale"]
    s["grad"].copy_(s["grad"].float() + acc if c["accumulate"] else acc)
    return s["grad"]


def _plain_gate(s, c):
    T, hc, dim = c["T"], c["hc"], c["dim"]
    h, u = s["x"].float(), s["dout"].float()
    kv = s["kv"].float().reshape(T, hc + 1, dim)
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
    return {"dx": dh.to(torch.bfloat16), "dkv": torch.cat([dkey, dv], 1).reshape(T, -1).to(torch.bfloat16),
            "dq": dw * w, "dk": dw * q}


def _in_use(g, count):
    """The rows of a gradient that count: the first `count` of them (all where there is no count)."""
    return g.float() if count is None else torch.where(torch.arange(g.shape[0], device="cuda")[:, None] < count, g.float(), 0.0)


def _plain_norm(s, c):
    return torch.stack([(_in_use(g, n) ** 2).sum() for g, n in zip(s["grads"], s["counts"])]).sum().sqrt()


def _plain_clip(s, c):
    norm = _plain_norm(s, c)
    coef = (1.0 / (norm + CLIP_EPS)).clamp(max=1.0)
    done = [o.copy_(_in_use(g, n) * coef) for o, g, n in zip(s["outs"], s["grads"], s["counts"])]
    return {"norm": norm, "grads": s["flat"]} if done else None


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
    if op in ("embed", "rows", "dense"):
        n, dim, rows = case["T"] * case["C"], case["dim"], case["rows"]
        distinct = min(_unique(n, rows // case["C"], case["C"]), n)
        if op == "embed":  # each distinct row read once, each output row written once
            return {"bytes": 8 * n + distinct * dim * size[case["table"]] + n * dim * size[case["out"]],
                    "flops": n * dim}
        moved = 8 * n + 0.98 * n * dim * size[case["dout"]]
        if op == "rows":
            return {"bytes": moved + 8 * n + distinct * dim * size[case["grad"]], "flops": n * dim}
        out = (2 * distinct if case["accumulate"] else rows) * dim * size[case["grad"]]
        return {"bytes": moved + out, "flops": n * dim}
    if op == "gate":
        T, hc, dim = case["T"], case["hc"], case["dim"]
        # x, the keys and the value, the output's gradient; dx and dkv; the weights and their gradients
        return {"bytes": 2 * T * dim * (3 * hc + 1) + 2 * T * dim * (2 * hc + 1) + hc * dim * (4 + 8),
                "flops": 30 * T * hc * dim}
    sizes, kinds = _sizes(case)
    read = sum(n * size[k] for n, k in zip(sizes, kinds)) + int(0.6 * case["sparse"]) * case["dim"] * 4
    values = sum(sizes) + int(0.6 * case["sparse"]) * case["dim"]
    return {"bytes": read + (4 * values if op == "clip" else 0), "flops": 2 * values + (values if op == "clip" else 0)}


def exact(case, seed):
    """The definitions in 64 bits, from the same inputs, one row or copy at a time where that is the
    definition's own shape."""
    s, op = prepare(case, seed), case["op"]
    if op == "embed":
        idx, W = s["idx"], s["W"]
        out = torch.zeros(idx.shape + (case["dim"],), device="cuda", dtype=torch.float64)
        at = ((idx >= 0) & (idx < case["rows"])).nonzero(as_tuple=True)
        out[at] = W[idx[at]].double() * float(np.float32(case["scale"]))
        return out
    if op in ("rows", "dense"):
        idx, dim = s["idx"].reshape(-1), case["dim"]
        at = ((idx >= 0) & (idx < case["rows"])).nonzero()[:, 0]
        distinct, which = torch.unique(idx[at], return_inverse=True)
        sums = torch.zeros((distinct.numel(), dim), device="cuda", dtype=torch.float64)
        sums.index_add_(0, which, s["dout"].reshape(-1, dim)[at].double())
        sums *= float(np.float32(case["scale"]))
        if op == "rows":
            out = torch.zeros((idx.numel(), dim), device="cuda", dtype=torch.float64)
            out[:distinct.numel()] = sums
            return {"rows": None, "grad": out, "count": None}
        out = s["grad"].double() if case["accumulate"] else torch.zeros((case["rows"], dim), device="cuda",
                                                                        dtype=torch.float64)
        out[distinct] += sums
        return out
    if op in ("norm", "clip"):
        return _exact_norm(s, case)
    # out_i = h_i + gate_i * value, differentiated by hand through u = h/|h| and y = key/|key|:
    # dot = sqrt(dim) * sum(u q k y), because mean squares are |.|^2 / dim (eps is far below them)
    T, hc, dim = case["T"], case["hc"], case["dim"]
    kv = s["kv"].reshape(T, hc + 1, dim)
    value = kv[:, hc].double()
    live = s["mask"].double()[:, None]
    dx = torch.empty((T, hc, dim), device="cuda", dtype=torch.float64)
    dkv = torch.zeros((T, hc + 1, dim), device="cuda", dtype=torch.float64)
    dq = torch.empty((hc, dim), device="cuda", dtype=torch.float64)
    dk = torch.empty((hc, dim), device="cuda", dtype=torch.float64)
    for i in range(hc):
        h, key, up = s["x"][:, i].double(), kv[:, i].double(), s["dout"][:, i].double()
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


def _exact_norm(s, case):
    parts = [g if n is None else g[:int(n)] for g, n in zip(s["grads"], s["counts"])]
    norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(p, dtype=torch.float64)) ** 2 for p in parts))
    if case["op"] == "norm":
        return torch.tensor(norm, dtype=torch.float64)
    flat = torch.zeros(s["flat"].shape, device="cuda", dtype=torch.float64)
    coef, at = min(1.0, 1.0 / (norm + CLIP_EPS)), 0
    for g, p in zip(s["grads"], parts):
        flat[at:at + p.numel()] = p.reshape(-1).double() * coef
        at += (g.numel() + 7) // 8 * 8
    return {"norm": torch.tensor(norm, dtype=torch.float64), "grads": flat}
