"""Four operators of a layer whose activations and weights are held in rows of 8 bits, as they are called
and as plain torch computes them.

  norm     h = x + residual; y = h / sqrt(mean(h^2) + eps) * weight, as values of the dtype or as 8-bit rows
  rows     the 8-bit rows of a matrix, and the values that they stand for
  linear8  y = x W^T of 8-bit rows: whole sums of code products, times the scales of the two rows; gated: W
           holds the gate rows and then the up rows, and y = silu(x Wg^T) * (x Wu^T)
  experts8 the products of ``linear8`` with another weight for each group of rows
  choose   a router's scores -> the experts of each token and their weights

An 8-bit row is a row of signed bytes and an fp32 scale, the largest magnitude over 127; rows are padded
with zeros to whole runs of 128.
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # one token before a 4096-wide projection: nothing but latency
        dict(name="norm_one_token", op="norm", dtype="bf16", rows=1, k=4096, residual=True, bits8=False),
        # the 32 x 1024 tokens of a 4096-wide layer, on their way into an 8-bit product
        dict(name="norm_prefill_32768", op="norm", dtype="bf16", rows=32768, k=4096, residual=True, bits8=True),
        # a chunk of odd length and width
        dict(name="rows_odd_777", op="rows", dtype="fp16", rows=777, k=5003),
        # the hidden values of 32 x 1024 tokens before the second product
        dict(name="rows_prefill_32768", op="rows", dtype="bf16", rows=32768, k=4096),
        # one token through a square projection: one read of the weight
        dict(name="linear8_one_row", op="linear8", dtype="fp16", rows=1, n=4096, k=4096, gated=False),
        # a batch of sixteen decoding sequences through a gated projection of an 8192-wide layer
        dict(name="linear8_gated_16", op="linear8", dtype="bf16", rows=16, n=8192, k=8192, gated=True),
        # a short chunk through a projection of odd width and depth
        dict(name="linear8_odd_137", op="linear8", dtype="fp16", rows=137, n=5003, k=4129, gated=False),
        # 8192 prompt tokens of an 8192-wide layer: the largest product
        dict(name="linear8_prompt_8192", op="linear8", dtype="bf16", rows=8192, n=8192, k=8192, gated=False),
        # 64 decoding sequences, eight of 64 small experts each
        dict(name="experts8_decode_64", op="experts8", dtype="bf16", tokens=64, top=8, experts=64, n=1024, k=2048,
             gated=True, dropped=0.0),
        # a prefill batch with some padding tokens
        dict(name="experts8_prefill_8192", op="experts8", dtype="bf16", tokens=8192, top=2, experts=16, n=4096,
             k=4096, gated=True, dropped=0.05),
        # the choice of one decoding step
        dict(name="choose_decode_64", op="choose", dtype="bf16", tokens=64, experts=64, top=8, score="softmax",
             bias=False, groups=1, top_groups=1, best=1, renormalise=True, masked=0.0),
        # the choice of a 32 x 1024 prefill: balanced by a bias, four of eight groups, with padding tokens
        dict(name="choose_prefill_32768", op="choose", dtype="fp32", tokens=32768, experts=256, top=8,
             score="sigmoid", bias=True, groups=8, top_groups=4, best=2, renormalise=True, masked=0.05),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, hi):
    """A power of two, whole runs of 128, or any width."""
    kind = rng.randrange(3)
    if kind == 0:
        return 1 << rng.randint(6, hi.bit_length() - 1)
    v = _log_int(rng, 64, hi)
    return max(1, v // 128) * 128 if kind == 1 else min(v | 1, hi - 1)


def draw(rng):
    op = rng.choice(["norm", "rows", "linear8", "linear8", "linear8", "experts8", "experts8", "choose", "choose"])
    dtype = rng.choice(["fp16", "bf16"])
    if op in ("norm", "rows"):
        while True:
            c = dict(op=op, dtype=dtype, rows=_log_int(rng, 1, 65536), k=_width(rng, 16384))
            if c["rows"] * c["k"] <= 1 << 27:
                break
        if op == "norm":
            c.update(residual=rng.random() < 0.6, bits8=rng.random() < 0.5)
        return c
    if op == "linear8":
        while True:
            c = dict(op=op, dtype=dtype, rows=_log_int(rng, 1, 8192), n=_width(rng, 16384), k=_width(rng, 16384),
                     gated=rng.random() < 0.5)
            wide = c["n"] * c["k"] * (2 if c["gated"] else 1)
            if wide <= 1 << 28 and c["rows"] * wide <= 1 << 38:
                return c
    if op == "experts8":
        while True:
            experts = _log_int(rng, 2, 128)
            c = dict(op=op, dtype=dtype, tokens=_log_int(rng, 1, 8192), top=rng.randint(1, min(8, experts)),
                     experts=experts, n=_width(rng, 4096), k=_width(rng, 4096), gated=rng.random() < 0.5,
                     dropped=rng.choice([0.0, 0.0, 0.1, 0.5]))
            wide = c["n"] * c["k"] * (2 if c["gated"] else 1)
            if experts * wide <= 1 << 29 and c["tokens"] * c["top"] * wide <= 1 << 38:
                return c
    each = _log_int(rng, 2, 64)
    groups = rng.choice([1, 1, 2, 4, 8])
    while each * groups > 512:
        groups //= 2
    top_groups = rng.randint(1, groups)
    return dict(op="choose", dtype=rng.choice(["fp16", "bf16", "fp32"]), tokens=_log_int(rng, 1, 32768),
                experts=each * groups, top=rng.randint(1, min(8, each * top_groups)),
                score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups,
                top_groups=top_groups, best=rng.choice([1, 2]), renormalise=rng.random() < 0.7,
                masked=rng.choice([0.0, 0.05, 0.5]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _pad_to(v, m):
    return (v + m - 1) // m * m


def _activations(gen, rows, k, dtype):
    """Normal values, one in a thousand twenty times as large."""
    x = torch.randn(rows, k, generator=gen, device=DEVICE)
    x = torch.where(torch.rand(rows, k, generator=gen, device=DEVICE) < 1e-3, x * 20, x)
    return x.to(DTYPES[dtype])


def _quantized(x):
    """8-bit rows of fp32 values: codes without padding, and the scales."""
    largest = x.abs().amax(-1)
    scales = largest / 127.0
    inverse = torch.where(largest > 0, 127.0 / largest, torch.zeros_like(largest))
    return torch.round(x * inverse[..., None]).clamp(-127, 127).to(torch.int8), scales


def _weight8(gen, rows, k):
    """Codes [rows, k padded] and scales of normal values, some rows larger than others."""
    codes = torch.zeros(rows, _pad_to(k, 128), dtype=torch.int8, device=DEVICE)
    scales = torch.empty(rows, device=DEVICE)
    step = max(1, (1 << 26) // k)
    for r in range(0, rows, step):
        m = min(step, rows - r)
        size = (torch.rand(m, 1, generator=gen, device=DEVICE) * 1.5 + 0.25) / math.sqrt(k)
        codes[r:r + m, :k], scales[r:r + m] = _quantized(torch.randn(m, k, generator=gen, device=DEVICE) * size)
    return codes, scales


def _plan(gen, case):
    """Where the rows of each expert begin and the token of each, some experts far more popular than
    others; a dropped token has no row."""
    tokens, top, experts = case["tokens"], case["top"], case["experts"]
    popular = torch.randn(experts, generator=gen, device=DEVICE) * 0.7
    noise = torch.rand(tokens, experts, generator=gen, device=DEVICE).clamp(min=1e-9)
    ids = (popular - torch.log((-torch.log(noise)).clamp(min=1e-9))).topk(top, 1).indices
    gone = torch.rand(tokens, 1, generator=gen, device=DEVICE) < case["dropped"]
    ids = torch.where(gone, experts, ids).reshape(-1)
    order = torch.sort(ids, stable=True)
    offsets = torch.searchsorted(order.values, torch.arange(experts + 1, device=DEVICE)).to(torch.int32)
    rows = torch.div(order.indices, top, rounding_mode="floor").to(torch.int32)
    rows = torch.where(order.values < experts, rows, -1)
    return offsets, rows.to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    state = dict(case)
    op = case["op"]
    if op == "choose":
        logits = torch.randn(case["tokens"], case["experts"], generator=gen, device=DEVICE) * 1.5
        logits += torch.randn(case["experts"], generator=gen, device=DEVICE)
        if case["masked"]:
            # experts that are out of use, and the rows of padding tokens
            none = torch.rand(case["experts"], generator=gen, device=DEVICE) < case["masked"] / 4
            gone = torch.rand(case["tokens"], 1, generator=gen, device=DEVICE) < case["masked"]
            logits = logits.masked_fill(none | gone, -math.inf)
        state["logits"] = logits.to(DTYPES[case["dtype"]])
        state["bias"] = torch.randn(case["experts"], generator=gen, device=DEVICE) * 0.1 if case["bias"] else None
        return state
    if op in ("norm", "rows"):
        state["x"] = _activations(gen, case["rows"], case["k"], case["dtype"])
        if op == "norm":
            dt = DTYPES[case["dtype"]]
            state["weight"] = (1 + 0.2 * torch.randn(case["k"], generator=gen, device=DEVICE)).to(dt)
            state["res"] = None
            if case["residual"]:
                state["res"] = (3 * torch.randn(case["rows"], case["k"], generator=gen, device=DEVICE)).to(dt)
        return state
    k, wide = case["k"], case["n"] * (2 if case["gated"] else 1)
    rows = case["rows"] if op == "linear8" else case["tokens"]
    codes, state["xs"] = _quantized(_activations(gen, rows, k, case["dtype"]).float())
    state["x"] = torch.zeros(rows, _pad_to(k, 128), dtype=torch.int8, device=DEVICE)
    state["x"][:, :k] = codes
    if op == "linear8":
        state["w"], state["ws"] = _weight8(gen, wide, k)
    else:
        w, ws = _weight8(gen, case["experts"] * wide, k)
        state["w"], state["ws"] = w.view(case["experts"], wide, -1), ws.view(case["experts"], wide)
        state["offsets"], state["token"] = _plan(gen, case)
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

_library = None


def _package():
    global _library
    if _library is None:
        import bit_quantized_all_amd
        _library = bit_quantized_all_amd
    return _library


def _product(x, xs, w, ws, n, gated):
    """x and w: codes in fp32, whose products and their sums are whole numbers."""
    h = (x @ w.t()) * xs[:, None] * ws
    if gated:
        gate, up = h[:, :n], h[:, n:]
        h = gate / (1 + torch.exp(-gate)) * up
    return h


def _choice(s):
    """Experts and weights of each token, in 64 bits: the order of two scores may hang on the last ones."""
    logits = s["logits"].double()
    here = logits > -math.inf
    if s["score"] == "softmax":
        e = torch.exp(logits - logits.amax(1, keepdim=True).clamp(min=-1e300)) * here
        p = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        p = torch.where(here, 1 / (1 + torch.exp(-logits)), 0)
    rank = torch.where(here, p + s["bias"].double() if s["bias"] is not None else p, -math.inf)
    if s["groups"] > 1:
        r = rank.view(rank.shape[0], s["groups"], -1)
        value = r.topk(s["best"], 2).values
        value = torch.where(value[..., :1] > -math.inf, value.clamp(min=-1e300).where(value > -math.inf, 0).sum(2, True),
                            -math.inf)[..., 0]
        taken = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :s["top_groups"]]
        kept = torch.zeros_like(value, dtype=torch.bool).scatter_(1, taken, True)
        rank = torch.where(kept[..., None], r, -math.inf).view(rank.shape)
    order = torch.sort(rank, dim=1, descending=True, stable=True)
    ids, rank = order.indices[:, :s["top"]], order.values[:, :s["top"]]
    gates = torch.where(rank > -math.inf, p.gather(1, ids), 0)
    if s["renormalise"]:
        gates = gates / gates.sum(1, keepdim=True).clamp(min=1e-300)
    return gates.float(), torch.where(rank > -math.inf, ids, -1).to(torch.int32)


def run(state):
    op = state["op"]
    if own:
        qa = _package()
        if op == "norm":
            if not state["bits8"]:
                return qa.qr_norm(state["x"], state["weight"], EPS, residual=state["res"])
            codes, scales, total, _ = qa.qr_norm_rows(state["x"], state["weight"], EPS, residual=state["res"])
            return qa.qr_decode_rows(codes, scales, state["k"], state["x"].dtype), total
        if op == "rows":
            codes, scales = qa.qr_encode_rows(state["x"])
            return qa.qr_decode_rows(codes, scales, state["k"], state["x"].dtype), scales
        if op == "linear8":
            return qa.qr_linear8(state["x"], state["xs"], state["w"], state["ws"], DTYPES[state["dtype"]],
                                 gated=state["gated"])
        if op == "experts8":
            return qa.qr_experts8(state["x"], state["xs"], state["w"], state["ws"], state["offsets"],
                                  DTYPES[state["dtype"]], rows=state["token"], gated=state["gated"])
        return qa.qr_choose(state["logits"], state["top"], score=state["score"], bias=state["bias"],
                            groups=state["groups"], top_groups=state["top_groups"], group_best=state["best"],
                            renormalise=state["renormalise"])

    if op == "norm":
        h = state["x"].float()
        if state["res"] is not None:
            h = h + state["res"].float()
        y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * state["weight"].float()
        if state["bits8"]:
            codes, scales = _quantized(y)
            y = codes.float() * scales[:, None]
        return y.to(state["x"].dtype), h.to(state["x"].dtype) if state["res"] is not None else None
    if op == "rows":
        codes, scales = _quantized(state["x"].float())
        return (codes.float() * scales[:, None]).to(state["x"].dtype), scales
    if op == "linear8":
        y = _product(state["x"].float(), state["xs"], state["w"].float(), state["ws"], state["n"], state["gated"])
        return y.to(DTYPES[state["dtype"]])
    if op == "experts8":
        offsets = state["offsets"].tolist()
        y = torch.zeros(state["token"].numel(), state["n"], dtype=DTYPES[state["dtype"]], device=state["x"].device)
        for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
            if hi > lo:
                t = state["token"][lo:hi].long()
                y[lo:hi] = _product(state["x"][t].float(), state["xs"][t], state["w"][e].float(), state["ws"][e],
                                    state["n"], state["gated"]).to(y.dtype)
        return y
    return _choice(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "norm":
        values = case["rows"] * case["k"]
        return {"bytes": 2 * values * (4 if case["residual"] else 2) + 2 * case["k"],
                "flops": values * (8 if case["bits8"] else 5)}
    if op == "rows":
        return {"bytes": 4 * case["rows"] * case["k"] + 4 * case["rows"], "flops": 4 * case["rows"] * case["k"]}
    if op == "choose":
        values = case["tokens"] * case["experts"]
        return {"bytes": values * (4 if case["dtype"] == "fp32" else 2) + 8 * case["tokens"] * case["top"]
                + (4 * case["experts"] if case["bias"] else 0), "flops": 4 * values}
    n, k = case["n"], case["k"]
    wide = n * (2 if case["gated"] else 1)
    if op == "linear8":
        m = case["rows"]
        return {"bytes": (wide + m) * (k + 4) + 2 * m * n, "flops": 2 * m * wide * k}
    kept = (1 - case["dropped"]) * case["tokens"]
    slots = case["tokens"] * case["top"]
    # each kept token picks ``top`` different experts: the share of experts that some token picks
    used = case["experts"] * (1 - (1 - case["top"] / case["experts"]) ** kept)
    return {"bytes": int((used * wide + kept) * (k + 4) + 2 * slots * n + 4 * slots + 4 * (case["experts"] + 1)),
            "flops": int(2 * kept * case["top"] * wide * k)}


# ---------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _rows64(y):
    top = np.abs(y).max(1, keepdims=True)
    step = np.where(top > 0, top / 127, 1)
    return np.rint(y / step) * step, top[:, 0] / 127


def _matrix64(x, k):
    return x[:, :k].double()


def _layer64(x, xs, w, ws, n, gated):
    out = torch.empty(x.shape[0], n, dtype=torch.float64, device=x.device)
    for c in range(0, n, 2048):
        m = min(2048, n - c)
        scaled = w[c:c + m].double() * ws[c:c + m, None].double()
        out[:, c:c + m] = torch.mm(x * xs[:, None].double(), scaled.t().contiguous())
        if gated:
            scaled = w[n + c:n + c + m].double() * ws[n + c:n + c + m, None].double()
            up = torch.mm(x * xs[:, None].double(), scaled.t().contiguous())
            out[:, c:c + m] *= torch.sigmoid(out[:, c:c + m]) * up
    return out


def _choose64(case, logits, bias):
    """A token's experts one after another, each the first of the largest rank that is left."""
    tokens, experts = logits.shape
    with np.errstate(over="ignore", invalid="ignore"):
        if case["score"] == "sigmoid":
            p = np.where(logits >= 0, 1 / (1 + np.exp(-logits)), np.exp(logits) / (1 + np.exp(logits)))
        else:
            e = np.exp(logits - np.maximum(logits.max(1, keepdims=True), -1e300))
            p = e / np.maximum(e.sum(1, keepdims=True), 1e-300)
    rank = p.copy() if bias is None else p + bias
    rank[np.isneginf(logits)] = -np.inf
    every = np.arange(tokens)
    if case["groups"] > 1:
        each = experts // case["groups"]
        value = np.full((tokens, case["groups"]), -np.inf)
        for g in range(case["groups"]):
            part = np.sort(rank[:, g * each:(g + 1) * each], 1)[:, ::-1][:, :case["best"]]
            some = part[:, 0] > -np.inf
            value[some, g] = np.where(part[some] > -np.inf, part[some], 0).sum(1)
        left = np.zeros_like(rank, dtype=bool)
        for _ in range(case["top_groups"]):
            g = value.argmax(1)
            for i in range(each):
                left[every, g * each + i] = True
            value[every, g] = -np.inf
            if np.isneginf(value).all():
                break
        rank[~left] = -np.inf
    ids = np.full((tokens, case["top"]), -1, np.int32)
    gates = np.zeros((tokens, case["top"]))
    for j in range(case["top"]):
        e = rank.argmax(1)
        some = rank[every, e] > -np.inf
        ids[some, j] = e[some]
        gates[some, j] = p[every, e][some]
        rank[every, e] = -np.inf
    if case["renormalise"]:
        total = gates.sum(1, keepdims=True)
        gates = np.where(total > 0, gates / np.where(total > 0, total, 1), 0)
    return gates, ids


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "choose":
        gates, ids = _choose64(case, s["logits"].double().cpu().numpy(),
                               None if s["bias"] is None else s["bias"].double().cpu().numpy())
        return torch.from_numpy(gates), torch.from_numpy(ids)
    if op == "rows":
        values, scales = zip(*(_rows64(x.double().cpu().numpy()) for x in s["x"].split(4096)))
        return torch.from_numpy(np.concatenate(values)), torch.from_numpy(np.concatenate(scales))
    if op == "norm":
        weight = s["weight"].double().cpu().numpy()
        values, totals = [], []
        for i in range(0, case["rows"], 4096):
            h = s["x"][i:i + 4096].double().cpu().numpy()
            if s["res"] is not None:
                h = h + s["res"][i:i + 4096].double().cpu().numpy()
            y = h / np.sqrt((h * h).mean(1, keepdims=True) + EPS) * weight
            values.append(_rows64(y)[0] if case["bits8"] else y)
            totals.append(h)
        return (torch.from_numpy(np.concatenate(values)),
                torch.from_numpy(np.concatenate(totals)) if s["res"] is not None else None)
    x = _matrix64(s["x"], case["k"])
    if op == "linear8":
        return _layer64(x, s["xs"], s["w"][:, :case["k"]], s["ws"], case["n"], case["gated"])
    out = torch.zeros(s["token"].numel(), case["n"], dtype=torch.float64, device=s["x"].device)
    begin = s["offsets"].cpu()
    for e in range(case["experts"]):
        mine = s["token"][begin[e]:begin[e + 1]].long()
        if mine.numel():
            out[begin[e]:begin[e + 1]] = _layer64(x[mine], s["xs"][mine], s["w"][e][:, :case["k"]], s["ws"][e],
                                                  case["n"], case["gated"])
    return out
