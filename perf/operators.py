"""Four operators of a mixture-of-experts layer whose weights are held in the 4-bit block formats, as
they are called and as plain torch computes them.

  linear   y = x W^T for few or many rows of x, W packed in "int4", "asym4" or "fp4"; gated: W holds
           the gate rows and then the up rows, and y = silu(x Wg^T) * (x Wu^T)
  route    expert ids of every token -> where each expert's rows begin, which token each row comes
           from, and where each token's rows went
  experts  the products of ``linear`` with another weight for each group of rows
  combine  the weighted sum of a token's expert rows

A packed weight is the packed form of its rows, one after another, each padded to whole blocks of 32
values ("int4", "fp4") or groups of 128 ("asym4"): tiles of 2048 values, each 1024 bytes of codes (value
2i in the low half of byte i) and then the scales (64 fp16; "asym4" 16 fp16 and 16 zero points).
"""
import math

import torch

own = False

DEVICE = "cuda"
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
GROUP = {"int4": 32, "asym4": 128, "fp4": 32}
TILE = {"int4": 1152, "asym4": 1072, "fp4": 1152}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one token through a square projection: nothing but latency and one read of the weight
        dict(name="linear_one_row", op="linear", fmt="int4", dtype="fp16", rows=1, n=4096, k=4096, gated=False),
        # a batch of sixteen decoding sequences through a gated projection of an 8192-wide layer
        dict(name="linear_gated_16", op="linear", fmt="asym4", dtype="bf16", rows=16, n=8192, k=8192, gated=True),
        # a short chunk through a projection whose width, depth and row stride are all odd
        dict(name="linear_odd_37", op="linear", fmt="fp4", dtype="bf16", rows=37, n=5003, k=4129, gated=False),
        # 1024 prompt tokens of an 8192-wide layer
        dict(name="linear_prompt_1024", op="linear", fmt="int4", dtype="bf16", rows=1024, n=8192, k=8192, gated=False),
        # one token, two of eight experts: single-sequence decoding
        dict(name="experts_one_token", op="experts", fmt="int4", dtype="fp16", tokens=1, top=2, experts=8, n=2048,
             k=4096, gated=True, dropped=0.0),
        # 64 decoding sequences, eight of 64 small experts each
        dict(name="experts_decode_64", op="experts", fmt="asym4", dtype="bf16", tokens=64, top=8, experts=64, n=1024,
             k=2048, gated=True, dropped=0.0),
        # an uneven mid-size batch with odd widths, dropped tokens and experts that get nothing
        dict(name="experts_ragged_1000", op="experts", fmt="fp4", dtype="fp16", tokens=1000, top=4, experts=40, n=1001,
             k=2080, gated=False, dropped=0.1),
        # a full prefill batch: the largest product
        dict(name="experts_prefill_8192", op="experts", fmt="int4", dtype="bf16", tokens=8192, top=2, experts=16,
             n=4096, k=4096, gated=True, dropped=0.0),
        # the plan of one decoding step
        dict(name="route_decode_64", op="route", tokens=64, top=8, experts=64, dropped=0.0),
        # the plan of a 32 x 1024 prefill over many experts, with padding tokens that go nowhere
        dict(name="route_prefill_32768", op="route", tokens=32768, top=8, experts=256, dropped=0.05),
        # the sums of one decoding step
        dict(name="combine_decode_64", op="combine", dtype="bf16", tokens=64, top=8, n=2048, dropped=0.0),
        # the sums of a 32 x 1024 prefill of a 4096-wide layer
        dict(name="combine_prefill_32768", op="combine", dtype="fp16", tokens=32768, top=2, n=4096, dropped=0.05),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _depth(rng, hi):
    """Whole groups (an odd number or a power of two of them), whole blocks, or any length."""
    kind = rng.randrange(4)
    if kind == 0:
        return 128 * rng.choice([g for g in (1, 2, 4, 8, 16, 32, 64) if 128 * g <= hi])
    v = _log_int(rng, 64, hi)
    if kind == 1:
        return max(1, v // 128) // 2 * 256 + 128 if v > 256 else 128
    if kind == 2:
        return v // 64 * 64 + 32 if v + 32 <= hi else hi - 32
    return min(v | 1, hi - 1)


def draw(rng):
    op = rng.choice(["linear", "linear", "experts", "experts", "route", "combine"])
    if op == "linear":
        while True:
            c = dict(op=op, fmt=rng.choice(sorted(GROUP)), dtype=rng.choice(sorted(DTYPES)), rows=_log_int(rng, 1, 4096),
                     n=_depth(rng, 8192), k=_depth(rng, 8192), gated=rng.random() < 0.5)
            if c["rows"] * c["n"] * c["k"] * (2 if c["gated"] else 1) <= 1 << 37:
                return c
    if op == "experts":
        while True:
            experts = _log_int(rng, 2, 128)
            c = dict(op=op, fmt=rng.choice(sorted(GROUP)), dtype=rng.choice(sorted(DTYPES)),
                     tokens=_log_int(rng, 1, 8192), top=rng.randint(1, min(8, experts)), experts=experts,
                     n=_depth(rng, 4096), k=_depth(rng, 4096), gated=rng.random() < 0.5,
                     dropped=rng.choice([0.0, 0.0, 0.1, 0.5]))
            wide = c["n"] * c["k"] * (2 if c["gated"] else 1)
            if experts * wide <= 1 << 29 and c["tokens"] * c["top"] * wide <= 1 << 38:
                return c
    if op == "route":
        experts = _log_int(rng, 2, 256)
        return dict(op=op, tokens=_log_int(rng, 1, 32768), top=rng.randint(1, min(8, experts)), experts=experts,
                    dropped=rng.choice([0.0, 0.0, 0.1, 0.9]))
    while True:
        c = dict(op=op, dtype=rng.choice(sorted(DTYPES)), tokens=_log_int(rng, 1, 32768), top=rng.randint(1, 8),
                 n=_depth(rng, 8192), dropped=rng.choice([0.0, 0.1, 0.5]))
        if c["tokens"] * (c["top"] + 1) * c["n"] <= 3 << 27:
            return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _pad_to(v, m):
    return (v + m - 1) // m * m


def _pack(fmt, gen, rows, k):
    """Packed form of a [rows, k] weight of normal values, some rows larger than others."""
    kp = _pad_to(k, GROUP[fmt])
    total = rows * kp
    tiles = (total + 2047) // 2048
    packed = torch.empty(tiles, TILE[fmt], dtype=torch.uint8, device=DEVICE)
    size = (torch.rand(rows, generator=gen, device=DEVICE) * 1.5 + 0.25) / math.sqrt(k)
    step = 1 << 15
    for t0 in range(0, tiles, step):
        t1 = min(t0 + step, tiles)
        i = torch.arange(t0 * 2048, t1 * 2048, device=DEVICE)
        row = torch.div(i, kp, rounding_mode="floor")
        w = torch.randn(i.numel(), generator=gen, device=DEVICE) * size[row.clamp(max=rows - 1)]
        w = torch.where((i - row * kp < k) & (i < total), w, torch.zeros_like(w))
        if fmt == "asym4":
            g = w.view(-1, 128)
            lo, hi = g.amin(1).clamp(max=0.0), g.amax(1).clamp(min=0.0)
            s = ((hi - lo) / 15.0).half()
            e = torch.where(s > 0, 1.0 / s.float(), torch.zeros_like(lo))
            z = torch.round(-lo * e).clamp(0, 15)
            code = (torch.round(g * e[:, None]) + z[:, None]).clamp(0, 15)
            tail = [s.view(-1, 16).view(torch.uint8), z.to(torch.uint8).view(-1, 16)]
        else:
            g = w.view(-1, 32)
            s = (g.abs().amax(1) / (6.0 if fmt == "fp4" else 8.0)).half()
            e = torch.where(s > 0, 1.0 / s.float(), torch.zeros(1, device=DEVICE))
            v = g * e[:, None]
            if fmt == "fp4":
                edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEVICE)
                code = torch.bucketize(v.abs(), edges) + 8 * (v < 0)
            else:
                code = torch.round(v).clamp(-8, 7) + 8
            tail = [s.view(-1, 64).view(torch.uint8)]
        code = code.to(torch.uint8).view(t1 - t0, 1024, 2)
        packed[t0:t1, :1024] = code[..., 0] | (code[..., 1] << 4)
        packed[t0:t1, 1024:] = torch.cat(tail, 1)
    return packed.view(-1)


def _activations(gen, rows, k, dtype):
    """Normal values, one in a thousand twenty times as large."""
    x = torch.randn(rows, k, generator=gen, device=DEVICE)
    x = torch.where(torch.rand(rows, k, generator=gen, device=DEVICE) < 1e-3, x * 20, x)
    return x.to(DTYPES[dtype])


def _ids(gen, case, experts):
    """``top`` different experts for each token, some experts far more popular than others; a dropped
    token has -1 throughout, as a padding token does."""
    popular = torch.randn(experts, generator=gen, device=DEVICE) * 0.7
    noise = torch.rand(case["tokens"], experts, generator=gen, device=DEVICE).clamp(min=1e-9)
    score = popular - torch.log((-torch.log(noise)).clamp(min=1e-9))
    ids = score.topk(case["top"], 1).indices.to(torch.int32)
    gone = torch.rand(case["tokens"], 1, generator=gen, device=DEVICE) < case["dropped"]
    return torch.where(gone, torch.full_like(ids, -1), ids)


def _plan(ids, experts):
    """Plan of ``route`` from its definition, in plain torch."""
    flat = ids.reshape(-1)
    hit = torch.arange(experts, device=flat.device, dtype=flat.dtype)[:, None] == flat
    upto = torch.cumsum(hit, 1, dtype=torch.int32)
    count = hit.sum(1, dtype=torch.int32)
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device=flat.device)
    offsets[1:] = torch.cumsum(count, 0)
    within = (upto * hit).sum(0, dtype=torch.int32) - 1
    kept = (flat >= 0) & (flat < experts)
    begin = offsets[flat.clamp(0, experts - 1).long()]
    pos = torch.where(kept, begin + within, torch.full_like(within, -1))
    rows = torch.full((flat.numel() + 1,), -1, dtype=torch.int32, device=flat.device)
    token = torch.div(torch.arange(flat.numel(), device=flat.device), ids.shape[1], rounding_mode="floor")
    # a dropped slot writes to the spare last place
    rows[torch.where(kept, pos, torch.full_like(pos, flat.numel())).long()] = token.to(torch.int32)
    rows[-1] = -1
    return offsets, rows[:-1].clone(), pos.view(ids.shape)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    state = dict(case)
    op = case["op"]
    wide = case["n"] * (2 if case.get("gated") else 1) if "n" in case else 0
    if op == "linear":
        state["x"] = _activations(gen, case["rows"], case["k"], case["dtype"])
        state["w"] = _pack(case["fmt"], gen, wide, case["k"])
    elif op == "experts":
        state["x"] = _activations(gen, case["tokens"], case["k"], case["dtype"])
        state["w"] = _pack(case["fmt"], gen, case["experts"] * wide, case["k"])
        ids = _ids(gen, case, case["experts"])
        state["offsets"], state["token"], _ = _plan(ids, case["experts"])
    elif op == "route":
        state["ids"] = _ids(gen, case, case["experts"])
    else:
        slots = case["tokens"] * case["top"]
        ids = _ids(gen, case, max(8, case["top"]))
        _, _, state["pos"] = _plan(ids, max(8, case["top"]))
        state["y"] = torch.randn(slots, case["n"], generator=gen, device=DEVICE).to(DTYPES[case["dtype"]])
        state["gates"] = torch.softmax(torch.randn(case["tokens"], case["top"], generator=gen, device=DEVICE), 1)
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


def _decoded(fmt, packed, rows, k):
    """The weight [rows, k] in fp32."""
    kp = _pad_to(k, GROUP[fmt])
    b = packed.view(-1, TILE[fmt])
    code = torch.stack([b[:, :1024] & 15, b[:, :1024] >> 4], 2).view(-1, GROUP[fmt])
    if fmt == "asym4":
        scale = b[:, 1024:1056].contiguous().view(torch.float16).view(-1, 1).float()
        value = code.float() - b[:, 1056:].reshape(-1, 1).float()
    else:
        scale = b[:, 1024:].contiguous().view(torch.float16).view(-1, 1).float()
        if fmt == "fp4":
            value = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=b.device)[code.int()]
        else:
            value = code.float() - 8
    return (value * scale).view(-1)[:rows * kp].view(rows, kp)[:, :k]


def _product(x, w, n, gated):
    h = x @ w.t()
    if gated:
        gate, up = h[:, :n], h[:, n:]
        h = gate / (1 + torch.exp(-gate)) * up
    return h


def run(state):
    op = state["op"]
    if own:
        qa = _package()
        if op == "linear":
            return qa.qr_linear(state["fmt"], state["x"], state["w"], state["n"], gated=state["gated"])
        if op == "experts":
            return qa.qr_experts(state["fmt"], state["x"], state["w"], state["n"], state["offsets"],
                                 rows=state["token"], gated=state["gated"])
        if op == "route":
            return qa.qr_route(state["ids"], state["experts"])
        return qa.qr_combine(state["y"], state["pos"], state["gates"])

    if op == "linear":
        wide = state["n"] * (2 if state["gated"] else 1)
        w = _decoded(state["fmt"], state["w"], wide, state["k"])
        return _product(state["x"].float(), w, state["n"], state["gated"]).to(state["x"].dtype)
    if op == "experts":
        wide = state["n"] * (2 if state["gated"] else 1)
        w = _decoded(state["fmt"], state["w"], state["experts"] * wide, state["k"])
        offsets = state["offsets"].tolist()
        y = torch.zeros(state["token"].numel(), state["n"], dtype=state["x"].dtype, device=w.device)
        for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
            if hi > lo:
                x = state["x"][state["token"][lo:hi].long()].float()
                y[lo:hi] = _product(x, w[e * wide:(e + 1) * wide], state["n"], state["gated"]).to(y.dtype)
        return y
    if op == "route":
        return _plan(state["ids"], state["experts"])
    pos = state["pos"]
    kept = pos >= 0
    terms = state["y"][pos.clamp(min=0).long()].float() * state["gates"][..., None]
    terms = torch.where(kept[..., None], terms, torch.zeros_like(terms))
    return terms.sum(1).to(state["y"].dtype)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def _weight_bytes(fmt, rows, k):
    return (rows * _pad_to(k, GROUP[fmt]) + 2047) // 2048 * TILE[fmt]


def work(case):
    op = case["op"]
    n = case.get("n", 0)
    wide = n * (2 if case.get("gated") else 1)
    if op == "linear":
        m = case["rows"]
        return {"bytes": _weight_bytes(case["fmt"], wide, case["k"]) + 2 * m * (case["k"] + n),
                "flops": 2 * m * wide * case["k"]}
    tokens, top = case["tokens"], case["top"]
    kept = (1 - case["dropped"]) * tokens
    slots = tokens * top
    if op == "experts":
        # each kept token picks ``top`` different experts: the share of experts that some token picks
        used = case["experts"] * (1 - (1 - top / case["experts"]) ** kept)
        return {"bytes": int(used * _weight_bytes(case["fmt"], wide, case["k"]) + 2 * kept * case["k"]
                             + 2 * slots * n + 4 * slots + 4 * (case["experts"] + 1)),
                "flops": int(2 * kept * top * wide * case["k"])}
    if op == "route":
        return {"bytes": 4 * (3 * slots + case["experts"] + 1), "flops": slots}
    return {"bytes": int(2 * kept * top * n + 2 * tokens * n + 8 * slots), "flops": int(2 * kept * top * n)}


# ---------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _weight64(fmt, packed, first, rows, k):
    """Rows ``first`` to ``first + rows`` of the weight in fp64, each value looked up by its own number."""
    group, tile = GROUP[fmt], TILE[fmt]
    kp = _pad_to(k, group)
    v = ((first + torch.arange(rows, device=packed.device)) * kp)[:, None] + torch.arange(k, device=packed.device)
    base, at = v // 2048 * tile, v % 2048
    code = (packed[base + at // 2] >> (4 * (at % 2)).to(torch.uint8)) & 15
    block = base + 1024 + at // group * 2
    bits = packed[block].int() | (packed[block + 1].int() << 8)
    exponent, mantissa = (bits >> 10) & 31, (bits & 1023).double()
    scale = torch.where(exponent == 0, torch.ldexp(mantissa, torch.tensor(-24, device=bits.device)),
                        torch.ldexp(1024 + mantissa, exponent - 25))
    if fmt == "fp4":
        e, m = (code >> 1) & 3, (code & 1).double()
        value = torch.where(e == 0, m * 0.5, torch.ldexp(1 + 0.5 * m, e.int() - 1))
        value = torch.where(code >= 8, -value, value)
    else:
        zero = packed[base + 1056 + at // 128].double() if fmt == "asym4" else 8.0
        value = code.double() - zero
    return value * scale


def _layer64(fmt, packed, first, x, n, k, gated):
    out = torch.empty(x.shape[0], n, dtype=torch.float64, device=x.device)
    for c in range(0, n, 1024):
        m = min(1024, n - c)
        out[:, c:c + m] = torch.mm(x, _weight64(fmt, packed, first + c, m, k).t().contiguous())
        if gated:
            up = torch.mm(x, _weight64(fmt, packed, first + n + c, m, k).t().contiguous())
            out[:, c:c + m] *= torch.sigmoid(out[:, c:c + m]) * up
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        return _layer64(case["fmt"], s["w"], 0, s["x"].double(), case["n"], case["k"], case["gated"])
    if op == "experts":
        wide = case["n"] * (2 if case["gated"] else 1)
        out = torch.zeros(s["token"].numel(), case["n"], dtype=torch.float64, device=s["x"].device)
        begin = s["offsets"].cpu()
        for e in range(case["experts"]):
            mine = s["token"][begin[e]:begin[e + 1]].long()
            if mine.numel():
                out[begin[e]:begin[e + 1]] = _layer64(case["fmt"], s["w"], e * wide, s["x"].double()[mine], case["n"],
                                                      case["k"], case["gated"])
        return out
    if op == "route":
        ids = s["ids"].cpu().tolist()
        groups = [[] for _ in range(case["experts"])]
        pos = [[-1] * case["top"] for _ in ids]
        for t, row in enumerate(ids):
            for j, e in enumerate(row):
                if 0 <= e < case["experts"]:
                    groups[e].append((t, j))
        offsets, rows = [0], []
        for g in groups:
            for t, j in g:
                pos[t][j] = len(rows)
                rows.append(t)
            offsets.append(len(rows))
        rows += [-1] * (case["tokens"] * case["top"] - len(rows))
        return tuple(torch.tensor(v, dtype=torch.int32, device=DEVICE) for v in (offsets, rows, pos))
    out = torch.zeros(case["tokens"], case["n"], dtype=torch.float64, device=s["y"].device)
    for j in range(case["top"]):
        p = s["pos"][:, j].long()
        here = (p >= 0).nonzero()[:, 0]
        out.index_add_(0, here, s["y"].double().index_select(0, p[here]) * s["gates"][here, j].double()[:, None])
    return out
