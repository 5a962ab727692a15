"""One mixture-of-experts layer, tensor-parallel over simulated ranks on one GPU, with
4-bit weights and a compressed all-reduce.

Each rank holds a slice of every expert's hidden width.  A rank's part of the layer is

    plan = qr_route(ids)                      where each token's rows go
    h    = qr_experts(x, w1, gated)           silu(gate) * up of its slice
    y    = qr_experts(h, w2)                  its part of the expert's output
    out  = qr_combine(y, gates)               the weighted sum of a token's experts

and then the ranks' partial outputs are added up as a compressed all-reduce does:
``qr_encode`` on every rank, ``qr_reduce_compressed`` on the encoded buffers.

    python examples/tensor_parallel_moe.py [--tokens T] [--ranks R] [--fmt int4|asym4|fp4]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bit_quantized_all_amd as qa  # noqa: E402


class Rank:
    """One rank's weights: columns [lo, hi) of the hidden width of each expert."""

    def __init__(self, fmt, gate_up, down, lo, hi):
        self.fmt, self.inner = fmt, hi - lo
        inner = down.shape[2]
        rows = torch.cat([torch.arange(lo, hi), torch.arange(inner + lo, inner + hi)])
        self.w1 = qa.qr_encode_weight(fmt, gate_up[:, rows.to(gate_up.device)].contiguous())
        self.w2 = qa.qr_encode_weight(fmt, down[:, :, lo:hi].contiguous())

    def partial(self, x, plan, gates):
        offsets, rows, pos = plan
        h = qa.qr_experts(self.fmt, x, self.w1, self.inner, offsets, rows=rows, gated=True)
        y = qa.qr_experts(self.fmt, h, self.w2, x.shape[1], offsets)
        return qa.qr_combine(y, pos, gates)


def layer(ranks, x, ids, gates, experts, wire="int8"):
    """The layer's output on every rank: plan, partial outputs, compressed all-reduce."""
    plan = qa.qr_route(ids, experts)
    packed = [qa.qr_encode(wire, r.partial(x, plan, gates)) for r in ranks]
    _, out = qa.qr_reduce_compressed(wire, x.dtype, packed, x.numel())
    return out.view_as(x)


def reference(gate_up, down, x, ids, gates):
    """The same layer in fp32 with the unpacked weights."""
    out = torch.zeros(x.shape, dtype=torch.float32, device=x.device)
    for e in range(gate_up.shape[0]):
        hit = (ids == e).any(1)
        if hit.any():
            g, u = (x[hit].float() @ gate_up[e].float().t()).chunk(2, 1)
            y = (torch.nn.functional.silu(g) * u) @ down[e].float().t()
            out[hit] += y * (gates[hit] * (ids[hit] == e)).sum(1, keepdim=True)
    return out


def make(tokens, width, inner, experts, top, dtype, device, seed=0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(tokens, width, generator=gen)
    gate_up = torch.randn(experts, 2 * inner, width, generator=gen) / width ** 0.5
    down = torch.randn(experts, width, inner, generator=gen) / inner ** 0.5
    gates, ids = torch.softmax(torch.randn(tokens, experts, generator=gen), 1).topk(top, 1)
    gates = gates / gates.sum(1, keepdim=True)
    return (x.to(device, dtype), gate_up.to(device, dtype), down.to(device, dtype), ids.to(device),
            gates.contiguous().to(device))


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--ranks", type=int, default=4)
    ap.add_argument("--fmt", default="int4", choices=["int4", "asym4", "fp4"])
    ap.add_argument("--width", type=int, default=2048)
    ap.add_argument("--inner", type=int, default=1024)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--top", type=int, default=2)
    a = ap.parse_args(argv)
    if a.inner % (128 * a.ranks) or (a.tokens * a.width) % qa.TILE_VALUES:
        ap.error("inner: a multiple of 128 for each rank; tokens * width: whole tiles of 2048 values")
    x, gate_up, down, ids, gates = make(a.tokens, a.width, a.inner, a.experts, a.top, torch.bfloat16, "cuda")
    part = a.inner // a.ranks
    ranks = [Rank(a.fmt, gate_up, down, r * part, (r + 1) * part) for r in range(a.ranks)]
    out = layer(ranks, x, ids, gates, a.experts)
    want = reference(gate_up, down, x, ids, gates)
    err = ((out.float() - want).norm() / want.norm()).item()
    times = []
    for _ in range(20):
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        layer(ranks, x, ids, gates, a.experts)
        end.record()
        end.synchronize()
        times.append(begin.elapsed_time(end))
    print(f"{a.fmt}, {a.tokens} tokens, {a.ranks} ranks: relative error against fp32 weights {err:.3f}, "
          f"{sorted(times)[10] * 1e3:.0f} us", flush=True)
    return err


if __name__ == "__main__":
    main()
