"""Decode a batch whose pooled KV rows are kept in pages, in 4 bits or bf16, one layer, token by token.

  python examples/paged_decode.py [--batch 64] [--pooled 4096] [--hidden 4096] [--steps 16] [--select 512] [--bf16]

Weights and states are random; each sequence's prompt has left between none and --pooled pooled rows and the
KV rows of its last positions (as far back as the window reaches), and every fourth token completes one more.
With --select each step combines that many rows of each sequence, drawn at random. Every step's output is
compared with the same step in f64 on the cached rows as they stand and the queries and KV rows rounded as
the layer stores them, and the time of a step is printed.
"""
import argparse
import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from deepseek_sparse_attention_hisa_gb300.paged import DH, H, ROPE_DIMS, PagedDecode  # noqa: E402

EPS = 1e-6


def turn(x, pos, sign):
    """Interleaved rotary positions of the last ROPE_DIMS dims, f64."""
    f = 160000.0 ** (-2 * torch.arange(ROPE_DIMS // 2, device=x.device, dtype=torch.float64) / ROPE_DIMS)
    z = torch.view_as_complex(x[..., -ROPE_DIMS:].unflatten(-1, (-1, 2)).contiguous())
    z = torch.view_as_real(z * torch.polar(torch.ones_like(f), sign * pos * f)).flatten(-2)
    return torch.cat([x[..., :-ROPE_DIMS], z], -1)


def normed(x, w):
    x = x.double()
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w.double()


def run(batch=64, pooled=4096, hidden=4096, steps=16, select=0, bits4=True, page_rows=64, seed=0, window=128, say=print):
    """Returns the largest error of any step relative to the largest output."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    bf16 = torch.bfloat16

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda") * std

    w = {"norm": 1 + normal(hidden, std=0.1), "q": normal(hidden, H * DH, std=hidden**-0.5).to(bf16),
         "kv": normal(hidden, DH, std=hidden**-0.5).to(bf16), "sinks": normal(H) + 4, "q_norm": 2 + normal(DH, std=0.1),
         "kv_norm": 1 + normal(DH, std=0.1)}
    have = torch.randint(0, pooled + 1, (batch,), generator=g, device="cuda").tolist()
    have[0] = pooled
    start = [4 * n for n in have]
    most = pooled + steps
    recent = [normal(min(t, window - 1), DH).to(bf16) for t in start]
    layer = PagedDecode(batch, w, start, steps, batch * -(-most // page_rows), most, page_rows, window, bits4=bits4, eps=EPS, recent=recent)
    layer.append(normal(sum(have), DH, std=2).to(bf16), have)
    worst, spent = 0.0, []
    check = sorted({0, batch // 2, batch - 1})
    local = {b: list(recent[b].double()) for b in check}
    for n in range(steps):
        x, residual = normal(batch, hidden).to(bf16), normal(batch, hidden, std=3).to(bf16)
        I = None
        if select:
            order = torch.rand((batch, max(most, select)), generator=g, device="cuda")
            order[torch.arange(order.shape[1], device="cuda") >= layer.cache_len[:, None]] = 2
            val, I = order.topk(select, -1, largest=False)
            I = torch.where(val < 1.5, I, -1).to(torch.int32)
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        out = layer.step(x, residual, I)
        b.record()
        torch.cuda.synchronize()
        spent.append(a.elapsed_time(b) * 1e3)
        q = normed((layer.act @ w["q"]).view(batch, H, DH), w["q_norm"])
        kv = normed(layer.act @ w["kv"], w["kv_norm"])
        for s in check:
            at = start[s] + n
            local[s].append(turn(kv[s], at, 1).to(bf16).double())
            rows = layer.rows(s, torch.float32).double()
            if I is not None:
                rows = rows[I[s][I[s] >= 0].long()]
            v = torch.cat([torch.stack(local[s][-window:]), rows])
            z = turn(q[s], at, 1).to(bf16).double() @ v.t() / math.sqrt(DH)
            p = torch.softmax(torch.cat([z, w["sinks"].double()[:, None]], -1), -1)[:, :-1]
            want = turn(p @ v, at, -1)
            worst = max(worst, ((out[s].double() - want).abs().max() / want.abs().max()).item())
        done = [int((start[s] + n + 1) % 4 == 0) for s in range(batch)]
        layer.append(normal(sum(done), DH, std=2).to(bf16), done)
    if layer.status():
        raise RuntimeError(f"device status {layer.status():#x}")
    say(f"{batch} sequences of up to {pooled} pooled rows in {'4 bits' if bits4 else 'bf16'}, {select or 'all'} combined, {steps} tokens each: "
        f"median step {sorted(spent)[len(spent) // 2]:.0f} us, largest error {worst:.2%} of the largest output")
    return worst


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("batch", 64), ("pooled", 4096), ("hidden", 4096), ("steps", 16), ("select", 0)):
        ap.add_argument(f"--{name}", type=int, default=value)
    ap.add_argument("--bf16", action="store_true")
    a = ap.parse_args()
    run(a.batch, a.pooled, a.hidden, a.steps, a.select, not a.bf16)
