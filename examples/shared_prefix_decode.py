"""Decode a batch whose sequences share one long prompt, one layer, token by token.

  python examples/shared_prefix_decode.py [--batch 64] [--prefix 8192] [--hidden 4096] [--steps 16]

Weights and states are random. Every step's output is compared with the same step in f64 on the
activations that the norm produced and the queries and KV rows rounded as the layer stores them, and
the time of a step is printed.
"""
import argparse
import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from deepseek_sparse_attention_hisa_gb300.prefix import DH, H, ROPE_DIMS, PrefixDecode  # noqa: E402


def turn(x, pos, sign):
    """Interleaved rotary positions of the last ROPE_DIMS dims, f64."""
    f = 160000.0 ** (-2 * torch.arange(ROPE_DIMS // 2, device=x.device, dtype=torch.float64) / ROPE_DIMS)
    z = torch.view_as_complex(x[..., -ROPE_DIMS:].unflatten(-1, (-1, 2)).contiguous())
    z = torch.view_as_real(z * torch.polar(torch.ones_like(f), sign * pos * f)).flatten(-2)
    return torch.cat([x[..., :-ROPE_DIMS], z], -1)


def run(batch=64, prefix=8192, hidden=4096, steps=16, own_rows=96, seed=0, window=128, say=print):
    """Returns the largest error of any step relative to the largest output."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    bf16 = torch.bfloat16

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda") * std

    w = {"norm": 1 + normal(hidden, std=0.1), "q": normal(hidden, H * DH, std=2 * hidden**-0.5).to(bf16),
         "kv": normal(hidden, DH, std=hidden**-0.5).to(bf16), "sinks": normal(H) + 4}
    start = 4 * prefix + 3
    layer = PrefixDecode(batch, w, normal(prefix, DH).to(bf16), start, steps, own_rows, window)
    own = [normal(int(torch.randint(0, own_rows + 1, (1,), generator=g, device="cuda")), DH).to(bf16) for _ in range(batch)]
    layer.set_pooled(own)
    worst, spent = 0.0, []
    check = sorted({0, batch // 2, batch - 1})
    rows = {b: [] for b in check}
    for n in range(steps):
        x, residual = normal(batch, hidden).to(bf16), normal(batch, hidden, std=3).to(bf16)
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        out = layer.step(x, residual)
        b.record()
        torch.cuda.synchronize()
        spent.append(a.elapsed_time(b) * 1e3)
        act = layer.activations()
        q = (act @ w["q"]).view(batch, H, DH).double()
        kv = (act @ w["kv"]).double()
        for s in check:
            rows[s].append(turn(kv[s], start + n, 1).to(bf16).double())
            v = torch.cat([torch.stack(rows[s][-window:]), layer.prefix_kv.double(), own[s].double()])
            z = turn(q[s], start + n, 1).to(bf16).double() @ v.t() / math.sqrt(DH)
            p = torch.softmax(torch.cat([z, w["sinks"].double()[:, None]], -1), -1)[:, :-1]
            want = turn(p @ v, start + n, -1)
            worst = max(worst, ((out[s].double() - want).abs().max() / want.abs().max()).item())
    if layer.status():
        raise RuntimeError(f"device status {layer.status():#x}")
    say(f"{batch} sequences behind {prefix} shared pooled rows, {steps} tokens each: median step {sorted(spent)[len(spent) // 2]:.0f} us, "
        f"largest error {worst:.2%} of the largest output")
    return worst


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("batch", 64), ("prefix", 8192), ("hidden", 4096), ("steps", 16)):
        ap.add_argument(f"--{name}", type=int, default=value)
    a = ap.parse_args()
    run(a.batch, a.prefix, a.hidden, a.steps)
