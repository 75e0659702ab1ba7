"""What the operators around the HiSA step are measured on: the residual's addition with the
root-mean-square norm and its 8-bit output, the rotary positions of queries and KV rows, and
the dense combine of a batch whose sequences share one long pooled prefix.

Every case runs either in its plain form (elementary torch operations in f32, angles in f64)
or through libhisa's entry points, on the same inputs; exact() states the same results from
the definitions in f64. Shapes are those of the DeepSeek-V4 workloads of this package
(64 query heads x 512 dims, 64 x 128 for the indexer, 64 trailing rotated dims, rotary base
160000, a sliding window of 128) and generic hidden sizes.
"""
from __future__ import annotations

import math

import torch

own = False

THETA, ORIG_LEN, BETA_FAST, BETA_SLOW = 160000.0, 65536, 32.0, 1.0
EPS = 1e-6
RATIO, WINDOW = 4, 128
TINY = 1e-10                     # the least largest magnitude of an 8-bit group
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
BYTES = {"none": 0, "f32": 4, "bf16": 2, "e4m3": 1}
MOST_BYTES = 800_000_000         # of the largest norm and the largest rotation
MOST_POW2 = 32768                # power-of-two scales of a drawn case: few enough that none sits on a border
MOST_ROWS = 304 * 16384          # query rows x prefix rows of the largest combine


# ------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------
def _norm(name, rows, cols, x="bf16", res="bf16", out="bf16", group=0, pow2=False):
    c = dict(op="norm", rows=rows, cols=cols, x=x, res=res, out=out, group=group, pow2=pow2)
    return dict(name=name, **c) if name else c


def _rope(name, tokens, heads, heads2, D, dims, first, half=False, src="bf16", dst="bf16", inplace=False,
          inverse=False, scaling="none", factor=1.0, start=0, spread=False):
    c = dict(op="rope", tokens=tokens, heads=heads, heads2=heads2, D=D, dims=dims, first=first, half=half,
             src=src, dst=dst, inplace=inplace, inverse=inverse, scaling=scaling, factor=factor, start=start,
             spread=spread)
    return dict(name=name, **c) if name else c


def _prefix(name, B, L, H, Dh, P, own_rows, dtype="bf16"):
    c = dict(op="prefix", B=B, L=L, H=H, Dh=Dh, P=P, own_rows=own_rows, dtype=dtype)
    return dict(name=name, **c) if name else c


def listed():
    return [
        # one token of one user: nothing but the latency of a call
        _norm("norm_one_token", 1, 4096),
        # a decode batch ahead of an 8-bit projection: power-of-two scales of 128 columns
        _norm("norm_decode_8bit", 304, 7168, out="e4m3", group=128, pow2=True),
        # a prompt's chunk ahead of an 8-bit projection, the largest
        _norm("norm_prompt_8bit", 16384, 7168, out="e4m3", group=128),
        # f32 rows of an odd length, no residual: no wide access fits every row
        _norm("norm_odd_f32", 1001, 5003, x="f32", res="none", out="f32"),
        # one speculative step of one user: query heads and the KV row, in place
        _rope("rope_one_token", 1, 64, 1, 512, 64, 448, inplace=True, start=61440),
        # a decode batch at far positions, in place: only the rotated tail moves
        _rope("rope_decode_tail", 304, 64, 1, 512, 64, 448, inplace=True, start=1 << 20, spread=True),
        # a prompt's queries as the projection leaves them (f32) to roped bf16, the largest
        _rope("rope_prompt_f32", 4096, 64, 1, 512, 64, 448, src="f32", start=61440),
        # indexer queries in the half layout, stretched to 16 times the trained length
        _rope("rope_half_yarn", 2047, 64, 0, 128, 64, 64, half=True, scaling="yarn", factor=16.0, start=1000000),
        # a few users on a short prefix, two tokens each (a speculative pair)
        _prefix("prefix_small", 3, 2, 64, 512, 1000, 100),
        # a decode batch on an ordinary prompt of odd length
        _prefix("prefix_decode", 64, 1, 64, 512, 8191, 512),
        # a full decode batch on a long document, the largest
        _prefix("prefix_long", 304, 1, 64, 512, 16384, 512),
        # f32 heads of 128 dims
        _prefix("prefix_f32", 7, 3, 16, 128, 1003, 200, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "rope", "prefix"])
    if op == "norm":
        out = rng.choice(["bf16", "e4m3", "f32"])
        group = 0
        if out == "e4m3":
            group = rng.choice([0, 32, 64, 128])
        cols = _log(rng, 64, 16384)
        if group:
            cols = max(group, cols // group * group)
        x, res = rng.choice(["bf16", "f32"]), rng.choice(["none", "bf16", "f32"])
        pow2 = out == "e4m3" and rng.random() < 0.5
        top = min(16384, MOST_BYTES // (cols * (BYTES[x] + 2 * BYTES[res] + BYTES[out])))
        if pow2:
            top = min(top, MOST_POW2 * (group or cols) // cols)
        return _norm(None, _log(rng, 1, top), cols, x=x, res=res, out=out, group=group, pow2=pow2)
    if op == "rope":
        D = rng.choice([64, 128, 512])
        dims = rng.choice([d for d in (32, 64, 128) if d <= D])
        heads, heads2 = rng.choice([(1, 0), (8, 1), (16, 2), (64, 1), (64, 0)])
        src, dst = rng.choice([("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
        tokens = _log(rng, 1, min(16384, MOST_BYTES // ((heads + heads2) * D * (BYTES[src] + BYTES[dst]))))
        scaling = rng.choice(["none", "linear", "yarn"])
        inplace = src == dst and rng.random() < 0.5
        return _rope(None, tokens, heads, heads2, D, dims, rng.choice([0, D - dims]), half=rng.random() < 0.5, src=src,
                     dst=dst, inplace=inplace, inverse=rng.random() < 0.3, scaling=scaling,
                     factor=1.0 if scaling == "none" else rng.choice([4.0, 16.0, 40.0]),
                     start=_log(rng, 1, 1 << 20), spread=rng.random() < 0.5)
    H, Dh, dtype = rng.choice([(64, 512, "bf16"), (64, 512, "bf16"), (64, 512, "bf16"), (16, 128, "bf16"), (16, 128, "f32"),
                               (8, 64, "f32")])
    L = rng.choice([1, 1, 1, 2, 4])
    B = _log(rng, 1, 304 // L)
    top = MOST_ROWS // (B * L)
    if dtype == "f32":
        top //= 64
    return _prefix(None, B, L, H, Dh, _log(rng, 1, max(1, min(65536, top))), rng.choice([0, 60, 512]), dtype=dtype)


# ------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------
def _frequencies(c):
    """Radians per position of the rotated pairs, in f64 (host). Linear scaling divides every
    frequency by the factor. The ramp of "yarn" divides those that turn less than beta_slow
    times over the trained length, keeps those that turn more than beta_fast times, and goes
    over from one to the other linearly in the pair's index."""
    d = c["dims"]
    i = torch.arange(d // 2, dtype=torch.float64)
    f = THETA ** (-2.0 * i / d)
    if c["scaling"] == "linear":
        return f / c["factor"]
    if c["scaling"] == "yarn":
        at = lambda turns: d * math.log(ORIG_LEN / (turns * 2 * math.pi)) / (2 * math.log(THETA))  # noqa: E731
        low, high = max(math.floor(at(BETA_FAST)), 0), min(math.ceil(at(BETA_SLOW)), d - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        return f / c["factor"] * ramp + f * (1 - ramp)
    return f


def _magnitude(c):
    # in place the pairs keep their length, so that a buffer can be rotated again and again
    return 0.1 * math.log(c["factor"]) + 1.0 if c["scaling"] == "yarn" and not c["inplace"] else 1.0


def _inputs(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(shape, dtype, std=1.0, mean=0.0):
        z = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
        return z.mul_(std).add_(mean).to(DT[dtype])

    s = {"case": c}
    if c["op"] == "norm":
        rows, cols = c["rows"], c["cols"]
        s["x"] = normal((rows, cols), c["x"])
        s["w"] = normal((cols,), "f32", 0.1, 1.0)
        if c["res"] != "none":
            r = torch.randn((rows, cols), generator=g, device="cuda")
            loud = torch.randint(0, cols, (max(1, cols // 512),), generator=g, device="cuda")
            r[:, loud] *= 20.0                       # the few loud channels of a residual stream
            s["res"] = r.to(DT[c["res"]])
    elif c["op"] == "rope":
        s["q"] = normal((c["tokens"], c["heads"], c["D"]), c["src"])
        s["k"] = normal((c["tokens"], c["heads2"], c["D"]), c["src"]) if c["heads2"] else None
        if c["spread"]:
            pos = torch.randint(0, c["start"] + 1, (c["tokens"],), generator=g, device="cuda")
        else:
            pos = torch.arange(c["start"], c["start"] + c["tokens"], device="cuda")
        s["pos"] = pos.to(torch.int32)
        s["freq"] = _frequencies(c).cuda()
        s["mscale"] = _magnitude(c)
    else:
        B, L, H, Dh, P = c["B"], c["L"], c["H"], c["Dh"], c["P"]
        W = WINDOW + L - 1
        counts = torch.randint(0, c["own_rows"] + 1, (B,), generator=g, device="cuda") if c["own_rows"] else torch.zeros(
            B, dtype=torch.int64, device="cuda")
        s["off"] = torch.zeros(B + 1, dtype=torch.int64, device="cuda")
        s["off"][1:] = counts.cumsum(0)
        s["q"] = normal((B, L, H, Dh), c["dtype"], 3.0)
        s["local"] = normal((B, W, Dh), c["dtype"])
        s["prefix"] = normal((P, Dh), c["dtype"])
        s["own"] = normal((B * c["own_rows"], Dh), c["dtype"])   # rows allocated: as many as can be there
        s["sinks"] = normal((H,), "f32", 1.0, 9.0)
        # row 0 sits so that the last query row is the token that completed the newest pooled row
        t0 = RATIO * (P + counts) - L
        s["len"] = torch.clamp(t0 + L, 0, W).to(torch.int32)
        s["pos0"] = (t0 + L - s["len"]).to(torch.int32)
        s["t0"] = t0.to(torch.int32)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    c = case
    if own:
        from deepseek_sparse_attention_hisa_gb300 import binding as hb
        code = {"none": hb.HISA_F32, "f32": hb.HISA_F32, "bf16": hb.HISA_BF16, "e4m3": hb.HISA_E4M3}
        if c["op"] == "norm":
            rows, cols = c["rows"], c["cols"]
            s["desc"] = hb.NormDesc(rows=rows, cols=cols, x_dtype=code[c["x"]], res_dtype=code[c["res"]],
                                    out_dtype=code[c["out"]], scale_group=c["group"], scale_pow2=int(c["pow2"]),
                                    eps=EPS, ld_x=cols, ld_res=cols, ld_out=cols)
            s["out"] = torch.empty((rows, cols), device="cuda", dtype=DT[c["out"]])
            s["res_out"] = torch.empty_like(s["res"]) if c["res"] != "none" else None
            s["scales"] = torch.empty((rows, cols // (c["group"] or cols)), device="cuda") if c["out"] == "e4m3" else None
        elif c["op"] == "rope":
            kind = {"none": hb.ROPE_PLAIN, "linear": hb.ROPE_LINEAR, "yarn": hb.ROPE_YARN}[c["scaling"]]
            s["table"] = hb.rope_table(hb.RopeScaling(rope_dims=c["dims"], kind=kind, theta=THETA, factor=c["factor"],
                                                      orig_len=ORIG_LEN, beta_fast=BETA_FAST, beta_slow=BETA_SLOW),
                                       "cuda")
            if c["inplace"]:
                s["yq"], s["yk"] = s["q"], s["k"]
            else:
                s["yq"] = torch.empty(s["q"].shape, device="cuda", dtype=DT[c["dst"]])
                s["yk"] = None if s["k"] is None else torch.empty(s["k"].shape, device="cuda", dtype=DT[c["dst"]])
            s["desc"] = hb.RopeDesc(tokens=c["tokens"], heads=c["heads"], heads2=c["heads2"], D=c["D"],
                                    rope_dims=c["dims"], rope_first=c["first"], half=int(c["half"]),
                                    inverse=int(c["inverse"]), src_dtype=code[c["src"]], dst_dtype=code[c["dst"]],
                                    mscale=s["mscale"], x_token=c["heads"] * c["D"], x_head=c["D"],
                                    y_token=c["heads"] * c["D"], y_head=c["D"], x2_token=c["heads2"] * c["D"],
                                    x2_head=c["D"], y2_token=c["heads2"] * c["D"], y2_head=c["D"])
        else:
            s["desc"] = hb.PrefixDesc(B=c["B"], L=c["L"], H=c["H"], Dh=c["Dh"], window=WINDOW, W_max=s["local"].shape[1],
                                      r=RATIO, prefix_rows=c["P"], Np_max=c["own_rows"], kv_rows=s["own"].shape[0],
                                      scale=0.0, q_dtype=code[c["dtype"]], kv_dtype=code[c["dtype"]],
                                      out_dtype=code[c["dtype"]])
            s["ws"] = hb.alloc_workspace(hb.workspace_bytes(hb.OP_PREFIX_ATTEND, s["desc"]))
            s["out"] = torch.empty((c["B"], c["L"], c["H"], c["Dh"]), device="cuda", dtype=DT[c["dtype"]])
    return s


# ------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------
def _plain_norm(s, c):
    h = s["x"].float()
    got = {}
    if c["res"] != "none":
        h = (s["res"].float() + h).to(DT[c["res"]])      # the norm takes the sum as it is stored
        got["residual"] = h
        h = h.float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["w"]
    if c["out"] != "e4m3":
        got["out"] = y.to(DT[c["out"]])
        return got
    group = c["group"] or c["cols"]
    y = y.view(c["rows"], -1, group)
    scale = y.abs().amax(-1, keepdim=True).clamp_min(TINY) / 448.0
    if c["pow2"]:
        m, e = torch.frexp(scale)                         # the next power of two, itself if it is one
        scale = torch.ldexp(torch.ones_like(scale), e - (m == 0.5).to(e.dtype))
    got["out"] = (y / scale).clamp(-448.0, 448.0).to(DT["e4m3"]).view(c["rows"], c["cols"])
    got["scales"] = scale.view(c["rows"], -1)
    return got


def _plain_rotate(x, c, cos, sin):
    d, first = c["dims"], c["first"]
    z = x[..., first:first + d].float()
    a, b = (z[..., : d // 2], z[..., d // 2:]) if c["half"] else (z[..., 0::2], z[..., 1::2])
    ya, yb = a * cos - b * sin, a * sin + b * cos
    y = torch.cat([ya, yb], -1) if c["half"] else torch.stack([ya, yb], -1).flatten(-2)
    if c["inplace"]:
        x[..., first:first + d] = y.to(x.dtype)
        return x
    return torch.cat([x[..., :first].to(DT[c["dst"]]), y.to(DT[c["dst"]]), x[..., first + d:].to(DT[c["dst"]])], -1)


def _plain_rope(s, c):
    angle = s["pos"].double()[:, None, None] * s["freq"]
    cos = (torch.cos(angle) * s["mscale"]).float()
    sin = (torch.sin(angle) * (-s["mscale"] if c["inverse"] else s["mscale"])).float()
    got = {"q": _plain_rotate(s["q"], c, cos, sin)}
    if s["k"] is not None:
        got["k"] = _plain_rotate(s["k"], c, cos, sin)
    return got


def _plain_prefix(s, c):
    B, L, H, Dh, P = c["B"], c["L"], c["H"], c["Dh"], c["P"]
    q, pre, loc = s["q"].float(), s["prefix"].float(), s["local"].float()
    scale = Dh ** -0.5
    t = s["t0"].long()[:, None] + torch.arange(L, device="cuda")                       # [B, L]
    # the shared rows: one product for all
    sp = (q.view(-1, Dh) @ pre.t()).view(B, L * H, P) * scale
    # the local window
    W = loc.shape[1]
    slot = torch.arange(W, device="cuda")
    at = s["pos0"].long()[:, None] + slot
    gone = t[:, :, None] - at[:, None, :]
    seen = (gone >= 0) & (gone < WINDOW) & (slot < s["len"].long()[:, None])[:, None, :]   # [B, L, W]
    sl = (q.view(B, L * H, Dh) @ loc.transpose(1, 2)).view(B, L, H, W) * scale
    sl = sl.masked_fill(~seen[:, :, None, :], -math.inf).view(B, L * H, W)
    parts = [sp, sl]
    N = c["own_rows"]
    if N:
        # the sequence's own pooled rows, padded to the longest
        count = s["off"][1:] - s["off"][:-1]
        row = torch.arange(N, device="cuda")
        there = row < count[:, None]
        kv = s["own"][(s["off"][:-1, None] + row).clamp_max(s["own"].shape[0] - 1)].float()   # [B, N, Dh]
        there = there[:, None, :].expand(B, L, N)
        if L > 1:
            there = there & (P + row < ((t + 1) // RATIO)[:, :, None])
        so = (q.view(B, L * H, Dh) @ kv.transpose(1, 2)).view(B, L, H, N) * scale
        parts.append(so.masked_fill(~there[:, :, None, :], -math.inf).view(B, L * H, N))
    sink = s["sinks"].repeat(L).view(1, L * H, 1).expand(B, -1, -1)
    top = torch.cat([p.amax(-1, keepdim=True) for p in parts] + [sink], -1).amax(-1, keepdim=True)
    e = [torch.exp(p.sub_(top)) for p in parts]
    norm = torch.exp(sink - top)
    norm = norm + e[0].sum(-1, keepdim=True) + e[1].sum(-1, keepdim=True)
    out = (e[0].view(-1, P) @ pre).view(B, L * H, Dh) + e[1] @ loc
    if N:
        norm = norm + e[2].sum(-1, keepdim=True)
        out = out + e[2] @ kv
    return {"out": (out / norm).view(B, L, H, Dh).to(DT[c["dtype"]])}


def run(state):
    s, c = state, state["case"]
    if own:
        from deepseek_sparse_attention_hisa_gb300 import binding as hb
        if c["op"] == "norm":
            hb.rms_norm(s["desc"], s["x"], s.get("res"), s["w"], s["res_out"], s["out"], s["scales"])
            got = {"out": s["out"]}
            if s["res_out"] is not None:
                got["residual"] = s["res_out"]
            if s["scales"] is not None:
                got["scales"] = s["scales"]
            return got
        if c["op"] == "rope":
            hb.rope(s["desc"], s["table"], s["pos"], s["q"], s["yq"], s["k"], s["yk"])
            return {"q": s["yq"]} if s["yk"] is None else {"q": s["yq"], "k": s["yk"]}
        hb.prefix_attend(s["desc"], s["q"], s["local"], s["len"], s["pos0"], s["prefix"], s["own"], s["off"], s["sinks"],
                         s["t0"], s["out"], s["ws"])
        return {"out": s["out"]}
    if c["op"] == "norm":
        return _plain_norm(s, c)
    if c["op"] == "rope":
        return _plain_rope(s, c)
    return _plain_prefix(s, c)


# ------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "norm":
        n = c["rows"] * c["cols"]
        scales = 4 * (n // (c["group"] or c["cols"])) if c["out"] == "e4m3" else 0
        return {"bytes": n * (BYTES[c["x"]] + 2 * BYTES[c["res"]] + BYTES[c["out"]]) + 4 * c["cols"] + scales, "flops": 6 * n}
    if c["op"] == "rope":
        per = c["tokens"] * (c["heads"] + c["heads2"])
        moved = c["dims"] if c["inplace"] else c["D"]
        return {"bytes": per * moved * (BYTES[c["src"]] + BYTES[c["dst"]]) + 4 * c["tokens"] + 4 * c["dims"],
                "flops": 3 * per * c["dims"]}
    size = BYTES[c["dtype"]]
    rows = c["B"] * c["L"] * c["H"]
    mean = WINDOW + c["own_rows"] / 2
    kv = c["P"] + c["B"] * mean
    return {"bytes": size * c["Dh"] * (2 * rows + kv) + 4 * c["H"], "flops": 4 * rows * (c["P"] + mean) * c["Dh"]}


# ------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------
def exact(case, seed):
    c = case
    s = _inputs(c, seed)
    if c["op"] == "norm":
        h = s["x"].double()
        got = {}
        if c["res"] != "none":
            h = h + s["res"].double()
            got["residual"] = h
            if c["res"] == "bf16":
                h = h.to(torch.float32).to(torch.bfloat16).double()     # the operator norms the stored sum
        y = h / torch.sqrt(torch.linalg.vector_norm(h, dim=-1, keepdim=True).square() / c["cols"] + EPS) * s["w"].double()
        if c["out"] != "e4m3":
            got["out"] = y
            return got
        y = y.unflatten(-1, (-1, c["group"] or c["cols"]))
        scale = torch.maximum(y.max(-1).values, -y.min(-1).values).clamp_min(TINY) / 448
        if c["pow2"]:
            scale = torch.exp2(torch.ceil(torch.log2(scale)))
        got["out"] = (y / scale[..., None]).flatten(-2)
        got["scales"] = scale
        return got
    if c["op"] == "rope":
        turn = torch.polar(torch.full_like(s["freq"], s["mscale"]).expand(c["tokens"], -1).contiguous(),
                           torch.outer(s["pos"].double(), -s["freq"] if c["inverse"] else s["freq"]))[:, None, :]

        def rotated(x):
            y = x.double().clone()
            z = y[..., c["first"]:c["first"] + c["dims"]]
            pairs = z.unflatten(-1, (2, -1)).transpose(-1, -2) if c["half"] else z.unflatten(-1, (-1, 2))
            w = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
            z.copy_((w.transpose(-1, -2) if c["half"] else w).flatten(-2))
            return y

        return {"q": rotated(s["q"])} if s["k"] is None else {"q": rotated(s["q"]), "k": rotated(s["k"])}
    B, L, H, Dh, P = c["B"], c["L"], c["H"], c["Dh"], c["P"]
    off, t0, n, p0 = s["off"].tolist(), s["t0"].tolist(), s["len"].tolist(), s["pos0"].tolist()
    pre = s["prefix"].double()
    out = torch.empty((B, L, H, Dh), device="cuda", dtype=torch.float64)
    for b in range(B):
        for j in range(L):
            t = t0[b] + j
            lo, hi = max(0, t - WINDOW + 1 - p0[b]), min(n[b], t - p0[b] + 1)
            mine = off[b + 1] - off[b]
            if L > 1:
                mine = max(0, min(mine, (t + 1) // RATIO - P))
            rows = torch.cat([s["local"][b, lo:max(hi, lo)].double(), pre, s["own"][off[b]:off[b] + mine].double()])
            z = torch.cat([s["q"][b, j].double() @ rows.t() / math.sqrt(Dh), s["sinks"].double()[:, None]], -1)
            out[b, j] = torch.softmax(z, -1)[:, :-1] @ rows
    return {"out": out}
