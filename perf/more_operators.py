"""What the operators of a paged KV cache are measured on: the norms of query and key heads with
the position rotation in the same pass, rows appended to pages (normed, rotated and held in bf16 or
in 4 bits), rows read back out of them, and the combine over a cache of pages.

Every case runs either in its plain form (elementary torch operations in f32, angles in f64)
or through libhisa's entry points, on the same inputs; exact() states the same results from
the definitions in f64. Shapes are those of the DeepSeek-V4 workloads of this package
(64 query heads x 512 dims, 64 x 128 for the indexer, 64 trailing rotated dims, rotary base
160000, a sliding window of 128, 512 selected rows) and generic ones.

Rows in 4 bits: sixteen neighbouring dims share a scale s of type e4m3, and a dim holds a value c of
{0, 0.5, 1, 1.5, 2, 3, 4, 6} with a sign, two to a byte, the even dim low; the row is c * s * g with one
factor g for the cache.
"""
from __future__ import annotations

import math

import torch

own = False

THETA, ORIG_LEN, BETA_FAST, BETA_SLOW = 160000.0, 65536, 32.0, 1.0
EPS = 1e-6
RATIO, WINDOW = 4, 128
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}
GROUP = 16
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
MOST_BYTES = 800_000_000         # of the largest heads
MOST_ROWS = 65536                # of the largest append and read
MOST_SEEN = 64 * 16384           # query rows x rows seen of the largest combine


# ------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------
def _heads(name, tokens, heads, heads2, D, dims, half=False, src="bf16", dst="bf16", weights=True, factor=1.0, start=0):
    c = dict(op="heads", tokens=tokens, heads=heads, heads2=heads2, D=D, dims=dims, half=half, src=src, dst=dst,
             weights=weights, factor=factor, start=start)
    return dict(name=name, **c) if name else c


def _append(name, B, new, old, D, dims, page, cache="4bit", src="bf16", half=False, norm=True, even=False):
    c = dict(op="append", B=B, new=new, old=old, D=D, dims=dims, page=page, cache=cache, src=src, half=half, norm=norm,
             even=even)
    return dict(name=name, **c) if name else c


def _read(name, B, rows, D, page, cache="4bit", dst="bf16", even=False):
    c = dict(op="read", B=B, rows=rows, D=D, page=page, cache=cache, dst=dst, even=even)
    return dict(name=name, **c) if name else c


def _attend(name, B, L, H, Dh, rows, page, select=0, cache="4bit", q="bf16", dst="bf16", window=WINDOW, sinks=True):
    c = dict(op="attend", B=B, L=L, H=H, Dh=Dh, rows=rows, page=page, select=select, cache=cache, q=q, dst=dst,
             window=window, sinks=sinks)
    return dict(name=name, **c) if name else c


def listed():
    return [
        # one token of one user: nothing but the latency of a call
        _heads("heads_one_token", 1, 64, 1, 512, 64, start=61440),
        # a prompt's queries and KV rows as the projections leave them (f32), the largest
        _heads("heads_prompt_f32", 4096, 64, 1, 512, 64, src="f32", start=61440),
        # indexer queries in the half layout, stretched to 16 times the trained length, no weights
        _heads("heads_half_yarn", 2047, 64, 0, 128, 64, half=True, weights=False, factor=16.0, start=1000000),
        # a decode batch: one row for each sequence, and its pages read back
        _append("append_decode", 304, 1, 15, 512, 64, 16, even=True),
        # prompts of different lengths in one call, the largest, and their pages read back
        _append("append_prompts", 5, 13107, 0, 512, 64, 64),
        # f32 rows of 128 dims in bf16 pages of an odd size, behind rows that are there already
        _append("append_bf16_odd", 33, 601, 300, 128, 64, 48, cache="bf16", src="f32", half=True),
        # one prompt's rows as a contiguous prefix for others to share
        _read("read_prefix", 1, 8191, 512, 64, even=True),
        # many sequences moved out of their pages in f32, the largest
        _read("read_many_f32", 37, 3542, 512, 64, dst="f32"),
        # one user on a long dense cache: the split over a long axis
        _attend("attend_one_long", 1, 1, 64, 512, 20001, 64),
        # a full decode batch with 512 selected rows each
        _attend("attend_selected", 304, 1, 64, 512, 4096, 64, select=512),
        # a decode batch over all rows of its caches, the largest
        _attend("attend_dense", 64, 1, 64, 512, 16384, 64),
        # a few speculative tokens over f32 heads of 128 dims, bf16 pages
        _attend("attend_verify_f32", 7, 3, 16, 128, 1003, 48, cache="bf16", q="f32", dst="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["heads", "append", "read", "attend", "attend"])
    page = rng.choice([1, 16, 48, 64, 100, 256])
    if op == "heads":
        D = rng.choice([64, 128, 192, 512])
        dims = rng.choice([d for d in (0, 32, 64, 128) if d <= D])
        heads, heads2 = rng.choice([(1, 0), (8, 1), (16, 2), (24, 8), (64, 1), (64, 0)])
        src, dst = rng.choice([("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
        top = min(16384, MOST_BYTES // ((heads + heads2) * D * (BYTES[src] + BYTES[dst])))
        return _heads(None, _log(rng, 1, top), heads, heads2, D, dims, half=rng.random() < 0.5, src=src, dst=dst,
                      weights=rng.random() < 0.7, factor=rng.choice([1.0, 1.0, 16.0]), start=_log(rng, 1, 1 << 20))
    cache = rng.choice(["4bit", "4bit", "bf16"])
    if op == "append":
        D = rng.choice([64, 128, 512])
        B = _log(rng, 1, 304)
        page = max(page, 16)
        return _append(None, B, _log(rng, 1, MOST_ROWS // B), rng.choice([0, 15, 300]) if B < 100 else 15, D,
                       rng.choice([d for d in (0, 32, 64) if d <= D]), page, cache=cache, src=rng.choice(["bf16", "f32"]),
                       half=rng.random() < 0.5, norm=rng.random() < 0.5, even=rng.random() < 0.3)
    if op == "read":
        B = _log(rng, 1, 304)
        return _read(None, B, _log(rng, 1, MOST_ROWS // B), rng.choice([64, 128, 512]), page, cache=cache,
                     dst=rng.choice(["bf16", "f32"]), even=rng.random() < 0.3)
    H, Dh, q, dst = rng.choice([(64, 512, "bf16", "bf16"), (64, 512, "bf16", "bf16"), (64, 512, "bf16", "f32"),
                                (16, 128, "bf16", "bf16"), (16, 128, "f32", "f32"), (8, 64, "f32", "f32")])
    L = rng.choice([1, 1, 1, 2, 4])
    B = _log(rng, 1, 304 // L)
    rows = _log(rng, 1, max(1, min(65536, MOST_SEEN // (B * L * (1 if Dh == 512 else 4)))))
    select = rng.choice([0, 0, 64, 512]) if rows > 64 else 0
    return _attend(None, B, L, H, Dh, rows, page, select=select, cache=cache, q=q, dst=dst,
                   window=rng.choice([WINDOW, WINDOW, 0]), sinks=rng.random() < 0.8)


# ------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------
def _frequencies(dims, factor):
    """Radians per position of the rotated pairs, in f64 (host). A factor above 1 stretches: it
    divides the pairs that turn less than beta_slow times over the trained length, keeps those that
    turn more than beta_fast times, and goes over linearly in the pair's index between them."""
    i = torch.arange(dims // 2, dtype=torch.float64)
    f = THETA ** (-2.0 * i / max(dims, 1))
    if factor > 1:
        at = lambda turns: dims * math.log(ORIG_LEN / (turns * 2 * math.pi)) / (2 * math.log(THETA))  # noqa: E731
        low, high = max(math.floor(at(BETA_FAST)), 0), min(math.ceil(at(BETA_SLOW)), dims - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        return f / factor * ramp + f * (1 - ramp)
    return f


def _pool(g, pages, page, D, cache):
    """Pages that hold rows of N(0, 1), in 4 bits as the quantiser leaves such rows: the group's
    largest magnitude near 1.8, so a scale near 0.3."""
    if cache == "bf16":
        return torch.randn((pages, page, D), generator=g, device="cuda").to(torch.bfloat16), None
    scales = (torch.rand((pages, page, D // GROUP), generator=g, device="cuda") * 0.2 + 0.2).to(torch.float8_e4m3fn)
    edge = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64) * 0.3
    quantile = torch.special.ndtri((torch.arange(256, dtype=torch.float64) + 0.5) / 256)
    nibble = torch.bucketize(quantile.abs(), edge) | torch.where(quantile < 0, 8, 0)
    pair = (nibble[:, None] * 16 + nibble[None, :]).flatten().to(torch.uint8).cuda()
    n = pages * page * D // 2
    codes = torch.empty(n, dtype=torch.uint8, device="cuda")
    for at in range(0, n, 1 << 28):
        m = min(1 << 28, n - at)
        codes[at:at + m] = pair[torch.randint(0, 65536, (m,), generator=g, device="cuda")]
    return codes.view(pages, page, D // 2), scales


def _tables(g, counts, most, page):
    """Page numbers of each sequence's rows, in no order; -1 where it has no rows."""
    B, cols = counts.numel(), -(-most // page)
    table = torch.randperm(B * cols, generator=g, device="cuda").view(B, cols)
    there = torch.arange(cols, device="cuda") * page < counts[:, None]
    return torch.where(there, table, -1).to(torch.int32), B * cols


def _inputs(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(shape, dtype, std=1.0, mean=0.0):
        z = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
        return z.mul_(std).add_(mean).to(DT[dtype])

    def some(hi, n):                 # up to hi each, the first one hi
        v = torch.randint(0, hi + 1, (n,), generator=g, device="cuda")
        v[0] = hi
        return v

    s = {"case": c}
    if c["op"] == "heads":
        s["q"] = normal((c["tokens"], c["heads"], c["D"]), c["src"], 2.0)
        s["k"] = normal((c["tokens"], c["heads2"], c["D"]), c["src"], 2.0) if c["heads2"] else None
        s["wq"] = normal((c["D"],), "f32", 0.1, 1.0) if c["weights"] else None
        s["wk"] = normal((c["D"],), "f32", 0.1, 1.0) if c["weights"] and c["heads2"] else None
        s["pos"] = torch.arange(c["start"], c["start"] + c["tokens"], device="cuda").to(torch.int32)
        s["freq"] = _frequencies(c["dims"], c["factor"]).cuda()
        s["mscale"] = 0.1 * math.log(c["factor"]) + 1.0
    elif c["op"] == "append":
        B, D = c["B"], c["D"]
        new = torch.full((B,), c["new"], device="cuda") if c["even"] else some(c["new"], B)
        s["first"] = some(c["old"], B).to(torch.int32)
        s["off"] = torch.zeros(B + 1, dtype=torch.int64, device="cuda")
        s["off"][1:] = new.cumsum(0)
        s["x"] = normal((B * c["new"], D), c["src"], 2.0 if c["norm"] else 1.0)
        s["w"] = normal((D,), "f32", 0.1, 1.0) if c["norm"] else None
        s["table"], pages = _tables(g, s["first"] + new, c["old"] + c["new"], c["page"])
        s["cache"], s["scales"] = _pool(g, pages, c["page"], D, c["cache"])
        s["freq"] = _frequencies(c["dims"], 1.0).cuda()
        s["g"] = 0.75
    elif c["op"] == "read":
        count = torch.full((c["B"],), c["rows"], device="cuda") if c["even"] else some(c["rows"], c["B"])
        s["off"] = torch.zeros(c["B"] + 1, dtype=torch.int64, device="cuda")
        s["off"][1:] = count.cumsum(0)
        s["first"] = torch.zeros(c["B"], dtype=torch.int32, device="cuda")
        s["table"], pages = _tables(g, count, c["rows"], c["page"])
        s["cache"], s["scales"] = _pool(g, pages, c["page"], c["D"], c["cache"])
        s["out"] = torch.zeros((c["B"] * c["rows"], c["D"]), device="cuda", dtype=DT[c["dst"]])
        s["g"] = 0.75
    else:
        B, L, H, Dh = c["B"], c["L"], c["H"], c["Dh"]
        W = c["window"] + L - 1 if c["window"] else 0
        count = some(c["rows"], B)
        s["count"] = count.to(torch.int32)
        s["table"], pages = _tables(g, count, c["rows"], c["page"])
        s["cache"], s["scales"] = _pool(g, pages, c["page"], Dh, c["cache"])
        s["q"] = normal((B, L, H, Dh), c["q"], 3.0)
        s["local"] = normal((B, W, Dh), c["q"])
        s["sinks"] = normal((H,), "f32", 1.0, 9.0) if c["sinks"] else None
        # row 0 sits so that the last query row is the token that completed the newest row
        t0 = RATIO * count - L
        s["len"] = torch.clamp(t0 + L, 0, W).to(torch.int32)
        s["pos0"] = (t0 + L - s["len"]).to(torch.int32)
        s["t0"] = t0.to(torch.int32)
        s["I"] = None
        if c["select"]:
            k = c["select"]
            order = torch.rand((B, L, max(c["rows"], k)), generator=g, device="cuda")
            order.masked_fill_(torch.arange(order.shape[-1], device="cuda") >= count[:, None, None], 2.0)
            val, idx = order.topk(k, -1, largest=False)
            idx = idx.masked_fill(val > 1.5, 1 << 30).sort(-1).values
            s["I"] = torch.where(idx < 1 << 30, idx, -1).to(torch.int32)
        s["g"] = 1.0
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    c = case
    if own:
        from deepseek_sparse_attention_hisa_gb300 import binding as hb
        code = {"f32": hb.HISA_F32, "bf16": hb.HISA_BF16, "4bit": hb.HISA_E2M1}
        if c["op"] in ("heads", "append"):
            yarn = c["op"] == "heads" and c["factor"] > 1
            s["turns"] = None if not c["dims"] else hb.rope_table(
                hb.RopeScaling(rope_dims=c["dims"], kind=hb.ROPE_YARN if yarn else hb.ROPE_PLAIN, theta=THETA,
                               factor=c["factor"] if yarn else 1.0, orig_len=ORIG_LEN, beta_fast=BETA_FAST,
                               beta_slow=BETA_SLOW), "cuda")
        if c["op"] == "heads":
            D = c["D"]
            s["yq"] = torch.empty(s["q"].shape, device="cuda", dtype=DT[c["dst"]])
            s["yk"] = None if s["k"] is None else torch.empty(s["k"].shape, device="cuda", dtype=DT[c["dst"]])
            s["desc"] = hb.NormRopeDesc(tokens=c["tokens"], heads=c["heads"], heads2=c["heads2"], D=D, norm=1,
                                        norm2=int(c["heads2"] > 0), rope_dims=c["dims"], rope_first=D - c["dims"],
                                        half=int(c["half"]), src_dtype=code[c["src"]], dst_dtype=code[c["dst"]],
                                        eps=EPS, mscale=s["mscale"], x_token=c["heads"] * D, x_head=D,
                                        y_token=c["heads"] * D, y_head=D, x2_token=c["heads2"] * D, x2_head=D,
                                        y2_token=c["heads2"] * D, y2_head=D)
        elif c["op"] == "append":
            pages, D = s["cache"].shape[0], c["D"]
            form = dict(pages=pages, page_rows=c["page"], D=D, cache_dtype=code[c["cache"]], cache_scale=s["g"], ld=D)
            s["desc"] = hb.CacheDesc(B=c["B"], table_cols=s["table"].shape[1], rows=s["x"].shape[0],
                                     io_dtype=code[c["src"]], norm=int(c["norm"]), eps=EPS, rope_dims=c["dims"],
                                     rope_first=D - c["dims"], half=int(c["half"]), r=RATIO, mscale=1.0, **form)
            s["ws"] = hb.alloc_workspace(hb.workspace_bytes(hb.OP_CACHE, s["desc"]))
            if c["cache"] == "4bit":                  # all pages in their order, as one sequence
                n = pages * c["page"]
                s["all"] = hb.CacheDesc(B=1, table_cols=pages, rows=n, io_dtype=hb.HISA_E4M3, **form)
                s["all_off"] = torch.tensor([0, n], device="cuda")
                s["all_first"] = torch.zeros(1, device="cuda", dtype=torch.int32)
                s["all_table"] = torch.arange(pages, device="cuda", dtype=torch.int32)
                s["codes"] = torch.empty((pages, c["page"], D), device="cuda", dtype=torch.float8_e4m3fn)
        elif c["op"] == "read":
            s["desc"] = hb.CacheDesc(pages=s["cache"].shape[0], page_rows=c["page"], D=c["D"], cache_dtype=code[c["cache"]],
                                     cache_scale=s["g"], B=c["B"], table_cols=s["table"].shape[1], rows=s["out"].shape[0],
                                     io_dtype=code[c["dst"]], ld=c["D"])
            s["ws"] = hb.alloc_workspace(hb.workspace_bytes(hb.OP_CACHE, s["desc"]))
        else:
            s["desc"] = hb.CacheAttnDesc(B=c["B"], L=c["L"], H=c["H"], Dh=c["Dh"], window=c["window"],
                                         W_max=s["local"].shape[1], r=RATIO, k=c["select"], page_rows=c["page"],
                                         table_cols=s["table"].shape[1], pages=s["cache"].shape[0], Np_max=c["rows"],
                                         scale=0.0, cache_scale=s["g"], q_dtype=code[c["q"]],
                                         cache_dtype=code[c["cache"]], out_dtype=code[c["dst"]])
            s["ws"] = hb.alloc_workspace(hb.workspace_bytes(hb.OP_CACHE_ATTEND, s["desc"]))
            s["out"] = torch.empty(s["q"].shape, device="cuda", dtype=DT[c["dst"]])
    return s


# ------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------
def _plain_norm(x, w):
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return y if w is None else y * w


def _plain_rotate(x, first, half, cos, sin):
    d = 2 * cos.shape[-1]
    if d == 0:
        return x
    z = x[..., first:first + d]
    a, b = (z[..., : d // 2], z[..., d // 2:]) if half else (z[..., 0::2], z[..., 1::2])
    ya, yb = a * cos - b * sin, a * sin + b * cos
    y = torch.cat([ya, yb], -1) if half else torch.stack([ya, yb], -1).flatten(-2)
    return torch.cat([x[..., :first], y, x[..., first + d:]], -1)


def _plain_heads(s, c):
    angle = s["pos"].double()[:, None, None] * s["freq"]
    cos, sin = ((f(angle) * s["mscale"]).float() for f in (torch.cos, torch.sin))
    first = c["D"] - c["dims"]
    got = {"q": _plain_rotate(_plain_norm(s["q"].float(), s["wq"]), first, c["half"], cos, sin).to(DT[c["dst"]])}
    if s["k"] is not None:
        got["k"] = _plain_rotate(_plain_norm(s["k"].float(), s["wk"]), first, c["half"], cos, sin).to(DT[c["dst"]])
    return got


def _grid():
    return torch.tensor(GRID + [-v for v in GRID], device="cuda")


def _slots(table, seq, p, page):
    """The row in the pool of row p of sequence seq."""
    return table[seq, p // page].long() * page + p % page


def _packed(off, first, n):
    """The sequence and the row in it of the first off[-1] of n packed rows; the others are padding."""
    row = torch.arange(n, device="cuda")
    seq = torch.searchsorted(off, row, right=True) - 1
    there = seq < off.numel() - 1
    seq, row = seq[there], row[there]
    return row, seq, first[seq].long() + row - off[seq]


def _plain_rows(s, slot, cache, D):
    """Rows of the pool by their place in it, f32."""
    if cache == "bf16":
        return s["cache"].view(-1, D)[slot].float()
    codes = s["cache"].view(-1, D // 2)[slot]
    grid = _grid()
    c = torch.stack([grid[(codes & 15).long()], grid[(codes >> 4).long()]], -1).flatten(-2)
    scale = s["scales"].view(torch.uint8).view(-1, D // GROUP)[slot].view(torch.float8_e4m3fn).float() * s["g"]
    return (c.unflatten(-1, (-1, GROUP)) * scale[..., None]).flatten(-2)


def _plain_append(s, c):
    D = c["D"]
    row, seq, p = _packed(s["off"], s["first"], s["x"].shape[0])
    angle = (p * RATIO).double()[:, None] * s["freq"]
    x = s["x"][row].float()
    if c["norm"]:
        x = _plain_norm(x, s["w"])
    y = _plain_rotate(x, D - c["dims"], c["half"], torch.cos(angle).float(), torch.sin(angle).float())
    slot = _slots(s["table"], seq, p, c["page"])
    if c["cache"] == "bf16":
        s["cache"].view(-1, D)[slot] = y.to(torch.bfloat16)
        return {"cache": s["cache"]}
    y = y.unflatten(-1, (-1, GROUP))
    top = y.abs().amax(-1)
    scale = (top / torch.full_like(top, 6.0 * s["g"])).clamp_max(448.0).to(torch.float8_e4m3fn)     # a quotient, not a product by 1 / 6g
    step = scale.float()[..., None] * s["g"]
    v = torch.where(step > 0, y / step, 0.0)
    a = v.abs()
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
            + (a >= 3.5).int() + (a > 5.0).int() + torch.signbit(v).int() * 8).flatten(-2)
    s["cache"].view(-1, D // 2)[slot] = (code[:, 0::2] + code[:, 1::2] * 16).to(torch.uint8)
    s["scales"].view(torch.uint8).view(-1, D // GROUP)[slot] = scale.view(torch.uint8)
    grid = _grid()
    codes = torch.stack([grid[(s["cache"] & 15).long()], grid[(s["cache"] >> 4).long()]], -1).flatten(-2)
    return {"codes": codes.to(torch.float8_e4m3fn), "scales": s["scales"]}


def _plain_read(s, c):
    row, seq, p = _packed(s["off"], s["first"], s["out"].shape[0])
    s["out"][row] = _plain_rows(s, _slots(s["table"], seq, p, c["page"]), c["cache"], c["D"]).to(DT[c["dst"]])
    return {"out": s["out"]}


def _plain_attend(s, c):
    B, L, H, Dh = c["B"], c["L"], c["H"], c["Dh"]
    q, loc = s["q"].float(), s["local"].float()
    count, W = s["count"].long(), loc.shape[1]
    t = s["t0"].long()[:, None] + torch.arange(L, device="cuda")                            # [B, L]
    b = torch.arange(B, device="cuda")[:, None, None]
    seen = torch.minimum((t + 1) // RATIO, count[:, None]) if L > 1 else count[:, None]     # rows before this one are seen
    parts, values = [], []
    if c["select"]:
        ids = s["I"].long()                                                                 # [B, L, k]
        there = (ids >= 0) & (ids < seen[:, :, None])
        ids = ids.clamp_min(0)
        kv = _plain_rows(s, _slots(s["table"], b, ids, c["page"]).clamp_min(0), c["cache"], Dh)     # [B, L, k, Dh]
        z = q @ kv.transpose(-1, -2)
        there = there[:, :, None, :]
    else:
        p = torch.arange(c["rows"], device="cuda")
        kv = _plain_rows(s, _slots(s["table"], b[:, 0], p[None], c["page"]).clamp_min(0), c["cache"], Dh)   # [B, N, Dh]
        there = (p < seen[:, :, None])[:, :, None, :]
        z = (q.view(B, L * H, Dh) @ kv.transpose(1, 2)).view(B, L, H, -1)
    parts.append((z * Dh ** -0.5).masked_fill(~there, -math.inf))
    values.append(kv)
    if W:
        slot = torch.arange(W, device="cuda")
        gone = t[:, :, None] - (s["pos0"].long()[:, None] + slot)[:, None, :]
        near = (gone >= 0) & (gone < c["window"]) & (slot < s["len"].long()[:, None])[:, None, :]    # [B, L, W]
        z = (q.view(B, L * H, Dh) @ loc.transpose(1, 2)).view(B, L, H, W) * Dh ** -0.5
        parts.append(z.masked_fill(~near[:, :, None, :], -math.inf))
        values.append(loc)
    top = torch.cat([z.amax(-1, keepdim=True) for z in parts], -1).amax(-1, keepdim=True)
    sink = s["sinks"].view(H, 1) if c["sinks"] else None
    if c["sinks"]:
        top = torch.maximum(top, sink)
    top = torch.where(top == -math.inf, 0.0, top)
    norm = torch.exp(sink - top) if c["sinks"] else 0.0
    out = 0.0
    for z, kv in zip(parts, values):
        e = torch.exp(z.sub_(top))
        norm = norm + e.sum(-1, keepdim=True)
        out = out + (e @ kv if kv.dim() == 4 else (e.view(B, L * H, -1) @ kv).view(B, L, H, Dh))
    return {"out": torch.where(norm > 0, out / norm, 0.0).to(DT[c["dst"]])}


def run(state):
    s, c = state, state["case"]
    if own:
        from deepseek_sparse_attention_hisa_gb300 import binding as hb
        if c["op"] == "heads":
            hb.norm_rope(s["desc"], s["turns"], s["pos"], s["q"], s["wq"], s["yq"], s["k"], s["wk"], s["yk"])
            return {"q": s["yq"]} if s["yk"] is None else {"q": s["yq"], "k": s["yk"]}
        if c["op"] == "append":
            hb.cache_append(s["desc"], s["turns"], s["x"], s["w"], s["off"], s["first"], s["table"], s["cache"], s["scales"],
                            s["ws"])
            if c["cache"] == "bf16":
                return {"cache": s["cache"]}
            hb.cache_read(s["all"], s["all_off"], s["all_first"], s["all_table"], s["cache"], s["scales"], s["codes"], s["ws"])
            return {"codes": s["codes"], "scales": s["scales"]}
        if c["op"] == "read":
            hb.cache_read(s["desc"], s["off"], s["first"], s["table"], s["cache"], s["scales"], s["out"], s["ws"])
            return {"out": s["out"]}
        hb.cache_attend(s["desc"], s["q"], s["local"], s["len"], s["pos0"], s["cache"], s["scales"], s["table"], s["count"],
                        s["I"], s["sinks"], s["t0"], s["out"], s["ws"])
        return {"out": s["out"]}
    return {"heads": _plain_heads, "append": _plain_append, "read": _plain_read, "attend": _plain_attend}[c["op"]](s, c)


# ------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------
def _mean(c, n):
    """Of as many as n in each sequence, n in the first."""
    return n if c.get("even") else n * (c["B"] + 1) / (2 * c["B"])


def _row_bytes(D, cache):
    return 2 * D if cache == "bf16" else D // 2 + D // GROUP


def work(case):
    c = case
    if c["op"] == "heads":
        n = c["tokens"] * (c["heads"] + c["heads2"])
        return {"bytes": n * c["D"] * (BYTES[c["src"]] + BYTES[c["dst"]]) + 4 * c["tokens"],
                "flops": n * (4 * c["D"] + 3 * c["dims"])}
    if c["op"] == "append":
        n = c["B"] * _mean(c, c["new"])
        size = n * (c["D"] * BYTES[c["src"]] + _row_bytes(c["D"], c["cache"]))
        if c["cache"] == "4bit":                       # the codes of all pages, read back in 8 bits
            size += c["B"] * -(-(c["old"] + c["new"]) // c["page"]) * c["page"] * (c["D"] // 2 + c["D"])
        return {"bytes": size, "flops": n * (6 * c["D"] + 3 * c["dims"])}
    if c["op"] == "read":
        n = c["B"] * _mean(c, c["rows"])
        return {"bytes": n * (_row_bytes(c["D"], c["cache"]) + c["D"] * BYTES[c["dst"]]), "flops": n * c["D"]}
    rows = c["B"] * c["L"]
    mean = _mean(c, c["rows"])
    if c["select"]:
        seen = min(mean, c["select"])
        held = rows * seen
    else:
        seen, held = mean, c["B"] * mean
    size = rows * c["H"] * c["Dh"] * (BYTES[c["q"]] + BYTES[c["dst"]]) + held * _row_bytes(c["Dh"], c["cache"])
    size += c["B"] * c["window"] * c["Dh"] * BYTES[c["q"]]
    return {"bytes": size, "flops": 4 * rows * c["H"] * (seen + c["window"]) * c["Dh"]}


# ------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------
def _exact_turned(x, w, norm, pos, freq, mscale, first, half):
    """x [n, heads, D] in 64 bits: the norm of each head, then its pairs as complex numbers turned."""
    y = x.double()
    if norm:
        y = y / torch.sqrt(torch.linalg.vector_norm(y, dim=-1, keepdim=True).square() / y.shape[-1] + EPS)
        y = y if w is None else y * w.double()
    y = y.clone()
    d = 2 * freq.numel()
    if d:
        turn = torch.polar(torch.full_like(freq, mscale).expand(pos.numel(), -1).contiguous(),
                           torch.outer(pos.double(), freq))[:, None, :]
        z = y[..., first:first + d]
        pairs = z.unflatten(-1, (2, -1)).transpose(-1, -2) if half else z.unflatten(-1, (-1, 2))
        v = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        z.copy_((v.transpose(-1, -2) if half else v).flatten(-2))
    return y


def _nearest(v, low, bits, most):
    """v >= 0 to the nearest float of `bits` bits after the leading one and a least exponent `low`."""
    e = torch.frexp(v.clamp_min(2.0 ** low))[1] - 1
    step = torch.ldexp(torch.ones_like(v), e - bits)
    return (torch.round(v / step) * step).clamp_max(most)


def _exact_values(codes, D):
    """The values that packed codes stand for, by the bits of a float of one bit after the leading one."""
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).to(torch.int32)
    e, m = (n >> 1) & 3, (n & 1).double()
    v = torch.where(e == 0, m / 2, torch.ldexp(1 + m / 2, e - 1))
    return torch.where(n >= 8, -v, v)


def _exact_rows(s, slot, cache, D):
    if cache == "bf16":
        return s["cache"].view(-1, D)[slot].double()
    scale = s["scales"].view(torch.uint8).view(-1, D // GROUP)[slot].view(torch.float8_e4m3fn).double()
    return _exact_values(s["cache"].view(-1, D // 2)[slot], D) * scale.repeat_interleave(GROUP, -1) * s["g"]


def exact(case, seed):
    c = case
    s = _inputs(c, seed)
    if c["op"] == "heads":
        first = c["D"] - c["dims"]
        got = {"q": _exact_turned(s["q"], s["wq"], True, s["pos"], s["freq"], s["mscale"], first, c["half"])}
        if s["k"] is not None:
            got["k"] = _exact_turned(s["k"], s["wk"], True, s["pos"], s["freq"], s["mscale"], first, c["half"])
        return got
    if c["op"] in ("append", "read"):
        D, page = c["D"], c["page"]
        off, first, table = s["off"].tolist(), s["first"].tolist(), s["table"].long()
        places, positions = [], []
        for b in range(c["B"]):
            p = torch.arange(first[b], first[b] + off[b + 1] - off[b], device="cuda")
            places.append(table[b].repeat_interleave(page)[p] * page + p % page)
            positions.append(p * RATIO)
        slot, pos = torch.cat(places), torch.cat(positions)
        if c["op"] == "read":
            out = torch.zeros(s["out"].shape, device="cuda", dtype=torch.float64)
            out[off[0]:off[-1]] = _exact_rows(s, slot, c["cache"], D)
            return {"out": out}
        y = _exact_turned(s["x"][off[0]:off[-1], None], s["w"], c["norm"], pos, s["freq"], 1.0, D - c["dims"], c["half"])[:, 0]
        if c["cache"] == "bf16":
            cache = s["cache"].double()
            cache.view(-1, D)[slot] = y
            return {"cache": cache}
        codes, scales = _exact_values(s["cache"], D), s["scales"].double()
        y = y.unflatten(-1, (-1, GROUP))
        scale = _nearest(torch.maximum(y.amax(-1), -y.amin(-1)) / (6 * s["g"]), -6, 3, 448.0)
        v = y / (scale.where(scale > 0, 1.0) * s["g"])[..., None]
        v = torch.where(scale[..., None] > 0, _nearest(v.abs(), 0, 1, 6.0) * torch.sign(v), 0.0)
        codes.view(-1, D)[slot] = v.flatten(-2)
        scales.view(-1, D // GROUP)[slot] = scale
        return {"codes": codes, "scales": scales}
    B, L, H, Dh, page = c["B"], c["L"], c["H"], c["Dh"], c["page"]
    count, t0, n, p0 = (s[k].tolist() for k in ("count", "t0", "len", "pos0"))
    out = torch.zeros((B, L, H, Dh), device="cuda", dtype=torch.float64)
    for b in range(B):
        for j in range(L):
            t = t0[b] + j
            lo, hi = max(0, t - c["window"] + 1 - p0[b]), min(n[b], t - p0[b] + 1)
            seen = count[b] if L == 1 else max(0, min(count[b], (t + 1) // RATIO))
            if c["select"]:
                p = s["I"][b, j].long()
                p = p[(p >= 0) & (p < seen)]
            else:
                p = torch.arange(seen, device="cuda")
            rows = _exact_rows(s, s["table"][b].long()[p // page] * page + p % page, c["cache"], Dh)
            if c["window"]:
                rows = torch.cat([s["local"][b, lo:max(hi, lo)].double(), rows])
            z = s["q"][b, j].double() @ rows.t() / math.sqrt(Dh)
            if c["sinks"]:
                z = torch.cat([z, s["sinks"].double()[:, None]], -1)
            if z.shape[-1]:
                out[b, j] = torch.softmax(z, -1)[:, :rows.shape[0]] @ rows
    return {"out": out}
