"""The operators around the step against plain 64-bit implementations (GB300).

Tolerances count roundings: half a step of the output type, u = 2^-24 for each f32 operation on
the way, and, where a kernel sums n terms in f32, n u times the sum of the terms' magnitudes.
"""
import math

import pytest

torch = pytest.importorskip("torch")

from deepseek_sparse_attention_hisa_gb300 import binding as hb  # noqa: E402

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

U = 2.0**-24
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
CODE = {"f32": hb.HISA_F32, "bf16": hb.HISA_BF16, "e4m3": hb.HISA_E4M3}
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from deepseek_sparse_attention_hisa_gb300 import build
    build.build_library()
    hb.lib()


def half_step(dt):
    return torch.finfo(DT[dt]).eps / 2


def randn(shape, dt, seed, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(DT[dt])


def strided(rows, cols, dt, ld, off, fill):
    """A [rows, cols] view, rows ld apart, starting off elements into a buffer full of `fill`."""
    buf = torch.empty(off + max(rows, 1) * ld, device="cuda", dtype=torch.float32).fill_(fill).to(DT[dt])
    return buf, buf[off:off + rows * ld].view(rows, ld)[:, :cols]


# ------------------------------------------------------------------------------------
# residual addition, root-mean-square norm, 8-bit output
# ------------------------------------------------------------------------------------
def run_norm(x, res, w, out_dt, group=0, pow2=0, keep=True, out=None, res_out=None, eps=1e-6, stream=None):
    rows, cols = x.shape
    if out is None:
        out = torch.empty((rows, cols), device="cuda", dtype=DT[out_dt])
    if res is not None and keep and res_out is None:
        res_out = torch.empty_strided(res.shape, res.stride(), device="cuda", dtype=res.dtype)
    scales = torch.full((rows, cols // (group or cols)), -7.0, device="cuda") if out_dt == "e4m3" else None
    d = hb.NormDesc(rows=rows, cols=cols, x_dtype=hb.dtype_code(x), res_dtype=hb.dtype_code(res) if res is not None else 0,
                    out_dtype=CODE[out_dt], scale_group=group, scale_pow2=pow2, eps=eps, ld_x=x.stride(0),
                    ld_res=res.stride(0) if res is not None else 0, ld_out=out.stride(0))
    hb.rms_norm(d, x, res, w, res_out if keep else None, out, scales, stream=stream)
    return out, res_out, scales


def check_norm(x, res, w, out_dt, out, res_out, scales, group=0, pow2=0, eps=1e-6):
    """Sums of squares: at most 32 terms per thread in order, 5 + 32 steps over lanes and warps,
    the square and the mean: 71 roundings, halved by the root; the root, the reciprocal and two
    products add 5."""
    cols = x.shape[1]
    h = x.float()
    if res is not None:
        h = (h + res.float()).to(res.dtype)          # one f32 addition, one rounding: the same bits
        if res_out is not None:
            assert torch.equal(h, res_out)
    h = h.double()
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * w.double()
    rel = (71 / 2 + 5) * U
    if out_dt != "e4m3":
        err = (out.double() - y).abs()
        assert (err <= y.abs() * (rel + half_step(out_dt)) + 1e-37).all(), err.max().item()
        return
    g = group or cols
    yg = y.view(x.shape[0], -1, g)
    top = yg.abs().amax(-1).clamp_min(1e-10) / 448
    s = scales.double()
    if pow2:
        assert torch.equal(torch.frexp(scales)[0], torch.full_like(scales, 0.5))
        assert (s >= top * (1 - rel - U)).all() and (s / 2 < top * (1 + rel + U)).all()
    else:
        assert ((s - top).abs() <= top * (rel + 2 * U)).all()
    want = (yg / s[..., None]).view_as(y)            # by the scale that was written
    err = (out.double() - want).abs()
    step = torch.maximum(want.abs() * half_step("e4m3"), torch.tensor(2.0**-10, device="cuda", dtype=torch.float64))
    assert (err <= step * (1 + 1e-6) + want.abs() * (rel + 4 * U)).all(), err.max().item()


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 64), (2, 1000), (9, 512), (7, 1024), (4, 1032), (3, 4096), (2, 5003),
                                       (2, 7168), (2, 8193), (1, 16384), (2, 32768), (700, 1024), (1300, 1096), (2500, 264)])
@pytest.mark.parametrize("xt,rt,ot", [("bf16", None, "bf16"), ("bf16", "bf16", "bf16"), ("f32", "f32", "f32"),
                                      ("bf16", "f32", "bf16"), ("f32", "bf16", "f32"), ("f32", None, "f32")])
def test_norm(rows, cols, xt, rt, ot):
    x, w = randn((rows, cols), xt, 1), 1 + randn((cols,), "f32", 2, 0.1)
    res = None if rt is None else randn((rows, cols), rt, 3, 4.0)
    out, res_out, _ = run_norm(x, res, w, ot)
    check_norm(x, res, w, ot, out, res_out, None)


@pytest.mark.parametrize("rows,cols", [(1, 256), (3, 1024), (5, 768), (2, 4096), (3, 7168), (1, 32768), (400, 2560)])
@pytest.mark.parametrize("group", [0, 32, 64, 128, 256])
@pytest.mark.parametrize("pow2", [0, 1])
@pytest.mark.parametrize("off", [0, 1])
def test_norm_8bit(rows, cols, group, pow2, off):
    # off = 1: no row start is aligned
    _, x = strided(rows, cols, "bf16", cols + 8 * off + off, off, 3.0)
    x.copy_(randn((rows, cols), "bf16", 4))
    res, w = randn((rows, cols), "bf16", 5, 2.0), 1 + randn((cols,), "f32", 6, 0.1)
    out, res_out, scales = run_norm(x, res, w, "e4m3", group, pow2)
    assert scales.shape == (rows, cols // (group or cols))
    check_norm(x, res, w, "e4m3", out, res_out, scales, group, pow2)


def test_norm_8bit_odd_row_scale():
    x, w = randn((37, 5003), "f32", 7), torch.ones(5003, device="cuda")
    out, _, scales = run_norm(x, None, w, "e4m3")
    check_norm(x, None, w, "e4m3", out, None, scales)


@pytest.mark.parametrize("ld,off", [(1032, 0), (1031, 0), (1040, 8), (1040, 3)])
@pytest.mark.parametrize("ot", ["bf16", "f32"])
def test_norm_strides_leave_the_rest(ld, off, ot):
    rows, cols = 11, 1024
    bx, x = strided(rows, cols, "bf16", ld, off, 3.0)
    br, res = strided(rows, cols, "f32", ld, off, 5.0)
    bo, out = strided(rows, cols, ot, ld, off, 9.0)
    x.copy_(randn((rows, cols), "bf16", 8))
    res.copy_(randn((rows, cols), "f32", 9))
    keep = res.clone()
    w = 1 + randn((cols,), "f32", 10, 0.1)
    run_norm(x, res, w, ot, out=out, res_out=res)                # residual in place
    check_norm(x, keep, w, ot, out, res, None)
    for buf, view, fill in ((bx, x, 3.0), (br, res, 5.0), (bo, out, 9.0)):
        view.fill_(fill)
        assert (buf == fill).all()                               # nothing outside the rows was written


@pytest.mark.parametrize("rows,cols", [(13, 1), (20, 3), (2500, 333), (1300, 1003), (1300, 5003), (900, 9001), (700, 20011)])
@pytest.mark.parametrize("off", [0, 5])
@pytest.mark.parametrize("xt,rt,ot", [("bf16", "bf16", "bf16"), ("f32", None, "f32"), ("bf16", "f32", "e4m3"),
                                      ("f32", "bf16", "bf16")])
def test_norm_rows_start_anywhere(rows, cols, off, xt, rt, ot):
    # rows one after another: they start at every remainder, the same in all arrays
    bx, x = strided(rows, cols, xt, cols, off, 3.0)
    bo, out = strided(rows, cols, ot, cols, off, 9.0)
    x.copy_(randn((rows, cols), xt, 16))
    br = res = keep = None
    if rt is not None:
        br, res = strided(rows, cols, rt, cols, off, 5.0)
        res.copy_(randn((rows, cols), rt, 17, 2.0))
        keep = res.clone()
    w = 1 + randn((cols,), "f32", 18, 0.1)
    _, _, scales = run_norm(x, res, w, ot, out=out, res_out=res)
    check_norm(x, keep, w, ot, out, res, scales)
    for buf, view, fill in ((bx, x, 3.0), (br, res, 5.0), (bo, out, 9.0)):
        if buf is not None:
            view.fill_(fill)
            assert (buf.float() == fill).all()                   # nothing outside the rows was written


@pytest.mark.parametrize("cols", [512, 4096, 1001])
def test_norm_residual_sum_of_any_bits(cols):
    # every exponent, subnormals, infinities and NaN: the sum kept is the f32 sum, rounded
    g = torch.Generator(device="cuda").manual_seed(21)
    x, res = (torch.randint(-32768, 32768, (300, cols), generator=g, device="cuda", dtype=torch.int32).to(torch.int16)
              .view(torch.bfloat16) for _ in range(2))
    near = torch.arange(300 * cols, device="cuda").view(300, cols) % 2 == 0
    res = torch.where(near, (x.view(torch.int16) ^ -32768 ^ (res.view(torch.int16) & 1023)).view(torch.bfloat16), res)
    want = (x.float() + res.float()).to(torch.bfloat16)
    _, got, _ = run_norm(x, res, torch.ones(cols, device="cuda"), "bf16")
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))


def test_norm_ragged_in_place():
    x, w = randn((1500, 5003), "f32", 19), 1 + randn((5003,), "f32", 20, 0.1)
    old = x.clone()
    run_norm(x, None, w, "f32", out=x)
    check_norm(old, None, w, "f32", x, None, None)


def test_norm_in_place_and_sum_not_kept():
    x, res, w = randn((50, 4096), "bf16", 11), randn((50, 4096), "bf16", 12), torch.ones(4096, device="cuda")
    old, before = x.clone(), res.clone()
    run_norm(x, res, w, "bf16", keep=False, out=x)
    check_norm(old, before, w, "bf16", x, None, None)
    assert torch.equal(res, before)


@pytest.mark.parametrize("cols", [1000, 1024, 4096, 5003])
def test_norm_bad_rows_stay_alone(cols):
    x, w = randn((6, cols), "f32", 13), torch.ones(cols, device="cuda")
    x[1, 5], x[3, cols - 1], x[4] = NAN, float("inf"), 0.0
    out, _, _ = run_norm(x, None, w, "f32")
    good = [0, 2, 4, 5]
    check_norm(x[good], None, w, "f32", out[good], None, None)
    assert out[1].isnan().all() and (out[4] == 0).all()
    assert out[3, cols - 1].isnan() and (out[3, :cols - 1] == 0).all()     # x / inf, inf / inf
    q, _, s = run_norm(x, None, w, "e4m3")
    assert s[1].isnan().all() and s[3].isnan().all() and q[1].float().isnan().all()
    assert s[4, 0] == torch.tensor(1e-10) / 448 and (q[4].float() == 0).all()
    check_norm(x[good], None, w, "e4m3", q[good], None, s[good])


def test_norm_rows_do_not_depend_on_the_batch():
    x, res, w = randn((2000, 7168), "bf16", 14), randn((2000, 7168), "bf16", 15), torch.ones(7168, device="cuda")
    whole, _, s = run_norm(x, res, w, "e4m3", 128)
    for r in (0, 777, 1999):
        one, _, s1 = run_norm(x[r:r + 1], res[r:r + 1], w, "e4m3", 128)
        assert torch.equal(one.view(torch.uint8), whole[r:r + 1].view(torch.uint8)) and torch.equal(s1, s[r:r + 1])


# ------------------------------------------------------------------------------------
# rotary positions
# ------------------------------------------------------------------------------------
def rope_exact(x, pos, dims, first, half, inverse, scaling, mscale):
    """In f64 from the angle pos * f_i; also the bound's |a| + |b| per rotated value."""
    i = torch.arange(dims // 2, device="cuda", dtype=torch.float64)
    f = 160000.0 ** (-2 * i / dims) / (scaling if scaling else 1.0)
    ang = pos.double()[:, None, None] * f * (-1 if inverse else 1)
    z = x.double()[..., first:first + dims]
    a, b = (z[..., :dims // 2], z[..., dims // 2:]) if half else (z[..., 0::2], z[..., 1::2])
    ya, yb = mscale * (a * ang.cos() - b * ang.sin()), mscale * (a * ang.sin() + b * ang.cos())
    mag = mscale * (a.abs() + b.abs())
    y, m = x.double().clone(), torch.zeros_like(x, dtype=torch.float64)
    if half:
        y[..., first:first + dims], m[..., first:first + dims] = torch.cat([ya, yb], -1), torch.cat([mag, mag], -1)
    else:
        y[..., first:first + dims] = torch.stack([ya, yb], -1).flatten(-2)
        m[..., first:first + dims] = torch.stack([mag, mag], -1).flatten(-2)
    return y, m


def check_rope(y, exact, mag, dt):
    """The turn's rounding to f32 (2^-26 turns, 1.6 u radians), sincospi (2 u), the product with
    mscale and the two products and the sum of the rotation (4 u); the reference's own angle is
    off by 2^-53 of up to 2^31 radians. Then the output's rounding."""
    err = (y.double() - exact).abs()
    ok = err <= mag * (7.6 * U + 2.0**-22) + exact.abs() * half_step(dt)
    assert ok.all(), err.max().item()


def run_rope(x, y, pos, dims, first, half=0, inverse=0, scaling=0.0, mscale=1.0, x2=None, y2=None, stream=None):
    t = hb.rope_table(hb.RopeScaling(rope_dims=dims, kind=hb.ROPE_LINEAR if scaling else hb.ROPE_PLAIN, theta=160000.0,
                                     factor=scaling or 1.0), "cuda")
    st = dict(x_token=x.stride(0), x_head=x.stride(1), y_token=y.stride(0), y_head=y.stride(1))
    if x2 is not None:
        st.update(x2_token=x2.stride(0), x2_head=x2.stride(1), y2_token=y2.stride(0), y2_head=y2.stride(1))
    d = hb.RopeDesc(tokens=x.shape[0], heads=x.shape[1], heads2=0 if x2 is None else x2.shape[1], D=x.shape[2], rope_dims=dims,
                    rope_first=first, half=half, inverse=inverse, src_dtype=hb.dtype_code(x), dst_dtype=hb.dtype_code(y),
                    mscale=mscale, **st)
    hb.rope(d, t, pos, x, y, x2, y2, stream=stream)


def positions(tokens, kind):
    if kind == "far":
        g = torch.Generator(device="cuda")
        g.manual_seed(tokens)
        return torch.randint(-(2**31), 2**31, (tokens,), generator=g, device="cuda").to(torch.int32)
    return torch.arange(tokens, device="cuda", dtype=torch.int32) + 61440


@pytest.mark.parametrize("tokens,heads,heads2", [(1, 1, 0), (1, 64, 1), (3, 5, 2), (67, 64, 1), (500, 1, 0), (2049, 2, 1)])
@pytest.mark.parametrize("D,dims,first", [(512, 64, 448), (128, 64, 64), (128, 128, 0), (64, 32, 0), (6, 2, 3), (72, 24, 16),
                                          (1024, 2, 1)])
@pytest.mark.parametrize("half", [0, 1])
@pytest.mark.parametrize("src,dst", [("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32"), ("bf16", "f32")])
def test_rope(tokens, heads, heads2, D, dims, first, half, src, dst):
    x = randn((tokens, heads, D), src, 20)
    x2 = randn((tokens, heads2, D), src, 21) if heads2 else None
    y = torch.empty((tokens, heads, D), device="cuda", dtype=DT[dst])
    y2 = torch.empty((tokens, heads2, D), device="cuda", dtype=DT[dst]) if heads2 else None
    pos = positions(tokens, "near")
    run_rope(x, y, pos, dims, first, half, x2=x2, y2=y2)
    for a, b in ((x, y), (x2, y2)):
        if a is not None:
            check_rope(b, *rope_exact(a, pos, dims, first, half, 0, 0.0, 1.0), dst)
            for part in (slice(0, first), slice(first + dims, D)):
                assert torch.equal(b[..., part], a[..., part].to(DT[dst]))


@pytest.mark.parametrize("half", [0, 1])
@pytest.mark.parametrize("inverse", [0, 1])
@pytest.mark.parametrize("scaling,mscale", [(0.0, 1.0), (40.0, 1.37)])
def test_rope_in_place_at_far_positions(half, inverse, scaling, mscale):
    # f32, any int32 position: the whole turns drop out exactly. The reference's own product is
    # off by pos * f * 2^-53 <= 2^-22 radians, counted in the bound.
    x, k = randn((130, 7, 128), "f32", 22), randn((130, 1, 128), "f32", 23)
    was, kwas = x.clone(), k.clone()
    pos = positions(130, "far")
    pos[0], pos[1], pos[2] = 0, 2**31 - 1, -(2**31)
    run_rope(x, x, pos, 64, 64, half, inverse, scaling, mscale, x2=k, y2=k)
    check_rope(x, *rope_exact(was, pos, 64, 64, half, inverse, scaling, mscale), "f32")
    check_rope(k, *rope_exact(kwas, pos, 64, 64, half, inverse, scaling, mscale), "f32")
    assert torch.equal(x[..., :64], was[..., :64]) and torch.equal(k[..., :64], kwas[..., :64])


def test_rope_inverse_returns():
    x = randn((40, 64, 512), "f32", 24)
    y, z = torch.empty_like(x), torch.empty_like(x)
    pos = positions(40, "far")
    run_rope(x, y, pos, 64, 448)
    run_rope(y, z, pos, 64, 448, inverse=1)
    # the same sine and cosine both ways: two rotations' roundings
    a = x[..., 448:].abs()
    assert ((x - z).abs()[..., 448:] <= 16 * U * (a + a.view(40, 64, 32, 2).flip(-1).reshape(a.shape))).all()
    assert torch.equal(x[..., :448], z[..., :448])


@pytest.mark.parametrize("pad,off", [(0, 0), (8, 0), (3, 0), (8, 1), (8, 8)])
def test_rope_strided_heads(pad, off):
    # heads sliced out of a wider row (a fused projection's output), written into a cache's slots
    tokens, heads, D = 33, 5, 128
    buf = randn((off + tokens * heads * (D + pad) + 64,), "bf16", 25)
    x = buf[off:off + tokens * heads * (D + pad)].view(tokens, heads, D + pad)[..., :D]
    cache = torch.full((tokens, 2 * heads, D), 9.0, device="cuda", dtype=torch.bfloat16)
    y = cache[:, 1::2]
    pos = positions(tokens, "near")
    run_rope(x, y, pos, 64, 64)
    check_rope(y, *rope_exact(x, pos, 64, 64, 0, 0, 0.0, 1.0), "bf16")
    assert (cache[:, 0::2] == 9.0).all()


# ------------------------------------------------------------------------------------
# shared-prefix combine
# ------------------------------------------------------------------------------------
SHAPES = {8: 64, 16: 128, 64: 512}


def prefix_case(B, L, H, P, own, dt, seed=0, W=None, window=128, t0=None, q_std=2.0):
    """Sequences with `own[b]` own pooled rows. Rows that no query may read hold NaN: the ends
    of the window buffers and of the own rows' allocation."""
    Dh = SHAPES[H]
    W = window + L - 1 if W is None else W
    off = torch.tensor([0] + list(own), dtype=torch.int64).cumsum(0)
    c = dict(B=B, L=L, H=H, Dh=Dh, P=P, W=W, window=window, dt=dt, Np_max=max(own) if own else 0)
    c["q"] = randn((B, L, H, Dh), dt, seed, q_std)
    c["prefix"] = randn((P, Dh), dt, seed + 1)
    c["pooled"] = torch.cat([randn((int(off[-1]), Dh), dt, seed + 2), torch.full((3, Dh), NAN, device="cuda", dtype=DT[dt])])
    c["local"] = randn((B, W, Dh), dt, seed + 3)
    c["sinks"] = randn((H,), "f32", seed + 4) + 2.0
    t = [4 * (P + n) - L if t0 is None else t0 for n in own]
    n_loc = [max(0, min(W, x + L)) for x in t]
    for b in range(B):
        c["local"][b, n_loc[b]:] = NAN
    c["len"] = torch.tensor(n_loc, dtype=torch.int32, device="cuda")
    c["pos0"] = torch.tensor([x + L - n for x, n in zip(t, n_loc)], dtype=torch.int32, device="cuda")
    c["t0"] = torch.tensor(t, dtype=torch.int32, device="cuda")
    c["off"] = off.cuda()
    return c


def run_prefix(c, out_dt, ws=None, stream=None, flags=0, kv_rows=None, sinks="own", out=None):
    d = hb.PrefixDesc(B=c["B"], L=c["L"], H=c["H"], Dh=c["Dh"], window=c["window"], W_max=c["W"], r=4, prefix_rows=c["P"],
                      Np_max=c["Np_max"], kv_rows=c["pooled"].shape[0] if kv_rows is None else kv_rows, scale=0.0,
                      q_dtype=CODE[c["dt"]], kv_dtype=CODE[c["dt"]], out_dtype=CODE[out_dt], flags=flags)
    if ws is None:
        ws = hb.alloc_workspace(hb.workspace_bytes(hb.OP_PREFIX_ATTEND, d))
        ws[256:] = 255                                        # NaN patterns: nothing is read before it is written
    if out is None:
        out = torch.full((c["B"], c["L"], c["H"], c["Dh"]), NAN, device="cuda", dtype=DT[out_dt])
    hb.prefix_attend(d, c["q"], c["local"] if c["W"] else None, c["len"], c["pos0"], c["prefix"] if c["P"] else None,
                     c["pooled"] if c["Np_max"] else None, c["off"], c["sinks"] if isinstance(sinks, str) else sinks,
                     c["t0"], out, ws, stream=stream)
    return out, ws


def prefix_rows(c, b, j):
    """The rows that query row (b, j) sees, in f64."""
    t, n = int(c["t0"][b]) + j, int(c["len"][b])
    p0 = int(c["pos0"][b])
    loc = [s for s in range(n) if 0 <= t - (p0 + s) < c["window"]]
    k0, k1 = int(c["off"][b]), int(c["off"][b + 1])
    if c["L"] > 1:
        k1 = max(k0, min(k1, k0 + (t + 1) // 4 - c["P"]))
    return torch.cat([c["local"][b, loc].double(), c["prefix"].double(), c["pooled"][k0:k1].double()])


def check_prefix(c, out, out_dt, sinks="own"):
    """Logits: Dh products summed in f32, off by e = Dh u scale sum|q k| + 2 u |z| (and 2 u |z|
    of the exponent's argument in base 2); weights by 2 e, and their f32 sums over n rows by
    n u. bf16 inputs may round each weight to bf16 (2^-9) before the product with the values."""
    sinks = c["sinks"] if isinstance(sinks, str) else sinks
    scale = c["Dh"] ** -0.5
    for b in range(c["B"]):
        for j in range(c["L"]):
            v, q = prefix_rows(c, b, j), c["q"][b, j].double()
            got = out[b, j].double()
            s = torch.full((c["H"],), -math.inf, device="cuda", dtype=torch.float64) if sinks is None else sinks.double()
            if v.shape[0] == 0:
                assert (got == 0).all()
                continue
            z = q @ v.t() * scale
            e = (c["Dh"] * U * (q.abs() @ v.abs().t() * scale) + 4 * U * z.abs()).amax(-1, keepdim=True)
            p = torch.softmax(torch.cat([z, s[:, None]], -1), -1)[:, :-1]
            want, mag = p @ v, p @ v.abs()
            tol = mag * (4 * e + 2 * v.shape[0] * U + (half_step("bf16") / 2 if c["dt"] == "bf16" else 0)) \
                + want.abs() * half_step(out_dt) + 1e-37
            err = (got - want).abs()
            assert (err <= tol).all(), (b, j, (err / tol).max().item())


OWN = [[0], [1], [5, 0, 70], [130, 64, 1, 63, 200], [33] * 9]


@pytest.mark.parametrize("H,dt,out_dt", [(8, "f32", "f32"), (16, "f32", "bf16"), (16, "bf16", "bf16"), (8, "bf16", "f32"),
                                         (64, "f32", "f32"), (64, "bf16", "bf16"), (64, "bf16", "f32")])
@pytest.mark.parametrize("P", [0, 1, 31, 64, 65, 1000])
@pytest.mark.parametrize("own", OWN, ids=[str(len(o)) + "x" + str(max(o)) for o in OWN])
@pytest.mark.parametrize("L", [1, 3])
def test_prefix(H, dt, out_dt, P, own, L):
    c = prefix_case(len(own), L, H, P, own, dt, seed=P + L)
    out, ws = run_prefix(c, out_dt)
    assert hb.device_status(ws) == 0
    check_prefix(c, out, out_dt)


@pytest.mark.parametrize("H,dt", [(8, "f32"), (16, "bf16"), (64, "f32"), (64, "bf16")])
def test_prefix_empty_parts(H, dt):
    # no window buffer; no window; no own rows at all; no shared rows; nothing
    for P, own, W, window in ((70, [5, 0], 0, 128), (70, [5, 0], 16, 0), (70, [0, 0], 16, 16), (0, [9, 0], 0, 0), (0, [0, 0], 0, 0)):
        c = prefix_case(2, 1, H, P, own, dt, W=W, window=window)
        out, _ = run_prefix(c, "f32")
        check_prefix(c, out, "f32")
        for sinks in (None, torch.full((H,), -math.inf, device="cuda")):
            out, _ = run_prefix(c, "f32", sinks=sinks)
            check_prefix(c, out, "f32", sinks)


@pytest.mark.parametrize("H,dt", [(16, "f32"), (64, "bf16")])
def test_prefix_masks_own_rows_by_position(H, dt):
    # early tokens: own rows that their windows have not completed are not seen (they hold NaN)
    c = prefix_case(3, 4, H, 40, [20, 3, 0], dt, t0=4 * 40 + 5)
    c["pooled"][int(c["off"][0]) + 3:int(c["off"][1])] = NAN     # t = 168 at most sees rows 0 and 1
    c["pooled"][int(c["off"][1]) + 2:int(c["off"][2])] = NAN
    out, _ = run_prefix(c, "f32")
    check_prefix(c, out, "f32")


@pytest.mark.parametrize("H,dt", [(16, "f32"), (64, "bf16")])
def test_prefix_rising_and_extreme_logits(H, dt):
    # the running maximum moves in every chunk; some heads' logits are hundreds apart
    c = prefix_case(3, 1, H, 700, [50, 9, 0], dt, q_std=1.0)
    ramp = torch.linspace(0.01, 6.0, 700, device="cuda")[:, None]
    c["prefix"] = (c["prefix"].float().sign() * ramp).to(DT[dt])
    c["q"][:, :, 0] = 6.0 * c["prefix"][699]
    c["q"][:, :, 1] = -6.0 * c["prefix"][699]
    out, _ = run_prefix(c, "f32")
    check_prefix(c, out, "f32")


@pytest.mark.parametrize("H,dt", [(16, "f32"), (64, "bf16")])
def test_prefix_many_rows(H, dt):
    # several query-row tiles, several segments, an odd number of stacked rows
    c = prefix_case(37, 1, H, 3001 if H == 16 else 5001, [(7 * b) % 90 for b in range(37)], dt)
    out, _ = run_prefix(c, "f32")
    check_prefix(c, out, "f32")


@pytest.mark.parametrize("H,dt", [(16, "f32"), (64, "bf16")])
@pytest.mark.parametrize("bad", ["negative", "falling", "past", "long"])
def test_prefix_bad_offsets_are_flagged(H, dt, bad):
    c = prefix_case(3, 1, H, 50, [6, 7, 8], dt)
    good = c["off"].clone()
    off = good.clone()
    kv_rows = None
    if bad == "negative":
        off[0] = -1
        skipped = [0]
    elif bad == "falling":
        off[1] = off[2] + 1
        skipped = [0, 1] if int(off[1]) > c["Np_max"] else [1]
    elif bad == "past":
        kv_rows = int(good[2]) + 1
        skipped = [2]
    else:
        c["Np_max"] = 7
        skipped = [2]
    c["off"] = off
    out, ws = run_prefix(c, "f32", kv_rows=kv_rows)
    assert hb.device_status(ws) == hb.DEV_BAD_OFFSETS
    ok = dict(c)
    for b in range(3):                                          # sequence b alone, its own rows dropped if skipped
        o = torch.zeros(4, dtype=torch.int64)
        o[b], o[b + 1] = int(off[b]), int(off[b]) if b in skipped else int(off[b + 1])
        ok["off"] = o.clamp_min(0)
        one = {**ok, "B": 1, "q": c["q"][b:b + 1], "local": c["local"][b:b + 1], "len": c["len"][b:b + 1],
               "pos0": c["pos0"][b:b + 1], "t0": c["t0"][b:b + 1], "off": ok["off"][b:b + 2]}
        check_prefix(one, out[b:b + 1], "f32")


@pytest.mark.parametrize("L", [1, 2])
def test_prefix_is_the_dense_branch(L):
    # the same rows as one packed stream through hisa_sparse_attend (I = NULL), which sees the
    # shared rows whole once t0 + 1 >= r P: two kernels of the same function, each within its
    # bound of the f64 result
    c = prefix_case(3, L, 64, 300, [40, 0, 17], "bf16")
    for k in ("t0", "pos0"):
        c[k] += L - 1
    out, _ = run_prefix(c, "f32")
    kv = torch.cat([torch.cat([c["prefix"], c["pooled"][int(c["off"][b]):int(c["off"][b + 1])]]) for b in range(3)])
    off = c["off"] + 300 * torch.arange(4, device="cuda")
    d = hb.AttnDesc(B=3, L=L, H=64, Dh=512, window=128, W_max=c["W"], r=4, k=0, Np_max=340, kv_rows=kv.shape[0], scale=0.0,
                    q_dtype=hb.HISA_BF16, kv_dtype=hb.HISA_BF16)
    ws = hb.alloc_workspace(hb.workspace_bytes(hb.OP_SPARSE_ATTEND, d))
    ref = torch.empty_like(out)
    hb.sparse_attend(d, c["q"], c["local"], c["len"], c["pos0"], kv, off, None, c["sinks"], c["t0"], ref, ws)
    check_prefix(c, out, "f32")
    check_prefix(c, ref, "f32")


@pytest.mark.parametrize("H,dt", [(16, "f32"), (64, "bf16")])
def test_prefix_same_bits_every_time(H, dt):
    c = prefix_case(5, 2, H, 2000, [100, 3, 0, 64, 65], dt)
    a, _ = run_prefix(c, "f32")
    for _ in range(3):
        b, _ = run_prefix(c, "f32")
        assert torch.equal(a, b)


@pytest.mark.parametrize("H,dt", [(16, "bf16"), (64, "bf16"), (16, "f32")])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_prefix_sequences_do_not_meet(H, dt, bad):
    # a sequence whose own or local rows hold a NaN or an infinity spoils no other
    c = prefix_case(5, 1, H, 130, [70, 33, 64, 5, 0], dt)
    clean, _ = run_prefix(c, "f32")
    c["pooled"][int(c["off"][1]) + 7] = bad
    c["pooled"][int(c["off"][2]) + 63] = bad
    c["local"][4, 3] = bad
    out, _ = run_prefix(c, "f32")
    for b in range(5):
        if b in (0, 3):
            assert torch.equal(out[b], clean[b])
        else:
            assert not torch.isfinite(out[b]).all()


@pytest.mark.parametrize("H,dt,P,own", [(64, "bf16", 1500, [5, 0, 40]), (64, "bf16", 10, [0, 31, 32, 33]), (16, "bf16", 1500, [5, 0])])
def test_prefix_chained(H, dt, P, own):
    c = prefix_case(len(own), 1, H, P, own, dt)
    out, ws = run_prefix(c, "bf16", flags=hb.FLAG_CHAINED)
    for _ in range(3):                                           # a call directly behind another, same workspace
        out, ws = run_prefix(c, "bf16", ws=ws, out=out.zero_(), flags=hb.FLAG_CHAINED)
    assert hb.device_status(ws) == 0
    check_prefix(c, out, "bf16")


@pytest.mark.parametrize("B,L,P,own", [(58, 4, 18796, 0), (107, 2, 22071, 3), (185, 1, 21246, 40), (43, 4, 24075, 300)])
def test_prefix_many_items_per_pair(B, L, P, own):
    # query rows that keep every pair of CTAs at several segments: the same bits every time
    c = prefix_case(B, L, 64, P, [own] * B, "bf16")
    first = run_prefix(c, "bf16")[0].clone()
    assert torch.isfinite(first.float()).all()
    for _ in range(8):
        out, ws = run_prefix(c, "bf16")
        assert torch.equal(out, first) and hb.device_status(ws) == 0


@pytest.mark.parametrize("offset", [8, 16])
def test_prefix_output_aligned_to_16_bytes_alone(offset):
    c = prefix_case(2, 1, 64, 100, [3, 40], "bf16")
    buf = torch.zeros(2 * 64 * 512 + 64, device="cuda", dtype=torch.bfloat16)
    out = buf[offset:offset + 2 * 64 * 512].view(2, 1, 64, 512)
    run_prefix(c, "bf16", out=out)
    check_prefix(c, out, "bf16")
    assert (buf[:offset] == 0).all() and (buf[offset + 2 * 64 * 512:] == 0).all()


@pytest.mark.parametrize("window,L", [(16, 1), (33, 5), (128, 9)])
def test_prefix_windows(window, L):
    # windows that start and end inside the buffer
    c = prefix_case(3, L, 64, 70, [9, 0, 40], "bf16", window=window, W=window + 40, t0=4 * 70 + 60)
    for b in range(3):
        c["len"][b] = window + 30 - 11 * b
        c["pos0"][b] = c["t0"][b] - window - 5 + b
        n = int(c["len"][b])
        c["local"][b] = randn(tuple(c["local"][b].shape), "bf16", 40 + b)
        c["local"][b, n:] = NAN
    out, _ = run_prefix(c, "f32")
    check_prefix(c, out, "f32")


# ------------------------------------------------------------------------------------
# offsets past 32 bits
# ------------------------------------------------------------------------------------
def test_norm_past_32_bits():
    rows, cols = 300001, 8192                                    # 2.46e9 elements
    x, w = torch.zeros((rows, cols), device="cuda", dtype=torch.bfloat16), torch.ones(cols, device="cuda")
    pick = [0, 131072, 262144, rows - 1]
    x[pick] = randn((4, cols), "bf16", 60)
    out, _, _ = run_norm(x, None, w, "bf16", out=x)
    assert torch.equal(x[1], torch.zeros_like(x[1]))
    check_norm(randn((4, cols), "bf16", 60), None, w, "bf16", x[pick], None, None)


def test_rope_past_32_bits():
    tokens, heads, D = 66000, 64, 512                            # 2.16e9 elements, in place
    x = torch.zeros((tokens, heads, D), device="cuda", dtype=torch.bfloat16)
    pick = torch.tensor([0, 65535, 65536, tokens - 1], device="cuda")
    x[pick] = randn((4, heads, D), "bf16", 61)
    was, pos = x[pick].clone(), torch.arange(tokens, device="cuda", dtype=torch.int32)
    run_rope(x, x, pos, 64, 448)
    check_rope(x[pick], *rope_exact(was, pos[pick], 64, 448, 0, 0, 0.0, 1.0), "bf16")


def test_prefix_own_rows_past_32_bits():
    c = prefix_case(3, 1, 64, 100, [40, 7, 33], "bf16")
    far = 4_300_000                                              # rows of 1 KiB: past 2^32 bytes and 2^31 elements
    pool = torch.empty((far + 100, 512), device="cuda", dtype=torch.bfloat16)
    pool[far:far + 80] = c["pooled"][:80]
    pool[far + 80:] = NAN
    c["pooled"], c["off"] = pool, c["off"] + far
    out, ws = run_prefix(c, "f32")
    assert hb.device_status(ws) == 0
    check_prefix(c, out, "f32")


# ------------------------------------------------------------------------------------
# streams and graphs
# ------------------------------------------------------------------------------------
def test_another_stream_and_a_graph():
    c = prefix_case(4, 1, 64, 500, [30, 0, 7, 64], "bf16")
    want, ws = run_prefix(c, "bf16")
    x, res, w = randn((4, 4096), "bf16", 30), randn((4, 4096), "bf16", 31), torch.ones(4096, device="cuda")
    n_want, r_want, _ = run_norm(x, res, w, "bf16")
    q = randn((4, 64, 512), "bf16", 32)
    r_rope = torch.empty_like(q)
    pos = positions(4, "near")
    table = hb.rope_table(hb.RopeScaling(rope_dims=64, kind=hb.ROPE_PLAIN, theta=160000.0), "cuda")
    rd = hb.RopeDesc(tokens=4, heads=64, heads2=0, D=512, rope_dims=64, rope_first=448, src_dtype=hb.HISA_BF16,
                     dst_dtype=hb.HISA_BF16, mscale=1.0, x_token=64 * 512, x_head=512, y_token=64 * 512, y_head=512)
    hb.rope(rd, table, pos, q, r_rope)
    out, y, got, res2 = (torch.zeros_like(t) for t in (want, n_want, r_rope, res))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def calls():
        run_norm(x, res, w, "bf16", out=y, res_out=res2)
        hb.rope(rd, table, pos, q, got)
        run_prefix(c, "bf16", ws=ws, out=out)

    def check():
        for a, b in ((out, want), (y, n_want), (got, r_rope), (res2, r_want)):
            assert torch.equal(a, b)
            a.zero_()

    with torch.cuda.stream(s):
        calls()
    s.synchronize()
    check()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        check()


# ------------------------------------------------------------------------------------
# together: a layer's decode step
# ------------------------------------------------------------------------------------
@pytest.mark.parametrize("batch,prefix,hidden,steps", [(5, 300, 1024, 6), (2, 64, 1000, 3)])
def test_shared_prefix_decode(batch, prefix, hidden, steps):
    # Roped queries and rows, the weights of the softmax, and the output are each rounded to bf16
    # (half a step, 2^-8 of a value at most); logits of about 4 standard deviations turn the queries'
    # and rows' share into 2 * 2^-8 * 8 of the weights. The last rotation rounds once more. All of it
    # stays below a tenth of the largest output.
    import sys

    import deepseek_sparse_attention_hisa_gb300 as pkg
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(pkg.__file__)))
    sys.path.insert(0, os.path.join(root, "examples"))
    import shared_prefix_decode
    assert shared_prefix_decode.run(batch, prefix, hidden, steps, own_rows=40, say=lambda *_: None) < 0.1
