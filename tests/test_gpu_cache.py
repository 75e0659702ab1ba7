"""Head norms with rotary positions and the cache in pages against plain 64-bit implementations (GB300).

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
CODE = {"f32": hb.HISA_F32, "bf16": hb.HISA_BF16, "e4m3": hb.HISA_E4M3, "4bit": hb.HISA_E2M1}
NAN = float("nan")
EPS = 1e-6
THETA = 160000.0


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


def ints(values, dt=torch.int32):
    return torch.tensor(values, device="cuda", dtype=dt)


def table_of(dims):
    return hb.rope_table(hb.RopeScaling(rope_dims=dims, kind=hb.ROPE_PLAIN, theta=THETA), "cuda") if dims else None


# ------------------------------------------------------------------------------------
# the norm of each head and rotary positions
# ------------------------------------------------------------------------------------
def turned(x, w, norm, pos, dims, first, half, mscale=1.0):
    """x [n, heads, D] in f64, and a bound of what f32 may be off: the square's sum takes at most 16
    products in order, 2 + 5 sums over them and the lanes and a division (halved by the root: 12), the
    epsilon, root, reciprocal and two products 5; so 17 u of each value, 20 u counted. A rotation adds 3 roundings and a sine and
    cosine that are off by pi u (the turn as f32) + 4 u (their function, mscale): 12 u of both of a pair."""
    y = x.double()
    if norm:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS)
        if w is not None:
            y = y * w.double()
    off = y.abs() * 20 * U
    if dims:
        i = torch.arange(dims // 2, device="cuda", dtype=torch.float64)
        a = pos.double()[:, None, None] * THETA ** (-2 * i / dims)
        c, s = torch.cos(a) * mscale, torch.sin(a) * mscale
        at = torch.arange(dims // 2, device="cuda")
        lo = first + (at if half else 2 * at)
        hi = lo + (dims // 2 if half else 1)
        p, q = y[..., lo], y[..., hi]
        y = y.clone()
        y[..., lo], y[..., hi] = p * c - q * s, p * s + q * c
        both = (p.abs() + q.abs()) * 32 * U * max(mscale, 1.0)
        off[..., lo] = off[..., hi] = both
    return y, off


def check_turned(got, y, off, dt):
    err = (got.double() - y).abs()
    assert (err <= off + y.abs() * half_step(dt) + 1e-37).all(), (err / (off + y.abs() * half_step(dt) + 1e-37)).max().item()


def run_norm_rope(x, y, pos, dims, first, half=0, w=None, x2=None, y2=None, w2=None, norm=1, norm2=1, mscale=1.0, stream=None,
                  flags=0):
    strides = lambda t: (t.stride(0), t.stride(1)) if t is not None else (0, 0)  # noqa: E731
    d = hb.NormRopeDesc(tokens=x.shape[0], heads=x.shape[1], heads2=0 if x2 is None else x2.shape[1], D=x.shape[2], norm=norm,
                        norm2=norm2 if x2 is not None else 0, rope_dims=dims, rope_first=first, half=half,
                        src_dtype=hb.dtype_code(x), dst_dtype=hb.dtype_code(y), eps=EPS, mscale=mscale, flags=flags)
    (d.x_token, d.x_head), (d.y_token, d.y_head) = strides(x), strides(y)
    (d.x2_token, d.x2_head), (d.y2_token, d.y2_head) = strides(x2), strides(y2)
    hb.norm_rope(d, table_of(dims), pos, x, w, y, x2, w2, y2, stream=stream)


def positions(n, seed=3, far=1 << 20):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randint(-far, far, (n,), generator=g, device="cuda").to(torch.int32)


SHAPES = [(1, 64, 1, 512, 64, 448), (3, 64, 1, 512, 64, 448), (700, 9, 2, 128, 64, 64), (5, 3, 0, 64, 64, 0), (2, 1, 1, 1024, 1024, 0),
          (4, 7, 1, 1024, 64, 960), (33, 5, 3, 192, 128, 32), (6, 2, 0, 16, 16, 0), (257, 16, 2, 8, 0, 0), (3, 17, 1, 576, 64, 512),
          # no units of 8: D, or where the rotated dims start or end
          (5, 3, 1, 100, 20, 80), (2, 4, 0, 2, 2, 0), (3, 2, 1, 7, 6, 1), (4, 5, 1, 512, 60, 451), (3, 2, 2, 1023, 512, 3), (2, 3, 1, 128, 24, 100)]


@pytest.mark.parametrize("tokens,heads,heads2,D,dims,first", SHAPES)
@pytest.mark.parametrize("half", [0, 1])
@pytest.mark.parametrize("src,dst", [("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32"), ("bf16", "f32")])
def test_norm_rope(tokens, heads, heads2, D, dims, first, half, src, dst):
    x, w = randn((tokens, heads, D), src, 1, 3.0), 1 + randn((D,), "f32", 2, 0.1)
    x2 = randn((tokens, heads2, D), src, 4, 0.01) if heads2 else None
    pos = positions(tokens)
    y = torch.full(x.shape, NAN, device="cuda", dtype=DT[dst])
    y2 = torch.full(x2.shape, NAN, device="cuda", dtype=DT[dst]) if heads2 else None
    run_norm_rope(x, y, pos, dims, first, half, w, x2, y2, None, mscale=1.25)
    check_turned(y, *turned(x, w, True, pos, dims, first, half, 1.25), dst)
    if heads2:
        check_turned(y2, *turned(x2, None, True, pos, dims, first, half, 1.25), dst)


@pytest.mark.parametrize("norm,norm2", [(0, 1), (1, 0), (0, 0)])
def test_norm_rope_norms_one_of_two(norm, norm2):
    x, x2, w = randn((5, 8, 128), "f32", 1), randn((5, 1, 128), "f32", 2), 1 + randn((128,), "f32", 3, 0.1)
    y, y2, pos = torch.empty_like(x), torch.empty_like(x2), positions(5)
    run_norm_rope(x, y, pos, 64, 64, 1, w if norm else None, x2, y2, w if norm2 else None, norm, norm2)
    check_turned(y, *turned(x, w, norm, pos, 64, 64, 1), "f32")
    check_turned(y2, *turned(x2, w, norm2, pos, 64, 64, 1), "f32")


@pytest.mark.parametrize("half", [0, 1])
@pytest.mark.parametrize("D,dims,first", [(512, 64, 448), (1024, 1024, 0), (100, 50, 25)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_norm_rope_in_place_and_strides(half, D, dims, first, dt):
    # heads 3 D + 5 (or 3 D + 8) apart within tokens, the rest of the buffer left alone
    gap = 8 if D % 8 == 0 else 5
    buf = torch.full((6, 4, 3 * D + gap), 7.0, device="cuda", dtype=DT[dt])
    x = buf[:, :, D:2 * D]
    x.copy_(randn(x.shape, dt, 5))
    was, pos, w = x.clone(), positions(6), 1 + randn((D,), "f32", 6, 0.1)
    run_norm_rope(x, x, pos, dims, first, half, w)
    check_turned(x, *turned(was, w, True, pos, dims, first, half), dt)
    x.fill_(7.0)
    assert (buf == 7.0).all()


def test_norm_rope_reads_a_broadcast_head():
    x, pos = randn((4, 1, 128), "bf16", 9).expand(4, 6, 128), positions(4)
    y = torch.empty((4, 6, 128), device="cuda", dtype=torch.bfloat16)
    run_norm_rope(x, y, pos, 64, 64)
    check_turned(y, *turned(x, None, True, pos, 64, 64, 0), "bf16")


def test_norm_rope_keeps_heads_apart():
    x, pos = randn((3, 4, 512), "f32", 11), positions(3)
    y, want = torch.empty_like(x), torch.empty_like(x)
    run_norm_rope(x, want, pos, 64, 448)
    x[1, 2, 5], x[2, 0, 500], x[0, 1] = NAN, math.inf, 0.0
    run_norm_rope(x, y, pos, 64, 448)
    bad = torch.zeros((3, 4), dtype=torch.bool, device="cuda")
    bad[1, 2] = bad[2, 0] = bad[0, 1] = True
    assert torch.equal(y[~bad], want[~bad])
    assert y[1, 2].isnan().all() and (y[0, 1] == 0).all()
    assert y[2, 0, 500].isnan() and (y[2, 0, :448] == 0).all()


def test_norm_rope_past_32_bits():
    tokens, heads, D = 66000, 64, 512                            # 2.16e9 elements
    x = torch.zeros((tokens, heads, D), device="cuda", dtype=torch.bfloat16)
    pick = torch.tensor([0, 65535, 65536, tokens - 1], device="cuda")
    x[pick] = randn((4, heads, D), "bf16", 61)
    was, pos = x[pick].clone(), torch.arange(tokens, device="cuda", dtype=torch.int32)
    run_norm_rope(x, x, pos, 64, 448)
    check_turned(x[pick], *turned(was, None, True, pos[pick], 64, 448, 0), "bf16")


# ------------------------------------------------------------------------------------
# a cache in pages
# ------------------------------------------------------------------------------------
GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], dtype=torch.float64)


def values(codes):
    """The 4-bit floats of packed bytes, f64."""
    return torch.stack([GRID.cuda()[(codes & 15).long()], GRID.cuda()[(codes >> 4).long()]], -1).flatten(-2)


def e4m3(scales):
    return scales.view(torch.float8_e4m3fn).double()


def pool_rows(cache, scales, g):
    """All rows of a pool, f64."""
    if scales is None:
        return cache.flatten(0, 1).double()
    return values(cache.flatten(0, 1)) * (e4m3(scales.flatten(0, 1)) * g).repeat_interleave(16, -1)


def empty_pool(pages, page, D, cache):
    """Pages whose rows read as NaN."""
    if cache == "bf16":
        return torch.full((pages, page, D), NAN, device="cuda", dtype=torch.bfloat16), None
    return (torch.full((pages, page, D // 2), 0xA5, device="cuda", dtype=torch.uint8),
            torch.full((pages, page, D // 16), 0x7F, device="cuda", dtype=torch.uint8))


def page_tables(lens, cols, page, spare=3, seed=0):
    """Pages in no order for sequences of `lens` rows; -7 where a sequence has none. Returns the pages too."""
    g = torch.Generator()
    g.manual_seed(seed)
    need = [-(-n // page) for n in lens]
    order = torch.randperm(sum(need) + spare, generator=g).tolist()
    t = torch.full((len(lens), cols), -7, dtype=torch.int32)
    for b, n in enumerate(need):
        for i in range(n):
            t[b, i] = order.pop()
    return t.cuda(), sum(need) + spare


def slots(table, b, index, page):
    return table[b].long()[index // page] * page + index % page


def append_desc(x, pool, B, cols, page, cache, norm=0, dims=0, first=0, half=0, r=4, g=0.75, mscale=1.0, ld=None, rows=None):
    return hb.CacheDesc(pages=pool.shape[0], page_rows=page, D=x.shape[1], cache_dtype=CODE[cache], cache_scale=g, B=B,
                        table_cols=cols, rows=x.shape[0] if rows is None else rows, ld=x.stride(0) if ld is None else ld,
                        io_dtype=hb.dtype_code(x), norm=norm, eps=EPS, rope_dims=dims, rope_first=first, half=half, r=r, mscale=mscale)


def workspace(op, d):
    ws = hb.alloc_workspace(hb.workspace_bytes(op, d))
    ws[256:] = 255                                                # NaN patterns: nothing is read before it is written
    return ws


def check_codes(codes, scales, y, off, g):
    """codes, scales (bytes) of rows y [n, D] known to `off`: each scale a nearest e4m3 to its group's
    largest magnitude / 6 g, each code a nearest 4-bit float to y / (scale g), as far as y is known."""
    n, D = y.shape
    top, slack = y.abs().view(n, -1, 16).amax(-1) / (6 * g), off.view(n, -1, 16).amax(-1) / (6 * g)
    grid = torch.arange(0x7F, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    s = e4m3(scales)
    t = top.clamp(max=448.0)
    best = torch.stack([(grid[i:i + 16] - t[..., None]).abs().amin(-1) for i in range(0, 127, 16)]).amin(0)
    assert ((s - t).abs() <= best + 2 * (slack + 2 * U * top)).all()
    step = (s * g).repeat_interleave(16, -1)
    c = values(codes)
    assert (c[step == 0] == 0).all()
    v = torch.where(step > 0, y / step.clamp_min(1e-300), 0.0)
    d = torch.where(step > 0, off / step.clamp_min(1e-300), 0.0) + 2 * U * v.abs()
    near = torch.stack([(v - f).abs() for f in GRID.tolist()]).amin(0)
    assert ((c - v).abs() <= near + 2 * d).all(), ((c - v).abs() - near - 2 * d).max().item()


def check_appended(x, w, norm, pos, dims, first, half, mscale, cache, scales, place, g):
    y, off = turned(x[:, None], w, norm, pos, dims, first, half, mscale)
    y, off = y[:, 0], off[:, 0]
    if scales is None:
        check_turned(cache.flatten(0, 1)[place], y, off, "bf16")
    else:
        check_codes(cache.flatten(0, 1)[place], scales.flatten(0, 1)[place], y, off, g)


@pytest.mark.parametrize("D,dims,first", [(512, 64, 448), (128, 64, 64), (64, 64, 0), (16, 0, 0), (1024, 128, 512), (240, 48, 192), (272, 30, 5)])
@pytest.mark.parametrize("new,old,page", [([1], [0], 1), ([1] * 9, [5, 0, 63, 64, 65, 7, 100, 1, 2], 64), ([0, 130, 1, 0, 33], [3, 0, 90, 8, 47], 48),
                                          ([700], [0], 100)])
@pytest.mark.parametrize("cache", ["4bit", "bf16"])
@pytest.mark.parametrize("src,half,norm", [("bf16", 0, 1), ("f32", 1, 0)])
def test_append(D, dims, first, new, old, page, cache, src, half, norm):
    B, n = len(new), sum(new)
    if half and dims % 4:
        dims -= 2
    x = randn((n + 5, D), src, 1, 2.0)                            # five rows of padding
    x[n:] = NAN
    w = 1 + randn((D,), "f32", 2, 0.1) if norm else None
    cols = max(-(-(a + b) // page) for a, b in zip(new, old)) + 1
    table, pages = page_tables([a + b for a, b in zip(new, old)], cols, page)
    pool, scales = empty_pool(pages, page, D, cache)
    was, was_s = pool.clone(), None if scales is None else scales.clone()
    d = append_desc(x, pool, B, cols, page, cache, norm, dims, first, half, mscale=1.25)
    ws = workspace(hb.OP_CACHE, d)
    off = torch.tensor([0] + new).cumsum(0).cuda()
    hb.cache_append(d, table_of(dims), x, w, off, ints(old), table, pool, scales, ws)
    assert hb.device_status(ws) == 0
    place, pos = [], []
    for b in range(B):
        i = torch.arange(old[b], old[b] + new[b], device="cuda")
        place.append(slots(table, b, i, page))
        pos.append(4 * i)
    place, pos = torch.cat(place), torch.cat(pos)
    check_appended(x[:n], w, norm, pos, dims, first, half, 1.25, pool, scales, place, 0.75)
    rest = torch.ones(pages * page, dtype=torch.bool, device="cuda")
    rest[place] = False
    assert torch.equal(pool.flatten(0, 1)[rest].view(torch.uint8), was.flatten(0, 1)[rest].view(torch.uint8))
    if scales is not None:
        assert torch.equal(scales.flatten(0, 1)[rest], was_s.flatten(0, 1)[rest])


@pytest.mark.parametrize("ld,skew", [(136, 0), (131, 0), (136, 3)])
@pytest.mark.parametrize("src", ["bf16", "f32"])
def test_append_takes_slices(ld, skew, src):
    buf = torch.full((40 * ld + 8,), NAN, device="cuda", dtype=DT[src])
    x = buf[skew:skew + 40 * ld].view(40, ld)[:, :128]
    x.copy_(randn((40, 128), src, 3))
    table, pages = page_tables([40], 2, 32)
    pool, scales = empty_pool(pages, 32, 128, "4bit")
    d = append_desc(x, pool, 1, 2, 32, "4bit", 1, 64, 64)
    ws = workspace(hb.OP_CACHE, d)
    hb.cache_append(d, table_of(64), x, None, ints([0, 40], torch.int64), ints([0]), table, pool, scales, ws)
    i = torch.arange(40, device="cuda")
    check_appended(x, None, 1, 4 * i, 64, 64, 0, 1.0, pool, scales, slots(table, 0, i, 32), 0.75)


def test_append_special_groups():
    # exact quotients at the middle between two codes go to the even one, on both sides
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    x = torch.zeros((4, 128), device="cuda")
    x[0, :16] = torch.cat([ties, -ties]).cuda() * 0.375 * 1.5    # scale 0.375 at factor 1.5
    x[0, 16:32] = 1e-30                                          # rounds to scale 0
    x[0, 32:48] = 1e30                                           # saturates
    x[0, 33] = -1e30
    x[0, 48] = 2.0**-9 * 6 * 1.5                                 # the least scale
    x[1, 3] = NAN
    x[1, 20], x[1, 40] = math.inf, -math.inf
    x[1, 64:80] = torch.cat([ties, -ties]).cuda() * 64 * 1.5
    x[2] = 3.4e38
    pool, scales = empty_pool(1, 4, 128, "4bit")
    d = append_desc(x, pool, 1, 1, 4, "4bit", g=1.5)
    ws = workspace(hb.OP_CACHE, d)
    hb.cache_append(d, None, x, None, ints([0, 4], torch.int64), ints([0]), ints([[0]]), pool, scales, ws)
    c, s = values(pool[0]), scales[0].view(torch.float8_e4m3fn).float()
    even = torch.tensor([0, 1, 1, 2, 2, 4, 4, 6], device="cuda", dtype=torch.float64)
    assert s[0, 0] == 0.375 and torch.equal(c[0, :16], torch.cat([even, -even]))
    assert s[0, 1] == 0 and (c[0, 16:32] == 0).all()
    assert s[0, 2] == 448 and c[0, 32] == 6 and c[0, 33] == -6 and (c[0, 34:48] == 6).all()
    assert s[0, 3] == 2.0**-9 and c[0, 48] == 6 and (c[0, 49:64] == 0).all()
    assert s[1, :3].isnan().all() and (s[1, 3] == 0).all()
    assert s[1, 4] == 64 and torch.equal(c[1, 64:80], torch.cat([even, -even]))
    assert (s[2] == 448).all() and (c[2] == 6).all()
    assert (s[3] == 0).all() and (c[3] == 0).all()


def test_bad_places_are_left_out():
    page, D = 8, 64
    for cache in ("4bit", "bf16"):
        x = randn((50, D), "bf16", 5)
        pool, scales = empty_pool(6, page, D, cache)
        table = ints([[0, 6, 1], [-1, 2, 3], [4, 5, 1 << 30]])   # sequence 0: a page too far; 1: none; 2: far
        good = torch.zeros(48, dtype=torch.bool, device="cuda")
        d = append_desc(x, pool, 3, 3, page, cache)
        ws = workspace(hb.OP_CACHE, d)
        args = (None, x, None, ints([0, 16, 30, 50], torch.int64), ints([0, 0, 8]), table, pool, scales, ws)
        hb.cache_append(d, *args)
        assert hb.device_status(ws) == hb.DEV_BAD_OFFSETS
        rows = pool_rows(pool, scales, 0.75)
        good[0:8] = True                                         # sequence 0, page 0
        good[16:22] = True                                       # sequence 1, rows 8..13 on page 2
        good[40:48] = True                                       # sequence 2, rows 8..15 on page 5; then past its table
        assert torch.equal(~rows.isnan().any(-1), good)
        out = torch.full((50, D), 5.0, device="cuda")
        hb.workspace_init(ws)
        rd = append_desc(out, pool, 3, 3, page, cache)
        hb.cache_read(rd, *args[3:6], pool, scales, out, ws)
        assert hb.device_status(ws) == hb.DEV_BAD_OFFSETS
        want = torch.zeros(50, dtype=torch.bool, device="cuda")
        want[0:8] = want[24:30] = want[30:38] = True
        assert torch.equal((out != 5.0).any(-1), want)
    # offsets that do not ascend, start below 0 or pass the rows; a negative first row
    for off, first in (([0, 30, 20, 50], [0, 0, 0]), ([-3, 10, 20, 30], [0, 0, 0]), ([0, 10, 20, 60], [0, 0, 0]), ([0, 10, 20, 30], [0, -1, 0])):
        pool, scales = empty_pool(24, page, D, "4bit")
        table = torch.arange(24, device="cuda", dtype=torch.int32).view(3, 8)
        d = append_desc(x, pool, 3, 8, page, "4bit")
        ws = workspace(hb.OP_CACHE, d)
        hb.cache_append(d, None, x, None, ints(off, torch.int64), ints(first), table, pool, scales, ws)
        assert hb.device_status(ws) == hb.DEV_BAD_OFFSETS


def test_append_without_rows():
    pool, scales = empty_pool(2, 4, 64, "4bit")
    d = append_desc(torch.empty((0, 64), device="cuda"), pool, 2, 1, 4, "4bit", ld=64)
    ws = workspace(hb.OP_CACHE, d)
    hb.cache_append(d, None, None, None, None, None, None, pool, scales, ws)
    x = randn((3, 64), "f32", 1)
    d = append_desc(x, pool, 2, 1, 4, "4bit")
    hb.cache_append(d, None, x, None, ints([1, 1, 1], torch.int64), ints([0, 0]), ints([[0], [1]]), pool, scales, ws)
    assert hb.device_status(ws) == 0 and (scales == 0x7F).all()


def random_pool(pages, page, D, cache, seed):
    if cache == "bf16":
        return randn((pages, page, D), "bf16", seed), None
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    codes = torch.randint(0, 256, (pages, page, D // 2), generator=g, device="cuda", dtype=torch.uint8)
    return codes, (torch.rand((pages, page, D // 16), generator=g, device="cuda") * 0.6 + 0.05).to(torch.float8_e4m3fn).view(torch.uint8)


@pytest.mark.parametrize("D", [512, 128, 64, 16, 1024, 240])
@pytest.mark.parametrize("count,first,page", [([1], [0], 1), ([3, 0, 70, 64], [60, 5, 0, 1], 64), ([130, 1], [0, 99], 48)])
@pytest.mark.parametrize("cache,out", [("4bit", "f32"), ("4bit", "bf16"), ("4bit", "e4m3"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("wider", [0, 16])
def test_read(D, count, first, page, cache, out, wider):
    n, B = sum(count), len(count)
    cols = max(-(-(a + b) // page) for a, b in zip(count, first))
    table, pages = page_tables([a + b for a, b in zip(count, first)], cols, page)
    pool, scales = random_pool(pages, page, D, cache, 7)
    buf = torch.full((n + 4, D + wider), 9.0, device="cuda").to(DT[out])
    d = hb.CacheDesc(pages=pages, page_rows=page, D=D, cache_dtype=CODE[cache], cache_scale=0.3, B=B, table_cols=cols, rows=n + 4,
                     ld=D + wider, io_dtype=CODE[out])
    ws = workspace(hb.OP_CACHE, d)
    off = torch.tensor([2] + count).cumsum(0).cuda()              # two rows before the first, two behind the last
    out_scales = torch.full((n + 4, D // 16), 9.0, device="cuda") if out == "e4m3" else None
    hb.cache_read(d, off, ints(first), table, pool, scales, buf, ws, out_scales)
    assert hb.device_status(ws) == 0
    place = torch.cat([slots(table, b, torch.arange(first[b], first[b] + count[b], device="cuda"), page) for b in range(B)])
    got = buf[2:2 + n, :D]
    if out == "e4m3":
        assert torch.equal(got.double(), values(pool.flatten(0, 1)[place]))
        want = e4m3(scales.flatten(0, 1)[place]) * 0.3
        assert ((out_scales[2:2 + n].double() - want).abs() <= 2 * U * want).all()
        assert (out_scales[:2] == 9).all() and (out_scales[2 + n:] == 9).all()
    else:
        want = pool_rows(pool, scales, 0.3)[place]                # the factor as f32, two products, the output's rounding
        assert ((got.double() - want).abs() <= want.abs() * (3 * U + (half_step("bf16") if out == "bf16" else 0))).all()
        if cache == "bf16":
            assert torch.equal(got.double(), want)
    buf[2:2 + n, :D] = 9.0
    assert (buf.float() == 9.0).all()


def test_pages_past_32_bits():
    page, D = 64, 512
    pages = (1 << 32) // (page * D // 2) + 40                     # past 2^32 bytes of codes
    pool = torch.empty((pages, page, D // 2), device="cuda", dtype=torch.uint8)
    scales = torch.empty((pages, page, D // 16), device="cuda", dtype=torch.uint8)
    x = randn((100, D), "bf16", 5)
    table = ints([[pages - 1, pages - 2]])
    d = append_desc(x, pool, 1, 2, page, "4bit", 1, 64, 448)
    ws = workspace(hb.OP_CACHE, d)
    off, first = ints([0, 100], torch.int64), ints([0])
    hb.cache_append(d, table_of(64), x, None, off, first, table, pool, scales, ws)
    i = torch.arange(100, device="cuda")
    y, e = turned(x[:, None], None, True, 4 * i, 64, 448, 0)
    at = table[0].long()[i // page], i % page
    check_codes(pool[at], scales[at], y[:, 0], e[:, 0], 0.75)
    out = torch.empty((100, D), device="cuda")
    hb.cache_read(append_desc(out, pool, 1, 2, page, "4bit"), off, first, table, pool, scales, out, ws)
    want = values(pool[at]) * (e4m3(scales[at]) * 0.75).repeat_interleave(16, -1)
    assert ((out.double() - want).abs() <= 3 * U * want.abs()).all()
    # and the combine reads them there
    c = attend_case([100], 1, 64, "4bit", "bf16", page)
    c.update(pool=pool, scales=scales, table=table, cols=2, pages=pages, g=0.75)
    out, ws = run_attend(c, "f32")
    assert hb.device_status(ws) == 0
    check_attend(c, out, "f32", rows=lambda b, place: values(pool[at]) * (e4m3(scales[at]) * 0.75).repeat_interleave(16, -1))


# ------------------------------------------------------------------------------------
# the combine over a cache in pages
# ------------------------------------------------------------------------------------
DIMS = {64: 512, 16: 128, 8: 64}


def attend_case(lens, L, H, cache, q, page, select=0, seed=0, window=128, W=None, t0=None, q_std=2.0, g=0.75, cols=None):
    """Sequences of `lens` pooled rows. Rows that no query may read hold NaN: the ends of the window
    buffers and of the last pages, and the pages of nobody."""
    B, Dh = len(lens), DIMS[H]
    W = window + L - 1 if W is None else W
    cols = max(1, max(-(-n // page) for n in lens)) if cols is None else cols
    table, pages = page_tables(lens, cols, page, seed=seed)
    pool, scales = empty_pool(pages, page, Dh, cache)
    full, full_s = random_pool(pages, page, Dh, cache, seed + 2)
    for b, n in enumerate(lens):
        at = slots(table, b, torch.arange(n, device="cuda"), page)
        pool.view(pages * page, -1)[at] = full.view(pages * page, -1)[at]
        if scales is not None:
            scales.view(pages * page, -1)[at] = full_s.view(pages * page, -1)[at]
    c = dict(B=B, L=L, H=H, Dh=Dh, W=W, window=window, cache=cache, qt=q, page=page, table=table, cols=cols, pages=pages, pool=pool,
             scales=scales, g=g, Np_max=max(lens), lens=lens, k=select, I=None)
    c["q"] = randn((B, L, H, Dh), q, seed, q_std)
    c["local"] = randn((B, W, Dh), q, seed + 3)
    c["sinks"] = randn((H,), "f32", seed + 4) + 2.0
    t = [4 * n - L if t0 is None else t0 for n in lens]
    n_loc = [max(0, min(W, x + L)) for x in t]
    for b in range(B):
        c["local"][b, n_loc[b]:] = NAN
    c["len"], c["pos0"] = ints(n_loc), ints([x + L - n for x, n in zip(t, n_loc)])
    c["t0"], c["count"] = ints(t), ints(lens)
    if select:
        gen = torch.Generator()
        gen.manual_seed(seed + 9)
        I = torch.full((B, L, select), -1, dtype=torch.int32)
        for b, n in enumerate(lens):
            for j in range(L):
                m = min(n, select)
                I[b, j, torch.randperm(select, generator=gen)[:m]] = torch.randperm(n, generator=gen)[:m].to(torch.int32)
        c["I"] = I.cuda()
    return c


def run_attend(c, out_dt, ws=None, stream=None, sinks="own", out=None, flags=0):
    d = hb.CacheAttnDesc(B=c["B"], L=c["L"], H=c["H"], Dh=c["Dh"], window=c["window"], W_max=c["W"], r=4, k=c["k"], page_rows=c["page"],
                         table_cols=c["cols"], pages=c["pages"], Np_max=c["Np_max"], scale=0.0, cache_scale=c["g"], q_dtype=CODE[c["qt"]],
                         cache_dtype=CODE[c["cache"]], out_dtype=CODE[out_dt], flags=flags)
    if ws is None:
        ws = workspace(hb.OP_CACHE_ATTEND, d)
    if out is None:
        out = torch.full((c["B"], c["L"], c["H"], c["Dh"]), NAN, device="cuda", dtype=DT[out_dt])
    hb.cache_attend(d, c["q"], c["local"] if c["W"] else None, c["len"], c["pos0"], c["pool"], c["scales"], c["table"], c["count"], c["I"],
                    c["sinks"] if isinstance(sinks, str) else sinks, c["t0"], out, ws, stream=stream)
    return out, ws


def check_attend(c, out, out_dt, sinks="own", rows=None, skip=None, weight=None):
    """Logits: Dh products summed in f32, off by e = Dh u scale sum|q k| + 4 u |z|; rows in 4 bits by 2 u
    of theirs; weights by 2 e, and their f32 sums over n rows by n u. bf16 queries may round each weight
    to bf16 (2^-8) before its product with the values."""
    sinks = c["sinks"] if isinstance(sinks, str) else sinks
    scale = c["Dh"] ** -0.5
    if rows is None:
        every = pool_rows(c["pool"], c["scales"], c["g"])
        rows = lambda b, place: every[place]  # noqa: E731
    for b in range(c["B"]):
        for j in range(c["L"]):
            t, n, p0 = int(c["t0"][b]) + j, int(c["len"][b]), int(c["pos0"][b])
            loc = [s for s in range(n) if 0 <= t - (p0 + s) < c["window"]]
            seen = c["lens"][b] if c["L"] == 1 else max(0, min(c["lens"][b], (t + 1) // 4))
            i = torch.arange(seen, device="cuda")
            if c["I"] is not None:
                i = c["I"][b, j].long()
                i = i[(i >= 0) & (i < seen)]
            if skip is not None:
                i = i[~skip(b, i)]
            v = torch.cat([c["local"][b, loc].double(), rows(b, slots(c["table"], b, i, c["page"]))])
            q, got = c["q"][b, j].double(), out[b, j].double()
            s = torch.full((c["H"],), -math.inf, device="cuda", dtype=torch.float64) if sinks is None else sinks.double()
            if v.shape[0] == 0:
                assert (got == 0).all()
                continue
            z = q @ v.t() * scale
            e = ((c["Dh"] + 2) * U * (q.abs() @ v.abs().t() * scale) + 4 * U * z.abs()).amax(-1, keepdim=True)
            p = torch.softmax(torch.cat([z, s[:, None]], -1), -1)[:, :-1]
            want, mag = p @ v, p @ v.abs()
            # weights w (1 + d) with |d| <= r, in the sum and in the normaliser: off by the sum of w d (v - out), so
            # by r (mag + |out|) at most
            r = weight if weight is not None else half_step("bf16") if c["qt"] == "bf16" else 0
            tol = mag * (4 * e + (2 * v.shape[0] + 2) * U + r) + want.abs() * (r + half_step(out_dt)) + 1e-37
            err = (got - want).abs()
            assert (err <= tol).all(), (b, j, (err / tol).max().item())


LENS = [[0], [1], [5, 0, 70], [130, 64, 1, 63, 200, 65], [33] * 9]


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("L", [1, 3])
@pytest.mark.parametrize("H,q", [(64, "bf16"), (64, "f32"), (16, "bf16"), (16, "f32"), (8, "bf16"), (8, "f32")])
@pytest.mark.parametrize("cache,page", [("4bit", 64), ("bf16", 48), ("4bit", 1)])
@pytest.mark.parametrize("select", [0, 40])
def test_attend(lens, L, H, q, cache, page, select):
    c = attend_case(lens, L, H, cache, q, page, select)
    for out_dt in ("f32", "bf16"):
        out, ws = run_attend(c, out_dt)
        assert hb.device_status(ws) == 0
        check_attend(c, out, out_dt)


@pytest.mark.parametrize("H,q", [(64, "bf16"), (16, "f32")])
@pytest.mark.parametrize("lens,select", [([5000, 3000, 1, 4097], 0), ([20001], 0), ([40000], 600), ([700] * 160, 0), ([300] * 200, 200), ([1500] * 310, 512)])
@pytest.mark.parametrize("cache", ["4bit", "bf16"])
def test_attend_long(H, q, lens, select, cache):
    c = attend_case(lens, 1, H, cache, q, 64, select, seed=5)
    out, ws = run_attend(c, "f32")
    assert hb.device_status(ws) == 0
    check_attend(c, out, "f32")


@pytest.mark.parametrize("H,q", [(64, "bf16"), (16, "bf16"), (8, "f32")])
@pytest.mark.parametrize("window,W,t0", [(0, 0, None), (128, 0, None), (0, 5, None), (7, 20, 3), (64, 64, 63), (128, 131, 1), (200, 300, 5000), (1000, 1500, 4000)])
def test_attend_windows(H, q, window, W, t0):
    c = attend_case([9, 0, 77], 2, H, "4bit", q, 16, window=window, W=W, t0=t0, seed=3)
    out, ws = run_attend(c, "f32")
    assert hb.device_status(ws) == 0
    check_attend(c, out, "f32")


@pytest.mark.parametrize("H,q", [(64, "bf16"), (64, "f32"), (16, "bf16"), (8, "f32")])
@pytest.mark.parametrize("cache", ["4bit", "bf16"])
def test_attend_sees_nothing(H, q, cache):
    # a window that holds nothing yet, no rows, no sinks; ids that are all skipped or masked
    c = attend_case([0, 6, 0], 2, H, cache, q, 8, window=128, t0=-3)
    out, ws = run_attend(c, "f32", sinks=None)
    assert hb.device_status(ws) == 0 and (out == 0).all()
    out, _ = run_attend(c, "bf16")
    assert (out == 0).all()
    c = attend_case([30, 30], 1, H, cache, q, 8, select=8, window=0)
    c["I"].fill_(-1)
    out, ws = run_attend(c, "f32", sinks=None)
    assert hb.device_status(ws) == 0 and (out == 0).all()
    out, _ = run_attend(c, "f32", sinks=torch.full((c["H"],), -math.inf, device="cuda"))
    assert (out == 0).all()


@pytest.mark.parametrize("H,q", [(64, "bf16"), (16, "f32")])
def test_attend_sinks(H, q):
    c = attend_case([50, 3], 1, H, "4bit", q, 16)
    c["sinks"][::2] = -math.inf
    c["sinks"][1] = 80.0
    out, _ = run_attend(c, "f32")
    check_attend(c, out, "f32")
    out, _ = run_attend(c, "f32", sinks=None)
    check_attend(c, out, "f32", sinks=None)


@pytest.mark.parametrize("H,q", [(64, "bf16"), (16, "f32")])
@pytest.mark.parametrize("cache", ["4bit", "bf16"])
def test_attend_large_logits_that_grow(H, q, cache):
    # the running maximum moves up many times along the list
    c = attend_case([900], 1, H, cache, q, 64, window=0, q_std=1.0)
    grow = torch.linspace(0.1, 6.0, 900, device="cuda")
    at = slots(c["table"], 0, torch.arange(900, device="cuda"), 64)
    base = randn((c["Dh"],), "f32", 3)
    if cache == "bf16":
        c["pool"].view(-1, c["Dh"])[at] = (base * grow[:, None]).to(torch.bfloat16)
    else:
        c["scales"].view(-1, c["Dh"] // 16)[at] = (grow[:, None] / 6).to(torch.float8_e4m3fn).expand(-1, c["Dh"] // 16).contiguous().view(torch.uint8)
    out, _ = run_attend(c, "f32")
    check_attend(c, out, "f32")


@pytest.mark.parametrize("H,q", [(64, "bf16"), (16, "f32")])
@pytest.mark.parametrize("cache", ["4bit", "bf16"])
def test_attend_scale_range(H, q, cache):
    # every scale of type e4m3 from the least to the largest, with a factor that brings the rows back
    if cache == "bf16":
        c = attend_case([127], 1, H, cache, q, 64, q_std=0.01)
    else:
        c = attend_case([127], 1, H, cache, q, 64, window=0, g=2.0**-8, q_std=1.0)
        at = slots(c["table"], 0, torch.arange(127, device="cuda"), 64)
        c["scales"].view(-1, c["Dh"] // 16)[at] = torch.arange(127, device="cuda", dtype=torch.uint8)[:, None].expand(-1, c["Dh"] // 16)
    out, _ = run_attend(c, "f32")
    check_attend(c, out, "f32")


@pytest.mark.parametrize("H,q", [(64, "bf16"), (64, "f32"), (16, "bf16")])
@pytest.mark.parametrize("lens,select", [([70, 0, 130], 0), ([900, 400], 200), ([9000, 5000], 0)])
@pytest.mark.parametrize("cache", ["4bit", "bf16"])
def test_attend_f32_output_keeps_the_weights(H, q, lens, select, cache):
    # bf16 queries with an output in f32: a weight is off by 2^-22, its exponential's error; all else is f32 too
    c = attend_case(lens, 1, H, cache, q, 16, select, seed=8)
    out, ws = run_attend(c, "f32")
    assert hb.device_status(ws) == 0
    check_attend(c, out, "f32", weight=2.0**-22)


@pytest.mark.parametrize("H,q", [(64, "bf16"), (64, "f32"), (16, "bf16")])
@pytest.mark.parametrize("W", [0, 128])
def test_attend_ids_of_no_rows(H, q, W):
    c = attend_case([70, 5], 1, H, "4bit", q, 16, W=W, seed=3)
    c["I"] = torch.empty((2, 1, 0), dtype=torch.int32, device="cuda")
    out, ws = run_attend(c, "f32")
    assert hb.device_status(ws) == 0
    check_attend(c, out, "f32")


@pytest.mark.parametrize("H,q", [(64, "bf16"), (64, "f32"), (16, "bf16"), (8, "f32")])
@pytest.mark.parametrize("power", [-60, -7, 60])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_attend_cache_scale(H, q, power, out):
    # factors at the ends of their range, with queries that bring the logits back; a window of ordinary rows beside them
    c = attend_case([200, 50], 1, H, "4bit", q, 16, q_std=2.0**-power, g=2.0**power, seed=6)
    if power > 0:
        c["len"].zero_()                                         # rows that queries this small could not tell apart
    else:
        c["local"] *= 2.0**power
    got, ws = run_attend(c, out)
    assert hb.device_status(ws) == 0
    check_attend(c, got, out)


@pytest.mark.parametrize("H,q", [(64, "bf16"), (16, "f32")])
@pytest.mark.parametrize("L", [1, 2])
def test_attend_nan_stays_in_its_sequence(H, q, L):
    c = attend_case([70, 80, 90], L, H, "4bit", q, 16)
    want, _ = run_attend(c, "f32")
    row = slots(c["table"], 1, torch.tensor([3], device="cuda"), 16)
    c["scales"].view(-1, c["Dh"] // 16)[row, 0] = 0x7F
    out, ws = run_attend(c, "f32")
    assert hb.device_status(ws) == 0
    assert torch.equal(out[0], want[0]) and torch.equal(out[2], want[2]) and out[1].isnan().all()


@pytest.mark.parametrize("H,q", [(64, "bf16"), (16, "f32")])
@pytest.mark.parametrize("cache", ["4bit", "bf16"])
def test_attend_bad_places_are_skipped(H, q, cache):
    c = attend_case([70, 80, 90], 1, H, cache, q, 16)
    c["table"][0, 1], c["table"][2, 5] = -1, c["pages"]          # rows 16..31 and 80..89
    out, ws = run_attend(c, "f32")
    assert hb.device_status(ws) == hb.DEV_BAD_OFFSETS
    c2 = dict(c, table=c["table"].clamp(0, c["pages"] - 1))
    check_attend(c2, out, "f32", skip=lambda b, i: ((i // 16 == 1) & (b == 0)) | ((i // 16 == 5) & (b == 2)))
    # lengths that do not fit: that sequence has none
    for bad in (-1, 91, 1 << 30):
        c = attend_case([70, 80, 90], 1, H, cache, q, 16)
        c["count"][1] = bad
        out, ws = run_attend(c, "f32")
        assert hb.device_status(ws) == hb.DEV_BAD_OFFSETS
        check_attend(dict(c, lens=[70, 0, 90]), out, "f32")
    # ids out of range are skipped
    c = attend_case([70, 80, 90], 1, H, cache, q, 16, select=20)
    c["I"][0, 0, 3], c["I"][1, 0, 0], c["I"][2, 0, 19] = 70, -2, 1 << 30
    out, ws = run_attend(c, "f32")
    assert hb.device_status(ws) == hb.DEV_BAD_ID
    check_attend(c, out, "f32")


@pytest.mark.parametrize("H,q", [(64, "bf16"), (16, "f32")])
def test_attend_shared_pages_and_repeated_ids(H, q):
    c = attend_case([60, 60], 1, H, "4bit", q, 16, select=30)
    c["table"][1] = c["table"][0]
    c["I"][1, 0, 5:9] = c["I"][1, 0, 4]                          # the same row five times: five entries
    out, ws = run_attend(c, "f32")
    assert hb.device_status(ws) == 0
    check_attend(c, out, "f32")


@pytest.mark.parametrize("H,q", [(64, "bf16"), (16, "f32")])
def test_attend_same_bits_and_workspace_reuse(H, q):
    big = attend_case([3000, 10, 900], 1, H, "4bit", q, 64)
    small = attend_case([5, 300], 2, H, "4bit", q, 64, seed=4)
    first, ws = run_attend(big, "bf16")
    alone, _ = run_attend(small, "f32")
    need = max(ws.numel(), 1 << 26)
    ws = hb.alloc_workspace(need)
    ws[256:] = 255
    for _ in range(3):
        assert torch.equal(run_attend(big, "bf16", ws=ws)[0], first)
        assert torch.equal(run_attend(small, "f32", ws=ws)[0], alone)


def test_streams_and_graphs():
    c = attend_case([300, 0, 70, 64], 1, 64, "4bit", "bf16", 16)
    d = attend_case([33, 90], 1, 16, "bf16", "f32", 16)
    x, pos = randn((4, 9, 512), "bf16", 1), positions(4)
    y, want_y = torch.zeros_like(x), torch.zeros_like(x)
    rows = randn((2, 512), "bf16", 4)
    ad = append_desc(rows, c["pool"], 2, c["cols"], 16, "4bit", 1, 64, 448)
    aws = workspace(hb.OP_CACHE, ad)
    off, first, turns = ints([0, 1, 2], torch.int64), ints([299, 0]), table_of(64)
    tab = torch.stack([c["table"][0], c["table"][2]])
    read = torch.zeros((2, 512), device="cuda")
    rd = append_desc(read, c["pool"], 2, c["cols"], 16, "4bit")
    nd = hb.NormRopeDesc(tokens=4, heads=9, heads2=0, D=512, norm=1, rope_dims=64, rope_first=448, src_dtype=hb.HISA_BF16,
                         dst_dtype=hb.HISA_BF16, eps=EPS, mscale=1.0, x_token=9 * 512, x_head=512, y_token=9 * 512, y_head=512)
    out, out2 = (torch.zeros((t["B"], 1, t["H"], t["Dh"]), device="cuda") for t in (c, d))
    wc, wd = run_attend(c, "f32")[1], run_attend(d, "f32")[1]

    def calls():
        hb.norm_rope(nd, turns, pos, x, None, y)
        hb.cache_append(ad, turns, rows, None, off, first, tab, c["pool"], c["scales"], aws)
        hb.cache_read(rd, off, first, tab, c["pool"], c["scales"], read, aws)
        run_attend(c, "f32", ws=wc, out=out)
        run_attend(d, "f32", ws=wd, out=out2)

    calls()
    torch.cuda.synchronize()
    want = [t.clone() for t in (y, read, out, out2)]
    check_attend(c, out, "f32")

    def check():
        for t, w in zip((y, read, out, out2), want):
            assert torch.equal(t, w)
            t.zero_()

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    check()
    s.wait_stream(torch.cuda.current_stream())
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


def test_calls_follow_one_another():
    # appended rows are seen by the combine that is enqueued right behind, at every step
    B, H, Dh, page, steps = 3, 64, 512, 16, 40
    table, pages = page_tables([steps] * B, 3, page)
    pool, scales = empty_pool(pages, page, Dh, "4bit")
    rows = randn((steps, B, Dh), "bf16", 1)
    q = randn((steps, B, 1, H, Dh), "bf16", 2, 2.0)
    off, turns = torch.arange(B + 1, device="cuda"), table_of(64)
    d = append_desc(rows[0], pool, B, 3, page, "4bit", 1, 64, 448, r=1, g=1.0)
    ad = hb.CacheAttnDesc(B=B, L=1, H=H, Dh=Dh, window=0, W_max=0, r=1, k=0, page_rows=page, table_cols=3, pages=pages, Np_max=steps,
                          scale=0.0, cache_scale=1.0, q_dtype=hb.HISA_BF16, cache_dtype=hb.HISA_E2M1, out_dtype=hb.HISA_F32)
    ws, aws = workspace(hb.OP_CACHE, d), workspace(hb.OP_CACHE_ATTEND, ad)
    outs = torch.full((steps, B, 1, H, Dh), NAN, device="cuda")
    first, count, t0 = torch.zeros(B, device="cuda", dtype=torch.int32), torch.ones(B, device="cuda", dtype=torch.int32), ints([0] * B)
    for n in range(steps):
        hb.cache_append(d, turns, rows[n], None, off, first, table, pool, scales, ws)
        hb.cache_attend(ad, q[n], None, None, None, pool, scales, table, count, None, None, t0, outs[n], aws)
        first += 1
        count += 1
    assert hb.device_status(ws) == 0 and hb.device_status(aws) == 0
    every = pool_rows(pool, scales, 1.0)
    for n in (0, 1, 15, 16, 39):
        for b in range(B):
            v = every[slots(table, b, torch.arange(n + 1, device="cuda"), page)]
            p = torch.softmax(q[n, b, 0].double() @ v.t() / math.sqrt(Dh), -1)
            err = (outs[n, b, 0].double() - p @ v).abs()
            assert (err <= (p @ v.abs()) * (half_step("bf16") + 1e-3)).all()


# ------------------------------------------------------------------------------------
# together: a layer's decode step
# ------------------------------------------------------------------------------------
@pytest.mark.parametrize("batch,pooled,hidden,steps,select,bits4,page", [(5, 300, 1024, 9, 0, True, 64), (3, 70, 1000, 6, 0, False, 16),
                                                                          (9, 900, 1024, 5, 128, True, 48), (2, 10, 512, 5, 64, False, 1)])
def test_paged_decode(batch, pooled, hidden, steps, select, bits4, page):
    # Queries and rows, the weights of the softmax, and the output are each rounded to bf16 (half a
    # step, 2^-8 of a value at most); normed queries of weight 2 give logits of about 2 standard deviations, up to
    # 10, whose share turns into 2 * 2^-8 * 10 of the weights. The last rotation rounds once more. All of it
    # stays below a tenth of the largest output.
    import os
    import sys

    import deepseek_sparse_attention_hisa_gb300 as pkg
    root = os.path.dirname(os.path.dirname(os.path.abspath(pkg.__file__)))
    sys.path.insert(0, os.path.join(root, "examples"))
    import paged_decode
    assert paged_decode.run(batch, pooled, hidden, steps, select, bits4, page, say=lambda *_: None) < 0.1


# ------------------------------------------------------------------------------------
# what offsets that do not fit leave in the cache, and in the rows read
# ------------------------------------------------------------------------------------
FAR = 1 << 62
BAD_OFFSETS = [
    # offsets, first rows; the packed rows that have a place, with their sequence
    ([-3, 10, 20, 30], [0, 0, 0], {n: n // 10 for n in range(10, 30)}),
    ([-FAR, 10, 20, 30], [0, 0, 0], {n: n // 10 for n in range(10, 30)}),
    ([-2 * FAR, 10, 20, 30], [5, 0, 0], {n: n // 10 for n in range(10, 30)}),
    ([0, 10, 20, 60], [0, 0, 0], {n: n // 10 for n in range(20)}),
    ([0, 10, 20, FAR], [0, 0, 0], {n: n // 10 for n in range(20)}),
    ([0, 10, 20, 30], [0, -1, 0], {n: n // 10 for n in (*range(10), *range(20, 30))}),
    ([0, 10, -2 * FAR, 30], [0, 0, 0], {n: 0 for n in range(10)}),
    ([40, 30, 20, 10], [0, 0, 0], {}),
]


@pytest.mark.parametrize("off,first,rows", BAD_OFFSETS)
@pytest.mark.parametrize("cache", ["4bit", "bf16"])
def test_offsets_that_do_not_fit_leave_their_rows_out(off, first, rows, cache):
    page, D, n = 8, 64, 50
    x = randn((n, D), "bf16", 5)
    pool, scales = empty_pool(24, page, D, cache)
    table = torch.arange(24, device="cuda", dtype=torch.int32).view(3, 8)
    d = append_desc(x, pool, 3, 8, page, cache)
    ws = workspace(hb.OP_CACHE, d)
    off, first = ints(off, torch.int64), ints(first)
    hb.cache_append(d, None, x, None, off, first, table, pool, scales, ws)
    assert hb.device_status(ws) == hb.DEV_BAD_OFFSETS
    want = torch.zeros(24 * page, dtype=torch.bool, device="cuda")
    for i, b in rows.items():
        want[64 * b + int(first[b]) + i - int(off[b])] = True
    assert torch.equal(~pool_rows(pool, scales, 0.75).isnan().any(-1), want)
    full, full_s = random_pool(24, page, D, cache, 3)
    out = torch.full((n, D), NAN, device="cuda")
    hb.workspace_init(ws)
    hb.cache_read(append_desc(out, pool, 3, 8, page, cache), off, first, table, full, full_s, out, ws)
    assert hb.device_status(ws) == hb.DEV_BAD_OFFSETS
    assert (~out.isnan().any(-1)).nonzero().flatten().tolist() == sorted(rows)


@pytest.mark.parametrize("cache", ["4bit", "bf16"])
def test_offsets_that_go_back(cache):
    # rows 20 to 29 lie in sequences 0 and 2: each goes to one of them, or to none; all others have their place
    page, D, n = 8, 64, 50
    x = randn((n, D), "bf16", 5)
    pool, scales = empty_pool(24, page, D, cache)
    table = torch.arange(24, device="cuda", dtype=torch.int32).view(3, 8)
    d = append_desc(x, pool, 3, 8, page, cache)
    ws = workspace(hb.OP_CACHE, d)
    hb.cache_append(d, None, x, None, ints([0, 30, 20, 50], torch.int64), ints([0, 0, 0]), table, pool, scales, ws)
    assert hb.device_status(ws) == hb.DEV_BAD_OFFSETS
    there = (~pool_rows(pool, scales, 0.75).isnan().any(-1)).view(3, 64).cpu()
    assert there[0, :20].all() and not there[0, 30:].any() and not there[1].any()
    assert there[2, 10:30].all() and not there[2, 30:].any()
    assert not (there[0, 20:30] & there[2, :10]).any()


@pytest.mark.parametrize("token,head", [(512, 5 * 512), (512, 4 * 512 + 600), (1600, 520), (1536, 1024)])
def test_norm_rope_heads_before_tokens(token, head):
    # tokens within heads, or heads between those of the tokens beside: all apart
    tokens, heads = (5, 3) if token != 1536 else (2, 2)
    buf = torch.full((8 * 5 * 1536,), 7.0, device="cuda", dtype=torch.bfloat16)
    x, pos, w = randn((tokens, heads, 512), "bf16", 2), positions(tokens), 1 + randn((512,), "f32", 3, 0.1)
    y = buf.as_strided((tokens, heads, 512), (token, head, 1))
    run_norm_rope(x, y, pos, 64, 448, 0, w)
    check_turned(y, *turned(x, w, True, pos, 64, 448, 0), "bf16")
    y.fill_(7.0)
    assert (buf == 7.0).all()


@pytest.mark.parametrize("bits4", [True, False])
def test_a_sequence_begins_behind_its_own_rows(bits4):
    # three sequences with unequal rows before them; the second is released, then another takes its place twice. Queries, rows,
    # weights and outputs are rounded to bf16 (2^-8 each, weights by logits up to 10 more): below a tenth of the largest output, where
    # a row too many or too few of the 20 that a window holds shows as several tenths.
    import os
    import sys

    import deepseek_sparse_attention_hisa_gb300 as pkg
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(pkg.__file__))), "examples"))
    from paged_decode import normed, turn

    from deepseek_sparse_attention_hisa_gb300.paged import DH, H, PagedDecode
    B, hidden, window = 3, 512, 20
    w = {"norm": 1 + randn((hidden,), "f32", 1, 0.1), "q": randn((hidden, H * DH), "bf16", 2, hidden**-0.5),
         "kv": randn((hidden, DH), "bf16", 3, hidden**-0.5), "sinks": randn((H,), "f32", 4) + 1, "q_norm": 1 + randn((DH,), "f32", 5, 0.1),
         "kv_norm": 1 + randn((DH,), "f32", 6, 0.1)}
    start = [100, 3, 40]
    recent = [randn((n, DH), "bf16", 7 + n) for n in (19, 3, 30)]
    p = PagedDecode(B, w, start, 12, pages=40, max_rows=30, page_rows=4, window=window, bits4=bits4, recent=recent)
    p.append(randn((35, DH), "bf16", 8, 2.0), [25, 0, 10])
    local, at = [list(x.double()) for x in recent], list(start)

    def begin(b, t, n, seed):
        x = randn((n, DH), "bf16", seed)
        p.admit(b, t, x)
        local[b], at[b] = list(x.double()), t

    for n in range(10):
        if n == 3:
            p.release(1)
        if n == 4:
            begin(1, 50, 0, 0)
            p.append(randn((7, DH), "bf16", 21, 2.0), [0, 7, 0])
        if n == 7:
            begin(1, 9, 9, 22)
        out = p.step(randn((B, hidden), "bf16", 30 + n), randn((B, hidden), "bf16", 50 + n))
        q = normed((p.act @ w["q"]).view(B, H, DH), w["q_norm"])
        kv = normed(p.act @ w["kv"], w["kv_norm"])
        for b in range(B):
            local[b].append(turn(kv[b], at[b], 1).to(torch.bfloat16).double())
            v = torch.cat([torch.stack(local[b][-window:]), p.rows(b, torch.float32).double()])
            z = turn(q[b], at[b], 1).to(torch.bfloat16).double() @ v.t() / math.sqrt(DH)
            pr = torch.softmax(torch.cat([z, w["sinks"].double()[:, None]], -1), -1)[:, :-1]
            want = turn(pr @ v, at[b], -1)
            assert (out[b].double() - want).abs().max() < 0.1 * want.abs().max(), (n, b)
            at[b] += 1
    assert p.status() == 0 and p.lens == [25, 0, 10]


# ------------------------------------------------------------------------------------
# how near the combine's outputs are by norm, and what an f32 output keeps of a weight
# ------------------------------------------------------------------------------------
def wanted(c, b, j):
    """Query row j of sequence b in f64, [H, Dh]."""
    t, n, p0 = int(c["t0"][b]) + j, int(c["len"][b]), int(c["pos0"][b])
    loc = [s for s in range(n) if 0 <= t - (p0 + s) < c["window"]]
    seen = c["lens"][b] if c["L"] == 1 else max(0, min(c["lens"][b], (t + 1) // 4))
    i = torch.arange(seen, device="cuda")
    if c["I"] is not None:
        i = c["I"][b, j].long()
        i = i[(i >= 0) & (i < seen)]
    v = torch.cat([c["local"][b, loc].double(), pool_rows(c["pool"], c["scales"], c["g"])[slots(c["table"], b, i, c["page"])]])
    z = c["q"][b, j].double() @ v.t() * c["Dh"] ** -0.5
    return torch.softmax(torch.cat([z, c["sinks"].double()[:, None]], -1), -1)[:, :-1] @ v


@pytest.mark.parametrize("H,q", [(64, "bf16"), (64, "f32"), (16, "bf16"), (16, "f32"), (8, "bf16")])
@pytest.mark.parametrize("lens,L,select", [([70, 0, 130], 1, 0), ([70, 5, 130], 3, 0), ([900, 400], 1, 200), ([2000, 600], 1, 512), ([9000, 5000], 1, 0)])
@pytest.mark.parametrize("cache", ["4bit", "bf16"])
def test_attend_f32_output_by_norm(H, q, lens, L, select, cache):
    # Twice the 2e-6 of an output's norm that the header gives for 64 bf16 heads (f32 sums of the tensor cores, cut off by up to 2^-23 at
    # each of some 70 steps over 512 rows and a window, half of that in the mean and of a sum that grows). Weights
    # rounded to bf16 alone are 0.6e-3 to 1e-3 off.
    c = attend_case(lens, L, H, cache, q, 16, select, seed=8)
    out, ws = run_attend(c, "f32")
    assert hb.device_status(ws) == 0
    for b in range(c["B"]):
        for j in range(L):
            want = wanted(c, b, j)
            assert (out[b, j].double() - want).norm() <= 4e-6 * want.norm(), (b, j)


@pytest.mark.parametrize("H,q", [(64, "bf16"), (64, "f32"), (16, "bf16"), (8, "bf16")])
@pytest.mark.parametrize("cache", ["4bit", "bf16"])
def test_attend_f32_output_takes_all_of_a_weight(H, q, cache):
    # Two rows: the first has a logit of (h + 1) scale for head h and one dim, the second a logit of 0 and the other dims, all ones, so
    # that an output is w / (1 + w) there, w = exp(-(h + 1) scale), and 1 / (1 + w) in the first dim. The products are exact.
    # The exponent's argument, up to 4.1 in log2 units, carries 4 roundings (scale, log2 e, their product, the sum): 4 * 4.1 ln 2 u
    # = 6.8e-7 of w; the exponential 2^-22; sums, quotient and product 5 u; three sums of planes 2^-23 each: 1.6e-6 in all, below
    # 2^-19. Weights as two bf16 planes would be up to 5e-6 off.
    c = attend_case([2], 1, H, cache, q, 16, window=0, W=0, g=1.0)
    at = slots(c["table"], 0, torch.arange(2, device="cuda"), 16)
    rows = torch.zeros((2, c["Dh"]), device="cuda")
    rows[0, 0] = rows[1, 1:] = 1.0
    if cache == "bf16":
        c["pool"].view(-1, c["Dh"])[at] = rows.to(torch.bfloat16)
    else:
        codes = (rows * 2).to(torch.uint8)                       # code 2 is 1
        c["pool"].view(-1, c["Dh"] // 2)[at] = codes[:, ::2] | codes[:, 1::2] << 4
        c["scales"].view(-1, c["Dh"] // 16)[at] = 0x38
    h = torch.arange(1, H + 1, device="cuda", dtype=torch.float64)
    c["q"].zero_()
    c["q"][0, 0, :, 0] = h.to(DT[q])
    out, ws = run_attend(c, "f32", sinks=None)
    assert hb.device_status(ws) == 0
    w = torch.exp(-h * c["Dh"] ** -0.5)
    if H == 64:
        two = w.float()
        for _ in range(2):
            two = two - two.bfloat16().float()
        assert (two / w).abs().max() > 2.0**-18                 # the inputs tell two planes from three
    want = torch.where(torch.arange(c["Dh"], device="cuda") == 0, (1 / (1 + w))[:, None], (w / (1 + w))[:, None])
    assert ((out[0, 0].double() - want).abs() <= 2.0**-19 * want).all(), ((out[0, 0].double() - want).abs() / want).max().item()


@pytest.mark.parametrize("H,q", [(64, "f32"), (16, "bf16"), (16, "f32"), (8, "bf16"), (8, "f32")])
@pytest.mark.parametrize("lens,L,select", [([130, 64, 1, 0, 200], 1, 0), ([70, 5], 3, 40), ([5000, 3], 1, 0)])
@pytest.mark.parametrize("cache", ["4bit", "bf16"])
def test_attend_bf16_output_is_the_f32_one_rounded(H, q, lens, L, select, cache):
    # on CUDA cores weights and sums are f32 whatever the output's type
    c = attend_case(lens, L, H, cache, q, 16, select, seed=9)
    assert torch.equal(run_attend(c, "bf16")[0], run_attend(c, "f32")[0].bfloat16())


# ------------------------------------------------------------------------------------
# calls that nothing above makes
# ------------------------------------------------------------------------------------
@pytest.mark.parametrize("D,dims,first", [(512, 64, 448), (512, 512, 0), (320, 128, 96), (272, 32, 240), (128, 64, 64), (1024, 128, 512), (272, 28, 5)])
@pytest.mark.parametrize("cache", ["4bit", "bf16"])
@pytest.mark.parametrize("src", ["bf16", "f32"])
def test_append_halves_with_a_norm(D, dims, first, cache, src):
    n, page = 150, 48
    x, w = randn((n, D), src, 1, 2.0), 1 + randn((D,), "f32", 2, 0.3)
    table, pages = page_tables([n + 7], 5, page)
    pool, scales = empty_pool(pages, page, D, cache)
    d = append_desc(x, pool, 1, 5, page, cache, 1, dims, first, 1, mscale=1.25)
    ws = workspace(hb.OP_CACHE, d)
    hb.cache_append(d, table_of(dims), x, w, ints([0, n], torch.int64), ints([7]), table, pool, scales, ws)
    assert hb.device_status(ws) == 0
    i = torch.arange(7, n + 7, device="cuda")
    check_appended(x, w, 1, 4 * i, dims, first, 1, 1.25, pool, scales, slots(table, 0, i, page), 0.75)


@pytest.mark.parametrize("power", [-60, 60])
@pytest.mark.parametrize("like", [True, False])
def test_append_cache_scale(power, like):
    # factors at the ends of their range: rows of their size, and rows of size 1, which saturate or vanish
    x = randn((40, 128), "f32", 3) * (2.0**power if like else 1.0)
    table, pages = page_tables([40], 2, 32)
    pool, scales = empty_pool(pages, 32, 128, "4bit")
    d = append_desc(x, pool, 1, 2, 32, "4bit", 0, 64, 64, g=2.0**power)
    ws = workspace(hb.OP_CACHE, d)
    hb.cache_append(d, table_of(64), x, None, ints([0, 40], torch.int64), ints([0]), table, pool, scales, ws)
    i = torch.arange(40, device="cuda")
    check_appended(x, None, 0, 4 * i, 64, 64, 0, 1.0, pool, scales, slots(table, 0, i, 32), 2.0**power)


def moved(t, by=16):
    """The same tensor `by` bytes past where it would begin."""
    skip = by // t.element_size()
    u = torch.empty(t.numel() + skip, device="cuda", dtype=t.dtype)[skip:].view(t.shape)
    u.copy_(t)
    assert u.data_ptr() % 32 == by % 32
    return u


@pytest.mark.parametrize("H,q", [(64, "bf16"), (64, "f32"), (16, "bf16"), (8, "f32")])
@pytest.mark.parametrize("cache", ["4bit", "bf16"])
def test_attend_tensors_16_bytes_on(H, q, cache):
    c = attend_case([300, 0, 70], 1, H, cache, q, 16, 40)
    want, _ = run_attend(c, "f32")
    d = dict(c, **{k: moved(c[k]) for k in ("q", "local", "pool")}, scales=None if c["scales"] is None else moved(c["scales"]))
    out, ws = run_attend(d, "f32", out=moved(torch.full_like(want, NAN)))
    assert hb.device_status(ws) == 0 and torch.equal(out, want)


@pytest.mark.parametrize("D", [512, 1024, 48])
@pytest.mark.parametrize("cache,out", [("4bit", "f32"), ("4bit", "bf16"), ("4bit", "e4m3"), ("bf16", "f32"), ("bf16", "bf16")])
def test_rows_16_bytes_on(D, cache, out):
    n, page = 100, 16
    table, pages = page_tables([n], 7, page)
    off, first = ints([0, n], torch.int64), ints([0])
    got = []
    for at in (lambda t: t, moved):
        x = at(randn((n, D), "bf16", 4))
        pool, scales = empty_pool(pages, page, D, cache)
        pool, scales = at(pool), None if scales is None else at(scales)
        d = append_desc(x, pool, 1, 7, page, cache, 1, 16, 16)
        ws = workspace(hb.OP_CACHE, d)
        hb.cache_append(d, table_of(16), x, None, off, first, table, pool, scales, ws)
        rows = at(torch.zeros((n, D), device="cuda").to(DT[out]))
        r = hb.CacheDesc(pages=pages, page_rows=page, D=D, cache_dtype=CODE[cache], cache_scale=0.75, B=1, table_cols=7, rows=n, ld=D,
                         io_dtype=CODE[out])
        hb.cache_read(r, off, first, table, pool, scales, rows, ws)
        assert hb.device_status(ws) == 0 and (rows.float() != 0).any()
        got.append(rows.float())
    assert torch.equal(*got)


def test_chained_calls():
    # calls that may overlap the end of the one before them give the same bits
    c = attend_case([300, 0, 70], 1, 64, "4bit", "bf16", 16)
    e = attend_case([300, 0, 70], 1, 16, "bf16", "f32", 16)
    x, pos = randn((4, 9, 512), "bf16", 1), positions(4)
    rows, tab, off, first = randn((2, 512), "bf16", 4), c["table"][:2].contiguous(), ints([0, 1, 2], torch.int64), ints([299, 0])
    tab[1, 0] = c["table"][2, 0]
    got = []
    for flags in (0, hb.FLAG_CHAINED):
        y, read, pool, scales = torch.zeros_like(x), torch.zeros((2, 512), device="cuda"), c["pool"].clone(), c["scales"].clone()
        ad, rd = append_desc(rows, pool, 2, c["cols"], 16, "4bit", 1, 64, 448), append_desc(read, pool, 2, c["cols"], 16, "4bit")
        ad.flags = rd.flags = flags
        ws = workspace(hb.OP_CACHE, ad)
        turns = table_of(64)
        run_norm_rope(x, y, pos, 64, 448, flags=flags)
        hb.cache_append(ad, turns, rows, None, off, first, tab, pool, scales, ws)
        hb.cache_read(rd, off, first, tab, pool, scales, read, ws)
        a, ws2 = run_attend(dict(c, pool=pool, scales=scales), "f32", flags=flags)
        b, ws3 = run_attend(e, "f32", flags=flags)
        assert hb.device_status(ws) == hb.device_status(ws2) == hb.device_status(ws3) == 0
        got.append((y, read, pool, scales, a, b))
    for u, v in zip(*got):
        assert torch.equal(u, v)


def test_paged_decode_combines_what_the_selection_names():
    # the step's selection, then a layer's decode over the rows it names; bounds as in test_a_sequence_begins_behind_its_own_rows
    import os
    import sys

    import deepseek_sparse_attention_hisa_gb300 as pkg
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(pkg.__file__))), "examples"))
    from paged_decode import normed, turn

    from deepseek_sparse_attention_hisa_gb300 import inputs
    from deepseek_sparse_attention_hisa_gb300.paged import DH, H, PagedDecode
    from deepseek_sparse_attention_hisa_gb300.problem import Problem
    B, hidden = 3, 512
    prob = Problem(inputs.generate(inputs.WORKLOADS["ragged_decode"].replace(B=B, Np_range=(1024, 2000), with_attention=False, seed=31)))
    prob.block_means()
    prob.hisa_step()
    have = [int(n) for n in prob.Np]
    w = {"norm": 1 + randn((hidden,), "f32", 1, 0.1), "q": randn((hidden, H * DH), "bf16", 2, hidden**-0.5),
         "kv": randn((hidden, DH), "bf16", 3, hidden**-0.5), "sinks": None, "q_norm": 1 + randn((DH,), "f32", 5, 0.1), "kv_norm": None}
    p = PagedDecode(B, w, [4 * n for n in have], 2, pages=100, max_rows=2000, recent=randn((B, 127, DH), "bf16", 6))
    p.append(randn((sum(have), DH), "bf16", 7, 2.0), have)
    out = p.step(randn((B, hidden), "bf16", 8), randn((B, hidden), "bf16", 9), prob.I)
    assert p.status() == 0 and prob.status() == 0
    q = normed((p.act @ w["q"]).view(B, H, DH), w["q_norm"])
    for b in range(B):
        ids = prob.I[b].long()
        assert (ids >= 0).all() and (ids < have[b]).all() and len(set(ids.tolist())) == 512
        v = torch.cat([p.local[b, :128].double(), p.rows(b, torch.float32).double()[ids]])
        pr = torch.softmax(turn(q[b], 4 * have[b], 1).to(torch.bfloat16).double() @ v.t() / math.sqrt(DH), -1)
        want = turn(pr @ v, 4 * have[b], -1)
        assert (out[b].double() - want).abs().max() < 0.1 * want.abs().max()


# ------------------------------------------------------------------------------------
# long lists in one span: what the tensor cores cut off does not add up
# ------------------------------------------------------------------------------------
def of_the_same_rows(c, B):
    """Case c of one sequence for B queries over its pages, and three of them as a case of their own."""
    d = dict(c, B=B, lens=c["lens"] * B)
    d["q"] = randn((B, *c["q"].shape[1:]), c["qt"], 77, 2.0)
    for k in ("local", "len", "pos0", "t0", "count", "table"):
        d[k] = c[k].expand(B, *c[k].shape[1:]).contiguous()
    if c["I"] is not None:
        d["I"] = c["I"].expand(B, *c["I"].shape[1:]).contiguous()
    pick = [0, B // 2, B - 1]
    some = dict(d, B=3, lens=c["lens"] * 3, **{k: d[k][pick] for k in ("q", "local", "len", "pos0", "t0", "count", "table")})
    return d, some, pick


@pytest.mark.parametrize("B,n", [(160, 600), (160, 769), (160, 3000), (160, 12000), (16, 100000)])
@pytest.mark.parametrize("cache", ["4bit", "bf16"])
def test_attend_f32_output_by_norm_of_long_lists(B, n, cache):
    # as test_attend_f32_output_by_norm: the 3e-6 of the header, and a third of it again. Sums that stayed in the tensor cores' accumulators
    # would be 8e-6 off over 3000 rows.
    c, some, pick = of_the_same_rows(attend_case([n], 1, 64, cache, "bf16", 64, seed=3), B)
    out, ws = run_attend(c, "f32")
    assert hb.device_status(ws) == 0
    for j, b in enumerate(pick):
        want = wanted(some, j, 0)
        assert (out[b, 0].double() - want).norm() <= 4e-6 * want.norm(), b


@pytest.mark.parametrize("cache", ["4bit", "bf16"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("most", [6.0, 60.0])
def test_attend_large_logits_that_grow_over_long_lists(cache, out, most):
    # the running maximum moves between sums that are put by, also by more than f32's exponents span
    c = attend_case([4000], 1, 64, cache, "bf16", 64, window=0, q_std=1.0)
    grow = torch.linspace(0.1, most, 4000, device="cuda")
    at = slots(c["table"], 0, torch.arange(4000, device="cuda"), 64)
    base = randn((512,), "f32", 3)
    if cache == "bf16":
        c["pool"].view(-1, 512)[at] = (base * grow[:, None]).to(torch.bfloat16)
    else:
        c["scales"].view(-1, 32)[at] = (grow[:, None] / 6).to(torch.float8_e4m3fn).expand(-1, 32).contiguous().view(torch.uint8)
    c, some, pick = of_the_same_rows(c, 160)
    got, ws = run_attend(c, out)
    assert hb.device_status(ws) == 0
    check_attend(some, got[pick], out, weight=2.0**-22 if out == "f32" else None)
    again, _ = run_attend(c, out, ws=ws)
    assert torch.equal(again, got)


def test_attend_sums_that_see_nothing_yet():
    # long lists whose first tiles are skipped ids: what is put by is nothing, and what comes later counts
    c = attend_case([3000], 1, 64, "4bit", "bf16", 64, select=2500, window=0)
    c["I"][0, 0, :2000] = -1
    c, some, pick = of_the_same_rows(c, 160)
    some["I"] = c["I"][pick]
    out, ws = run_attend(c, "f32")
    assert hb.device_status(ws) == 0
    for j, b in enumerate(pick):
        want = wanted(some, j, 0)
        assert (out[b, 0].double() - want).norm() <= 4e-6 * want.norm(), b
    c["I"].fill_(-1)
    assert (run_attend(c, "f32", sinks=None)[0] == 0).all()


@pytest.mark.parametrize("H,q", [(64, "bf16")])
def test_attend_two_graphs_share_a_workspace(H, q):
    # two captured calls of different shapes, one workspace, replayed in turn
    a, _, _ = of_the_same_rows(attend_case([2000], 1, H, "4bit", q, 64, seed=3), 20)
    b = attend_case([700, 30, 5000], 1, H, "bf16", q, 16, seed=4)
    want = [run_attend(c, "f32")[0] for c in (a, b)]
    out = [torch.zeros_like(w) for w in want]
    ws = max((run_attend(c, "f32")[1] for c in (a, b)), key=lambda t: t.numel())
    torch.cuda.synchronize()
    graphs = []
    for c, o in zip((a, b), out):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run_attend(c, "f32", ws=ws, out=o)
        graphs.append(g)
    for _ in range(3):
        for g, o, w in zip(graphs, out, want):
            o.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, w)
