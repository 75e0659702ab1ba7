"""Head norms with rotary positions and the cache in pages without a GPU: struct layouts and refusals
(every one returned before anything is enqueued)."""
import ctypes
import os
import shutil
import subprocess

import pytest

from deepseek_sparse_attention_hisa_gb300 import binding as hb
from deepseek_sparse_attention_hisa_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p
FAKE = P(1 << 20)                  # never dereferenced: validation fails first
EINVAL, EDTYPE, EWS = hb.HISA_EINVAL, hb.HISA_EDTYPE, hb.HISA_EWORKSPACE


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return hb.lib()


def heads_desc(**kw):
    d = dict(tokens=4, heads=64, heads2=1, D=512, norm=1, norm2=1, rope_dims=64, rope_first=448, src_dtype=hb.HISA_BF16,
             dst_dtype=hb.HISA_BF16, eps=1e-6, mscale=1.0, x_token=64 * 512, x_head=512, y_token=64 * 512, y_head=512,
             x2_token=512, x2_head=512, y2_token=512, y2_head=512)
    d.update(kw)
    return hb.NormRopeDesc(**d)


def cache_desc(**kw):
    d = dict(pages=10, page_rows=64, D=512, cache_dtype=hb.HISA_E2M1, cache_scale=1.0, B=3, table_cols=4, rows=100, ld=512,
             io_dtype=hb.HISA_BF16, norm=1, eps=1e-6, rope_dims=64, rope_first=448, r=4, mscale=1.0)
    d.update(kw)
    return hb.CacheDesc(**d)


def attn_desc(**kw):
    d = dict(B=2, L=1, H=64, Dh=512, window=128, W_max=128, r=4, k=512, page_rows=64, table_cols=4, pages=10, Np_max=200, scale=0.0,
             cache_scale=1.0, q_dtype=hb.HISA_BF16, cache_dtype=hb.HISA_E2M1, out_dtype=hb.HISA_BF16)
    d.update(kw)
    return hb.CacheAttnDesc(**d)


@pytest.mark.parametrize("name,cls", [("hisa_norm_rope_desc", hb.NormRopeDesc), ("hisa_cache_desc", hb.CacheDesc),
                                      ("hisa_cache_attn_desc", hb.CacheAttnDesc)])
def test_struct_layouts(name, cls, tmp_path):
    gcc = shutil.which("gcc") or shutil.which("cc")
    if gcc is None:
        pytest.skip("no C compiler")
    fields = [f[0] for f in cls._fields_]
    src = '#include <stdio.h>\n#include <stddef.h>\n#include "hisa.h"\nint main(void) {\nprintf("%zu", sizeof(' + name + "));\n"
    src += "".join(f'printf(" %zu", offsetof({name}, {f}));\n' for f in fields) + "return 0;}\n"
    (tmp_path / "p.c").write_text(src)
    subprocess.run([gcc, "-I", os.path.join(ROOT, "include"), str(tmp_path / "p.c"), "-o", str(tmp_path / "p")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "p")], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f in fields]


def test_the_enum_values(tmp_path):
    gcc = shutil.which("gcc") or shutil.which("cc")
    if gcc is None:
        pytest.skip("no C compiler")
    (tmp_path / "p.c").write_text('#include <stdio.h>\n#include "hisa.h"\nint main(void) {printf("%d %d %d", HISA_E2M1, HISA_OP_CACHE, '
                                  "HISA_OP_CACHE_ATTEND); return 0;}\n")
    subprocess.run([gcc, "-I", os.path.join(ROOT, "include"), str(tmp_path / "p.c"), "-o", str(tmp_path / "p")], check=True)
    got = subprocess.run([str(tmp_path / "p")], capture_output=True, text=True, check=True).stdout
    assert got == f"{hb.HISA_E2M1} {hb.OP_CACHE} {hb.OP_CACHE_ATTEND}"


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), EINVAL), (dict(heads=0), EINVAL), (dict(heads2=-1), EINVAL), (dict(D=1), EINVAL), (dict(D=1025), EINVAL),
    (dict(norm=2), EINVAL), (dict(norm2=-1), EINVAL), (dict(rope_dims=63), EINVAL), (dict(rope_dims=-2), EINVAL),
    (dict(rope_dims=514, rope_first=0), EINVAL), (dict(rope_first=449), EINVAL), (dict(rope_first=-1), EINVAL), (dict(half=2), EINVAL),
    (dict(eps=0.0), EINVAL), (dict(eps=float("nan")), EINVAL), (dict(norm=0, eps=0.0), EINVAL), (dict(flags=2), EINVAL),
    (dict(mscale=float("inf")), EINVAL), (dict(src_dtype=hb.HISA_E4M3), EDTYPE), (dict(dst_dtype=hb.HISA_E2M1), EDTYPE),
    (dict(x_token=-1), EINVAL), (dict(dst_dtype=hb.HISA_F32), EINVAL), (dict(y_head=1024), EINVAL), (dict(y2_token=1024), EINVAL),
    (dict(tokens=1 << 31, heads=1), EINVAL), (dict(tokens=(1 << 31) - 1, heads=64), EINVAL)])
def test_norm_rope_refusals(lib, kw, code):
    d = heads_desc(**kw)
    assert lib.hisa_norm_rope(ctypes.byref(d), *[FAKE] * 8, None) == code


def test_norm_rope_refuses_pointers(lib):
    d = heads_desc()
    a = [FAKE] * 8 + [None]                                 # table, pos, x, w, y, x2, w2, y2, stream
    for i in (0, 1, 2, 4, 5, 7):
        b = list(a)
        b[i] = None
        assert lib.hisa_norm_rope(ctypes.byref(d), *b) == EINVAL, i
    for i, off in ((0, 4), (1, 2), (2, 1), (3, 2), (4, 1), (5, 1), (6, 1), (7, 1)):
        b = list(a)
        b[i] = P((1 << 20) + off)
        assert lib.hisa_norm_rope(ctypes.byref(d), *b) == EINVAL, i
    one = heads_desc(heads2=0)                              # a second tensor, or its weights, that are not there
    for i in (5, 6, 7):
        b = [FAKE] * 5 + [None] * 4
        b[i] = FAKE
        assert lib.hisa_norm_rope(ctypes.byref(one), *b) == EINVAL, i
    for kw in (dict(norm=0), dict(norm2=0)):                # weights of a norm that is not taken
        assert lib.hisa_norm_rope(ctypes.byref(heads_desc(**kw)), *a) == EINVAL
    b = list(a)
    b[4] = P(1 << 21)                                       # one tensor in place, the other not
    assert lib.hisa_norm_rope(ctypes.byref(d), *b) == EINVAL
    for kw in (dict(y_head=511), dict(y_token=0), dict(heads2=2, y2_head=0, y2_token=1024)):   # heads that overlap
        b = [FAKE, FAKE, FAKE, None, P(1 << 22), P(1 << 23), None, P(1 << 24), None]
        assert lib.hisa_norm_rope(ctypes.byref(heads_desc(**kw)), *b) == EINVAL, kw
    assert lib.hisa_norm_rope(None, *a) == EINVAL
    assert lib.hisa_norm_rope(ctypes.byref(heads_desc(tokens=0)), *[None] * 9) == hb.HISA_OK


COMMON = [(dict(pages=0), EINVAL), (dict(pages=1 << 31), EINVAL), (dict(page_rows=0), EINVAL), (dict(page_rows=65537), EINVAL),
          (dict(table_cols=0), EINVAL), (dict(cache_dtype=hb.HISA_F32), EDTYPE), (dict(cache_dtype=hb.HISA_E4M3), EDTYPE),
          (dict(cache_scale=0.0), EINVAL), (dict(cache_scale=-1.0), EINVAL), (dict(cache_scale=float("nan")), EINVAL),
          (dict(cache_scale=2.0**61), EINVAL), (dict(B=0), EINVAL), (dict(flags=2), EINVAL)]
ROWS = COMMON + [(dict(D=24), EINVAL), (dict(D=0), EINVAL), (dict(D=1040, ld=1040), EINVAL), (dict(rows=-1), EINVAL), (dict(ld=511), EINVAL)]


@pytest.mark.parametrize("kw,code", ROWS + [
    (dict(io_dtype=hb.HISA_E4M3), EDTYPE), (dict(io_dtype=9), EDTYPE), (dict(norm=2), EINVAL), (dict(eps=0.0), EINVAL), (dict(r=0), EINVAL),
    (dict(mscale=float("nan")), EINVAL), (dict(rope_dims=65), EINVAL), (dict(rope_first=449), EINVAL), (dict(half=-1), EINVAL)])
def test_append_refusals(lib, kw, code):
    d = cache_desc(**kw)
    assert lib.hisa_cache_append(ctypes.byref(d), *[FAKE] * 9, 256, None) == code


@pytest.mark.parametrize("kw,code", ROWS + [(dict(io_dtype=hb.HISA_E2M1), EDTYPE), (dict(cache_dtype=hb.HISA_BF16, io_dtype=hb.HISA_E4M3), EDTYPE),
                                            (dict(ld=516), EINVAL), (dict(io_dtype=hb.HISA_E4M3, ld=520), EINVAL)])
def test_read_refusals(lib, kw, code):
    d = cache_desc(**kw)
    assert lib.hisa_cache_read(ctypes.byref(d), *[FAKE] * 6, None, FAKE, 256, None) == code


@pytest.mark.parametrize("kw,code", ROWS)
def test_workspace_of_bad_descriptors(lib, kw, code):
    assert hb.workspace_bytes(hb.OP_CACHE, cache_desc(**kw)) == 0
    assert hb.workspace_bytes(hb.OP_CACHE, cache_desc()) == 256


def test_append_refuses_pointers(lib):
    d = cache_desc()
    a = [FAKE] * 9                                          # table, x, w, row_off, first, page_table, cache, scales, ws
    call = lambda d, b, n=256: lib.hisa_cache_append(ctypes.byref(d), *b, n, None)  # noqa: E731
    for i in (0, 1, 3, 4, 5, 6, 7):
        b = list(a)
        b[i] = None
        assert call(d, b) == EINVAL, i
    for i, off in ((0, 4), (1, 1), (2, 2), (3, 4), (4, 2), (5, 1), (6, 8), (7, 8)):
        b = list(a)
        b[i] = P((1 << 20) + off)
        assert call(d, b) == EINVAL, i
    assert call(cache_desc(norm=0), a) == EINVAL            # weights without the norm
    assert call(cache_desc(cache_dtype=hb.HISA_BF16), a) == EINVAL     # scales of a bf16 cache
    assert call(d, a, 255) == EWS and call(d, a[:8] + [None]) == EWS and call(d, a[:8] + [P((1 << 20) + 64)]) == EWS
    assert call(cache_desc(rows=0), [None] * 8 + [FAKE]) == hb.HISA_OK
    assert lib.hisa_cache_append(None, *a, 256, None) == EINVAL


def test_read_refuses_pointers(lib):
    d = cache_desc()
    a = [FAKE] * 6 + [None, FAKE]                           # row_off, first, page_table, cache, scales, out, out_scales, ws
    call = lambda d, b, n=256: lib.hisa_cache_read(ctypes.byref(d), *b, n, None)  # noqa: E731
    for i in range(6):
        b = list(a)
        b[i] = None
        assert call(d, b) == EINVAL, i
    for i, off in ((0, 4), (1, 2), (2, 1), (3, 8), (4, 8), (5, 8)):
        b = list(a)
        b[i] = P((1 << 20) + off)
        assert call(d, b) == EINVAL, i
    b = list(a)
    b[6] = FAKE                                             # scales of an output that has none
    assert call(d, b) == EINVAL
    b[6] = P((1 << 20) + 2)
    assert call(cache_desc(io_dtype=hb.HISA_E4M3), b) == EINVAL
    assert call(d, a, 255) == EWS and call(d, a[:7] + [None]) == EWS
    assert lib.hisa_cache_read(None, *a, 256, None) == EINVAL


ATTN = COMMON + [(dict(L=0), EINVAL), (dict(window=-1), EINVAL), (dict(W_max=-1), EINVAL), (dict(r=0), EINVAL), (dict(k=-1), EINVAL),
                 (dict(k=65537), EINVAL), (dict(Np_max=-1), EINVAL), (dict(Np_max=(1 << 31) - 1), EINVAL), (dict(B=1 << 20, L=64), EINVAL),
                 (dict(Np_max=1 << 30, W_max=1 << 30, window=1 << 30), EINVAL), (dict(W_max=(1 << 31) - 1, window=(1 << 31) - 1), EINVAL),
                 (dict(H=32), EDTYPE), (dict(Dh=128), EDTYPE), (dict(q_dtype=hb.HISA_E2M1), EDTYPE), (dict(out_dtype=hb.HISA_E4M3), EDTYPE)]


@pytest.mark.parametrize("kw,code", ATTN)
def test_attend_refusals(lib, kw, code):
    d = attn_desc(**kw)
    assert lib.hisa_cache_attend(ctypes.byref(d), *[FAKE] * 13, 1 << 40, None) == code
    assert hb.workspace_bytes(hb.OP_CACHE_ATTEND, d) == 0


def test_attend_refuses_pointers(lib):
    d = attn_desc()
    need = hb.workspace_bytes(hb.OP_CACHE_ATTEND, d)
    assert need >= 256
    # q, local_kv, local_len, local_pos0, cache, scales, page_table, cache_len, I, sinks, t0, out, ws
    a = [FAKE] * 13
    call = lambda d, b, n=need: lib.hisa_cache_attend(ctypes.byref(d), *b, n, None)  # noqa: E731
    for i in (0, 1, 2, 3, 4, 5, 6, 7, 10, 11):
        b = list(a)
        b[i] = None
        assert call(d, b) == EINVAL, i
    for i, off in ((0, 8), (1, 2), (2, 2), (3, 1), (4, 4), (5, 8), (6, 2), (7, 2), (8, 1), (9, 2), (10, 2), (11, 8)):
        b = list(a)
        b[i] = P((1 << 20) + off)
        assert call(d, b) == EINVAL, i
    assert call(attn_desc(cache_dtype=hb.HISA_BF16), a) == EINVAL
    assert call(d, a, need - 1) == EWS and call(d, a[:12] + [None]) == EWS and call(d, a[:12] + [P((1 << 20) + 16)]) == EWS
    assert lib.hisa_cache_attend(None, *a, need, None) == EINVAL


def test_one_workspace_with_and_without_ids(lib):
    # the size does not depend on whether ids are passed, and sizes past 32 bits are computed in 64
    need = hb.workspace_bytes(hb.OP_CACHE_ATTEND, attn_desc(H=16, Dh=128, B=1, k=0, Np_max=1 << 20, table_cols=1 << 15, pages=1 << 15))
    assert need >= 256 + 64 * 16 * (128 + 2) * 4
    big = hb.workspace_bytes(hb.OP_CACHE_ATTEND, attn_desc(B=1 << 15, L=16, q_dtype=hb.HISA_F32))
    assert big >= (1 << 15) * 16 * 64 * 514 * 4


CUTS = r"""
#include <cstdio>
#include <cstring>
#include "cache_cuts.h"
using namespace hisa;
static int bad = 0;
static void want(bool v, const char *what) { if (!v) { std::printf("%s\n", what); bad = 1; } }
int main() {
    // every tile lies in the span that span_of names
    const int64_t totals[] = {1, 2, 7, 100, 151, 152, 153, 999, 65536, (1 << 24) - 1, 1 << 24, (1 << 24) + 1, (int64_t)1 << 40};
    for (int64_t total : totals)
        for (int groups = 1; groups <= 152 && groups <= total; ++groups) {
            want(span_start(0, total, groups) == 0 && span_start(groups, total, groups) == total, "ends");
            for (int c = 0; c < groups; ++c) {
                const int64_t s0 = span_start(c, total, groups), s1 = span_start(c + 1, total, groups);
                want(s0 < s1 && span_of(s0, total, groups) == c && span_of(s1 - 1, total, groups) == c, "span_of");
            }
        }
    // an entry is used only if it names a row and parts that there are
    const Cut good = {9, 3, 5, 7, {0, 0, 0}};
    want(cut_fits(good, 10, 6), "a good one");
    auto with = [&](int64_t row, int first, int last, int place) { Cut k = good; k.row = row; k.first = first; k.last = last; k.place = place; return cut_fits(k, 10, 6); };
    want(with(0, 0, 0, 0) && with(0, 0, 5, 1) && with(9, 5, 5, 11), "the ends");
    want(!with(-1, 3, 5, 7) && !with(10, 3, 5, 7) && !with((int64_t)1 << 40, 3, 5, 7), "row");
    want(!with(9, -1, 5, 7) && !with(9, 5, 3, 7) && !with(9, 3, 6, 7) && !with(9, 6, 6, 12), "span");
    want(!with(9, 3, 5, 5) && !with(9, 3, 5, 8) && !with(9, 3, 5, -1) && !with(9, 2147483647, 2147483647, 0), "place");
    for (int byte = 1; byte < 256; ++byte) {            // memory that nothing has written
        Cut k;
        std::memset(static_cast<void *>(&k), byte, sizeof k);
        want(!cut_fits(k, 152, 152), "garbage");
    }
    return bad;
}
"""


def test_the_join_takes_addresses_from_entries_that_fit(tmp_path):
    # after a wait that ran out, entries of the list of cuts may hold anything
    gxx = shutil.which("g++") or shutil.which("c++")
    if gxx is None:
        pytest.skip("no C++ compiler")
    (tmp_path / "p.cc").write_text(CUTS)
    subprocess.run([gxx, "-std=c++17", "-O1", "-I", build.CSRC, str(tmp_path / "p.cc"), "-o", str(tmp_path / "p")], check=True)
    r = subprocess.run([str(tmp_path / "p")], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout[:400]


APART = r"""
#include <cstdio>
#include "heads_apart.h"
using namespace hisa;
int main() {
    // against every pair of heads
    for (int64_t w = 1; w <= 4; ++w)
        for (int64_t tokens = 1; tokens <= 5; ++tokens)
            for (int64_t heads = 1; heads <= 4; ++heads)
                for (int64_t token = 0; token <= 26; ++token)
                    for (int64_t head = 0; head <= 26; ++head) {
                        bool apart = true;
                        for (int64_t i = 0; i < tokens * heads && apart; ++i)
                            for (int64_t j = 0; j < i && apart; ++j) {
                                const int64_t d = (i / heads - j / heads) * token + (i % heads - j % heads) * head;
                                apart = d >= w || d <= -w;
                            }
                        if (apart != heads_apart(tokens, heads, token, head, w)) {
                            std::printf("%d x %d, %d and %d apart, %d wide\n", (int)tokens, (int)heads, (int)token, (int)head, (int)w);
                            return 1;
                        }
                    }
    const int64_t far = (int64_t)1 << 40;
    return heads_apart(((int64_t)1 << 31) - 1, 1, 512, far, 512) && heads_apart(1 << 20, 65536, far, 512, 512) &&
           heads_apart(1 << 20, 65536, 512, far, 512) && !heads_apart(1 << 20, 65536, far, far, 512) &&
           !heads_apart(65536, 65536, far - 1, far, 512) ? 0 : 2;
}
"""


def test_strides_that_keep_heads_apart(tmp_path):
    gxx = shutil.which("g++") or shutil.which("c++")
    if gxx is None:
        pytest.skip("no C++ compiler")
    (tmp_path / "p.cc").write_text(APART)
    subprocess.run([gxx, "-std=c++17", "-O1", "-I", build.CSRC, str(tmp_path / "p.cc"), "-o", str(tmp_path / "p")], check=True)
    r = subprocess.run([str(tmp_path / "p")], capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stdout)


# tokens token apart and heads head apart such that a head of one token is one of another's, or overlaps it
CROSSED = [(3, 2, 512, 1024), (2, 3, 1024, 512), (4, 3, 1024, 1536), (3, 8, 700, 1300), (9, 2, 600, 4700)]


@pytest.mark.parametrize("tokens,heads,token,head", CROSSED)
def test_outputs_whose_heads_cross_are_refused(lib, tokens, heads, token, head):
    far = P(1 << 32)
    d = heads_desc(tokens=tokens, heads=heads, heads2=0, y_token=token, y_head=head)
    assert lib.hisa_norm_rope(ctypes.byref(d), FAKE, FAKE, FAKE, None, far, None, None, None, None) == EINVAL
    d = heads_desc(tokens=tokens, heads=1, heads2=heads, y2_token=token, y2_head=head)
    assert lib.hisa_norm_rope(ctypes.byref(d), FAKE, FAKE, FAKE, None, far, FAKE, None, P(1 << 33), None) == EINVAL
    kw = dict(tokens=tokens, heads=heads, heads2=0, D=512, rope_dims=64, rope_first=448, src_dtype=hb.HISA_BF16, dst_dtype=hb.HISA_BF16,
              mscale=1.0, x_token=heads * 512, x_head=512, y_token=token, y_head=head)
    assert lib.hisa_rope(ctypes.byref(hb.RopeDesc(**kw)), FAKE, FAKE, FAKE, far, None, None, None) == EINVAL
    kw.update(x_token=token, x_head=token, y_head=token)   # in place, token after token at the same dims
    assert lib.hisa_rope(ctypes.byref(hb.RopeDesc(**kw)), FAKE, FAKE, FAKE, FAKE, None, None, None) == EINVAL


def test_an_f32_output_of_long_lists_takes_more_workspace():
    # 64 x 512 sums per CTA, where a list may have more than 16 tiles of 48 rows (the window's 3 among them)
    build.build_library()
    need = lambda n, out, B=304: hb.workspace_bytes(hb.OP_CACHE_ATTEND, attn_desc(  # noqa: E731
        B=B, Np_max=n, k=0, table_cols=1 << 12, pages=1 << 12, out_dtype=out))
    assert need(13 * 48, hb.HISA_F32) == need(13 * 48, hb.HISA_BF16)
    assert need(13 * 48 + 1, hb.HISA_F32) == need(13 * 48 + 1, hb.HISA_BF16) + 152 * 64 * 512 * 4
    assert need(1 << 17, hb.HISA_F32, 1) == need(1 << 17, hb.HISA_BF16, 1) + 152 * 64 * 512 * 4
