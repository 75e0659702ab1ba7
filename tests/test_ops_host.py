"""The operators around the step without a GPU: struct layouts, refusals (every one returned
before anything is enqueued) and the rotary frequency table against its definition."""
import ctypes
import math
import os
import shutil
import subprocess

import numpy as np
import pytest

from deepseek_sparse_attention_hisa_gb300 import binding as hb
from deepseek_sparse_attention_hisa_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p
FAKE = P(1 << 20)                  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return hb.lib()


def norm_desc(**kw):
    d = dict(rows=4, cols=4096, x_dtype=hb.HISA_BF16, res_dtype=hb.HISA_BF16, out_dtype=hb.HISA_BF16, eps=1e-6,
             ld_x=4096, ld_res=4096, ld_out=4096)
    d.update(kw)
    return hb.NormDesc(**d)


def rope_desc(**kw):
    d = dict(tokens=4, heads=64, heads2=1, D=512, rope_dims=64, rope_first=448, src_dtype=hb.HISA_BF16,
             dst_dtype=hb.HISA_BF16, mscale=1.0, x_token=64 * 512, x_head=512, y_token=64 * 512, y_head=512,
             x2_token=512, x2_head=512, y2_token=512, y2_head=512)
    d.update(kw)
    return hb.RopeDesc(**d)


def prefix_desc(**kw):
    d = dict(B=2, L=1, H=64, Dh=512, window=128, W_max=128, r=4, prefix_rows=1000, Np_max=100, kv_rows=200, scale=0.0,
             q_dtype=hb.HISA_BF16, kv_dtype=hb.HISA_BF16, out_dtype=hb.HISA_BF16)
    d.update(kw)
    return hb.PrefixDesc(**d)


@pytest.mark.parametrize("name,cls", [("hisa_norm_desc", hb.NormDesc), ("hisa_rope_scaling", hb.RopeScaling),
                                      ("hisa_rope_desc", hb.RopeDesc), ("hisa_prefix_desc", hb.PrefixDesc)])
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


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), hb.HISA_EINVAL), (dict(cols=0), hb.HISA_EINVAL), (dict(cols=32769, ld_x=32769), hb.HISA_EINVAL),
    (dict(eps=0.0), hb.HISA_EINVAL), (dict(eps=float("nan")), hb.HISA_EINVAL), (dict(flags=2), hb.HISA_EINVAL),
    (dict(x_dtype=hb.HISA_E4M3), hb.HISA_EDTYPE), (dict(res_dtype=3), hb.HISA_EDTYPE), (dict(out_dtype=3), hb.HISA_EDTYPE),
    (dict(scale_group=128), hb.HISA_EINVAL), (dict(scale_pow2=1), hb.HISA_EINVAL),
    (dict(out_dtype=hb.HISA_E4M3, scale_group=48), hb.HISA_EINVAL),
    (dict(out_dtype=hb.HISA_E4M3, scale_group=128, cols=4000), hb.HISA_EINVAL),
    (dict(out_dtype=hb.HISA_E4M3, scale_group=128, scale_pow2=2), hb.HISA_EINVAL),
    (dict(out_dtype=hb.HISA_E4M3, scale_group=128), hb.HISA_EINVAL),          # no scales
    (dict(ld_x=4095), hb.HISA_EINVAL), (dict(ld_res=4095), hb.HISA_EINVAL), (dict(ld_out=4095), hb.HISA_EINVAL)])
def test_norm_refusals(lib, kw, code):
    d = norm_desc(**kw)
    assert lib.hisa_rms_norm(ctypes.byref(d), FAKE, FAKE, FAKE, FAKE, FAKE, None, None) == code


def test_norm_refuses_pointers(lib):
    d = norm_desc()
    a = [FAKE, FAKE, FAKE, FAKE, FAKE, None, None]          # x, residual, w, residual_out, out, scales, stream
    for i in (0, 1, 2, 4):                                  # a residual_out without a residual is one
        b = list(a)
        b[i] = None
        assert lib.hisa_rms_norm(ctypes.byref(d), *b) == hb.HISA_EINVAL, i
    for i, off in ((0, 1), (1, 1), (2, 2), (3, 1), (4, 1)):
        b = list(a)
        b[i] = P((1 << 20) + off)
        assert lib.hisa_rms_norm(ctypes.byref(d), *b) == hb.HISA_EINVAL, i
    b = list(a)
    b[5] = FAKE                                             # scales without an 8-bit output
    assert lib.hisa_rms_norm(ctypes.byref(d), *b) == hb.HISA_EINVAL
    f = norm_desc(out_dtype=hb.HISA_F32)                    # in place with another dtype
    assert lib.hisa_rms_norm(ctypes.byref(f), FAKE, None, FAKE, None, FAKE, None, None) == hb.HISA_EINVAL
    assert lib.hisa_rms_norm(None, *a) == hb.HISA_EINVAL
    z = norm_desc(rows=0)
    assert lib.hisa_rms_norm(ctypes.byref(z), None, None, None, None, None, None, None) == hb.HISA_OK


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), hb.HISA_EINVAL), (dict(heads=0), hb.HISA_EINVAL), (dict(heads2=-1), hb.HISA_EINVAL),
    (dict(D=1), hb.HISA_EINVAL), (dict(D=1025), hb.HISA_EINVAL), (dict(rope_dims=63), hb.HISA_EINVAL),
    (dict(rope_dims=0), hb.HISA_EINVAL), (dict(rope_dims=514, rope_first=0), hb.HISA_EINVAL),
    (dict(rope_first=449), hb.HISA_EINVAL), (dict(rope_first=-1), hb.HISA_EINVAL), (dict(half=2), hb.HISA_EINVAL),
    (dict(inverse=-1), hb.HISA_EINVAL), (dict(flags=4), hb.HISA_EINVAL), (dict(mscale=float("inf")), hb.HISA_EINVAL),
    (dict(src_dtype=hb.HISA_E4M3), hb.HISA_EDTYPE), (dict(dst_dtype=7), hb.HISA_EDTYPE), (dict(x_token=-1), hb.HISA_EINVAL),
    (dict(dst_dtype=hb.HISA_F32), hb.HISA_EINVAL),          # in place with another dtype
    (dict(y_head=1024), hb.HISA_EINVAL), (dict(y2_token=1024), hb.HISA_EINVAL)])
def test_rope_refusals(lib, kw, code):
    d = rope_desc(**kw)
    assert lib.hisa_rope(ctypes.byref(d), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None) == code


def test_rope_refuses_pointers(lib):
    d = rope_desc()
    a = [FAKE] * 6 + [None]                                 # table, pos, x, y, x2, y2, stream
    for i in range(6):
        b = list(a)
        b[i] = None
        assert lib.hisa_rope(ctypes.byref(d), *b) == hb.HISA_EINVAL, i
    for i, off in ((0, 4), (1, 2), (2, 1), (3, 1), (4, 1), (5, 1)):
        b = list(a)
        b[i] = P((1 << 20) + off)
        assert lib.hisa_rope(ctypes.byref(d), *b) == hb.HISA_EINVAL, i
    # one tensor in place, the other not; a second tensor that the descriptor does not name
    assert lib.hisa_rope(ctypes.byref(d), FAKE, FAKE, FAKE, FAKE, FAKE, P(1 << 21), None) == hb.HISA_EINVAL
    one = rope_desc(heads2=0)
    assert lib.hisa_rope(ctypes.byref(one), *a) == hb.HISA_EINVAL
    z = rope_desc(tokens=0)
    assert lib.hisa_rope(ctypes.byref(z), None, None, None, None, None, None, None) == hb.HISA_OK


@pytest.mark.parametrize("inplace,kw", [
    (True, dict(x_head=0, y_head=0)), (True, dict(x_head=63, y_head=63)), (True, dict(x_token=0, y_token=0)),
    (True, dict(x_token=512, y_token=512)), (True, dict(x2_token=0, y2_token=0)), (False, dict(y_head=0)), (False, dict(y_head=511)),
    (False, dict(y_token=511)), (False, dict(y_token=512)), (False, dict(heads2=2, y2_head=256, y2_token=1024)),
    (False, dict(heads2=2, y2_head=512, y2_token=512))])
def test_rope_refuses_rows_that_overlap(lib, inplace, kw):
    # a broadcast view rotated in place would turn as often as it repeats, in no order
    d = rope_desc(**kw)
    y = FAKE if inplace else P(1 << 21)
    assert lib.hisa_rope(ctypes.byref(d), FAKE, FAKE, FAKE, y, FAKE, y, None) == hb.HISA_EINVAL


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), hb.HISA_EINVAL), (dict(L=0), hb.HISA_EINVAL), (dict(window=-1), hb.HISA_EINVAL),
    (dict(W_max=-1), hb.HISA_EINVAL), (dict(r=0), hb.HISA_EINVAL), (dict(flags=2), hb.HISA_EINVAL),
    (dict(prefix_rows=-1), hb.HISA_EINVAL), (dict(prefix_rows=1 << 31), hb.HISA_EINVAL), (dict(Np_max=-1), hb.HISA_EINVAL),
    (dict(kv_rows=-1), hb.HISA_EINVAL), (dict(H=32), hb.HISA_EDTYPE), (dict(Dh=128), hb.HISA_EDTYPE),
    (dict(q_dtype=hb.HISA_F32), hb.HISA_EDTYPE), (dict(out_dtype=hb.HISA_E4M3), hb.HISA_EDTYPE)])
def test_prefix_refusals(lib, kw, code):
    d = prefix_desc(**kw)
    assert lib.hisa_prefix_attend(ctypes.byref(d), *[FAKE] * 11, 1 << 30, None) == code
    assert hb.workspace_bytes(hb.OP_PREFIX_ATTEND, d) == 0


def test_prefix_refuses_pointers(lib):
    d = prefix_desc()
    need = hb.workspace_bytes(hb.OP_PREFIX_ATTEND, d)
    assert need >= 256
    # q, local_kv, local_len, local_pos0, prefix_kv, pooled_kv, kv_off, sinks, t0, out, ws
    a = [FAKE] * 11
    for i in (0, 1, 2, 3, 4, 5, 6, 8, 9):
        b = list(a)
        b[i] = None
        assert lib.hisa_prefix_attend(ctypes.byref(d), *b, need, None) == hb.HISA_EINVAL, i
    for i, off in ((0, 8), (1, 2), (4, 4), (5, 8), (9, 4), (2, 2), (3, 1), (6, 4), (7, 2), (8, 2)):
        b = list(a)
        b[i] = P((1 << 20) + off)
        assert lib.hisa_prefix_attend(ctypes.byref(d), *b, need, None) == hb.HISA_EINVAL, i
    assert lib.hisa_prefix_attend(ctypes.byref(d), *a, need - 1, None) == hb.HISA_EWORKSPACE
    b = list(a)
    b[10] = P((1 << 20) + 16)
    assert lib.hisa_prefix_attend(ctypes.byref(d), *b, need, None) == hb.HISA_EWORKSPACE
    b[10] = None
    assert lib.hisa_prefix_attend(ctypes.byref(d), *b, need, None) == hb.HISA_EWORKSPACE


def table(**kw):
    d = dict(rope_dims=64, kind=hb.ROPE_PLAIN, theta=160000.0, factor=1.0, orig_len=65536, beta_fast=32.0, beta_slow=1.0)
    d.update(kw)
    return [int(v) & (2**64 - 1) for v in hb.rope_table(hb.RopeScaling(**d), "cpu").tolist()]


def radians(table):
    return np.array([float(v) / 2.0**64 * 2 * math.pi for v in table])


# The table's own step (2^-64 of a turn) and the steps of the doubles it is computed in
STEP = 2 * math.pi * 2.0**-64


def test_rope_table_plain_and_linear(lib):
    i = np.arange(32)
    f = 160000.0 ** (-i / 32)
    assert np.allclose(radians(table()), f, rtol=8 * 2.0**-53, atol=STEP)
    assert np.allclose(radians(table(kind=hb.ROPE_LINEAR, factor=40.0)), f / 40, rtol=8 * 2.0**-53, atol=STEP)
    # a factor below 1 / (2 pi) turns more than once per position: the whole turns drop out
    fast = radians(table(kind=hb.ROPE_LINEAR, factor=0.1))
    whole = f / 0.1 / (2 * math.pi)
    assert np.allclose(fast, (whole - np.floor(whole)) * 2 * math.pi, atol=16 * 2.0**-53 * 2 * math.pi)


@pytest.mark.parametrize("dims,factor,orig", [(64, 16.0, 65536), (128, 4.0, 4096), (32, 40.0, 4096), (2, 2.0, 100)])
def test_rope_table_yarn(lib, dims, factor, orig):
    got = radians(table(rope_dims=dims, kind=hb.ROPE_YARN, factor=factor, orig_len=orig))
    lo = max(math.floor(dims * math.log(orig / (32 * 2 * math.pi)) / (2 * math.log(160000.0))), 0)
    hi = min(math.ceil(dims * math.log(orig / (1 * 2 * math.pi)) / (2 * math.log(160000.0))), dims - 1)
    for i in range(dims // 2):
        f = 160000.0 ** (-2.0 * i / dims)
        g = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
        want = f / factor * g + f * (1 - g)
        assert abs(got[i] - want) <= 16 * 2.0**-53 * f + STEP, i


@pytest.mark.parametrize("kw", [dict(rope_dims=0), dict(rope_dims=3), dict(rope_dims=1026), dict(theta=1.0),
                                dict(theta=float("inf")), dict(kind=3), dict(kind=hb.ROPE_LINEAR, factor=0.0),
                                dict(kind=hb.ROPE_YARN, factor=float("nan")), dict(kind=hb.ROPE_YARN, orig_len=0.0),
                                dict(kind=hb.ROPE_YARN, beta_fast=0.0), dict(kind=hb.ROPE_YARN, beta_slow=-1.0)])
def test_rope_table_refusals(lib, kw):
    with pytest.raises(hb.HisaError):
        table(**kw)


def test_largest_descriptors_size(lib):
    # sizes that pass 32 bits are computed in 64
    kw = dict(B=304, L=64, prefix_rows=1 << 20, Np_max=1 << 20, kv_rows=1 << 30)
    # f32: own and shared rows are summed apart, 512 sums, a maximum and a sum per row and segment
    sums = 304 * 64 * 64 * (512 + 2) * 4
    d = prefix_desc(**kw, q_dtype=hb.HISA_F32, kv_dtype=hb.HISA_F32)
    assert hb.workspace_bytes(hb.OP_PREFIX_ATTEND, d) >= 2 * sums
    # bf16: this many query rows fill the GPU with one segment each, which needs no sums in memory
    assert hb.workspace_bytes(hb.OP_PREFIX_ATTEND, prefix_desc(**kw)) == 256
