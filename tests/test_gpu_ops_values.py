"""More of the operators around the step (GB300): full batches of the shared-prefix combine against
f64, whose pairs of CTAs each take several items; calls made with HISA_FLAG_CHAINED."""
import pytest

torch = pytest.importorskip("torch")

from deepseek_sparse_attention_hisa_gb300 import binding as hb  # noqa: E402
from test_gpu_ops import (CODE, DT, U, _built, check_norm, half_step, prefix_case, prefix_rows, randn, run_norm,  # noqa: E402, F401
                          run_prefix)

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def check_rows(c, out, out_dt, rows):
    """Query rows [(b, j)] against f64. Logits: Dh products and sums in f32 and the scale, off by
    e = Dh u scale sum|q k| + 4 u |z| (the product with the scale, the exponent's argument in base 2
    and a segment's maximum in base e each round values up to |z|), so weights and their sum by 2 e each;
    f32 sums over n rows by n u twice. bf16: each weight is rounded once, by half a step, before its
    product with the values; the normaliser sums the unrounded ones."""
    scale, worst = c["Dh"] ** -0.5, 0.0
    for b, j in rows:
        v, q = prefix_rows(c, b, j), c["q"][b, j].double()
        z = q @ v.t() * scale
        e = (c["Dh"] * U * (q.abs() @ v.abs().t() * scale) + 4 * U * z.abs()).amax(-1, keepdim=True)
        p = torch.softmax(torch.cat([z, c["sinks"].double()[:, None]], -1), -1)[:, :-1]
        want, mag = p @ v, p @ v.abs()
        tol = mag * (4 * e + 2 * v.shape[0] * U + (half_step("bf16") if c["dt"] == "bf16" else 0)) \
            + want.abs() * half_step(out_dt) + 1e-37
        err = (out[b, j].double() - want).abs()
        assert (err <= tol).all(), (b, j, (err / tol).max().item())
        worst = max(worst, (err / tol).max().item())
    return worst


# sequences, query rows, shared rows. 76 pairs of CTAs: (153, 1) is 77 pairs of query rows, the last
# of one row alone; (109, 3) an odd number of rows whose pairs straddle sequences
@pytest.mark.parametrize("out_dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,L,P", [(153, 1, 100), (153, 1, 4000), (304, 1, 1200), (109, 3, 333), (58, 4, 9001)])
def test_prefix_values_of_every_item(B, L, P, out_dt):
    own = [(37 * b) % 301 if b % 5 else 0 for b in range(B)]
    c = prefix_case(B, L, 64, P, own, "bf16", seed=P)
    out, ws = run_prefix(c, out_dt)
    assert hb.device_status(ws) == 0 and torch.isfinite(out.float()).all()
    pairs = (B * L + 1) // 2
    # both rows of the first, middle and last pairs, and of those either side of a full round of clusters
    at = sorted({min(r, B * L - 1) for p in (0, 1, 75, 76, 77, pairs // 2, 151, 152, pairs - 2, pairs - 1)
                 for r in (2 * p, 2 * p + 1)})
    check_rows(c, out, out_dt, [(r // L, r % L) for r in at])


@pytest.mark.parametrize("B,L,H,dt", [(700, 4, 8, "bf16"), (608, 3, 16, "bf16"), (304, 2, 16, "f32"), (160, 1, 64, "f32")])
def test_prefix_values_of_many_rows(B, L, H, dt):
    # more tiles of stacked rows than SMs
    c = prefix_case(B, L, H, 777, [(11 * b) % 97 for b in range(B)], dt, seed=B)
    out, ws = run_prefix(c, "f32")
    assert hb.device_status(ws) == 0 and torch.isfinite(out).all()
    check_rows(c, out, "f32", [(b, j) for b in (0, 1, B // 3, B // 2, B - 2, B - 1) for j in range(L)])


def test_prefix_call_of_a_third_of_a_second():
    # two prompt chunks of 2048 tokens before 1.2 million shared rows: a call that outlasts the limit of a
    # wait, with the rows' values at its start, middle and end
    c = prefix_case(2, 2048, 64, 1_200_000, [0, 37], "bf16", seed=3)
    out, ws = run_prefix(c, "f32")
    assert hb.device_status(ws) == 0 and torch.isfinite(out).all()
    check_rows(c, out, "f32", [(0, 0), (0, 1), (0, 2047), (1, 0), (1, 1023), (1, 2047)])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("lead", [0.0, 2.0, 5.4])
def test_prefix_one_row_outweighs_all(dt, lead):
    # one row of a late tile holds nearly all the weight, and exceeds the running maximum by less than
    # what makes the bf16 kernel rescale: the weight that is rounded is no power of two
    c = prefix_case(3, 1, 64, 700, [0, 5, 40], dt, q_std=0.01)
    c["q"] = torch.where(torch.arange(512, device="cuda") == 0, 16.0, c["q"].float()).to(c["q"].dtype)
    c["prefix"][:, 0] = 0.0
    c["prefix"][3, 0] = 30.0
    c["prefix"][650, 0] = 30.0 + lead
    c["local"][:, :, 0] = torch.where(c["local"][:, :, 0].isnan(), c["local"][:, :, 0], torch.zeros_like(c["local"][:, :, 0]))
    c["pooled"][:-3, 0] = 0.0
    out, _ = run_prefix(c, "f32")
    check_rows(c, out, "f32", [(0, 0), (1, 0), (2, 0)])


@pytest.mark.parametrize("H,dt", [(16, "bf16"), (16, "f32"), (64, "bf16")])
def test_prefix_local_lengths_that_do_not_fit(H, dt):
    # more rows than the buffer has are those it has, fewer than none are none
    c = prefix_case(3, 1, H, 70, [5, 0, 9], dt)
    c["local"] = randn(tuple(c["local"].shape), dt, 50)
    want = dict(c, len=torch.tensor([c["W"], 0, c["W"]], dtype=torch.int32, device="cuda"))
    got = dict(c, len=torch.tensor([c["W"] + 50, -3, 2**31 - 1], dtype=torch.int32, device="cuda"))
    assert torch.equal(run_prefix(got, "f32")[0], run_prefix(want, "f32")[0])
    far = dict(want, pos0=torch.tensor([-(2**31), 2**31 - 1, 2**31 - 1], dtype=torch.int32, device="cuda"))
    none = dict(want, len=torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert torch.equal(run_prefix(far, "f32")[0], run_prefix(none, "f32")[0])


# ------------------------------------------------------------------------------------
# chained calls
# ------------------------------------------------------------------------------------
# every form of the norm: a warp per row, a CTA with one, two and four units per thread, cut units,
# rows at different remainders, rows too long to be staged
@pytest.mark.parametrize("cols,ld,xt,rt,ot", [(512, 512, "bf16", "bf16", "bf16"), (1001, 1001, "f32", None, "f32"),
                                              (1000, 1003, "bf16", "f32", "bf16"), (4096, 4096, "bf16", "bf16", "e4m3"),
                                              (7168, 7168, "bf16", "bf16", "e4m3"), (5003, 5003, "f32", "f32", "f32"),
                                              (20000, 20000, "bf16", None, "bf16"), (9000, 9003, "bf16", None, "bf16"),
                                              (20000, 20003, "bf16", "bf16", "bf16"), (32768, 32768, "f32", "f32", "f32")])
def test_norm_chained(cols, ld, xt, rt, ot):
    # a chain in which each norm reads what the one before wrote, and weights that no kernel writes
    rows, n = 700, 3
    w = [1 + randn((cols,), "f32", 70 + i, 0.1) for i in range(n)]
    x0 = torch.zeros((rows, ld), device="cuda", dtype=DT[xt])
    x0[:, :cols] = randn((rows, cols), xt, 80)
    res = None if rt is None else randn((rows, cols), rt, 81, 2.0)

    def chain(flags):
        x, got = x0[:, :cols], []
        for i in range(n):
            last = i == n - 1
            out_dt = ot if last else xt
            out = torch.empty((rows, cols if last else ld), device="cuda", dtype=DT[out_dt])[:, :cols]
            res_out = None if res is None else torch.empty_like(res)
            scales = torch.empty((rows, 1), device="cuda") if out_dt == "e4m3" else None
            got.append((x, out, res_out, scales, hb.NormDesc(
                rows=rows, cols=cols, x_dtype=CODE[xt], res_dtype=CODE[rt or "f32"], out_dtype=CODE[out_dt], eps=1e-6,
                ld_x=x.stride(0), ld_res=cols, ld_out=out.stride(0), flags=flags)))
            x = out
        torch.cuda.synchronize()                      # nothing but the chain runs from here on
        for (a, out, res_out, scales, d), wi in zip(got, w):
            hb.rms_norm(d, a, res, wi, res_out, out, scales)
        torch.cuda.synchronize()
        return [t.float() for g in got for t in g[1:4] if t is not None]

    want = chain(0)
    assert all(torch.isfinite(t).all() for t in want)
    for _ in range(5):
        for a, b in zip(chain(hb.FLAG_CHAINED), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("cols,xt,rt,ot,group", [(512, "bf16", None, "bf16", 0), (1001, "f32", "f32", "f32", 0),
                                                 (7168, "bf16", "bf16", "bf16", 0), (5003, "bf16", None, "f32", 0),
                                                 (4096, "bf16", "bf16", "e4m3", 128), (20000, "bf16", "bf16", "e4m3", 32),
                                                 (32768, "f32", "f32", "f32", 0)])
@pytest.mark.parametrize("off", [1, 2])
def test_norm_weights_start_anywhere(cols, xt, rt, ot, group, off):
    # the values do not depend on where the weights start
    x, w = randn((40, cols), xt, 93), 1 + randn((cols,), "f32", 94, 0.1)
    res = None if rt is None else randn((40, cols), rt, 95)
    at = torch.full((cols + off,), float("nan"), device="cuda")
    at[off:] = w
    out, kept, s = run_norm(x, res, at[off:], ot, group)
    check_norm(x, res, w, ot, out, kept, s, group)


@pytest.mark.parametrize("rows,cols", [(900, 1001), (700, 5003), (500, 9001)])
@pytest.mark.parametrize("xt,rt,ot", [("f32", None, "f32"), ("bf16", "bf16", "bf16"), ("bf16", "f32", "e4m3")])
def test_norm_rows_of_odd_widths_do_not_depend_on_the_batch(rows, cols, xt, rt, ot):
    # rows that start at every remainder: the same row in place, by itself and among a few
    x, w = randn((rows, cols), xt, 90), 1 + randn((cols,), "f32", 91, 0.1)
    res = None if rt is None else randn((rows, cols), rt, 92, 2.0)
    whole, kept, s = run_norm(x, res, w, ot)
    for a, n in ((0, 1), (1, 1), (rows // 2 + 3, 1), (rows - 1, 1), (5, 9), (rows - 30, 30)):
        part = slice(a, a + n)
        out, res_out = torch.empty_like(whole), None if res is None else torch.empty_like(res)
        _, _, s1 = run_norm(x[part], None if res is None else res[part], w, ot, out=out[part],
                            res_out=None if res is None else res_out[part])
        assert torch.equal(out[part].float(), whole[part].float())
        assert res is None or torch.equal(res_out[part], kept[part])
        assert s is None or torch.equal(s1, s[part])


# ------------------------------------------------------------------------------------
# together: a layer's decode step
# ------------------------------------------------------------------------------------
@pytest.mark.parametrize("batch,prefix,hidden,steps,window", [(3, 40, 512, 12, 5), (2, 9, 1000, 140, 128)])
def test_shared_prefix_decode_past_the_window(batch, prefix, hidden, steps, window):
    # More tokens than the window holds. With queries and rows rounded alike, what is left are a weight's
    # rounding and the two of the output, before and after it is turned back (a pair's two values mix:
    # sqrt(2) of each): (1 + 2 sqrt(2)) 2^-8 of the weighted rows' magnitudes. Those of N(0, 1) rows are at
    # most a few times the largest output, by at most the weights' effective number: below
    # 4 (1 + 2 sqrt(2)) 2^-8 = 0.06. Dropping or keeping one row of the window too many moves a step of few
    # rows by more.
    import os
    import sys

    import deepseek_sparse_attention_hisa_gb300 as pkg
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(pkg.__file__))), "examples"))
    import shared_prefix_decode
    assert shared_prefix_decode.run(batch, prefix, hidden, steps, own_rows=3, window=window, say=lambda *_: None) < 0.06


@pytest.mark.parametrize("own_each", [False, True])
def test_decode_sees_the_prompts_last_rows(own_each):
    # The window's rows of before the first token count as the tokens' own do; those out of the window
    # (NaN here) do not. Queries and rows rounded alike, the bound as above.
    from deepseek_sparse_attention_hisa_gb300.prefix import PrefixDecode
    B, P, hidden, steps, window, held, start = 3, 20, 512, 5, 8, 11, 90
    w = {"norm": 1 + randn((hidden,), "f32", 1, 0.1), "q": randn((hidden, 64 * 512), "bf16", 2, 2 * hidden**-0.5),
         "kv": randn((hidden, 512), "bf16", 3, hidden**-0.5), "sinks": randn((64,), "f32", 4)}
    recent = randn((B, held, 512) if own_each else (held, 512), "bf16", 5)
    recent[..., :held - window + 1, :] = float("nan")
    layer = PrefixDecode(B, w, randn((P, 512), "bf16", 6), start, steps, 0, window, recent=recent)
    for n in range(steps):
        out = layer.step(randn((B, hidden), "bf16", 10 + n), randn((B, hidden), "bf16", 20 + n)).double()
        assert layer.status() == 0
        q = layer.q.double()
        for b in range(B):
            lo = max(0, held + n + 1 - window)
            v = torch.cat([layer.local[b, lo:held + n + 1].double(), layer.prefix_kv.double()])
            p = torch.softmax(torch.cat([q[b] @ v.t() * 512**-0.5, w["sinks"].double()[:, None]], -1), -1)[:, :-1]
            want = p @ v
            f = 160000.0 ** (-torch.arange(32, device="cuda", dtype=torch.float64) / 32) * (start + n)
            c, s = f.cos(), f.sin()
            a, d = want[:, 448::2].clone(), want[:, 449::2].clone()
            want[:, 448::2], want[:, 449::2] = a * c + d * s, d * c - a * s
            assert ((out[b] - want).abs().max() / want.abs().max()).item() < 0.06
