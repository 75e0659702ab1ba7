"""More of the operators around the step against their definitions in f64 (GB300): full batches of
the shared-prefix combine, whose pairs of CTAs each take several items."""
import pytest

torch = pytest.importorskip("torch")

from deepseek_sparse_attention_hisa_gb300 import binding as hb  # noqa: E402
from test_gpu_ops import U, _built, half_step, prefix_case, prefix_rows, run_prefix  # noqa: E402, F401

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
