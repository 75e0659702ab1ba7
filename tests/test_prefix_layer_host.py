"""PrefixDecode without a GPU: what it refuses before any call, and the descriptors it passes on."""
import pytest

torch = pytest.importorskip("torch")

from deepseek_sparse_attention_hisa_gb300 import binding as hb  # noqa: E402
from deepseek_sparse_attention_hisa_gb300 import build  # noqa: E402
from deepseek_sparse_attention_hisa_gb300.prefix import DH, H, PrefixDecode  # noqa: E402

BF16, HIDDEN = torch.bfloat16, 64


@pytest.fixture
def calls(monkeypatch):
    """The entry points that need a GPU record their descriptors instead of running."""
    build.build_library()
    seen = []
    monkeypatch.setattr(hb, "alloc_workspace", lambda n, device: torch.zeros(max(n, 256), dtype=torch.uint8))
    monkeypatch.setattr(hb, "rms_norm", lambda d, x, r, *a: seen.append(("norm", d.ld_x, d.ld_res, x.data_ptr(), r.data_ptr())))
    monkeypatch.setattr(hb, "rope", lambda *a: seen.append(("rope",)))
    monkeypatch.setattr(hb, "prefix_attend", lambda *a: seen.append(("attend",)))
    return seen


def weights(**kw):
    w = {"norm": torch.ones(HIDDEN), "q": torch.zeros(HIDDEN, H * DH, dtype=BF16), "kv": torch.zeros(HIDDEN, DH, dtype=BF16),
         "sinks": torch.zeros(H)}
    w.update(kw)
    return w


def layer(B=3, w=None, prefix=None, **kw):
    prefix = torch.zeros(8, DH, dtype=BF16) if prefix is None else prefix
    d = dict(start=32, steps=4, own_rows=2, device="cpu")
    d.update(kw)
    return PrefixDecode(B, w or weights(), prefix, **d)


def rows(B=3, hidden=HIDDEN, dtype=BF16):
    return torch.zeros(B, hidden, dtype=dtype)


@pytest.mark.parametrize("which", ["x", "residual"])
@pytest.mark.parametrize("bad", [rows(2), rows(4), rows(3, HIDDEN - 8), rows(3, 2 * HIDDEN), rows(dtype=torch.float32),
                                 rows(dtype=torch.float16), rows()[0], rows(HIDDEN, 3).t(), rows(3, 2 * HIDDEN)[:, ::2],
                                 rows(1).expand(3, HIDDEN), torch.empty(3, HIDDEN, dtype=BF16, device="meta")])
def test_step_refuses_other_tensors(calls, which, bad):
    p = layer()
    with pytest.raises(ValueError):
        p.step(*((bad, rows()) if which == "x" else (rows(), bad)))
    assert calls == [] and p.n == 0


def test_step_takes_slices_of_wider_rows(calls):
    p = layer()
    x, r = rows(3, 3 * HIDDEN)[:, HIDDEN:2 * HIDDEN], rows(6)[::2]
    p.step(x, r)
    assert calls[0] == ("norm", 3 * HIDDEN, 2 * HIDDEN, x.data_ptr(), r.data_ptr())
    p.step(rows(), rows())
    assert calls[4][1:3] == (HIDDEN, HIDDEN)
    one = layer(B=1)
    one.step(rows(1).expand(1, HIDDEN), rows(5)[4:5])
    assert calls[8][1:3] == (HIDDEN, HIDDEN)


@pytest.mark.parametrize("name,bad", [("norm", torch.ones(HIDDEN, dtype=BF16)), ("norm", torch.ones(2 * HIDDEN)[::2]),
                                      ("q", torch.zeros(HIDDEN, DH, dtype=BF16)), ("q", torch.zeros(HIDDEN, H * DH)),
                                      ("kv", torch.zeros(HIDDEN, DH // 2, dtype=BF16)), ("sinks", torch.zeros(H - 1)),
                                      ("sinks", torch.zeros(H, dtype=BF16))])
def test_weights_are_checked(calls, name, bad):
    with pytest.raises(ValueError, match=name):
        layer(w=weights(**{name: bad}))


@pytest.mark.parametrize("bad", [torch.zeros(8, DH), torch.zeros(8, DH // 2, dtype=BF16), torch.zeros(8, 2 * DH, dtype=BF16)[:, :DH],
                                 torch.zeros(16, DH, dtype=BF16)[::2]])
def test_prefix_is_checked(calls, bad):
    with pytest.raises(ValueError, match="prefix_kv"):
        layer(prefix=bad)


@pytest.mark.parametrize("kw", [dict(B=0), dict(steps=0), dict(own_rows=-1), dict(start=-1), dict(start=2**31 - 3)])
def test_sizes_are_checked(calls, kw):
    with pytest.raises(ValueError):
        layer(**kw)


def test_pooled_rows_are_checked(calls):
    p = layer()
    good = [torch.ones(n, DH, dtype=BF16) for n in (2, 0, 1)]
    for bad in (good[:2], good[:2] + [torch.ones(3, DH, dtype=BF16)], good[:2] + [torch.ones(1, 1, dtype=BF16)],
                good[:2] + [torch.ones(DH, dtype=BF16)]):
        with pytest.raises(ValueError):
            p.append_pooled(bad)
    assert (p.pooled == 0).all() and (p.kv_off == 0).all()
    p.append_pooled(good)
    assert p.kv_off.tolist() == [0, 2, 2, 3] and (p.pooled[:3] == 1).all() and (p.pooled[3:] == 0).all()


def test_no_prefix_and_no_sinks(calls):
    p = layer(w=weights(sinks=None), prefix=torch.zeros(0, DH, dtype=BF16))
    p.step(rows(), rows())
    assert [c[0] for c in calls] == ["norm", "rope", "attend", "rope"]


def test_weights_may_be_transposed(calls):
    p = layer(w=weights(q=torch.zeros(H * DH, HIDDEN, dtype=BF16).t(), kv=torch.zeros(DH, HIDDEN, dtype=BF16).t()))
    p.step(rows(), rows())
    assert len(calls) == 4


def test_pooled_rows_are_replaced(calls):
    p = layer()
    p.set_pooled([torch.full((2, DH), 1.0, dtype=BF16)] * 3)
    p.set_pooled([torch.full((n, DH), 2.0, dtype=BF16) for n in (0, 1, 2)])
    assert p.kv_off.tolist() == [0, 0, 1, 3] and (p.pooled[:3] == 2).all()
    p.append_pooled([torch.full((1, DH), 3.0, dtype=BF16)] * 3)
    assert p.kv_off.tolist() == [0, 1, 2, 3] and (p.pooled[:3] == 3).all()


@pytest.mark.parametrize("bad", [torch.zeros(3, 5, DH), torch.zeros(2, 5, DH, dtype=BF16), torch.zeros(5, DH // 2, dtype=BF16),
                                 torch.zeros(33, DH, dtype=BF16)])
def test_recent_rows_are_checked(calls, bad):
    with pytest.raises(ValueError, match="recent"):
        layer(recent=bad)                                # start is 32


@pytest.mark.parametrize("shape", [(7, DH), (3, 7, DH)])
def test_recent_rows_precede_the_steps(calls, shape):
    recent = torch.arange(shape[-2]).to(BF16)[:, None].expand(shape).clone()
    p = layer(recent=recent)
    assert (p.local[:, :7, 0] == torch.arange(7)).all() and (p.local[:, 7:] == 0).all()
    assert p.local_pos0.tolist() == [25] * 3 and p.desc.W_max == 11 and p.rope_desc.y2_token == 11 * DH
    p.step(rows(), rows())
    assert p.local_len.tolist() == [8] * 3 and p.pos.tolist() == [33] * 3
