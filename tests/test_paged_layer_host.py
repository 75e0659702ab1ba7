"""PagedDecode without a GPU: what it refuses before any call, how it shares out pages, and the
descriptors it passes on."""
import pytest

torch = pytest.importorskip("torch")

from deepseek_sparse_attention_hisa_gb300 import binding as hb  # noqa: E402
from deepseek_sparse_attention_hisa_gb300 import build  # noqa: E402
from deepseek_sparse_attention_hisa_gb300.paged import DH, H, PagedDecode  # noqa: E402

BF16, HIDDEN = torch.bfloat16, 64


@pytest.fixture
def calls(monkeypatch):
    """The entry points that need a GPU record their descriptors instead of running."""
    build.build_library()
    seen = []
    monkeypatch.setattr(hb, "alloc_workspace", lambda n, device: torch.zeros(max(n, 256), dtype=torch.uint8))
    monkeypatch.setattr(hb, "rms_norm", lambda d, x, r, *a: seen.append(("norm", d.ld_x, d.ld_res, x.data_ptr(), r.data_ptr())))
    monkeypatch.setattr(hb, "norm_rope", lambda d, *a: seen.append(("heads", d.y2_token, a[-1].data_ptr())))
    monkeypatch.setattr(hb, "rope", lambda *a: seen.append(("rope",)))
    monkeypatch.setattr(hb, "cache_append", lambda d, t, x, w, off, first, *a: seen.append(
        ("append", d.rows, d.ld, off.tolist(), first.tolist())))
    monkeypatch.setattr(hb, "cache_read", lambda d, *a: seen.append(("read", d.rows)))
    monkeypatch.setattr(hb, "cache_attend", lambda d, *a: seen.append(("attend", d.k, a[8] is None, a[7].tolist())))
    return seen


def weights(**kw):
    w = {"norm": torch.ones(HIDDEN), "q": torch.zeros(HIDDEN, H * DH, dtype=BF16), "kv": torch.zeros(HIDDEN, DH, dtype=BF16),
         "sinks": torch.zeros(H), "q_norm": None, "kv_norm": torch.ones(DH)}
    w.update(kw)
    return w


def layer(B=3, w=None, **kw):
    d = dict(start=32, steps=4, pages=6, max_rows=12, page_rows=4, device="cpu")
    d.update(kw)
    return PagedDecode(B, w or weights(), **d)


def rows(n=3, hidden=HIDDEN, dtype=BF16):
    return torch.zeros(n, hidden, dtype=dtype)


def test_pages_are_shared_out(calls):
    p = layer()
    p.append(rows(9, DH), [1, 4, 4])
    assert calls[-1] == ("append", 9, DH, [0, 1, 5, 9], [0, 0, 0])
    assert [len(x) for x in p.owned] == [1, 1, 1] and p.cache_len.tolist() == [1, 4, 4]
    p.append(rows(4, DH, torch.float32), [3, 0, 1])
    assert calls[-1] == ("append", 4, DH, [0, 3, 3, 4], [1, 4, 4])
    assert [len(x) for x in p.owned] == [1, 1, 2] and len(p.free) == 2
    used = p.page_table[p.page_table >= 0].tolist()
    assert sorted(used) == sorted(sum(p.owned, [])) and len(set(used)) == 4
    with pytest.raises(ValueError, match="pages"):
        p.append(rows(16, DH), [8, 8, 0])
    assert p.lens == [4, 4, 5] and len(p.free) == 2              # nothing has changed
    with pytest.raises(ValueError, match="max_rows"):
        p.append(rows(9, DH), [9, 0, 0])
    p.release(2)
    assert len(p.free) == 4 and p.cache_len.tolist() == [4, 4, 0] and (p.page_table[2] == -1).all()
    p.append(rows(8, DH), [0, 8, 0])
    assert calls[-1][3:] == ([0, 0, 8, 8], [4, 4, 0]) and p.lens == [4, 12, 0]
    n = len(calls)
    p.append(rows(0, DH), [0, 0, 0])
    assert len(calls) == n


@pytest.mark.parametrize("bad,counts", [(rows(3, DH), [1, 1]), (rows(3, DH), [2, 2, 0]), (rows(2, DH), [3, -1, 0]), (rows(3, DH, torch.float16), [1, 1, 1]),
                                        (rows(3, DH // 2), [1, 1, 1]), (rows(3, 2 * DH)[:, ::2], [1, 1, 1])])
def test_appended_rows_are_checked(calls, bad, counts):
    p = layer()
    with pytest.raises(ValueError):
        p.append(bad, counts)
    assert calls == [] and p.lens == [0, 0, 0] and len(p.free) == 6


def test_rows_are_read_by_their_length(calls):
    p = layer()
    assert p.rows(0).shape == (0, DH) and calls == []
    p.append(rows(5, 2 * DH)[:, DH:], [0, 5, 0])
    assert calls[-1][2] == 2 * DH
    assert p.rows(1).shape == (5, DH) and calls[-1] == ("read", 5)
    assert p.rows(1, torch.float32).dtype == torch.float32
    with pytest.raises(ValueError):
        p.rows(1, torch.float16)


def test_a_step_in_order(calls):
    p = layer(start=[5, 6, 7])
    x, r = rows(3, 3 * HIDDEN)[:, HIDDEN:2 * HIDDEN], rows(6)[::2]
    p.step(x, r)
    assert [c[0] for c in calls] == ["norm", "heads", "attend", "rope"]
    assert calls[0] == ("norm", 3 * HIDDEN, 2 * HIDDEN, x.data_ptr(), r.data_ptr())
    assert calls[1][1:] == (4 * DH, p.local.data_ptr())
    assert p.pos.tolist() == [6, 7, 8] and p.local_pos0.tolist() == [5, 6, 7] and p.local_len.tolist() == [1, 1, 1]
    p.step(rows(), rows(), torch.zeros(3, 2, dtype=torch.int32))
    assert calls[5][2] == p.local[:, 1].data_ptr() and calls[6][:3] == ("attend", 2, False)
    p.step(rows(), rows(), torch.zeros(3, 0, dtype=torch.int32))
    assert calls[10][:3] == ("attend", 0, False)                  # ids of no rows are not all rows
    p.step(rows(), rows())
    with pytest.raises(ValueError, match="full"):
        p.step(rows(), rows())


def test_the_status_survives_a_larger_workspace(calls, monkeypatch):
    p = layer()
    before = p.ws
    monkeypatch.setattr(hb, "workspace_bytes", lambda op, d: before.numel() + d.k)
    before[0] = hb.DEV_BAD_ID
    p.step(rows(), rows(), torch.zeros(3, 8, dtype=torch.int32))
    assert p.ws.numel() == before.numel() + 8 and p.ws[0] == hb.DEV_BAD_ID


@pytest.mark.parametrize("which", ["x", "residual"])
@pytest.mark.parametrize("bad", [rows(2), rows(3, HIDDEN - 8), rows(dtype=torch.float32), rows()[0], rows(HIDDEN, 3).t(), rows(3, 2 * HIDDEN)[:, ::2],
                                 rows(1).expand(3, HIDDEN), torch.empty(3, HIDDEN, dtype=BF16, device="meta")])
def test_step_refuses_other_tensors(calls, which, bad):
    p = layer()
    with pytest.raises(ValueError):
        p.step(*((bad, rows()) if which == "x" else (rows(), bad)))
    assert calls == [] and p.n == 0


@pytest.mark.parametrize("bad", [torch.zeros(2, 4, dtype=torch.int32), torch.zeros(3, 4, dtype=torch.int64), torch.zeros(3, dtype=torch.int32),
                                 torch.zeros(3, 8, dtype=torch.int32)[:, ::2], torch.zeros(3, 65537, dtype=torch.int32)])
def test_step_refuses_other_ids(calls, bad):
    p = layer()
    with pytest.raises(ValueError):
        p.step(rows(), rows(), bad)
    assert calls == [] and p.n == 0


@pytest.mark.parametrize("name,bad", [("norm", torch.ones(HIDDEN, dtype=BF16)), ("q", torch.zeros(HIDDEN, DH, dtype=BF16)),
                                      ("kv", torch.zeros(HIDDEN, DH)), ("sinks", torch.zeros(H - 1)), ("q_norm", torch.ones(H)),
                                      ("kv_norm", torch.ones(DH, dtype=BF16)), ("kv_norm", torch.ones(2 * DH)[::2])])
def test_weights_are_checked(calls, name, bad):
    with pytest.raises(ValueError, match=name):
        layer(w=weights(**{name: bad}))


@pytest.mark.parametrize("kw", [dict(B=0), dict(steps=0), dict(start=-1), dict(start=2**31 - 3), dict(start=[1, 2]), dict(pages=0), dict(page_rows=0),
                                dict(max_rows=-1), dict(r=0)])
def test_sizes_are_checked(calls, kw):
    with pytest.raises(ValueError):
        layer(**kw)


def test_bf16_pages(calls):
    p = layer(bits4=False, w=weights(sinks=None, kv_norm=None))
    assert p.scales is None and p.pool.dtype == BF16 and p.pool.shape == (6, 4, DH)
    p.append(rows(3, DH), [1, 1, 1])
    p.step(rows(), rows())
    assert [c[0] for c in calls] == ["append", "norm", "heads", "attend", "rope"]


def kv_rows(n, first=1):
    return torch.arange(first, first + n, dtype=BF16)[:, None].repeat(1, DH)


def test_the_window_holds_the_prompts_last_rows(calls):
    # as many as the window reaches, for all the same: KV rows go straight behind them
    p = layer(window=5, start=[9, 7, 4], recent=torch.stack([kv_rows(4, b) for b in (1, 11, 21)]))
    assert p.local.shape == (3, 8, DH) and p.local[:, :4, 0].tolist() == [[1, 2, 3, 4], [11, 12, 13, 14], [21, 22, 23, 24]]
    assert p.local_len.tolist() == [4, 4, 4] and p.local_pos0.tolist() == [5, 3, 0] and p.desc.W_max == 8
    for n in range(4):
        p.step(rows(), rows())
        assert calls[-3][1:] == (8 * DH, p.local[:, 4 + n].data_ptr())
    assert p.local_len.tolist() == [8, 8, 8] and p.local_pos0.tolist() == [5, 3, 0] and p.pos.tolist() == [13, 11, 8]
    with pytest.raises(ValueError, match="full"):
        p.step(rows(), rows())


def test_sequences_may_have_unequal_rows_before(calls, monkeypatch):
    # more than the window reaches are cut; each sequence's KV row goes behind its own
    p = layer(window=3, steps=2, start=[9, 1, 4], recent=[kv_rows(5), kv_rows(1, 40), kv_rows(0)])
    assert p.local.shape == (3, 4, DH) and p.local[0, :2, 0].tolist() == [4, 5] and p.local[1, 0, 0] == 40
    assert p.local_len.tolist() == [2, 1, 0] and p.local_pos0.tolist() == [7, 0, 4]

    def heads(d, *a):
        assert d.y2_token == DH
        a[-1].copy_(torch.tensor([100.0, 110.0, 120.0])[:, None] + p.n)

    monkeypatch.setattr(hb, "norm_rope", heads)
    p.step(rows(), rows())
    p.step(rows(), rows())
    assert p.local[..., 0].tolist() == [[4, 5, 100, 101], [40, 110, 111, 0], [120, 121, 0, 0]]
    assert p.local_len.tolist() == [4, 3, 2] and p.local_pos0.tolist() == [7, 0, 4]
    with pytest.raises(ValueError, match="full"):
        p.step(rows(), rows())


@pytest.mark.parametrize("bad", [[kv_rows(1)] * 2, [kv_rows(33)] * 3, [kv_rows(1).float()] * 3, [kv_rows(1)[0]] * 3, [kv_rows(1)[:, 1:]] * 3,
                                 torch.zeros(4, 2, DH, dtype=BF16), torch.zeros(3, 2, DH // 2, dtype=BF16)])
def test_rows_before_are_checked(calls, bad):
    with pytest.raises(ValueError):
        layer(recent=bad)


def test_a_sequence_begins_in_the_place_of_another(calls, monkeypatch):
    p = layer(window=4, steps=5, start=[40, 50, 60])
    monkeypatch.setattr(hb, "norm_rope", lambda d, *a: a[-1].copy_(torch.tensor([100.0, 110.0, 120.0])[:, None] + p.n))
    p.append(rows(9, DH), [4, 4, 1])
    p.step(rows(), rows())
    p.step(rows(), rows())
    p.admit(1, 7, kv_rows(6))
    assert p.lens == [4, 0, 1] and len(p.free) == 4 and p.cache_len.tolist() == [4, 0, 1] and (p.page_table[1] == -1).all()
    assert p.local_len.tolist() == [2, 3, 2] and p.local_pos0.tolist() == [40, 4, 60] and p.pos.tolist() == [42, 7, 62]
    p.append(rows(2, DH), [0, 2, 0])
    assert calls[-1] == ("append", 2, DH, [0, 0, 2, 2], [4, 0, 1])
    p.step(rows(), rows())
    assert p.local[..., 0].tolist() == [[100, 101, 102, 0, 0], [4, 5, 6, 112, 0], [120, 121, 122, 0, 0]]
    assert p.local_len.tolist() == [3, 4, 3] and p.local_pos0.tolist() == [40, 4, 60] and p.pos.tolist() == [43, 8, 63]
    p.admit(1, 0)
    p.step(rows(), rows())
    p.step(rows(), rows())
    assert p.local[1, :2, 0].tolist() == [113, 114] and p.local_len.tolist() == [5, 2, 5] and p.local_pos0.tolist() == [40, 0, 60]
    with pytest.raises(ValueError, match="full"):                 # the buffers of those that were there
        p.step(rows(), rows())
    p.admit(0, 5, p.local[0, 2:5])
    p.admit(2, 9, p.local[2, 3:5])
    p.step(rows(), rows())
    assert p.local[0, :4, 0].tolist() == [102, 103, 104, 105] and p.local[2, :3, 0].tolist() == [123, 124, 125]


@pytest.mark.parametrize("b,start,recent", [(3, 0, None), (-1, 0, None), (0, -1, None), (0, 2**31 - 3, None), (0, 2, kv_rows(3)), (0, 9, kv_rows(2).float()),
                                            (0, 9, kv_rows(4)), (0, 9, kv_rows(1)[0])])
def test_what_cannot_begin(calls, b, start, recent):
    p = layer(window=9)
    p.append(rows(3, DH), [1, 1, 1])
    with pytest.raises(ValueError):
        p.admit(b, start, recent)
    assert p.lens == [1, 1, 1] and p.pos.tolist() == [32] * 3 and p.local_len.tolist() == [0] * 3


@pytest.mark.parametrize("b", [-1, 3])
def test_sequences_that_are_not_there(calls, b):
    p = layer()
    p.append(rows(3, DH), [1, 1, 1])
    n = len(calls)
    for f in (p.rows, p.release):
        with pytest.raises(ValueError, match="no sequence"):
            f(b)
    assert len(calls) == n and p.lens == [1, 1, 1]


@pytest.mark.parametrize("kw", [dict(cache_scale=0.0), dict(cache_scale=2.0**61), dict(page_rows=65537), dict(max_rows=2**31 - 1, page_rows=65536),
                                dict(window=-1), dict(eps=0.0)])
def test_what_no_call_would_take_is_refused_at_once(calls, kw):
    # not by the first append, when pages have changed hands
    with pytest.raises(ValueError, match="do not take"):
        layer(**kw)


def test_positions_end_with_the_window_buffer(calls):
    # the third sequence has room for two tokens more than steps, once the others have given their places to new ones
    far, before = [9, 9, 2**31 - 4], [kv_rows(2), kv_rows(2), kv_rows(0)]
    with pytest.raises(ValueError, match="positions"):
        layer(start=far, recent=before)
    layer(start=[9, 9, 2**31 - 6], recent=before)
    layer(start=far)
