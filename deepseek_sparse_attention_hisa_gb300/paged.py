"""Device-resident state of one attention layer's decode whose pooled KV rows are kept in pages, in 4 bits or
bf16, and the calls of a step, in order.

Marshalling only: torch allocates the tensors, owns the stream and multiplies by the projection
weights; everything else is one libhisa entry point each (include/hisa.h):

  hisa_rms_norm      residual addition and norm
  (projections)      queries and the token's KV row, torch matmul
  hisa_norm_rope     the norm of each query head and of the KV row, their rotary positions, the KV row
                     straight into its slot of the window buffer
  hisa_cache_append  pooled rows, as they complete: normed, turned, into pages (append)
  hisa_cache_attend  the combine over window, all or selected pooled rows, and sinks
  hisa_rope          the output turned back (K = V: its rotated dims carry positions), in place
  hisa_cache_read    a sequence's pooled rows out of its pages, for instance as another batch's
                     shared prefix (rows)
"""
from __future__ import annotations

from . import binding as hb
from .prefix import DH, H, ROPE_DIMS, _expect


class PagedDecode:
    """B sequences that decode in step, each with pooled rows in pages of its own.

    weights: norm [hidden] f32, q [hidden, H * DH] bf16, kv [hidden, DH] bf16, and in f32 or None for ones
    q_norm [DH], kv_norm [DH] (heads and KV rows are normed), sinks [H] f32 (or None).
    start: the position of the first token decoded, one for all or a list of one each. steps: how many
    tokens the window buffer takes. pages: pages of page_rows rows that the sequences share out among
    themselves, also with those that begin later in the place of others (admit); max_rows: pooled rows of a
    sequence at most. r: tokens per pooled row; pooled row p sits at position p r. bits4: rows in 4 bits (16
    dims share a scale), else bf16; cache_scale: the factor of all rows in 4 bits. recent: the KV rows of the
    positions before start, normed and rotated, bf16: [B, n, DH], or a list of [n_b, DH] (the last window - 1
    matter); without them the first tokens see nothing of the prompt but its pooled rows.
    Tensors of another shape, type, device or layout raise ValueError, and so does a cache that is full."""

    def __init__(self, B, weights, start, steps, pages, max_rows, page_rows=64, window=128, r=4, bits4=True, cache_scale=1.0,
                 eps=1e-6, theta=160000.0, device="cuda", recent=None):
        import torch
        self.B, self.w, self.n, self.r = B, weights, 0, r
        self.steps, self.hidden, self.page_rows, self.max_rows = steps, weights["norm"].numel(), page_rows, max_rows
        self.window = window
        if B < 1 or steps < 1 or pages < 1 or max_rows < 0 or page_rows < 1 or r < 1:
            raise ValueError("B, steps, pages, page_rows and r of 1 at least expected")
        starts = [int(start)] * B if not hasattr(start, "__len__") else [int(t) for t in start]
        if len(starts) != B or min(starts) < 0 or max(starts) + steps > 2**31:
            raise ValueError("a start for all sequences or one each, and positions from 0 to 2^31 - 1, expected")
        self.device = torch.empty(0, device=device).device
        at = self.device
        _expect(weights["norm"], "weights['norm']", (self.hidden,), torch.float32, at)
        _expect(weights["q"], "weights['q']", (self.hidden, H * DH), torch.bfloat16, at, "any")
        _expect(weights["kv"], "weights['kv']", (self.hidden, DH), torch.bfloat16, at, "any")
        for name, n in (("q_norm", DH), ("kv_norm", DH), ("sinks", H)):
            if weights[name] is not None:
                _expect(weights[name], f"weights['{name}']", (n,), torch.float32, at)
        bf16, i32 = dict(device=device, dtype=torch.bfloat16), dict(device=device, dtype=torch.int32)
        self.norm_desc = hb.NormDesc(rows=B, cols=self.hidden, x_dtype=hb.HISA_BF16, res_dtype=hb.HISA_BF16, out_dtype=hb.HISA_BF16,
                                     eps=eps, ld_x=self.hidden, ld_res=self.hidden, ld_out=self.hidden)
        self.act = torch.empty((B, self.hidden), **bf16)
        self.table = hb.rope_table(hb.RopeScaling(rope_dims=ROPE_DIMS, kind=hb.ROPE_PLAIN, theta=theta), device)
        # sequence b's next row of the window buffer is n + ahead[b]: where all are the same, the KV rows go straight
        # into it, else by way of kv_row
        recent = [None] * B if recent is None else list(recent)
        if len(recent) != B:
            raise ValueError(f"recent: rows of {B} sequences expected, got {len(recent)}")
        recent = [self._reached(x, t) for x, t in zip(recent, starts)]
        self.ahead = [x.shape[0] for x in recent]
        self._order()
        self.capacity = self.top + steps
        if any(t + self.capacity - n > 2**31 for t, n in zip(starts, self.ahead)):
            raise ValueError("positions from 0 to 2^31 - 1 expected, for as many tokens as the window buffer takes")
        self.local = torch.zeros((B, self.capacity, DH), **bf16)
        for b, x in enumerate(recent):
            self.local[b, :x.shape[0]] = x
        self.kv_row = torch.empty((B, DH), **bf16)
        self.row0 = torch.arange(B, device=device) * self.capacity
        self.q, self.out = torch.empty((B, H, DH), **bf16), torch.empty((B, H, DH), **bf16)
        dense = dict(x_token=H * DH, x_head=DH, y_token=H * DH, y_head=DH)
        self.head_desc = hb.NormRopeDesc(tokens=B, heads=H, heads2=1, D=DH, norm=1, norm2=1, rope_dims=ROPE_DIMS, rope_first=DH - ROPE_DIMS,
                                         src_dtype=hb.HISA_BF16, dst_dtype=hb.HISA_BF16, eps=eps, mscale=1.0, x2_token=DH, x2_head=DH,
                                         y2_head=DH, **dense)
        self.back_desc = hb.RopeDesc(tokens=B, heads=H, heads2=0, D=DH, rope_dims=ROPE_DIMS, rope_first=DH - ROPE_DIMS, inverse=1,
                                     src_dtype=hb.HISA_BF16, dst_dtype=hb.HISA_BF16, mscale=1.0, **dense)
        cols = max(1, -(-max_rows // page_rows))
        kind = hb.HISA_E2M1 if bits4 else hb.HISA_BF16
        self.pool = torch.zeros((pages, page_rows, DH // 2 if bits4 else DH), device=device, dtype=torch.uint8 if bits4 else torch.bfloat16)
        self.scales = torch.zeros((pages, page_rows, DH // 16), device=device, dtype=torch.uint8) if bits4 else None
        self.free, self.owned, self.lens = list(range(pages))[::-1], [[] for _ in range(B)], [0] * B
        self.page_table = torch.full((B, cols), -1, **i32)
        self.cache_len = torch.zeros(B, **i32)
        self.cache_desc = dict(pages=pages, page_rows=page_rows, D=DH, cache_dtype=kind, cache_scale=cache_scale, table_cols=cols,
                               norm=1, eps=eps, rope_dims=ROPE_DIMS, rope_first=DH - ROPE_DIMS, r=r, mscale=1.0)
        self.desc = hb.CacheAttnDesc(B=B, L=1, H=H, Dh=DH, window=window, W_max=self.capacity, r=r, k=0, page_rows=page_rows, table_cols=cols,
                                     pages=pages, Np_max=max_rows, scale=0.0, cache_scale=cache_scale, q_dtype=hb.HISA_BF16,
                                     cache_dtype=kind, out_dtype=hb.HISA_BF16)
        self.pos = torch.tensor(starts, **i32)
        self.local_len = torch.tensor(self.ahead, **i32)
        self.local_pos0 = self.pos - self.local_len
        self.cache_ws = hb.alloc_workspace(256, device)
        need = hb.workspace_bytes(hb.OP_CACHE_ATTEND, self.desc)
        if need == 0 or hb.workspace_bytes(hb.OP_CACHE, hb.CacheDesc(B=B, ld=DH, **self.cache_desc)) == 0 or not eps > 0:
            raise ValueError("sizes, a cache_scale or an eps that the library's calls do not take")
        self.ws, self.ws_k = hb.alloc_workspace(need, device), 0

    def _there(self, b):
        if not 0 <= b < self.B:                          # -1 would name the last one here and no row of the page table there
            raise ValueError(f"no sequence {b} of {self.B}")

    def _order(self):
        self.top, self.together = max(self.ahead), min(self.ahead) == max(self.ahead)

    def _reached(self, rows, start):
        """The rows before position start that the window reaches."""
        import torch
        if rows is None:
            return torch.empty((0, DH), device=self.device, dtype=torch.bfloat16)
        if rows.dim() != 2:
            raise ValueError("recent: [n, DH] expected for a sequence")
        n = rows.shape[0]
        _expect(rows, "recent", (n, DH), torch.bfloat16, self.device, "any")
        if n > start:
            raise ValueError(f"recent: {n} rows before position {start}")
        return rows[n - min(n, max(self.window - 1, 0)):]

    def append(self, rows, counts):
        """Pooled rows that have completed, counts[b] of sequence b, packed in the sequences' order: [n, DH] bf16 or
        f32, before the norm and the rotation. They follow those that the sequence has."""
        import torch
        counts = [int(n) for n in counts]
        if len(counts) != self.B or min(counts) < 0:
            raise ValueError("a count of rows for each sequence expected")
        if rows.dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("rows: bf16 or f32 expected")
        _expect(rows, "rows", (sum(counts), DH), rows.dtype, self.device, "rows")
        if sum(counts) == 0:
            return
        need = [-(-(have + n) // self.page_rows) - len(own) for have, n, own in zip(self.lens, counts, self.owned)]
        if any(have + n > self.max_rows for have, n in zip(self.lens, counts)):
            raise ValueError("more pooled rows than max_rows")
        if sum(need) > len(self.free):
            raise ValueError(f"{sum(need)} pages needed, {len(self.free)} free")
        first = torch.tensor(self.lens, dtype=torch.int32).to(self.device)
        for b, n in enumerate(need):
            if n:
                new = [self.free.pop() for _ in range(n)]
                have = len(self.owned[b])
                self.page_table[b, have:have + n] = torch.tensor(new, dtype=torch.int32)
                self.owned[b] += new
        self.lens = [have + n for have, n in zip(self.lens, counts)]
        off = torch.tensor([0] + counts).cumsum(0).to(self.device)
        d = hb.CacheDesc(B=self.B, rows=rows.shape[0], ld=rows.stride(0) if rows.shape[0] > 1 else DH, io_dtype=hb.dtype_code(rows),
                         **self.cache_desc)
        hb.cache_append(d, self.table, rows, self.w["kv_norm"], off, first, self.page_table, self.pool, self.scales, self.cache_ws)
        self.cache_len.copy_(torch.tensor(self.lens, dtype=torch.int32))

    def rows(self, b, dtype=None):
        """Sequence b's pooled rows as the combine sees them, [len, DH] in bf16 (or f32)."""
        import torch
        self._there(b)
        out = torch.empty((self.lens[b], DH), device=self.device, dtype=dtype or torch.bfloat16)
        if out.dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("bf16 or f32 expected")
        if self.lens[b]:
            d = hb.CacheDesc(B=1, rows=out.shape[0], ld=DH, io_dtype=hb.dtype_code(out), **self.cache_desc)
            off = torch.tensor([0, out.shape[0]]).to(self.device)
            hb.cache_read(d, off, torch.zeros(1, device=self.device, dtype=torch.int32), self.page_table[b:b + 1], self.pool, self.scales,
                          out, self.cache_ws)
        return out

    def release(self, b):
        """Sequence b's pages are free again; it has no pooled rows. It decodes on behind its window alone, and rows
        appended to it start at position 0: admit begins another sequence in its place."""
        import torch
        self._there(b)
        self.free += self.owned[b][::-1]
        self.owned[b], self.lens[b] = [], 0
        self.page_table[b].fill_(-1)
        self.cache_len.copy_(torch.tensor(self.lens, dtype=torch.int32))

    def admit(self, b, start, recent=None):
        """Another sequence begins in the place of sequence b, which ends: its first token decoded has position start,
        recent [n, DH] are the KV rows before it (as the constructor takes them), and its pooled rows are those that are
        appended from now on. Of the sequence before it nothing is seen any more."""
        start = int(start)
        self._there(b)
        recent = self._reached(recent, start)
        n = recent.shape[0]
        if start < 0 or start + self.capacity - n > 2**31:
            raise ValueError("positions from 0 to 2^31 - 1 expected")
        if n >= self.capacity:
            raise ValueError(f"recent: {n} rows fill the window buffer of {self.capacity}")
        self.release(b)
        self.local[b, :n] = recent.clone()               # it may be rows of this buffer
        self.ahead[b] = n - self.n
        self._order()
        self.local_len[b], self.local_pos0[b], self.pos[b] = n, start - n, start

    def step(self, x, residual, I=None):
        """One token per sequence: x, residual [B, hidden] bf16, rows dense (residual is updated in place).
        I [B, k] int32: the pooled rows that each sequence combines (-1: none), from the selection; None: all.
        Returns the combine's output [B, H, DH] bf16, turned back to position-free dims; the next step
        writes it anew."""
        import torch
        if self.n + self.top == self.capacity:
            raise ValueError("the window buffer is full")
        for t, name in ((x, "x"), (residual, "residual")):
            _expect(t, name, (self.B, self.hidden), torch.bfloat16, self.device, "rows")
        k = 0
        if I is not None:
            if I.dim() != 2:
                raise ValueError("I: [B, k] expected")
            k = I.shape[1]
            _expect(I, "I", (self.B, k), torch.int32, self.device)
        self.desc.k = k
        if k > self.ws_k:
            need = hb.workspace_bytes(hb.OP_CACHE_ATTEND, self.desc)
            if need == 0:
                raise ValueError(f"I: {k} rows are too many")
            if need > self.ws.numel():
                old, self.ws = self.ws, hb.alloc_workspace(need, self.device)
                self.ws[:256] = old[:256]                # the status so far
            self.ws_k = k
        self.norm_desc.ld_x = x.stride(0) if self.B > 1 else self.hidden
        self.norm_desc.ld_res = residual.stride(0) if self.B > 1 else self.hidden
        hb.rms_norm(self.norm_desc, x, residual, self.w["norm"], residual, self.act)
        q, kv = self.act @ self.w["q"], self.act @ self.w["kv"]
        row = self.local[:, self.n + self.top] if self.together else self.kv_row
        self.head_desc.y2_token = row.stride(0)
        hb.norm_rope(self.head_desc, self.table, self.pos, q, self.w["q_norm"], self.q, kv, self.w["kv_norm"], row)
        if not self.together:
            self.local.view(-1, DH).index_copy_(0, self.row0 + self.local_len, row)
        self.n += 1
        self.local_len += 1
        hb.cache_attend(self.desc, self.q, self.local, self.local_len, self.local_pos0, self.pool, self.scales, self.page_table,
                        self.cache_len, I, self.w["sinks"], self.pos, self.out, self.ws)
        hb.rope(self.back_desc, self.table, self.pos, self.out, self.out)
        self.pos += 1
        return self.out

    def status(self) -> int:
        """The device status bits of all calls so far (0 = clean)."""
        return hb.device_status(self.ws) | hb.device_status(self.cache_ws)
