"""Device-resident state of one attention layer's decode for a batch that shares a long prefix,
and the calls of a step, in order.

Marshalling only: torch allocates the tensors, owns the stream and multiplies by the projection
weights; everything else is one libhisa entry point each (include/hisa.h):

  hisa_rms_norm       residual addition, norm, 8-bit activations with scales
  (projections)       queries and the token's KV row, torch matmul
  hisa_rope           queries, and the KV row straight into its slot of the window buffer
  hisa_prefix_attend  the dense combine over window, shared pooled rows, own pooled rows and sinks
  hisa_rope           the output turned back (K = V: its rotated dims carry positions), in place
"""
from __future__ import annotations

from . import binding as hb

H, DH, ROPE_DIMS = 64, 512, 64


def _expect(t, name, shape, dtype, device, layout="dense"):
    """The kernels get pointers: whatever a tensor is not, they would read or write past its end.
    layout: "rows" may lie further apart than they are wide (a slice of a wider tensor); "any" is
    for what torch multiplies by."""
    if tuple(t.shape) != shape or t.dtype != dtype or t.device != device:
        raise ValueError(f"{name}: {list(shape)} {dtype} on {device} expected, "
                         f"got {list(t.shape)} {t.dtype} on {t.device}")
    fits = {"dense": t.is_contiguous(), "any": True,
            "rows": t.stride(-1) == 1 and (t.shape[0] == 1 or t.stride(0) >= shape[-1])}
    if not fits[layout]:
        raise ValueError(f"{name}: strides {t.stride()} are not dense")


class PrefixDecode:
    """B sequences that decode in step behind one shared prefix of P pooled rows.

    weights: norm [hidden] f32, q [hidden, H * DH] bf16, kv [hidden, DH] bf16, sinks [H] f32 (or None).
    prefix_kv: [P, DH] bf16; the combine is dense, as a layer's is whose pooled rows are few for its
    context (one row for 128 tokens, or the first 512 of one for 4): longer streams of a ratio-4 layer
    select rows instead (problem.py). r is that ratio; a step's single query row per sequence sees all
    its pooled rows, whatever r. start: the position of the first token decoded. steps: how many tokens
    the window buffer takes. own_rows: pooled rows each sequence may add (set_pooled).
    recent: [n, DH] or, one's own for each sequence, [B, n, DH] bf16: the KV rows of the n positions
    before start, rotated, as far back as the window reaches (n up to window - 1 matter); without
    them the first tokens see nothing of the prompt but its pooled rows.
    Tensors of another shape, type, device or layout raise ValueError."""

    def __init__(self, B, weights, prefix_kv, start, steps, own_rows=0, window=128, r=4, eps=1e-6, theta=160000.0,
                 device="cuda", recent=None):
        import torch
        self.B, self.w, self.prefix_kv, self.n = B, weights, prefix_kv, 0
        self.start, self.steps, self.hidden = start, steps, weights["norm"].numel()
        if B < 1 or steps < 1 or own_rows < 0 or start < 0 or start + steps > 2**31:
            raise ValueError("B and steps of 1 at least, own_rows and positions from 0 to 2^31 - 1 expected")
        self.device = torch.empty(0, device=device).device
        at = self.device
        _expect(weights["norm"], "weights['norm']", (self.hidden,), torch.float32, at)
        _expect(weights["q"], "weights['q']", (self.hidden, H * DH), torch.bfloat16, at, "any")
        _expect(weights["kv"], "weights['kv']", (self.hidden, DH), torch.bfloat16, at, "any")
        if weights["sinks"] is not None:
            _expect(weights["sinks"], "weights['sinks']", (H,), torch.float32, at)
        _expect(prefix_kv, "prefix_kv", (prefix_kv.shape[0], DH), torch.bfloat16, at)
        self.held = 0 if recent is None else recent.shape[-2]          # rows of the window buffer before start
        if recent is not None:
            _expect(recent, "recent", (*((B,) if recent.dim() == 3 else ()), self.held, DH), torch.bfloat16, at, "any")
            if self.held > start:
                raise ValueError(f"recent: {self.held} rows before position {start}")
        bf16 = dict(device=device, dtype=torch.bfloat16)
        i32 = dict(device=device, dtype=torch.int32)
        group = 128 if self.hidden % 128 == 0 else 0
        self.norm_desc = hb.NormDesc(rows=B, cols=self.hidden, x_dtype=hb.HISA_BF16, res_dtype=hb.HISA_BF16,
                                     out_dtype=hb.HISA_E4M3, scale_group=group, eps=eps, ld_x=self.hidden,
                                     ld_res=self.hidden, ld_out=self.hidden)
        self.codes = torch.empty((B, self.hidden), device=device, dtype=torch.float8_e4m3fn)
        self.scales = torch.empty((B, self.hidden // (group or self.hidden)), device=device)
        self.table = hb.rope_table(hb.RopeScaling(rope_dims=ROPE_DIMS, kind=hb.ROPE_PLAIN, theta=theta), device)
        self.local = torch.zeros((B, self.held + steps, DH), **bf16)
        if recent is not None:
            self.local[:, :self.held] = recent
        self.q = torch.empty((B, H, DH), **bf16)
        rope = dict(tokens=B, heads=H, D=DH, rope_dims=ROPE_DIMS, rope_first=DH - ROPE_DIMS, mscale=1.0,
                    x_token=H * DH, x_head=DH, y_token=H * DH, y_head=DH)
        self.rope_desc = hb.RopeDesc(heads2=1, src_dtype=hb.HISA_BF16, dst_dtype=hb.HISA_BF16, x2_token=DH, x2_head=DH,
                                     y2_token=self.local.stride(0), y2_head=DH, **rope)
        self.back_desc = hb.RopeDesc(heads2=0, inverse=1, src_dtype=hb.HISA_BF16, dst_dtype=hb.HISA_BF16, **rope)
        self.pooled = torch.zeros((max(B * own_rows, 1), DH), **bf16)
        self.own_rows = own_rows
        self.kv_off = torch.zeros(B + 1, device=device, dtype=torch.int64)
        self.pos = torch.full((B,), start, **i32)
        self.local_pos0 = torch.full((B,), start - self.held, **i32)
        self.local_len = torch.zeros(B, **i32)
        self.desc = hb.PrefixDesc(B=B, L=1, H=H, Dh=DH, window=window, W_max=self.local.shape[1], r=r, prefix_rows=prefix_kv.shape[0],
                                  Np_max=own_rows, kv_rows=self.pooled.shape[0], scale=0.0, q_dtype=hb.HISA_BF16,
                                  kv_dtype=hb.HISA_BF16, out_dtype=hb.HISA_BF16)
        self.ws = hb.alloc_workspace(hb.workspace_bytes(hb.OP_PREFIX_ATTEND, self.desc), device)
        self.out = torch.empty((B, H, DH), **bf16)

    def set_pooled(self, rows):
        """The sequences' own pooled rows, in place of those they had: a list of [n_b, DH] bf16 tensors."""
        import torch
        if len(rows) != self.B or any(x.dim() != 2 or x.shape[0] > self.own_rows or x.shape[1] != DH for x in rows):
            raise ValueError(f"one tensor of at most own_rows rows of {DH} per sequence")
        off = [0]
        for x in rows:
            self.pooled[off[-1]:off[-1] + x.shape[0]] = x
            off.append(off[-1] + x.shape[0])
        self.kv_off.copy_(torch.tensor(off, dtype=torch.int64))

    append_pooled = set_pooled        # the name it had, though it never appended

    def activations(self):
        """The norm's 8-bit output as bf16: what projections of 8-bit activations are given, for weights
        in bf16."""
        import torch
        groups = self.scales.shape[1]
        return (self.codes.float().view(self.B, groups, -1) * self.scales[..., None]).view(self.B, -1).to(torch.bfloat16)

    def step(self, x, residual):
        """One token per sequence: x, residual [B, hidden] bf16, rows dense (residual is updated in place).
        Returns the combine's output [B, H, DH] bf16, turned back to position-free dims; the next step
        writes it anew."""
        import torch
        if self.n == self.steps:
            raise ValueError("the window buffer is full")
        for t, name in ((x, "x"), (residual, "residual")):
            _expect(t, name, (self.B, self.hidden), torch.bfloat16, self.device, "rows")
        self.norm_desc.ld_x = x.stride(0) if self.B > 1 else self.hidden
        self.norm_desc.ld_res = residual.stride(0) if self.B > 1 else self.hidden
        hb.rms_norm(self.norm_desc, x, residual, self.w["norm"], residual, self.codes, self.scales)
        a = self.activations()
        q, kv = a @ self.w["q"], a @ self.w["kv"]
        hb.rope(self.rope_desc, self.table, self.pos, q, self.q, kv, self.local[:, self.held + self.n])
        self.n += 1
        self.local_len.fill_(self.held + self.n)
        hb.prefix_attend(self.desc, self.q, self.local, self.local_len, self.local_pos0, self.prefix_kv, self.pooled,
                         self.kv_off, self.w["sinks"], self.pos, self.out, self.ws)
        hb.rope(self.back_desc, self.table, self.pos, self.out, self.out)
        self.pos += 1
        return self.out

    def status(self) -> int:
        return hb.device_status(self.ws)
