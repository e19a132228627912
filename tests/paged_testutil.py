"""Shared by the paged-cache tests: problems with ragged sequences over scattered pages, and
the three operators from their formulas in 64 bits (torch float64, one sequence at a time).

Every cache row that no sequence holds is filled with NaN (codes, scales and values), so
anything read from outside a sequence's tokens shows.

Bounds, element by element (u8 = 2^-8, half a step of bf16 relative to the value):
  rotation in fp32: the products and their sum round, the cosine and sine are
      rounded once: at most 4 * 2^-24 * (|x| + |partner|)
  bf16 row: u8 * |x| on top;  e4m3 row: half a step is 2^-4 |x|, or 2^-10 * scale
      where x is below the normal codes
  attention, with P_j the softmax weights: scores are fp32 sums of 256 products, off by at
      most 256 * 2^-24 * scale * sum|q k| =: d, which moves a weight by a factor e^(2 d);
      exponentials and sums add less than 2^-19; each weight enters the product with V
      rounded to 8 significant bits, so
          |y - ref| <= (u8 + 2 d + 2^-19) sum_j P_j |v_j|   (times the gate)
      and u8 |y| more for a bf16 output.  Over a code cache the weight that is
      rounded is P_j * v_scale_j, first to f16 (2^-11) and then in two e4m3 parts (2^-4 of
      2^-4: u8 again); their smallest step is 2^-9 at a scale where the row's reference weight is 2^6, and the reference is within 2^2 of the
      largest weight: 2^-14 of the largest P_j v_scale_j per code, at most.
  A relative L2 over all rows: the roundings are independent and uniform, u8 / sqrt(3)
      each at most, for the weights and again for a bf16 output.
"""
import math

import torch

import linear_attention_recurrence_10_b200 as gdr

D = 256
U8 = 2.0 ** -8
NAN = float("nan")


class Problem:
    """Packed sequences with `new` tokens over caches of `past` tokens each."""

    def __init__(self, new, past, H_q=16, H_kv=2, page=16, kind="bf16", seed=0, spare=3, tail=0,
                 width=None, v_scale_spread=0.0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.new, self.past, self.H_q, self.H_kv, self.page, self.kind = new, past, H_q, H_kv, page, kind
        self.n_seq, self.n_tok = len(new), sum(new)
        self.rows = self.n_tok + tail
        self.len = [n + p for n, p in zip(new, past)]
        need = [-(-l // page) for l in self.len]
        self.n_pages = sum(need) + spare
        self.width = max(need + [1]) if width is None else width
        order = torch.randperm(self.n_pages, generator=g).tolist()
        table = torch.full((self.n_seq, self.width), -1, dtype=torch.int32)
        for s, n in enumerate(need):
            table[s, :n] = torch.tensor([order.pop() for _ in range(n)], dtype=torch.int32)
        bf = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)
        self.q, self.gate = bf(self.rows, H_q, D), bf(self.rows, H_q, D)
        self.k, self.v = bf(self.rows, H_kv, D), bf(self.rows, H_kv, D)
        if v_scale_spread:
            self.v = (self.v.float() * torch.exp2(v_scale_spread * torch.randn(
                self.rows, H_kv, 1, generator=g))).to(torch.bfloat16)
        shape = (self.n_pages, H_kv, page)
        self.held = torch.zeros(self.n_pages, page, dtype=torch.bool)  # rows of cached tokens
        for s in range(self.n_seq):
            for t in range(self.past[s]):
                self.held[table[s, t // page], t % page] = True
        held = self.held[:, None].expand(shape)
        self.k_scale = self.v_scale = None
        if kind == "bf16":
            fill = lambda: torch.where(held[..., None], bf(*shape, D), torch.tensor(NAN).bfloat16())
            self.k_pages, self.v_pages = fill(), fill()
        else:
            def fill():
                codes = (torch.randn(*shape, D, generator=g) * 120).clamp(-448, 448).to(torch.float8_e4m3fn)
                codes = torch.where(held[..., None], codes.view(torch.uint8), torch.tensor(0x7f, dtype=torch.uint8))
                scale = torch.exp2(torch.rand(*shape, generator=g) - 7.5 +
                                   v_scale_spread * torch.randn(*shape, generator=g))
                return codes.view(torch.float8_e4m3fn), torch.where(held, scale, torch.tensor(NAN))
            self.k_pages, self.k_scale = fill()
            self.v_pages, self.v_scale = fill()
        self.table = table
        self.cu = torch.tensor([0] + new, dtype=torch.int64).cumsum(0).to(torch.int32)
        self.cache_len = torch.tensor(past, dtype=torch.int32)
        for n in ("q", "gate", "k", "v", "k_pages", "v_pages", "k_scale", "v_scale", "table", "cu",
                  "cache_len"):
            if getattr(self, n) is not None:
                setattr(self, n, getattr(self, n).to(device))

    @property
    def pages(self):
        return self.k_pages, self.v_pages, self.table, self.cu

    @property
    def scales(self):
        return dict(k_scale=self.k_scale, v_scale=self.v_scale)

    def append(self, **kw):
        q_out = torch.full_like(self.q, NAN) if "q_out" not in kw else kw.pop("q_out")
        gdr.kv_append(self.k, self.v, self.k_pages, self.v_pages, self.table, self.cu, self.cache_len,
                      q=kw.pop("q", self.q), q_out=q_out, **self.scales, **kw)
        return q_out

    def put_plain(self):
        """The new tokens into their pages without the library: k and v unrotated, as bf16,
        or as codes by the definition."""
        for s in range(self.n_seq):
            if not self.new[s]:
                continue
            t = torch.arange(self.past[s], self.len[s], device=self.cu.device)
            at = (self.table[s].long()[t // self.page], t % self.page)
            r = slice(int(self.cu[s]), int(self.cu[s + 1]))
            for x, pages, scale in ((self.k[r], self.k_pages, self.k_scale),
                                    (self.v[r], self.v_pages, self.v_scale)):
                if scale is None:
                    pages[at[0], :, at[1]] = x
                else:
                    x = x.float()
                    sc = (x.abs().amax(-1) / 448).clamp_min(2.0 ** -40)
                    codes = (x / sc[..., None]).to(torch.float8_e4m3fn)
                    pages.view(torch.uint8)[at[0], :, at[1]] = codes.view(torch.uint8)
                    scale[at[0], :, at[1]] = sc

    def cached(self, which, s, length=None):
        """(values, scales) of sequence s's rows in float64: [length, H_kv, D], [length, H_kv]."""
        t = torch.arange(self.len[s] if length is None else length, device=self.cu.device)
        at = (self.table[s].long()[t // self.page], t % self.page)
        x = getattr(self, which + "_pages")[at[0], :, at[1]].double()
        sc = getattr(self, which + "_scale")
        sc = torch.ones(x.shape[:2], dtype=torch.float64, device=x.device) if sc is None else sc[at[0], :, at[1]].double()
        return x * sc[..., None], sc

    def attend(self, gate=True, out_dtype=torch.bfloat16, lse=True, scale=None, workspace=None,
               q=None, stream=None):
        q = self.q if q is None else q
        out = torch.full((self.rows, self.H_q, D), NAN, dtype=out_dtype, device=q.device)
        lse = torch.full((self.rows, self.H_q), NAN, device=q.device) if lse else None
        args = (q, *self.pages, self.cache_len, out)
        kw = dict(**self.scales, gate=self.gate if gate else None, lse=lse, scale=scale)
        if workspace is None:
            n = gdr.attn_paged_workspace_size(*args, **kw)
            workspace = torch.full((max(n, 16),), 0xAB, dtype=torch.uint8, device=q.device)
        gdr.attn_paged(*args, **kw, workspace=workspace, stream=stream)
        return out, lse, workspace

    def check_attend(self, out, lse, gate=True, scale=None, q=None, only=None, what=""):
        """out and lse against the formula, sequence by sequence; rows of no sequence untouched."""
        scale = D ** -0.5 if scale is None else scale
        q = (self.q if q is None else q).double()
        num = den = 0.0
        for s in range(self.n_seq):
            if not self.new[s] or (only is not None and s not in only):
                continue
            r0 = int(self.cu[s])
            k, _ = self.cached("k", s)
            v, vs = self.cached("v", s)
            for a in range(0, self.new[s], 256):
                n = min(256, self.new[s] - a)
                rows = slice(r0 + a, r0 + a + n)
                qs = q[rows].unflatten(1, (self.H_kv, -1))
                sc = torch.einsum("igrd,tgd->igrt", qs, k) * scale
                mag = torch.einsum("igrd,tgd->igrt", qs.abs(), k.abs()) * scale
                pos = self.past[s] + a + torch.arange(n, device=q.device)
                off = (torch.arange(self.len[s], device=q.device) > pos[:, None])[:, None, None]
                sc = sc.masked_fill(off, -math.inf)
                d = mag.masked_fill(off, 0).amax(-1, keepdim=True) * 256 * 2.0 ** -24
                ref_lse = torch.logsumexp(sc, -1)
                P = torch.exp(sc - ref_lse[..., None])
                y = torch.einsum("igrt,tgd->igrd", P, v)
                part = 2.0 ** -11 if self.kind == "e4m3" else 0.0
                tol = (U8 + part + 2 * d + 2.0 ** -19) * torch.einsum("igrt,tgd->igrd", P, v.abs())
                if self.kind == "e4m3":
                    top = (P * vs.t()[None, :, None]).amax(-1)
                    codes = (v / vs[..., None]).abs().sum(0)
                    tol = tol + 2.0 ** -14 * top[..., None] * codes[None, :, None]
                g = torch.sigmoid(self.gate[rows].double()) if gate else torch.ones_like(q[rows])
                y, tol = y.flatten(1, 2) * g, tol.flatten(1, 2) * g * (1 + 2.0 ** -18)
                if out.dtype == torch.bfloat16:
                    tol = tol + U8 * (y.abs() + tol)
                got = out[rows].double()
                assert torch.isfinite(got).all(), (what, s, "not finite")
                err = (got - y).abs()
                assert (err <= tol + 1e-12).all(), (what, s, a, float((err - tol).max()), float((err / tol).max()))
                num += float((err ** 2).sum())
                den += float((y ** 2).sum())
                if lse is not None:
                    e = (lse[rows].double() - ref_lse.flatten(1)).abs()
                    assert (e <= d.flatten(1) + 2.0 ** -19 + 2.0 ** -22 * ref_lse.flatten(1).abs()).all(), \
                        (what, s, float(e.max()))
        bar = U8 / math.sqrt(3) * (math.sqrt(2) if out.dtype == torch.bfloat16 else 1.0)
        # a few hundred values estimate the mean of squares within a few per cent: 1.25
        assert den == 0 or math.sqrt(num / den) <= 1.25 * bar, (what, math.sqrt(num / den))
        tail = slice(int(self.cu[-1]), None)
        assert torch.isnan(out[tail]).all()
        if lse is not None:
            assert torch.isnan(lse[tail]).all()


def status_of(workspace):
    return int(workspace[:4].view(torch.int32).item())


def rope64(x, pos, rot_dim, theta):
    """x [n, H, D] float64 turned at pos [n], and the bound on fp32 rounding."""
    x = x.double()
    half = rot_dim // 2
    i = torch.arange(half, dtype=torch.float64, device=x.device)
    ang = pos.double()[:, None] * theta ** (-2 * i / rot_dim) if half else pos.double()[:, None] * i
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    a, b = x[..., :half], x[..., half:rot_dim]
    y = torch.cat([a * c - b * s, b * c + a * s, x[..., rot_dim:]], -1)
    m = a.abs() + b.abs()
    return y, 4 * 2.0 ** -24 * torch.cat([m, m, torch.zeros_like(x[..., rot_dim:])], -1)
