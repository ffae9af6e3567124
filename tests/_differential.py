"""Test helpers of differential attention: seeded cases, the formula in 64 bits, and
the error bound of each output element that the kernels' arithmetic allows."""
from __future__ import annotations

import math

import numpy as np
import torch

import paged_kv_cache_decode_gb300 as pkv

EPS, SCALE = 1e-5, 0.8
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


class Case:
    """Requests of lengths `lens` (the new tokens included; `new` of them new, default one
    each) over one layer of a differential pool whose pages (from `first_page` on) are handed
    out in a shuffled order; unused slots hold NaN."""

    def __init__(self, lens, H, G, D, P=16, dtype="bf16", window=0, new=None, seed=0, layers=1, layer=0,
                 amp=1.0, max_context=None, table_pad=1, norm=True, weight=True, first_page=0):
        self.lens = np.asarray(lens, dtype=np.int64)
        self.B, self.H, self.G, self.D, self.P, self.window = len(self.lens), H, G, D, P, window
        self.new = np.asarray(new, dtype=np.int64) if new is not None else None
        self.dtype, self.layer, self.HQ = DT[dtype], layer, H * G
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed + 1)

        def normal(*shape, dtype=torch.float32, amp=1.0):
            return (amp * torch.randn(*shape, generator=g, device="cuda")).to(dtype)

        need = -(-self.lens // P)
        pages = int(need.sum()) + 2 + first_page
        perm = first_page + rng.permutation(pages - first_page)
        tables = np.full((self.B, int(need.max(initial=0)) + table_pad), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            tables[b, :n] = perm[at:at + n]
            at += int(n)
        self.tables = torch.from_numpy(tables).cuda()
        self.max_len = max(1, int(self.lens.max(initial=1)))
        self.pool = pkv.Pool(layers, pages, H, D, P, dtype, max_context or max(P, self.max_len),
                             query_heads=self.HQ, window=window, differential=True)
        self.k, self.v = self.pool.kv_pages(layer)
        self.k.fill_(math.nan)
        self.v.fill_(math.nan)
        # logical rows, then into the pages (all but the new ones)
        self.K, self.V = [], []
        n_new = self.new if self.new is not None else np.minimum(self.lens, 1)
        kn, vn = [], []
        for b in range(self.B):
            t, n = int(self.lens[b]), int(n_new[b])
            K, V = normal(t, H, D, dtype=self.dtype, amp=amp), normal(t, H, D, dtype=self.dtype)
            self.K.append(K)
            self.V.append(V)
            if t > n:
                pos = torch.arange(t - n, device="cuda")
                pg = self.tables[b, pos // P].long()
                self.k[pg, :, pos % P] = K[:t - n]
                self.v[pg, :, pos % P] = V[:t - n]
            if self.new is None and t == 0:
                K = V = normal(1, H, D, dtype=self.dtype)        # an empty slot's row
                n = 1
            kn.append(K[K.shape[0] - n:])
            vn.append(V[V.shape[0] - n:])
        self.k_new, self.v_new = torch.cat(kn).contiguous(), torch.cat(vn).contiguous()
        self.rows = self.k_new.shape[0]
        self.q = normal(self.rows, self.HQ, D, dtype=torch.float32 if self.new is None else self.dtype)
        self.cu = torch.from_numpy(np.concatenate([[0], np.cumsum(n_new)]).astype(np.int32)).cuda()
        self.dlens = torch.from_numpy(self.lens.astype(np.int32)).cuda()
        self.lam = 0.2 + 0.6 * torch.rand(self.HQ // 2, generator=g, device="cuda")
        self.weight = 1.0 + 0.1 * normal(2 * D) if weight else None
        self.norm = norm
        self.diff = pkv.Differential(self.lam, norm_weight=self.weight, norm_eps=EPS, out_scale=SCALE,
                                     normalise=norm)
        self.out = torch.full((self.rows, self.HQ // 2, 2 * D), math.nan, device="cuda")

    def run(self, **kw):
        if self.new is None:
            return self.pool.paged_differential_decode(
                self.layer, self.q, self.k_new, self.v_new, self.tables, self.dlens, self.max_len,
                self.diff, out=self.out, **kw)
        return self.pool.paged_differential_prefill(
            self.layer, self.q, self.k_new, self.v_new, self.cu, self.tables, self.dlens, self.diff,
            out=self.out, **kw)

    def reference(self):
        """(out, bound) in 64 bits, [rows, HQ / 2, 2 D]: `bound` is the largest error an
        element may have (see `bound_of`)."""
        out = torch.zeros(self.rows, self.HQ // 2, 2 * self.D, dtype=torch.float64, device="cuda")
        bound = torch.zeros_like(out)
        at = 0
        for b in range(self.B):
            t = int(self.lens[b])
            n = int(self.new[b]) if self.new is not None else 1
            if t > 0 and n > 0:
                sl = slice(at, at + n)
                out[sl], bound[sl] = formula(
                    self.q[sl], self.K[b], self.V[b], self.lam, self.weight if self.norm else None,
                    self.norm, self.window, self.dtype == torch.bfloat16)
            at += n
        return out, bound

    def check(self, what=""):
        assert self.pool.check_device_status() == 0
        ref, bound = self.reference()
        got = self.out.double()
        assert torch.isfinite(got).all(), f"{what}: not finite"
        off = (got - ref).abs()
        worst = (off / bound.clamp(min=1e-30)).max().item() if bound.numel() else 0.0
        assert (off <= bound).all(), f"{what}: {worst:.3g} of the bound, off by {off.max().item():.3g}"
        self.check_rows(what)
        return worst

    def check_rows(self, what=""):
        """Every row of the requests is in its page, bit for bit; other slots still hold NaN."""
        for pages, rows in ((self.k, self.K), (self.v, self.V)):
            seen = torch.zeros(pages.shape[0], self.P, dtype=torch.bool, device="cuda")
            for b in range(self.B):
                pos = torch.arange(int(self.lens[b]), device="cuda")
                pg = self.tables[b, pos // self.P].long()
                seen[pg, pos % self.P] = True
                assert torch.equal(pages[pg, :, pos % self.P], rows[b]), f"{what}: rows of request {b}"
            if pages.numel() < 1 << 30:
                rest = pages.transpose(1, 2)[~seen]
                assert torch.isnan(rest).all(), f"{what}: a slot of nobody was written"

    def close(self):
        self.pool.close()


def formula(q, K, V, lam, weight, norm, window, bf16):
    """The operator on one request: q [n, HQ, D] of the last n positions, K, V [t, H, D]."""
    n, HQ, D = q.shape
    t, H, _ = K.shape
    G = HQ // H
    q, K, V, lam = q.double(), K.double(), V.double(), lam.double()
    pos = torch.arange(t - n, t, device=q.device)
    keys = torch.arange(t, device=q.device)
    seen = keys[None] <= pos[:, None]
    if window:
        seen &= keys[None] > pos[:, None] - window
    out = torch.empty(n, HQ // 2, 2 * D, dtype=torch.float64, device=q.device)
    bound = torch.empty_like(out)
    for i in range(HQ // 2):
        p = i // G
        vv = torch.cat([V[:, 2 * p], V[:, 2 * p + 1]], dim=1)
        d = torch.zeros(n, 2 * D, dtype=torch.float64, device=q.device)
        off = torch.zeros_like(d)
        for m in range(2):
            s = q[:, 2 * i + m] @ K[:, 2 * p + m].T / math.sqrt(D)
            mag = q[:, 2 * i + m].abs() @ K[:, 2 * p + m].abs().T / math.sqrt(D)
            a = torch.softmax(s.masked_fill(~seen, -math.inf), dim=1)
            c = lam[i] if m else 1.0
            d = d - c * (a @ vv) if m else a @ vv
            off = off + c * (delta_of(mag.masked_fill(~seen, 0.0), D, t, bf16) * a) @ vv.abs()
        bound[:, i], out[:, i] = bound_of(d, off, weight, norm), finish(d, weight, norm)
    return out, bound


def finish(d, weight, norm):
    if not norm:
        return SCALE * d
    x = SCALE * d / torch.sqrt((d * d).mean(-1, keepdim=True) + EPS)
    return x * weight.double() if weight is not None else x


def delta_of(mag, D, t, bf16):
    """Largest relative error of one softmax weight times its value.  mag = sum |q k| / sqrt(D)
    of the score (natural-log units).  A half step of fp32 is 2^-24, of bf16 2^-9:
      score       (D + 4) roundings of fp32 at most; with q as bf16 hi + lo, 2^-18 of each
                  term more (half a step of lo, which is half a step of q at most)
      exponent    twice the score's error (the weight and the sum it is divided by), 2^-21
                  for exp2 and the scaling of the exponent's argument
      products    weights as bf16 hi + lo: 2^-18; sums over t keys: errors of either sign, 8
                  standard deviations of sqrt(t) roundings, sums and accumulators alike"""
    score = mag * ((D + 4) * 2.0 ** -24 + (2.0 ** -18 if bf16 else 0.0))
    return 2 * score + 2.0 ** -21 + (2.0 ** -18 if bf16 else 0.0) + 2 * 8 * math.sqrt(t) * 2.0 ** -24


def bound_of(d, off, weight, norm):
    """Error of the output element when d is off by at most `off`, plus the roundings of the
    epilogue (difference, mean of 2 D squares, root, quotient, two products: under 2^-20)."""
    if not norm:
        return SCALE * off + SCALE * d.abs() * 2.0 ** -20 + 1e-30
    r = torch.sqrt((d * d).mean(-1, keepdim=True) + EPS)
    # |d + e| / r' - |d| / r with |r' - r| <= rms(e)
    er = torch.sqrt((off * off).mean(-1, keepdim=True))
    x = SCALE * ((off + d.abs() * er / r) / r * (1 + er / r) + d.abs() / r * 2.0 ** -20)
    return (x * weight.double().abs() if weight is not None else x) + 1e-30
