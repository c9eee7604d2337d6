"""64-bit definitions of the paged operators (chunks of new tokens, the 8-bit latent cache) and the
inputs their tests share.  Everything here is numpy or torch in float64, from the formulas; none
of it calls the library.

Error bounds (u = 2^-8 is half a bf16 step relative to a value, 2^-24 half an fp32 step):
  logits  the tensor cores add 16 products at a time to an fp32 sum; each of the n / 16 + 1 sums
          is off by at most 2^-22 of the magnitudes summed so far (truncating accumulation), so
          |dl| <= (n / 16 + 1) 2^-22 sigma sum_d |q_d k_d| =: D
  exp     the fp32 argument and the 2^x approximation: below 2^-18 relative while |l| < 64
  output  probabilities are rounded to bf16 once (u each), the sums are fp32, the result is
          rounded to bf16 (u): |dO| <= A (u + 2 D + 2^-18) + u |O|, A = sum_s p_s |v_s|
          (a logit off by D moves a normalised probability by at most 2 D)
  LSE     D + 2^-18 and a rounding of the result
"""
from __future__ import annotations

import math

import numpy as np
import torch

U = 2.0 ** -8
FULL = dict(h_idx=64, d_idx=128, h=128, d_qk=576, d_v=512)
TINY = dict(h_idx=4, d_idx=32, h=16, d_qk=160, d_v=128)


# ------------------------------------------------------------------------------- 8-bit rows

def e4m3_values() -> np.ndarray:
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7.0))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b >= 128, -v, v)


def e4m3_nearest(y: np.ndarray) -> np.ndarray:
    """Codes of the e4m3 values nearest to y (float64, finite): ties to even, saturating."""
    y = np.asarray(y, np.float64)
    a = np.minimum(np.abs(y), 448.0)
    e = np.floor(np.log2(np.maximum(a, 2.0 ** -6)))
    step = 2.0 ** (e - 3)
    q = np.rint(a / step) * step                           # may reach the next power of two
    e2 = np.floor(np.log2(np.maximum(q, 2.0 ** -6)))
    sub = q < 2.0 ** -6
    code = np.where(sub, np.rint(q * 2.0 ** 9), (e2 + 7) * 8 + np.rint((q / 2.0 ** e2 - 1) * 8))
    return code.astype(np.uint8) | np.where(np.signbit(y), 128, 0).astype(np.uint8)


def row_bytes(d) -> int:
    return d["d_v"] + (4 * (d["d_v"] // 128) + 15) // 16 * 16 + 2 * (d["d_qk"] - d["d_v"])


def pack_rows(latent: torch.Tensor, d) -> np.ndarray:
    """8-bit rows (uint8 [n, row_bytes]) of bf16 latent rows, from the definition."""
    lat = latent.detach().cpu()
    x = lat.double().numpy()
    n, dv = x.shape[0], d["d_v"]
    g = dv // 128
    val = x[:, :dv].reshape(n, g, 128)
    finite = np.isfinite(val).all(axis=2)
    val = np.where(finite[:, :, None], val, 0.0)
    top = np.abs(val).max(axis=2)
    e = np.zeros_like(top)
    pos = top > 0
    e[pos] = np.ceil(np.log2(top[pos] / 448.0))
    # the logarithm's last bit at exact powers: correct by comparison
    e = np.where(pos & (top > 448.0 * 2.0 ** e), e + 1, e)
    e = np.where(pos & (top <= 448.0 * 2.0 ** (e - 1)), e - 1, e)
    e = np.where(pos, np.clip(e, -100, 119), 0)
    codes = e4m3_nearest(val / (2.0 ** e)[:, :, None]).reshape(n, dv)
    codes = np.where(np.repeat(finite, 128, axis=1), codes, 0)
    slots = (4 * g + 15) // 16 * 4
    scale = np.zeros((n, slots), np.float32)
    scale[:, :g] = np.where(finite, 2.0 ** e, np.nan).astype(np.float32)
    rope = lat[:, dv:].contiguous().view(torch.int16).numpy().view(np.uint8)
    return np.concatenate([codes, scale.view(np.uint8), rope], axis=1)


def unpack_rows(rows: np.ndarray, d) -> np.ndarray:
    """float64 values [n, d_qk] of 8-bit rows."""
    dv = d["d_v"]
    g, off = dv // 128, dv + (4 * (dv // 128) + 15) // 16 * 16
    scale = np.ascontiguousarray(rows[:, dv:dv + 4 * g]).view(np.float32).astype(np.float64)
    v = e4m3_values()[rows[:, :dv]] * np.repeat(scale, 128, axis=1)
    bits = np.ascontiguousarray(rows[:, off:]).view(np.uint16).astype(np.uint32) << 16
    return np.concatenate([v, bits.view(np.float32).astype(np.float64)], axis=1)


def key_codes(k: np.ndarray):
    """Indexer key codes and fp32 scales: amax / 448, x / scale in fp32."""
    k = np.asarray(k, np.float32)
    top = np.abs(k).max(axis=1)
    s = np.where(top > 0, top / np.float32(448), np.float32(1)).astype(np.float32)
    return e4m3_nearest((k / s[:, None]).astype(np.float32).astype(np.float64)), s


# ------------------------------------------------------------------------------- geometry

class Pages:
    """Sequences over paged (or contiguous) caches: new tokens, contexts, a scattered table."""

    def __init__(self, new, ctx, paged=True, spare=2, seed=0, device="cuda", max_seqlen=None):
        self.new, self.ctx = list(new), list(ctx)
        self.batch, self.rows = len(ctx), sum(new)
        self.max_seqlen = max_seqlen or max(ctx)
        rng = np.random.default_rng(seed)
        if paged:
            per = [(c + 63) // 64 for c in ctx]
            perm = rng.permutation(sum(per) + spare)
            width = (self.max_seqlen + 63) // 64
            table = np.zeros((self.batch, width), np.int32)
            at = 0
            for b, n in enumerate(per):
                table[b, :n] = perm[at:at + n]
                at += n
            self.table, self.kv_rows = table, (sum(per) + spare) * 64
        else:
            self.table, self.kv_rows = None, (self.batch * self.max_seqlen + 63) // 64 * 64
        self.cu = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        dev = lambda a: torch.tensor(a, dtype=torch.int32, device=device)
        self.d_cu, self.d_ctx = dev(self.cu), dev(self.ctx)
        self.d_table = dev(self.table) if paged else None

    def phys(self, b, pos):
        pos = np.asarray(pos, np.int64)
        if self.table is None:
            return b * self.max_seqlen + pos
        return self.table[b, pos // 64].astype(np.int64) * 64 + pos % 64

    def row(self, r):
        """(sequence, position) of query row r."""
        b = int(np.searchsorted(self.cu, r, side="right") - 1)
        return b, self.ctx[b] - (int(self.cu[b + 1]) - r)

    def problem(self, dsa, d, topk, mode="chunk", sigma=None):
        return dsa.make_problem(mode=mode, topk=topk, softmax_scale=sigma or d["d_qk"] ** -0.5,
                                num_kv_rows=self.kv_rows,
                                seqlens=self.new if mode == "chunk" else self.ctx,
                                cu_seqlens=self.d_cu, seq_lens=self.d_ctx,
                                block_table=self.d_table, max_seqlen=self.max_seqlen, **d)


def latents(n, d, seed, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    size = torch.exp(0.5 * torch.randn(n, 1, generator=g, device=device))
    return (torch.randn(n, d["d_qk"], generator=g, device=device) * size).to(torch.bfloat16)


def random_selection(pages: Pages, topk, seed, holes=0.0):
    """int32 [rows, topk]: distinct keys of each row in increasing order, then -1 (and a share of
    the entries replaced by -1)."""
    rng = np.random.default_rng(seed)
    idx = np.full((pages.rows, topk), -1, np.int32)
    for r in range(pages.rows):
        _, pos = pages.row(r)
        k = min(topk, pos + 1)
        idx[r, :k] = np.sort(rng.permutation(pos + 1)[:k])
        if holes:
            idx[r, rng.random(topk) < holes] = -1
    return idx


# ------------------------------------------------------------------------------- attention

def attention(q, keys, sel, sigma, d_v):
    """One row in float64: q [h, d_qk], keys [n, d_qk] (logical order), sel logical keys.
    Returns out, lse and the bounds on their errors."""
    h = q.shape[0]
    sel = sel[sel >= 0]
    if len(sel) == 0:
        z = torch.zeros(h, d_v, dtype=torch.float64, device=q.device)
        ninf = torch.full((h,), -math.inf, dtype=torch.float64, device=q.device)
        return z, ninf, z, torch.zeros(h, dtype=torch.float64, device=q.device)
    kv = keys[sel]
    l = q @ kv.T * sigma
    D = (q.shape[1] / 16 + 1) * 2.0 ** -22 * sigma * (q.abs() @ kv.abs().T).amax(dim=1)
    lse = torch.logsumexp(l, dim=1)
    p = torch.exp(l - lse[:, None])
    out = p @ kv[:, :d_v]
    A = p @ kv[:, :d_v].abs()
    tol = A * (U + 2 * D[:, None] + 2.0 ** -18) + U * out.abs()
    return out, lse, tol, D + 2.0 ** -18 + 2.0 ** -22 * lse.abs()


def check_attention_rows(out, lse, q, values, idx, pages: Pages, sigma, d, rows=None, what=""):
    """out, lse of the library against attention() on `values` ([kv_rows, d_qk] float64, the
    cache's contents by physical row).  idx None: every key of the row."""
    for r in (range(pages.rows) if rows is None else rows):
        b, pos = pages.row(r)
        if pos < 0:
            keys = values[:0]
            sel = torch.zeros(0, dtype=torch.long, device=values.device)
        else:
            keys = values[torch.as_tensor(pages.phys(b, np.arange(pos + 1)), device=values.device)]
            sel = (torch.arange(pos + 1, device=values.device) if idx is None
                   else idx[r].long())
        ro, rl, to, tl = attention(q[r].double(), keys, sel, sigma, d["d_v"])
        eo = (out[r].double() - ro).abs() - to
        assert (eo <= 0).all(), f"{what} row {r}: out off by {eo.max().item():.3e} over its bound"
        fin = torch.isfinite(rl)
        assert torch.equal(fin, torch.isfinite(lse[r])), f"{what} row {r}: -inf pattern"
        el = ((lse[r].double() - rl).abs() - tl)[fin]
        assert el.numel() == 0 or (el <= 0).all(), f"{what} row {r}: LSE off by {el.max().item():.3e}"


# ------------------------------------------------------------------------------- indexer

def indexer_inputs(rows, kv_rows, d, seed, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device=device)
    f8 = lambda x: x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).contiguous()
    q8 = f8(rnd(rows, d["h_idx"], d["d_idx"]) * 100)
    qs = torch.rand(rows, d["h_idx"], generator=g, device=device) * 0.02 + 0.001
    w = torch.rand(rows, d["h_idx"], generator=g, device=device)
    k8 = f8(rnd(kv_rows, d["d_idx"]) * 100)
    ks = torch.rand(kv_rows, generator=g, device=device) * 0.02 + 0.001
    return q8, qs, w, k8, ks


def interleave(k8, ks):
    nb, d = k8.shape[0] // 64, k8.shape[1]
    return torch.cat([k8.reshape(nb, 64 * d), ks.view(torch.uint8).reshape(nb, 256)],
                     dim=1).contiguous()


def scores_row(q8, qs, w, k8, ks, pages: Pages, r):
    """float64 scores of row r over keys 0..pos."""
    b, pos = pages.row(r)
    rows = torch.as_tensor(pages.phys(b, np.arange(max(pos + 1, 0))), device=q8.device)
    val = torch.as_tensor(e4m3_values(), device=q8.device)
    dots = torch.relu(val[q8[r].long()] @ val[k8[rows].long()].T)
    return ((w[r].double() * qs[r].double()) @ dots) * ks[rows].double()
