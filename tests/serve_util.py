"""The serving operators in 64 bits (numpy) and the ragged, paged inputs of their tests."""
from __future__ import annotations

import numpy as np
import torch

import hybrid_attention_ssm_hymba_b200 as H
from hybrid_attention_ssm_hymba_b200 import host

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
CACHE = {"f32": H.HYMBA_CACHE_F32, "bf16": H.HYMBA_CACHE_BF16, "e4m3": H.HYMBA_CACHE_E4M3}
DTYPE = {"f32": H.HYMBA_F32, "bf16": H.HYMBA_BF16}
TINY = np.float32(2.0 ** -126)
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def quantise_e4m3(x):
    """x [..., dh] fp32 -> (codes as a float8 tensor, scales): the documented fp32 steps, each
    of which IEEE arithmetic fixes to the last bit."""
    x = np.asarray(x, np.float32)
    amax = np.abs(x).max(axis=-1)
    scale = np.maximum(amax / np.float32(448), TINY).astype(np.float32)
    with np.errstate(invalid="ignore"):
        y = x * (np.float32(1) / scale)[..., None]
    return torch.from_numpy(y).to(torch.float8_e4m3fn), scale


class Paged:
    """A paged cache of random rows with shuffled pages, and a ragged batch over it.
    `ns`: new rows, `pasts`: rows before them.  Rows the batch does not own hold NaN."""

    def __init__(self, dtype, cache, hkv, dh, page, ns, pasts, seed=0, pad=3, spare=2, device="cuda"):
        self.dtype, self.cache, self.hkv, self.dh, self.page = dtype, cache, hkv, dh, page
        self.ns, self.lens = np.array(ns), np.array(ns) + np.array(pasts)
        self.batch, self.device = len(ns), device
        r = self.rng = np.random.default_rng(seed)
        need = -(-self.lens // page)
        self.n_pages = int(need.sum()) + spare
        order = r.permutation(self.n_pages)
        self.table = np.full((self.batch, int(need.max()) + 2), -7, np.int32)
        at = 0
        for b in range(self.batch):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
        self.first = np.concatenate([[0], np.cumsum(self.ns)]).astype(np.int32)
        self.total = int(self.first[-1]) + pad
        self.pages = torch.full((2, self.n_pages, page, hkv, dh), float("nan")).to(TORCH[cache])
        self.scales = torch.full((2, self.n_pages, hkv, page), float("nan")) if cache == "e4m3" else None
        for b in range(self.batch):
            for which in range(2):
                x = r.standard_normal((self.lens[b], hkv, dh)).astype(np.float32) * \
                    np.exp(r.uniform(-2, 1, (self.lens[b], hkv, 1))).astype(np.float32)
                self.put(which, b, 0, x)

    def slots(self, b, lo, hi):
        rows = np.arange(lo, hi)
        return torch.from_numpy(self.table[b, rows // self.page].astype(np.int64)), torch.from_numpy(rows % self.page)

    def put(self, which, b, lo, x):
        pg, at = self.slots(b, lo, lo + len(x))
        if self.cache == "e4m3":
            codes, scale = quantise_e4m3(x)
            self.pages[which].view(torch.uint8)[pg, at] = codes.view(torch.uint8)
            self.scales[which][pg, :, at] = torch.from_numpy(scale)
        else:
            self.pages[which][pg, at] = torch.from_numpy(np.asarray(x, np.float32)).to(TORCH[self.cache])

    def rows(self, which, b, lo, hi, pages=None, scales=None):
        """Cache rows [lo, hi) of sequence b in 64 bits [rows, hkv, dh]."""
        pages = self.pages if pages is None else pages
        scales = self.scales if scales is None else scales
        pg, at = self.slots(b, lo, hi)
        if self.cache == "e4m3":
            x = pages[which].view(torch.uint8)[pg, at].view(torch.float8_e4m3fn).float().double().numpy()
            return x * scales[which][pg, :, at].double().numpy()[..., None]
        return pages[which][pg, at].double().numpy()

    def upload(self):
        d = self.device
        self.g_pages = self.pages.to(d)
        self.g_scales = None if self.scales is None else self.scales.to(d)
        self.g_table = torch.from_numpy(self.table).to(d)
        self.g_first = torch.from_numpy(self.first).to(d)
        self.g_lens = torch.from_numpy(self.lens.astype(np.int32)).to(d)
        self.kv = H.make_paged_kv(self.g_pages, self.g_table, self.page, self.hkv, self.dh, CACHE[self.cache],
                                  scales=self.g_scales)
        return self

    # ---- the three calls (raise on a non-OK status)
    def attend(self, q, out, hq, meta, window, max_rows=None, ws=None, q_ld=None, out_ld=None, stream=None):
        most = int(max(1, self.ns.max())) if max_rows is None else max_rows
        if ws is None:
            ws = self.workspace(hq, most)
        H.check(H.hymba_paged_attention(q, q_ld or hq * self.dh, self.kv, out, out_ld or hq * self.dh, self.batch,
                                        self.g_first, self.g_lens, self.total, most, hq, meta, window,
                                        DTYPE[self.dtype], ws, stream=stream), "paged_attention")
        return ws

    def workspace(self, hq, most=None):
        most = int(max(1, self.ns.max())) if most is None else most
        n = H.hymba_paged_attention_workspace_size(self.kv, self.batch, self.total, most, hq, DTYPE[self.dtype])
        assert n >= 256
        return host.workspace(n)

    def append(self, k, v, ld, ws=None, stream=None):
        ws = host.workspace(256) if ws is None else ws
        H.check(H.hymba_paged_kv_append(self.kv, k, v, ld, self.batch, self.g_first, self.g_lens, self.total,
                                        DTYPE[self.dtype], ws, stream=stream), "paged_kv_append")
        return ws

    def read(self, k, v, ld, ws=None, stream=None):
        ws = host.workspace(256) if ws is None else ws
        H.check(H.hymba_paged_kv_read(self.kv, k, v, ld, self.batch, self.g_first, self.g_lens, self.total,
                                      DTYPE[self.dtype], ws, stream=stream), "paged_kv_read")
        return ws

    # ---- the oracle
    def visible(self, b, meta, window):
        i = np.arange(self.lens[b] - self.ns[b], self.lens[b])[:, None]
        j = np.arange(self.lens[b])[None]
        return (j <= i) & ((window < 0) | (i - j <= window) | (j < meta))

    def attention(self, q, hq, meta, window, hidden=None):
        """(out, tolerance) [total, hq, dh] in 64 bits; rows outside the batch are NaN.  `hidden`
        (b, j) -> bool: keys whose page number is invalid.

        The tolerance, with A = sum_j p_j |v_j|: bf16 rounds P once (half a step of p_j v_j
        each, so HALF_STEP * A in all) and the output once; fp32 sums of dh products and of L
        terms add (dh + 2) 2^-24 sum |q k| to a score (twice that to p, after the scale) and
        (L + 16) 2^-23 A to the sums."""
        out = np.full((self.total, hq, self.dh), np.nan)
        tol = np.zeros_like(out)
        g = hq // self.hkv
        for b in range(self.batch):
            if self.ns[b] == 0:
                continue
            k, v = self.rows(0, b, 0, self.lens[b]), self.rows(1, b, 0, self.lens[b])
            k, v = np.nan_to_num(k), np.nan_to_num(v)
            see = self.visible(b, meta, window)
            if hidden is not None:
                see = see & ~np.array([hidden(b, j) for j in range(self.lens[b])])[None]
            at = slice(self.first[b], self.first[b + 1])
            for h in range(hq):
                qq = q[at, h]
                s = np.where(see, qq @ k[:, h // g].T / np.sqrt(self.dh), -np.inf)
                m = s.max(1, keepdims=True)
                p = np.exp(s - np.where(np.isfinite(m), m, 0.0))
                p /= np.maximum(p.sum(1, keepdims=True), 1e-300)
                out[at, h] = p @ v[:, h // g]
                a = p @ np.abs(v[:, h // g])
                ds = np.where(see, np.abs(qq) @ np.abs(k[:, h // g]).T, 0).max() / np.sqrt(self.dh) * \
                    (self.dh + 2) * 2.0 ** -24
                t = a * (2 * ds + (self.lens[b] + 16) * 2.0 ** -23) + np.abs(out[at, h]) * HALF_STEP[self.dtype]
                if self.dtype == "bf16":
                    t += a * HALF_STEP["bf16"]
                tol[at, h] = t
        return out, tol
