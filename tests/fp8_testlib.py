"""The 8-bit cache for tests: a cache filled through the library, the definition of its bytes and
of its attention in float64, written from include/kvq.h and apart from the kernels."""
from __future__ import annotations

import math

import numpy as np
import torch

from rotated_int2_kv_kvq_gb300 import kvq as K

D, PAGE, REC = 128, 16, 4112


def i32(values):
    return torch.tensor([int(v) for v in values], dtype=torch.int32, device="cuda")


def cu_of(counts):
    return i32([0] + list(np.cumsum(counts, dtype=np.int64)))


def code_values():
    """The value of each of the 256 codes (NaN for 0x7f and 0xff)."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v[[127, 255]] = np.nan
    return np.where(b >= 128, -v, v)


def encode(x):
    """Nearest codes of x (float64, |x| <= 448 or NaN), ties to even, as uint8."""
    up = code_values()[:127]
    a = np.abs(x)
    hi = np.clip(np.searchsorted(up, np.nan_to_num(a)), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - up[lo], up[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.isnan(a), 127, code)
    # the sign of a NaN is not defined: callers compare NaN codes by their value
    return (code + np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def exponent(top):
    """The least e >= -100 with top <= 448 * 2^e."""
    if not top > 0:
        return -100
    e = math.ceil(math.log2(top / 448.0))
    while top > 448.0 * 2.0 ** e:
        e += 1
    while top <= 448.0 * 2.0 ** (e - 1):
        e -= 1
    return max(e, -100)


def places():
    """Byte of slot tau's element d in a record: keys, values [16, 128]."""
    k, v = np.zeros((PAGE, D), np.int64), np.zeros((PAGE, D), np.int64)
    for tau in range(PAGE):
        for d in range(D):
            w, r = d >> 4, d & 15
            t, e = (r >> 1) & 3, r & 1
            k[tau, d] = 512 * (w >> 1) + 16 * (4 * (tau & 7) + t) + 4 * ((tau >> 3) + 2 * (r >> 3)) \
                + 2 * (w & 1) + e
            t, e = (tau & 7) >> 1, tau & 1
            v[tau, d] = 2048 + 512 * (w >> 1) + 16 * (4 * (r & 7) + t) + 4 * (2 * (w & 1) + (r >> 3)) \
                + 2 * (tau >> 3) + e
    return k, v


PLACES = places()


class Model:
    """The definition, page by page: codes and exponents of a pool of `pages` pages."""

    def __init__(self, pages, hkv):
        self.hkv = hkv
        self.codes = np.zeros((2, pages, hkv, PAGE, D), np.uint8)
        self.e = np.full((2, pages, hkv), -100)
        self.nan = np.zeros((pages, hkv), np.uint32)
        self.known = np.zeros(pages, bool)           # begun by an append

    def append(self, k, v, new, lens, pt):
        """k, v: float64 [n, hkv, D]; new rows of each sequence, the last of its lens."""
        at = 0
        for b, (n, length) in enumerate(zip(new, lens)):
            p = length - n
            while p < length:
                count = min(PAGE - p % PAGE, length - p)
                self._page(int(pt[b, p // PAGE]), p % PAGE, k[at:at + count], v[at:at + count])
                p += count
                at += count

    def _page(self, page, slot, k, v):
        if slot == 0:
            self.codes[:, page] = 0
            self.e[:, page] = -100
            self.nan[page] = 0
            self.known[page] = True
        for which, x in enumerate((k, v)):
            for kv in range(self.hkv):
                fine = np.where(np.isfinite(x[:, kv]), x[:, kv], 0.0)
                e0 = self.e[which, page, kv]
                e = max(exponent(np.abs(fine).max()), e0)
                old = code_values()[self.codes[which, page, kv]] * 2.0 ** float(e0 - e)
                c = encode(old)
                y = np.where(np.isfinite(x[:, kv]), x[:, kv], np.nan) * 2.0 ** float(-e)
                c[slot:slot + len(y)] = encode(y)
                if np.isnan(y).any():
                    self.nan[page, kv] |= 1 << which
                self.codes[which, page, kv] = c
                self.e[which, page, kv] = e

    def check(self, pool, pages):
        """The bytes of `pages` in the library's pool."""
        rec = pool.cpu().numpy().reshape(-1, self.hkv, REC)[pages]
        scale = rec[..., 4096:4104].copy().view(np.float32)
        flags = rec[..., 4104:4112].copy().view(np.uint32)
        value = code_values()
        for which in range(2):
            assert np.array_equal(scale[..., which], 2.0 ** self.e[which][pages]), which
            got, want = rec[..., PLACES[which]], self.codes[which][pages]
            same = (got == want) | (np.isnan(value[got]) & np.isnan(value[want]))
            assert same.all(), (which, int((~same).sum()))
        assert np.array_equal(flags[..., 0], self.nan[pages]) and not flags[..., 1].any()


class Cache8:
    """An 8-bit cache of sequences with `lens` positions, filled through kvq_fp8_append."""

    def __init__(self, H, Hkv, lens, seed=0, extra=2, max_pages=None, scale_k=1.5, scale_v=1.0,
                 fill=True):
        self.H, self.Hkv, self.lens = H, Hkv, list(lens)
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.h = K.kvq_create(K.make_layout(H, Hkv))
        need = [(c + 15) // 16 for c in lens]
        self.pages = sum(need) + extra
        perm = np.random.default_rng(seed).permutation(self.pages).astype(np.int32)
        pt = np.full((len(lens), max([max_pages or 1] + need)), -1, np.int32)
        o = 0
        for b, m in enumerate(need):
            pt[b, :m] = perm[o:o + m]
            o += m
        self.pt = torch.from_numpy(pt).cuda()
        # 0xFF bytes: NaN wherever nothing is appended
        self.pool = torch.full((self.pages * Hkv * REC,), 255, dtype=torch.uint8, device="cuda")
        n = sum(lens)
        self.k = self.randn(max(n, 1), Hkv, scale=scale_k)
        self.v = self.randn(max(n, 1), Hkv, scale=scale_v)
        self.seq_lens = i32(self.lens)
        if n and fill:
            self.append(self.k[:n], self.v[:n], self.lens)

    def randn(self, n, heads, scale=1.0):
        return (scale * torch.randn(n, heads, D, generator=self.g, device="cuda")).bfloat16()

    def append(self, k, v, new, lens=None, pt=None):
        K.kvq_fp8_append(self.h, self.pool, self.pages, k, v, cu_of(new),
                         self.pt if pt is None else pt,
                         self.seq_lens if lens is None else i32(lens))

    def read(self, new, lens=None):
        n = sum(new)
        out = [torch.full((n, self.Hkv, D), 9.0, dtype=torch.bfloat16, device="cuda")
               for _ in range(2)]
        K.kvq_fp8_read(self.h, self.pool, self.pages, *out, cu_of(new), self.pt,
                       self.seq_lens if lens is None else i32(lens))
        return out

    def entries(self, b, length=None):
        """float64 keys and values [Hkv, len, 128] of sequence b, from the pool's bytes."""
        c = self.lens[b] if length is None else length
        ids = self.pt[b, :(c + 15) // 16].long()
        rec = self.pool.view(self.pages, self.Hkv, REC)[ids]
        scale = rec[..., 4096:4104].contiguous().view(torch.float32).double()
        value = torch.from_numpy(code_values()).cuda()
        got = []
        for which in range(2):
            x = value[rec[..., torch.from_numpy(PLACES[which]).cuda()].long()]
            x = x * scale[..., which, None, None]
            got.append(x.permute(1, 0, 2, 3).reshape(self.Hkv, -1, D)[:, :c])
        return got

    def decode(self, q, window=0, sinks=0, lens=None, out=None, ws=None, pt=None):
        B = self.pt.shape[0]
        out = torch.full((B, self.H, D), 9.0, device="cuda") if out is None else out
        if ws is None:      # contents on entry do not matter: NaN bytes
            ws = torch.full((K.kvq_fp8_workspace_bytes(self.h, B),), 255, dtype=torch.uint8,
                            device="cuda")
        K.kvq_fp8_decode(self.h, self.pool, self.pages, q, self.pt if pt is None else pt,
                         self.seq_lens if lens is None else i32(lens), out, ws, window=window,
                         sinks=sinks)
        return out

    def prefill(self, q, new, window=0, sinks=0, lens=None, out=None, ws=None, pt=None, cu=None):
        n, B = q.shape[0], self.pt.shape[0]
        if out is None:
            out = torch.full((n, self.H, D), 9.0, dtype=torch.bfloat16, device="cuda")
        if ws is None:
            ws = torch.full((K.kvq_fp8_prefill_workspace_bytes(self.h, B, n),), 255,
                            dtype=torch.uint8, device="cuda")
        K.kvq_fp8_prefill(self.h, self.pool, self.pages, q, cu_of(new) if cu is None else cu,
                          self.pt if pt is None else pt,
                          self.seq_lens if lens is None else i32(lens), out, ws, window=window,
                          sinks=sinks)
        return out


def seen(length, n, window, sinks):
    """[n, length] bool: what each of the last n positions sees."""
    row = torch.arange(length - n, length, device="cuda")[:, None]
    col = torch.arange(length, device="cuda")[None]
    mask = col <= row
    if window:
        mask &= (col > row - window) | (col < sinks)
    return mask


def attend(q, k, v, mask, scale=None):
    """float64 attention of q [n, D] over k, v [len, D]: output, sum of p |v|, and the largest
    sum of |q_d k_td| of a visible position (what a score's rounding is relative to)."""
    scale = scale or 1 / math.sqrt(D)
    s = (q @ k.T * scale).masked_fill(~mask, -math.inf)
    p = torch.nan_to_num(torch.softmax(s, 1))
    size = (q.abs() @ k.abs().T * scale).masked_fill(~mask, 0).amax(1)
    return p @ v, p @ v.abs(), size
