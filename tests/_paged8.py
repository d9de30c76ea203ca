"""64-bit references and input builders of the 8-bit paged cache's tests (test infrastructure only).

An element is an e4m3 number (4 significant bits, steps of 2^-9 below 2^-6) times a power of two.
Rounding to e4m3 is off by at most half a step: 2^-4 relative, or 2^-10 of the scale.

Bounds of the attention output, per element, with A = sum_t w_t |v_t| (the reference run on |V|)
and u = eps/2 of the output's type:
  * a probability is rounded to fp16 before the second product: <= 2^-11 A, and below 2^-14 (of the
    largest product of a probability and its block's scale) by up to 2^-25: <= 2^-25 keys vmax, vmax
    the largest 448 * scale;
  * the result is rounded to the type: <= u (|ref| + the error before it);
  * fp32 scores and sums: 1.5e-4 A in all, as in _paged.py (sum |q k| scale D^1/2 <= 100 per score).
The log-sum-exp is off by the score bound, 6e-5, plus a few steps of fp32 (2^-22 |lse|).
"""
import numpy as np
import torch

import _paged as pg

NAN_CODE = 0x7F      # what nothing may read is NaN, with a scale of no value
NO_SCALE = 255


def nearest(y):
    """The nearest e4m3 numbers to finite values of magnitude up to 448, ties to even."""
    step = np.exp2(np.maximum(np.frexp(y)[1] - 1, -6) - 3.0)
    return np.rint(y / step) * step


def need(a):
    """The least exponent e >= -64 with a <= 448 * 2^e."""
    m, e = np.frexp(a)
    return np.where(a > 0, np.maximum(e - 9 + (m > 0.875), -64), -64)


def codes(values):
    """Bytes of e4m3 numbers."""
    return torch.from_numpy(np.ascontiguousarray(values)).to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8)


def numbers(code):
    return code.view(torch.float8_e4m3fn).float().double().cpu().numpy()


def append_reference(num, exp, x, slots, block):
    """Rows x [T, Hkv, D] into a cache of numbers [pages, page, Hkv, D] and exponents [pages, page / block, Hkv], by
    the definition, one run after the other; both are changed in place."""
    pages, page = num.shape[:2]
    t, T = 0, len(slots)
    while t < T:
        s = int(slots[t])
        if not 0 <= s < pages * page:
            t += 1
            continue
        end = t + 1
        while end < T and slots[end] == slots[end - 1] + 1 and slots[end] % block:
            end += 1
        at, off = divmod(s, page)
        b, o = off // block, off % block
        e = need(np.abs(x[t:end]).max(axis=(0, 2)))
        if o:
            old = exp[at, b]
            e = np.maximum(e, old)
            kept = num[at, off - o:off]
            kept[:] = nearest(kept * np.exp2(old - e.astype(float))[:, None])
        exp[at, b] = e
        num[at, off:off + end - t] = nearest(x[t:end] * np.exp2(-e.astype(float))[:, None])
        t = end


def to_cache(code, scale, heads_first, device, one_buffer=None):
    """uint8 arrays [pages, page, Hkv, D] and [pages, blocks, Hkv] as device tensors of that shape."""
    code, scale = torch.as_tensor(code).to(device), torch.as_tensor(scale).to(device)
    if heads_first:
        code, scale = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (code, scale))
    return code.view(torch.float8_e4m3fn), scale.view(torch.float8_e8m0fnu)


class Paged8Case(pg.PagedCase):
    """A batch over an 8-bit cache.  Pages of nobody, page rows past a sequence and (window) pages before what any row
    sees hold NaN, blocks without a token that is read have no scale; ``freed``: such pages' table entries are
    out of range.  Blocks' magnitudes differ by powers of two up to 2^spread either way."""

    def __init__(self, q_lens, kv_lens, H, Hkv, D, page, block=16, dtype=torch.bfloat16, seed=0, heads_first=False,
                 one_buffer=False, extra_rows=0, q_pad=0, table_pad=0, window=0, freed=False, gain=1.0, spread=1,
                 v_spread=None, device="cuda"):
        r = np.random.default_rng(seed)
        self.q_lens, self.kv_lens = list(q_lens), list(kv_lens)
        self.H, self.Hkv, self.D, self.page, self.block, self.dtype = H, Hkv, D, page, block, dtype
        n = self.n = len(self.q_lens)
        rows = sum(self.q_lens)
        self.T = max(1, rows + extra_rows)
        held = [pg.ceil_div(c, page) for c in self.kv_lens]
        n_pages, blocks = sum(held) + 5, page // block
        order = r.permutation(n_pages)
        width = max(max(held), 1) + 2
        table = r.integers(-(1 << 30), 1 << 30, size=(n, width + table_pad))   # nonsense where nothing is to be read
        caches = [(np.full((n_pages, page, Hkv, D), NAN_CODE, np.uint8), np.full((n_pages, blocks, Hkv), NO_SCALE, np.uint8))
                  for _ in range(2)]
        self.keys, self.values, self.vmax, at = [], [], 0.0, 0
        for i in range(n):
            c = self.kv_lens[i]
            first_seen = max(0, c - self.q_lens[i] - window + 1) if window else 0
            for j in range(held[i]):
                if j < width:
                    table[i, j] = n_pages + 7 if freed and min(c, (j + 1) * page) <= first_seen else order[at + j]
            for (code, scale), store, how in zip(caches, (self.keys, self.values), (spread, spread if v_spread is None else v_spread)):
                exp = r.integers(-how, how + 1, size=(pg.ceil_div(c, block), Hkv)) - 6
                num = nearest(np.clip(r.standard_normal((c, Hkv, D)) * 64, -448, 448))
                which = np.arange(c) // block
                store.append(gain * num * np.exp2(exp[which].astype(float))[..., None] if c else num)
                assert gain == 2.0 ** round(np.log2(gain))
                exp = exp + int(np.log2(gain))
                if c and store is self.values:
                    self.vmax = max(self.vmax, 448 * 2.0 ** exp.max())
                bytes_ = codes(num).numpy()
                for j in range(held[i]):
                    lo, hi = j * page, min(c, (j + 1) * page)
                    if hi <= first_seen:
                        continue
                    e = order[at + j]
                    code[e, :hi - lo] = bytes_[lo:hi]
                    b0, b1 = lo // block, pg.ceil_div(hi, block)
                    scale[e, :b1 - b0] = exp[b0:b1] + 127
            at += held[i]
        q = torch.from_numpy(r.standard_normal((self.T, H + q_pad, D))).to(dtype)
        self.q64 = q[:, :H].double().numpy()
        self.q = q.to(device)[:, :H]
        if one_buffer:      # K and V of a page side by side, and their scales
            both = [to_cache(np.stack([a[k] for a in caches], axis=1), np.zeros(1, np.uint8), False, device)[0].view(torch.uint8)
                    for k in (0, 1)]
            (self.k, self.v), (self.ks, self.vs) = ([b[:, i] for i in (0, 1)] for b in both)
            self.k, self.v = self.k.view(torch.float8_e4m3fn), self.v.view(torch.float8_e4m3fn)
        else:
            (self.k, self.ks), (self.v, self.vs) = (to_cache(*c, heads_first, device) for c in caches)
        self.cache = (self.k, self.v, self.ks, self.vs)
        self.table = torch.from_numpy(table.astype(np.int32)).to(device)[:, :width]
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(self.q_lens)]), dtype=torch.int32, device=device)
        self.kv = torch.tensor(self.kv_lens, dtype=torch.int32, device=device)

    def check(self, out, lse, causal, window, scale, heads=None, where=""):
        ref, mass, z = self.reference(causal, window, scale, heads)
        rows = sum(self.q_lens)
        hs = list(range(self.H)) if heads is None else list(heads)
        got = out.double().cpu().numpy()[:rows][:, hs]
        ref, mass, z = ref[:rows][:, hs], mass[:rows][:, hs], z[:rows][:, hs]
        u = pg.U[self.dtype]
        before = (2.0 ** -11 + 1.5e-4) * mass + 2.0 ** -25 * max(self.kv_lens + [0]) * self.vmax
        tol = before + u * (np.abs(ref) + before) + 1e-30
        assert np.isfinite(got).all(), f"{where}: {np.argwhere(~np.isfinite(got))[:4]}"
        bad = np.abs(got - ref) > tol
        assert not bad.any(), (f"{where}: {bad.sum()} of {bad.size} out of tolerance, first {np.argwhere(bad)[0]}, worst "
                               f"{(np.abs(got - ref) / tol).max():.2f} times")
        if rows and np.linalg.norm(ref):
            rel = np.linalg.norm(got - ref) / np.linalg.norm(ref)
            assert rel <= u, f"{where}: relative L2 {rel}"
        if lse is not None:
            g = lse.double().cpu().numpy()[:rows][:, hs]
            empty = np.isneginf(z)
            assert np.array_equal(np.isneginf(g), empty), where
            d = np.abs(g[~empty] - z[~empty])
            assert (d <= 6e-5 + 2.0 ** -22 * np.abs(z[~empty])).all(), f"{where}: lse off by {d.max(initial=0)}"
