"""64-bit references and input builders of the paged-cache tests (test infrastructure only).

Rounding: u = eps/2 of the 16-bit type (bf16 2^-8, fp16 2^-11).  Bounds of the attention
output, per element, with A = sum_t w_t |v_t| (the reference run on |V|):
  * every probability is rounded to the type before the second product: <= u A;
  * the result is rounded to the type: <= u (|ref| + the error before it);
  * fp32: a score is a sum of D products, off by at most D 2^-24 sum_d |q_d k_d| scale; the
    tests' inputs keep that below 6e-5 (D = 128, sum |q k| <= 100 at unit variance, scale
    D^-1/2), so that a probability and the sum of them are off by 2 * 6e-5 together, plus
    2^-21 for the exponentials: 1.5e-4 A in all;
  * fp16 probabilities below 2^-14 round by up to 2^-25 (the row's sum is at least 1, the
    running maximum being at most the true one): <= 2^-25 * keys * max |v|.
The log-sum-exp is off by the score bound, 6e-5, plus a few steps of fp32 (2^-22 |lse|).
"""
import numpy as np
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def ceil_div(a, b):
    return -(-a // b)


# ------------------------------------------------------------------------------- step
def step_reference(cache_lens, new_lens, table, free_pages, free_count, page, rows):
    """xs_paged_step by its definition, one request after the other.  numpy int arrays."""
    n, width = table.shape
    n_pages = len(free_pages)
    table, free = table.copy(), free_pages.copy()
    status, kv = np.zeros(n, np.int32), np.zeros(n, np.int32)
    fc = min(max(int(free_count), 0), n_pages)
    pages = list(free[:fc])
    ended = [False] * n
    for i in range(n):
        c, a = int(cache_lens[i]), int(new_lens[i])
        if c < 0 or ceil_div(max(c, 0) + max(a, 0), page) > width:
            status[i] = 2
        elif a < 0:
            ended[i] = True
            pages += list(table[i, :ceil_div(c, page)])
    pages = pages[:n_pages]
    free[fc:len(pages)] = pages[fc:]
    seen = 0
    for i in range(n):
        if status[i] == 0 and not ended[i] and new_lens[i] > 0:
            seen += int(new_lens[i])
            if seen > rows:
                status[i] = 3
    want, taken = 0, 0
    cu = [0]
    pos_out, slot_out = np.zeros(rows, np.int32), np.full(rows, -1, np.int64)
    for i in range(n):
        c, a = max(int(cache_lens[i]), 0), int(new_lens[i])
        tokens = a if status[i] == 0 and not ended[i] else 0
        if tokens > 0:
            held, need = ceil_div(c, page), ceil_div(c + a, page) - ceil_div(c, page)
            want += need
            if need > 0 and want > len(pages):
                status[i], tokens = 1, 0
            else:
                for j in range(need):
                    table[i, held + j] = pages[len(pages) - 1 - (want - need + j)]
                taken = max(taken, want) if need else taken
        for j in range(tokens):
            p = c + j
            pos_out[cu[-1] + j] = p
            e = int(table[i, p // page])
            slot_out[cu[-1] + j] = e * page + p % page if 0 <= e < n_pages else -1
        cu.append(cu[-1] + tokens)
        kv[i] = 0 if ended[i] else c + tokens
    return dict(table=table, free=free, kv_lens=kv, cu_q=np.array(cu, np.int32), positions=pos_out, slots=slot_out,
                free_count=len(pages) - taken, status=status)


# ------------------------------------------------------------------------------- rope
def frequencies(rot, base=10000.0, scaling="plain", factor=1.0, context=0.0, low=1.0, high=32.0):
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "stretch":
        base = base * factor ** (rot / (rot - 2))
    theta = base ** (-2 * i / rot)
    if scaling == "linear":
        theta = theta / factor
    if scaling == "by_parts":
        keep = np.clip((theta * context / (2 * np.pi) - low) / (high - low), 0, 1)
        theta = theta * keep + theta / factor * (1 - keep)
    return theta


def rope_reference(x, positions, theta, interleaved, magnitude=1.0, sign=1):
    """x: float64 [T, H, D]; returns (rotated, sum of the pair's magnitudes per channel)."""
    rot = 2 * len(theta)
    t = sign * positions.astype(np.float64)[:, None, None] * theta
    c, s = magnitude * np.cos(t), magnitude * np.sin(t)
    y, mass = x.copy(), np.abs(x) * 0
    lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = x[..., lo], x[..., hi]
    y[..., lo], y[..., hi] = a * c - b * s, a * s + b * c
    mass[..., lo] = mass[..., hi] = abs(magnitude) * (np.abs(a) + np.abs(b))
    return y, mass


def rope_tolerance(ref, mass, dtype):
    """Half a step of the type, plus fp32: an angle off by pi 2^-24 (its conversion to fp32)
    and sines and cosines off by two steps of 2^-23, with their products and sums."""
    return U[dtype] * np.abs(ref) * 1.0001 + (np.pi * 2.0 ** -24 + 4 * 2.0 ** -23) * mass + 2.0 ** -25


# -------------------------------------------------------------------------- attention
def attention_reference(q, k, v, kv_len, causal, window, scale):
    """One sequence and head in float64: q [nq, D], k and v [kv_len, D] -> out, mass, lse."""
    nq = q.shape[0]
    p = kv_len - nq + np.arange(nq)[:, None]
    t = np.arange(kv_len)[None, :]
    seen = np.ones((nq, kv_len), bool)
    if causal:
        seen &= t <= p
    if window:
        seen &= t > p - window
    x = np.where(seen, scale * (q @ k.T), -np.inf) if kv_len else np.zeros((nq, 0))
    m = x.max(axis=1, initial=-np.inf)
    w = np.exp(x - np.where(np.isinf(m), 0, m)[:, None])
    total = w.sum(axis=1)
    some = total > 0
    w = w / np.where(some, total, 1)[:, None]
    lse = np.where(some, m + np.log(np.where(some, total, 1)), -np.inf)
    return w @ v, w @ np.abs(v), lse


class PagedCase:
    """A batch over a paged cache.  Everything the operator must not read holds NaN: pages of
    nobody, page rows past a sequence, and (window) pages before what any row sees.  ``freed``:
    such pages' table entries are replaced by an out-of-range number."""

    def __init__(self, q_lens, kv_lens, H, Hkv, D, page, dtype=torch.bfloat16, seed=0, heads_first=False, one_buffer=False,
                 extra_rows=0, q_pad=0, width=None, table_pad=0, window=0, freed=False, gain=1.0, device="cuda"):
        r = np.random.default_rng(seed)
        self.q_lens, self.kv_lens = list(q_lens), list(kv_lens)
        self.H, self.Hkv, self.D, self.page, self.dtype = H, Hkv, D, page, dtype
        n = self.n = len(self.q_lens)
        rows = sum(self.q_lens)
        self.T = max(1, rows + extra_rows)
        held = [ceil_div(c, page) for c in self.kv_lens]
        n_pages = sum(held) + 5
        order = r.permutation(n_pages)
        width = max(max(held), 1) + 2 if width is None else width
        table = r.integers(-(1 << 30), 1 << 30, size=(n, width + table_pad))   # nonsense where nothing is to be read
        k = np.full((n_pages, page, Hkv, D), np.nan)
        v = np.full((n_pages, page, Hkv, D), np.nan)
        self.keys, self.values, at = [], [], 0
        for i in range(n):
            c = self.kv_lens[i]
            ki, vi = (gain * r.standard_normal((c, Hkv, D)) for _ in range(2))
            ki, vi = (torch.from_numpy(x).to(dtype).double().numpy() for x in (ki, vi))
            self.keys.append(ki)
            self.values.append(vi)
            first_seen = max(0, c - self.q_lens[i] - window + 1) if window else 0
            for j in range(held[i]):
                e = order[at + j]
                lo, hi = j * page, min(c, (j + 1) * page)
                if j < width:
                    table[i, j] = e
                if hi <= first_seen and freed:
                    table[i, j] = n_pages + 7
                    continue
                k[e, :hi - lo], v[e, :hi - lo] = ki[lo:hi], vi[lo:hi]
            at += held[i]
        q = torch.from_numpy(r.standard_normal((self.T, H + q_pad, D))).to(dtype)
        self.q64 = q[:, :H].double().numpy()
        self.q = q.to(device)[:, :H]
        to = lambda x: torch.from_numpy(x).to(dtype).to(device)   # noqa: E731
        if one_buffer:      # K and V of a page side by side
            kv = to(np.stack([k, v], axis=1))
            self.k, self.v = kv[:, 0], kv[:, 1]
        elif heads_first:
            self.k, self.v = (to(np.ascontiguousarray(x.transpose(0, 2, 1, 3))).transpose(1, 2) for x in (k, v))
        else:
            self.k, self.v = to(k), to(v)
        self.table = torch.from_numpy(table.astype(np.int32)).to(device)[:, :width]
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(self.q_lens)]), dtype=torch.int32, device=device)
        self.kv = torch.tensor(self.kv_lens, dtype=torch.int32, device=device)

    def reference(self, causal, window, scale, heads=None):
        """out, mass [T, H, D], lse [T, H] (rows past the sequences: NaN)."""
        out, mass = (np.full((self.T, self.H, self.D), np.nan) for _ in range(2))
        lse = np.full((self.T, self.H), np.nan)
        row, G = 0, self.H // self.Hkv
        for i in range(self.n):
            nq = self.q_lens[i]
            for h in (range(self.H) if heads is None else heads):
                o, a, z = attention_reference(self.q64[row:row + nq, h], self.keys[i][:, h // G],
                                              self.values[i][:, h // G], self.kv_lens[i], causal, window, scale)
                out[row:row + nq, h], mass[row:row + nq, h], lse[row:row + nq, h] = o, a, z
            row += nq
        return out, mass, lse

    def check(self, out, lse, causal, window, scale, heads=None, where=""):
        ref, mass, z = self.reference(causal, window, scale, heads)
        rows = sum(self.q_lens)
        hs = list(range(self.H)) if heads is None else list(heads)
        got = out.double().cpu().numpy()[:rows][:, hs]
        ref, mass, z = ref[:rows][:, hs], mass[:rows][:, hs], z[:rows][:, hs]
        vmax = max((np.abs(v).max() for v in self.values if v.size), default=0.0)
        u = U[self.dtype]
        before = u * mass + 1.5e-4 * mass + 2.0 ** -25 * max(self.kv_lens + [0]) * vmax * (self.dtype == torch.float16)
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
