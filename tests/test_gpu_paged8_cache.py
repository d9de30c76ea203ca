"""xs_rope_append_paged8 and xs_paged_read8 on the GPU against their definitions in 64 bits (_paged8.py)."""
import numpy as np
import pytest

import _paged as pg
import _paged8 as p8

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def xs():
    from conftest import build_library
    build_library()
    import dit_attention_ulysses_gb300 as xs
    assert torch.cuda.is_available()
    return xs


class Append:
    """Rows for a cache in which every request holds `cached` tokens: requests' pages in any order, rows of a fused
    projection, magnitudes that differ by row.  What no token has been written to is NaN, without a scale."""

    def __init__(self, new, cached, Hkv, D, page, block, H=2, dtype=torch.bfloat16, seed=0, heads_first=False, pad=0,
                 spread=3, one_buffer=False):
        r = np.random.default_rng(seed)
        self.Hkv, self.D, self.page, self.block, self.dtype = Hkv, D, page, block, dtype
        held = [pg.ceil_div(a + c, page) for a, c in zip(new, cached)]
        pages, blocks = sum(held) + 2, page // block
        order, at = r.permutation(pages), 0
        self.num = [np.full((pages, page, Hkv, D), np.nan) for _ in range(2)]
        self.exp = [np.full((pages, blocks, Hkv), 128.0) for _ in range(2)]   # byte 255
        self.before = [np.full((pages, page, Hkv, D), p8.NAN_CODE, np.uint8) for _ in range(2)]
        slots, pos = [], []
        for a, c, n in zip(new, cached, held):
            mine = order[at:at + n]
            at += n
            for p in range(c, c + a):
                slots.append(mine[p // page] * page + p % page)
                pos.append(p)
            for num, exp, code in zip(self.num, self.exp, self.before):
                for j in range(pg.ceil_div(c, block)):
                    lo, hi = j * block, min(c, (j + 1) * block)
                    e, o = mine[lo // page], lo % page
                    exp[e, o // block] = r.integers(-12, -4, size=Hkv)
                    x = p8.nearest(np.clip(r.standard_normal((hi - lo, Hkv, D)) * 64, -448, 448))
                    num[e, o:o + hi - lo] = x
                    code[e, o:o + hi - lo] = p8.codes(x).numpy()
        T = self.T = len(slots) + pad
        # padding: negative, and the first slot past the cache
        slots += [-1 if i % 2 else pages * page for i in range(pad)]
        pos += [0] * pad
        self.slots, self.pos = np.array(slots, np.int64), np.array(pos, np.int32)
        x = r.standard_normal((T, H + 2 * Hkv, D)) * np.exp2(r.integers(-spread, spread + 1, size=(T, 1, 1)))
        if T > 3:
            x[r.integers(0, T, size=T // 4), :, :] = 0.0
        self.qkv = torch.from_numpy(x).to(dtype)
        self.x64 = self.qkv.double().numpy()
        qkv = self.qkv.cuda()
        self.q, self.k, self.v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        scales = [(e + 127).astype(np.uint8) for e in self.exp]
        if one_buffer:
            both = torch.from_numpy(np.stack(self.before, axis=1)).cuda(), torch.from_numpy(np.stack(scales, axis=1)).cuda()
            self.cache = [both[0][:, 0].view(torch.float8_e4m3fn), both[0][:, 1].view(torch.float8_e4m3fn), both[1][:, 0],
                          both[1][:, 1]]
        else:
            (k, ks), (v, vs) = (p8.to_cache(c, s, heads_first, "cuda") for c, s in zip(self.before, scales))
            self.cache = [k, v, ks, vs]
        self.slots_d, self.pos_d = torch.from_numpy(self.slots).cuda(), torch.from_numpy(self.pos).cuda()
        self.H = H

    def launch(self, xs, rope):
        if rope is None:
            xs.xs_rope_append_paged8(None, self.k, self.v, None, self.slots_d, None, *self.cache, None)
            out = None
        else:
            out = torch.full((self.T, self.H, self.D), float("nan"), dtype=self.dtype, device="cuda")
            xs.xs_rope_append_paged8(self.q, self.k, self.v, self.pos_d, self.slots_d, out, *self.cache, rope)
        torch.cuda.synchronize()
        return out

    def check_exact(self, i, x):
        """Cache i (0: K, 1: V) bit for bit after rows `x` have been appended by the definition."""
        num, exp = self.num[i].copy(), self.exp[i].copy()
        p8.append_reference(num, exp, x, self.slots, self.block)
        assert np.array_equal(self.cache[2 + i].view(torch.uint8).cpu().numpy(), (exp + 127).astype(np.uint8))
        want = p8.codes(num).numpy()
        want[np.isnan(num)] = p8.NAN_CODE
        got = self.cache[i].view(torch.uint8).cpu().numpy()
        assert np.array_equal(got, want), np.argwhere(got != want)[:5]


# new, cached, Hkv, D, page, block
APPENDS = [
    ([1], [0], 1, 64, 16, 16),
    ([1], [7], 1, 128, 16, 16),
    ([1] * 70, list(range(70)), 3, 128, 32, 32),
    ([1, 2, 3, 20, 5], [15, 14, 16, 3, 127], 2, 64, 128, 16),
    ([33, 31, 1, 64], [0, 31, 62, 64], 8, 128, 64, 32),
    ([300, 1, 7], [5, 63, 120], 5, 128, 128, 64),
    ([257, 130, 2], [100, 127, 126], 2, 128, 128, 128),
    ([400, 129], [1, 250], 2, 64, 256, 128),
    ([90, 90], [10, 1000], 4, 64, 1024, 64),
    ([1000], [0], 1, 128, 16, 16),
    ([513], [37], 7, 64, 64, 32),
]


@pytest.mark.parametrize("form", [dict(), dict(heads_first=True), dict(one_buffer=True)], ids=str)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("case", APPENDS, ids=lambda c: "T%d_kv%d_D%d_p%d_b%d" % (sum(c[0]), *c[2:]))
def test_append_without_rotation(xs, case, dtype, form):
    a = Append(*case, dtype=dtype, seed=sum(case[0]), pad=3, **form)
    a.launch(xs, None)
    H, Hkv = a.H, a.Hkv
    a.check_exact(0, a.x64[:, H:H + Hkv])
    a.check_exact(1, a.x64[:, H + Hkv:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("case,rot", [(APPENDS[i], r) for i, r in ((1, 128), (2, 48), (3, 64), (4, 128), (6, 16), (7, 32), (9, 128))],
                         ids=lambda c: str(c) if isinstance(c, int) else "T%d" % sum(c[0]))
def test_append_with_rotation(xs, case, rot, dtype, layout):
    a = Append(*case, dtype=dtype, seed=7, pad=2)
    rope = xs.Rope(a.D, rot, layout=("half", "interleaved").index(layout), base=5e5)
    out = a.launch(xs, rope)
    H, Hkv = a.H, a.Hkv
    plain = torch.empty_like(out)
    xs.xs_rope_fwd(a.q, a.pos_d, plain, rope)
    assert torch.equal(out, plain)                      # q: the rotation's own bits
    a.check_exact(1, a.x64[:, H + Hkv:])                # V: nothing but the quantisation
    x, mass = pg.rope_reference(a.x64[:, H:H + Hkv], a.pos, pg.frequencies(rot, base=5e5), layout == "interleaved")
    off = (np.pi * 2.0 ** -24 + 4 * 2.0 ** -23) * mass + 2.0 ** -25 * np.abs(x)    # of the fp32 values (_paged.py)
    num, exp = a.num[0].copy(), a.exp[0].copy()
    p8.append_reference(num, exp, x, a.slots, a.block)
    got_e = a.cache[2].view(torch.uint8).cpu().numpy().astype(float) - 127
    # a scale differs only where the largest magnitude lies within its error of 448 * 2^e
    differs = np.argwhere(got_e != exp)
    lo, hi = p8.need(np.abs(x) - off), p8.need(np.abs(x) + off)
    assert len(differs) <= (lo != hi).sum()
    assert np.abs(got_e - exp).max() <= 1
    got = p8.numbers(a.cache[0].view(torch.uint8))
    at = a.slots[:a.T - 2]
    p, o = at // a.page, at % a.page
    scale = np.exp2(got_e[p, o // a.block])[..., None]
    value, want = got[p, o] * scale, x[:a.T - 2]
    # half a step of e4m3 (2^-4 of the value, 2^-10 of the scale where it is larger) from the exact value
    tol = np.maximum(2.0 ** -4 * (np.abs(want) + off[:a.T - 2]), 2.0 ** -10 * scale) + off[:a.T - 2]
    assert (np.abs(value - want) <= tol).all()
    # and the tokens that were there, by the definition, wherever the scale is the same
    rows = np.zeros(num.shape[:2], bool)
    rows[p, o] = True
    same = np.repeat(got_e == exp, a.block, axis=1) & ~rows[..., None]
    w = np.where(np.isnan(num), 0, num)
    g = np.where(np.isnan(got), 0, got)
    assert np.array_equal(np.isnan(num), np.isnan(got)) and np.array_equal(g[same], w[same])


def test_a_token_at_a_time_is_near_all_at_once(xs):
    """A block that grows: its scale ends as if it had been written at once, and numbers that were moved to a larger
    scale are off by what they lost below 2^-6 at most."""
    Hkv, D, n = 3, 128, 64
    whole = Append([n], [0], Hkv, D, 64, 32, seed=3, spread=4)
    x = whole.x64[:, whole.H:]
    steps = Append([n], [0], Hkv, D, 64, 32, seed=3, spread=4)
    whole.launch(xs, None)
    for t in range(n):
        xs.xs_rope_append_paged8(None, steps.k[t:t + 1], steps.v[t:t + 1], None, steps.slots_d[t:t + 1], None, *steps.cache, None)
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(whole.cache[2 + i].view(torch.uint8), steps.cache[2 + i].view(torch.uint8))
        at = steps.slots
        p, o = at // 64, at % 64
        e = steps.cache[2 + i].view(torch.uint8).cpu().numpy()[p, o // 32].astype(float) - 127
        a, b = (p8.numbers(c.cache[i].view(torch.uint8))[p, o] for c in (whole, steps))
        want = x[:, i * Hkv:(i + 1) * Hkv] / np.exp2(e)[..., None]
        # each move rounds numbers below 2^-6 to steps of 2^-9; the moves halve, so all together add at most 2^-9
        assert (np.abs(b - want) <= np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10) + 2.0 ** -9).all()
        assert (a == b).mean() > 0.5


def test_append_is_repeatable_and_on_any_stream(xs):
    a, b = (Append([40, 1, 130], [3, 17, 60], 4, 128, 64, 64, seed=11) for _ in range(2))
    rope = xs.Rope(128, 64)
    first = a.launch(xs, rope)
    kept = [c.view(torch.uint8).clone() for c in a.cache]
    again = a.launch(xs, rope)                           # the same rows once more: the same cache
    assert torch.equal(first, again) and all(torch.equal(x, c.view(torch.uint8)) for x, c in zip(kept, a.cache))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(first)
    xs.xs_rope_append_paged8(b.q, b.k, b.v, b.pos_d, b.slots_d, out, *b.cache, rope, stream=side)
    side.synchronize()
    assert torch.equal(out, first) and all(torch.equal(x, c.view(torch.uint8)) for x, c in zip(kept, b.cache))


@pytest.mark.parametrize("value", [0.0, -0.0, 2.0 ** -70, 2.0 ** -100, 448 * 2.0 ** -10, 449 * 2.0 ** -10, 3.0e38, 1.0])
def test_append_of_extreme_magnitudes(xs, value):
    """One value everywhere: nothing, less than the least scale, on both sides of 448 * 2^e, near the type's largest."""
    a = Append([20], [0], 2, 64, 32, 16, seed=1, spread=0)
    x = torch.full((20, 2, 64), value, dtype=torch.bfloat16, device="cuda")
    x[::2] *= -1
    xs.xs_rope_append_paged8(None, x, x, None, a.slots_d, None, *a.cache, None)
    for i in range(2):
        a.check_exact(i, x.double().cpu().numpy())


# ------------------------------------------------------------------------------- read
# rows, first (None: 0), Hkv, D, page, block
READS = [
    ([1], None, 1, 64, 16, 16),
    ([40], [0], 2, 128, 16, 16),
    ([33, 0, 1, 64, 0], [5, 9, 0, 100, 0], 3, 128, 32, 16),
    ([200, 1000], [1000, 24], 8, 64, 128, 64),
    ([3] * 100, list(range(100)), 1, 128, 64, 32),
    ([1] * 700, None, 2, 64, 16, 16),
    ([0, 0, 500], None, 5, 128, 256, 128),
]


@pytest.mark.parametrize("form", [dict(), dict(heads_first=True), dict(one_buffer=True)], ids=str)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("case", READS, ids=lambda c: "n%d_%d_kv%d_D%d_p%d_b%d" % (len(c[0]), sum(c[0]), *c[2:]))
def test_read(xs, case, dtype, form):
    rows, first, Hkv, D, page, block = case
    start = first or [0] * len(rows)
    c = p8.Paged8Case([0] * len(rows), [a + b for a, b in zip(rows, start)], Hkv, Hkv, D, page, block, dtype=dtype, seed=5,
                      spread=12, table_pad=2, **form)
    T = sum(rows) + 4
    wide = [torch.full((T, Hkv + 1, D), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    out = [w[:, :Hkv] for w in wide]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32, device="cuda")
    f = None if first is None else torch.tensor(first, dtype=torch.int32, device="cuda")
    xs.xs_paged_read8(*c.cache, c.table, cu, f, *out)
    torch.cuda.synchronize()
    for o, w, values in zip(out, wide, (c.keys, c.values)):
        want = np.concatenate([v[s:s + a] for v, s, a in zip(values, start, rows)])
        most = torch.finfo(dtype).max
        assert torch.equal(o[:sum(rows)].cpu(), torch.from_numpy(np.clip(want, -most, most)).to(dtype))
        assert (o[sum(rows):] == 7).all() and (w[:, Hkv:] == 7).all()


def test_read_of_what_is_not_there(xs):
    """Pages out of range, positions before the first and past the table: zeros; more sequences' rows than fit: cut."""
    c = p8.Paged8Case([0, 0], [64, 64], 2, 2, 64, 16, seed=2)
    table = c.table[:, :4].clone()
    table[0, 1], table[1, 2] = -1, 1 << 20
    cu = torch.tensor([0, 80, 200], dtype=torch.int32, device="cuda")
    first = torch.tensor([0, -10], dtype=torch.int32, device="cuda")
    out = [torch.full((150, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    xs.xs_paged_read8(*c.cache, table, cu, first, *out)
    torch.cuda.synchronize()
    for o, values in zip(out, (c.keys, c.values)):
        want = np.zeros((150, 2, 64))
        want[:64] = values[0]
        want[16:32] = 0
        want[90:150] = values[1][:60]
        want[90 + 32:90 + 48] = 0
        assert torch.equal(o.cpu(), torch.from_numpy(want).bfloat16())


def test_read_saturates(xs):
    """Elements past fp16's largest number become it; bf16 holds them."""
    c = p8.Paged8Case([0], [16], 1, 1, 64, 16, seed=1)
    c.ks.view(torch.uint8)[c.table[0, 0].long()] = 127 + 15
    cu = torch.tensor([0, 16], dtype=torch.int32, device="cuda")
    for dtype in (torch.float16, torch.bfloat16):
        k, v = (torch.empty((16, 1, 64), dtype=dtype, device="cuda") for _ in range(2))
        xs.xs_paged_read8(*c.cache, c.table, cu, None, k, v)
        want = torch.from_numpy(c.keys[0]) / c.keys[0].max() * c.keys[0].max()
        num = p8.numbers(c.k.view(torch.uint8))[int(c.table[0, 0])][:16]
        want = torch.from_numpy(num * 2.0 ** 15)
        most = torch.finfo(dtype).max
        assert torch.equal(k.cpu(), want.clamp(-most, most).to(dtype))
