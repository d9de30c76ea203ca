"""The 8-bit paged cache at the ends of what it holds.  References and roundings: _paged8.py."""
import numpy as np
import pytest

import _paged as pg
import _paged8 as p8
from test_gpu_paged8_attn import _run
from test_gpu_paged8_cache import APPENDS, Append
from test_gpu_paged_attn import _run as _run16

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

DTYPES = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])


@pytest.fixture(scope="module")
def xs():
    from conftest import build_library
    build_library()
    import dit_attention_ulysses_gb300 as xs
    assert torch.cuda.is_available()
    return xs


def _same(got, want):
    assert np.array_equal(np.isnan(got), np.isnan(want)), np.argwhere(np.isnan(got) != np.isnan(want))[:5]
    bad = ~np.isnan(want) & (got != want)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])


# ------------------------------------------------------------------------------- read
def _read_all_numbers(xs, scales, dtype):
    """Every e4m3 number under each of the scale bytes, read back: got and wanted, [scale, number], of K and of V."""
    n = len(scales)
    code = torch.arange(256, dtype=torch.uint8).view(1, 2, 1, 128).repeat(n, 8, 1, 1)    # two tokens hold them all
    scale = torch.tensor(scales, dtype=torch.uint8).view(n, 1, 1)
    k, v = (c.cuda().view(torch.float8_e4m3fn) for c in (code, code.flip(-1)))
    table = torch.arange(n, dtype=torch.int32, device="cuda").view(1, n)
    out = [torch.full((16 * n, 1, 128), 7.0, dtype=dtype, device="cuda") for _ in "kv"]
    xs.xs_paged_read8(k, v, scale.cuda(), scale.cuda(), table, torch.tensor([0, 16 * n], dtype=torch.int32, device="cuda"), None, *out)
    number = code[0, :2].view(torch.float8_e4m3fn).float().double().numpy()
    with np.errstate(over="ignore"):
        # four bits times a power of two: exact in 32 bits, so that what follows is the one rounding
        by = [np.float64("nan") if s == 255 else 2.0 ** (s - 127) for s in scales]
        most = torch.finfo(dtype).max
        want = [torch.from_numpy(np.clip(number * b, -most, most)).float().to(dtype).double().numpy() for b in by]
    got = [o.double().cpu().numpy().reshape(n, 8, 2, 1, 128) for o in out]
    for o, flip in zip(got, (False, True)):
        for s in range(n):
            w = want[s][..., ::-1] if flip else want[s]
            for t in range(8):
                yield o[s, t], w


@DTYPES
def test_read_of_every_number_under_every_scale(xs, dtype):
    """numbers * scale, rounded once, what is past the type's largest its largest, NaN as NaN."""
    for got, want in _read_all_numbers(xs, list(range(1, 255)), dtype):
        _same(got, want)


@DTYPES
def test_read_of_a_scale_that_is_nan(xs, dtype):
    for got, want in _read_all_numbers(xs, [127, 255, 130], dtype):
        _same(got, want)


@DTYPES
def test_what_is_not_finite_comes_back(xs, dtype):
    """Appended, then read: NaN stays NaN beside its neighbours, an infinity becomes the type's largest number."""
    x = torch.ones((48, 2, 64), dtype=dtype, device="cuda")
    x[3, 0, 5], x[4, 1, 60] = float("nan"), float("nan")           # a block with NaN
    x[20, 0, 7], x[21, 0, 8], x[22, 1, 9] = float("inf"), float("-inf"), float("nan")
    cache = [torch.zeros((3, 16, 2, 64), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in "kv"] + \
            [torch.zeros((3, 1, 2), dtype=torch.uint8, device="cuda") for _ in "kv"]
    xs.xs_rope_append_paged8(None, x, -x, None, torch.arange(48, device="cuda"), None, *cache, None)
    table = torch.arange(3, dtype=torch.int32, device="cuda").view(1, 3)
    k, v = (torch.empty_like(x) for _ in "kv")
    xs.xs_paged_read8(*cache, table, torch.tensor([0, 48], dtype=torch.int32, device="cuda"), None, k, v)
    want = np.ones((48, 2, 64))
    want[3, 0, 5] = want[4, 1, 60] = want[22, 1, 9] = np.nan
    want[16:32, 0] = 0                                             # beside an infinity 1 is nothing
    most = torch.finfo(dtype).max
    want[20, 0, 7], want[21, 0, 8] = most, -most
    _same(k.double().cpu().numpy(), want)
    _same(v.double().cpu().numpy(), -want)


@DTYPES
def test_read_of_the_least_scale(xs, dtype):
    """Byte 0 stands for 2^-127 as every other for its power."""
    for got, want in _read_all_numbers(xs, [0, 1, 2], dtype):
        _same(got, want)


# ----------------------------------------------------------------------------- append
@pytest.mark.parametrize("before", [0, 1, 50, 62, 63, 64, 119, 247, 248, 253, 254])
@pytest.mark.parametrize("size", [2.0 ** -120, 1.0, 2.0 ** 124])
def test_append_under_a_scale_that_another_program_wrote(xs, before, size):
    """Rows into a begun block whose scale is any power of two: the numbers kept and the new ones by the definition."""
    a = Append([3, 40], [5, 18], 2, 64, 32, 16, seed=before, spread=0)
    a.x64 *= size
    x = torch.from_numpy(a.x64).to(a.dtype)
    a.x64 = x.double().numpy()
    k, v = (x[:, a.H + i * a.Hkv:a.H + (i + 1) * a.Hkv].cuda() for i in (0, 1))
    for i in (0, 1):
        given = a.exp[i] != 128
        a.exp[i][given] = before - 127
        a.cache[2 + i].view(torch.uint8)[torch.from_numpy(given).cuda()] = before
    xs.xs_rope_append_paged8(None, k, v, None, a.slots_d, None, *a.cache, None)
    a.check_exact(0, a.x64[:, a.H:a.H + a.Hkv])
    a.check_exact(1, a.x64[:, a.H + a.Hkv:])


def test_append_under_a_scale_that_is_nan(xs):
    """A begun block whose scale is NaN: it stays so, and what is appended is NaN by itself too."""
    a = Append([3], [5], 1, 64, 16, 16, seed=1, spread=0)
    at = a.slots_d[0].item() // 16
    a.cache[2].view(torch.uint8)[at] = 255
    kept = a.cache[0].view(torch.uint8)[at, :5].clone()
    xs.xs_rope_append_paged8(None, a.k, a.v, None, a.slots_d, None, *a.cache, None)
    assert a.cache[2].view(torch.uint8)[at].item() == 255
    assert torch.equal(a.cache[0].view(torch.uint8)[at, :5], kept)
    assert a.cache[0][at, 5:8].float().isnan().all()
    a.check_exact(1, a.x64[:, a.H + a.Hkv:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@DTYPES
@pytest.mark.parametrize("case,rot", [(APPENDS[i], r) for i, r in ((1, 128), (2, 48), (3, 64), (4, 128), (6, 16), (7, 32), (9, 128))],
                         ids=lambda c: str(c) if isinstance(c, int) else "T%d" % sum(c[0]))
def test_scales_of_rotated_keys(xs, case, rot, dtype, layout):
    """Every block's and head's scale lies between those of magnitudes lowered and raised by the rotation's error: it is
    the definition's but where the largest magnitude lies within that error of 448 times a scale."""
    a = Append(*case, dtype=dtype, seed=7, pad=2)
    rope = xs.Rope(a.D, rot, layout=("half", "interleaved").index(layout), base=5e5)
    a.launch(xs, rope)
    x, mass = pg.rope_reference(a.x64[:, a.H:a.H + a.Hkv], a.pos, pg.frequencies(rot, base=5e5), layout == "interleaved")
    off = (np.pi * 2.0 ** -24 + 4 * 2.0 ** -23) * mass + 2.0 ** -25 * np.abs(x)
    ends = []
    for y in (np.maximum(np.abs(x) - off, 0), np.abs(x) + off):
        num, exp = a.num[0].copy(), a.exp[0].copy()
        p8.append_reference(num, exp, y, a.slots, a.block)
        ends.append(exp)
    got = a.cache[2].view(torch.uint8).cpu().numpy().astype(float) - 127
    bad = (got < ends[0]) | (got > ends[1])
    assert not bad.any(), np.argwhere(bad)[:5]
    assert (ends[0] == ends[1]).mean() > 0.9      # nearly all are pinned


# -------------------------------------------------------------------------- attention
@pytest.mark.parametrize("q", [1, 90])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("apart", [0, 1, 9], ids=lambda a: "apart%d" % a)
def test_values_under_the_largest_scale(xs, apart, D, q):
    """V's scales at the upper end of their range, 2^127, alone or beside smaller ones: outputs of up to 2^127, and the
    log-sum-exp as ever."""
    c = p8.Paged8Case([q, q], [300, 40], 4, 2, D, 32, block=16, seed=apart)
    r = np.random.default_rng(apart)
    c.vmax = 2.0 ** 127
    for i, kv in enumerate(c.kv_lens):
        blocks = pg.ceil_div(kv, 16)
        num = p8.nearest(np.clip(r.standard_normal((kv, 2, D)) * 0.25, -0.9375, 0.9375))
        exp = 127 - apart * r.integers(0, 2, size=(blocks, 2))
        c.values[i] = num * np.exp2(exp[np.arange(kv) // 16].astype(float))[..., None]
        code = p8.codes(num)
        for j in range(pg.ceil_div(kv, 32)):
            e = int(c.table[i, j])
            hi = min(kv - 32 * j, 32)
            c.v.view(torch.uint8)[e, :hi] = code[32 * j:32 * j + hi].cuda()
            n = pg.ceil_div(hi, 16)
            c.vs.view(torch.uint8)[e, :n] = torch.from_numpy((exp[2 * j:2 * j + n] + 127).astype(np.uint8)).cuda()
    out, lse = _run(xs, c)
    c.check(out, lse, True, 0, c.D ** -0.5)


@DTYPES
@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("q", [1, 3, 90])
def test_rows_that_are_nan(xs, q, bits, dtype):
    """Their outputs are NaN and so are their log-sum-exps, whole tiles and cut ones; the other rows keep their bits."""
    make, run = (p8.Paged8Case, _run) if bits == 8 else (pg.PagedCase, _run16)
    c = make([q, q, 1], [500, 70, 20000], 8, 2, 128, 32, seed=3, dtype=dtype)
    want, z = run(xs, c)
    hit = torch.zeros((2 * q + 1, 8), dtype=torch.bool, device="cuda")
    for t, h, d in [(0, 5, 17), (2 * q - 1, 0, 127), (2 * q, 7, 0)]:
        c.q[t, h, d] = float("nan")
        hit[t, h] = True
    out, lse = run(xs, c)
    assert out[hit].isnan().all() and lse[hit].isnan().all()
    assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse[~hit], z[~hit])


@DTYPES
@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
@pytest.mark.parametrize("q", [1, 90])
def test_rows_of_q_that_are_not_finite(xs, q, value, dtype):
    """Their outputs and log-sum-exps are NaN; the other rows keep their bits."""
    c = p8.Paged8Case([q, q], [500, 70], 8, 2, 128, 32, seed=3, dtype=dtype)
    want, z = _run(xs, c)
    rows = [(0, 5, 17), (2 * q - 1, 0, 127)]
    for t, h, d in rows:
        c.q[t, h, d] = value
    out, lse = _run(xs, c)
    hit = torch.zeros((2 * q, 8), dtype=torch.bool, device="cuda")
    for t, h, _ in rows:
        hit[t, h] = True
    assert out[hit].isnan().all() and lse[hit].isnan().all()
    assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse[~hit], z[~hit])


@DTYPES
@pytest.mark.parametrize("q", [1, 90])
def test_a_row_that_is_not_finite_and_sees_no_key(xs, q, dtype):
    c = p8.Paged8Case([q, 2], [0, 30], 4, 1, 64, 16, seed=3, dtype=dtype)
    c.q[:q] = float("inf")
    out, lse = _run(xs, c)
    assert not out[:q].any() and torch.isneginf(lse[:q]).all()
    assert out[q:].isfinite().all()


@DTYPES
@pytest.mark.parametrize("q,heads", [(1, 1), (2, 2), (70, 2)])
@pytest.mark.parametrize("down", [22, 24, 26, 28])
def test_small_probabilities_beside_large_ones(xs, q, heads, down, dtype):
    """A key of 32 has a probability 2^down times the others' and values of 0: the output is what the others add up to.
    A probability is off by half a step of fp16, 2^-11, or by 2^-32 of its row's largest where it is small."""
    kv = 640
    c = p8.Paged8Case([q], [kv], heads, 1, 64, 32, block=32, seed=1, dtype=dtype)
    few = np.arange(kv) % 32 == 5
    k, v = np.zeros((kv, 1, 64)), np.full((kv, 1, 64), 256.0)
    k[~few, 0, 0], v[few] = -down, 0.0                       # (four significant bits)
    for cache, scale, x, e in ((c.k, c.ks, k, 0), (c.v, c.vs, v, 6)):
        for j in range(kv // 32):
            at = int(c.table[0, j])
            cache.view(torch.uint8)[at] = p8.codes(x[32 * j:32 * j + 32]).cuda()
            scale.view(torch.uint8)[at] = 127 + e
    c.keys, c.values = [k], [v * 2.0 ** 6]
    c.q.zero_()
    c.q[:, :, 0] = 1.0
    c.q64 = c.q.double().cpu().numpy()
    scale = float(np.log(2.0))                               # a score is a power of two's exponent
    out, lse = _run(xs, c, scale=scale)
    ref, mass, z = c.reference(True, 0, scale)
    # every 32 keys have a large one, so that the small ones are 31 of at most 2^-down / (keys / 32) each
    floor = 2.0 ** -32 * 32 * 256 * 2.0 ** 6
    before = (2.0 ** -11 + 1.5e-4) * mass + floor
    got = out.double().cpu().numpy()
    u = pg.U[dtype]
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0     # half of fp16's least step
    assert (np.abs(got - ref) <= before + u * (np.abs(ref) + before) + tiny).all(), (got.ravel()[0], ref.ravel()[0])
    assert (np.abs(lse.double().cpu().numpy() - z) <= 6e-5 + 2.0 ** -22 * np.abs(z)).all()
