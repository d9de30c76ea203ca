"""xs_paged_step, xs_rope_fwd and xs_rope_append_paged on the GPU against their
definitions in 64 bits (whole numbers: equal; see _paged.py for the bounds)."""
import numpy as np
import pytest

import _paged as pg

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def xs():
    from conftest import build_library
    build_library()
    import dit_attention_ulysses_gb300 as xs
    assert torch.cuda.is_available()
    return xs


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


# ------------------------------------------------------------------------------- step
def _step_case(n, page, width, seed, max_new=1, spare=None, rows=None, ended=0.1, bad=0.0):
    r = np.random.default_rng(seed)
    cap = width * page
    cached = r.integers(0, cap - min(cap - 1, max_new), size=n, endpoint=True).astype(np.int32)
    cached[r.random(n) < 0.2] = 0
    new = r.integers(0, max_new, size=n, endpoint=True).astype(np.int32)
    new[r.random(n) < ended] = -1
    if bad:
        cached[r.random(n) < bad] = -3
        new[r.random(n) < bad] = cap + 1
        new[r.random(n) < bad] = 2 ** 31 - 1
        cached[r.random(n) < bad] = 2 ** 31 - 1
    held = np.minimum(-(-np.maximum(cached, 0).astype(np.int64) // page), width)
    need = int(held.sum())
    n_pages = need + (n + 3 if spare is None else spare) + 1
    order = r.permutation(n_pages).astype(np.int32)
    table = r.integers(-5, n_pages + 5, size=(n, width)).astype(np.int32)
    at = 0
    for i in range(n):
        table[i, :held[i]] = order[at:at + held[i]]
        at += held[i]
    free = r.integers(-9, -1, size=n_pages).astype(np.int32)
    count = min(n_pages - need, n_pages) if spare is None else spare
    free[:count] = order[need:need + count]
    total = int(np.clip(new, 0, cap).sum())
    return dict(cache_lens=cached, new_lens=new, table=table, free=free, count=count, page=page,
                rows=max(1, total + 3 if rows is None else rows))


def _run_step(xs, c):
    n, rows = len(c["cache_lens"]), c["rows"]
    t = dict(table=_dev(c["table"]), free=_dev(c["free"]), kv_lens=torch.full((n,), -7, dtype=torch.int32).cuda(),
             cu_q=torch.full((n + 1,), -7, dtype=torch.int32).cuda(),
             positions=torch.full((rows,), -7, dtype=torch.int32).cuda(),
             slots=torch.full((rows,), -7, dtype=torch.int64).cuda(),
             free_count=torch.full((1,), -7, dtype=torch.int32).cuda(),
             status=torch.full((n,), -7, dtype=torch.int32).cuda())
    ins = _dev(c["cache_lens"]), _dev(c["new_lens"]), torch.tensor([c["count"]], dtype=torch.int32, device="cuda")
    call = lambda: xs.xs_paged_step(ins[0], ins[1], t["table"], t["free"], ins[2], c["page"], t["kv_lens"],  # noqa: E731
                                    t["cu_q"], t["positions"], t["slots"], t["free_count"], t["status"])
    return t, call, ins


def _check_step(t, c, where=""):
    ref = pg.step_reference(c["cache_lens"], c["new_lens"], c["table"], c["free"], c["count"], c["page"], c["rows"])
    for k, v in t.items():
        np.testing.assert_array_equal(v.cpu().numpy().reshape(-1), np.asarray(ref[k]).reshape(-1), err_msg=f"{where} {k}")


STEPS = [  # n, page, width, max_new, spare, rows, bad
    (1, 16, 4, 1, None, None, 0.0),
    (1, 16, 1, 16, 1, None, 0.0),
    (1, 1024, 3, 3000, 3, None, 0.0),
    (7, 32, 9, 40, None, None, 0.2),
    (256, 16, 64, 1, None, None, 0.0),
    (300, 64, 6, 100, 40, None, 0.1),        # pages run out
    (300, 16, 30, 100, None, 2000, 0.1),     # rows run out
    (513, 16, 30, 50, 700, 9000, 0.1),       # both
    (100, 128, 4, 2, 0, None, 0.0),          # an empty free list: only the ended requests' pages
    (1025, 16, 8, 3, None, 1, 0.05),         # a single row
    (8192, 32, 5, 9, None, None, 0.02),      # the most requests
    (3, 16, 5000, 60000, None, None, 0.0),   # long prompts: many pages per request
]


@pytest.mark.parametrize("case", STEPS, ids=lambda c: "n%d_p%d_w%d_a%d" % c[:4])
def test_step_equals_definition(xs, case):
    n, page, width, max_new, spare, rows, bad = case
    for seed in range(3):
        c = _step_case(n, page, width, seed, max_new, spare, rows, bad=bad)
        t, call, ins = _run_step(xs, c)
        call()
        _check_step(t, c, f"seed {seed}")
        call()   # the same call again: the same result
        _check_step(t, c, f"seed {seed} again")
        for a, k in zip(ins[:2], ("cache_lens", "new_lens")):
            np.testing.assert_array_equal(a.cpu().numpy(), c[k])


def test_step_all_ended_or_idle(xs):
    for new in (-1, 0):
        c = _step_case(40, 16, 6, 5)
        c["new_lens"][:] = new
        t, call, _ = _run_step(xs, c)
        call()
        _check_step(t, c)


@pytest.mark.parametrize("count", [-4, 10 ** 9])
def test_step_free_count_out_of_range(xs, count):
    """A count outside the list is taken as its nearest end."""
    c = _step_case(20, 16, 4, 3)
    c["free"] = np.random.default_rng(0).permutation(len(c["free"])).astype(np.int32)
    c["count"] = count
    t, call, _ = _run_step(xs, c)
    call()
    _check_step(t, c)


# ------------------------------------------------------------------------------- rope
ROPES = [  # T, H, D, rot, interleaved, scaling arguments
    (1, 1, 64, 64, False, {}),
    (3, 5, 64, 16, True, {}),
    (33, 24, 128, 128, False, {}),
    (257, 3, 128, 48, False, dict(scaling="by_parts", factor=8.0, context=8192.0, base=5e5)),
    (100, 7, 128, 96, True, dict(scaling="by_parts", factor=4.0, context=1000.0, low=2.0, high=20.0)),
    (2000, 40, 128, 128, True, {}),
    (19, 2, 64, 32, False, dict(scaling="linear", factor=3.5)),
    (64, 33, 64, 64, True, dict(scaling="stretch", factor=16.0)),
    (5, 130, 128, 80, False, {}),
]
FAR = [0, 1, -1, 7, -12345, 1 << 20, (1 << 24) + 1, (1 << 31) - 1, -(1 << 31)]


def _rope(xs, D, rot, interleaved, kw, magnitude=1.0):
    kw = dict(kw)
    kw["scaling"] = {"plain": 0, "linear": 1, "stretch": 2, "by_parts": 3}[kw.get("scaling", "plain")]
    return xs.Rope(D, rot, layout=xs.XS_ROPE_INTERLEAVED if interleaved else xs.XS_ROPE_HALF, magnitude=magnitude, **kw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("grad", [False, True], ids=["fwd", "grad"])
@pytest.mark.parametrize("case", ROPES, ids=lambda c: "T%d_H%d_D%d_r%d_%s" % (*c[:4], "il" if c[4] else "half"))
def test_rope_against_definition(xs, case, grad, dtype):
    T, H, D, rot, il, kw = case
    r = np.random.default_rng(T + rot)
    x = torch.from_numpy(r.standard_normal((T, H, D))).to(dtype)
    pos = r.integers(0, 1 << 20, size=T).astype(np.int32)
    pos[:min(T, len(FAR))] = FAR[:min(T, len(FAR))]
    magnitude = 1.3 if kw.get("scaling") == "by_parts" else 1.0
    rope = _rope(xs, D, rot, il, kw, magnitude)
    out = torch.full((T, H, D), float("nan"), dtype=dtype, device="cuda")
    dx = x.cuda()
    xs.xs_rope_fwd(dx, _dev(pos), out, rope, grad=grad)
    ref, mass = pg.rope_reference(x.double().numpy(), pos, pg.frequencies(rot, **kw), il, magnitude, -1 if grad else 1)
    err = np.abs(out.double().cpu().numpy() - ref)
    tol = pg.rope_tolerance(ref, mass, dtype)
    assert (err <= tol).all(), (err / tol).max()
    assert torch.equal(out[..., rot:], dx[..., rot:])          # channels that do not rotate: the same bits
    assert torch.equal(dx.cpu(), x)
    xs.xs_rope_fwd(dx, _dev(pos), dx, rope, grad=grad)          # in place
    assert torch.equal(dx, out)


def test_rope_rows_of_a_wider_matrix(xs):
    """Input and output as column ranges of fused projections; everything beside them stays."""
    T, H, D = 50, 4, 64
    g = torch.Generator(device="cuda").manual_seed(0)
    wide = torch.randn((T, 3 * H, D), generator=g, device="cuda").bfloat16()
    before = wide.clone()
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    rope = xs.Rope(D)
    dense = torch.empty((T, H, D), dtype=torch.bfloat16, device="cuda")
    xs.xs_rope_fwd(wide[:, H:2 * H], pos, dense, rope)
    xs.xs_rope_fwd(wide[:, H:2 * H], pos, wide[:, :H], rope)     # into other columns of the same matrix
    assert torch.equal(wide[:, :H], dense) and torch.equal(wide[:, H:], before[:, H:])
    xs.xs_rope_fwd(wide[:, H:2 * H], pos, wide[:, H:2 * H], rope)
    assert torch.equal(wide[:, H:2 * H], dense) and torch.equal(wide[:, 2 * H:], before[:, 2 * H:])


def test_rope_passes_infinities_of_channels_that_do_not_rotate(xs):
    x = torch.ones((2, 1, 64), dtype=torch.bfloat16, device="cuda")
    x[0, 0, 40], x[1, 0, 63] = float("inf"), float("nan")
    out = torch.empty_like(x)
    xs.xs_rope_fwd(x, torch.tensor([5, 9], dtype=torch.int32, device="cuda"), out, xs.Rope(64, 32))
    assert torch.equal(out[..., 32:].view(torch.int16), x[..., 32:].view(torch.int16))
    assert torch.isfinite(out[..., :32]).all()


@pytest.mark.parametrize("il", [False, True])
def test_rope_gradient_against_differences(xs, il):
    """L(x) = <g, R x> is linear: (L(x + e_i) - L(x - e_i)) / 2 at x = 0 is its i-th derivative.
    Each side carries one rounding of the type per element."""
    D, rot = 64, 48
    rope = _rope(xs, D, rot, il, {}, 0.75)
    r = np.random.default_rng(3)
    pos = torch.full((D,), 977, dtype=torch.int32, device="cuda")
    g = torch.from_numpy(r.standard_normal((1, 1, D))).bfloat16().cuda()
    basis = torch.eye(D, dtype=torch.bfloat16, device="cuda")[:, None, :].contiguous()
    plus, minus, dx = torch.empty_like(basis), torch.empty_like(basis), torch.empty_like(g)
    xs.xs_rope_fwd(basis, pos, plus, rope)
    xs.xs_rope_fwd(-basis, pos, minus, rope)
    xs.xs_rope_fwd(g, pos[:1].contiguous(), dx, rope, grad=True)
    diff = ((plus.double() - minus.double())[:, 0] / 2) @ g.double()[0, 0]
    u = pg.U[torch.bfloat16]
    mass = (plus.double().abs()[:, 0]) @ g.double()[0, 0].abs()
    assert ((diff - dx.double()[0, 0]).abs() <= 1.01 * u * (mass + diff.abs()) + 1e-6).all()


def test_rope_largest_rows(xs):
    """More than 2^31 elements: offsets pass 32 bits."""
    T, H, D = 131200, 128, 128
    assert T * H * D > 2 ** 31
    x = torch.zeros((T, H, D), dtype=torch.bfloat16, device="cuda")
    x[-3:] = 1.0
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    pos[-3:] = torch.tensor([0, 3, 11])
    xs.xs_rope_fwd(x, pos, x, xs.Rope(D))
    assert not x[:-3].any()
    ref, mass = pg.rope_reference(np.ones((3, H, D)), np.array([0, 3, 11]), pg.frequencies(D), False)
    assert (np.abs(x[-3:].double().cpu().numpy() - ref) <= pg.rope_tolerance(ref, mass, torch.bfloat16)).all()


# ----------------------------------------------------------------------------- append
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("T,H,Hkv,D,rot,page,il,form", [
    (1, 1, 1, 64, 64, 16, False, "tokens"), (37, 8, 2, 128, 128, 16, False, "heads"),
    (300, 6, 3, 64, 32, 64, True, "buffer"), (1000, 7, 7, 128, 48, 128, False, "tokens"),
    (65, 24, 1, 128, 128, 1024, True, "heads")])
def test_append(xs, T, H, Hkv, D, rot, page, il, form, dtype):
    r = np.random.default_rng(T)
    n_pages = T // page + 4
    qkv = torch.from_numpy(r.standard_normal((T, H + 2 * Hkv, D))).to(dtype).cuda()
    q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    shape = (n_pages, page, Hkv, D)
    if form == "buffer":
        both = torch.full((n_pages, 2, page, Hkv, D), 7.0, dtype=dtype, device="cuda")
        kc, vc = both[:, 0], both[:, 1]
    elif form == "heads":
        kc, vc = (torch.full((n_pages, Hkv, page, D), 7.0, dtype=dtype, device="cuda").transpose(1, 2) for _ in "kv")
    else:
        kc, vc = (torch.full(shape, 7.0, dtype=dtype, device="cuda") for _ in "kv")
    pos = torch.from_numpy(r.integers(0, 1 << 17, size=T).astype(np.int32)).cuda()
    slots = r.permutation(n_pages * page)[:T].astype(np.int64)
    if T > 5:
        slots[-1], slots[3], slots[4], slots[2] = -1, n_pages * page, 2 ** 62, -2 ** 63
    good = (slots >= 0) & (slots < n_pages * page)
    rope = _rope(xs, D, rot, il, {})
    want_q, want_k = torch.empty((T, H, D), dtype=dtype, device="cuda"), torch.empty((T, Hkv, D), dtype=dtype, device="cuda")
    xs.xs_rope_fwd(q, pos, want_q, rope)
    xs.xs_rope_fwd(k, pos, want_k, rope)
    want_v = v.clone()
    ek, ev = torch.full(shape, 7.0, dtype=dtype, device="cuda"), torch.full(shape, 7.0, dtype=dtype, device="cuda")
    rows = torch.from_numpy(np.nonzero(good)[0]).cuda()
    at = torch.from_numpy(slots[good]).cuda()
    ek[at // page, at % page], ev[at // page, at % page] = want_k[rows], want_v[rows]
    q_out = torch.full((T, H, D), float("nan"), dtype=dtype, device="cuda")
    before = qkv.clone()
    xs.xs_rope_append_paged(q, k, v, pos, _dev(slots), q_out, kc, vc, rope)
    assert torch.equal(q_out, want_q) and torch.equal(kc, ek) and torch.equal(vc, ev) and torch.equal(qkv, before)
    xs.xs_rope_append_paged(q, k, v, pos, _dev(slots), q, kc, vc, rope)     # q in place, beside k and v
    assert torch.equal(q, want_q) and torch.equal(kc, ek) and torch.equal(qkv[:, H:], before[:, H:])
