"""xs_attn_paged_fwd on the GPU against plain attention in 64 bits (_paged.py has the
bounds), and whole serving steps: step, plan, append and attention together."""
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


def _run(xs, c, causal=True, window=0, scale=None, max_q=None, ws=None, lse=True, layout=None, P=1, fill=float("nan")):
    scale = c.D ** -0.5 if scale is None else scale
    max_q = max(max(c.q_lens), 1) if max_q is None else max_q
    ws = ws or xs.PagedWorkspace(c.n, c.H, c.Hkv, c.D)
    layout = xs.XS_LAYOUT_CONTIGUOUS if layout is None else layout
    shape = {xs.XS_LAYOUT_A2A: (c.T // P, c.H, c.D), xs.XS_LAYOUT_HEADS: (c.T, c.H // P, c.D)}.get(layout, (c.T, c.H, c.D))
    outs = [torch.full(shape, fill, dtype=c.dtype, device="cuda") for _ in range(P)]
    z = torch.full((c.T, c.H), fill, dtype=torch.float32, device="cuda") if lse else None
    xs.xs_attn_paged_plan(c.cu, c.kv, max_q, ws, causal=causal, window=window)
    xs.xs_attn_paged_fwd(c.q, c.k, c.v, c.table, layout, outs, scale, ws, lse=z)
    assert xs.xs_attn_get_device_error_info() [0] == xs.XS_OK
    return (outs if P > 1 else outs[0]), z


# q_lens, kv_lens, H, Hkv, D, page
DECODE = [
    ([1], [1], 1, 1, 64, 16),
    ([1], [33], 2, 1, 128, 16),
    ([1], [5000], 8, 2, 128, 16),
    ([1, 1, 1], [31, 32, 33], 4, 4, 64, 32),
    ([1, 0, 1, 0, 1], [700, 50, 1, 0, 257], 12, 4, 128, 64),
    ([1] * 40, [1 + 97 * i for i in range(40)], 8, 1, 128, 16),
    ([2, 1, 4, 3], [900, 3, 4, 130], 8, 2, 64, 128),
    ([1, 1], [3000, 2100], 28, 4, 128, 256),      # 7 heads to a KV head
    ([1, 5], [70, 900], 5, 1, 128, 1024),
    ([1], [700], 32, 1, 128, 32),                 # 32 heads to a KV head
    ([1, 2], [500, 3000], 40, 1, 128, 16),        # 40, and 128: a tile of its own size
    ([1, 1, 0, 3], [900, 128, 5, 40000], 128, 1, 64, 64),
    ([33], [1300], 48, 2, 128, 128),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("case", DECODE, ids=lambda c: "n%d_kv%d_H%d_%d_D%d_p%d" % (len(c[0]), max(c[1]), *c[2:]))
def test_few_tokens(xs, case, dtype):
    c = pg.PagedCase(*case, dtype=dtype, seed=len(case[0]), extra_rows=2)
    out, lse = _run(xs, c)
    c.check(out, lse, True, 0, c.D ** -0.5)
    rows = sum(c.q_lens)
    assert out[rows:].isnan().all() and lse[rows:].isnan().all()     # rows behind the last sequence
    out2, _ = _run(xs, c, lse=False)
    assert torch.equal(out2[:rows], out[:rows])


CHUNKS = [  # q_lens, kv_lens, H, Hkv, D, page, causal, window
    ([130], [130], 2, 2, 128, 16, True, 0),
    ([128], [256], 2, 1, 64, 64, False, 0),
    ([257, 1, 64], [1000, 700, 64], 8, 2, 128, 16, True, 0),
    ([100, 3, 0, 31], [100, 900, 77, 2000], 6, 2, 64, 32, True, 100),
    ([300], [1111], 3, 1, 128, 128, True, 1),
    ([200, 129], [200, 1500], 5, 5, 128, 256, True, 200),
    ([65, 200], [500, 201], 4, 4, 128, 32, False, 0),
    ([90], [2500], 24, 8, 64, 1024, False, 0),
    ([10, 6], [4, 0], 4, 2, 128, 16, True, 0),      # more new tokens than keys: rows that see nothing
    ([10, 6], [4, 0], 4, 2, 64, 16, False, 0),
    ([40, 200], [30, 150], 2, 1, 128, 16, True, 7),
    ([17] * 33, [17 + 13 * i for i in range(33)], 4, 1, 128, 16, True, 0),
    ([515], [2061], 8, 1, 128, 64, True, 0),
    ([77, 400], [1500, 400], 7, 1, 128, 32, True, 0),     # 18 tokens of 7 heads: 126 of 128 rows
    ([301], [700], 24, 1, 64, 16, True, 333),
    ([2000], [2000], 2, 1, 64, 16, True, 0),
    ([129] * 9, [129 * (i + 1) for i in range(9)], 12, 3, 128, 64, False, 0),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("case", CHUNKS, ids=lambda c: "q%d_kv%d_H%d_%d_D%d_p%d_%s_w%d" % (
    max(c[0]), max(c[1]), *c[2:6], "causal" if c[6] else "full", c[7]))
def test_chunks(xs, case, dtype):
    *shape, causal, window = case
    c = pg.PagedCase(*shape, dtype=dtype, seed=sum(case[0]), extra_rows=1, window=window, freed=window > 0)
    out, lse = _run(xs, c, causal, window)
    c.check(out, lse, causal, window, c.D ** -0.5)
    rows = sum(c.q_lens)
    assert out[rows:].isnan().all() and lse[rows:].isnan().all()


@pytest.mark.parametrize("n", [38, 39, 76, 77, 130, 257, 1024, 1025])
def test_many_ragged_tiles(xs, n):
    """Four tiles per sequence: one to 27 tiles per CTA, some CTAs with one fewer, and both sides of the
    number up to which the plan sorts them."""
    r = np.random.default_rng(n)
    q_lens = r.integers(1, 41, size=n).tolist()
    c = pg.PagedCase(q_lens, [q + int(r.integers(0, 400)) for q in q_lens], 8, 4, 64, 16, seed=n, extra_rows=1)
    ws = xs.PagedWorkspace(n, 8, 4, 64)
    out, lse = _run(xs, c, ws=ws, max_q=64)
    c.check(out, lse, True, 0, c.D ** -0.5)
    rows = sum(q_lens)
    out2, lse2 = _run(xs, c, ws=ws, max_q=64)      # a plan of the same lengths is the same plan
    assert torch.equal(out2[:rows], out[:rows]) and torch.equal(lse2[:rows], lse[:rows])


@pytest.mark.parametrize("max_q", [1, 3, 8, 5000])
def test_max_q_is_only_an_estimate(xs, max_q):
    c = pg.PagedCase([5, 150, 1], [400, 300, 90], 4, 2, 128, 16, seed=9)
    out, lse = _run(xs, c, max_q=max_q)
    c.check(out, lse, True, 0, c.D ** -0.5)


@pytest.mark.parametrize("form", [dict(heads_first=True), dict(one_buffer=True), dict(q_pad=5), dict(table_pad=3),
                                  dict(heads_first=True, q_pad=2, table_pad=1)], ids=str)
@pytest.mark.parametrize("q", [1, 70])
def test_strides(xs, form, q):
    c = pg.PagedCase([q, 2], [333, 200], 6, 2, 128, 32, seed=4, **form)
    out, lse = _run(xs, c)
    c.check(out, lse, True, 0, c.D ** -0.5)


@pytest.mark.parametrize("q", [[1, 1, 2], [60, 4, 100]], ids=["few", "chunk"])
def test_layouts_hold_the_same_bits(xs, q):
    P = 4
    c = pg.PagedCase(q, [300, 17, 900], 8, 4, 64, 16, seed=1, extra_rows=-sum(q) % P)
    full, _ = _run(xs, c, fill=3.0)
    shards, _ = _run(xs, c, layout=xs.XS_LAYOUT_A2A, P=P, fill=3.0)
    heads, _ = _run(xs, c, layout=xs.XS_LAYOUT_HEADS, P=P, fill=3.0)
    assert torch.equal(torch.cat(shards), full) and torch.equal(torch.cat(heads, 1), full)


@pytest.mark.parametrize("scale", [0.0, 0.01, 3.0])
@pytest.mark.parametrize("q", [1, 90])
def test_scales(xs, scale, q):
    """0: the mean of the values.  3: one key takes nearly all, and maxima move often."""
    c = pg.PagedCase([q], [500], 2, 1, 64, 16, seed=2, gain=0.2 if scale > 1 else 1.0)
    out, lse = _run(xs, c, scale=scale)
    c.check(out, lse, True, 0, scale)


@pytest.mark.parametrize("q", [1, 40])
def test_rising_scores_move_the_maximum(xs, q):
    """Keys whose scores grow along the sequence: every block has a new maximum."""
    c = pg.PagedCase([q], [2000], 2, 2, 128, 16, seed=6)
    up = np.linspace(0, 1, 2000)[:, None, None] * np.ones((1, 2, 128)) * 0.6
    x = torch.from_numpy(up).to(c.dtype)
    c.keys[0] = x.double().numpy()
    for j in range(pg.ceil_div(2000, 16)):
        c.k[c.table[0, j].long()] = x[16 * j:16 * j + 16].cuda()
    c.q.copy_(torch.ones_like(c.q) * 4)
    c.q64 = c.q.double().cpu().numpy()
    out, lse = _run(xs, c, scale=0.2)
    # scores up to 61: sum |q_d k_d| scale = 61, so 128 * 2^-24 * 61 = 4.7e-4 bounds their error
    ref, mass, z = c.reference(True, 0, 0.2)
    tol = pg.U[c.dtype] * (mass + np.abs(ref)) * 1.01 + 1.2e-3 * mass
    assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()
    assert (np.abs(lse.double().cpu().numpy() - z) <= 5e-4 + 2.0 ** -22 * np.abs(z)).all()


@pytest.mark.parametrize("q,power", [(1, 55), (200, 12)], ids=["few", "chunk"])
def test_scores_far_from_zero(xs, q, power):
    """All scores alike far below zero (a row that sees keys, however low), and one key far above the
    others: no overflow on the way, the mean and that key's values.  A chunk's exponents subtract the
    rounded maximum from the exact product, so its scores stay below 1e9; a few tokens' may be any."""
    c = pg.PagedCase([q], [700], 2, 2, 64, 16, seed=6)
    big = 2.0 ** power
    score = 64 * big * big / 8
    c.q.fill_(big)
    c.k.fill_(-big)
    out, lse = _run(xs, c, causal=False)
    v = np.mean(c.values[0], axis=0)
    a = np.mean(np.abs(c.values[0]), axis=0)
    assert (np.abs(out.double().cpu().numpy() - v) <= 2.0 ** -8 * (a + np.abs(v)) * 1.01 + 2e-4 * a).all()
    # log2(e), ln 2 and their products in fp32: four steps; the logarithm of 700 is below one
    assert ((lse.double() / -score - 1).abs() <= 2.0 ** -21).all()
    c.k[c.table[0, 30].long(), 5] = big
    out, lse = _run(xs, c, causal=False)
    one = torch.from_numpy(c.values[0][30 * 16 + 5]).cuda()
    # a chunk's only probability is a power of two near 1, rounded to the type: half a step, and the output's
    assert ((out.double() - one).abs() <= (2.0 ** -8 * 2.02 if q > 1 else 0.0) * one.abs()).all()
    assert ((lse.double() / score - 1).abs() <= 2.0 ** -21).all()


def test_nan_rows_of_q_behind_the_last_sequence(xs):
    """Padding rows may hold anything."""
    for q in ([1, 1], [70, 30]):
        c = pg.PagedCase(q, [300, 200], 6, 2, 128, 16, seed=6, extra_rows=40)
        c.q[sum(q):] = float("nan")
        out, lse = _run(xs, c)
        c.check(out, lse, True, 0, c.D ** -0.5)


@pytest.mark.parametrize("q", [1, 300])
def test_workspace_of_more_sequences_and_used_again(xs, q):
    """A workspace serves one step after the other, of other lengths, causal or not, few or many."""
    ws = xs.PagedWorkspace(3, 4, 2, 128)
    for kv, causal, window in (((500, 0, 90), True, 0), ((1, 3000, 700), False, 0), ((800, 900, 1000), True, 64)):
        c = pg.PagedCase([q, 1, 0], [max(kv[0], q), kv[1], kv[2]], 4, 2, 128, 32, seed=q)
        out, lse = _run(xs, c, causal, window, ws=ws)
        c.check(out, lse, causal, window, c.D ** -0.5)


def test_lengths_that_are_not_the_caches(xs):
    """Nonsense on the device reads and writes nothing out of range; the next step is right."""
    c = pg.PagedCase([2, 3], [60, 70], 4, 2, 64, 16, seed=1)
    ws = xs.PagedWorkspace(2, 4, 2, 64)
    guard = torch.full((c.T + 64, 4, 64), 5.0, dtype=c.dtype, device="cuda")
    for cu, kv in (([5, 1, 3], [60, 70]), ([-7, 3, 9], [-1, 5000]), ([0, 2, 4000], [60, 20]), ([100, 101, 102], [10, 10]),
                   ([0, 0, 0], [2 ** 20, 2 ** 20]), ([2, 5, 5], [0, 0])):
        for max_q in (1, 100):
            xs.xs_attn_paged_plan(torch.tensor(cu, dtype=torch.int32, device="cuda"),
                                  torch.tensor(kv, dtype=torch.int32, device="cuda"), max_q, ws)
            xs.xs_attn_paged_fwd(c.q, c.k, c.v, c.table, xs.XS_LAYOUT_CONTIGUOUS, [guard[32:32 + c.T]], 0.1, ws)
            xs.xs_attn_get_device_error()
            assert (guard[:32] == 5.0).all() and (guard[32 + c.T:] == 5.0).all()
    out, lse = _run(xs, c, ws=ws)
    c.check(out, lse, True, 0, c.D ** -0.5)


def test_long_split_is_repeatable(xs):
    """One sequence cut over many SMs; ten calls on one plan give the same bits, and a plan made
    anew does too."""
    c = pg.PagedCase([1], [40000], 8, 2, 128, 64, seed=8)
    ws = xs.PagedWorkspace(c.n, c.H, c.Hkv, c.D)
    out, lse = _run(xs, c, ws=ws)
    c.check(out, lse, True, 0, c.D ** -0.5)
    for _ in range(10):
        o, z = torch.full_like(out, float("nan")), torch.full_like(lse, float("nan"))
        xs.xs_attn_paged_fwd(c.q, c.k, c.v, c.table, xs.XS_LAYOUT_CONTIGUOUS, [o], c.D ** -0.5, ws, lse=z)
        assert torch.equal(o, out) and torch.equal(z, lse)
    o, z = _run(xs, c, ws=ws)
    assert torch.equal(o, out) and torch.equal(z, lse)


def test_offsets_past_32_bits(xs):
    """A cache of more than 2^31 elements, the sequence's pages at its end."""
    H, Hkv, D, page = 2, 2, 128, 256
    n_pages = 2 ** 31 // (page * Hkv * D) + 40
    kc, vc = (torch.empty((n_pages, page, Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    for q_len, kv_len in ((1, 1000), (200, 1000)):
        c = pg.PagedCase([q_len], [kv_len], H, Hkv, D, page, seed=q_len)
        used = c.table[0, :4].long()
        far = n_pages - 4 + torch.tensor([2, 0, 3, 1], device="cuda")
        kc[far], vc[far] = c.k[used], c.v[used]
        c.table[0, :4] = far.int()
        c.k, c.v = kc, vc
        out, lse = _run(xs, c)
        c.check(out, lse, True, 0, D ** -0.5)


@pytest.mark.parametrize("most", [1, 40], ids=["one", "up_to_40"])
def test_most_sequences(xs, most):
    """8192 sequences, the limit, some without new tokens."""
    r = np.random.default_rng(most)
    q = r.integers(0, most, size=8192, endpoint=True)
    kv = q + r.integers(0, 30, size=8192)
    c = pg.PagedCase(q.tolist(), kv.tolist(), 2, 1, 64, 16, seed=most)
    out, lse = _run(xs, c)
    c.check(out, lse, True, 0, c.D ** -0.5)


@pytest.mark.parametrize("q", [1, 70])
def test_a_million_keys(xs, q):
    """2^20 keys of one head: Q = 0 weighs every key alike, so a row is the mean of what it sees."""
    D, page, keys = 64, 512, 1 << 20
    kc, vc = (torch.randn((keys // page, page, 1, D), device="cuda").bfloat16() for _ in "kv")
    table = torch.randperm(keys // page, device="cuda").int()[None]
    cu, kv = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, q], [keys]))
    query = torch.zeros((q, 1, D), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty_like(query), torch.empty((q, 1), dtype=torch.float32, device="cuda")
    ws = xs.PagedWorkspace(1, 1, 1, D)
    xs.xs_attn_paged_plan(cu, kv, q, ws)
    xs.xs_attn_paged_fwd(query, kc, vc, table, xs.XS_LAYOUT_CONTIGUOUS, [out], 0.1, ws, lse=lse)
    assert xs.xs_attn_get_device_error() == xs.XS_OK
    v = vc[table[0].long()].double().view(keys, D)
    seen = torch.arange(keys - q + 1, keys + 1, device="cuda").double()
    ref = torch.cumsum(v, 0)[keys - q:] / seen[:, None]
    # probabilities are exactly 1: a sum of 2^20 terms in fp32 over 2^20, in hundreds of separate runs of
    # at most a few thousand blocks' partial sums (each step 2^-24 of a partial sum below 5000)
    assert ((out[:, 0].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1e-5).all()
    assert ((lse[:, 0].double() - seen.log()).abs() <= 6e-5).all()


def test_pages_out_of_range_read_as_zeros(xs):
    """Bad page numbers and a table too narrow for the sequence read as zeros: no fault."""
    H, D, page = 2, 64, 16
    for q_len in (1, 50):
        c = pg.PagedCase([q_len], [200], H, H, D, page, seed=3)
        bad = {2: -1, 5: c.k.shape[0], 7: 2 ** 31 - 1, 9: -2 ** 31}
        for j, e in bad.items():
            c.table[0, j] = e
            c.keys[0][j * page:(j + 1) * page] = 0
            c.values[0][j * page:(j + 1) * page] = 0
        c.table = c.table[:, :11].contiguous()     # 176 of 200 keys
        c.keys[0][176:], c.values[0][176:] = 0, 0
        out, lse = _run(xs, c)
        c.check(out, lse, True, 0, D ** -0.5)


def test_plan_of_other_arguments_is_reported(xs):
    c = pg.PagedCase([1, 1], [100, 50], 4, 2, 64, 16, seed=3)
    ws = xs.PagedWorkspace(c.n, c.H, c.Hkv, c.D)
    xs.xs_attn_paged_plan(c.cu, c.kv, 1, ws)
    out = torch.full((c.T, c.H, c.D), 5.0, dtype=c.dtype, device="cuda")
    for planned in ((1, 0, 0), (1, 1, 9), (8, 1, 0), (1000, 1, 0)):     # causal, window, max_q
        ws.planned = planned
        xs.xs_attn_paged_fwd(c.q, c.k, c.v, c.table, xs.XS_LAYOUT_CONTIGUOUS, [out], 0.1, ws)
        if planned == (8, 1, 0):
            assert xs.xs_attn_get_device_error() == xs.XS_OK            # 8 tokens of 2 heads: the same tiles
            assert not (out == 5.0).all()
            out.fill_(5.0)
            continue
        code, rec = xs.xs_attn_get_device_error_info()
        assert code == xs.XS_ERR_DEVICE_BOUNDS and rec["site"] == 3
        assert (out == 5.0).all()
    xs.xs_attn_paged_plan(c.cu, c.kv, 1, ws)
    xs.xs_attn_paged_fwd(c.q, c.k, c.v, c.table, xs.XS_LAYOUT_CONTIGUOUS, [out], 0.1, ws)
    c.check(out, None, True, 0, 0.1)


@pytest.mark.parametrize("q", [1, 300])
def test_expired_wait_is_reported(xs, monkeypatch, q):
    """With a limit of 0 the first copy that has not landed when it is looked for ends the launch.  A
    cache of 1.6 GB, far more than L2, so that some has not; afterwards the context still works."""
    H, D, page, keys = 8, 128, 64, 400000
    n_pages = keys // page
    kc, vc = (torch.zeros((n_pages, page, H, D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    table = torch.arange(n_pages, dtype=torch.int32, device="cuda")[None]
    cu, kv = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, q], [keys]))
    query, out = (torch.zeros((q, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = xs.PagedWorkspace(1, H, H, D)
    xs.xs_attn_paged_plan(cu, kv, q, ws)
    monkeypatch.setenv("XSATTN_WAIT_TIMEOUT_NS", "0")
    xs.xs_attn_paged_fwd(query, kc, vc, table, xs.XS_LAYOUT_CONTIGUOUS, [out], 0.1, ws)
    code, rec = xs.xs_attn_get_device_error_info()
    assert code == xs.XS_ERR_DEVICE_TIMEOUT and rec["kind"] == 1
    monkeypatch.delenv("XSATTN_WAIT_TIMEOUT_NS")
    c = pg.PagedCase([q], [3000], 4, 2, 128, 16, seed=3)
    out, lse = _run(xs, c)
    c.check(out, lse, True, 0, c.D ** -0.5)


def test_no_sequence_has_new_tokens(xs):
    c = pg.PagedCase([0, 0], [100, 0], 4, 2, 64, 16, seed=3)
    out, lse = _run(xs, c)
    assert out.isnan().all() and lse.isnan().all()


def test_prompt_equals_dense_causal_attention(xs):
    """A prompt without a prefix, through the pages, against the library's causal attention of the
    same tensors: the same sums in another order (two bounds of the type)."""
    S, H, D = 1000, 4, 128
    c = pg.PagedCase([S], [S], H, H, D, 64, seed=5)
    out, _ = _run(xs, c)
    k, v = (torch.from_numpy(x[0]).to(c.dtype).cuda()[None].contiguous() for x in (c.keys, c.values))
    dense = torch.empty((1, S, H, D), dtype=c.dtype, device="cuda")
    xs.xs_attn_causal_fwd(c.q[None].contiguous(), k, v, xs.XS_LAYOUT_CONTIGUOUS, [dense], D ** -0.5)
    _, mass, _ = c.reference(True, 0, D ** -0.5)
    u = pg.U[c.dtype]
    d = (out.double() - dense[0].double()).abs().cpu().numpy()
    assert (d <= 2.02 * u * (mass + np.abs(dense[0].double().cpu().numpy())) + 3e-4 * mass).all()


# ---------------------------------------------------------------------- serving, whole
class _Server:
    """The buffers of a small server, and the same state in 64 bits on the host."""

    def __init__(self, xs, n, H, Hkv, D, page, n_pages, rows, seed, causal=True, dtype=torch.bfloat16):
        self.xs, self.n, self.H, self.Hkv, self.D, self.page, self.rows = xs, n, H, Hkv, D, page, rows
        self.dtype, self.causal, self.max_q = dtype, causal, rows
        self.r = np.random.default_rng(seed)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.width = n_pages
        self.table = torch.full((n, self.width), -9, **i32)
        self.free = torch.randperm(n_pages).to(**i32)
        self.count, self.count_out = torch.tensor([n_pages], **i32), torch.empty(1, **i32)
        self.lens, self.new, self.kv = torch.zeros(n, **i32), torch.zeros(n, **i32), torch.zeros(n, **i32)
        self.cu, self.status = torch.zeros(n + 1, **i32), torch.zeros(n, **i32)
        self.positions, self.slots = torch.zeros(rows, **i32), torch.zeros(rows, dtype=torch.int64, device="cuda")
        t = dict(dtype=dtype, device="cuda")
        self.kc, self.vc = (torch.full((n_pages, page, Hkv, D), float("nan"), **t) for _ in "kv")
        self.qkv = torch.zeros((rows, H + 2 * Hkv, D), **t)
        self.q_rot, self.out = torch.zeros((rows, H, D), **t), torch.zeros((rows, H, D), **t)
        self.lse = torch.zeros((rows, H), dtype=torch.float32, device="cuda")
        self.rope = xs.Rope(D)
        self.ws = xs.PagedWorkspace(n, H, Hkv, D)
        self.past = [np.zeros((0, H + 2 * Hkv, D)) for _ in range(n)]

    def launch(self):
        xs, H, Hkv = self.xs, self.H, self.Hkv
        xs.xs_paged_step(self.lens, self.new, self.table, self.free, self.count, self.page, self.kv, self.cu,
                         self.positions, self.slots, self.count_out, self.status)
        xs.xs_attn_paged_plan(self.cu, self.kv, self.max_q, self.ws, causal=self.causal)
        q, k, v = self.qkv[:, :H], self.qkv[:, H:H + Hkv], self.qkv[:, H + Hkv:]
        xs.xs_rope_append_paged(q, k, v, self.positions, self.slots, self.q_rot, self.kc, self.vc, self.rope)
        xs.xs_attn_paged_fwd(self.q_rot, self.kc, self.vc, self.table, xs.XS_LAYOUT_CONTIGUOUS, [self.out],
                             self.D ** -0.5, self.ws, lse=self.lse)
        self.lens.copy_(self.kv)
        self.count.copy_(self.count_out)

    def step(self, new, launch):
        """One step with `new` tokens per request (-1: ended) through `launch`, checked in 64 bits."""
        rows = sum(max(a, 0) for a in new)
        x = torch.from_numpy(self.r.standard_normal((rows, self.H + 2 * self.Hkv, self.D))).to(self.dtype)
        self.qkv[:rows] = x.cuda()
        self.new.copy_(torch.tensor(new, dtype=torch.int32))
        self.out.fill_(9.0)
        launch()
        assert self.xs.xs_attn_get_device_error() == self.xs.XS_OK
        assert not self.status.any()
        row, theta = 0, pg.frequencies(self.D)
        for i, a in enumerate(new):
            if a < 0:
                self.past[i] = self.past[i][:0]
                continue
            self.past[i] = np.concatenate([self.past[i], x[row:row + a].double().numpy()])
            y, c = self.past[i], len(self.past[i])
            qk, _ = pg.rope_reference(y[:, :self.H + self.Hkv], np.arange(c), theta, False)
            # the operator rounds what it rotates
            qk = torch.from_numpy(qk).to(self.dtype).double().numpy()
            for h in range(self.H if a else 0):
                g = h // (self.H // self.Hkv)
                ref, mass, z = pg.attention_reference(qk[c - a:, h], qk[:, self.H + g], y[:, self.H + self.Hkv + g], c,
                                                      self.causal, 0, self.D ** -0.5)
                got = self.out[row:row + a, h].double().cpu().numpy()
                # beside attention's own bound: a rotated q or k may round to the other neighbour (a whole step,
                # 2u) where the angle's fp32 error decides; a score then moves by up to 2u |q_d k_d| scale for
                # that pair, below 2u * 4 * 4 / 8 = 4u
                u = pg.U[self.dtype]
                assert (np.abs(got - ref) <= u * (mass + np.abs(ref)) * 1.01 + (1.5e-4 + 4 * u) * mass).all()
            row += a
        assert (self.out[row:] == 9.0).all()
        held = [pg.ceil_div(len(p), self.page) for p in self.past]
        used = [int(e) for i, h in enumerate(held) for e in self.table[i, :h].cpu()]
        left = [int(e) for e in self.free[:int(self.count)].cpu()]
        assert sorted(used + left) == list(range(self.kc.shape[0]))      # every page has one owner


STEPS = [[40, 0, 7, 1], [1, 33, 1, 1], [1, 1, 1, 1], [-1, 1, 16, 1], [25, -1, 1, 1], [1, 1, 0, -1], [2, 5, 1, 50]]


@pytest.mark.parametrize("D,page,causal", [(128, 16, True), (64, 32, True), (128, 64, False)])
def test_serving_steps(xs, D, page, causal):
    s = _Server(xs, 4, 4, 2, D, page, 40, 100, seed=D + page, causal=causal)
    for new in STEPS:
        s.step(new, s.launch)


@pytest.mark.parametrize("max_q", [1, 100])
def test_serving_steps_in_a_graph(xs, max_q):
    """One captured step replayed with other lengths: nothing is baked into the launches."""
    s = _Server(xs, 4, 8, 2, 128, 16, 40, 100, seed=1)
    s.max_q = max_q
    s.launch()      # warm-up: every request idle
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        s.launch()
    for new in STEPS:
        s.step(new, graph.replay)
    for new in STEPS[::-1]:      # eager and replayed steps in turn
        s.step([a if a >= 0 else 0 for a in new], s.launch if sum(new) % 2 else graph.replay)


def test_readme_example(xs):
    """The README's serving step runs as printed, and computes what the entry points say."""
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "README.md")).read()
    code = next(b for b in re.findall(r"```python\n(.*?)```", text, re.S) if "xs_paged_step" in b)
    ns = dict(torch=torch, xs=xs)
    exec(code, ns)
    assert xs.xs_attn_get_device_error() == xs.XS_OK
    n, H, Hkv, D = (ns[k] for k in ("n", "H", "Hkv", "D"))
    assert ns["cache_lens"].tolist() == [20] * n and int(ns["count"]) == ns["n_pages"] - 2 * n
    # first tokens of the first and the last request: the whole attention of a prompt in 64 bits
    q, k, v = (x.double().cpu().numpy() for x in (ns["q"], ns["k"], ns["v"]))
    k, _ = pg.rope_reference(k, ns["positions"].cpu().numpy(), pg.frequencies(D), False)
    k = torch.from_numpy(k).bfloat16().double().numpy()
    for i in (0, n - 1):
        rows = slice(20 * i, 20 * i + 20)
        for h in (0, H - 1):
            g = h // (H // Hkv)
            ref, mass, _ = pg.attention_reference(q[rows, h], k[rows, g], v[rows, g], 20, True, 0, D ** -0.5)
            got = ns["out"][rows, h].double().cpu().numpy()
            u = pg.U[torch.bfloat16]     # k may round to the other neighbour: 4 u of a score, as in _Server.step
            assert (np.abs(got - ref) <= u * (mass + np.abs(ref)) * 1.01 + (1.5e-4 + 4 * u) * mass).all()


def test_two_streams_with_their_own_workspaces(xs):
    cases = [pg.PagedCase([1] * 5, [3000, 10, 900, 4000, 77], 8, 2, 128, 16, seed=i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cases]
    ws = [xs.PagedWorkspace(c.n, c.H, c.Hkv, c.D) for c in cases]
    outs = [torch.empty((c.T, c.H, c.D), dtype=c.dtype, device="cuda") for c in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, w, o, st in zip(cases, ws, outs, streams):
            xs.xs_attn_paged_plan(c.cu, c.kv, 1, w, stream=st)
            xs.xs_attn_paged_fwd(c.q, c.k, c.v, c.table, xs.XS_LAYOUT_CONTIGUOUS, [o], 0.1, w, stream=st)
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        c.check(o, None, True, 0, 0.1)


def test_two_graphs_share_a_workspace(xs):
    """Each captured plan and attention replayed in turn, the two kernels and cut tiles among them."""
    cases = [pg.PagedCase([1] * 6, [5000, 10, 900, 4000, 77, 1], 8, 2, 128, 16, seed=1),
             pg.PagedCase([90, 0, 1, 40, 7, 200], [2500, 3, 1, 4000, 77, 230], 8, 2, 128, 32, seed=2)]
    ws = xs.PagedWorkspace(6, 8, 2, 128)
    outs = [torch.empty((c.T, 8, 128), dtype=c.dtype, device="cuda") for c in cases]

    def launch(c, o):
        xs.xs_attn_paged_plan(c.cu, c.kv, max(c.q_lens), ws)
        xs.xs_attn_paged_fwd(c.q, c.k, c.v, c.table, xs.XS_LAYOUT_CONTIGUOUS, [o], 0.1, ws)

    graphs = []
    for c, o in zip(cases, outs):
        launch(c, o)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            launch(c, o)
    for turn in range(3):
        for g, c, o in zip(graphs, cases, outs):
            o.fill_(float("nan"))
            g.replay()
            c.check(o, None, True, 0, 0.1)
    assert xs.xs_attn_get_device_error() == xs.XS_OK


PLANS_IN_TURN = """
import torch
import dit_attention_ulysses_gb300 as xs
for n in (1, 2, 31, 64, 100, 130, 131, 200, 300, 400, 420, 421, 422, 500, 1000, 2000, 2500, 2700, 3000, 5000, 8192):
    cu = torch.arange(n + 1, dtype=torch.int32, device="cuda") * 2
    kv = torch.full((n,), 5, dtype=torch.int32, device="cuda")
    for max_q in (1, 300):
        xs.xs_attn_paged_plan(cu, kv, max_q, xs.PagedWorkspace(n, 8, 2, 64))
torch.cuda.synchronize()
assert xs.xs_attn_get_device_error() == xs.XS_OK
print("planned")
"""


def test_plans_of_growing_batches_in_a_new_process(xs):
    """The plan's shared memory grows with the sequences: each size launches, whatever ran before."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", PLANS_IN_TURN], cwd=root, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.strip() == "planned", r.stderr[-2000:]


def test_native_binding_and_python_checks_make_the_same_calls(xs, monkeypatch):
    """One step through the binding and through the checks in Python: the same bits, and the same refusals."""
    xs._device()
    if xs._native is None:
        pytest.skip("the binding needs PyTorch's and Python's headers")
    seen = []

    class Spy:
        def __getattr__(self, name):
            def f(*args):
                seen.append((name, getattr(native, name)(*args)))
                return seen[-1][1]
            return f

    native, outs = xs._native, []
    side = torch.cuda.Stream()
    for binding in (Spy(), None):
        monkeypatch.setattr(xs, "_native", binding)
        s = _Server(xs, 4, 8, 2, 128, 16, 40, 100, seed=1)
        for new in STEPS:
            s.step(new, s.launch)
        c = pg.PagedCase([90, 1, 7], [300, 200, 7], 8, 2, 128, 16, seed=2, q_pad=3, table_pad=2)
        ws, lse = xs.PagedWorkspace(3, 8, 2, 128), torch.empty((c.T, 8), device="cuda")
        shards = [torch.empty((c.T, 4, 128), dtype=c.dtype, device="cuda") for _ in range(2)]
        turned = torch.empty((c.T, 8, 128), dtype=c.dtype, device="cuda")
        side.wait_stream(torch.cuda.current_stream())
        xs.xs_attn_paged_plan(c.cu, c.kv, 90, ws, stream=side)
        xs.xs_attn_paged_fwd(c.q, c.k, c.v, c.table, xs.XS_LAYOUT_HEADS, shards, 0.1, ws, lse=lse, stream=side.cuda_stream)
        xs.xs_rope_fwd(c.q, torch.arange(c.T, device="cuda").int(), turned, xs.Rope(128, 64), grad=True)
        torch.cuda.synchronize()
        outs.append([*shards, lse, turned])
        with pytest.raises(TypeError, match="contiguous"):
            xs.xs_attn_paged_plan(torch.zeros(8, dtype=torch.int32, device="cuda")[::2], c.kv, 90, ws)
        with pytest.raises(TypeError, match="shapes do not match|shape"):
            xs.xs_attn_paged_fwd(c.q, c.k, c.v, c.table, xs.XS_LAYOUT_HEADS, shards[:1], 0.1, ws)
        with pytest.raises(TypeError, match="current device"):
            xs.xs_attn_paged_fwd(c.q, c.k, c.v, c.table.cpu(), xs.XS_LAYOUT_HEADS, shards, 0.1, ws)
        with pytest.raises(xs.XsError) as e:
            xs.xs_attn_paged_fwd(c.q, c.k, c.v, c.table, xs.XS_LAYOUT_HEADS, shards, -1.0, ws)
        assert e.value.code == xs.XS_ERR_SCALE
        with pytest.raises(ValueError, match="no plan"):
            xs.xs_attn_paged_fwd(c.q, c.k, c.v, c.table, xs.XS_LAYOUT_HEADS, shards, 0.1, xs.PagedWorkspace(3, 8, 2, 128))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    taken = {name for name, code in seen if code == xs.XS_OK}
    assert taken == {"rope", "append", "step", "plan", "attn"}
