"""Windowed attention over a cache whose keys and values before the window hold NaN or infinities,
those of the page in which the window begins among them: no row sees them, so none of them may
reach an output (_paged.py has the bounds)."""
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


def spoil(c, window, what):
    """Every key and value that no row of its sequence sees becomes `what`."""
    for i in range(c.n):
        first = max(0, c.kv_lens[i] - c.q_lens[i] - window + 1)
        for t in range(first):
            e = int(c.table[i, t // c.page])
            c.k[e, t % c.page] = what
            c.v[e, t % c.page] = what


# q_lens, kv_lens, H, Hkv, D, page, window
CASES = [
    ([1], [300], 4, 2, 64, 16, 20),
    ([1, 1, 1], [700, 33, 1], 8, 2, 128, 64, 7),
    ([3, 1, 2], [900, 1300, 40], 4, 1, 64, 128, 100),
    ([1], [9000], 8, 1, 128, 1024, 4000),                       # cut among CTAs
    ([70], [700], 4, 2, 64, 16, 30),
    ([200, 1, 40], [1000, 400, 40], 8, 2, 128, 64, 90),
    ([300, 17], [3000, 2500], 6, 6, 64, 256, 1000),
    ([20], [20000], 32, 2, 128, 128, 15001),                    # cut among CTAs
]


@pytest.mark.parametrize("what", [float("nan"), float("inf")], ids=["nan", "inf"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "q%d_kv%d_D%d_p%d_w%d" % (max(c[0]), max(c[1]), *c[4:]))
def test_what_lies_before_the_window(xs, case, dtype, what):
    *shape, window = case
    c = pg.PagedCase(*shape, dtype=dtype, seed=window, window=window)
    spoil(c, window, what)
    ws = xs.PagedWorkspace(c.n, c.H, c.Hkv, c.D)
    out = torch.full((c.T, c.H, c.D), float("nan"), dtype=dtype, device="cuda")
    lse = torch.full((c.T, c.H), float("nan"), device="cuda")
    xs.xs_attn_paged_plan(c.cu, c.kv, max(c.q_lens), ws, causal=True, window=window)
    xs.xs_attn_paged_fwd(c.q, c.k, c.v, c.table, xs.XS_LAYOUT_CONTIGUOUS, [out], c.D ** -0.5, ws, lse=lse)
    assert xs.xs_attn_get_device_error() == xs.XS_OK
    c.check(out, lse, True, window, c.D ** -0.5)
