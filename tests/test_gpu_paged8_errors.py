"""Device errors of the kernels over both paged caches: found by one look, the earliest reported, all cleared; and what a
read of a clean state costs."""
import itertools
import time

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


FAMILIES = [(8, 1), (8, 100), (16, 1), (16, 100)]      # bits, the upper estimate of new tokens that chooses the kernel


def _mismatch(xs, bits, max_q):
    """A call whose window is not its plan's: it computes nothing.  The record holds the plan's tokens of a tile."""
    c = (p8.Paged8Case if bits == 8 else pg.PagedCase)([1], [40], 4, 2, 64, 16, seed=3)
    ws = xs.PagedWorkspace(c.n, c.H, c.Hkv, c.D)
    out = torch.full((c.T, c.H, c.D), 5.0, dtype=c.dtype, device="cuda")
    cache = c.cache if bits == 8 else (c.k, c.v)
    name = "xs_attn_paged8" if bits == 8 else "xs_attn_paged"
    getattr(xs, name + "_plan")(c.cu, c.kv, max_q, ws)
    ws.planned = (max_q, 1, 9)
    getattr(xs, name + "_fwd")(c.q, *cache, c.table, xs.XS_LAYOUT_CONTIGUOUS, [out], 0.1, ws)
    torch.cuda.synchronize()
    assert (out == 5.0).all()
    return {(8, 1): 4, (16, 1): 8}.get((bits, max_q), 64)


@pytest.mark.parametrize("order", [o for n in (1, 2) for o in itertools.permutations(FAMILIES, n)] + [FAMILIES, FAMILIES[::-1]],
                         ids=lambda o: "_".join("%d-%d" % x for x in o))
def test_the_earliest_of_all_families(xs, order):
    assert xs.xs_attn_get_device_error() == xs.XS_OK
    tokens = [_mismatch(xs, *f) for f in order]
    code, rec = xs.xs_attn_get_device_error_info()
    assert code == xs.XS_ERR_DEVICE_BOUNDS and rec["site"] == 3 and rec["detail1"] == tokens[0]
    assert xs.xs_attn_get_device_error_info() == (xs.XS_OK, {k: 0 for k in rec})


def test_a_read_of_a_clean_state_is_a_few_copies(xs):
    """At most what six blocking copies of four bytes take (it is a look at all words of the paged kernels, one copy of
    what it found, and two of the dense kernels' words; two of every family were ten)."""
    x = torch.zeros(1, dtype=torch.int32, device="cuda")

    def best(f):
        times = []
        for _ in range(300):
            t = time.perf_counter()
            f()
            times.append(time.perf_counter() - t)
        return sorted(times)[15]

    assert xs.xs_attn_get_device_error() == xs.XS_OK
    assert best(xs.xs_attn_get_device_error) <= 6 * best(x.item)
