"""The record of the first device error, whichever kernel reports it: attention of few tokens and of
chunks find a plan that was made for other arguments, compute nothing, and say so."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def xs():
    from conftest import build_library
    build_library()
    import dit_attention_ulysses_gb300 as xs
    assert torch.cuda.is_available()
    return xs


def _mismatch(xs, planned, called):
    """A plan of 4-head tiles for up to `planned` tokens, called as one for up to `called`."""
    cu, kv = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 1], [40]))
    q, out = (torch.full((1, 4, 64), 5.0, device="cuda").bfloat16() for _ in range(2))
    k, v = (torch.zeros((3, 16, 1, 64), device="cuda").bfloat16() for _ in "kv")
    table = torch.arange(3, dtype=torch.int32, device="cuda")[None]
    ws = xs.PagedWorkspace(1, 4, 1, 64)
    xs.xs_attn_paged_plan(cu, kv, planned, ws)
    ws.planned = (called, *ws.planned[1:])
    xs.xs_attn_paged_fwd(q, k, v, table, xs.XS_LAYOUT_CONTIGUOUS, [out], 0.1, ws)
    torch.cuda.synchronize()
    assert (out == 5.0).all()


FEW, CHUNK = (1, 1000), (1000, 1)      # the record holds the plan's tokens per tile: 16 / 4 or 128 / 4
TOKENS = {FEW: 4, CHUNK: 32}


@pytest.mark.parametrize("order", [(FEW,), (CHUNK,), (FEW, CHUNK), (CHUNK, FEW), (FEW, CHUNK, FEW), (CHUNK, CHUNK, FEW)],
                         ids=lambda o: "-".join({FEW: "few", CHUNK: "chunk"}[x] for x in o))
def test_the_first_error_is_the_one_recorded(xs, order):
    assert xs.xs_attn_get_device_error() == xs.XS_OK
    for planned, called in order:
        _mismatch(xs, planned, called)
    code, rec = xs.xs_attn_get_device_error_info()
    assert code == xs.XS_ERR_DEVICE_BOUNDS and rec["kind"] == 3 and rec["site"] == 3
    assert (rec["detail0"], rec["detail1"]) == (1, TOKENS[order[0]])
    assert xs.xs_attn_get_device_error_info() == (xs.XS_OK, {k: 0 for k in rec})   # all of them are cleared
