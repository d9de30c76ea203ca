"""The Python side of the serving calls without a GPU: a rotation filled anew, and whole numbers
that a C int does not hold.  Host tensors only, which every call refuses in the end."""
import copy
import pickle

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def xs():
    from conftest import build_library
    build_library()
    import dit_attention_ulysses_gb300 as xs
    return xs


OTHER = dict(D=64, rot=32, layout=1, base=5e5, scaling=3, factor=8.0, context=8192.0, low=1.0, high=32.0, magnitude=1.25)


def test_a_rotation_filled_anew_is_the_new_one(xs):
    """xs_rope_init on a Rope: its dimensions, its table and its copies are the new rotation's."""
    a = xs.Rope(128, 48)
    xs.xs_rope_init(a, *OTHER.values())
    want = bytes(xs.Rope(**OTHER)._struct)
    assert (a.D, a.rot) == (64, 32) and bytes(a._struct) == want
    for b in (copy.copy(a), copy.deepcopy(a), pickle.loads(pickle.dumps(a))):
        assert (b.D, b.rot) == (64, 32) and bytes(b._struct) == want and b.ptr != a.ptr


def test_a_rotation_that_is_refused_stays_as_it_was(xs):
    a = xs.Rope(128, 48)
    before = bytes(a._struct)
    with pytest.raises(xs.XsError) as e:
        xs.xs_rope_init(a, *{**OTHER, "rot": 40}.values())
    assert e.value.code == xs.XS_ERR_ROPE
    assert (a.D, a.rot) == (128, 48) and bytes(a._struct) == before and bytes(copy.copy(a)._struct) == before


WIDE = [2 ** 31, 2 ** 32 + 16, -2 ** 31 - 1, -2 ** 32, 2 ** 40, 2 ** 64 + 16]


@pytest.mark.parametrize("value", WIDE)
def test_numbers_that_no_c_int_holds_are_refused(xs, value, monkeypatch):
    """ctypes would pass their lower 32 bits on: a page size of 2^32 + 16 would be one of 16."""
    i32 = dict(dtype=torch.int32)
    ints = lambda n: torch.zeros(n, **i32)   # noqa: E731
    for name, code in (("D", xs.XS_ERR_HEAD_DIM), ("rot", xs.XS_ERR_ROPE), ("layout", xs.XS_ERR_LAYOUT), ("scaling", xs.XS_ERR_ROPE)):
        with pytest.raises(xs.XsError) as e:
            xs.Rope(**{**OTHER, name: value})
        assert e.value.code == code
    xs._device()
    # the checks see host tensors as ones of the current device; no call may reach the library
    monkeypatch.setattr(xs, "_on_device", lambda t, name, dev: None)
    monkeypatch.setattr(xs, "_native", None)
    monkeypatch.setattr(xs, "_vec", lambda t, name, dtype, n, dev: 0)

    class Library:
        xs_attn_error_string = xs.lib.xs_attn_error_string

        def __getattr__(self, name):
            raise AssertionError(f"{name} was called")

    monkeypatch.setattr(xs, "lib", Library())
    with pytest.raises(xs.XsError) as e:
        xs.xs_paged_step(ints(2), ints(2), torch.zeros((2, 3), **i32), ints(9), ints(1), value, ints(2), ints(3), ints(4),
                         torch.zeros(4, dtype=torch.int64), ints(1), ints(2))
    assert e.value.code == xs.XS_ERR_PAGE

    class Workspace:
        n, H, Hkv, D, ptr, nbytes, planned = 2, 4, 2, 64, 256, 1 << 20, None
        _buf = ints(1)
        _dims = (n, H, Hkv, D, ptr, nbytes)

    for max_q, window in ((value, 0), (1, value)):
        with pytest.raises(xs.XsError) as e:
            xs.xs_attn_paged_plan(ints(3), ints(2), max_q, Workspace, window=window)
        assert e.value.code == xs.XS_ERR_SHAPE and Workspace.planned is None
