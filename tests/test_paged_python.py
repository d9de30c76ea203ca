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
