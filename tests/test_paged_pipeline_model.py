"""The mbarrier protocol of the paged chunk kernel on a host model (_paged_pipeline_model.py): for
random lists of pieces (one block to many, cut tiles among them) and random timing no parity
alias, no buffer or descriptor overwritten too early, no deadlock, at both head sizes; planted
errors are caught."""
import random

import pytest

import _paged_pipeline_model as pm


def _pieces(r):
    sizes = r.choice([[1], [1, 2], [1, 2, 3], [2, 3, 4, 5], [1, 4, 9, 30], [12], [1, 1, 1, 17]])
    n = r.randint(1, 14)
    blocks = [r.choice(sizes) for _ in range(n)]
    return blocks, [r.random() < 0.4 for _ in blocks]


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("stall", [0.3, 0.85, 0.97])
def test_protocol(D, stall):
    r = random.Random(D)
    for seed in range(60):
        blocks, parts = _pieces(r)
        pm.run_cta(blocks, parts, D=D, seed=seed, stall=stall)


@pytest.mark.parametrize("mutate", pm.MUTATIONS)
def test_planted_errors_are_caught(mutate):
    r = random.Random(1)
    caught = 0
    for seed in range(40):
        blocks, parts = _pieces(r)
        try:
            pm.run_cta(blocks, parts, D=128, seed=seed, mutate=mutate)
        except AssertionError:
            caught += 1
    assert caught > 0
