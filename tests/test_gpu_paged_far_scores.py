"""Scores so far from 0 that fp32 holds few of their digits: attention over the paged caches."""
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


@pytest.mark.parametrize("base", range(0, 2048, 512))
def test_a_maximum_that_rises_by_one_step(xs, base):
    """Two keys whose scores are fp32's neighbours, 16 apart in powers of two, the rest 2^28 below: the second takes all
    but 2^-16, wherever the first falls on the even or the odd number."""
    from test_gpu_paged_attn import _run
    c = pg.PagedCase([1], [300], 1, 1, 64, 16, seed=6, dtype=torch.float16)
    c.q.zero_(), c.k.zero_()
    c.q[0, 0, :3] = torch.tensor([65504.0, 65504.0, 1.0])
    for key, e in ((0, base), (128, base + 512)):        # of one warp, one group after the other
        c.k[c.table[0, key // 16].long(), key % 16, 0, :3] = torch.tensor([65504.0, 65504.0, e], dtype=torch.float16).cuda()
    out, lse = _run(xs, c, causal=False, scale=float(np.log(2) / 32))
    want = c.values[0][128, 0]
    # 2^-16 of the values beside it, and half a step of fp16
    assert (np.abs(out.double().cpu().numpy()[0, 0] - want) <= 2.0 ** -14 + 2.0 ** -11 * np.abs(want)).all()
    assert lse.isfinite().all()
