"""Scores so far from 0 that fp32 holds few of their digits: attention over the paged caches."""
import numpy as np
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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("q", [1, 200])
@pytest.mark.parametrize("power", [4, 6, 8, 9])
def test_scores_far_from_zero_over_8_bits(xs, power, q, dtype):
    """All scores alike and far below zero, up to -2.1e6: the mean of the values, of blocks with unlike scales; and one key as
    far above: its values."""
    from test_gpu_paged8_attn import _run
    c = p8.Paged8Case([q], [700], 2, 2, 64, 16, seed=6, dtype=dtype, spread=3)
    big = 2.0 ** power
    score = 64 * big * big / 8
    c.q.fill_(big)
    c.k.view(torch.uint8)[:] = int(p8.codes(np.array([-1.0]))[0])
    c.ks.view(torch.uint8)[:] = 127 + power
    out, lse = _run(xs, c, causal=False)
    u = pg.U[dtype]
    v, a = np.mean(c.values[0], axis=0), np.mean(np.abs(c.values[0]), axis=0)
    # the maximum, the block's exponent and their difference are rounded once each: 2^-22 |score log2(e)| powers of two
    # in all, ln 2 times as much of a weight; numerator and denominator are weighed alike but for v_inv
    off = 2 * np.expm1(score * 2.0 ** -22)
    before = (off + 2.0 ** -11 + 1.5e-4) * a + 2.0 ** -32 * 700 * c.vmax
    got = out.double().cpu().numpy()
    assert (np.abs(got - v) <= before + u * (np.abs(v) + before)).all()
    assert ((lse.double() / -score - 1).abs() <= 2.0 ** -21 + 8 / score).all()     # the logarithm of 700, and its error
    c.k.view(torch.uint8)[c.table[0, 30].long(), 5] = int(p8.codes(np.array([1.0]))[0])
    out, lse = _run(xs, c, causal=False)
    one = torch.from_numpy(c.values[0][30 * 16 + 5]).cuda()
    # its probability is rounded to fp16, its quotient by the sum to the type
    assert ((out.double() - one).abs() <= (2.0 ** -11 + 1e-6 + u) * 1.01 * one.abs()).all()
    assert ((lse.double() / score - 1).abs() <= 2.0 ** -21).all()
