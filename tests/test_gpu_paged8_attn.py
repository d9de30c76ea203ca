"""xs_attn_paged8_fwd on the GPU against plain attention in 64 bits over the elements that the cache stands
for (_paged8.py has the bounds)."""
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


def _run(xs, c, causal=True, window=0, scale=None, max_q=None, ws=None, lse=True, layout=None, P=1, fill=float("nan")):
    scale = c.D ** -0.5 if scale is None else scale
    max_q = max(max(c.q_lens), 1) if max_q is None else max_q
    ws = ws or xs.PagedWorkspace(c.n, c.H, c.Hkv, c.D)
    layout = xs.XS_LAYOUT_CONTIGUOUS if layout is None else layout
    shape = {xs.XS_LAYOUT_A2A: (c.T // P, c.H, c.D), xs.XS_LAYOUT_HEADS: (c.T, c.H // P, c.D)}.get(layout, (c.T, c.H, c.D))
    outs = [torch.full(shape, fill, dtype=c.dtype, device="cuda") for _ in range(P)]
    z = torch.full((c.T, c.H), fill, dtype=torch.float32, device="cuda") if lse else None
    xs.xs_attn_paged8_plan(c.cu, c.kv, max_q, ws, causal=causal, window=window)
    xs.xs_attn_paged8_fwd(c.q, *c.cache, c.table, layout, outs, scale, ws, lse=z)
    assert xs.xs_attn_get_device_error_info()[0] == xs.XS_OK
    return (outs if P > 1 else outs[0]), z


# q_lens, kv_lens, H, Hkv, D, page, block
DECODE = [
    ([1], [1], 1, 1, 64, 16, 16),
    ([1], [33], 2, 1, 128, 16, 16),
    ([1], [5000], 8, 2, 128, 32, 32),
    ([1, 1, 1], [31, 32, 33], 4, 4, 64, 32, 16),
    ([1, 0, 1, 0, 1], [700, 50, 1, 0, 257], 12, 4, 128, 64, 64),
    ([1] * 40, [1 + 97 * i for i in range(40)], 8, 1, 128, 16, 16),
    ([2, 1, 4, 3], [900, 3, 4, 130], 8, 2, 64, 128, 128),
    ([1, 1], [3000, 2100], 28, 4, 128, 256, 32),   # 7 heads to a KV head
    ([1, 3], [70, 900], 5, 1, 128, 1024, 128),
    ([3, 3], [4000, 2], 10, 2, 64, 64, 16),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("case", DECODE, ids=lambda c: "n%d_kv%d_H%d_%d_D%d_p%d_b%d" % (len(c[0]), max(c[1]), *c[2:]))
def test_few_tokens(xs, case, dtype):
    c = p8.Paged8Case(*case, dtype=dtype, seed=len(case[0]), extra_rows=2)
    out, lse = _run(xs, c)
    c.check(out, lse, True, 0, c.D ** -0.5)
    rows = sum(c.q_lens)
    assert out[rows:].isnan().all() and lse[rows:].isnan().all()     # rows behind the last sequence
    out2, _ = _run(xs, c, lse=False)
    assert torch.equal(out2[:rows], out[:rows])


FEW_HEADS = [   # one tile of a few rows of the chunk kernel, and of heads that do not divide its 128
    ([1], [700], 32, 1, 128, 32, 16),
    ([1, 2], [500, 3000], 40, 1, 128, 16, 16),
    ([1, 1, 0, 3], [900, 128, 5, 40000], 128, 1, 64, 64, 64),
    ([5, 6, 1], [20, 5000, 300], 32, 8, 128, 32, 32),
    ([33], [1300], 48, 2, 128, 128, 128),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("case", FEW_HEADS, ids=lambda c: "n%d_kv%d_H%d_%d_D%d_p%d_b%d" % (len(c[0]), max(c[1]), *c[2:]))
def test_many_heads_to_a_key(xs, case, dtype):
    c = p8.Paged8Case(*case, dtype=dtype, seed=len(case[0]), extra_rows=2)
    out, lse = _run(xs, c)
    c.check(out, lse, True, 0, c.D ** -0.5)
    rows = sum(c.q_lens)
    assert out[rows:].isnan().all() and lse[rows:].isnan().all()


CHUNKS = [  # q_lens, kv_lens, H, Hkv, D, page, block, causal, window
    ([130], [130], 2, 2, 128, 16, 16, True, 0),
    ([128], [256], 2, 1, 64, 64, 32, False, 0),
    ([257, 1, 64], [1000, 700, 64], 8, 2, 128, 16, 16, True, 0),
    ([100, 3, 0, 31], [100, 900, 77, 2000], 6, 2, 64, 32, 32, True, 100),
    ([300], [1111], 3, 1, 128, 128, 128, True, 1),
    ([200, 129], [200, 1500], 5, 5, 128, 256, 64, True, 200),
    ([65, 200], [500, 201], 4, 4, 128, 32, 16, False, 0),
    ([90], [2500], 24, 8, 64, 1024, 128, False, 0),
    ([10, 6], [4, 0], 4, 2, 128, 16, 16, True, 0),      # more new tokens than keys: rows that see nothing
    ([10, 6], [4, 0], 4, 2, 64, 16, 16, False, 0),
    ([40, 200], [30, 150], 2, 1, 128, 16, 16, True, 7),
    ([17] * 33, [17 + 13 * i for i in range(33)], 4, 1, 128, 16, 16, True, 0),
    ([515], [2061], 8, 1, 128, 64, 32, True, 0),
    ([77, 400], [1500, 400], 7, 1, 128, 32, 32, True, 0),     # 18 tokens of 7 heads: 126 of 128 rows
    ([301], [700], 24, 1, 64, 16, 16, True, 333),
    ([2000], [2000], 2, 1, 64, 16, 16, True, 0),
    ([129] * 9, [129 * (i + 1) for i in range(9)], 12, 3, 128, 64, 64, False, 0),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("case", CHUNKS, ids=lambda c: "q%d_kv%d_H%d_%d_D%d_p%d_b%d_%s_w%d" % (
    max(c[0]), max(c[1]), *c[2:7], "causal" if c[7] else "full", c[8]))
def test_chunks(xs, case, dtype):
    *shape, causal, window = case
    c = p8.Paged8Case(*shape, dtype=dtype, seed=sum(case[0]), extra_rows=1, window=window, freed=window > 0)
    out, lse = _run(xs, c, causal, window)
    c.check(out, lse, causal, window, c.D ** -0.5)
    rows = sum(c.q_lens)
    assert out[rows:].isnan().all() and lse[rows:].isnan().all()


PAIRS = [   # q_lens, kv_lens, H, Hkv, D, page, block, causal, window: enough sequences for tiles of two KV heads, and odd heads
    ([1] * 80, [1 + (37 * i) % 700 for i in range(80)], 16, 4, 128, 16, 16, True, 0),
    ([1] * 160, [1 + (61 * i) % 500 for i in range(160)], 2, 2, 64, 64, 32, True, 0),
    ([(i * 5) % 3 for i in range(90)], [3 + (53 * i) % 400 for i in range(90)], 12, 4, 64, 16, 16, True, 100),
    ([1] * 53, [2000 - 31 * i for i in range(53)], 48, 6, 128, 32, 16, False, 0),
    ([2] * 40, [2 + (97 * i) % 3000 for i in range(40)], 32, 8, 128, 128, 64, True, 33),
    ([1] * 110, [1 + (37 * i) % 300 for i in range(110)], 6, 3, 128, 16, 16, True, 0),
]


@pytest.mark.parametrize("form", [dict(), dict(heads_first=True), dict(one_buffer=True), dict(q_pad=3, table_pad=2)], ids=str)
@pytest.mark.parametrize("case", PAIRS, ids=lambda c: "n%d_H%d_%d_D%d_p%d_b%d_w%d" % (len(c[0]), *c[2:7], c[8]))
def test_many_sequences(xs, case, form):
    *shape, causal, window = case
    dtype = torch.bfloat16 if len(form) != 1 else torch.float16
    c = p8.Paged8Case(*shape, dtype=dtype, seed=sum(case[0]), extra_rows=1, window=window, freed=window > 0, **form)
    ws = xs.PagedWorkspace(c.n, c.H, c.Hkv, c.D)
    out, lse = _run(xs, c, causal, window, ws=ws)
    c.check(out, lse, causal, window, c.D ** -0.5)
    rows = sum(c.q_lens)
    assert out[rows:].isnan().all() and lse[rows:].isnan().all()
    out2, lse2 = _run(xs, c, causal, window, ws=ws)      # the same plan and the same bits
    assert torch.equal(out2[:rows], out[:rows]) and torch.equal(lse2[:rows], lse[:rows])
