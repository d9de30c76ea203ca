"""The division of work that xs_attn_paged8_plan writes, read back from the workspace (_paged_plan.py): every key block of
every tile exactly once, the records of cut tiles right, tiles of two KV heads among them, and what counts as fitting L2."""
import random

import pytest

import _paged_plan as pp

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def xs():
    from conftest import build_library
    build_library()
    import dit_attention_ulysses_gb300 as xs
    assert torch.cuda.is_available()
    return xs


def _plan(xs, call, q_lens, kv_lens, H, Hkv, D, max_q, causal, window):
    n = len(q_lens)
    cu = torch.tensor([0] + q_lens, dtype=torch.int64).cumsum(0).int().cuda()
    ws = xs.PagedWorkspace(n, H, Hkv, D)
    ws._buf.fill_(0xab)
    getattr(xs, call)(cu, torch.tensor(kv_lens, dtype=torch.int32).cuda(), max_q, ws, causal=causal, window=window)
    start = ws.ptr - ws._buf.data_ptr()
    raw = ws._buf[start:start + ws.nbytes].cpu().numpy().tobytes()
    plan = pp.Plan(raw, n, torch.cuda.get_device_properties(0).multi_processor_count)
    heads = int(plan.header["Hkv"])
    assert heads == Hkv or 2 * heads == Hkv
    return pp.check(plan, q_lens, kv_lens, H, heads, int(causal), window), heads


# What the batch is for: q_lens, kv_lens, H, Hkv, D, max_q, window, and what the plan of it has to be
CHOSEN = {
    "one token, one sequence: cut": (([1], [131072], 8, 1, 128, 1, 0), lambda w, s, whole, cut, parts, heads: cut == 1 and parts > 64),
    "pairs of heads": (([1] * 80, [900] * 80, 32, 8, 128, 1, 0), lambda w, s, whole, cut, parts, heads: heads == 4),
    "heads that are no pairs": (([1] * 120, [900] * 120, 6, 3, 128, 1, 0), lambda w, s, whole, cut, parts, heads: heads == 3),
    "few sequences: single heads": (([1] * 30, [900] * 30, 32, 8, 128, 1, 0), lambda w, s, whole, cut, parts, heads: heads == 8),
    "sorted whole tiles": (([2048], [2048], 32, 8, 128, 2048, 0), lambda w, s, whole, cut, parts, heads: w > 1 and cut == 0),
    "keys that stay in L2 (61 MB): cut": (([96] * 8, [3896] * 8, 32, 8, 128, 96, 0), lambda w, s, whole, cut, parts, heads: w == 0),
    "keys that do not (111 MB): a wave": (([96] * 8, [7096] * 8, 32, 8, 128, 96, 0), lambda w, s, whole, cut, parts, heads: w == 1),
    "heads of 64 that stay in L2 (42 MB)": (([192] * 8, [5392] * 8, 16, 8, 64, 192, 0), lambda w, s, whole, cut, parts, heads: w == 0),
    "waves, then cuts": (([4608], [18432], 24, 24, 128, 4608, 0), lambda w, s, whole, cut, parts, heads: w > 1),
    "a window": (([512, 3, 77, 1] * 6, [6000, 50, 77, 4000] * 6, 12, 6, 64, 512, 1000), lambda w, s, whole, cut, parts, heads: w >= 1),
    "nothing to do": (([0, 0], [5, 0], 2, 1, 64, 1, 0), lambda w, s, whole, cut, parts, heads: whole == cut == 0),
}


@pytest.mark.parametrize("name", CHOSEN, ids=lambda x: x.replace(" ", "_"))
def test_chosen_batches(xs, name):
    (q_lens, kv_lens, H, Hkv, D, max_q, window), expected = CHOSEN[name]
    got, heads = _plan(xs, "xs_attn_paged8_plan", q_lens, kv_lens, H, Hkv, D, max_q, True, window)
    assert expected(*got, heads), (got, heads)


@pytest.mark.parametrize("seed", range(4))
def test_random_batches(xs, seed):
    r = random.Random(seed)
    for _ in range(12):
        Hkv, D, n = r.choice([1, 2, 3, 4, 8]), r.choice([64, 128]), r.choice([1, 3, 40, 200])
        most = r.choice([1, 1, 7, 300])
        q_lens = [r.randint(0, most) for _ in range(n)]
        kv_lens = [q + r.randint(0, r.choice([10, 1000, 20000])) for q in q_lens]
        causal = r.random() < 0.7
        window = r.choice([0, 0, 333]) if causal else 0
        for call in ("xs_attn_paged8_plan", "xs_attn_paged_plan"):
            _plan(xs, call, q_lens, kv_lens, Hkv * r.choice([1, 4, 8]), Hkv, D, max(most, 1), causal, window)
