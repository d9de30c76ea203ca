"""The division of work that xs_attn_paged_plan writes, read back from the workspace: every key block of
every tile exactly once and the records of cut tiles right, for random and for chosen batches, with the
tilings that the library uses (waves, sorted whole tiles, slots of many tiles, parts limited by their
join, even parts, few keys)."""
import math
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


def _plan(xs, q_lens, kv_lens, H, Hkv, D, max_q, causal, window):
    n = len(q_lens)
    cu = torch.tensor([0] + q_lens, dtype=torch.int64).cumsum(0).int().cuda()
    ws = xs.PagedWorkspace(n, H, Hkv, D)
    ws._buf.fill_(0xab)
    xs.xs_attn_paged_plan(cu, torch.tensor(kv_lens, dtype=torch.int32).cuda(), max_q, ws, causal=causal, window=window)
    start = ws.ptr - ws._buf.data_ptr()
    raw = ws._buf[start:start + ws.nbytes].cpu().numpy().tobytes()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return pp.check(pp.Plan(raw, n, sms), q_lens, kv_lens, H, Hkv, int(causal), window)


# What the batch is for: q_lens, kv_lens, H, Hkv, D, max_q, window, and what the plan of it has to be
CHOSEN = {
    "one token, one sequence: cut": (([1], [131072], 8, 1, 128, 1, 0), lambda w, s, whole, cut, parts: cut == 1 and parts > 64),
    "few keys, even parts": (([1], [6000], 32, 8, 128, 1, 0), lambda w, s, whole, cut, parts: cut == 8 and 31 <= parts <= 32),
    "short sequences: whole": (([1] * 40, [100] * 40, 8, 2, 128, 1, 0), lambda w, s, whole, cut, parts: cut == 0 and whole == 80),
    "drafts: cut": (([8], [32768], 32, 8, 128, 8, 0), lambda w, s, whole, cut, parts: cut == 8 and parts > 8),
    "sorted whole tiles": (([2048], [2048], 32, 8, 128, 2048, 0), lambda w, s, whole, cut, parts: w > 1 and cut == 0),
    "a partial last wave": (([64] * 8, [8192] * 8, 32, 8, 128, 64, 0), lambda w, s, whole, cut, parts: w == 1 and cut == 0),
    "waves, then cuts": (([4608], [18432], 24, 24, 128, 4608, 0), lambda w, s, whole, cut, parts: w > 1),
    "slots of many tiles": (([300] * 300, [900] * 300, 64, 64, 64, 300, 0), lambda w, s, whole, cut, parts: w > 1 and s > 1),
    "a window": (([512, 3, 77, 1] * 6, [6000, 50, 77, 4000] * 6, 12, 6, 64, 512, 1000), lambda w, s, whole, cut, parts: w >= 1),
    "nothing to do": (([0, 0], [5, 0], 2, 1, 64, 1, 0), lambda w, s, whole, cut, parts: whole == cut == 0),
    "rows that see nothing": (([50, 3], [2, 0], 4, 4, 64, 50, 0), lambda w, s, whole, cut, parts: whole + cut == 8),
}


@pytest.mark.parametrize("name", CHOSEN, ids=lambda x: x.replace(" ", "_"))
def test_chosen_batches(xs, name):
    (q_lens, kv_lens, H, Hkv, D, max_q, window), expected = CHOSEN[name]
    got = _plan(xs, q_lens, kv_lens, H, Hkv, D, max_q, True, window)
    assert expected(*got), got


def draw(r):
    """Batches of up to some 6000 tiles: few or many sequences, ragged or even, short or long."""
    log = lambda lo, hi: min(hi, int(math.exp(r.uniform(math.log(lo), math.log(hi + 1)))))   # noqa: E731
    while True:
        Hkv, G, D = r.choice([1, 2, 3, 8, 24]), r.choice([1, 2, 3, 4, 5, 8, 16, 40, 128]), r.choice([64, 128])
        n, most_q, most_kv = log(1, 500), r.choice([1, 1, log(1, 16), log(2, 4000)]), log(1, r.choice([2000, 40000, 300000]))
        even = r.random() < 0.4
        q, kv = [], []
        for _ in range(n):
            q.append(most_q if even else r.choice([0, 1, log(1, most_q), most_q]))
            kv.append(q[-1] + most_kv if even else max(0, r.choice([q[-1] + log(1, most_kv), q[-1], q[-1] - r.randint(0, q[-1]), 0])))
        causal = r.random() < 0.7
        window = log(1, 5000) if causal and r.random() < 0.4 else 0
        max_q = r.choice([max(q + [1])] * 4 + [1, 5000])
        tokens = max(1, (16 if G * max_q <= 16 else 128) // G)
        if Hkv * sum(-(-x // tokens) for x in q) <= 6000 and Hkv * G <= 4096:
            return q, kv, Hkv * G, Hkv, D, max_q, causal, window


@pytest.mark.parametrize("seed", range(6))
def test_random_batches(xs, seed):
    r = random.Random(seed)
    forms = set()
    for _ in range(60):
        case = draw(r)
        try:
            w, slot, whole, cut, parts = _plan(xs, *case)
        except AssertionError as e:
            raise AssertionError(f"{case}: {e}") from e
        forms.add((w > 0, whole > 0, cut > 0, parts > 2))
    assert len(forms) >= 4
