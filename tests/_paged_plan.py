"""Reader of a planned workspace of the paged attention, and the check of its division of work (test
infrastructure only).  Layout and records are those of csrc/paged.h and csrc/api_paged.cu."""
import numpy as np

MAX_WAVES = 64
POS = [("seq", "i4"), ("head", "i4"), ("tile", "i4"), ("k", "i4")]
SEQ = [("q_start", "i4"), ("q_len", "i4"), ("kv_len", "i4"), ("index", "i4")]
HEADER = np.dtype([(n, "i4") for n in ("n_seqs", "ranges", "n", "H", "Hkv", "D", "tokens", "block", "grid", "causal", "window",
                                       "waves", "slot", "slot_ctas", "unused0", "unused1")])
RANGE = np.dtype([("start", POS), ("end", POS), ("first", SEQ), ("c0", "i4"), ("c1", "i4"), ("c1_last", "i4"), ("unused", "i4")])
SLOT = np.dtype([("pos", POS), ("seq", SEQ)])


class Plan:
    """Header, counters, ranges, sequences and slots of a workspace (`raw`: its bytes from the aligned start)."""

    def __init__(self, raw, n, sms):
        at = 0

        def take(dtype, count):
            nonlocal at
            x = np.frombuffer(raw, dtype, count, at)
            at += (x.nbytes + 255) // 256 * 256
            return x

        self.header = take(HEADER, 1)[0]
        self.counters = take(np.dtype("u4"), 2 * sms)
        self.ranges = take(RANGE, 2 * sms)
        self.seqs = take(np.dtype(SEQ), n)
        self.slots = take(SLOT, 2 * sms * MAX_WAVES).reshape(2 * sms, MAX_WAVES)


def tile_blocks(q_len, kv_len, t, tokens, block, causal, window):
    """First key block of a tile and their number, from its rows: the blocks from the first key that a row
    sees to the last (one key where the rows see none)."""
    base = kv_len - q_len
    first, last = base + t * tokens, base + min((t + 1) * tokens, q_len) - 1
    hi = max(1, last + 1 if causal else kv_len)
    lo = max(0, first - window + 1) if window else 0
    return lo // block, -(-hi // block) - lo // block


def check(plan, q_lens, kv_lens, H, Hkv, causal, window):
    """Every block of every tile exactly once; a cut tile's pieces on the CTAs c0 .. c1 that all its records
    name, one each, in the order of the keys.  Returns (waves, tiles of a slot, whole tiles, cut tiles, most
    parts of a tile)."""
    h = plan.header
    tokens, block, grid = int(h["tokens"]), int(h["block"]), int(h["grid"])
    kept = [i for i in range(len(q_lens)) if q_lens[i] > 0]
    assert (h["n"], h["H"], h["Hkv"], h["causal"], h["window"]) == (len(q_lens), H, Hkv, causal, window)
    assert h["n_seqs"] == len(kept) and 0 <= h["waves"] <= MAX_WAVES and 1 <= h["slot"] <= 64 and not plan.counters[:grid].any()
    starts = np.concatenate([[0], np.cumsum(q_lens)])
    want = [(int(starts[i]), int(q_lens[i]), int(kv_lens[i]), i) for i in kept]
    assert [tuple(s) for s in plan.seqs[:len(kept)].tolist()] == want
    tiles_of = [-(-s[1] // tokens) for s in want]
    blocks = {}

    def count(pos):
        seq, head, tile, _ = pos
        assert 0 <= seq < len(kept) and 0 <= head < Hkv and 0 <= tile < tiles_of[seq], pos
        if (seq, tile) not in blocks:
            blocks[seq, tile] = tile_blocks(want[seq][1], want[seq][2], tile, tokens, block, causal, window)[1]
        return blocks[seq, tile]

    def after(pos):
        seq, head, tile, _ = pos
        if tile + 1 < tiles_of[seq]:
            return seq, head, tile + 1, 0
        return (seq, head + 1, 0, 0) if head + 1 < Hkv else (seq + 1, 0, 0, 0)

    whole, pieces = set(), {}
    for c in range(grid):
        for w in range(int(h["waves"]) - (c >= h["slot_ctas"])):
            slot = plan.slots[c, w]
            pos = tuple(slot["pos"].tolist())
            assert tuple(slot["seq"].tolist()) == want[pos[0]] and pos[3] == 0
            for _ in range(int(h["slot"])):
                count(pos)
                assert pos[:3] not in whole, (c, w, pos)
                whole.add(pos[:3])
                pos = after(pos)
        r = plan.ranges[c]
        pos, end = tuple(r["start"].tolist()), tuple(r["end"].tolist())
        if pos < end:
            assert tuple(r["first"].tolist()) == want[pos[0]]
        while pos < end:
            n = count(pos)
            cut_end = pos[:3] == end[:3]
            k1 = min(end[3], n) if cut_end else n
            assert k1 > pos[3], (c, pos, end)
            if pos[3] == 0 and not cut_end:
                assert pos[:3] not in whole, (c, pos)
                whole.add(pos[:3])
            else:
                c0, c1 = (c, int(r["c1_last"])) if pos[3] == 0 else (int(r["c0"]), int(r["c1"]))
                pieces.setdefault(pos[:3], []).append((pos[3], k1, c, c0, c1))
            if cut_end:
                break
            pos = after(pos)
    for tile, parts in pieces.items():
        assert tile not in whole, tile
        c0, c1 = parts[0][3:]
        assert [p[2:] for p in parts] == [(c, c0, c1) for c in range(c0, c1 + 1)], (tile, parts)
        assert [p[0] for p in parts] == [0] + [p[1] for p in parts[:-1]] and parts[-1][1] == count((*tile, 0)), (tile, parts)
    assert len(whole) + len(pieces) == Hkv * sum(tiles_of)
    return int(h["waves"]), int(h["slot"]), len(whole), len(pieces), max((len(p) for p in pieces.values()), default=0)
