"""Measured cases of the paged-cache operators: the step that lays out new tokens in a
paged cache, rotary positions, their fusion with the cache append, and the attention of
new tokens over the cache.

``run`` computes a pass either with this package's entry points (``own = True``) or in
plain torch operations (``own = False``, 32-bit arithmetic, 64-bit angles); ``exact`` is
the same result from the operators' definitions in 64 bits.
"""
import math
import random

import torch

own = False

LAYOUTS = {"half": 0, "interleaved": 1}
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
NEG = float("-inf")


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decoding step of a serving batch: 256 requests, one new token each
        dict(name="step decode 256", op="step", n=256, page=16, ctx=8192, new=1, lens_seed=1),
        # a large mixed step: prompts beside decoding and finished requests
        dict(name="step mixed 4096", op="step", n=4096, page=32, ctx=4096, new=64, lens_seed=2),
        # Q or K of the image model before its attention
        dict(name="rope image", op="rope", T=4608, H=24, D=128, rot=128, layout="half", scaled=False, grad=False,
             dtype="bf16", fused=False, far=4608),
        # the gradient of Q or K of the large video model
        dict(name="rope grad video", op="rope", T=75776, H=40, D=128, rot=128, layout="interleaved", scaled=False,
             grad=True, dtype="bf16", fused=False, far=75776),
        # a short odd prompt, half of each head rotated, far positions of a scaled context, rows of a fused projection
        dict(name="rope part scaled", op="rope", T=777, H=5, D=64, rot=32, layout="half", scaled=True, grad=False,
             dtype="fp16", fused=True, far=1 << 20),
        # one decoding step of 64 requests: rotate and append one token each
        dict(name="append decode 64", op="append", T=64, H=32, Hkv=8, D=128, rot=128, layout="half", page=16,
             pages=8192, pad=0, dtype="bf16", heads_first=False),
        # a chunk of a long prompt: rotate and append, pages stored head by head, the last rows padding
        dict(name="append chunk 8192", op="append", T=8192, H=32, Hkv=8, D=128, rot=128, layout="interleaved", page=64,
             pages=512, pad=100, dtype="bf16", heads_first=True),
        # a single user decoding: latency
        dict(name="attn decode 1", op="attn", n=1, q=1, ctx=4096, H=32, Hkv=8, D=128, page=16, even=True, causal=True,
             window=0, P=1, dtype="bf16", heads_first=False, lens_seed=3),
        # a ragged decoding batch: bandwidth
        dict(name="attn decode 64", op="attn", n=64, q=1, ctx=16384, H=32, Hkv=8, D=128, page=16, even=False,
             causal=True, window=0, P=1, dtype="bf16", heads_first=False, lens_seed=4),
        # two prompts in chunks over a long prefix: matrix products
        dict(name="attn chunk causal", op="attn", n=2, q=2048, ctx=14336, H=32, Hkv=8, D=128, page=64, even=True,
             causal=True, window=0, P=1, dtype="bf16", heads_first=True, lens_seed=5),
        # the next chunk of a video over the chunks before it, stored to 4 sequence shards
        dict(name="attn chunk video", op="attn", n=1, q=4608, ctx=13824, H=24, Hkv=24, D=128, page=128, even=True,
             causal=False, window=0, P=4, dtype="bf16", heads_first=False, lens_seed=6),
        # prompts and decoding requests in one ragged batch, attention within a window
        dict(name="attn mixed window", op="attn", n=24, q=512, ctx=6000, H=12, Hkv=6, D=64, page=32, even=False,
             causal=True, window=1000, P=1, dtype="fp16", heads_first=False, lens_seed=7),
    ]


def _log(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(["step", "rope", "append", "attn", "attn"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    D = rng.choice([64, 128])
    rot = rng.choice([D, D, D // 2, 16, 48])
    layout = rng.choice(["half", "interleaved"])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    if op == "step":
        return dict(op=op, n=_log(rng, 1, 4096), page=rng.choice([16, 32, 64, 128]), ctx=_log(rng, 16, 8192),
                    new=rng.choice([1, _log(rng, 1, 64)]), lens_seed=rng.randrange(1 << 20))
    if op == "rope":
        T, H = _log(rng, 1, 75776), rng.choice([1, 3, 8, 24, 40])
        return dict(op=op, T=T, H=H, D=D, rot=rot, layout=layout, scaled=rng.random() < 0.5, grad=rng.random() < 0.5,
                    dtype=dtype, fused=rng.random() < 0.3, far=_log(rng, T, 1 << 20))
    if op == "append":
        page, T = rng.choice([16, 32, 64, 128]), _log(rng, 1, 8192)
        return dict(op=op, T=T, H=Hkv * rng.choice([1, 2, 4, 7]), Hkv=Hkv, D=D, rot=rot, layout=layout, page=page,
                    pages=2 * (T // page) + 8, pad=rng.choice([0, T // 5]), dtype=dtype,
                    heads_first=rng.random() < 0.5)
    while True:
        even = rng.random() < 0.3
        P = rng.choice([1, 1, 1, 2])
        H = Hkv * rng.choice([1, 2, 4, 5, 8])
        causal = rng.random() < 0.7
        case = dict(op=op, n=_log(rng, 1, 64), q=rng.choice([1, 1, _log(rng, 2, 2048)]), ctx=_log(rng, 1, 32768), H=H,
                    Hkv=Hkv, D=D, page=rng.choice([16, 32, 64, 128]), even=even, causal=causal,
                    window=_log(rng, 1, 4096) if causal and rng.random() < 0.3 else 0, P=P, dtype=dtype,
                    heads_first=rng.random() < 0.5, lens_seed=rng.randrange(1 << 20))
        q_lens, kv_lens = _attn_lens(case)
        scores = case["n"] * H * max(q_lens) * max(kv_lens)
        pairs = sum(a * b for a, b in zip(q_lens, kv_lens)) * H
        if scores <= 1 << 31 and pairs <= 1 << 31 and sum(kv_lens) * Hkv <= 1 << 23 and H % P == 0:
            return case


def _step_lens(case):
    """Cached and new tokens of each request; -1 new tokens: the request has ended."""
    r = random.Random(case["lens_seed"])
    cached = [r.randint(0, case["ctx"]) for _ in range(case["n"])]
    new = [r.randint(1, case["new"]) for _ in cached]
    if case["n"] > 16:
        for i in range(0, case["n"], 16):
            new[i] = -1 if i % 32 else 0
    return cached, new


def _attn_lens(case):
    r = random.Random(case["lens_seed"])
    if case["even"]:
        return [case["q"]] * case["n"], [case["ctx"] + case["q"]] * case["n"]
    q = [case["q"]] + [_log(r, 1, case["q"]) for _ in range(case["n"] - 1)]
    ctx = [case["ctx"]] + [_log(r, 1, case["ctx"]) for _ in range(case["n"] - 1)]
    return q, [a + b for a, b in zip(q, ctx)]


def _attn_rows(case):
    """Rows of the query tensor: the new tokens, padded to the number of shards."""
    rows = sum(_attn_lens(case)[0])
    return -(-rows // case["P"]) * case["P"]


# ----------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(shape, dtype, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _cache(pages, page, Hkv, D, dtype, heads_first, g):
    """A cache of logical shape [pages, page, Hkv, D]."""
    if heads_first:
        return _randn((pages, Hkv, page, D), dtype, g).transpose(1, 2)
    return _randn((pages, page, Hkv, D), dtype, g)


ROPE_SCALED = dict(base=500000.0, factor=8.0, context=8192, low=1.0, high=32.0, magnitude=1.2)


def _rope_args(case):
    return dict(ROPE_SCALED) if case.get("scaled") else dict(base=10000.0)


def _rope_handle(case):
    import dit_attention_ulysses_gb300 as xs
    kw = _rope_args(case)
    if case.get("scaled"):
        kw["scaling"] = xs.XS_ROPE_BY_PARTS
    return xs.Rope(case["D"], case["rot"], layout=LAYOUTS[case["layout"]], **kw)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    if case["op"] == "step":
        cached, new = _step_lens(case)
        page = case["page"]
        held = [-(-c // page) for c in cached]
        width = -(-(case["ctx"] + case["new"]) // page)
        used = sum(held)
        spare = sum(-(-(c + max(a, 0)) // page) - h for c, a, h in zip(cached, new, held))
        spare = max(1, spare - spare // 8)   # the last requests find the list empty unless ended ones give pages back
        pages = used + spare
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        # columns past a request's pages hold what an earlier request left there
        table = torch.randint(0, pages, (case["n"], width), generator=g, device="cuda", dtype=torch.int32)
        held_t = _ints(held)
        first = torch.cumsum(held_t, 0) - held_t
        col = torch.arange(width, device="cuda")
        mine = col[None, :] < held_t[:, None]
        table = torch.where(mine, order[(first[:, None] + col[None, :]).clamp(max=pages - 1)], table)
        free = torch.zeros(pages, dtype=torch.int32, device="cuda")
        free[:spare] = order[used:]
        rows = sum(max(a, 0) for a in new) + 7   # a captured step has room for more tokens than this one brings
        s.update(cache_lens=_ints(cached), new_lens=_ints(new), table=table.contiguous(), free=free,
                 free_count=_ints([spare]), kv_lens=torch.empty(case["n"], dtype=torch.int32, device="cuda"),
                 cu_q=torch.empty(case["n"] + 1, dtype=torch.int32, device="cuda"),
                 positions=torch.empty(rows, dtype=torch.int32, device="cuda"),
                 slots=torch.empty(rows, dtype=torch.int64, device="cuda"),
                 free_count_out=torch.empty(1, dtype=torch.int32, device="cuda"),
                 status=torch.empty(case["n"], dtype=torch.int32, device="cuda"))
        return s
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "rope":
        T, H, D = case["T"], case["H"], case["D"]
        width = 3 * H if case["fused"] else H
        s["x"] = _randn((T, width, D), dtype, g)[:, :H]
        s["positions"] = torch.randint(0, case["far"], (T,), generator=g, device="cuda", dtype=torch.int32)
        s["out"] = torch.empty((T, H, D), dtype=dtype, device="cuda")
    elif case["op"] == "append":
        T, H, Hkv, D = case["T"], case["H"], case["Hkv"], case["D"]
        qkv = _randn((T, H + 2 * Hkv, D), dtype, g)   # one projection's rows
        s["q"], s["k"], s["v"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        s["positions"] = torch.randint(0, 1 << 17, (T,), generator=g, device="cuda", dtype=torch.int32)
        slots = torch.randperm(case["pages"] * case["page"], generator=g, device="cuda")[:T].clone()
        slots[T - case["pad"]:] = -1
        s["slots"] = slots
        s["q_out"] = torch.empty((T, H, D), dtype=dtype, device="cuda")
        for name in ("k_cache", "v_cache"):
            s[name] = _cache(case["pages"], case["page"], Hkv, D, dtype, case["heads_first"], g)
    else:
        q_lens, kv_lens = _attn_lens(case)
        H, Hkv, D, page = case["H"], case["Hkv"], case["D"], case["page"]
        T = _attn_rows(case)
        held = [-(-c // page) for c in kv_lens]
        pages = sum(held) + 3
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        held_t = _ints(held)
        first = torch.cumsum(held_t, 0) - held_t
        col = torch.arange(max(held), device="cuda")
        s["table"] = order[(first[:, None] + col[None, :]).clamp(max=pages - 1)].contiguous()
        s["q"] = _randn((T, H, D), dtype, g)
        for name in ("k_cache", "v_cache"):
            s[name] = _cache(pages, page, Hkv, D, dtype, case["heads_first"], g)
        cu = [0]
        for a in q_lens:
            cu.append(cu[-1] + a)
        s["cu_q"], s["kv_lens"] = _ints(cu), _ints(kv_lens)
        P = case["P"]
        s["outs"] = [torch.zeros((T // P, H, D), dtype=dtype, device="cuda") for _ in range(P)]
        s["lse"] = torch.zeros((T, H), dtype=torch.float32, device="cuda")
        s["max_q"], s["max_kv"] = max(q_lens), max(kv_lens)
    if own:
        # what a serving loop keeps: the frequencies of the model, and the plan of the step, which all its layers share
        if case["op"] == "attn":
            import dit_attention_ulysses_gb300 as xs
            s["ws"] = xs.PagedWorkspace(case["n"], case["H"], case["Hkv"], case["D"])
            xs.xs_attn_paged_plan(s["cu_q"], s["kv_lens"], s["max_q"], s["ws"], causal=case["causal"],
                                  window=case["window"])
        else:
            s["rope"] = _rope_handle(case)
    return s


# -------------------------------------------------------------------------------- run
def run(s):
    op = s["case"]["op"]
    if own:
        return {"step": _step_own, "rope": _rope_own, "append": _append_own, "attn": _attn_own}[op](s)
    return {"step": _step_plain, "rope": _rope_plain, "append": _append_plain, "attn": _attn_plain}[op](s)


def _step_own(s):
    import dit_attention_ulysses_gb300 as xs
    xs.xs_paged_step(s["cache_lens"], s["new_lens"], s["table"], s["free"], s["free_count"], s["case"]["page"],
                     s["kv_lens"], s["cu_q"], s["positions"], s["slots"], s["free_count_out"], s["status"])
    return [s[k] for k in ("table", "free", "kv_lens", "cu_q", "positions", "slots", "free_count_out", "status")]


def _rope_own(s):
    import dit_attention_ulysses_gb300 as xs
    xs.xs_rope_fwd(s["x"], s["positions"], s["out"], s["rope"], grad=s["case"]["grad"])
    return s["out"]


def _append_own(s):
    import dit_attention_ulysses_gb300 as xs
    xs.xs_rope_append_paged(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["q_out"], s["k_cache"],
                            s["v_cache"], s["rope"])
    return [s["q_out"], s["k_cache"], s["v_cache"]]


def _attn_own(s):
    import dit_attention_ulysses_gb300 as xs
    case = s["case"]
    layout = xs.XS_LAYOUT_A2A if case["P"] > 1 else xs.XS_LAYOUT_CONTIGUOUS
    xs.xs_attn_paged_fwd(s["q"], s["k_cache"], s["v_cache"], s["table"], layout, s["outs"], case["D"] ** -0.5,
                         s["ws"], lse=s["lse"])
    return [s["outs"], s["lse"]]


# ------------------------------------------------------------------------- plain forms
def _step_plain(s):
    page, table, free = s["case"]["page"], s["table"], s["free"]
    c, a = s["cache_lens"].long(), s["new_lens"].long()
    pages, rows, width = free.numel(), s["positions"].numel(), table.shape[1]
    ceil = lambda x: torch.div(x + page - 1, page, rounding_mode="floor")  # noqa: E731
    held = ceil(c.clamp(min=0))
    ended = (a < 0) & (c >= 0) & (held <= width)
    new = a.clamp(min=0)
    need = ceil(c.clamp(min=0) + new) - held
    status = torch.where((c < 0) | (held + need > width), 2, 0)
    tokens = torch.where((status == 0) & ~ended, new, 0)
    status = torch.where((status == 0) & (tokens > 0) & (torch.cumsum(tokens, 0) > rows), 3, status)
    gives = torch.where(ended, held, 0)
    gives_to = torch.cumsum(gives, 0)
    count = s["free_count"].long().clamp(0, pages)[0]
    avail = (count + gives_to[-1]).clamp(max=pages)
    # the free list with the ended requests' pages behind it
    at = torch.arange(pages, device=free.device)
    r = (at - count).clamp(min=0)
    giver = torch.searchsorted(gives_to, r, right=True).clamp(max=c.numel() - 1)
    given = table[giver, (r - (gives_to - gives)[giver]).clamp(0, width - 1)]
    back = (at >= count) & (at < avail)
    free.copy_(torch.where(back, given, free))
    need = torch.where((status == 0) & ~ended, need, 0)
    need_to = torch.cumsum(need, 0)
    status = torch.where((need > 0) & (need_to > avail), 1, status)
    need = torch.where(status == 0, need, 0)
    taken = torch.where(need > 0, need_to, 0).max()
    tokens = torch.where((status == 0) & ~ended, new, 0)
    # new pages from the end of the list, request by request
    col = torch.arange(width, device=free.device)[None, :]
    fresh = (col >= held[:, None]) & (col < (held + need)[:, None])
    k = (need_to - need)[:, None] + col - held[:, None]
    table.copy_(torch.where(fresh, free[(avail - 1 - k).clamp(0, pages - 1)], table))
    cu = torch.cumsum(tokens, 0)
    t = torch.arange(rows, device=free.device)
    i = torch.searchsorted(cu, t, right=True).clamp(max=c.numel() - 1)
    live = t < cu[-1]
    pos = torch.where(live, c[i] + t - (cu - tokens)[i], 0)
    entry = table[i, torch.div(pos, page, rounding_mode="floor")].long()
    good = live & (entry >= 0) & (entry < pages)
    slot = torch.where(good, entry * page + pos % page, -1)
    zero = torch.zeros(1, dtype=torch.int64, device=free.device)
    kv = torch.where(ended, 0, c.clamp(min=0) + tokens)
    return [table, free, kv.int(), torch.cat([zero, cu]).int(), pos.int(), slot, (avail - taken).int().view(1),
            status.int()]


def _frequencies(case, device):
    """Angle per position of each rotated pair, and the factor on cos and sin, in 64 bits."""
    kw, rot = _rope_args(case), case["rot"]
    theta = kw["base"] ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    if not case.get("scaled"):
        return theta, 1.0
    turns = theta * kw["context"] / (2 * math.pi)
    keep = ((turns - kw["low"]) / (kw["high"] - kw["low"])).clamp(0, 1)
    return theta * keep + theta / kw["factor"] * (1 - keep), kw["magnitude"]


def _rotate(x, positions, case, grad=False):
    rot = case["rot"]
    theta, magnitude = _frequencies(case, x.device)
    angle = positions.double()[:, None] * theta
    cos, sin = ((magnitude * f(angle)).float()[:, None, :] for f in (torch.cos, torch.sin))
    sin = -sin if grad else sin
    y = x.float()
    if case["layout"] == "half":
        a, b = y[..., : rot // 2], y[..., rot // 2: rot]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([turned, y[..., rot:]], -1).to(x.dtype)


def _rope_plain(s):
    return _rotate(s["x"], s["positions"], s["case"], s["case"]["grad"])


def _append_plain(s):
    case, slots = s["case"], s["slots"]
    page = case["page"]
    k = _rotate(s["k"], s["positions"], case)
    # rows of padding write the first row's token once more to its own place
    real = slots >= 0
    to = torch.where(real, slots, slots[0])
    at, off = torch.div(to, page, rounding_mode="floor"), to % page
    for cache, x in ((s["k_cache"], k), (s["v_cache"], s["v"])):
        cache[at, off] = torch.where(real[:, None, None], x, x[:1])
    return [_rotate(s["q"], s["positions"], case), s["k_cache"], s["v_cache"]]


def _attn_plain(s):
    case = s["case"]
    H, Hkv, D, page, P = case["H"], case["Hkv"], case["D"], case["page"], case["P"]
    n, G, T = case["n"], H // Hkv, s["q"].shape[0]
    cu, kv = s["cu_q"].long(), s["kv_lens"].long()
    nq, nk = s["max_q"], s["max_kv"]
    dev = cu.device
    j, t = torch.arange(nq, device=dev), torch.arange(nk, device=dev)
    rows = (cu[:-1, None] + j).clamp(max=T - 1)
    q = s["q"][rows].float().view(n, nq, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(n, Hkv, G * nq, D)
    held = t[None, :] < kv[:, None]
    entry = s["table"].long()[:, torch.div(t, page, rounding_mode="floor")]
    k, v = (torch.where(held[:, :, None, None], c[entry, t % page].float(), 0).transpose(1, 2)
            for c in (s["k_cache"], s["v_cache"]))
    x = torch.matmul(q * D ** -0.5, k.transpose(2, 3)).view(n, Hkv, G, nq, nk)
    pos = (kv - (cu[1:] - cu[:-1]))[:, None] + j     # position of each query row
    seen = held[:, None, :].expand(n, nq, nk)
    if case["causal"]:
        seen = seen & (t <= pos[:, :, None])
    if case["window"]:
        seen = seen & (t > pos[:, :, None] - case["window"])
    x = x.masked_fill_(~seen[:, None, None], NEG)
    m = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(m == NEG, 0, m)).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(n, Hkv, G * nq, nk), v).view(n, Hkv, G, nq, D) / torch.where(total == 0, 1, total)
    lse = (m + total.log()).squeeze(-1)
    # back to packed rows; rows behind the last sequence stay as they were
    r = torch.arange(T, device=dev)
    i = torch.searchsorted(cu, r, right=True).clamp(1, n) - 1
    jj = (r - cu[i]).clamp(max=nq - 1)
    live = r < cu[-1]
    o = o.permute(0, 3, 1, 2, 4).reshape(n, nq, H, D)[i, jj].to(s["q"].dtype)
    lse = lse.permute(0, 3, 1, 2).reshape(n, nq, H)[i, jj]
    o = torch.where(live[:, None, None], o, torch.cat(s["outs"]))
    return [list(o.chunk(P)), torch.where(live[:, None], lse, s["lse"])]


# ------------------------------------------------------------------- 64-bit definitions
def exact(case, seed):
    if case["op"] == "step":
        return None
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _turn(s["x"], s["positions"], case, -1 if case["grad"] else 1)
    if case["op"] == "append":
        caches = [s["k_cache"].double(), s["v_cache"].double()]
        rows = torch.nonzero(s["slots"] >= 0)[:, 0]
        at = s["slots"][rows]
        for c, x in zip(caches, (_turn(s["k"], s["positions"], case, 1), s["v"].double())):
            c[at // case["page"], at % case["page"]] = x[rows]
        return [_turn(s["q"], s["positions"], case, 1)] + caches
    q_lens, kv_lens = _attn_lens(case)
    H, Hkv, D, page, P = case["H"], case["Hkv"], case["D"], case["page"], case["P"]
    G = H // Hkv
    out, lse = torch.cat(s["outs"]).double(), s["lse"].double()
    row = 0
    for i, (nq, nk) in enumerate(zip(q_lens, kv_lens)):
        t = torch.arange(nk, device="cuda")
        at, off = s["table"][i, t // page].long(), t % page
        p = torch.arange(nk - nq, nk, device="cuda")[:, None]
        hidden = torch.zeros((nq, nk), dtype=torch.bool, device="cuda")
        if case["causal"]:
            hidden |= t > p
        if case["window"]:
            hidden |= t <= p - case["window"]
        for h in range(H):
            key, value = (c[at, off, h // G].double() for c in (s["k_cache"], s["v_cache"]))
            x = s["q"][row:row + nq, h].double() @ key.T / math.sqrt(D)
            x[hidden] = NEG
            z = torch.logsumexp(x, 1)
            out[row:row + nq, h] = torch.exp(x - z[:, None]) @ value
            lse[row:row + nq, h] = z
        row += nq
    return [list(out.chunk(P)), lse]


def _turn(x, positions, case, sign):
    """Rotation as a complex product."""
    rot, kw = case["rot"], _rope_args(case)
    pairs = []
    for i in range(rot // 2):
        f = math.exp(-2 * i / rot * math.log(kw["base"]))
        if case.get("scaled"):
            ramp = (f * kw["context"] / (2 * math.pi) - kw["low"]) / (kw["high"] - kw["low"])
            ramp = min(1.0, max(0.0, ramp))
            f = f * (ramp + (1 - ramp) / kw["factor"])
        pairs.append(f)
    angle = positions.double()[:, None, None] * torch.tensor(pairs, dtype=torch.float64, device=x.device)
    z = torch.polar(torch.full_like(angle, kw.get("magnitude", 1.0)), sign * angle)
    y = x.double().clone()
    lo, hi = (slice(0, rot // 2), slice(rot // 2, rot)) if case["layout"] == "half" else (slice(0, rot, 2),
                                                                                        slice(1, rot, 2))
    w = torch.complex(y[..., lo].contiguous(), y[..., hi].contiguous()) * z
    y[..., lo], y[..., hi] = w.real, w.imag
    return y


# ------------------------------------------------------------------------------- work
def work(case):
    if case["op"] == "step":
        cached, new = _step_lens(case)
        page = case["page"]
        rows = sum(max(a, 0) for a in new)
        touched = sum(-(-(c + a) // page) - c // page for c, a in zip(cached, new) if a > 0)   # pages tokens fall in
        given = sum(-(-c // page) for c, a in zip(cached, new) if a < 0)
        return dict(bytes=20 * case["n"] + 12 * (rows + 7) + 8 * touched + 8 * given, flops=0)
    if case["op"] == "rope":
        T, H, D = case["T"], case["H"], case["D"]
        return dict(bytes=4 * T * H * D + 4 * T, flops=3 * T * H * case["rot"])
    if case["op"] == "append":
        T, H, Hkv, D = case["T"], case["H"], case["Hkv"], case["D"]
        real = T - case["pad"]
        return dict(bytes=4 * T * H * D + 8 * real * Hkv * D + 12 * T, flops=3 * (T * H + real * Hkv) * case["rot"])
    q_lens, kv_lens = _attn_lens(case)
    H, Hkv, D, w = case["H"], case["Hkv"], case["D"], case["window"]
    pairs = keys = 0
    for nq, nk in zip(q_lens, kv_lens):
        keys += min(nk, nq + w - 1) if w else nk
        if not case["causal"]:
            pairs += nq * nk
        elif not w:
            pairs += nq * nk - nq * (nq - 1) // 2
        else:
            pairs += sum(min(p + 1, w) for p in range(nk - nq, nk))
    rows = sum(q_lens)
    return dict(bytes=4 * rows * H * D + 4 * rows * H + 4 * keys * Hkv * D, flops=4 * H * D * pairs)
