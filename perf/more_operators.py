"""Measured cases of the 8-bit paged cache: rotary positions fused with an append that
quantises K and V, the cache read back, and the attention of new tokens over it.

A cache holds e4m3 numbers, and for every block of tokens and head a scale, a power of two
(e8m0); an element stands for its number times its block's scale.

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
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
LARGEST = 448.0        # of e4m3
LEAST_SCALE = -64      # exponent of the smallest scale that is written
NEG = float("-inf")


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decoding step of 64 requests: rotate, quantise and append one token each, most of them into a begun block
        dict(name="append decode 64", op="append", n=64, new=1, ctx=2000, even=False, H=32, Hkv=8, D=128, rot=128,
             layout="half", page=16, block=16, pad=0, dtype="bf16", heads_first=False, lens_seed=1),
        # a step with prompts beside decoding requests: odd lengths, small heads, half of each rotated, larger blocks
        dict(name="append mixed", op="append", n=24, new=300, ctx=700, even=False, H=12, Hkv=6, D=64, rot=32,
             layout="half", page=128, block=64, pad=9, dtype="fp16", heads_first=False, lens_seed=2),
        # a chunk of two long prompts, pages stored head by head, the last rows padding
        dict(name="append chunk 8192", op="append", n=2, new=4096, ctx=4096, even=True, H=32, Hkv=8, D=128, rot=128,
             layout="interleaved", page=64, block=32, pad=100, dtype="bf16", heads_first=True, lens_seed=3),
        # a long prompt's keys and values read back in 16 bits
        dict(name="read prompt 32768", op="read", n=1, rows=32768, start=0, even=True, Hkv=8, D=128, page=64, block=16,
             pad=0, dtype="bf16", heads_first=False, lens_seed=4),
        # the newest tokens of ragged requests
        dict(name="read ragged", op="read", n=24, rows=500, start=3000, even=False, Hkv=6, D=64, page=32, block=32,
             pad=5, dtype="fp16", heads_first=True, lens_seed=5),
        # a single user decoding: latency
        dict(name="attn decode 1", op="attn", n=1, q=1, ctx=4096, H=32, Hkv=8, D=128, page=16, block=16, even=True,
             causal=True, window=0, P=1, dtype="bf16", heads_first=False, lens_seed=6),
        # a ragged decoding batch: bandwidth
        dict(name="attn decode 64", op="attn", n=64, q=1, ctx=16384, H=32, Hkv=8, D=128, page=16, block=16, even=False,
             causal=True, window=0, P=1, dtype="bf16", heads_first=False, lens_seed=7),
        # a few drafted tokens for each of 16 requests
        dict(name="attn drafts 16", op="attn", n=16, q=6, ctx=5000, H=32, Hkv=8, D=128, page=32, block=32, even=False,
             causal=True, window=0, P=1, dtype="fp16", heads_first=True, lens_seed=8),
        # two prompts in chunks over a long prefix: matrix products
        dict(name="attn chunk causal", op="attn", n=2, q=2048, ctx=14336, H=32, Hkv=8, D=128, page=64, block=32,
             even=True, causal=True, window=0, P=1, dtype="bf16", heads_first=True, lens_seed=9),
        # the next chunk of a video over the chunks before it, stored to 4 sequence shards
        dict(name="attn chunk video", op="attn", n=1, q=4608, ctx=13824, H=24, Hkv=24, D=128, page=128, block=128,
             even=True, causal=False, window=0, P=4, dtype="bf16", heads_first=False, lens_seed=10),
        # prompts and decoding requests in one ragged batch, attention within a window
        dict(name="attn mixed window", op="attn", n=24, q=512, ctx=6000, H=12, Hkv=6, D=64, page=32, block=16,
             even=False, causal=True, window=1000, P=1, dtype="fp16", heads_first=False, lens_seed=11),
    ]


def _log(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(["append", "read", "attn", "attn"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    common = dict(op=op, Hkv=Hkv, D=D, page=page, block=rng.choice([b for b in (16, 32, 64, 128) if b <= page]),
                  dtype=rng.choice(["bf16", "bf16", "fp16"]), heads_first=rng.random() < 0.5,
                  even=rng.random() < 0.3, lens_seed=rng.randrange(1 << 20))
    if op == "append":
        new = rng.choice([1, _log(rng, 1, 4096)])
        n = _log(rng, 1, 256 if new == 1 else max(1, 8192 // new))
        return dict(common, n=n, new=new, ctx=_log(rng, 1, 4096), H=Hkv * rng.choice([1, 2, 4, 7]),
                    rot=rng.choice([D, D, D // 2, 16, 48]), layout=rng.choice(["half", "interleaved"]),
                    pad=rng.choice([0, _log(rng, 1, 64)]))
    if op == "read":
        rows = _log(rng, 1, 32768)
        return dict(common, n=_log(rng, 1, max(1, 32768 // rows)), rows=rows, start=rng.choice([0, _log(rng, 1, 8192)]),
                    pad=rng.choice([0, _log(rng, 1, 64)]))
    while True:
        P = rng.choice([1, 1, 1, 2])
        causal = rng.random() < 0.7
        case = dict(common, n=_log(rng, 1, 64), q=rng.choice([1, 1, _log(rng, 2, 2048)]), ctx=_log(rng, 1, 32768),
                    H=Hkv * rng.choice([1, 2, 4, 5, 8]), causal=causal,
                    window=_log(rng, 1, 4096) if causal and rng.random() < 0.3 else 0, P=P)
        q_lens, kv_lens = _attn_lens(case)
        scores = case["n"] * case["H"] * max(q_lens) * max(kv_lens)
        pairs = sum(a * b for a, b in zip(q_lens, kv_lens)) * case["H"]
        if scores <= 1 << 31 and pairs <= 1 << 31 and sum(kv_lens) * Hkv <= 1 << 23 and case["H"] % P == 0:
            return case


def _ragged(case, most, least=1):
    """A length for each request, the first one the largest."""
    if case["even"]:
        return [most] * case["n"]
    r = random.Random("%s %d" % (case["lens_seed"], most))
    return [most] + [_log(r, least, most) for _ in range(case["n"] - 1)]


def _attn_lens(case):
    q = _ragged(case, case["q"])
    return q, [a + b for a, b in zip(q, _ragged(case, case["ctx"]))]


def _append_lens(case):
    """New tokens and cached tokens of each request."""
    return _ragged(case, case["new"]), [c - 1 for c in _ragged(case, case["ctx"])]


def _read_lens(case):
    """Rows that are read of each request, and the position of the first."""
    rows = _ragged(case, case["rows"])
    return rows, [c - 1 for c in _ragged(case, case["start"] + 1)]


# ----------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(shape, dtype, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _starts(lens):
    cu = [0]
    for a in lens:
        cu.append(cu[-1] + a)
    return cu


def _cache(case, pages, g):
    """e4m3 numbers [pages, page, Hkv, D] and e8m0 scales [pages, page / block, Hkv]: elements of about 1, which
    differ by channel and by block."""
    page, Hkv, D, blocks = case["page"], case["Hkv"], case["D"], case["page"] // case["block"]
    lead, scale_lead = ((pages, Hkv, page), (pages, Hkv, blocks)) if case["heads_first"] else ((pages, page, Hkv),
                                                                                              (pages, blocks, Hkv))
    width = torch.exp(0.4 * torch.randn(D, generator=g, device="cuda"))
    x = (torch.randn((*lead, D), generator=g, device="cuda") * (64.0 * width)).clamp(-LARGEST, LARGEST).to(E4M3)
    e = torch.randint(-8, -4, scale_lead, generator=g, device="cuda")
    scales = (e + 127).to(torch.uint8).view(E8M0)
    return (x.transpose(1, 2), scales.transpose(1, 2)) if case["heads_first"] else (x, scales)


def _table(kv_lens, page, spare, g):
    """Pages of every request in any order, and how many there are."""
    held = [-(-c // page) for c in kv_lens]
    pages = sum(held) + spare
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    held_t = _ints(held)
    first = torch.cumsum(held_t, 0) - held_t
    col = torch.arange(max(held), device="cuda")
    return order[(first[:, None] + col[None, :]).clamp(max=pages - 1)].contiguous(), pages


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    dtype, page, Hkv, D = DTYPES[case["dtype"]], case["page"], case["Hkv"], case["D"]
    if case["op"] == "append":
        new, cached = _append_lens(case)
        H, kv_lens = case["H"], [a + b for a, b in zip(new, cached)]
        table, pages = _table(kv_lens, page, 2, g)
        T = sum(new) + case["pad"]
        qkv = _randn((T, H + 2 * Hkv, D), dtype, g)   # one projection's rows
        s["q"], s["k"], s["v"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        cu, cached_t = _ints(_starts(new)), _ints(cached)
        t = torch.arange(T, device="cuda")
        i = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=case["n"] - 1)
        pos = cached_t[i] + t - cu[i]
        live = t < cu[-1]
        pos = torch.where(live, pos, 0)
        slots = table[i, pos // page].long() * page + pos % page
        s["slots"], s["positions"] = torch.where(live, slots, -1), pos.int()
        s["q_out"] = torch.empty((T, H, D), dtype=dtype, device="cuda")
    elif case["op"] == "read":
        rows, start = _read_lens(case)
        s["table"], pages = _table([a + b for a, b in zip(rows, start)], page, 2, g)
        s["cu_rows"], s["first"] = _ints(_starts(rows)), _ints(start)
        T = sum(rows) + case["pad"]
        s["k_out"], s["v_out"] = (torch.zeros((T, Hkv, D), dtype=dtype, device="cuda") for _ in range(2))
    else:
        q_lens, kv_lens = _attn_lens(case)
        H, P = case["H"], case["P"]
        T = -(-sum(q_lens) // P) * P   # the new tokens, padded to the number of shards
        s["table"], pages = _table(kv_lens, page, 3, g)
        s["q"] = _randn((T, H, D), dtype, g)
        s["cu_q"], s["kv_lens"] = _ints(_starts(q_lens)), _ints(kv_lens)
        s["outs"] = [torch.zeros((T // P, H, D), dtype=dtype, device="cuda") for _ in range(P)]
        s["lse"] = torch.zeros((T, H), dtype=torch.float32, device="cuda")
        s["max_q"], s["max_kv"] = max(q_lens), max(kv_lens)
    s["k_cache"], s["k_scales"] = _cache(case, pages, g)
    s["v_cache"], s["v_scales"] = _cache(case, pages, g)
    if own:
        # what a serving loop keeps: the frequencies of the model, and the plan of the step, which all its layers share
        import dit_attention_ulysses_gb300 as xs
        if case["op"] == "attn":
            s["ws"] = xs.PagedWorkspace(case["n"], case["H"], Hkv, D)
            xs.xs_attn_paged8_plan(s["cu_q"], s["kv_lens"], s["max_q"], s["ws"], causal=case["causal"],
                                   window=case["window"])
        elif case["op"] == "append":
            s["rope"] = xs.Rope(D, case["rot"], layout=LAYOUTS[case["layout"]], base=10000.0)
    return s


# -------------------------------------------------------------------------------- run
def run(s):
    op = s["case"]["op"]
    if own:
        return {"append": _append_own, "read": _read_own, "attn": _attn_own}[op](s)
    return {"append": _append_plain, "read": _read_plain, "attn": _attn_plain}[op](s)


def _append_own(s):
    import dit_attention_ulysses_gb300 as xs
    xs.xs_rope_append_paged8(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["q_out"], s["k_cache"],
                             s["v_cache"], s["k_scales"], s["v_scales"], s["rope"])
    return [s["q_out"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"]]


def _read_own(s):
    import dit_attention_ulysses_gb300 as xs
    xs.xs_paged_read8(s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["table"], s["cu_rows"], s["first"],
                      s["k_out"], s["v_out"])
    return [s["k_out"], s["v_out"]]


def _attn_own(s):
    import dit_attention_ulysses_gb300 as xs
    case = s["case"]
    layout = xs.XS_LAYOUT_A2A if case["P"] > 1 else xs.XS_LAYOUT_CONTIGUOUS
    xs.xs_attn_paged8_fwd(s["q"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["table"], layout,
                          s["outs"], case["D"] ** -0.5, s["ws"], lse=s["lse"])
    return [s["outs"], s["lse"]]


# ------------------------------------------------------------------------- plain forms
def _rotated(x, positions, case):
    """In 32 bits; the angles in 64."""
    rot = case["rot"]
    theta = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=x.device) / rot)
    angle = positions.double()[:, None] * theta
    cos, sin = (f(angle).float()[:, None, :] for f in (torch.cos, torch.sin))
    y = x.float()
    if case["layout"] == "half":
        a, b = y[..., : rot // 2], y[..., rot // 2: rot]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([turned, y[..., rot:]], -1)


def _append_one(cache, scales, x, slots, block):
    """x [T, Hkv, D] in 32 bits into the slots of an 8-bit cache."""
    pages, page, Hkv, D = cache.shape
    n_blocks = pages * page // block
    at, off = torch.div(slots, block, rounding_mode="floor"), slots % block
    # the first token that a block gets; the ones before it stay
    first = torch.full((n_blocks,), block, device=x.device).scatter_reduce(0, at, off, "amin")
    largest = torch.zeros((n_blocks, Hkv), device=x.device).scatter_reduce(
        0, at[:, None].expand(-1, Hkv), x.abs().amax(-1), "amax")
    m, e = torch.frexp(largest)   # the smallest power of two whose 448-fold holds the largest
    need = torch.where(largest > 0, e - 9 + (m > 0.875), LEAST_SCALE).clamp(min=LEAST_SCALE)
    old = scales.view(torch.uint8).reshape(n_blocks, Hkv).int() - 127
    begun, touched = (first > 0)[:, None], (first < block)[:, None]
    e = torch.where(touched, torch.where(begun, torch.maximum(old, need), need), old)
    codes = cache.reshape(n_blocks, block, Hkv, D)
    held = torch.arange(block, device=x.device)[None, :] < first[:, None]
    again = (codes.float() * torch.exp2((old - e).float())[:, None, :, None]).to(E4M3)
    codes = torch.where((held & touched)[:, :, None, None], again.view(torch.uint8), codes.view(torch.uint8))
    codes[at, off] = (x * torch.exp2(-e[at].float())[:, :, None]).to(E4M3).view(torch.uint8)
    cache.view(torch.uint8).copy_(codes.view(pages, page, Hkv, D))
    scales.view(torch.uint8).copy_((e + 127).to(torch.uint8).view(scales.shape))


def _append_plain(s):
    case, slots = s["case"], s["slots"]
    # rows of padding write the first row's token once more to its own place
    row = torch.where(slots >= 0, torch.arange(slots.numel(), device=slots.device), 0)
    k, v = _rotated(s["k"], s["positions"], case)[row], s["v"].float()[row]
    _append_one(s["k_cache"], s["k_scales"], k, slots[row], case["block"])
    _append_one(s["v_cache"], s["v_scales"], v, slots[row], case["block"])
    q = _rotated(s["q"], s["positions"], case).to(s["q"].dtype)
    return [q, s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"]]


def _values(cache, scales, entry, off, block):
    """Elements of tokens `off` of pages `entry`, in 32 bits."""
    x = cache.view(torch.uint8)[entry, off].view(E4M3).float()
    e = scales.view(torch.uint8)[entry, torch.div(off, block, rounding_mode="floor")].float() - 127
    return x * torch.exp2(e)[..., None]


def _read_plain(s):
    case, cu = s["case"], s["cu_rows"].long()
    page = case["page"]
    r = torch.arange(s["k_out"].shape[0], device=cu.device)
    i = (torch.searchsorted(cu, r, right=True) - 1).clamp(max=case["n"] - 1)
    live = r < cu[-1]
    pos = torch.where(live, s["first"].long()[i] + r - cu[i], 0)
    entry = s["table"].long()[i, torch.div(pos, page, rounding_mode="floor")]
    most = torch.finfo(s["k_out"].dtype).max
    return [torch.where(live[:, None, None], _values(s[c], s[z], entry, pos % page, case["block"])
                        .clamp(-most, most).to(s[o].dtype), s[o])
            for c, z, o in (("k_cache", "k_scales", "k_out"), ("v_cache", "v_scales", "v_out"))]


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
    off = (t % page).expand(n, nk)
    k, v = (torch.where(held[:, :, None, None], _values(s[c], s[z], entry, off, case["block"]), 0).transpose(1, 2)
            for c, z in (("k_cache", "k_scales"), ("v_cache", "v_scales")))
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
def _numbers(cache):
    return cache.to(torch.float32).double()


def _nearest(y):
    """The nearest e4m3 numbers, ties to even: four significant bits, steps of 2^-9 below 2^-6."""
    step = torch.exp2((torch.frexp(y)[1] - 1).clamp(min=-6).double() - 3)
    return torch.round(y / step) * step


def _turn(x, positions, case):
    """Rotation as a complex product."""
    rot = case["rot"]
    theta = torch.tensor([math.exp(-2 * i / rot * math.log(10000.0)) for i in range(rot // 2)], dtype=torch.float64,
                         device=x.device)
    angle = positions.double()[:, None, None] * theta
    z = torch.polar(torch.ones_like(angle), angle)
    y = x.double().clone()
    lo, hi = (slice(0, rot // 2), slice(rot // 2, rot)) if case["layout"] == "half" else (slice(0, rot, 2),
                                                                                        slice(1, rot, 2))
    w = torch.complex(y[..., lo].contiguous(), y[..., hi].contiguous()) * z
    y[..., lo], y[..., hi] = w.real, w.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    caches = [(_numbers(s[c + "_cache"]), _numbers(s[c + "_scales"])) for c in "kv"]
    return {"append": _append_exact, "read": _read_exact, "attn": _attn_exact}[case["op"]](s, case, caches)


def _append_exact(s, case, caches):
    page, block = case["page"], case["block"]
    slots = s["slots"].tolist()
    runs, t = [], 0   # rows of one block, one after the other
    while t < len(slots):
        end = t + 1
        while end < len(slots) and slots[t] >= 0 and slots[end] == slots[end - 1] + 1 and slots[end] % block:
            end += 1
        if slots[t] >= 0:
            runs.append((t, end, slots[t]))
        t = end
    for (c, scale), x in zip(caches, (_turn(s["k"], s["positions"], case), s["v"].double())):
        largest = x.abs().amax(-1).cpu()
        for t0, t1, slot in runs:
            at, off = divmod(slot, page)
            b, before = off // block, off % block
            need = []
            for a in largest[t0:t1].amax(0).tolist():
                m, e = math.frexp(a)
                need.append(max(LEAST_SCALE, e - 8 if m > 0.875 else e - 9) if a else LEAST_SCALE)
            need = torch.exp2(torch.tensor(need, dtype=torch.float64, device=c.device))
            if before:
                need = torch.maximum(need, scale[at, b])
                tokens = slice(off - before, off)
                c[at, tokens] = _nearest(c[at, tokens] * (scale[at, b] / need)[:, None])
            scale[at, b] = need
            c[at, off:off + t1 - t0] = _nearest(x[t0:t1] / need[:, None])
    return [_turn(s["q"], s["positions"], case), caches[0][0], caches[1][0], caches[0][1], caches[1][1]]


def _read_exact(s, case, caches):
    page, block = case["page"], case["block"]
    outs = [s["k_out"].double(), s["v_out"].double()]
    row = 0
    for i, (count, start) in enumerate(zip(*_read_lens(case))):
        p = torch.arange(start, start + count, device="cuda")
        at, off = s["table"][i, p // page].long(), p % page
        for out, (c, scale) in zip(outs, caches):
            out[row:row + count] = c[at, off] * scale[at, off // block].unsqueeze(-1)
        row += count
    return outs


def _attn_exact(s, case, caches):
    q_lens, kv_lens = _attn_lens(case)
    H, Hkv, D, page, block, P = case["H"], case["Hkv"], case["D"], case["page"], case["block"], case["P"]
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
            key, value = (c[at, off, h // G] * scale[at, off // block, h // G][:, None] for c, scale in caches)
            x = s["q"][row:row + nq, h].double() @ key.T / math.sqrt(D)
            x[hidden] = NEG
            z = torch.logsumexp(x, 1)
            out[row:row + nq, h] = torch.exp(x - z[:, None]) @ value
            lse[row:row + nq, h] = z
        row += nq
    return [list(out.chunk(P)), lse]


# ------------------------------------------------------------------------------- work
def work(case):
    Hkv, D, block = case["Hkv"], case["D"], case["block"]
    if case["op"] == "append":
        new, cached = _append_lens(case)
        T, real, H = sum(new) + case["pad"], sum(new), case["H"]
        blocks = sum(-(-(c + a) // block) - c // block for a, c in zip(new, cached))
        # q in and out; k and v in 16 bits in, in 8 bits out; the scales of the blocks that get tokens
        return dict(bytes=4 * T * H * D + 6 * real * Hkv * D + 2 * blocks * Hkv + 12 * T,
                    flops=3 * (T * H + real * Hkv) * case["rot"] + 2 * real * Hkv * D)
    if case["op"] == "read":
        rows, start = _read_lens(case)
        blocks = sum(-(-(c + a) // block) - c // block for a, c in zip(rows, start))
        return dict(bytes=6 * sum(rows) * Hkv * D + 2 * blocks * Hkv, flops=2 * sum(rows) * Hkv * D)
    q_lens, kv_lens = _attn_lens(case)
    H, w = case["H"], case["window"]
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
    return dict(bytes=4 * rows * H * D + 4 * rows * H + 2 * keys * Hkv * D + 2 * keys * Hkv // block,
                flops=4 * H * D * pairs)
