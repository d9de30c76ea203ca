"""The 8-bit paged cache as a server uses it: whole steps (xs_paged_step, plan, append, attention, read back), captured
and replayed, streams and workspaces, strides and layouts, what is refused or reported, and the ends of the ranges."""
import numpy as np
import pytest

import _paged as pg
import _paged8 as p8
from test_gpu_paged8_attn import _run

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def xs():
    from conftest import build_library
    build_library()
    import dit_attention_ulysses_gb300 as xs
    assert torch.cuda.is_available()
    return xs


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Server:
    """The buffers of a small server over an 8-bit cache, and its state in 64 bits on the host."""

    def __init__(self, xs, n, H, Hkv, D, page, block, n_pages, rows, seed, causal=True, window=0, dtype=torch.bfloat16):
        self.xs, self.n, self.H, self.Hkv, self.D, self.page, self.block, self.rows = xs, n, H, Hkv, D, page, block, rows
        self.dtype, self.causal, self.window, self.max_q, self.n_pages = dtype, causal, window, rows, n_pages
        self.r = np.random.default_rng(seed)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.table = torch.full((n, n_pages), -9, **i32)
        self.free = torch.randperm(n_pages).to(**i32)
        self.count, self.count_out = torch.tensor([n_pages], **i32), torch.empty(1, **i32)
        self.lens, self.new, self.kv = torch.zeros(n, **i32), torch.zeros(n, **i32), torch.zeros(n, **i32)
        self.cu, self.status = torch.zeros(n + 1, **i32), torch.zeros(n, **i32)
        self.positions, self.slots = torch.zeros(rows, **i32), torch.zeros(rows, dtype=torch.int64, device="cuda")
        t = dict(dtype=dtype, device="cuda")
        self.cache = [torch.full((n_pages, page, Hkv, D), p8.NAN_CODE, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
                      for _ in "kv"] + \
                     [torch.full((n_pages, page // block, Hkv), p8.NO_SCALE, dtype=torch.uint8, device="cuda") for _ in "kv"]
        self.qkv = torch.zeros((rows, H + 2 * Hkv, D), **t)
        self.q_rot, self.out = torch.zeros((rows, H, D), **t), torch.zeros((rows, H, D), **t)
        self.lse = torch.zeros((rows, H), dtype=torch.float32, device="cuda")
        self.back = [torch.zeros((n_pages * page, Hkv, D), **t) for _ in "kv"]
        self.ends = torch.zeros(n + 1, **i32)
        self.rope = xs.Rope(D)
        self.ws = xs.PagedWorkspace(n, H, Hkv, D)
        # V by the definition, in the cache's places; what was appended, by request
        self.num, self.exp = np.full((n_pages, page, Hkv, D), np.nan), np.full((n_pages, page // block, Hkv), 128.0)
        self.past = [np.zeros((0, H + 2 * Hkv, D)) for _ in range(n)]

    def launch(self):
        xs, H, Hkv = self.xs, self.H, self.Hkv
        xs.xs_paged_step(self.lens, self.new, self.table, self.free, self.count, self.page, self.kv, self.cu,
                         self.positions, self.slots, self.count_out, self.status)
        xs.xs_attn_paged8_plan(self.cu, self.kv, self.max_q, self.ws, causal=self.causal, window=self.window)
        q, k, v = self.qkv[:, :H], self.qkv[:, H:H + Hkv], self.qkv[:, H + Hkv:]
        xs.xs_rope_append_paged8(q, k, v, self.positions, self.slots, self.q_rot, *self.cache, self.rope)
        xs.xs_attn_paged8_fwd(self.q_rot, *self.cache, self.table, xs.XS_LAYOUT_CONTIGUOUS, [self.out],
                              self.D ** -0.5, self.ws, lse=self.lse)
        torch.cumsum(self.kv, 0, dtype=torch.int32, out=self.ends[1:])
        xs.xs_paged_read8(*self.cache, self.table, self.ends, None, *self.back)
        self.lens.copy_(self.kv)
        self.count.copy_(self.count_out)

    def step(self, new, launch):
        """One step with `new` tokens per request (-1: ended) through `launch`, checked in 64 bits."""
        rows = sum(max(a, 0) for a in new)
        H, Hkv, D = self.H, self.Hkv, self.D
        x = self.r.standard_normal((rows, H + 2 * Hkv, D))
        x[:, H + Hkv:] *= np.exp2(self.r.integers(-3, 4, size=(rows, 1, 1)))      # V's blocks grow
        x = torch.from_numpy(x).to(self.dtype)
        self.qkv[:rows] = x.cuda()
        self.new.copy_(torch.tensor(new, dtype=torch.int32))
        self.out.fill_(9.0)
        for b in self.back:
            b.fill_(7.0)
        launch()
        assert self.xs.xs_attn_get_device_error() == self.xs.XS_OK
        assert not self.status.any()
        x = x.double().numpy()
        p8.append_reference(self.num, self.exp, x[:, H + Hkv:], self.slots.cpu().numpy()[:rows], self.block)
        scales = self.cache[2].cpu().numpy().astype(float) - 127
        k_back, v_back = (b.double().cpu().numpy() for b in self.back)
        q_rot, out, lse = (t.double().cpu().numpy() for t in (self.q_rot, self.out, self.lse))
        table, u = self.table.cpu().numpy(), pg.U[self.dtype]
        row, at, theta = 0, 0, pg.frequencies(D)
        for i, a in enumerate(new):
            if a < 0:
                self.past[i] = self.past[i][:0]
                continue
            self.past[i] = np.concatenate([self.past[i], x[row:row + a]])
            y, c = self.past[i], len(self.past[i])
            t = np.arange(c)
            where = table[i, t // self.page] if c else t
            kd, vd = k_back[at:at + c], v_back[at:at + c]
            # V: the definition's bits
            e = self.exp[where, t % self.page // self.block]
            assert np.array_equal(vd, self.num[where, t % self.page] * np.exp2(e)[..., None])
            # K: half a step relative, and of the least numbers half a step at every scale that the block has had, a
            # sum below 2^-9 of the last; the rotation's own error is 2^-20 of a pair of channels
            turned, size = pg.rope_reference(y[:, :H + Hkv], t, theta, False)
            kt = turned[:, H:]
            ks = np.exp2(scales[where, t % self.page // self.block])[..., None] if c else kt
            # (in fp16 what is read back is rounded below 2^-14)
            assert (np.abs(kd - kt) <= 2.0 ** -4 * np.abs(kt) + 2.0 ** -9 * ks + 2.0 ** -18 * np.abs(y[:, H:H + Hkv]).max(initial=1) + 2.0 ** -25).all()
            vmax = 448 * np.exp2(e.max(initial=-64))
            for h in range(H if a else 0):
                g = h // (H // Hkv)
                ref, mass, z = pg.attention_reference(q_rot[row:row + a, h], kd[:, g], vd[:, g], c, self.causal, self.window,
                                                      D ** -0.5)
                before = (2.0 ** -11 + 1.5e-4) * mass + 2.0 ** -25 * c * vmax
                assert (np.abs(out[row:row + a, h] - ref) <= before + u * (np.abs(ref) + before)).all()
                assert (np.abs(lse[row:row + a, h] - z) <= 6e-5 + 2.0 ** -22 * np.abs(z)).all()
            row += a
            at += c
        assert (self.out[row:] == 9.0).all()
        assert all((b[at:] == 7.0).all() for b in self.back)


STEPS = [[40, 0, 7, 1], [1, 33, 1, 1], [1, 1, 1, 1], [-1, 1, 16, 1], [25, -1, 1, 1], [1, 1, 0, -1], [2, 5, 1, 50]]


@pytest.mark.parametrize("D,page,block,causal,window,dtype", [
    (128, 16, 16, True, 0, torch.bfloat16), (64, 32, 16, True, 9, torch.float16), (128, 64, 64, False, 0, torch.bfloat16),
    (64, 128, 32, True, 30, torch.bfloat16)])
def test_serving_steps(xs, D, page, block, causal, window, dtype):
    s = Server(xs, 4, 4, 2, D, page, block, 40, 100, seed=D + page, causal=causal, window=window, dtype=dtype)
    for new in STEPS:
        s.step(new, s.launch)


@pytest.mark.parametrize("max_q", [1, 100])
def test_serving_steps_in_a_graph(xs, max_q):
    """One captured step replayed with other lengths: nothing is baked into the launches."""
    s = Server(xs, 4, 8, 2, 128, 16, 16, 40, 100, seed=1)
    s.max_q = max_q
    s.launch()      # warm-up: every request idle
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        s.launch()
    for new in STEPS:
        s.step(new, graph.replay)
    for new in STEPS[::-1]:      # eager and replayed steps in turn
        s.step([a if a >= 0 else 0 for a in new], s.launch if sum(new) % 2 else graph.replay)


def test_readme_example(xs):
    """The README's steps over both caches run as printed, and the second's results are those of its elements."""
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "README.md")).read()
    blocks = [b for b in re.findall(r"```python\n(.*?)```", text, re.S) if "xs_paged_step" in b or "xs_attn_paged8_fwd" in b]
    assert len(blocks) == 2
    ns = dict(torch=torch, xs=xs)
    for b in blocks:
        exec(b, ns)
    assert xs.xs_attn_get_device_error() == xs.XS_OK
    n, H, Hkv, D = (ns[k] for k in ("n", "H", "Hkv", "D"))
    q8, kd, vd = (ns[k].double().cpu().numpy() for k in ("q8", "k_back", "v_back"))
    k, v = (ns[x].double().cpu().numpy()[:20 * n] for x in "kv")
    k, _ = pg.rope_reference(k, ns["positions"].cpu().numpy()[:20 * n], pg.frequencies(D), False)
    # half a step, and of the smallest numbers half a step of a scale that is at most 2^-7 of a magnitude below 8
    assert (np.abs(vd - v) <= 2.0 ** -4 * np.abs(v) + 2.0 ** -16).all()
    assert (np.abs(kd - k) <= 2.0 ** -4 * np.abs(k) + 2.0 ** -15).all()
    u = pg.U[torch.bfloat16]
    for i in (0, n - 1):
        rows = slice(20 * i, 20 * i + 20)
        for h in (0, H - 1):
            g = h // (H // Hkv)
            ref, mass, _ = pg.attention_reference(q8[rows, h], kd[rows, g], vd[rows, g], 20, True, 0, D ** -0.5)
            before = (2.0 ** -11 + 1.5e-4) * mass + 2.0 ** -25 * 20 * 448 * 2.0 ** -6
            assert (np.abs(ns["out8"][rows, h].double().cpu().numpy() - ref) <= before + u * (np.abs(ref) + before)).all()


def test_two_graphs_share_a_workspace(xs):
    """Captured plans and attentions replayed in turn, both kernels of this cache and one of the 16-bit cache."""
    cases = [p8.Paged8Case([1] * 6, [5000, 10, 900, 4000, 77, 1], 8, 2, 128, 16, seed=1),
             p8.Paged8Case([90, 0, 1, 40, 7, 200], [2500, 3, 1, 4000, 77, 230], 8, 2, 128, 32, seed=2),
             pg.PagedCase([1, 3, 1, 1, 2, 1], [2500, 3, 1, 4000, 77, 230], 8, 2, 128, 32, seed=3)]
    ws = xs.PagedWorkspace(6, 8, 2, 128)
    outs = [torch.empty((c.T, 8, 128), dtype=c.dtype, device="cuda") for c in cases]

    def launch(c, o):
        if isinstance(c, p8.Paged8Case):
            xs.xs_attn_paged8_plan(c.cu, c.kv, max(c.q_lens), ws)
            xs.xs_attn_paged8_fwd(c.q, *c.cache, c.table, xs.XS_LAYOUT_CONTIGUOUS, [o], 0.1, ws)
        else:
            xs.xs_attn_paged_plan(c.cu, c.kv, max(c.q_lens), ws)
            xs.xs_attn_paged_fwd(c.q, c.k, c.v, c.table, xs.XS_LAYOUT_CONTIGUOUS, [o], 0.1, ws)

    graphs = []
    for c, o in zip(cases, outs):
        launch(c, o)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            launch(c, o)
    for turn in range(3):
        for g, c, o in zip(graphs, cases, outs):
            o.fill_(float("nan"))
            g.replay()
            c.check(o, None, True, 0, 0.1)
    assert xs.xs_attn_get_device_error() == xs.XS_OK


def test_two_streams_with_their_own_workspaces(xs):
    cases = [p8.Paged8Case([q] * 5, [3000, 10, 900, 4000, 77], 8, 2, 128, 16, seed=i) for i, q in enumerate((1, 9))]
    streams = [torch.cuda.Stream() for _ in cases]
    ws = [xs.PagedWorkspace(c.n, c.H, c.Hkv, c.D) for c in cases]
    outs = [torch.empty((c.T, c.H, c.D), dtype=c.dtype, device="cuda") for c in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, w, o, st in zip(cases, ws, outs, streams):
            xs.xs_attn_paged8_plan(c.cu, c.kv, 9, w, stream=st)
            xs.xs_attn_paged8_fwd(c.q, *c.cache, c.table, xs.XS_LAYOUT_CONTIGUOUS, [o], 0.1, w, stream=st)
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        c.check(o, None, True, 0, 0.1)


def test_native_binding_and_python_checks_make_the_same_calls(xs, monkeypatch):
    """Steps through the binding and through the checks in Python: the same bits, and the same refusals."""
    xs._device()
    if xs._native is None:
        pytest.skip("the binding needs PyTorch's and Python's headers")
    seen = []

    class Spy:
        def __getattr__(self, name):
            def f(*args):
                seen.append((name, getattr(native, name)(*args)))
                return seen[-1][1]
            return f

    native, outs = xs._native, []
    side = torch.cuda.Stream()
    for binding in (Spy(), None):
        monkeypatch.setattr(xs, "_native", binding)
        s = Server(xs, 4, 8, 2, 128, 16, 16, 40, 100, seed=1)
        for new in STEPS:
            s.step(new, s.launch)
        c = p8.Paged8Case([90, 1, 7], [300, 200, 7], 8, 2, 128, 16, seed=2, q_pad=3, table_pad=2)
        ws, lse = xs.PagedWorkspace(3, 8, 2, 128), torch.empty((c.T, 8), device="cuda")
        shards = [torch.empty((c.T, 4, 128), dtype=c.dtype, device="cuda") for _ in range(2)]
        rows = [torch.zeros((20, 2, 128), dtype=c.dtype, device="cuda") for _ in range(4)]
        table, cu, first = c.table[:2], _i32([0, 3, 17]), _i32([5, 30])
        slots = torch.arange(16, 36, device="cuda")
        side.wait_stream(torch.cuda.current_stream())
        ks = [t.view(torch.float8_e8m0fnu) for t in (c.ks, c.vs)]      # either type of the scales
        xs.xs_attn_paged8_plan(c.cu, c.kv, 90, ws, stream=side)
        xs.xs_attn_paged8_fwd(c.q, c.k, c.v, *ks, c.table, xs.XS_LAYOUT_HEADS, shards, 0.1, ws, lse=lse, stream=side.cuda_stream)
        xs.xs_paged_read8(*c.cache, table, cu, first, rows[0], rows[1], stream=side)
        torch.cuda.synchronize()
        mine = [t.clone() for t in c.cache]
        xs.xs_rope_append_paged8(None, rows[0], rows[1], None, slots, None, *mine, None)
        xs.xs_rope_append_paged8(c.q[:20], c.q[:20, :2], c.q[:20, 2:4], slots.int(), slots, turned := torch.empty_like(c.q[:20]),
                                 *mine, xs.Rope(128, 64))
        outs.append([*shards, lse, turned, *rows, *(t.view(torch.uint8) for t in mine), s.out, *s.back])
        with pytest.raises(TypeError, match="contiguous"):
            xs.xs_attn_paged8_plan(torch.zeros(8, dtype=torch.int32, device="cuda")[::2], c.kv, 90, ws)
        with pytest.raises(TypeError, match="shapes do not match|shape"):
            xs.xs_attn_paged8_fwd(c.q, *c.cache, c.table, xs.XS_LAYOUT_HEADS, shards[:1], 0.1, ws)
        with pytest.raises(TypeError, match="current device"):
            xs.xs_attn_paged8_fwd(c.q, *c.cache, c.table.cpu(), xs.XS_LAYOUT_HEADS, shards, 0.1, ws)
        with pytest.raises(TypeError, match="k_scales"):
            xs.xs_attn_paged8_fwd(c.q, c.k, c.v, c.ks[:1], c.vs, c.table, xs.XS_LAYOUT_HEADS, shards, 0.1, ws)
        with pytest.raises(TypeError, match="v_scales"):
            xs.xs_paged_read8(c.k, c.v, c.ks, c.vs.float(), table, cu, first, rows[0], rows[1])
        with pytest.raises(TypeError, match="v_cache"):
            xs.xs_paged_read8(c.k, c.v.float(), c.ks, c.vs, table, cu, first, rows[0], rows[1])
        with pytest.raises(TypeError, match="shapes do not match|shape"):
            xs.xs_rope_append_paged8(c.q[:20], rows[0][:, :1], rows[1], slots.int(), slots, turned, *mine, xs.Rope(128))
        with pytest.raises(TypeError):
            xs.xs_rope_append_paged8(c.q[:20], rows[0], rows[1], slots.int(), slots.int(), turned, *mine, xs.Rope(128))
        with pytest.raises(TypeError, match="D|shape"):
            xs.xs_rope_append_paged8(c.q[:20], rows[0], rows[1], slots.int(), slots, turned, *mine, xs.Rope(64))
        with pytest.raises(TypeError, match="None"):
            xs.xs_rope_append_paged8(None, rows[0], rows[1], slots.int(), slots, None, *mine, None)
        with pytest.raises(xs.XsError) as e:
            xs.xs_attn_paged8_fwd(c.q, *c.cache, c.table, xs.XS_LAYOUT_HEADS, shards, -1.0, ws)
        assert e.value.code == xs.XS_ERR_SCALE
        with pytest.raises(xs.XsError) as e:
            xs.xs_rope_append_paged8(c.q[:20], rows[0], rows[1], slots.int(), slots, turned, mine[0], mine[0], *mine[2:], xs.Rope(128))
        assert e.value.code == xs.XS_ERR_OVERLAP
        with pytest.raises(ValueError, match="no plan"):
            xs.xs_attn_paged8_fwd(c.q, *c.cache, c.table, xs.XS_LAYOUT_HEADS, shards, 0.1, xs.PagedWorkspace(3, 8, 2, 128))
        k16 = torch.zeros(c.k.shape, dtype=c.dtype, device="cuda")
        with pytest.raises(ValueError, match="no plan"):       # a plan of the other cache
            xs.xs_attn_paged_fwd(c.q, k16, k16, c.table, xs.XS_LAYOUT_HEADS, shards, 0.1, ws)
        xs.xs_attn_paged_plan(c.cu, c.kv, 90, ws)
        with pytest.raises(ValueError, match="xs_attn_paged8_plan"):
            xs.xs_attn_paged8_fwd(c.q, *c.cache, c.table, xs.XS_LAYOUT_HEADS, shards, 0.1, ws)
    # (the servers' caches differ: their pages are handed out in random orders)
    assert [torch.equal(a, b) for a, b in zip(*outs)] == [True] * len(outs[0])
    taken = {name for name, code in seen if code == xs.XS_OK}
    assert taken == {"append8", "read8", "step", "plan", "plan8", "attn8"}


def test_plan_of_other_arguments_is_reported(xs):
    c = p8.Paged8Case([1, 1], [100, 50], 4, 2, 64, 16, seed=3)
    c16 = pg.PagedCase([1, 1], [100, 50], 4, 2, 64, 16, seed=3)
    ws = xs.PagedWorkspace(c.n, c.H, c.Hkv, c.D)
    out = torch.full((c.T, c.H, c.D), 5.0, dtype=c.dtype, device="cuda")
    call = lambda: xs.xs_attn_paged8_fwd(c.q, *c.cache, c.table, xs.XS_LAYOUT_CONTIGUOUS, [out], 0.1, ws)   # noqa: E731

    def reported():
        code, rec = xs.xs_attn_get_device_error_info()
        assert code == xs.XS_ERR_DEVICE_BOUNDS and rec["site"] == 3 and (out == 5.0).all()

    xs.xs_attn_paged8_plan(c.cu, c.kv, 1, ws)
    for planned in ((1, 0, 0), (1, 1, 9), (1000, 1, 0)):     # max_q, causal, window
        ws.planned = planned
        call()
        reported()
    for max_q in (1, 100):          # plans of one cache for the other, the workspace's note of it set aside
        xs.xs_attn_paged_plan(c.cu, c.kv, max_q, ws)
        ws.cache8 = True
        call()
        reported()
        xs.xs_attn_paged8_plan(c.cu, c.kv, max_q, ws)
        ws.cache8 = False
        xs.xs_attn_paged_fwd(c16.q, c16.k, c16.v, c16.table, xs.XS_LAYOUT_CONTIGUOUS, [out], 0.1, ws)
        reported()
    xs.xs_attn_paged8_plan(c.cu, c.kv, 1, ws)
    call()
    c.check(out, None, True, 0, 0.1)


@pytest.mark.parametrize("q", [1, 300])
def test_expired_wait_is_reported(xs, monkeypatch, q):
    """With a limit of 0 the first copy that has not landed when it is looked for ends the launch.  A cache of 0.8 GB,
    far more than L2, so that some has not; afterwards the context still works."""
    H, D, page, keys = 8, 128, 64, 400000
    n_pages = keys // page
    cache = [torch.zeros((n_pages, page, H, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in "kv"] + \
            [torch.full((n_pages, 1, H), 127, dtype=torch.uint8, device="cuda") for _ in "kv"]
    table = torch.arange(n_pages, dtype=torch.int32, device="cuda")[None]
    query, out = (torch.zeros((q, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = xs.PagedWorkspace(1, H, H, D)
    xs.xs_attn_paged8_plan(_i32([0, q]), _i32([keys]), q, ws)
    monkeypatch.setenv("XSATTN_WAIT_TIMEOUT_NS", "0")
    xs.xs_attn_paged8_fwd(query, *cache, table, xs.XS_LAYOUT_CONTIGUOUS, [out], 0.1, ws)
    code, rec = xs.xs_attn_get_device_error_info()
    assert code == xs.XS_ERR_DEVICE_TIMEOUT and rec["kind"] == 1
    monkeypatch.delenv("XSATTN_WAIT_TIMEOUT_NS")
    c = p8.Paged8Case([q], [3000], 4, 2, 128, 16, seed=3)
    out, lse = _run(xs, c)
    c.check(out, lse, True, 0, c.D ** -0.5)


@pytest.mark.parametrize("form", [dict(heads_first=True), dict(one_buffer=True), dict(q_pad=5), dict(table_pad=3),
                                  dict(heads_first=True, q_pad=2, table_pad=1)], ids=str)
@pytest.mark.parametrize("q", [1, 70])
def test_strides(xs, form, q):
    c = p8.Paged8Case([q, 2], [333, 200], 6, 2, 128, 32, seed=4, **form)
    out, lse = _run(xs, c)
    c.check(out, lse, True, 0, c.D ** -0.5)


@pytest.mark.parametrize("q", [[1, 1, 2], [60, 4, 100]], ids=["few", "chunk"])
def test_layouts_hold_the_same_bits(xs, q):
    P = 4
    c = p8.Paged8Case(q, [300, 17, 900], 8, 4, 64, 16, seed=1, extra_rows=-sum(q) % P)
    full, _ = _run(xs, c, fill=3.0)
    shards, _ = _run(xs, c, layout=xs.XS_LAYOUT_A2A, P=P, fill=3.0)
    heads, _ = _run(xs, c, layout=xs.XS_LAYOUT_HEADS, P=P, fill=3.0)
    assert torch.equal(torch.cat(shards), full) and torch.equal(torch.cat(heads, 1), full)


@pytest.mark.parametrize("max_q", [1, 3, 8, 5000])
def test_max_q_is_only_an_estimate(xs, max_q):
    c = p8.Paged8Case([5, 150, 1], [400, 300, 90], 4, 2, 128, 16, seed=9)
    out, lse = _run(xs, c, max_q=max_q)
    c.check(out, lse, True, 0, c.D ** -0.5)


@pytest.mark.parametrize("q", [1, 90])
@pytest.mark.parametrize("scale,gain", [(0.0, 1.0), (0.01, 1.0), (3.0, 0.125), (0.125 * 2.0 ** -80, 2.0 ** 40), (0.125 * 2.0 ** 30, 2.0 ** -15)])
def test_scales(xs, scale, gain, q):
    """0: the mean of the values.  3: one key takes nearly all, and maxima move often.  The last two: keys and queries far
    from 1, the scores as ever (q is scaled by the gain below)."""
    c = p8.Paged8Case([q], [500], 2, 1, 64, 16, seed=2, gain=gain)
    if gain not in (1.0, 0.125):
        c.q.mul_(gain)
        c.q64 = c.q64 * gain
    out, lse = _run(xs, c, scale=scale)
    c.check(out, lse, True, 0, scale)


@pytest.mark.parametrize("q", [1, 90])
@pytest.mark.parametrize("v_spread", [8, 20, 45])
def test_values_of_unlike_blocks(xs, q, v_spread):
    """V's blocks apart by factors of up to 2^90: what counts is the largest product (the bound has its scale), and the
    log-sum-exp counts every key alike."""
    c = p8.Paged8Case([q, 2], [700, 40], 4, 2, 128, 32, block=16, seed=v_spread, v_spread=v_spread)
    out, lse = _run(xs, c)
    ref, mass, z = c.reference(True, 0, c.D ** -0.5)
    tol = (2.0 ** -11 + 1.5e-4) * mass + 2.0 ** -25 * 700 * c.vmax + pg.U[c.dtype] * (np.abs(ref) + mass)
    assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()
    assert (np.abs(lse.double().cpu().numpy() - z) <= 6e-5 + 2.0 ** -22 * np.abs(z)).all()


@pytest.mark.parametrize("q", [1, 90])
def test_zeros(xs, q):
    """Rows of q that are zero, blocks of zeros with the least scale."""
    c = p8.Paged8Case([q], [300], 2, 1, 128, 16, seed=5)
    c.q[:, 1] = 0
    c.q64[:, 1] = 0
    for j in (0, 3, 18):
        e = c.table[0, j].long()
        c.k[e], c.v[e] = 0, 0
        c.ks.view(torch.uint8)[e], c.vs.view(torch.uint8)[e] = 63, 63
        c.keys[0][16 * j:16 * j + 16], c.values[0][16 * j:16 * j + 16] = 0, 0
    out, lse = _run(xs, c)
    c.check(out, lse, True, 0, c.D ** -0.5)


@pytest.mark.parametrize("q", [1, 40])
def test_rising_scores_move_the_maximum(xs, q):
    """Keys whose scores grow along the sequence: every block has a new maximum."""
    c = p8.Paged8Case([q], [2000], 2, 2, 128, 16, seed=6)
    up = p8.nearest(np.linspace(0, 1, 2000)[:, None, None] * np.ones((1, 2, 128)) * 0.6 * 256)
    c.keys[0] = up / 256
    for j in range(pg.ceil_div(2000, 16)):
        e = c.table[0, j].long()
        c.k.view(torch.uint8)[e] = p8.codes(up[16 * j:16 * j + 16]).cuda()
        c.ks.view(torch.uint8)[e] = 127 - 8
    c.q.copy_(torch.ones_like(c.q) * 4)
    c.q64 = c.q.double().cpu().numpy()
    out, lse = _run(xs, c, scale=0.2)
    # scores up to 64: sum |q_d k_d| scale = 64, so 128 * 2^-24 * 64 = 4.9e-4 bounds their error
    ref, mass, z = c.reference(True, 0, 0.2)
    tol = (pg.U[c.dtype] * (mass + np.abs(ref)) + 2.0 ** -11 * mass) * 1.01 + 1.2e-3 * mass + 2.0 ** -25 * 2000 * c.vmax
    assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()
    assert (np.abs(lse.double().cpu().numpy() - z) <= 5e-4 + 2.0 ** -22 * np.abs(z)).all()


def test_nan_rows_of_q_behind_the_last_sequence(xs):
    """Padding rows may hold anything."""
    for q in ([1, 1], [70, 30]):
        c = p8.Paged8Case(q, [300, 200], 6, 2, 128, 16, seed=6, extra_rows=40)
        c.q[sum(q):] = float("nan")
        out, lse = _run(xs, c)
        c.check(out, lse, True, 0, c.D ** -0.5)


def test_no_sequence_has_new_tokens(xs):
    for max_q in (1, 100):
        c = p8.Paged8Case([0, 0], [100, 0], 4, 2, 64, 16, seed=3)
        out, lse = _run(xs, c, max_q=max_q)
        assert out.isnan().all() and lse.isnan().all()


def test_lengths_that_are_not_the_caches(xs):
    """Nonsense on the device reads and writes nothing out of range; the next step is right."""
    c = p8.Paged8Case([2, 3], [60, 70], 4, 2, 64, 16, seed=1)
    ws = xs.PagedWorkspace(2, 4, 2, 64)
    guard = torch.full((c.T + 64, 4, 64), 5.0, dtype=c.dtype, device="cuda")
    for cu, kv in (([5, 1, 3], [60, 70]), ([-7, 3, 9], [-1, 5000]), ([0, 2, 4000], [60, 20]), ([100, 101, 102], [10, 10]),
                   ([0, 0, 0], [2 ** 20, 2 ** 20]), ([2, 5, 5], [0, 0])):
        for max_q in (1, 100):
            xs.xs_attn_paged8_plan(_i32(cu), _i32(kv), max_q, ws)
            xs.xs_attn_paged8_fwd(c.q, *c.cache, c.table, xs.XS_LAYOUT_CONTIGUOUS, [guard[32:32 + c.T]], 0.1, ws)
            xs.xs_attn_get_device_error()
            assert (guard[:32] == 5.0).all() and (guard[32 + c.T:] == 5.0).all()
    out, lse = _run(xs, c, ws=ws)
    c.check(out, lse, True, 0, c.D ** -0.5)


def test_pages_out_of_range_read_as_zeros(xs):
    """Bad page numbers and a table too narrow for the sequence read as zeros: no fault."""
    H, D, page = 2, 64, 16
    for q_len in (1, 50):
        c = p8.Paged8Case([q_len], [200], H, H, D, page, seed=3)
        bad = {2: -1, 5: c.k.shape[0], 7: 2 ** 31 - 1, 9: -2 ** 31}
        for j, e in bad.items():
            c.table[0, j] = e
            c.keys[0][j * page:(j + 1) * page] = 0
            c.values[0][j * page:(j + 1) * page] = 0
        c.table = c.table[:, :11].contiguous()     # 176 of 200 keys
        c.keys[0][176:], c.values[0][176:] = 0, 0
        out, lse = _run(xs, c)
        c.check(out, lse, True, 0, D ** -0.5)


@pytest.mark.parametrize("q", [1, 2, 6])
def test_long_split_is_repeatable(xs, q):
    """One sequence cut over many SMs; ten calls on one plan give the same bits, and a plan made anew does too."""
    c = p8.Paged8Case([q], [40000], 8, 2, 128, 64, 32, seed=8)
    ws = xs.PagedWorkspace(c.n, c.H, c.Hkv, c.D)
    out, lse = _run(xs, c, ws=ws)
    c.check(out, lse, True, 0, c.D ** -0.5)
    for _ in range(10):
        o, z = torch.full_like(out, float("nan")), torch.full_like(lse, float("nan"))
        xs.xs_attn_paged8_fwd(c.q, *c.cache, c.table, xs.XS_LAYOUT_CONTIGUOUS, [o], c.D ** -0.5, ws, lse=z)
        assert torch.equal(o, out) and torch.equal(z, lse)
    o, z = _run(xs, c, ws=ws)
    assert torch.equal(o, out) and torch.equal(z, lse)


@pytest.mark.parametrize("most", [1, 40], ids=["one", "up_to_40"])
def test_most_sequences(xs, most):
    """8192 sequences, the limit, some without new tokens; with two KV heads few tokens' tiles are of both."""
    r = np.random.default_rng(most)
    q = r.integers(0, most, size=8192, endpoint=True)
    kv = q + r.integers(0, 30, size=8192)
    c = p8.Paged8Case(q.tolist(), kv.tolist(), 2, 2 if most == 1 else 1, 64, 16, seed=most)
    out, lse = _run(xs, c)
    c.check(out, lse, True, 0, c.D ** -0.5)


@pytest.mark.parametrize("q", [1, 70])
def test_a_million_keys(xs, q):
    """2^20 keys of one head: Q = 0 weighs every key alike, so a row is the mean of what it sees."""
    D, page, keys = 64, 512, 1 << 20
    cache = [(torch.randn((keys // page, page, 1, D), device="cuda") * 64).clamp(-448, 448).to(torch.float8_e4m3fn) for _ in "kv"] + \
            [torch.full((keys // page, page // 128, 1), 127 - 6, dtype=torch.uint8, device="cuda") for _ in "kv"]
    table = torch.randperm(keys // page, device="cuda").int()[None]
    query = torch.zeros((q, 1, D), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty_like(query), torch.empty((q, 1), dtype=torch.float32, device="cuda")
    ws = xs.PagedWorkspace(1, 1, 1, D)
    xs.xs_attn_paged8_plan(_i32([0, q]), _i32([keys]), q, ws)
    xs.xs_attn_paged8_fwd(query, *cache, table, xs.XS_LAYOUT_CONTIGUOUS, [out], 0.1, ws, lse=lse)
    assert xs.xs_attn_get_device_error() == xs.XS_OK
    v = cache[1][table[0].long()].double().view(keys, D) / 64
    seen = torch.arange(keys - q + 1, keys + 1, device="cuda").double()
    ref = torch.cumsum(v, 0)[keys - q:] / seen[:, None]
    # every probability is the same power of two: a sum of 2^20 terms in fp32 over 2^20, in hundreds of separate runs
    # of at most a few thousand blocks' partial sums (each step 2^-24 of a partial sum below 5000)
    assert ((out[:, 0].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1e-5).all()
    assert ((lse[:, 0].double() - seen.log()).abs() <= 6e-5).all()


def test_offsets_past_32_bits(xs):
    """A cache of more than 2^32 bytes, the sequence's pages at its end: append, attention, read back."""
    H, Hkv, D, page, block = 2, 2, 128, 256, 64
    n_pages = 2 ** 32 // (page * Hkv * D) + 40
    big = [torch.empty((n_pages, page, Hkv, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in "kv"] + \
          [torch.empty((n_pages, page // block, Hkv), dtype=torch.uint8, device="cuda") for _ in "kv"]
    far = n_pages - 4 + torch.tensor([2, 0, 3, 1], device="cuda")
    for q_len, kv_len in ((1, 1000), (200, 1000)):
        c = p8.Paged8Case([q_len], [kv_len], H, Hkv, D, page, block, seed=q_len)
        used = c.table[0, :4].long()
        for b, s in zip(big, c.cache):
            b.view(torch.uint8)[far] = s.view(torch.uint8)[used]
        c.table[0, :4] = far.int()
        small, c.cache = c.cache, big
        out, lse = _run(xs, c)
        c.check(out, lse, True, 0, D ** -0.5)
        # the last 300 tokens once more, by appending their elements: no bit changes (their blocks begin in them)
        k, v = (torch.empty((kv_len, Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
        ends = _i32([0, kv_len])
        xs.xs_paged_read8(*big, c.table, ends, None, k, v)
        assert np.array_equal(k.double().cpu().numpy(), c.keys[0]) and np.array_equal(v.double().cpu().numpy(), c.values[0])
        t = torch.arange(640, kv_len, device="cuda")
        slots = c.table[0].long()[t // page] * page + t % page
        assert int(slots.max()) * Hkv * D > 2 ** 32
        for b in big:
            b.view(torch.uint8)[far[2:], 128 if b.dim() == 4 else 2:] = 99
        xs.xs_rope_append_paged8(None, k[640:], v[640:], None, slots, None, *big, None)
        k2, v2 = torch.empty_like(k), torch.empty_like(v)
        xs.xs_paged_read8(*big, c.table, ends, None, k2, v2)
        assert torch.equal(k2[640:], k[640:]) and torch.equal(v2[640:], v[640:]) and torch.equal(k2[:512], k[:512])


def test_rows_past_32_bits(xs):
    """Rows of k and of what is read back more than 2^32 bytes apart."""
    T, stride, D = 20000, 1 << 17, 64
    wide = torch.empty(T * stride, dtype=torch.bfloat16, device="cuda")
    k, v, k2, v2 = (wide.as_strided((T, 1, D), (stride, D, 1), i * 4096) for i in range(4))
    page, block = 128, 32
    for x in (k, v):
        x.copy_(torch.randn((T, 1, D), device="cuda").bfloat16())
    cache = [torch.empty((160, page, 1, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in "kv"] + \
            [torch.empty((160, page // block, 1), dtype=torch.uint8, device="cuda") for _ in "kv"]
    perm = torch.randperm(160, device="cuda")
    t = torch.arange(T, device="cuda")
    xs.xs_rope_append_paged8(None, k, v, None, perm[t // page] * page + t % page, None, *cache, None)
    xs.xs_paged_read8(*cache, perm.int()[None], _i32([0, T]), None, k2, v2)
    for a, b in ((k, k2), (v, v2)):
        x, y = a.double().cpu().numpy()[:, 0], b.double().cpu().numpy()[:, 0]
        e = p8.need(np.abs(x).reshape(T // block, -1).max(1)).repeat(block)[:, None]
        assert np.array_equal(y, p8.nearest(x * np.exp2(-e.astype(float))) * np.exp2(e.astype(float)))


@pytest.mark.parametrize("first,second", [(float("inf"), 1.0), (float("nan"), 1.0), (float("-inf"), float("nan"))])
def test_append_of_what_is_not_finite(xs, first, second):
    x = torch.ones((2, 1, 64), dtype=torch.bfloat16, device="cuda")
    x[0, 0, 3], x[1, 0, 5] = first, second
    cache = [torch.zeros((2, 16, 1, 64), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in "kv"] + \
            [torch.zeros((2, 1, 1), dtype=torch.uint8, device="cuda") for _ in "kv"]
    xs.xs_rope_append_paged8(None, x, x.clone(), None, torch.tensor([16, 17], device="cuda"), None, *cache, None)
    for code, scale in zip(cache[:2], cache[2:]):
        e = 120 if np.isinf(first) or np.isinf(second) else -8
        assert int(scale[1, 0, 0]) == 127 + e
        got = code[1, :2, 0].double().cpu().numpy() * 2.0 ** e
        for row, at, value in ((0, 3, first), (1, 5, second)):
            if np.isnan(value):
                assert np.isnan(got[row, at])
            elif np.isinf(value):
                assert got[row, at] == np.sign(value) * 448 * 2.0 ** 120
            else:
                assert got[row, at] == value * (e < 0)
        assert (got[0, 10:] == (e < 0)).all()


@pytest.mark.parametrize("T", [1, 300])
def test_append_rotates_q_in_place(xs, T):
    """q_out may be q, a slice of a fused projection: the same bits, k and v left alone."""
    H, Hkv, D, page, block = 6, 2, 128, 64, 32
    qkv = torch.randn((T, H + 2 * Hkv, D), device="cuda").bfloat16()
    slots, rope = torch.randperm(40, device="cuda")[torch.arange(T, device="cuda") // page] * page + \
        torch.arange(T, device="cuda") % page, xs.Rope(D)
    results = []
    for in_place in (False, True):
        x = qkv.clone()
        q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
        out = q if in_place else torch.empty((T, H, D), dtype=x.dtype, device="cuda")
        cache = [torch.zeros((40, page, Hkv, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in "kv"] + \
                [torch.zeros((40, page // block, Hkv), dtype=torch.uint8, device="cuda") for _ in "kv"]
        xs.xs_rope_append_paged8(q, k, v, torch.arange(T, device="cuda").int(), slots, out, *cache, rope)
        assert torch.equal(x[:, H:], qkv[:, H:])
        results.append([out.clone(), *(c.view(torch.uint8) for c in cache)])
    assert all(torch.equal(a, b) for a, b in zip(*results))
    out16 = torch.empty((T, H, D), dtype=qkv.dtype, device="cuda")
    xs.xs_rope_fwd(qkv[:, :H], torch.arange(T, device="cuda").int(), out16, rope)
    assert torch.equal(out16, results[0][0])


def test_two_streams_append_to_one_cache(xs):
    """Requests' appends on streams of their own, twenty steps of them, equal those one after the other."""
    Hkv, D, page, block, n = 4, 64, 32, 16, 3
    streams = [torch.cuda.Stream() for _ in range(n)]
    x = torch.randn((n, 20, 7, Hkv, D), device="cuda").bfloat16()
    results = []
    for side in (True, False):
        cache = [torch.zeros((n * 5, page, Hkv, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in "kv"] + \
                [torch.zeros((n * 5, page // block, Hkv), dtype=torch.uint8, device="cuda") for _ in "kv"]
        slots = [[(i * 5) * page + 7 * s + torch.arange(7, device="cuda") for s in range(20)] for i in range(n)]
        torch.cuda.synchronize()
        for s in range(20):
            for i in range(n):
                xs.xs_rope_append_paged8(None, x[i, s], x[i, s], None, slots[i][s], None, *cache, None,
                                         stream=streams[i] if side else None)
        torch.cuda.synchronize()
        results.append([c.view(torch.uint8) for c in cache])
    assert all(torch.equal(a, b) for a, b in zip(*results))
