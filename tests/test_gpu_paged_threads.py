"""Serving threads of one process: plans and steps of unlike batches at the same time, each
thread with its own stream, workspace and buffers.  Both calls let go of the interpreter's lock,
so that what a call sets for a whole kernel another thread's call sees."""
import threading

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def xs():
    from conftest import build_library
    build_library()
    import dit_attention_ulysses_gb300 as xs
    assert torch.cuda.is_available()
    return xs


def _together(*loops):
    """Every loop in a thread of its own, all from the same moment; the first exception of each is returned."""
    start, faults = threading.Barrier(len(loops)), []

    def run(loop):
        try:
            start.wait()
            loop()
        except Exception as e:      # noqa: BLE001 (the test reports it)
            faults.append(repr(e))

    threads = [threading.Thread(target=run, args=(x,)) for x in loops]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return faults


def _plans(xs, n, max_q, turns):
    cu = torch.arange(n + 1, dtype=torch.int32, device="cuda") * 2
    kv = torch.full((n,), 5, dtype=torch.int32, device="cuda")
    ws, stream = xs.PagedWorkspace(n, 8, 2, 64), torch.cuda.Stream()
    q = torch.randn((2 * n, 8, 64), device="cuda").bfloat16()
    k, v = (torch.randn((n, 16, 2, 64), device="cuda").bfloat16() for _ in "kv")
    table = torch.arange(n, dtype=torch.int32, device="cuda")[:, None]
    torch.cuda.synchronize()

    def attend(out):
        xs.xs_attn_paged_fwd(q, k, v, table, xs.XS_LAYOUT_CONTIGUOUS, [out], 0.125, ws, stream=stream)

    def loop():
        for _ in range(turns):
            xs.xs_attn_paged_plan(cu, kv, max_q, ws, stream=stream)
        attend(got)

    got, want = torch.empty_like(q), torch.empty_like(q)
    xs.xs_attn_paged_plan(cu, kv, max_q, ws, stream=stream)
    attend(want)
    torch.cuda.synchronize()
    return loop, lambda: torch.equal(got, want)


@pytest.mark.parametrize("sizes", [(8192, 1), (4096, 300), (8192, 2000, 7)], ids=str)
@pytest.mark.parametrize("max_q", [1, 300], ids=["few", "chunk"])
def test_plans_of_unlike_batches(xs, sizes, max_q):
    plans = [_plans(xs, n, max_q, 1500) for n in sizes]
    assert _together(*(loop for loop, _ in plans)) == []
    assert all(same() for _, same in plans)
    assert xs.xs_attn_get_device_error() == xs.XS_OK


def _steps(xs, n, turns):
    i32 = dict(dtype=torch.int32, device="cuda")
    cached, new = torch.full((n,), 20, **i32), torch.full((n,), 3, **i32)
    table = torch.arange(n, **i32)[:, None] * 2 + torch.arange(2, **i32)
    free, count = torch.zeros(2 * n, **i32), torch.zeros(1, **i32)
    stream = torch.cuda.Stream()
    outs = [torch.full((k,), -7, **i32) for k in (n, n + 1, 3 * n)] + [torch.full((3 * n,), -7, dtype=torch.int64, device="cuda"),
                                                                     torch.full((1,), -7, **i32), torch.full((n,), -7, **i32)]
    torch.cuda.synchronize()

    def loop():
        for _ in range(turns):
            xs.xs_paged_step(cached, new, table, free, count, 16, *outs, stream=stream)

    def same():
        kv, cu, pos, slots, left, status = outs
        t = torch.arange(3 * n, device="cuda")
        return (bool((kv == 23).all()) and torch.equal(cu, torch.arange(n + 1, **i32) * 3) and
                torch.equal(pos, (20 + t % 3).int()) and torch.equal(slots, (t // 3 * 2 + 1) * 16 + 4 + t % 3) and
                int(left) == 0 and not status.any())

    return loop, same


@pytest.mark.parametrize("sizes", [(4096, 2600), (8192, 4200), (8192, 4500, 5000)], ids=str)
def test_steps_of_unlike_batches(xs, sizes):
    steps = [_steps(xs, n, 1500) for n in sizes]
    assert _together(*(loop for loop, _ in steps)) == []
    assert all(same() for _, same in steps)


def test_plans_and_steps_of_unlike_batches(xs):
    work = [_plans(xs, 8192, 300, 500), _plans(xs, 3, 300, 500), _steps(xs, 8192, 500), _steps(xs, 4200, 500)]
    assert _together(*(loop for loop, _ in work)) == []
    assert all(same() for _, same in work)
    assert xs.xs_attn_get_device_error() == xs.XS_OK
