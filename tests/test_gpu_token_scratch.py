"""GPU: the token operators' scratch. What a captured graph uses is its own for as long as it lives, and so is a stream's."""

import gc

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import newton_schulz_momentum_gb300 as dm
    return dm


def step_inputs(n, rows, dim, seed=0):
    """One of each operator that needs scratch."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    return dict(dy=randn(n, dim), h=randn(n, dim), gain=randn(dim), rows=rows,
                ids=torch.randint(0, rows, (n,), generator=g, device="cuda"),
                targets=torch.randint(0, dim, (n,), generator=g, device="cuda"),
                lp=-1.0 - torch.rand(n, generator=g, device="cuda"), adv=randn(n),
                w=torch.rand(n, generator=g, device="cuda") / n)


def step(dm, s):
    dx, dgain = dm.add_rmsnorm_grad(s["dy"], s["h"], s["gain"])
    grad = dm.embedding_grad(dx, s["ids"], s["rows"])
    return (dx, dgain, grad, *dm.policy_loss(s["h"], s["targets"], s["lp"], s["adv"], s["w"]))


def captured(dm, s):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(dm, s)
    return graph, held


def replayed(graph, held):
    for t in held:
        t.fill_(-7.0)
    graph.replay()
    torch.cuda.synchronize()
    return held


def equal(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_replays_survive_larger_calls_and_the_release(dm):
    """A capture as the library's first call, then calls that need more scratch, and the release of all of it, between
    the replays; memory that any of these gave back would be the fill's."""
    dm.release_workspace()
    small, large = step_inputs(700, 300, 520), step_inputs(40000, 5000, 1032, 1)
    graph, held = captured(dm, small)
    want = [t.clone() for t in step(dm, small)]
    assert equal(replayed(graph, held), want)
    big = [t.clone() for t in step(dm, large)]
    assert equal(replayed(graph, held), want)
    dm.release_workspace()
    fill = [torch.full((1 << 20,), 3.0, device="cuda") for _ in range(64)]
    assert equal(replayed(graph, held), want) and all(float(t.min()) == 3.0 for t in fill)
    assert equal(step(dm, large), big) and equal(replayed(graph, held), want)
    dm.check_status()


def test_graphs_do_not_share(dm):
    """Two graphs replayed side by side on two streams, and a call beside them."""
    a, b, c = (step_inputs(5000, 3000, 1032, k) for k in range(3))
    ga, ha = captured(dm, a)
    gb, hb = captured(dm, b)
    wa, wb, wc = ([t.clone() for t in step(dm, s)] for s in (a, b, c))
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(one):
            ga.replay()
        with torch.cuda.stream(two):
            gb.replay()
        got = step(dm, c)
        torch.cuda.synchronize()
        assert equal(ha, wa) and equal(hb, wb) and equal(got, wc)
    dm.check_status()


def test_streams_do_not_share(dm):
    """Calls that overlap on three streams, with scratch that grows on the way, give what they give one by one, and
    leave nothing behind for the calls that follow."""
    sizes = [(5000, 3000, 1032), (70, 50, 128256), (900, 200, 264)]
    some = [step_inputs(*size, seed=k) for k, size in enumerate(sizes)]
    more = step_inputs(30000, 3000, 1032, 7)
    want, big = [[t.clone() for t in step(dm, s)] for s in some], [t.clone() for t in step(dm, more)]
    streams = [torch.cuda.Stream() for _ in some]
    torch.cuda.synchronize()
    for turn in range(30):
        got = []
        for s, stream in zip(some, streams):
            with torch.cuda.stream(stream):
                got.append(step(dm, s))
        if turn == 15:
            with torch.cuda.stream(streams[2]):
                large = step(dm, more)
        torch.cuda.synchronize()
        assert all(equal(a, b) for a, b in zip(got, want))
    assert equal(large, big)
    for s, w in zip(some, want):
        assert equal(step(dm, s), w)
    dm.check_status()


def test_more_streams_than_have_scratch_at_a_time(dm):
    """Streams of the caller's own making (torch hands out the same few again and again)."""
    import ctypes
    rt = ctypes.CDLL("libcudart.so.13")
    s = step_inputs(600, 300, 136)
    want = [t.clone() for t in step(dm, s)]
    torch.cuda.synchronize()
    for _ in range(70):
        handle = ctypes.c_void_p()
        assert rt.cudaStreamCreateWithFlags(ctypes.byref(handle), 1) == 0
        with torch.cuda.stream(torch.cuda.ExternalStream(handle.value)):
            got = step(dm, s)
        assert rt.cudaStreamSynchronize(handle) == 0 and equal(got, want)
        assert rt.cudaStreamDestroy(handle) == 0
    dm.check_status()


def test_scratch_goes_with_its_graph(dm):
    """Graph after graph, each dropped: 5 MB of scratch each, over 300 MB in all if none came back."""
    s = step_inputs(20000, 100, 1032)
    grad = dm.embedding_grad(s["dy"], s["ids"], 100)
    left = []
    for _ in range(60):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            dm.embedding_grad(s["dy"], s["ids"], 100, grad=grad)
        graph.replay()
        torch.cuda.synchronize()
        del graph
        gc.collect()
        torch.cuda.empty_cache()
        left.append(torch.cuda.mem_get_info()[0])
    assert left[2] - left[-1] < 100 << 20, [v >> 20 for v in left]


@pytest.mark.parametrize("n,dim,dt,least", [(4096, 16384, torch.bfloat16, 10), (3000, 16384, torch.float32, 10),
                                            (4096, 65536, torch.bfloat16, 9), (65536, 128, torch.float32, 1)])
def test_norm_gradient_asks_for_what_it_uses(dm, n, dim, dt, least):
    """A row of gain sums per CTA that runs (152 of the longest rows', 64 KB each), or 32 of rows that no CTA holds: under a
    limit of `least` MB and a fifth, what is given without one."""
    g = torch.Generator(device="cuda").manual_seed(dim)
    dy, h = (torch.randn(n, dim, generator=g, device="cuda").to(dt) for _ in range(2))
    gain = torch.randn(dim, generator=g, device="cuda")
    want = dm.add_rmsnorm_grad(dy, h, gain)
    torch.cuda.synchronize()
    dm.release_workspace()
    dm.set_workspace_limit(int(1.2e6 * least))
    try:
        got = dm.add_rmsnorm_grad(dy, h, gain)
        assert equal(got, want)
        dm.set_workspace_limit(1)  # without a gain no scratch at all
        alone = dm.add_rmsnorm_grad(dy, h)[0]
    finally:
        dm.set_workspace_limit(0)
    assert torch.equal(alone, dm.add_rmsnorm_grad(dy, h, torch.ones_like(gain))[0])
    dm.check_status()


@pytest.mark.parametrize("where", ["same thread", "another thread"])
def test_calls_beside_a_capture(dm, where):
    """Calls that run at once on another stream while a stream is captured, with scratch that grows and scratch that is
    there: neither they nor the capture fails."""
    import threading
    small, large = step_inputs(700, 300, 520), step_inputs(20000, 900, 1032, 1)
    want, big = [t.clone() for t in step(dm, small)], [t.clone() for t in step(dm, large)]
    side, errors = torch.cuda.Stream(), []
    with torch.cuda.stream(side):
        step(dm, small)
    outs = [[torch.empty_like(t) for t in w] for w in (want, big, want)]
    torch.cuda.synchronize()
    dm.release_workspace()
    with torch.cuda.stream(side):
        dm.embedding_grad(small["dy"], small["ids"], 300)  # scratch for the small calls
    torch.cuda.synchronize()

    def beside():
        try:
            with torch.cuda.stream(side):
                for s, out in zip((small, large, small), outs):
                    dm.add_rmsnorm_grad(s["dy"], s["h"], s["gain"], dx=out[0], dgain=out[1])
                    dm.embedding_grad(out[0], s["ids"], s["rows"], grad=out[2])
        except Exception as e:  # noqa: BLE001 - whatever it is, it is reported
            errors.append(e)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(dm, small)
        if where == "same thread":
            beside()
        else:
            thread = threading.Thread(target=beside)
            thread.start()
            thread.join()
        more = step(dm, small)
    torch.cuda.synchronize()
    assert not errors, errors
    for out, w in zip(outs, (want, big, want)):
        assert equal(out[:3], w[:3])
    assert equal(replayed(graph, held), want) and equal(more, want)
    dm.check_status()
