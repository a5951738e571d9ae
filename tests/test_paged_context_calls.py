"""How page bounds, page selection, attention over chosen pages and behind shared prompts are called: workspaces, streams,
graphs, repeated calls, lengths that make no sense, large caches, waits that run out (GPU only)."""
import numpy as np
import pytest

from oracle import serving as S
from test_paged_context import Batch, check_prefix, check_select, check_selected, f64, finished, i32, shared

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from top_sparse_attention_row_gb300 import build, binding
    build.build()
    binding.load_library()
    return binding


class Ops:
    """The four calls over one batch, by name."""

    def __init__(self, B, b, n_select=6, groups=(0,), prefix=()):
        self.B, self.b, self.k = B, b, n_select
        self.groups, self.prefix = i32(groups), i32(prefix)
        self.bounds = b.bounds()
        self.lists = i32(b.lists(n_select + 3, n_select, seed=5))

    def call(self, name, batch=None, **kw):
        B, b = self.B, self.b
        batch = b.batch() if batch is None else batch
        if name == "bounds":
            out = kw.pop("out", None)
            return (B.page_bounds(b.k, *batch, self.bounds.clone() if out is None else out, **kw),)
        if name == "select":
            return (B.page_select(b.q, self.bounds, *batch, self.k, **kw),)
        if name == "selected":
            return B.selected_attention_paged(b.q, b.k, b.v, self.lists, *batch, b.scale, **kw)
        return B.prefix_attention_paged(b.q, b.k, b.v, *batch, b.scale, self.groups, self.prefix, **kw)

    def workspace_bytes(self, name):
        B, b = self.B, self.b
        n, ppr = b.table.shape
        if name == "select":
            return B.page_select_workspace_bytes(b.R, n, ppr, b.hq, b.hkv, b.dim)
        if name == "selected":
            return B.selected_workspace_bytes(b.R, n, ppr, b.ps, self.lists.shape[2], b.hq, b.hkv, b.dim)
        return B.prefix_workspace_bytes(b.R, n, self.prefix.numel(), ppr, b.ps, b.hq, b.hkv, b.dim)


NAMES = ["bounds", "select", "selected", "prefix"]


def ops(B, seed=0, new=lambda i: 1 + 7 * (i % 3)):
    b = shared(7, 640, lambda i: 30 + 41 * i, 12, 2, 128, 16, seed=seed, new=new)
    return Ops(B, b, groups=[0, 7], prefix=[640])


def same(a, b):
    import torch
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("name", NAMES[1:])
def test_workspaces(B, name):
    import torch
    o = ops(B)
    want = o.call(name)
    n = o.workspace_bytes(name)
    assert n > 0
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")                # NaN everywhere
    assert same(o.call(name, workspace=ws), want)
    assert same(o.call(name, workspace=ws), want)                               # as the call before left it
    for bad in (ws[:n - 1], ws[8:]):
        with pytest.raises(RuntimeError, match="WORKSPACE"):
            o.call(name, workspace=bad)
    finished(B)


def test_c_entries_take_workspaces_from_the_pool(B):
    import torch
    o = ops(B)
    b, lib = o.b, B.load_library()
    cu, kv, table = i32(b.cu), i32(b.kv), i32(b.table)
    n, ppr = b.table.shape
    at = lambda *t: [x.data_ptr() for x in t]  # noqa: E731
    stream = torch.cuda.current_stream().cuda_stream
    pages = torch.empty((b.R, 2, o.k), dtype=torch.int32, device="cuda")
    assert lib.qsa_page_select(*at(b.q, o.bounds, cu, kv, table, pages), b.R, n, ppr, 16, b.n_pages, 12, 2, 128, o.k, 1, 1, 0,
                               None, 0, stream) == 0
    out = torch.empty_like(b.q)
    assert lib.qsa_selected_attention_paged(*at(b.q, b.k, b.v, o.lists, cu, kv, table, out), None, b.R, n, ppr, 16, b.n_pages,
                                            o.lists.shape[2], 12, 2, 128, b.scale, 0, None, 0, stream) == 0
    out2 = torch.empty_like(b.q)
    assert lib.qsa_prefix_attention_paged(*at(b.q, b.k, b.v, cu, kv, table, o.groups, o.prefix, out2), None, b.R, n, 1, ppr, 16,
                                          b.n_pages, 12, 2, 128, b.scale, 0, None, 0, stream) == 0
    finished(B)
    assert torch.equal(pages, o.call("select")[0])
    assert torch.equal(out, o.call("selected")[0]) and torch.equal(out2, o.call("prefix")[0])


def test_unaligned_outputs(B):
    """Outputs on 16-byte boundaries that are not 32-byte ones."""
    import torch
    o = ops(B)
    for name in ("selected", "prefix"):
        want = o.call(name)
        odd = torch.empty(want[0].numel() + 8, dtype=want[0].dtype, device="cuda")[8:].view(want[0].shape)
        assert torch.equal(o.call(name, out=odd)[0], want[0])


@pytest.mark.parametrize("name", NAMES)
def test_two_streams_at_once(B, name):
    import torch
    os_ = [ops(B, seed=k) for k in range(2)]
    want = [o.call(name) for o in os_]
    batches = [o.b.batch() for o in os_]
    streams = [torch.cuda.Stream() for _ in os_]
    torch.cuda.synchronize()
    outs = [[o.bounds.clone() for _ in range(10)] for o in os_] if name == "bounds" else None
    torch.cuda.synchronize()
    got = [[o.call(name, batch=x, stream=s, **(dict(out=outs[k][t]) if outs else {}))
            for k, (o, x, s) in enumerate(zip(os_, batches, streams))] for t in range(10)]
    torch.cuda.synchronize()
    for pair in got:
        assert same(pair[0], want[0]) and same(pair[1], want[1])
    with torch.cuda.stream(streams[0]):
        a = os_[1].call(name)
    streams[0].synchronize()
    assert same(a, want[1])
    finished(B)


@pytest.mark.parametrize("name", NAMES)
def test_results_repeat(B, name):
    o = ops(B, seed=3)
    want = o.call(name)
    for _ in range(20):
        assert same(o.call(name), want)
    finished(B)


def test_rows_that_do_not_begin_at_zero(B):
    """Rows before the first request are left as they were, and the others get what they get without them."""
    import torch
    o = ops(B, seed=6)
    b, ahead = o.b, 70
    more = lambda t: torch.cat((torch.zeros_like(t[:1]).expand(ahead, *t.shape[1:]), t)).contiguous()  # noqa: E731
    q, batch = more(b.q), (i32(b.cu + ahead), i32(b.kv), i32(b.table), 16)
    pages = torch.full((ahead + b.R, 2, o.k), -5, dtype=torch.int32, device="cuda")
    B.page_select(q, o.bounds, *batch, o.k, out=pages)
    assert torch.equal(pages[ahead:], o.call("select")[0]) and bool((pages[:ahead] == -5).all())
    chosen = lambda v: S.selected_attention(f64(b.q), f64(b.k), v, o.lists.cpu().numpy(), *b.host(), b.scale)  # noqa: E731
    whole = lambda v: S.window_attention(f64(b.q), f64(b.k), v, *b.host(), b.scale)  # noqa: E731
    for name, want in (("selected", chosen), ("prefix", whole)):
        out = torch.full((ahead + b.R, 12, 128), 7, dtype=q.dtype, device="cuda")
        lse = torch.full((ahead + b.R, 12), 7, dtype=torch.float32, device="cuda")
        if name == "selected":
            B.selected_attention_paged(q, b.k, b.v, more(o.lists), *batch, b.scale, out=out, lse=lse)
        else:
            B.prefix_attention_paged(q, b.k, b.v, *batch, b.scale, o.groups, o.prefix, out=out, lse=lse)
        finished(B)
        b.compare((out[ahead:], lse[ahead:]), *want(f64(b.v)), want(np.abs(f64(b.v)))[0])
        assert bool((out[:ahead] == 7).all()) and bool((lse[:ahead] == 7).all())


@pytest.mark.parametrize("name", NAMES)
def test_no_rows(B, name):
    o = Ops(B, Batch([(30, 0), (0, 0)], 4, 2, 64, 16, seed=1))
    got = o.call(name)
    assert name == "bounds" or got[0].shape[0] == 0
    finished(B)


def test_prefix_replays_from_a_graph(B):
    """Decode steps behind one prompt, captured once; lengths grow past page and tile borders with every replay."""
    import torch
    b = shared(5, 256, lambda i: 140 + 60 * i, 8, 2, 64, 16, seed=7)
    kv, cu, table = i32([256 + 3 + 50 * i for i in range(5)]), i32(b.cu), i32(b.table)
    groups, prefix = i32([0, 5]), i32([256])
    call = lambda: B.prefix_attention_paged(b.q, b.k, b.v, cu, kv, table, 16, b.scale, groups, prefix)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for t in range(40):
        kv += 3
        graph.replay()
        torch.cuda.synchronize()
        if t % 4 == 0:
            b.kv = kv.cpu().numpy()
            o, z = S.window_attention(f64(b.q), f64(b.k), f64(b.v), *b.host(), b.scale)
            a, _ = S.window_attention(f64(b.q), f64(b.k), np.abs(f64(b.v)), *b.host(), b.scale)
            b.compare(got, o, z, a)
    for shorter in (100, 0):                               # not whole pages; nothing
        prefix.fill_(shorter)
        kv += 1
        graph.replay()
        torch.cuda.synchronize()
        b.kv = kv.cpu().numpy()
        o, z = S.window_attention(f64(b.q), f64(b.k), f64(b.v), *b.host(), b.scale)
        a, _ = S.window_attention(f64(b.q), f64(b.k), np.abs(f64(b.v)), *b.host(), b.scale)
        b.compare(got, o, z, a)
    finished(B)


def test_two_graphs_of_one_workspace_replay_in_turn(B):
    """Graphs that share a workspace are ordered by their stream."""
    import torch
    os_ = [ops(B, seed=k) for k in range(2)]
    for name in NAMES[1:]:
        want = [o.call(name) for o in os_]
        batches = [o.b.batch() for o in os_]
        ws = torch.empty(max(o.workspace_bytes(name) for o in os_), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        graphs, got = [], []
        for o, x in zip(os_, batches):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                got.append(o.call(name, batch=x, workspace=ws))
            graphs.append(g)
        for t in range(6):
            graphs[t % 2].replay()
        torch.cuda.synchronize()
        assert same(got[0], want[0]) and same(got[1], want[1])


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("cu,kv", [([0, 40, 5, 60], [1500, 1200, 900]), ([60, 40, 20, 0], [1500, 1200, 900]),
                                   ([50, -3, 20, 61], [-7, 1500, 2 ** 31 - 1]), ([0, 0, 0, 0], [1, 2, 3]),
                                   ([0, 20, 40, 60], [2 ** 31 - 1, -2 ** 31, 0]),
                                   ([0, 100000, 7, 100000], [-2 ** 31, 1500, 1500])])
def test_offsets_and_lengths_that_make_no_sense_stay_in_bounds(B, name, cu, kv):
    """No promise about the outputs, but the tensors around them stay as they are and the next call is right."""
    import torch
    b = Batch([(1500, 20), (1200, 20), (900, 20)], 4, 2, 128, 16, seed=9)
    o = Ops(B, b, n_select=9, groups=[0, 3], prefix=[320])
    want = o.call(name)
    room = torch.full((3, *want[0].shape), 7, dtype=want[0].dtype, device="cuda")
    o.call(name, batch=(i32(cu), i32(kv), i32(b.table), 16), out=room[1])
    torch.cuda.synchronize()
    assert B.device_status() == 0
    assert bool((room[0] == 7).all()) and bool((room[2] == 7).all())
    assert same(o.call(name), want)


@pytest.mark.parametrize("groups,prefix", [([0, 2, 1, 3], [320, 320, 320]), ([3, 2, 1, 0], [320] * 3), ([-5, 2, 9], [2 ** 31 - 1, 7]),
                                           ([0, 3], [-2 ** 31]), ([2 ** 31 - 1, -2 ** 31], [320])])
def test_groups_that_make_no_sense_stay_in_bounds(B, groups, prefix):
    import torch
    b = shared(3, 320, lambda i: 20 + i, 4, 2, 128, 16, seed=9, new=lambda i: 5)
    o = Ops(B, b, groups=groups, prefix=prefix)
    good = Ops(B, b, groups=[0, 3], prefix=[320])
    want = good.call("prefix")
    room = torch.full((3, *want[0].shape), 7, dtype=want[0].dtype, device="cuda")
    o.call("prefix", out=room[1])
    torch.cuda.synchronize()
    assert B.device_status() == 0
    assert bool((room[0] == 7).all()) and bool((room[2] == 7).all())
    assert same(good.call("prefix"), want)


@pytest.mark.parametrize("dim,hkv", [(256, 8), (64, 24)])
def test_caches_whose_offsets_pass_32_bits(B, dim, hkv):
    """The same batch with its pages at the far end of a cache of more than 2^31 elements."""
    import torch
    ps = 64
    b = shared(3, 256, lambda i: 70 + 90 * i, 2 * hkv, hkv, dim, ps, seed=11, new=lambda i: 1 + i)
    o = Ops(B, b, n_select=4, groups=[0, 3], prefix=[256])
    want = {name: o.call(name) for name in NAMES}
    pages = (2 ** 31 + 2 ** 28) // (ps * hkv * dim)
    far = pages - b.n_pages
    used = torch.from_numpy(np.unique(b.table[b.table >= 0])).long().cuda()

    def grow(t, per):
        x = torch.empty((pages * per, *t.shape[1:]), dtype=t.dtype, device="cuda")
        x[far * per:] = t
        return x
    b.k, b.v, o.bounds = grow(b.k, ps), grow(b.v, ps), grow(o.bounds, 1)
    b.table = np.where(b.table >= 0, b.table + far, -1)
    assert torch.equal(o.call("bounds")[0][used + far], want["bounds"][0][used])
    for name in NAMES[1:]:
        assert same(o.call(name), want[name])
    finished(B)


def test_bounds_beyond_32_bits(B):
    """Bounds of more than 2^31 elements (pages of one slot)."""
    import torch
    b = Batch([(40, 3), (33, 1)], 4, 2, 256, 1, seed=12)
    bounds = b.bounds()
    want = B.page_select(b.q, bounds, *b.batch(), 7)
    pages = (2 ** 31 + 2 ** 24) // (2 * 2 * 256)
    big = torch.empty((pages, 2, 2, 256), dtype=bounds.dtype, device="cuda")
    big[-b.n_pages:] = bounds
    table = np.where(b.table >= 0, b.table + pages - b.n_pages, -1)
    got = B.page_select(b.q, big, i32(b.cu), i32(b.kv), i32(table), 1, 7)
    assert torch.equal(got, want)
    finished(B)


@pytest.mark.parametrize("name", NAMES[1:])
def test_a_wait_that_runs_out(B, name):
    """The scheduler withholds its items: the waits run out after their limit, the call ends, its status is reported, and the
    next call is right."""
    import time
    import torch
    o = ops(B, seed=4)
    want = o.call(name)
    finished(B)
    B.debug_stall_next_call()
    t0 = time.time()
    o.call(name)
    torch.cuda.synchronize()
    assert 1.0 < time.time() - t0 < 30.0
    assert B.device_status() & 0x100
    assert same(o.call(name), want)
    finished(B)


@pytest.mark.parametrize("seed", range(12))
def test_random_batches(B, seed):
    """Lengths, heads, page sizes, groups and holes at random."""
    rng = np.random.default_rng(100 + seed)
    dim = int(rng.choice([64, 128, 256]))
    hkv = int(rng.choice([1, 2, 3]))
    hq = hkv * int(rng.choice([1, 2, 3, 4, 5, 8, 12, 17]))
    ps = int(rng.choice([8, 16, 24, 40, 64, 128]))
    n = int(rng.integers(1, 9))
    prefix = int(rng.integers(0, 20)) * ps
    new = [int(rng.choice([0, 1, 1, 2, 30, 75])) for _ in range(n)]
    own = [int(m + rng.integers(0, 200)) for m in new]
    b = shared(n, prefix, lambda i: own[i], hq, hkv, dim, ps, str(rng.choice(["bfloat16", "float16"])), seed=seed,
               new=lambda i: new[i], pad_rows=int(rng.integers(0, 4)), wide=int(rng.integers(0, 5)))
    if b.cu[-1] == 0:
        return
    cut = int(rng.integers(0, n + 1))
    check_prefix(B, b, [0, cut, n], [prefix, int(rng.integers(0, prefix + 1))])
    holes = rng.random(b.table.shape) < 0.05
    b.table = np.where(holes, rng.choice([-1, b.n_pages, 2 ** 31 - 1], b.table.shape), b.table)
    k = int(rng.integers(2, 30))
    got = check_select(B, b, b.bounds(), k, int(rng.integers(0, 2)), 1)
    check_selected(B, b, np.where(got == -2, -1, got))
    check_selected(B, b, b.lists(k + 2, k, seed=seed))
