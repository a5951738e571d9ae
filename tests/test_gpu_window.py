"""Sliding-window attention with sink tokens over paged caches, 16-bit and 4-bit, against its float64
restatement (GPU only)."""
import numpy as np
import pytest

from oracle import serving as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from top_sparse_attention_row_gb300 import build, binding
    build.build()
    binding.load_library()
    return binding


def i32(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


class Batch:
    """A ragged batch over a shuffled paged cache: lens = [(kv_len, new rows)]."""

    def __init__(self, lens, hq, hkv, dim, ps, dtype="bfloat16", fp4=False, seed=0, pad_rows=0, spread=1.0):
        import torch
        rng = np.random.default_rng(seed)
        self.dt = getattr(torch, dtype)
        self.ps, self.dim = ps, dim
        self.kv = np.array([a for a, _ in lens])
        self.cu = np.concatenate([[0], np.cumsum([b for _, b in lens])])
        self.R = int(self.cu[-1]) + pad_rows
        ppr = max(1, max(-(-a // ps) for a, _ in lens))
        used = sum(-(-a // ps) for a, _ in lens)
        self.n_pages = used + 3
        pages = rng.permutation(self.n_pages)
        self.table = np.full((len(lens), ppr), -1)
        at = 0
        for i, (a, _) in enumerate(lens):
            n = -(-a // ps)
            self.table[i, :n] = pages[at:at + n]
            at += n
        s = self.n_pages * ps
        to = lambda x: torch.from_numpy(x).to(self.dt).cuda()  # noqa: E731
        self.q = to(rng.standard_normal((self.R, hq, dim)) * spread)
        k, v = rng.standard_normal((2, s, hkv, dim))
        self.fp4 = fp4
        if fp4:
            self.kg, self.vg = 0.25, 0.5
            (kc, ks, k), (vc, vs, v) = S.fp4_quantise(k, self.kg), S.fp4_quantise(v, self.vg)
            u8 = lambda x: torch.from_numpy(x.astype(np.uint8)).cuda()  # noqa: E731
            self.k, self.v = u8(S.fp4_pack(kc)), u8(S.fp4_pack(vc))
            self.ks, self.vs = u8(ks), u8(vs)
            self.k64, self.v64 = k, v
        else:
            self.k, self.v = to(k), to(v)
            self.k64, self.v64 = self.k.double().cpu().numpy(), self.v.double().cpu().numpy()
        self.q64 = self.q.double().cpu().numpy()
        self.scale = dim ** -0.5

    def call(self, B, window, n_sink, **kw):
        common = (i32(self.cu), i32(self.kv), i32(self.table), self.ps, self.scale)
        kw = dict(window=window, n_sink=n_sink, **kw)
        if self.fp4:
            return B.window_attention_fp4_paged(self.q, self.k, self.ks, self.v, self.vs, *common,
                                                k_global=self.kg, v_global=self.vg, **kw)
        return B.window_attention_paged(self.q, self.k, self.v, *common, **kw)

    def check(self, B, window, n_sink, rows=None, **kw):
        import torch
        out, lse = self.call(B, window, n_sink, **kw)
        torch.cuda.synchronize()
        assert B.device_status() == 0
        self.compare(out, lse, window, n_sink, rows)
        return out, lse

    def compare(self, out, lse, window, n_sink, rows=None):
        import torch
        n = int(self.cu[-1])
        rows = np.arange(n) if rows is None else np.asarray(rows)
        args = (self.cu, self.kv, self.table, self.ps, self.scale, window, n_sink, rows)
        o, z = S.window_attention(self.q64, self.k64, self.v64, *args)
        a, _ = S.window_attention(self.q64, self.k64, np.abs(self.v64), *args)
        o, z, a = o[rows], z[rows], a[rows]
        got, zg = out.double().cpu().numpy()[rows], lse.double().cpu().numpy()[rows]
        assert np.array_equal(np.isneginf(zg), np.isneginf(z))
        # Weights and output are rounded to the type's half step u (weights of a 4-bit cache to fp16's);
        # with A = sum w |v| / l: |dO| <= u_w A (numerator) + u |O|.  A logit is a sum of dim products in
        # fp32, off by at most dim 2^-23 sum |q k| scale =: d (for N(0, 1) rows sum |q k| scale is at most
        # about 2 sqrt(dim) spread), which changes a weight by a factor e^d and l likewise: 2 d A.
        u = torch.finfo(self.dt).eps / 2
        uw = 2.0 ** -11 if self.fp4 or self.dt == torch.float16 else u
        spread = max(1.0, float(np.std(self.q64)))
        d = self.dim * 2.0 ** -23 * 2 * np.sqrt(self.dim) * spread + 2.0 ** -20
        if self.fp4 and self.dt == torch.bfloat16:
            pass                       # bf16 q is exact in fp16 above 2^-14
        bound = uw * a + u * np.abs(o) + 2 * d * a + 2.0 ** -24
        worst = np.max(np.abs(got - o) - bound)
        assert worst <= 0, (worst, np.max(np.abs(got - o)))
        fin = np.isfinite(z)
        assert np.all(np.abs(zg[fin] - z[fin]) <= d + 2.0 ** -21 * np.abs(z[fin]) + 2.0 ** -22)


DECODE = [(1, 1), (77, 1), (129, 1), (700, 1), (64, 1)]
MIXED = [(5, 5), (300, 40), (513, 1), (257, 130), (64, 64), (3, 3), (40, 2)]


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window,sink", [(0, 0), (100, 4), (1, 0), (33, 40)])
def test_decode(B, dim, window, sink, fp4):
    Batch(DECODE, 6, 2, dim, 16, fp4=fp4, seed=dim + window).check(B, window, sink)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window,sink", [(0, 0), (64, 3), (200, 130)])
def test_mixed_batch(B, dim, window, sink, dtype, fp4):
    Batch(MIXED, 8, 2, dim, 64, dtype, fp4=fp4, seed=dim + sink).check(B, window, sink)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("ps", [1, 2, 3, 7, 8, 12, 24, 48, 64, 100, 128, 256])
def test_page_sizes(B, ps, fp4):
    Batch([(1000, 30), (129, 1), (40, 40)], 4, 2, 128, ps, fp4=fp4, seed=ps).check(B, 150, 5)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (24, 2), (96, 1), (128, 1), (130, 2), (8, 8), (40, 5)])
def test_head_groups(B, hq, hkv):
    for fp4 in (False, True):
        Batch([(400, 37), (90, 1)], hq, hkv, 64, 16, fp4=fp4, seed=hq).check(B, 90, 2)


@pytest.mark.parametrize("hq", [33, 64])
def test_large_groups_over_a_4_bit_cache_of_256_dims(B, hq):
    """Query tiles of 64 rows there: one token of 33 or 64 heads."""
    Batch([(300, 9), (90, 1)], hq, 1, 256, 16, fp4=True, seed=hq).check(B, 90, 2)


@pytest.mark.parametrize("fp4", [False, True])
def test_non_finite_queries_stay_in_their_rows(B, fp4):
    import torch
    b = Batch([(400, 37), (90, 1)], 4, 2, 128, 16, fp4=fp4)
    want = b.check(B, 0, 0)
    b.q[5, 1, 7], b.q[30, 3], b.q[37, 0, 0] = float("nan"), float("inf"), float("-inf")
    got = b.call(B, 0, 0)
    torch.cuda.synchronize()
    rest = torch.ones(want[1].shape, dtype=torch.bool, device="cuda")
    rest[5, 1] = rest[30, 3] = rest[37, 0] = False
    assert torch.equal(got[0][rest], want[0][rest]) and torch.equal(got[1][rest], want[1][rest])
    assert bool(got[0][5, 1].isnan().all()) and bool(got[1][5, 1].isnan())


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("n,rows", [(60000, 1), (20000, 3), (900, 1)])
def test_non_finite_queries_in_equal_shares(B, n, rows, fp4):
    """Units in more parts than a warp joins, and in few: a NaN row is NaN in out and lse, the others are as
    they were."""
    import torch
    b = Batch([(n, rows), (40, 2)], 4, 1, 64, 64, fp4=fp4, seed=rows)
    assert B.window_workspace_bytes(rows + 2, 2, b.table.shape[1], 64, 4, 1, 64, 0, 0, fp4=fp4, num_sms=152) > 0
    want = b.check(B, 0, 0)
    b.q[0, 1, 3], b.q[rows + 1, 2], b.q[rows, 0, 0] = float("nan"), float("nan"), float("inf")
    out, lse = b.call(B, 0, 0)
    torch.cuda.synchronize()
    bad = torch.zeros(lse.shape, dtype=torch.bool, device="cuda")
    bad[0, 1] = bad[rows + 1, 2] = bad[rows, 0] = True
    assert torch.equal(out[~bad], want[0][~bad]) and torch.equal(lse[~bad], want[1][~bad])
    assert bool(out[bad].isnan().all()) and bool(lse[bad].isnan().all())


LAYOUTS = {      # how a call is dealt out: whole units, equal shares joined by warps, by blocks
    "whole": ([(2600, 2600), (300, 300)], 8, 2), "few parts": ([(900, 1), (40, 2)], 4, 1),
    "many parts": ([(60000, 1), (40, 2)], 4, 1)}


@pytest.mark.parametrize("how", LAYOUTS)
@pytest.mark.parametrize("what", ["k nan", "k inf", "k -inf", "v inf", "v -inf", "v nan"])
def test_non_finite_values_that_rows_see(B, how, what):
    """One element of the key at position 20 of the first request, q there positive for all: the logit is NaN, inf
    or -inf.  With v, the element's dim is non-finite in every row that sees it; rows of other requests and
    KV heads, and with k also the earlier rows, stay as they are."""
    import torch
    lens, hq, hkv = LAYOUTS[how]
    b = Batch(lens, hq, hkv, 64, 64, seed=3)
    R = b.R
    ws = B.window_workspace_bytes(R, 2, b.table.shape[1], 64, hq, hkv, 64, 0, 0, num_sms=152)
    assert (ws == 0) == (how == "whole")
    b.q[..., 5] = b.q[..., 5].abs() + 0.5
    want = b.call(B, 0, 0)
    value = float(what.split()[1])
    slot = int(b.table[0][0]) * 64 + 20
    (b.k if what[0] == "k" else b.v)[slot, 0, 5] = value
    out, lse = b.call(B, 0, 0)
    torch.cuda.synchronize()
    first, new = int(b.kv[0]), int(b.cu[1])
    sees = np.arange(R) >= max(0, 20 - (first - new))
    sees[new:] = False
    hit = torch.zeros((R, hq), dtype=torch.bool, device="cuda")
    hit[torch.from_numpy(sees).cuda(), :hq // hkv] = True
    if what in ("k nan", "k inf"):
        assert bool(out[hit].isnan().all()) and bool(lse[hit].isnan().all())
        assert torch.equal(out[~hit], want[0][~hit]) and torch.equal(lse[~hit], want[1][~hit])
    elif what == "k -inf":        # weight 0: as a batch that has the key's logit far below the others
        b.k[slot, 0, 5] = -1e30
        far = b.call(B, 0, 0)
        torch.cuda.synchronize()
        rows = torch.arange(R, device="cuda") != 20       # (the row at 20 sees earlier keys as well)
        assert bool(out.isfinite().all()) and bool(lse.isfinite().all())
        assert torch.equal(out[rows], far[0][rows]) and torch.equal(lse[rows], far[1][rows])
    else:
        got = out[hit][:, 5].float()
        assert not bool(got.isfinite().any())
        if what != "v nan" and how != "whole":            # decode rows: weights that are not 0
            near = lens[0][1] == 1 and first < 2000
            assert not near or bool((got == value).all())
        dims = torch.arange(64, device="cuda") != 5
        assert torch.equal(out[..., dims], want[0][..., dims]) and torch.equal(lse, want[1])
        other = torch.ones_like(hit)
        other[:new, :hq // hkv] = False
        assert torch.equal(out[other], want[0][other])


@pytest.mark.parametrize("n", [3, 900, 60000])
def test_rows_whose_logits_are_all_minus_infinity(B, n):
    """As rows that see nothing: out 0, lse -inf."""
    import torch
    b = Batch([(n, 1), (50, 3)], 4, 1, 128, 64)
    want = b.call(B, 0, 0)
    b.q[0, :, 0] = 1.0
    at = torch.from_numpy(np.concatenate([np.arange(64) + 64 * p for p in b.table[0] if p >= 0])).cuda()
    b.k[at, 0, 0] = -float("inf")
    out, lse = b.call(B, 0, 0)
    torch.cuda.synchronize()
    assert float(out[0].abs().max()) == 0 and bool((lse[0] == -float("inf")).all())
    assert torch.equal(out[1:], want[0][1:]) and torch.equal(lse[1:], want[1][1:])


def test_infinite_values_of_vanishing_weight_are_not_lost_in_a_join(B):
    """An infinite V whose part of a shared unit has a weight that fp32 cannot hold: inf or NaN, on both ways of
    joining."""
    import torch
    for n in (900, 60000):
        b = Batch([(n, 1)], 1, 1, 64, 64, seed=n)
        b.q[:] = 0.0
        b.q[..., 0] = 16.0
        b.k[..., 0] = 0.0
        far, near = int(b.table[0][0]) * 64 + 5, int(b.table[0][-1]) * 64 + (n - 1) % 64
        b.k[near, 0, 0] = 100.0                                  # 200 above the others
        b.v[far, 0, 7] = float("inf")
        out, lse = b.call(B, 0, 0)
        torch.cuda.synchronize()
        assert not bool(out[0, 0, 7].isfinite()) and bool(lse.isfinite().all())
        assert bool(out[0, 0, 8:].isfinite().all())


def test_first_call_inside_a_capture(B):
    """A fresh process whose very first calls are captured."""
    import subprocess
    import sys
    code = """
import torch
from top_sparse_attention_row_gb300 import binding as B
i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
q = torch.randn((1, 6, 256), device="cuda").bfloat16()
k, v = (torch.randn((4096, 1, 256), device="cuda").bfloat16() for _ in range(2))
args = (i(0, 1), i(4000), torch.arange(64, device="cuda").int()[None], 64, 0.0625)
past, new, table, free, head = i(5), i(1), i(7, 0)[None].contiguous(), i(3, 4), i(0)
rope, pos, slot = B.rope_table(256), i(9), i(11)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    plan = B.page_plan(past, new, table, free, head, 4, 1)
    x = B.rope_append(q, k[:1], v[:1], k, v, pos, slot, rope)
    out, lse = B.window_attention_paged(x, k, v, *args)
g.replay()
torch.cuda.synchronize()
a, b = out.clone(), lse.clone()
want = B.window_attention_paged(x, k, v, *args)
torch.cuda.synchronize()
assert torch.equal(a, want[0]) and torch.equal(b, want[1]) and int(plan.slots) == 1 and B.device_status() == 0
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


# ------------------------------------------------------------------------------ masks and bad places

def unseen_slots(b, window, sink):
    """Cache slots that no row sees."""
    seen = np.zeros(b.n_pages * b.ps, bool)
    for i, kv in enumerate(b.kv):
        new = b.cu[i + 1] - b.cu[i]
        for p in range(max(kv - new, 0), kv):
            lo = 0 if window <= 0 else max(0, p - window + 1)
            js = np.concatenate([np.arange(min(sink, lo)), np.arange(lo, p + 1)])
            js = js[js < b.table.shape[1] * b.ps]
            page = b.table[i][js // b.ps]
            js, page = js[page >= 0], page[page >= 0]
            seen[page * b.ps + js % b.ps] = True
    return np.flatnonzero(~seen)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), 3e38])
@pytest.mark.parametrize("dim,window,sink", [(64, 0, 0), (128, 70, 3), (256, 70, 3), (256, 1, 0), (128, 200, 150)])
def test_anything_in_unseen_places(B, dim, window, sink, value):
    """The rest of a page, tokens that left the window, unused pages: NaN, infinities and the largest
    values there change nothing."""
    import torch
    b = Batch([(300, 1), (95, 30), (777, 2), (5, 5)], 4, 2, dim, 64, seed=dim)
    want = b.check(B, window, sink)
    at = torch.from_numpy(unseen_slots(b, window, sink)).cuda()
    b.k[at], b.v[at] = value, value
    got = b.call(B, window, sink)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_anything_in_unseen_places_of_a_4_bit_cache(B, dim):
    import torch
    b = Batch([(300, 1), (95, 30), (777, 2), (5, 5)], 4, 2, dim, 64, fp4=True, seed=dim)
    want = b.check(B, 70, 3)
    at = torch.from_numpy(unseen_slots(b, 70, 3)).cuda()
    b.ks[at], b.vs[at], b.k[at], b.v[at] = 0x7F, 0xFF, 0x77, 0xFF       # NaN scales
    got = b.call(B, 70, 3)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("dim", [64, 256])
def test_rows_that_see_nothing(B, dim, fp4):
    """kv_len below the row count puts first rows at negative positions; empty requests and kv_len 0."""
    b = Batch([(40, 40), (10, 10), (300, 3), (20, 20)], 4, 2, dim, 16, fp4=fp4, seed=1)
    b.kv = np.array([25, 0, 300, 1])
    out, lse = b.check(B, 0, 0)
    assert float(out[:15].abs().max()) == 0 and bool((lse[:15] == -np.inf).all())
    b.check(B, 8, 2)
    e = Batch([(70, 0), (50, 50), (9, 0), (9, 0), (300, 7), (1, 0)], 4, 2, dim, 16, fp4=fp4, seed=2)
    e.check(B, 0, 0)
    e.check(B, 33, 1)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("ps", [1, 3, 16, 64])
def test_missing_and_bad_pages(B, ps, fp4):
    """Entries below 0, past the pool, and positions past the table's row are not seen, wherever they lie."""
    b = Batch([(400, 60), (333, 1), (200, 5)], 4, 2, 128, ps, fp4=fp4, seed=ps)
    rng = np.random.default_rng(ps)
    hit = rng.random(b.table.shape) < 0.2
    b.table = np.where(hit, rng.choice([-1, -7, b.n_pages, 2 ** 31 - 1], b.table.shape), b.table)
    b.check(B, 0, 0)
    b.check(B, 120, 9)
    b.table = b.table[:, :max(1, b.table.shape[1] // 2)]
    b.check(B, 0, 0)
    b.check(B, 120, 9)
    b.table[:] = -1                                   # no page at all
    out, lse = b.check(B, 50, 2)
    assert float(out.abs().max()) == 0


@pytest.mark.parametrize("fp4", [False, True])
def test_padded_batch_leaves_its_last_rows(B, fp4):
    import torch
    b = Batch([(100, 3), (300, 1)], 4, 2, 256, 64, fp4=fp4, pad_rows=37)
    out = torch.full_like(b.q, 7.0)
    lse = torch.full((b.R, 4), 5.0, device="cuda")
    b.check(B, 64, 4, out=out, lse=lse)
    assert bool((out[4:] == 7).all()) and bool((lse[4:] == 5).all())
    c = Batch([(1500, 600)], 4, 2, 64, 64, fp4=fp4, pad_rows=300)       # whole units
    out = torch.full_like(c.q, 7.0)
    c.check(B, 64, 4, out=out, rows=range(0, 600, 7))
    assert bool((out[600:] == 7).all())


# ------------------------------------------------------------------------------ numerics

@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("cu,kv", [([0, 40, 5, 60], [1500, 1200, 900]), ([60, 40, 20, 0], [1500, 1200, 900]),
                                   ([50, -3, 20, 61], [-7, 1500, 2 ** 31 - 1]), ([0, 0, 0, 0], [1, 2, 3]),
                                   ([0, 2 ** 31 - 1, 7, 2 ** 31 - 1], [-2 ** 31, 1500, 1500])])
def test_offsets_and_lengths_that_make_no_sense_stay_in_bounds(B, cu, kv, fp4):
    """Row offsets that do not increase or leave the rows, negative and huge lengths: no promise about the
    outputs, but the tensors around them stay as they are and the next call is right."""
    import torch
    b = Batch([(1500, 20), (1200, 20), (900, 20)], 4, 2, 128, 16, fp4=fp4)
    want = b.check(B, 0, 0)
    good = b.cu, b.kv
    room = torch.full((3, *want[0].shape), 7.0, dtype=b.dt, device="cuda")
    lroom = torch.full((3, *want[1].shape), 7.0, device="cuda")
    b.cu, b.kv = np.array(cu), np.array(kv)
    for window, sink in ((0, 0), (100, 3), (2 ** 31 - 1, 2 ** 31 - 1)):
        b.call(B, window, sink, out=room[1], lse=lroom[1])
    torch.cuda.synchronize()
    assert B.device_status() == 0
    for x in (room, lroom):
        assert bool((x[0] == 7).all()) and bool((x[2] == 7).all())
    b.cu, b.kv = good
    again = b.check(B, 0, 0)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


@pytest.mark.parametrize("dim", [64, 256])
@pytest.mark.parametrize("order", ["up", "down", "spike"])
def test_rising_logits(B, dim, order):
    """Logits that climb by far more than 2^8 from tile to tile, so that O is rescaled again and again."""
    import torch
    b = Batch([(900, 40), (640, 1)], 4, 1, dim, 64, seed=4)
    n = b.n_pages * b.ps
    ramp = {"up": np.arange(n), "down": n - np.arange(n), "spike": (np.arange(n) % 200 == 0) * n}[order] / n
    pos = np.zeros(n)
    for i, kv in enumerate(b.kv):
        js = np.arange(kv)
        pos[b.table[i][js // b.ps] * b.ps + js % b.ps] = ramp[js * n // 1000]
    # q and k along one direction: logits up to 300
    b.q = torch.zeros_like(b.q)
    b.q[..., 0] = 16.0
    b.k[..., 0] = torch.from_numpy(300 * np.sqrt(dim) / 16 * pos).to(b.dt).cuda()[:, None]
    b.q64, b.k64 = b.q.double().cpu().numpy(), b.k.double().cpu().numpy()
    b.check(B, 0, 0)
    b.check(B, 333, 2)


@pytest.mark.parametrize("dtype,fp4", [("float16", False), ("float16", True), ("bfloat16", True), ("bfloat16", False)])
@pytest.mark.parametrize("n,rows,heads", [(6000, 6000, 16), (60000, 1, 1)])
def test_a_long_tail_far_below_one_key(B, n, rows, heads, dtype, fp4):
    """One key 18 nats above all others (v 0 there, 1 elsewhere): the others' weights, 2^-26 each, still add up, in
    whole units and in shares.  A weight is off by half a step u_w of itself, in fp16 or by 2^-32 of the
    largest where that is more; the output by its own half step (or fp16's least, 2^-25)."""
    import torch
    b = Batch([(n, rows)], heads, heads, 64, 64, dtype, fp4=fp4)
    ws = B.window_workspace_bytes(rows, 1, b.table.shape[1], 64, heads, heads, 64, 0, 0, fp4=fp4, num_sms=152)
    assert (ws == 0) == (rows > 1)
    peak = int(b.table[0][0]) * 64 + 7
    b.q[:] = 0.0
    b.q[..., 0] = 96.0                                     # logit 96 k / 8
    if fp4:
        b.k[:], b.ks[:], b.v[:], b.vs[:] = 0, 0x38, 0x22, 0x40          # v = 1.0 * 2.0 * 0.5
        b.k[peak, :, 0], b.v[peak] = 7, 0                               # k = 6 * 1.0 * 0.25
    else:
        b.k[:], b.v[:] = 0.0, 1.0
        b.k[peak, :, 0], b.v[peak] = 1.5, 0.0
    out, lse = b.call(B, 0, 0)
    torch.cuda.synchronize()
    p = np.arange(n - rows, n)
    tail = np.where(p >= 7, p, 1) * np.exp(-18.0)
    o = np.where(p >= 7, tail / (1 + tail), 1.0)[:, None, None]
    z = np.where(p >= 7, 18.0 + np.log1p(tail), np.log(p + 1.0))[:, None]
    u = torch.finfo(b.dt).eps / 2
    uw = 2.0 ** -11 if fp4 or dtype == "float16" else 2.0 ** -8
    bound = o * (uw + u + 2.0 ** -18) + (n * 2.0 ** -32 if uw == 2.0 ** -11 else 0.0) + 2.0 ** -25
    assert np.all(np.abs(out.double().cpu().numpy() - o) <= bound)
    assert np.all(np.abs(lse.double().cpu().numpy() - z) <= 2.0 ** -19 * np.abs(z) + 2.0 ** -22)


@pytest.mark.parametrize("dim,n", [(128, 20000), (256, 9000)])
@pytest.mark.parametrize("fp4", [False, True])
def test_long_context_in_equal_shares(B, dim, n, fp4):
    """One and three decode rows over a long cache: every SM takes a share of the keys."""
    assert B.window_workspace_bytes(1, 1, n // 64, 64, 4, 1, dim, 0, 0, fp4=fp4, num_sms=152) > 0
    Batch([(n, 1)], 4, 1, dim, 64, fp4=fp4, seed=1).check(B, 0, 0)
    Batch([(n, 1), (3, 1), (n // 3, 1)], 4, 1, dim, 64, fp4=fp4, seed=2).check(B, 0, 0)
    Batch([(n, 3)], 4, 1, dim, 64, fp4=fp4, seed=3).check(B, n // 2, 700)


@pytest.mark.parametrize("fp4", [False, True])
def test_ragged_units_in_equal_shares(B, fp4):
    """More units than blocks, of no tile to many: shares that begin and end inside units, empty ones among them."""
    rng = np.random.default_rng(5)
    lens = [(int(rng.choice([0, 1, 5, 128, 129, 700, rng.integers(1, 5000)])), 1) for _ in range(230)]
    Batch(lens + [(5000, 1)], 3, 1, 64, 64, fp4=fp4).check(B, 0, 0)
    Batch(lens[:120] + [(5000, 40)], 4, 2, 64, 16, fp4=fp4).check(B, 0, 0)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("dim,hq,hkv", [(64, 8, 8), (128, 16, 2), (256, 6, 1)])
def test_long_prompt(B, dim, hq, hkv, dtype):
    """Enough query tiles for whole units, and a few more than SMs for equal shares with full tiles."""
    rng = np.random.default_rng(0)
    b = Batch([(3500, 2900)], hq, hkv, dim, 64, dtype, seed=dim)
    rows = rng.choice(2900, 60, replace=False)
    b.check(B, 0, 0, rows=rows)
    b.check(B, 500, 4, rows=rows)


def dealt_out(B, b, hq, hkv, window, sink, fp4):
    """"whole" units or "shares", as on a device of 152 SMs."""
    n = B.window_workspace_bytes(b.R, len(b.kv), b.table.shape[1], b.ps, hq, hkv, b.dim, window, sink, fp4=fp4, num_sms=152)
    return "shares" if n else "whole"


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lens,heads,window,sink", [
    ([(4000, 4000)], 12, 200, 3), ([(1400, 1400), (700, 150), (90, 90), (40, 1)], 24, 0, 0)])
def test_several_whole_units_per_block(B, dim, lens, heads, window, sink, fp4):
    """More than twice as many query tiles as SMs, so that blocks take over unit after unit: every ring, record and
    barrier goes round several times, with units of unequal length among them."""
    rng = np.random.default_rng(dim)
    b = Batch(lens, heads, heads, dim, 64, fp4=fp4, seed=dim)
    tile = 64 if fp4 and dim == 256 else 128
    assert sum(-(-m // tile) for _, m in lens) * heads > 2 * 152
    assert dealt_out(B, b, heads, heads, window, sink, fp4) == "whole"
    rows = np.unique(np.concatenate([rng.choice(b.R, 24, replace=False), [0, 127, 128, b.R - 1]]))
    b.check(B, window, sink, rows=rows)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("dim", [64, 256])
def test_equal_shares_over_more_tiles_than_threads(B, dim, fp4):
    """Every block adds up the units' tiles, its threads one each at a time: here in several rounds, with many requests
    that bring no row, and shares that begin in the later rounds."""
    rng = np.random.default_rng(dim)
    some = [(int(rng.integers(1, 400)), 1) for _ in range(600)]
    some[50], some[599] = (9000, 1), (2500, 1)
    sparse = [(int(rng.integers(1, 300)), int(rng.random() < 0.1)) for _ in range(2500)]
    sparse[2400], sparse[7] = (6000, 3), (3000, 2)
    for lens in (some, sparse):
        b = Batch(lens, 4, 1, dim, 64, fp4=fp4, seed=dim)
        assert b.R // (128 // 4) + len(lens) > 512 and dealt_out(B, b, 4, 1, 0, 0, fp4) == "shares"
        if lens is sparse:
            assert len(lens) > 3 * 768
        b.check(B, 0, 0)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("dim,hq,hkv", [(128, 32, 8), (256, 24, 2)])
def test_a_prompt_in_tables_of_any_width(B, dim, hq, hkv, fp4):
    """How a call is dealt out goes by the table's width; what it computes does not."""
    b = Batch([(1024, 1024)], hq, hkv, dim, 64, fp4=fp4, seed=1)
    rows = np.arange(0, 1024, 79)
    narrow, ways = b.table, set()
    for wide in (1, 4, 64):
        b.table = np.concatenate([narrow, np.full((1, narrow.shape[1] * (wide - 1)), -1)], 1)
        ways.add(dealt_out(B, b, hq, hkv, 0, 0, fp4))
        b.check(B, 0, 0, rows=rows)
    assert "shares" in ways


def test_many_requests(B):
    rng = np.random.default_rng(9)
    lens = [(int(n), int(min(n, m))) for n, m in zip(rng.integers(1, 200, 400), rng.integers(0, 4, 400))]
    for fp4 in (False, True):
        Batch(lens, 2, 1, 64, 16, fp4=fp4, seed=5).check(B, 40, 2)


@pytest.mark.parametrize("fp4", [False, True])
def test_tens_of_thousands_of_requests(B, fp4):
    """More units than shares are dealt out for, short and long ones in no order."""
    rng = np.random.default_rng(21)
    lens = [(int(n), 1) for n in rng.integers(1, 60, 20000)]
    lens[17], lens[12345], lens[19999] = (2000, 30), (1500, 1), (700, 2)
    b = Batch(lens, 2, 1, 64, 16, fp4=fp4, seed=3)
    rows = np.unique(np.concatenate([np.arange(0, b.R, 211), np.arange(17, 47), [12374], np.arange(b.R - 3, b.R)]))
    b.check(B, 0, 0, rows=rows)


def test_random_batches(B):
    """Shapes drawn at random over the whole range."""
    rng = np.random.default_rng(11)
    for k in range(24):
        n = int(rng.integers(1, 9))
        lens = []
        for _ in range(n):
            new = int(rng.choice([0, 1, 1, rng.integers(1, 150)]))
            lens.append((new + int(rng.integers(0, 700)), new))
        if sum(m for _, m in lens) == 0:
            lens[0] = (lens[0][0] + 1, 1)
        hkv = int(rng.choice([1, 2, 3]))
        b = Batch(lens, hkv * int(rng.choice([1, 2, 5, 7, 16])), hkv, int(rng.choice([64, 128, 256])),
                  int(rng.choice([1, 5, 8, 16, 40, 64, 128])), str(rng.choice(["bfloat16", "float16"])),
                  fp4=bool(rng.integers(2)), seed=100 + k, pad_rows=int(rng.integers(0, 3)))
        b.check(B, int(rng.choice([0, 1, 17, 128, 300])), int(rng.choice([0, 1, 4, 64, 129])))


def test_results_repeat_bit_for_bit(B):
    import torch
    for fp4 in (False, True):
        b = Batch([(5000, 1), (900, 200)], 8, 2, 128, 64, fp4=fp4)
        first = b.call(B, 700, 4)
        for _ in range(5):
            again = b.call(B, 700, 4)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_offsets_past_32_bits(B):
    """A cache of more than 4 GiB, the pages in use at its end."""
    import torch
    for fp4 in (False, True):
        b = Batch([(200, 3), (90, 1)], 2, 2, 256, 64, fp4=fp4)
        rows = (1 << 32) // (b.k.stride(0) * b.k.element_size()) + 64
        far = -(-rows // 64)                               # pages in front
        grow = lambda t: torch.cat([torch.zeros((far * 64, *t.shape[1:]), dtype=t.dtype, device="cuda"), t])  # noqa: E731
        want = b.check(B, 100, 4)
        b.k, b.v = grow(b.k), grow(b.v)
        if fp4:
            b.ks, b.vs = grow(b.ks), grow(b.vs)
        b.table = np.where(b.table >= 0, b.table + far, -1)
        got = b.call(B, 100, 4)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------------------------------------ how it is called

def test_outputs_workspaces_and_alignment(B):
    import torch
    b = Batch([(3000, 1), (800, 20)], 6, 1, 256, 64)
    want = b.check(B, 0, 0)
    odd = torch.empty(b.q.numel() + 8, dtype=b.dt, device="cuda")[8:].view(b.q.shape)      # 16-byte aligned only
    got = b.call(B, 0, 0, out=odd, want_lse=False)
    assert got[1] is None and got[0].data_ptr() % 32 == 16 and torch.equal(got[0], want[0])
    args = (b.R, 2, b.table.shape[1], 64, 6, 1, 256, 0, 0)
    n = B.window_workspace_bytes(*args)
    assert n > 0
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")                          # NaN everywhere
    assert torch.equal(b.call(B, 0, 0, workspace=ws)[0], want[0])
    for bad in (ws[:n - 1], ws[8:]):
        with pytest.raises(RuntimeError, match="WORKSPACE"):
            b.call(B, 0, 0, workspace=bad)
    # the C entry without a workspace takes one from the library's pool
    lib, out = B.load_library(), torch.empty_like(b.q)
    cu, kv, table = i32(b.cu), i32(b.kv), i32(b.table)
    st = lib.qsa_window_attention_paged(
        b.q.data_ptr(), b.k.data_ptr(), b.v.data_ptr(), cu.data_ptr(), kv.data_ptr(), table.data_ptr(), out.data_ptr(),
        None, b.R, 2, b.table.shape[1], 64, b.n_pages, 6, 1, 256, b.scale, 0, 0, 0, None, 0,
        torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0 and torch.equal(out, want[0])
    assert b.call(B, 0, 0, out=odd[:0] if False else None)[0].shape == b.q.shape
    empty = Batch([(30, 0)], 6, 1, 256, 64)
    assert empty.call(B, 0, 0)[0].shape == (0, 6, 256)


def test_two_streams_at_once(B):
    import torch
    bs = [Batch([(4000 + 7 * k, 1), (700, 30)], 6, 1, 256, 64, seed=k) for k in range(2)]
    want = [b.check(B, 0, 0) for b in bs]
    streams = [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    got = [[b.call(B, 0, 0, stream=s) for b, s in zip(bs, streams)] for _ in range(20)]
    torch.cuda.synchronize()
    for pair in got:
        for g, w in zip(pair, want):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
    with torch.cuda.stream(streams[0]):
        a = bs[1].call(B, 0, 0)
    streams[0].synchronize()
    assert torch.equal(a[0], want[1][0])


@pytest.mark.parametrize("fp4", [False, True])
def test_decode_steps_replay_from_a_graph(B, fp4):
    """Plan, append and attention of a decode step captured once; the lengths grow with every replay, past
    page and tile borders, and every step agrees with the oracle on the rows so far."""
    import torch
    rng = np.random.default_rng(3)
    n, hq, hkv, dim, ps, ppr, steps = 3, 4, 2, 64, 16, 24, 150
    start = np.array([0, 100, 250])
    table, free, head = i32(np.full((n, ppr), -1)), i32(rng.permutation(n * ppr)), i32([0])
    past, new = i32(np.zeros(n)), i32(start)
    s = n * ppr * ps
    dt = torch.bfloat16
    caches = ([torch.zeros((s, hkv, w), dtype=torch.uint8, device="cuda") for w in (dim // 2, dim // 16) * 2] if fp4 else
              [torch.zeros((s, hkv, dim), dtype=dt, device="cuda") for _ in range(2)])
    rope = B.rope_table(dim, 10000.0)

    def step(qkv, plan):
        q, k, v = (t.unflatten(1, (-1, dim)) for t in qkv.split([hq * dim, hkv * dim, hkv * dim], 1))
        if fp4:
            kc, ks, vc, vs = caches
            q = B.rope_append_fp4(q, k, v, kc, ks, vc, vs, plan.positions, plan.slots, rope)
            return q, B.window_attention_fp4_paged(q, kc, ks, vc, vs, plan.cu_seqlens_q, plan.kv_lens, table, ps, 0.125,
                                                   window=120, n_sink=3)
        q = B.rope_append(q, k, v, *caches, plan.positions, plan.slots, rope)
        return q, B.window_attention_paged(q, *caches, plan.cu_seqlens_q, plan.kv_lens, table, ps, 0.125, window=120,
                                           n_sink=3)

    width = (hq + 2 * hkv) * dim
    plan = B.page_plan(past, new, table, free, head, ps, int(start.sum()), free_head_out=head)     # the prompts
    step(torch.randn((int(start.sum()), width), device="cuda").to(dt), plan)
    past.copy_(plan.kv_lens)
    new.fill_(1)
    qkv = torch.randn((n, width), device="cuda").to(dt)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):                     # opt-ins outside the capture, on tables of their own
        t2, h2 = table.clone(), head.clone()
        B.page_plan(past, new, t2, free, h2, ps, n, free_head_out=h2)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan = B.page_plan(past, new, table, free, head, ps, n, free_head_out=head)
        q, (out, lse) = step(qkv, plan)
        past.copy_(plan.kv_lens)
    for t in range(steps):
        qkv.copy_(torch.from_numpy(rng.standard_normal((n, width))).to(dt))
        g.replay()
        torch.cuda.synchronize()
        assert B.device_status() == 0 and int(plan.shortfall) == 0
        if t % 29 and t != steps - 1:
            continue
        b = Batch.__new__(Batch)
        b.dt, b.dim, b.ps, b.fp4, b.scale = dt, dim, ps, fp4, 0.125
        b.cu, b.kv, b.table = np.arange(n + 1), start + t + 1, table.cpu().numpy()
        assert np.array_equal(plan.kv_lens.cpu().numpy(), b.kv)
        b.q64 = q.double().cpu().numpy()
        c = [x.cpu().numpy() if fp4 else x.double().cpu().numpy() for x in caches]
        b.k64, b.v64 = (S.fp4_values(c[0], c[1], 1.0), S.fp4_values(c[2], c[3], 1.0)) if fp4 else c
        b.compare(out, lse, 120, 3)


def test_prefill_and_decode_agree_with_dense_attention(B):
    """Prompt rows fed in chunks through plan, append and attention give what dense causal attention of the
    rotated rows gives; the last rows fed one by one give the same again."""
    import torch
    rng = np.random.default_rng(5)
    hq, hkv, dim, ps, n = 4, 2, 128, 32, 400
    q, k, v = (torch.from_numpy(rng.standard_normal((n, h, dim))).bfloat16().cuda() for h in (hq, hkv, hkv))
    w, mag = S.rope_frequencies(64, 10000.0)
    qr, kr = (S.rope(x.double().cpu().numpy(), np.arange(n), w, mag, True, 32) for x in (q, k))
    rope = B.rope_table(64, 10000.0)
    table, free, head = i32(np.full((1, 16), -1)), i32(rng.permutation(16)), i32([0])
    kc, vc = (torch.full((16 * ps, hkv, dim), float("nan"), device="cuda").bfloat16() for _ in range(2))
    rows, at = [], 0
    for m in [1, 150, 37, 200] + [1] * 12:
        plan = B.page_plan(i32([at]), i32([m]), table, free, head, ps, m, free_head_out=head)
        s = slice(at, at + m)
        x = B.rope_append(q[s], k[s], v[s], kc, vc, plan.positions, plan.slots, rope, layout="interleaved", rot_offset=32)
        out, lse = B.window_attention_paged(x, kc, vc, plan.cu_seqlens_q, plan.kv_lens, table, ps, dim ** -0.5)
        rows.append(out)
        at += m
    got = torch.cat(rows).double().cpu().numpy()
    vd = v.double().cpu().numpy()
    s = np.einsum("rhd,jhd->hrj", qr, np.repeat(kr, 2, 1)) * dim ** -0.5
    s = np.where(np.tril(np.ones((n, n), bool)), s, -np.inf)
    e = np.exp(s - s.max(-1, keepdims=True))
    e /= e.sum(-1, keepdims=True)
    want = np.einsum("hrj,jhd->rhd", e, np.repeat(vd, 2, 1))
    a = np.einsum("hrj,jhd->rhd", e, np.repeat(np.abs(vd), 2, 1))
    # weights, output, and q and k rounded to bf16 (half a step 2^-8 each): the latter move a logit by at most
    # 2 * 2^-8 sum |q k| scale, with sum |q k| scale <= 0.64 sqrt(dim) on average for N(0, 1) rows, taken twofold
    u = 2.0 ** -8
    bound = u * a + u * np.abs(want) + 2 * (2 * u * 2 * 0.64 * np.sqrt(dim)) * a
    assert np.all(np.abs(got - want) <= bound)


def test_stalled_call_times_out_and_the_context_recovers(B):
    import time
    import torch
    for lens in ([(700, 1)], [(3000, 2500)]):                # equal shares, whole units
        b = Batch(lens, 4, 4, 128, 64)
        B.debug_stall_next_call()
        t0 = time.time()
        b.call(B, 0, 0)
        torch.cuda.synchronize()
        assert B.device_status() == 0x142                    # the wait for a unit's record
        assert 1.0 < time.time() - t0 < 20.0
        b.check(B, 0, 0, rows=range(0, b.R, 97))


def test_a_unit_that_takes_longer_than_the_least_limit_of_waits(B):
    """600 million positions, all on one page, dealt out whole beside 1100 short requests: some waits last as long as that
    unit, some seconds, and none of them may be taken for a stall.  (Its own sums are beyond what fp32 can
    add up one by one and are not looked at.)"""
    import torch
    rng = np.random.default_rng(2)
    n, ps, D = 1100, 1 << 16, 64
    kv = rng.integers(1, 200, n)
    kv[0] = 600_000_000
    table = np.zeros((n, -(-int(kv[0]) // ps)), np.int64)
    q = torch.randn((n, 1, D), device="cuda").bfloat16()
    k, v = (torch.randn((ps, 1, D), device="cuda").bfloat16() for _ in range(2))
    assert B.window_workspace_bytes(n, n, table.shape[1], ps, 1, 1, D, 0, 0, num_sms=152) == 0      # whole units
    out, lse = B.window_attention_paged(q, k, v, i32(np.arange(n + 1)), i32(kv), i32(table), ps, D ** -0.5)
    torch.cuda.synchronize()
    assert B.device_status() == 0 and bool(out.isfinite().all()) and bool(lse.isfinite().all())
    b = Batch.__new__(Batch)
    b.dt, b.dim, b.ps, b.fp4, b.scale = torch.bfloat16, D, ps, False, D ** -0.5
    b.cu, b.kv, b.table = np.arange(n + 1), kv, table
    b.q64, b.k64, b.v64 = (x.double().cpu().numpy() for x in (q, k, v))
    b.compare(out, lse, 0, 0, rows=range(1, n, 31))
