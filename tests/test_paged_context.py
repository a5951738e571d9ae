"""Long contexts over paged caches: bounds of pages, pages chosen by them, attention over chosen pages and behind shared
prompts, against their float64 restatements (GPU only)."""
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


def f64(t):
    return t.double().cpu().numpy()


class Batch:
    """A ragged batch over a shuffled paged cache: lens = [(kv_len, new rows)]; share[i] = (request, positions)
    whose first pages request i shares."""

    def __init__(self, lens, hq, hkv, dim, ps, dtype="bfloat16", seed=0, pad_rows=0, extra_pages=3, share=None, wide=0):
        import torch
        rng = np.random.default_rng(seed)
        self.rng, self.dt, self.ps, self.dim, self.hq, self.hkv = rng, getattr(torch, dtype), ps, dim, hq, hkv
        self.kv = np.array([a for a, _ in lens])
        self.cu = np.concatenate([[0], np.cumsum([b for _, b in lens])])
        self.R = int(self.cu[-1]) + pad_rows
        held = [max(0, -(-a // ps)) for a, _ in lens]
        self.n_pages = sum(held) + extra_pages
        pages = rng.permutation(self.n_pages)
        self.table = np.full((len(lens), max(1, max(held)) + wide), -1)
        at = 0
        for i, n in enumerate(held):
            self.table[i, :n] = pages[at:at + n]
            at += n
            if share and share[i]:
                j, m = share[i]
                self.table[i, :m // ps] = self.table[j, :m // ps]
        s = self.n_pages * ps
        self.to = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(self.dt).cuda()  # noqa: E731
        self.q = self.to(rng.standard_normal((self.R, hq, dim)))
        self.k, self.v = (self.to(x) for x in rng.standard_normal((2, s, hkv, dim)))
        self.scale = dim ** -0.5

    def batch(self):
        return i32(self.cu), i32(self.kv), i32(self.table), self.ps

    def host(self):
        return self.cu, self.kv, self.table, self.ps

    def bounds(self):
        """Bounds of all pages, as if they had been filled."""
        pages = f64(self.k).reshape(self.n_pages, self.ps, self.hkv, self.dim)
        return self.to(np.stack((pages.min(1), pages.max(1)), 2))

    def lists(self, n, k=6, seed=0):
        """Lists of up to k different pages, in any order, some of them beyond the row or missing."""
        rng = np.random.default_rng(seed)
        out = np.full((self.R, self.hkv, n), -1)
        for r in range(self.R):
            for h in range(self.hkv):
                m = min(k, n, self.table.shape[1] + 1)
                at = rng.choice(n, size=m, replace=False)
                out[r, h, at] = rng.choice(self.table.shape[1] + 1, size=m, replace=False)
        return out

    def compare(self, got, want_o, want_lse, abs_o, rows=None):
        """abs_o: the output with |v| in place of v.  With u the type's half step and A = sum w |v| / l:
        weights and output are rounded, u A + u |O|.  A logit is a sum of dim products in fp32, off by at most
        dim 2^-23 sum |q k| scale =: d (N(0, 1) rows: sum |q k| scale <= 2 sqrt(dim) here), which changes a weight
        by e^d and the sum likewise: 2 d A.  Parts of a row joined in fp32 add 2^-20 A."""
        import torch
        n = int(self.cu[-1])
        rows = np.arange(n) if rows is None else rows
        o, z = f64(got[0])[rows], f64(got[1])[rows]
        wo, wz, a = want_o[rows], want_lse[rows], abs_o[rows]
        assert np.array_equal(np.isneginf(z), np.isneginf(wz))
        u = torch.finfo(self.dt).eps / 2
        d = self.dim * 2.0 ** -23 * 2 * np.sqrt(self.dim) + 2.0 ** -20
        worst = np.max(np.abs(o - wo) - (u * a + u * np.abs(wo) + 2 * d * a + 2.0 ** -24), initial=-1)
        assert worst <= 0, worst
        fin = np.isfinite(wz)
        assert np.all(np.abs(z[fin] - wz[fin]) <= d + 2.0 ** -21 * np.abs(wz[fin]) + 2.0 ** -22)


def finished(B):
    import torch
    torch.cuda.synchronize()
    assert B.device_status() == 0


RAGGED = [(5, 5), (300, 40), (513, 1), (257, 130), (64, 64), (3, 3), (40, 2), (129, 0), (1, 1)]


# ------------------------------------------------------------------------------ bounds
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("ps", [1, 7, 16, 64, 256])
def test_bounds(B, ps, dim, dtype):
    import torch
    b = Batch(RAGGED, 2, 2, dim, ps, dtype, seed=ps + dim)
    before = b.to(b.rng.standard_normal((b.n_pages, 2, 2, dim)))
    bounds = before.clone()
    assert B.page_bounds(b.k, *b.batch(), bounds) is bounds
    torch.cuda.synchronize()
    want = S.page_bounds(f64(b.k), *b.host(), f64(before))
    assert np.array_equal(f64(bounds), want)
    B.page_bounds(b.k, *b.batch(), bounds)                 # again, with the same result
    assert np.array_equal(f64(bounds), want)


def test_bounds_of_rows_that_do_not_begin_at_zero(B):
    """The first rows of the batch belong to no request: no page but the requests' own is touched, the ones that stand
    before the table's first row among them."""
    import torch
    b = Batch([(40, 20), (100, 30)], 4, 2, 64, 16, seed=4, extra_pages=40)
    wide = b.table.shape[1]
    ahead = np.setdiff1d(np.arange(b.n_pages), b.table)[:4 * wide].reshape(-1, wide)   # pages of nobody
    table = i32(np.concatenate([ahead, b.table]))[len(ahead):]
    cu, kv = i32(b.cu + 70), i32(b.kv)
    mark = torch.full((b.n_pages, 2, 2, 64), 9, dtype=b.dt, device="cuda")
    want = B.page_bounds(b.k, i32(b.cu), kv, table, 16, mark.clone())
    got = B.page_bounds(b.k, cu, kv, table, 16, mark.clone())
    finished(B)
    assert torch.equal(got, want)
    assert bool((got[torch.from_numpy(ahead).flatten().long().cuda()] == 9).all())


def test_bounds_of_missing_pages_short_tables_and_short_lengths(B):
    b = Batch([(200, 70), (90, 3), (64, 100), (0, 4), (0, 0), (50, 0)], 1, 1, 64, 16, seed=5)
    b.table[0, 9], b.table[1, 5] = -1, b.n_pages           # missing and out of range
    table = b.table[:, :11]                                # the first request has 13 pages
    before = b.to(b.rng.standard_normal((b.n_pages, 1, 2, 64)))
    bounds = before.clone()
    B.page_bounds(b.k, i32(b.cu), i32(b.kv), i32(table), 16, bounds)
    assert np.array_equal(f64(bounds), S.page_bounds(f64(b.k), b.cu, b.kv, table, 16, f64(before)))


def test_bounds_keep_nan_and_infinities(B):
    import torch
    b = Batch([(40, 40)], 1, 1, 64, 16, seed=6)
    b.k[b.table[0, 1] * 16 + 3, 0, 5] = float("nan")
    b.k[b.table[0, 2] * 16 + 1, 0, 6] = float("-inf")
    b.k[b.table[0, 2] * 16 + 9, 0, 7] = float("nan")       # position 41: not filled
    bounds = torch.zeros((b.n_pages, 1, 2, 64), dtype=b.dt, device="cuda")
    B.page_bounds(b.k, *b.batch(), bounds)
    got = f64(bounds)[b.table[0, :3], 0]
    assert np.isnan(got).sum() == 2 and np.isnan(got[1, :, 5]).all()
    assert np.isneginf(got[2, 0, 6]) and np.isfinite(got[2, 1]).all()


def test_bounds_of_many_requests(B):
    b = Batch([(1 + 5 * i % 90, 1) for i in range(700)], 1, 1, 64, 16, seed=7)
    before = b.to(b.rng.standard_normal((b.n_pages, 1, 2, 64)))
    bounds = before.clone()
    B.page_bounds(b.k, *b.batch(), bounds)
    assert np.array_equal(f64(bounds), S.page_bounds(f64(b.k), *b.host(), f64(before)))


# ------------------------------------------------------------------------------ choice
def check_select(B, b, bounds, n_select, first=1, last=1, **kw):
    import torch
    out = torch.full((b.R, b.hkv, n_select), -2, dtype=torch.int32, device="cuda")
    got = B.page_select(b.q, bounds, *b.batch(), n_select, n_first=first, n_last=last, out=out, **kw)
    assert got is out
    finished(B)
    want = S.page_select(f64(b.q), f64(bounds), *b.host(), n_select, first, last)
    got = out.cpu().numpy()
    assert np.array_equal(got, want), np.argwhere((got != want).any(-1))[:5]
    return got


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n_select,first,last", [(1, 0, 1), (5, 1, 2), (12, 2, 1), (64, 0, 1)])
def test_select(B, dim, n_select, first, last, dtype):
    b = Batch(RAGGED, 6, 2, dim, 8, dtype, seed=dim + n_select, pad_rows=3)
    check_select(B, b, b.bounds(), n_select, first, last)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (24, 2), (8, 8), (40, 5), (128, 1), (66, 2)])
def test_select_head_groups(B, hq, hkv):
    b = Batch([(400, 37), (90, 1), (700, 1)], hq, hkv, 64, 16, seed=hq)
    check_select(B, b, b.bounds(), 7, 1, 2)


@pytest.mark.parametrize("ps", [1, 3, 24, 100])
def test_select_page_sizes(B, ps):
    b = Batch([(600, 9), (90, 90)], 4, 2, 64, ps, seed=ps)
    check_select(B, b, b.bounds(), 6, 1, 1)


def test_select_equal_scores_go_to_the_lower_page(B):
    """Pages of equal bounds, many of them, among others; q of zeros makes all scores equal."""
    b = Batch([(1000, 5), (800, 1)], 4, 1, 64, 8, seed=1)
    bounds = b.bounds()
    bounds[b.rng.permutation(b.n_pages)[:150]] = bounds[0].clone()
    check_select(B, b, bounds, 20)
    b.q[:] = 0
    check_select(B, b, bounds, 20)
    b.q[:] = -b.q                                          # (-0)
    check_select(B, b, bounds, 20)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_select_decides_scores_that_32_bits_cannot_part(B, dtype):
    """All scores agree in 14 or more bits: one dim carries the same large bound everywhere, the others differ by
    multiples of 2^-10 and less, so that any rounding of a sum would change the order."""
    b = Batch([(1500, 4), (1024, 1)], 4, 2, 128, 8, dtype, seed=2)
    bounds = b.bounds() * 2.0 ** -8
    bounds[..., 17] = 8192.0
    b.q[:, :, 17] = 31.0
    check_select(B, b, bounds, 33)


def test_select_cancelling_sums(B):
    """Large products of both signs that cancel, in the first and the last dims."""
    b = Batch([(1500, 4)], 3, 1, 256, 8, seed=3)
    bounds = b.bounds()
    b.q[..., 0], b.q[..., 255] = 64.0, 64.0
    bounds[..., 0], bounds[..., 255] = 2.0 ** 14, -2.0 ** 14
    check_select(B, b, bounds, 33)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("dim", [64, 256])
def test_select_bounds_of_many_magnitudes(B, dim, dtype):
    """Dims that reach from 2^-12 to 2^12: the products' fp32 sums are furthest off here."""
    import torch
    b = Batch([(3000, 6), (2048, 1)], 6, 1, dim, 8, dtype, seed=dim)
    s = torch.exp2(torch.from_numpy(b.rng.integers(-12, 12, (b.n_pages, 1, 1, dim))).float()).cuda().to(b.dt)
    check_select(B, b, b.bounds() * s, 60)


def test_select_scores_beyond_fp32(B):
    """Sums that overflow fp32 are compared in 64 bits like any other."""
    b = Batch([(500, 4)], 3, 1, 64, 8, seed=4)
    bounds = b.bounds() * 2.0 ** 100
    b.q[:] = b.q * 2.0 ** 100
    check_select(B, b, bounds, 9)
    b.q[..., 0], b.q[..., 63] = 2.0 ** 120, 2.0 ** 120     # cancels
    bounds[..., 0], bounds[..., 63] = 2.0 ** 120, -2.0 ** 120
    check_select(B, b, bounds, 9)


def test_select_nan_scores_come_first(B):
    b = Batch([(500, 2)], 2, 1, 64, 8, seed=5)
    bounds = b.bounds()
    bounds[b.table[0, 7], 0, 1, 3] = float("nan")
    bounds[b.table[0, 30], 0, 0, 3] = float("nan")
    b.q[..., 3] = 1.0                                      # takes the upper bounds of this dim
    bounds[b.table[0, 30], 0, 1, 3] = 0.5
    got = check_select(B, b, bounds, 3, 0, 1)
    assert (got[..., 0] == 7).all()


def test_select_missing_pages_short_tables_and_rows_before_the_start(B):
    b = Batch([(300, 20), (90, 3), (10, 30), (0, 2)], 4, 2, 64, 16, seed=6)
    b.table[0, 3], b.table[0, 0], b.table[1, 5], b.table[0, 18] = -1, -7, b.n_pages, -1
    check_select(B, b, b.bounds(), 6, 2, 2)
    b.table = np.ascontiguousarray(b.table[:, :11])        # the rows' own pages are past the table
    check_select(B, b, b.bounds(), 6, 2, 2)


@pytest.mark.parametrize("n", [1, 2, 33, 255, 1000, 4000])
def test_select_context_lengths(B, n):
    b = Batch([(8 * n - 3, 1), (8, 1), (8 * n // 2 + 5, 1)], 2, 1, 64, 8, seed=n)
    check_select(B, b, b.bounds(), 19, 1, 3)


def test_select_long_tables(B):
    """As many pages as a request may have."""
    b = Batch([(32768, 1), (31000, 2)], 2, 1, 64, 1, seed=8)
    check_select(B, b, b.bounds(), 40)


def test_select_many_rows(B):
    b = Batch([(700, 600), (900, 333)], 8, 2, 64, 16, seed=9)
    check_select(B, b, b.bounds(), 9, 1, 2)


# ------------------------------------------------------------------------------ attention over chosen pages
def check_selected(B, b, lists, **kw):
    got = B.selected_attention_paged(b.q, b.k, b.v, i32(lists), *b.batch(), b.scale, **kw)
    finished(B)
    args = (lists, *b.host(), b.scale)
    o, z = S.selected_attention(f64(b.q), f64(b.k), f64(b.v), *args)
    a, _ = S.selected_attention(f64(b.q), f64(b.k), np.abs(f64(b.v)), *args)
    b.compare(got, o, z, a)
    return got


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("ps", [8, 16, 24, 64, 128])
def test_selected(B, ps, dim, dtype):
    b = Batch(RAGGED, 6, 2, dim, ps, dtype, seed=ps + dim)
    check_selected(B, b, b.lists(9, seed=ps))


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (24, 2), (8, 8), (40, 5), (128, 1), (66, 2)])
def test_selected_head_groups(B, hq, hkv):
    b = Batch([(400, 37), (90, 1), (700, 1)], hq, hkv, 64, 16, seed=hq)
    check_selected(B, b, b.lists(11, 9, seed=hq))


@pytest.mark.parametrize("dim", [64, 256])
@pytest.mark.parametrize("n", [1, 2, 7, 50])
def test_selected_decode(B, n, dim):
    b = Batch([(1 + (977 * i) % 3000, 1) for i in range(n)], 12, 2, dim, 64, seed=n)
    check_selected(B, b, b.lists(20, 16, seed=n))


def test_selected_all_pages_is_full_attention(B):
    b = Batch(RAGGED, 8, 2, 128, 16, seed=1)
    lists = np.broadcast_to(np.arange(b.table.shape[1]), (b.R, 2, b.table.shape[1]))
    got = check_selected(B, b, lists)
    full = B.window_attention_paged(b.q, b.k, b.v, *b.batch(), b.scale)
    assert (got[0].float() - full[0].float()).abs().max() <= 2.0 ** -6


def test_selected_repeated_future_and_missing_pages(B):
    """A page that is listed twice counts once; pages past the row, past the table and without an id count nothing."""
    b = Batch([(300, 50), (100, 1), (20, 33)], 4, 2, 64, 16, seed=2)
    lists = b.lists(12, 8, seed=2)
    lists[::3, 0, :6] = lists[::3, 0, 6:]                  # twice
    lists[1::3, 1, 0] = 2 ** 31 - 1
    lists[2::3, 1, 1] = -2 ** 31
    lists[5, :] = -1                                       # nothing listed
    lists[7, :] = b.table.shape[1] - 1                     # only the last page, which the row may not reach
    b.table[0, 4], b.table[0, 9] = -1, b.n_pages
    got = check_selected(B, b, lists)
    assert (got[0][5] == 0).all() and (got[1][5] == float("-inf")).all()


def test_selected_ignores_what_it_does_not_see(B):
    """NaN in pages that no row lists, in the rest of a row's last page and behind it."""
    b = Batch([(150, 1), (90, 1)], 4, 1, 128, 16, seed=3)
    lists = np.full((2, 1, 4), -1)
    lists[0, 0, :3], lists[1, 0, :2] = [0, 4, 9], [5, 1]
    seen = np.zeros(b.n_pages * 16, dtype=bool)
    for r, kv in enumerate(b.kv):
        for e in lists[r, 0]:
            n = min(16, kv - e * 16) if e >= 0 else 0
            seen[b.table[r, e] * 16:b.table[r, e] * 16 + n] = True
    want = check_selected(B, b, lists)
    for t in (b.k, b.v):
        t[i32(np.flatnonzero(~seen)).long()] = float("nan")
    got = B.selected_attention_paged(b.q, b.k, b.v, i32(lists), *b.batch(), b.scale)
    assert (got[0] == want[0]).all() and (got[1] == want[1]).all()


def test_selected_leaves_rows_behind_the_last_request(B):
    import torch
    b = Batch([(300, 20), (50, 1)], 4, 2, 64, 16, seed=4, pad_rows=30)
    out = torch.full_like(b.q, 7.0)
    lse = torch.full((b.R, 4), 7.0, device="cuda")
    got = check_selected(B, b, b.lists(5, seed=4), out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    assert (out[21:] == 7).all() and (lse[21:] == 7).all()
    assert B.selected_attention_paged(b.q, b.k, b.v, i32(b.lists(5, seed=4)), *b.batch(), b.scale, want_lse=False)[1] is None


def test_selected_many_rows(B):
    """Units for all SMs, which are dealt out whole; neighbouring rows list much the same pages."""
    b = Batch([(2500, 2400), (900, 700)], 4, 2, 64, 16, seed=12)
    lists = np.sort(b.rng.integers(0, 57, (b.R // 50 + 1, 2, 12)), -1).repeat(50, 0)[:b.R]
    moved = b.rng.random(lists.shape) < 0.05
    lists = np.where(moved, b.rng.integers(-1, 160, lists.shape), lists)
    got = B.selected_attention_paged(b.q, b.k, b.v, i32(lists), *b.batch(), b.scale)
    finished(B)
    for cut in (slice(0, 60), slice(1200, 1260), slice(2390, 2460), slice(3050, 3100)):
        rows = np.arange(cut.start, cut.stop)
        args = (lists, *b.host(), b.scale, rows)
        o, z = S.selected_attention(f64(b.q), f64(b.k), f64(b.v), *args)
        a, _ = S.selected_attention(f64(b.q), f64(b.k), np.abs(f64(b.v)), *args)
        b.compare(got, o, z, a, rows)


# ------------------------------------------------------------------------------ shared prompts
def check_prefix(B, b, groups, prefix, **kw):
    got = B.prefix_attention_paged(b.q, b.k, b.v, *b.batch(), b.scale, i32(groups), i32(prefix), **kw)
    finished(B)
    o, z = S.window_attention(f64(b.q), f64(b.k), f64(b.v), *b.host(), b.scale)
    a, _ = S.window_attention(f64(b.q), f64(b.k), np.abs(f64(b.v)), *b.host(), b.scale)
    b.compare(got, o, z, a)
    return got


def shared(n, prefix, own, hq, hkv, dim, ps, dtype="bfloat16", seed=0, new=lambda i: 1, **kw):
    """n requests behind one prompt, with own(i) positions behind it, the last new(i) of them the step's."""
    lens = [(prefix + own(i), new(i)) for i in range(n)]
    return Batch(lens, hq, hkv, dim, ps, dtype, seed, share=[None] + [(0, prefix)] * (n - 1), **kw)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n,prefix,ps", [(1, 64, 16), (5, 512, 64), (30, 320, 16), (3, 2048, 128), (17, 21, 7)])
def test_prefix_decode(B, n, prefix, ps, dim, dtype):
    b = shared(n, prefix, lambda i: 1 + 37 * i % 200, 6, 2, dim, ps, dtype, seed=n + dim)
    check_prefix(B, b, [0, n], [prefix])


@pytest.mark.parametrize("dim", [64, 256])
def test_prefix_rows_of_all_lengths(B, dim):
    new = [1, 40, 130, 2, 300, 1, 0, 9]
    b = shared(8, 256, lambda i: new[i] + 11 * i, 8, 2, dim, 16, seed=dim, new=lambda i: new[i], pad_rows=5)
    check_prefix(B, b, [0, 8], [256])


def test_prefix_groups(B):
    """Several groups, one of a single request, one that shares nothing, requests before and behind them all."""
    starts, prefix = [1, 4, 5, 9, 9, 12], [48, 160, 0, 16, 320]
    lens, share = [], []
    for i in range(14):
        g = next((g for g in range(5) if starts[g] <= i < starts[g + 1]), None)
        p = prefix[g] if g is not None else 0
        lens.append((p + 1 + 29 * i, 1 + i % 3 * 7 if 1 + i % 3 * 7 <= 1 + 29 * i else 1))
        share.append(None if g is None or i == starts[g] or p == 0 else (starts[g], p))
    b = Batch(lens, 4, 2, 64, 16, seed=3, share=share)
    check_prefix(B, b, starts, prefix)


def test_prefix_longer_than_a_request_has(B):
    """What a request of the group does not have as past is not shared, whatever the length says."""
    b = shared(4, 128, lambda i: 1 + 50 * i, 4, 1, 64, 16, seed=4)
    check_prefix(B, b, [0, 4], [10 ** 6])                  # only 128 positions are past of all
    b.kv[2] = 100                                          # a request that ends inside the prompt
    check_prefix(B, b, [0, 4], [128])
    b.kv[1] = 0                                            # one without any: its row sees nothing
    got = check_prefix(B, b, [0, 4], [128])
    assert (got[0][1] == 0).all()
    check_prefix(B, b, [0, 4], [-5])


def test_prefix_without_groups(B):
    b = Batch(RAGGED, 4, 2, 64, 16, seed=5)
    check_prefix(B, b, [0], [])


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (24, 2), (8, 8), (128, 1), (66, 2)])
def test_prefix_head_groups(B, hq, hkv):
    b = shared(6, 192, lambda i: 5 + 40 * i, hq, hkv, 64, 16, seed=hq, new=lambda i: 1 + i)
    check_prefix(B, b, [0, 6], [192])


def test_prefix_missing_pages(B):
    b = shared(4, 256, lambda i: 1 + 50 * i, 4, 2, 64, 16, seed=6)
    b.table[:, 3] = -1                                     # a hole in the prompt
    b.table[2, 17] = b.n_pages
    check_prefix(B, b, [0, 4], [256])


def test_prefix_many_requests_and_long_prompts(B):
    b = shared(300, 1024, lambda i: 1 + i % 5, 2, 1, 64, 64, seed=7)
    check_prefix(B, b, [0, 300], [1024])
    b = shared(2, 20000, lambda i: 1 + i, 2, 1, 64, 16, seed=8)
    check_prefix(B, b, [0, 2], [20000])


def test_prefix_leaves_rows_behind_the_last_request(B):
    import torch
    b = shared(3, 64, lambda i: 9, 4, 2, 64, 16, seed=9, new=lambda i: 3, pad_rows=40)
    out, lse = torch.full_like(b.q, 7.0), torch.full((b.R, 4), 7.0, device="cuda")
    got = check_prefix(B, b, [0, 3], [64], out=out, lse=lse)
    assert got[0] is out and (out[9:] == 7).all() and (lse[9:] == 7).all()


@pytest.mark.parametrize("dim", [64, 128])
def test_prefix_many_rows(B, dim):
    """More rows than the join gives four warps each."""
    b = shared(8, 512, lambda i: 300 + 40 * i, 8, 2, dim, 16, seed=dim, new=lambda i: 260 + 5 * i)
    got = B.prefix_attention_paged(b.q, b.k, b.v, *b.batch(), b.scale, i32([0, 8]), i32([512]))
    finished(B)
    rows = np.arange(0, b.R, 41)
    o, z = S.window_attention(f64(b.q), f64(b.k), f64(b.v), *b.host(), b.scale, rows=rows)
    a, _ = S.window_attention(f64(b.q), f64(b.k), np.abs(f64(b.v)), *b.host(), b.scale, rows=rows)
    b.compare(got, o, z, a, rows)


# ------------------------------------------------------------------------------ together
def test_a_decode_step_over_chosen_pages(B):
    """Plan, rotation and write, bounds, choice, attention: prompts first, then decode steps, captured and replayed."""
    import torch
    hq, hkv, dim, ps, n, K = 8, 2, 128, 16, 3, 4
    rng = np.random.default_rng(11)
    rope = B.rope_table(dim)
    prompts = [130, 40, 77]
    table = i32(np.full((n, 16), -1))
    free, head = i32(rng.permutation(60)), i32([0])
    k, v = (torch.zeros((60 * ps, hkv, dim), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    bounds = torch.zeros((60, hkv, 2, dim), dtype=torch.bfloat16, device="cuda")
    past = i32([0] * n)

    def step(x, new, rows):
        plan = B.page_plan(past, new, table, free, head, ps, rows, free_head_out=head, kv_lens=past)
        q, kn, vn = x.split([hq, hkv, hkv], 1)
        q = B.rope_append(q, kn, vn, k, v, plan.positions, plan.slots, rope)
        batch = (plan.cu_seqlens_q, plan.kv_lens, table, ps)
        B.page_bounds(k, *batch, bounds)
        pages = B.page_select(q, bounds, *batch, K, n_first=1, n_last=1)
        return q, pages, *B.selected_attention_paged(q, k, v, pages, *batch, dim ** -0.5)

    def check(got, new, kv):
        q, pages, out, lse = got
        cu = np.concatenate([[0], np.cumsum(new)])
        host = (cu, np.array(kv), table.cpu().numpy(), ps)
        b = S.page_bounds(f64(k), *host, f64(bounds))
        assert np.array_equal(b, f64(bounds))
        want = S.page_select(f64(q), b, *host, K, 1, 1)
        assert np.array_equal(pages.cpu().numpy(), want)
        o, z = S.selected_attention(f64(q), f64(k), f64(v), want, *host, dim ** -0.5)
        assert np.max(np.abs(f64(out) - o)) <= 2.0 ** -6 and np.max(np.abs(f64(lse) - z)) <= 1e-4

    x = torch.from_numpy(rng.standard_normal((sum(prompts), hq + 2 * hkv, dim))).bfloat16().cuda()
    check(step(x, i32(prompts), sum(prompts)), prompts, prompts)
    x = torch.zeros((n, hq + 2 * hkv, dim), dtype=torch.bfloat16, device="cuda")
    one = i32([1] * n)
    step(x.normal_(), one, n)                              # (past is now prompts + 1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(x, one, n)
    for t in range(20):
        x.normal_()
        graph.replay()
        check(got, [1] * n, [p + 2 + t for p in prompts])
    finished(B)
