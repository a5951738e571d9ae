"""Long contexts over paged caches, against their float64 restatements: more cases (GPU only)."""
import numpy as np
import pytest

from oracle import serving as S
from test_paged_context import Batch, check_prefix, check_select, f64, finished, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from top_sparse_attention_row_gb300 import build, binding
    build.build()
    binding.load_library()
    return binding


# ------------------------------------------------------------------------------ scores that are not finite
@pytest.mark.parametrize("value", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 8, 12, 16])
def test_select_of_zero_queries_over_bounds_that_are_not_finite(B, group, value):
    """Zero times such a bound is NaN: its page comes first, the others are equal, and the row's own page is there.  (A
    zero takes the lower bound, so an infinite upper one alone leaves the score 0.)"""
    b = Batch([(96, 3), (500, 2), (90, 1)], 2 * group, 2, 64, 8, "float16", seed=group)
    bounds = b.bounds()
    b.q[:4] = 0
    for i, pages in ((0, (3, 7, 10)), (1, (2, 40, 61)), (2, (0,))):
        for n, e in enumerate(pages):
            bounds[b.table[i, e], :, n % 2, 5 + n] = float(value)
    for n_select, first, last in ((10, 0, 1), (11, 1, 2), (4, 0, 1)):
        got = check_select(B, b, bounds, n_select, first, last)
        own = np.array([11, 11, 11, 62, 62, 11])
        assert (got == own[:, None, None]).any(-1).all()


@pytest.mark.parametrize("group", [1, 3, 8, 12])
def test_select_of_queries_that_are_not_finite(B, group):
    """NaN and infinities in one head's query, bounds of zeros among the others."""
    b = Batch([(300, 4), (96, 2)], group, 1, 128, 8, seed=group)
    bounds = b.bounds()
    b.q[0, group - 1, 7] = float("nan")
    b.q[1, 0, 9] = float("inf")
    b.q[2, 0, 9] = float("-inf")
    bounds[b.table[0, 5:20]] = 0
    check_select(B, b, bounds, 9, 1, 1)
    bounds[:] = 0                                          # 0 times infinity everywhere
    check_select(B, b, bounds, 9, 1, 1)


# ------------------------------------------------------------------------------ requests without rows
@pytest.mark.parametrize("kv", [0, 100, 700])
def test_prefix_group_that_begins_with_a_request_without_rows(B, kv):
    """Such a request has no part in its group: it may have ended, its pages gone to others or not in its table at all."""
    lens = [(kv, 0)] + [(512 + 3 + 20 * i, 1) for i in range(6)] + [(0, 0), (512 + 90, 2)]
    b = Batch(lens, 8, 2, 128, 16, seed=kv, share=[None, None] + [(1, 512)] * 5 + [None, (1, 512)])
    assert kv > 0 or (b.table[0] == -1).all()
    check_prefix(B, b, [0, 9], [512])
    check_prefix(B, b, [0, 1, 9], [512, 512])              # a group of that request alone
    check_prefix(B, b, [7, 9], [512])


# ------------------------------------------------------------------------------ large batches
def check_select_rows(B, b, rows, n_select, first, last):
    """As check_select, for some of the rows: each as a request of one row."""
    bounds = b.bounds()
    got = B.page_select(b.q, bounds, *b.batch(), n_select, n_first=first, n_last=last)
    finished(B)
    req = np.searchsorted(b.cu, rows, side="right") - 1
    kv = b.kv[req] - (b.cu[req + 1] - rows) + 1
    want = S.page_select(f64(b.q[rows]), f64(bounds), np.arange(len(rows) + 1), kv, b.table[req], b.ps, n_select, first, last)
    got = got.cpu().numpy()[rows]
    assert np.array_equal(got, want), rows[np.unique(np.argwhere((got != want).any(-1))[:, 0])]


@pytest.mark.parametrize("hq,hkv,dim,dtype,lens", [
    (64, 8, 64, "bfloat16", [(2400, 900), (1900, 600)]),   # up to 300 pages: three tiles of them to an item
    (48, 4, 256, "bfloat16", [(6000, 1300), (5000, 700)]),   # 750 pages, six tiles an item
    (32, 2, 128, "float16", [(16000, 1600)]),              # 2000 pages in runs of three tiles, the last one shorter
    (12, 1, 64, "float16", [(4096, 2500)]),                # 512 pages, the most of a warp with 16 keys a lane
    (8, 2, 64, "bfloat16", [(8192, 1300), (8000, 30)]),    # 1024 pages, the most of a warp
])
def test_select_large_batches(B, hq, hkv, dim, dtype, lens):
    b = Batch(lens, hq, hkv, dim, 8, dtype, seed=hq + dim)
    rows = np.unique(np.concatenate([np.linspace(0, b.R - 1, 40).astype(int), b.cu[:-1], b.cu[1:] - 1]))
    check_select_rows(B, b, rows, 29, 1, 2)


def test_prefix_of_very_many_tiles(B):
    """More tiles than are listed by a warp each: several groups, requests between and behind them, 64 heads a KV head."""
    starts, prefix = [2, 12, 12, 25, 31], [512, 512, 256, 1024]
    lens, share = [], []
    for i in range(34):
        g = next((g for g in range(4) if starts[g] <= i < starts[g + 1]), None)
        p = prefix[g] if g is not None else 0
        new = 1 + 37 * i % 130
        lens.append((p + new + 5 * i, new))
        share.append(None if g is None or i == starts[g] else (starts[g], p))
    b = Batch(lens, 64, 1, 64, 16, seed=3, share=share)
    assert 2 * (b.R // 2) + 4 + 34 > 2048                  # two tokens a tile, of the groups and of the requests
    got = B.prefix_attention_paged(b.q, b.k, b.v, *b.batch(), b.scale, i32(starts), i32(prefix))
    finished(B)
    rows = np.unique(np.concatenate([np.arange(0, b.R, 23), b.cu[:-1], b.cu[1:] - 1]))
    o, z = S.window_attention(f64(b.q), f64(b.k), f64(b.v), *b.host(), b.scale, rows=rows)
    a, _ = S.window_attention(f64(b.q), f64(b.k), np.abs(f64(b.v)), *b.host(), b.scale, rows=rows)
    b.compare(got, o, z, a, rows)
