"""Long contexts over paged caches, against their float64 restatements: more cases (GPU only)."""
import numpy as np
import pytest

from test_paged_context import Batch, check_prefix, check_select

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
