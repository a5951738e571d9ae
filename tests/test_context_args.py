"""Refusals and host-side parts of page bounds, page selection, attention over chosen pages and behind shared prompts
(no GPU needed)."""
import pytest

FAKE = 1 << 20          # 16-byte aligned stand-in for a device pointer, never read
OK, INVALID, UNSUPPORTED = 0, 1, 2


@pytest.fixture(scope="module")
def B():
    from top_sparse_attention_row_gb300 import build, binding
    build.build()
    binding.load_library()
    return binding


def args(defaults, kw):
    assert set(kw) <= set(defaults)
    return list({**defaults, **kw}.values())


def bounds_args(**kw):
    return args(dict(k=FAKE, cu=FAKE, kv=FAKE, table=FAKE, bounds=FAKE, n=4, ppr=8, ps=64, n_pages=32, hkv=2, dim=128,
                     dtype=0, stream=None), kw)


def select_args(**kw):
    return args(dict(q=FAKE, bounds=FAKE, cu=FAKE, kv=FAKE, table=FAKE, pages=FAKE, rows=8, n=4, ppr=8, ps=64, n_pages=32,
                     hq=8, hkv=2, dim=128, n_select=4, first=1, last=1, dtype=0, ws=None, ws_bytes=0, stream=None), kw)


def selected_args(**kw):
    return args(dict(q=FAKE, k=FAKE, v=FAKE, pages=FAKE, cu=FAKE, kv=FAKE, table=FAKE, out=FAKE, lse=FAKE, rows=8, n=4,
                     ppr=8, ps=64, n_pages=32, n_select=4, hq=8, hkv=2, dim=128, scale=0.1, dtype=0, ws=None, ws_bytes=0,
                     stream=None), kw)


def prefix_args(**kw):
    return args(dict(q=FAKE, k=FAKE, v=FAKE, cu=FAKE, kv=FAKE, table=FAKE, groups=FAKE, prefix=FAKE, out=FAKE, lse=FAKE,
                     rows=8, n=4, n_groups=2, ppr=8, ps=64, n_pages=32, hq=8, hkv=2, dim=128, scale=0.1, dtype=0, ws=None,
                     ws_bytes=0, stream=None), kw)


BATCH = [
    (dict(cu=None), INVALID), (dict(kv=None), INVALID), (dict(table=None), INVALID), (dict(n=0), INVALID),
    (dict(ppr=0), INVALID), (dict(ps=0), INVALID), (dict(n_pages=0), INVALID), (dict(hkv=0), INVALID),
    (dict(cu=FAKE + 2), INVALID), (dict(kv=FAKE + 1), INVALID), (dict(table=FAKE + 2), INVALID), (dict(dtype=2), INVALID),
    (dict(dim=96), UNSUPPORTED), (dict(dim=512), UNSUPPORTED), (dict(n_pages=1 << 26), UNSUPPORTED),
]
ROWS = [(dict(q=None), INVALID), (dict(q=FAKE + 8), INVALID), (dict(rows=-1), INVALID), (dict(hq=0), INVALID),
        (dict(hq=7), INVALID), (dict(hq=258), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED), (dict(rows=0), OK)]
CACHE = [(dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k=FAKE + 8), INVALID), (dict(v=FAKE + 8), INVALID),
         (dict(out=None), INVALID), (dict(out=FAKE + 8), INVALID), (dict(lse=FAKE + 2), INVALID), (dict(scale=0.0), INVALID),
         (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=3e38), INVALID)]


@pytest.mark.parametrize("kw,status", BATCH + [
    (dict(k=None), INVALID), (dict(bounds=None), INVALID), (dict(k=FAKE + 8), INVALID), (dict(bounds=FAKE + 2), INVALID)])
def test_page_bounds_refusals(B, kw, status):
    assert B.load_library().qsa_page_bounds(*bounds_args(**kw)) == status


@pytest.mark.parametrize("kw,status", BATCH + ROWS + [
    (dict(bounds=None), INVALID), (dict(pages=None), INVALID), (dict(bounds=FAKE + 8), INVALID),
    (dict(pages=FAKE + 2), INVALID), (dict(n_select=0), INVALID), (dict(first=-1), INVALID), (dict(last=0), INVALID),
    (dict(first=3, last=2), INVALID), (dict(first=2 ** 31 - 1, last=2 ** 31 - 1), INVALID),
    (dict(ppr=32769), UNSUPPORTED), (dict(rows=1 << 30), UNSUPPORTED)])
def test_page_select_refusals(B, kw, status):
    assert B.load_library().qsa_page_select(*select_args(**kw)) == status


@pytest.mark.parametrize("kw,status", BATCH + ROWS + CACHE + [
    (dict(pages=None), INVALID), (dict(pages=FAKE + 2), INVALID), (dict(n_select=0), INVALID),
    (dict(ps=12), UNSUPPORTED), (dict(ps=4), UNSUPPORTED), (dict(ppr=32769), UNSUPPORTED)])
def test_selected_attention_refusals(B, kw, status):
    assert B.load_library().qsa_selected_attention_paged(*selected_args(**kw)) == status


@pytest.mark.parametrize("kw,status", BATCH + ROWS + CACHE + [
    (dict(groups=None), INVALID), (dict(prefix=None), INVALID), (dict(groups=FAKE + 2), INVALID),
    (dict(prefix=FAKE + 1), INVALID), (dict(n_groups=-1), INVALID)])
def test_prefix_attention_refusals(B, kw, status):
    assert B.load_library().qsa_prefix_attention_paged(*prefix_args(**kw)) == status


def cpu_batch(n=2, ppr=3):
    import torch
    return torch.zeros(n + 1, dtype=torch.int32), torch.zeros(n, dtype=torch.int32), torch.zeros((n, ppr), dtype=torch.int32)


def test_binding_refuses_what_is_no_cuda_tensor(B):
    import torch
    h = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    cu, kv, table = cpu_batch()
    pages = torch.zeros((4, 1, 2), dtype=torch.int32)
    one = torch.zeros(1, dtype=torch.int32)
    calls = [lambda: B.page_bounds(h(64, 1, 64), cu, kv, table, 16, h(4, 1, 2, 64)),
             lambda: B.page_select(h(4, 2, 64), h(4, 1, 2, 64), cu, kv, table, 16, 2),
             lambda: B.selected_attention_paged(h(4, 2, 64), h(64, 1, 64), h(64, 1, 64), pages, cu, kv, table, 16, 1.0),
             lambda: B.prefix_attention_paged(h(4, 2, 64), h(64, 1, 64), h(64, 1, 64), cu, kv, table, 16, 1.0, cu[:2], one)]
    for c in calls:
        with pytest.raises(ValueError, match="CUDA"):
            c()


def test_binding_refuses_wrong_types_and_shapes(B):
    import torch
    h = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    cu, kv, table = cpu_batch()
    with pytest.raises(TypeError, match="bfloat16 or float16"):
        B.page_bounds(torch.zeros(64, 1, 64), cu, kv, table, 16, h(4, 1, 2, 64))
    with pytest.raises(ValueError, match="whole pages"):
        B.page_bounds(h(63, 1, 64), cu, kv, table, 16, h(4, 1, 2, 64))
    with pytest.raises(ValueError, match="bounds must have shape"):
        B.page_bounds(h(64, 1, 64), cu, kv, table, 16, h(3, 1, 2, 64))
    with pytest.raises(TypeError, match="bounds must be"):
        B.page_bounds(h(64, 1, 64), cu, kv, table, 16, h(4, 1, 2, 64).half())
    with pytest.raises(ValueError, match="bounds must have 4 dims"):
        B.page_select(h(4, 2, 64), h(4, 2, 64), cu, kv, table, 16, 2)
    with pytest.raises(ValueError, match="n_select"):
        B.page_select(h(4, 2, 64), h(4, 1, 2, 64), cu, kv, table, 16, 0)
    with pytest.raises(TypeError, match="kv_lens must be torch.int32"):
        B.page_select(h(4, 2, 64), h(4, 1, 2, 64), cu, kv.long(), table, 16, 2)
    with pytest.raises(ValueError, match="cu_seqlens_q must have shape"):
        B.page_select(h(4, 2, 64), h(4, 1, 2, 64), cu[:2], kv, table, 16, 2)
    k = h(64, 1, 64)
    with pytest.raises(ValueError, match="pages must have shape"):
        B.selected_attention_paged(h(4, 2, 64), k, k, torch.zeros((4, 2, 2), dtype=torch.int32), cu, kv, table, 16, 1.0)
    with pytest.raises(ValueError, match="cu_groups must have shape"):
        B.prefix_attention_paged(h(4, 2, 64), k, k, cu, kv, table, 16, 1.0, cu, torch.zeros(1, dtype=torch.int32))
    with pytest.raises(TypeError, match="v_cache must be"):
        B.prefix_attention_paged(h(4, 2, 64), k, k.half(), cu, kv, table, 16, 1.0, cu[:2], cu[:1])


def test_workspace_sizes(B):
    assert B.page_select_workspace_bytes(0, 1, 8, 8, 2, 128) == 0
    assert B.selected_workspace_bytes(0, 1, 8, 64, 4, 8, 2, 128, num_sms=152) == 0
    assert B.prefix_workspace_bytes(0, 1, 1, 8, 64, 8, 2, 128, num_sms=152) == 0
