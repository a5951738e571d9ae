"""The binding's sparse attention calls carry the rows of the caches they are given, so that the kernels' tensor maps end
where the caches end."""
import numpy as np
import pytest

SLOTS, HEADS = 4096, 2


@pytest.fixture
def calls(monkeypatch):
    """The binding over a library that records its calls' arguments (tensors of the meta device: no memory, no GPU)."""
    from top_sparse_attention_row_gb300 import binding
    seen = []

    class Library:
        def __getattr__(self, name):
            def entry(*args):
                seen.append((name, args))
                return 0
            return entry
    monkeypatch.setattr(binding, "load_library", lambda *a: Library())
    monkeypatch.setattr(binding, "_require", lambda *a, **k: None)
    monkeypatch.setattr(binding, "_stream_ptr", lambda s: 0)
    return binding, seen


def tensors(slots, heads, dim, rows=3, topk=128):
    import torch
    e = lambda *s, dt=torch.bfloat16: torch.empty(s, dtype=dt, device="meta")  # noqa: E731
    i = lambda *s: e(*s, dt=torch.int32)  # noqa: E731
    return e(rows, 4 if heads else 8, dim), e(*((slots, heads, dim) if heads else (slots, dim))), i(rows, topk), i


def call(B, name, slots, heads=HEADS, ps=64, **kw):
    mla = "mla" in name
    q, cache, idx, i = tensors(slots, 0 if mla else heads, 576 if mla else 256)
    args = [q, cache] if mla else [q, cache, cache]
    if "fp8" in name:
        args += [i(1), i(1), 128]
    args += [idx, None]
    if "paged" in name:
        args += [i(3), i(2), i(2, 8), ps]
    getattr(B, name)(*args, 0.1, **kw)


def count_of(name, entry, args):
    """The slots (paged: pages) among an entry's arguments."""
    if name == "sparse_prefill":
        return args[14] if entry == "qsa_sparse_prefill_ex" else 0
    if name == "sparse_prefill_fp8":
        return args[17]
    if name == "sparse_mla_prefill":
        return args[13]
    return args[{"sparse_prefill_paged": 14, "sparse_prefill_fp8_paged": 17, "sparse_mla_prefill_paged": 13}[name]]


NAMES = ["sparse_prefill", "sparse_prefill_fp8", "sparse_mla_prefill", "sparse_prefill_paged", "sparse_prefill_fp8_paged",
         "sparse_mla_prefill_paged"]


@pytest.mark.parametrize("name", NAMES)
def test_calls_carry_the_rows_of_their_caches(calls, name):
    B, seen = calls
    paged = "paged" in name
    for slots, kw, want in ((SLOTS, {}, SLOTS // 64 if paged else SLOTS),
                            (SLOTS, {"n_pages" if paged else "n_kv_slots": 9}, 9),
                            (SLOTS + 1, {}, 0 if paged else SLOTS + 1)):
        call(B, name, slots, **kw)
        (entry, args), = seen
        seen.clear()
        assert entry.startswith("qsa_" + name) and count_of(name, entry, args) == want


@pytest.mark.parametrize("name", NAMES)
def test_caches_that_the_library_does_not_count_stay_unchecked(calls, name):
    """2^31 - 1 rows (slot x KV head) and more were taken without a count before, and are."""
    B, seen = calls
    heads = 1 if "mla" in name else HEADS
    for slots, counted in ((2 ** 31 // heads, False), (2 ** 31 // heads - 64, True)):
        call(B, name, slots)
        (entry, args), = seen
        seen.clear()
        assert (count_of(name, entry, args) > 0) == counted


@pytest.mark.gpu
@pytest.mark.parametrize("mla", [False, True])
@pytest.mark.parametrize("union_g", [0, 4])
def test_slots_behind_the_cache_are_padding(mla, union_g):
    """As -1 in their place, in calls that give no count."""
    import torch
    from top_sparse_attention_row_gb300 import binding as B, build
    build.build()
    rng = np.random.default_rng(3)
    S, R, K = 200, 19, 160
    idx = np.stack([rng.permutation(S)[:K] for _ in range(R)])
    out_of = rng.random((R, K)) < 0.2
    idx[7], out_of[8] = -1, True
    far = np.where(out_of, rng.choice([S, S + 1, 10 ** 6, 2 ** 31 - 1], (R, K)), idx)
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    bf = lambda *s: torch.from_numpy(rng.standard_normal(s)).bfloat16().cuda()  # noqa: E731
    if mla:
        args = [bf(R, 8, 576), bf(S, 576)]
    else:
        args = [bf(R, 6, 256), bf(S, 1, 256), bf(S, 1, 256)]
    f = B.sparse_mla_prefill if mla else B.sparse_prefill
    want = f(*args, i32(np.where(out_of, -1, idx)), None, 0.05, union_g=union_g)
    got = f(*args, i32(far), None, 0.05, union_g=union_g)
    torch.cuda.synchronize()
    assert B.device_status() == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert bool((got[0][7:9] == 0).all()) and bool((got[1][7:9] == float("-inf")).all())
