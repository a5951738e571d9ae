"""Refusals and host-side parts of the serving-step operators (no GPU needed)."""
import ctypes
import math

import numpy as np
import pytest

from oracle import serving as S

FAKE = 1 << 20          # 16-byte aligned stand-in for a device pointer, never read
OK, INVALID, UNSUPPORTED = 0, 1, 2


@pytest.fixture(scope="module")
def B():
    from top_sparse_attention_row_gb300 import build, binding
    build.build()
    binding.load_library()
    return binding


def plan_args(**kw):
    a = dict(past=FAKE, new=FAKE, table=FAKE, free=FAKE, n_free=10, head=FAKE, head_out=FAKE, cu=FAKE,
             kv=FAKE, pos=FAKE, slots=FAKE, short=FAKE, n=4, ppr=8, ps=64, n_pages=0, max_rows=16,
             stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(past=None), INVALID), (dict(new=None), INVALID), (dict(table=None), INVALID),
    (dict(free=None), INVALID), (dict(head=None), INVALID), (dict(head_out=None), INVALID),
    (dict(cu=None), INVALID), (dict(kv=None), INVALID), (dict(n=0), INVALID), (dict(ppr=0), INVALID),
    (dict(ps=0), INVALID), (dict(n_pages=-1), INVALID), (dict(n_free=-1), INVALID),
    (dict(max_rows=-1), INVALID), (dict(past=FAKE + 2), INVALID), (dict(slots=FAKE + 1), INVALID),
    (dict(n=16385), UNSUPPORTED), (dict(max_rows=1 << 31), UNSUPPORTED), (dict(n_free=1 << 31), UNSUPPORTED),
])
def test_page_plan_refusals(B, kw, status):
    assert B.load_library().qsa_page_plan(*plan_args(**kw)) == status


def test_page_plan_refuses_tables_whose_pages_pass_32_bits(B):
    """A step's fresh pages are numbered in 32 bits."""
    f = B.load_library().qsa_page_plan
    assert f(*plan_args(n=16384, ppr=131072)) == UNSUPPORTED
    assert f(*plan_args(n=2, ppr=1 << 30)) == UNSUPPORTED


def rope_spec(B, **kw):
    steps = (ctypes.c_uint64 * 256)()
    a = dict(steps=ctypes.addressof(steps), rot_dim=64, rot_offset=0, layout=0, transpose=0, magnitude=1.0)
    a.update(kw)
    spec = B.RopeSpec(*a.values())
    spec.keep = steps
    return spec


def append_args(B, spec, **kw):
    a = dict(q=FAKE, q_out=FAKE, k=FAKE, v=FAKE, k_cache=FAKE, v_cache=FAKE, positions=FAKE, slots=FAKE,
             spec=None if spec is None else ctypes.byref(spec), rows=0, n_slots=100, hq=6, hkv=1, d=256,
             qs=6 * 256, qos=6 * 256, ks=256, vs=256, dtype=0, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("spec,kw,status", [
    ({}, {}, OK), (None, {}, OK), (None, dict(positions=None), OK), ({}, dict(v=None, v_cache=None), OK),
    ({}, dict(hq=0, q=None, q_out=None), OK), ({}, dict(q=None), INVALID), ({}, dict(q_out=None), INVALID),
    ({}, dict(k=None), INVALID), ({}, dict(k_cache=None), INVALID), ({}, dict(v=None), INVALID),
    ({}, dict(v_cache=None), INVALID), ({}, dict(slots=None), INVALID), ({}, dict(positions=None), INVALID),
    ({}, dict(rows=-1), INVALID), ({}, dict(hkv=0), INVALID), ({}, dict(hq=-1), INVALID),
    ({}, dict(d=0), INVALID), ({}, dict(n_slots=-1), INVALID), ({}, dict(dtype=2), INVALID),
    ({}, dict(qos=6 * 256 - 1), INVALID), ({}, dict(qs=7 * 256), INVALID),      # in place, other stride
    ({}, dict(ks=-1), INVALID), ({}, dict(q=FAKE + 1), INVALID), ({}, dict(rows=1 << 31), UNSUPPORTED),
    ({}, dict(d=1 << 20, qos=6 << 20, qs=6 << 20), UNSUPPORTED),
    (dict(rot_dim=63), {}, INVALID), (dict(rot_dim=-2), {}, INVALID), (dict(rot_offset=-1), {}, INVALID),
    (dict(rot_offset=200), {}, INVALID), (dict(rot_dim=258), {}, INVALID), (dict(layout=2), {}, INVALID),
    (dict(transpose=2), {}, INVALID), (dict(magnitude=math.nan), {}, INVALID), (dict(steps=None), {}, INVALID),
    (dict(rot_dim=514), dict(d=1024, qs=6 * 1024, qos=6 * 1024), UNSUPPORTED),
])
def test_rope_append_refusals(B, spec, kw, status):
    s = None if spec is None else rope_spec(B, **spec)
    assert B.load_library().qsa_rope_append(*append_args(B, s, **kw)) == status


def test_rope_append_limits_of_heads(B):
    """What the header states: 16384 query heads, 8192 KV heads, 16384 dims."""
    f, s = B.load_library().qsa_rope_append, rope_spec(B)
    for ok, bad in ((dict(hq=16384), dict(hq=16385)), (dict(hkv=8192), dict(hkv=8193)), (dict(d=16384), dict(d=16385))):
        wide = dict(qs=1 << 40, qos=1 << 40, ks=1 << 40, vs=1 << 40)
        assert f(*append_args(B, s, **wide, **ok)) == OK
        assert f(*append_args(B, s, **wide, **bad)) == UNSUPPORTED


def test_rope_refusals(B):
    f = B.load_library().qsa_rope
    s = rope_spec(B)
    ok = [FAKE, FAKE, FAKE, ctypes.byref(s), 0, 6, 256, 1536, 1536, 0, None]
    assert f(*ok) == OK
    for at, bad in ((0, None), (1, None), (2, None), (3, None), (4, -1), (5, 0), (6, 0), (8, 1535), (9, 5)):
        args = list(ok)
        args[at] = bad
        assert f(*args) == INVALID, (at, bad)


@pytest.mark.parametrize("spec,kw,status", [
    ({}, {}, OK), (None, {}, OK), ({}, dict(k_scale=None), INVALID), ({}, dict(v_scale=None), INVALID),
    ({}, dict(v=None, v_cache=None), INVALID), ({}, dict(kg=0.0), INVALID), ({}, dict(vg=math.inf), INVALID),
    ({}, dict(kg=math.nan), INVALID), ({}, dict(ks=260), INVALID), ({}, dict(k_seen=FAKE + 8), INVALID),
    ({}, dict(k_cache=FAKE + 8), INVALID), ({}, dict(d=240, qs=1440, qos=1440), UNSUPPORTED),
    (dict(rot_dim=48), {}, UNSUPPORTED), (dict(rot_dim=48, layout=1), {}, OK),
    (dict(rot_offset=8), {}, UNSUPPORTED),
])
def test_rope_append_fp4_refusals(B, spec, kw, status):
    s = None if spec is None else rope_spec(B, **spec)
    a = dict(q=FAKE, q_out=FAKE, k=FAKE, v=FAKE, k_cache=FAKE, k_scale=FAKE + 1, v_cache=FAKE, v_scale=FAKE + 3,
             kg=1.0, vg=1.0, k_seen=None, v_seen=None, positions=FAKE, slots=FAKE,
             spec=None if s is None else ctypes.byref(s), rows=0, n_slots=100, hq=6, hkv=1, d=256, qs=6 * 256,
             qos=6 * 256, ks=256, vs=256, dtype=0, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    assert B.load_library().qsa_rope_append_fp4(*a.values()) == status


SCALINGS = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
            dict(scaling="yarn", factor=4.0, original_len=4096), dict(scaling="yarn", factor=16.0, original_len=700),
            dict(scaling="turns", factor=8.0, original_len=8192, beta_fast=4.0, beta_slow=1.0)]


@pytest.mark.parametrize("kw", SCALINGS)
@pytest.mark.parametrize("rot,base", [(64, 10000.0), (128, 500000.0), (10, 2.5)])
def test_rope_table_against_the_formulas(B, rot, base, kw):
    t = B.rope_table(rot, base, **kw)
    w, mag = S.rope_frequencies(rot, base, **kw)
    assert t.rot_dim == rot and abs(t.magnitude - mag) <= 2.0 ** -24 * mag
    # a step is the frequency's fraction of a turn: off by the roundings of pow, of one quotient and of a
    # few products in doubles, some 1e-15 of it, and by the cut to a whole number of 2^-64 turns (a slow
    # pair's 1e-14 of w / 2 pi is less than that: w = 2.5e-6 gives 2.5e-20, against 2^-64 = 5.4e-20)
    got = np.array([s / 2.0 ** 64 for s in t.steps])
    assert np.all(np.abs(got - w / (2 * np.pi)) <= 1e-14 * w + 2.0 ** -64)


def test_rope_table_refusals(B):
    for kw in (dict(rot_dim=63), dict(rot_dim=0), dict(rot_dim=64, base=-1.0), dict(rot_dim=64, base=math.inf),
               dict(rot_dim=64, scaling="linear", factor=0.0), dict(rot_dim=2, scaling="ntk", factor=2.0),
               dict(rot_dim=64, scaling="yarn", factor=2.0), dict(rot_dim=514),
               dict(rot_dim=64, scaling="turns", factor=2.0, original_len=100, beta_fast=1.0, beta_slow=1.0),
               dict(rot_dim=64, scaling="yarn", factor=2.0, original_len=100, base=1.0)):
        with pytest.raises(RuntimeError):
            B.rope_table(**kw)
    with pytest.raises(ValueError):
        B.rope_table(64, scaling="other")
    t = B.RopeTable(4, [1, 2 ** 64 - 1], 1.5)      # a caller's own frequencies
    assert t.steps == [1, 2 ** 64 - 1] and t.magnitude == 1.5


PI = "3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803"


@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0)])
@pytest.mark.parametrize("rot,base", [(64, 10000.0), (128, 500000.0), (256, 1000000.0), (10, 2.5)])
def test_rope_steps_against_80_digits(B, rot, base, kw):
    """A step's error per token, and an angle's at the largest position.  In doubles, with e = 2 i / rot and the base b
    (for ntk b f^(rot / (rot - 2))): e is rounded (moves b^-e by e ln b 2^-53 of itself), b too (e times the roundings
    of its own power, (1 + 2 ln f + 2 + 1) 2^-53), pow is good to 2^-52, and 2 pi, its quotient and the
    scaling's round 2^-53 each: theta (e (ln b + 2 ln f + 4) + 6) 2^-53 / 2 pi, and 2^-64 from the cut to an
    integer.  theta falls with e faster than the bracket grows: 6 / 2 pi = 2^-0.06 covers all pairs."""
    from decimal import Decimal as D, localcontext
    got = B.rope_table(rot, base, **kw).steps
    with localcontext() as c:
        c.prec = 80
        f, b = D(kw.get("factor", 1.0)), D(base)
        if kw.get("scaling") == "ntk":
            b = b * f ** (D(rot) / D(rot - 2))
        for i, step in enumerate(got):
            e = D(2 * i) / D(rot)
            turns = b ** -e / (2 * D(PI))
            if kw.get("scaling") == "linear":
                turns /= f
            off = D(step) / D(2) ** 64 - turns
            bound = float(turns) * (float(e) * (math.log(float(b)) + 2 * math.log(float(f)) + 4) + 6) * 2.0 ** -53
            assert abs(float(off)) <= bound + 2.0 ** -64 <= 2.0 ** -53
            pos = 2 ** 31 - 1
            far = D((pos * step) % 2 ** 64) / D(2) ** 64 - (pos * turns) % 1
            far = abs(float(far))
            assert min(far, 1 - far) <= 2.0 ** -22


def test_rope_table_wants_a_step_for_every_pair(B):
    """Too few would leave pairs unturned, silently."""
    for rot, steps in ((8, [1, 2, 3]), (8, [1, 2, 3, 4, 5]), (8, []), (7, [1, 2, 3]), (-2, []), (0, [1])):
        with pytest.raises(ValueError):
            B.RopeTable(rot, steps, 1.0)
    assert B.RopeTable(0, [], 1.0).steps == [] and B.RopeTable(8, range(4), 1.0).steps == [0, 1, 2, 3]


def test_binding_refuses_cpu_and_mismatched_tensors(B):
    import torch
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        B.page_plan(i(2), i(2), i(2, 4), i(5), i(1), 64, 8)                      # not on a GPU
    with pytest.raises(TypeError):
        B.page_plan(i(2).long(), i(2), i(2, 4), i(5), i(1), 64, 8)
    with pytest.raises(ValueError):
        B.page_plan(i(2), i(3), i(2, 4), i(5), i(1), 64, 8)
    with pytest.raises(ValueError):
        B.page_plan(i(2), i(2), i(2, 4), i(5), i(1), 64, -1)
    t = B.rope_table(64)
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        B.rope(x, i(3), t)                                                       # not on a GPU
    with pytest.raises(TypeError):
        B.rope(x.float(), i(3), t)
    with pytest.raises(ValueError):
        B.rope(x, i(2), t)
    with pytest.raises(ValueError):
        B.rope(x.transpose(1, 2).contiguous().transpose(1, 2), i(3), t)          # heads not contiguous
    with pytest.raises(ValueError):
        B.rope_append(None, x, x, x, None, i(3), i(3), t)                        # v without its cache
    with pytest.raises(TypeError):
        B.rope(x, i(3), None)
    with pytest.raises(TypeError):
        B.rope(x, [0, 1, 2], t)
    with pytest.raises(TypeError):
        B.rope(x, i(3), t, unknown=1)
    q, c, cu, kv, tab = torch.zeros(3, 2, 64).half(), torch.zeros(128, 1, 64).half(), i(2), i(1), i(1, 2)
    with pytest.raises(ValueError):
        B.window_attention_paged(q, c, c, cu, kv, tab, 64, 0.1)                  # not on a GPU
    with pytest.raises(ValueError):
        B.window_attention_paged(q, c, c, cu, kv, tab, 48, 0.1)                  # not whole pages
    with pytest.raises(ValueError):
        B.window_attention_paged(q, c, c[:64], cu, kv, tab, 64, 0.1)
    with pytest.raises(ValueError):
        B.window_attention_paged(q, c, c, kv, kv, tab, 64, 0.1)
    with pytest.raises(TypeError):
        B.window_attention_paged(q, c.float(), c, cu, kv, tab, 64, 0.1)
    with pytest.raises(AttributeError):
        B.no_such_call
    for name in B.SERVING:
        assert name in getattr(B, name).__doc__ or getattr(B, name).__text_signature__


def test_oracle_fp4_grid_and_ties():
    """Ties fall on the even code, values past 6 saturate, and e4m3 has the 127 values of its bit layout."""
    import torch
    f8 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(f8, S.E4M3)
    x = np.array([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -5.0, 5.01, -0.26, 0, 0, 0, 0])
    codes, sc, v = S.fp4_quantise(x, 1.0)
    assert S.E4M3[sc[0]] == 1.0
    assert list(v[:12]) == [6, 0, 1, 1, 2, 2, 4, 4, -0.0, -4, 6, -0.5]
    assert np.array_equal(S.fp4_values(S.fp4_pack(codes), sc, 1.0), v)


def test_oracle_rope_is_a_rotation():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 2, 16))
    w, _ = S.rope_frequencies(8, 100.0)
    y = S.rope(x, [0, 5, 77], w, 1.0, True, 4)
    assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., :4], x[..., :4])
    assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))
    assert np.allclose(S.rope(y, [0, 5, 77], w, 1.0, True, 4, transpose=True), x)
    # dot products depend on the distance alone
    a, b = rng.standard_normal((1, 1, 8)), rng.standard_normal((1, 1, 8))
    dot = lambda p, r: float(np.sum(S.rope(a, [p], w, 1.0, False, 0) * S.rope(b, [r], w, 1.0, False, 0)))  # noqa: E731
    assert abs(dot(10, 3) - dot(107, 100)) < 1e-12


def test_copies_of_a_rope_table_have_their_own_steps(B):
    import copy
    import ctypes
    import pickle
    t = B.rope_table(64, 500.0, scaling="yarn", factor=4.0, original_len=4096.0)
    for c in (copy.copy(t), copy.deepcopy(t), pickle.loads(pickle.dumps(t))):
        assert c.steps == t.steps and (c.rot_dim, c.magnitude) == (t.rot_dim, t.magnitude)
        assert c._raw[0] == ctypes.addressof(c._steps) != t._raw[0]
    with pytest.raises(AttributeError):
        t.magnitude = 2.0


def window_args(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, cu=FAKE, kv=FAKE, table=FAKE, out=FAKE, lse=None, rows=0, n=2, ppr=4, ps=64, n_pages=8,
             hq=6, hkv=1, d=256, scale=0.0625, window=0, sink=0, dtype=0, ws=None, ws_bytes=0, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return list(a.values())


WINDOW_REFUSALS = [
    ({}, OK), (dict(window=7, sink=3, dtype=1), OK), (dict(d=64), OK), (dict(d=128), OK),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(cu=None), INVALID),
    (dict(kv=None), INVALID), (dict(table=None), INVALID), (dict(out=None), INVALID), (dict(q=FAKE + 8), INVALID),
    (dict(out=FAKE + 8), INVALID), (dict(lse=FAKE + 2), INVALID), (dict(rows=-1), INVALID), (dict(n=0), INVALID),
    (dict(ppr=0), INVALID), (dict(ps=0), INVALID), (dict(n_pages=0), INVALID), (dict(hq=5, hkv=2), INVALID),
    (dict(window=-1), INVALID), (dict(sink=-1), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID), (dict(dtype=2), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(hq=129), UNSUPPORTED), (dict(rows=(1 << 31) - 2), UNSUPPORTED),
    (dict(ppr=1 << 25), UNSUPPORTED), (dict(n_pages=1 << 26), UNSUPPORTED), (dict(rows=(1 << 63) - 1), UNSUPPORTED), (dict(n_pages=1 << 24, hkv=2), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", WINDOW_REFUSALS)
def test_window_attention_refusals(B, kw, status):
    assert B.load_library().qsa_window_attention_paged(*window_args(**kw)) == status


@pytest.mark.parametrize("kw,extra,status", [
    (dict(), {}, OK), (dict(), dict(ks=None), INVALID), (dict(), dict(vs=FAKE + 4), INVALID), (dict(), dict(kg=0.0), INVALID),
    (dict(), dict(vg=math.inf), INVALID), (dict(hq=64), {}, OK), (dict(hq=65), {}, UNSUPPORTED), (dict(hq=128, d=128), {}, OK),
])
def test_window_attention_fp4_refusals(B, kw, extra, status):
    q, k, v, *rest = window_args(**kw)
    e = dict(ks=FAKE, vs=FAKE, kg=1.0, vg=1.0)
    e.update(extra)
    assert B.load_library().qsa_window_attention_fp4_paged(q, k, e["ks"], v, e["vs"], e["kg"], e["vg"], *rest) == status


def test_window_attention_refuses_scales_that_leave_fp32(B):
    """The kernel multiplies by scale log2(e), for a 4-bit cache by k_global too."""
    lib = B.load_library()
    assert lib.qsa_window_attention_paged(*window_args(scale=2.3e38)) == OK
    assert lib.qsa_window_attention_paged(*window_args(scale=2.4e38)) == INVALID
    for scale, kg, status in ((0.1, 1.0, OK), (1e30, 1e30, INVALID), (1e-30, 1e-30, INVALID), (1e30, 1e-30, OK)):
        q, k, v, *rest = window_args(scale=scale)
        assert lib.qsa_window_attention_fp4_paged(q, k, FAKE, v, FAKE, kg, 1.0, *rest) == status


def test_window_workspace_bytes(B):
    """Equal shares where there are few query tiles, whole units where there are many."""
    f = lambda rows, n, ppr, **kw: B.window_workspace_bytes(rows, n, ppr, 64, 24, 2, 256, 0, 0, num_sms=152, **kw)  # noqa: E731
    one = 2 * 128 * 257 * 4 + 32
    assert f(1, 1, 512) == 152 * one and f(1, 1, 40) == 40 * one     # two KV heads of 20 tiles each
    assert f(1, 1, 2) == 0                                           # one tile: nothing to share
    assert f(48, 48, 512, fp4=True) == 152 * one
    assert f(100000, 1, 2000) == 0
    assert B.window_workspace_bytes(0, 1, 4, 64, 24, 2, 256, 0, 0, num_sms=152) == 0
    assert B.window_workspace_bytes(1, 1, 4, 64, 24, 5, 256, 0, 0, num_sms=152) == 0
