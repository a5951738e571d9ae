"""Page plans, rotary positions and 4-bit cache rows against their float64 restatement (GPU only)."""
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


# ------------------------------------------------------------------------------ page plans

def plan_case(rng, n, new_max, past_max, ps, extra_pages=2, n_free=None):
    past = rng.integers(0, past_max + 1, n)
    new = rng.integers(0, new_max + 1, n)
    ppr = (past_max + new_max) // ps + extra_pages
    held = np.minimum(-(-past // ps), ppr)
    total = int(np.minimum(-(-(past + new) // ps), ppr).sum())
    pages = rng.permutation(total + 8)
    table = np.full((n, ppr), -7)
    at = 0
    for i in range(n):
        table[i, :held[i]] = pages[at:at + held[i]]
        at += held[i]
    free = pages[at:]
    return past, new, table, free if n_free is None else free[:n_free], total + 8


def check_plan(B, past, new, table, free, head, ps, max_rows, n_pages=0, in_place=False):
    import torch
    t, h = i32(table), i32([head])
    got = B.page_plan(i32(past), i32(new), t, i32(free), h, ps, max_rows, n_pages=n_pages,
                      free_head_out=h if in_place else None)
    torch.cuda.synchronize()
    want = S.page_plan(past, new, table, free, head, ps, max_rows, n_pages)
    for name, a, b in zip(("table", "cu", "kv", "positions", "slots", "head", "short"),
                          (t, got.cu_seqlens_q, got.kv_lens, got.positions, got.slots, got.free_head,
                           got.shortfall), want):
        assert np.array_equal(a.cpu().numpy().reshape(np.shape(b)), b), name
    return got


@pytest.mark.parametrize("ps", [1, 7, 16, 64])
@pytest.mark.parametrize("n,new_max,past_max", [(1, 1, 0), (3, 5, 20), (64, 1, 300), (37, 90, 400),
                                                (1025, 3, 40), (2500, 6, 9)])
def test_page_plan(B, n, new_max, past_max, ps):
    rng = np.random.default_rng(n * 100 + ps)
    past, new, table, free, n_pages = plan_case(rng, n, new_max, past_max, ps)
    rows = int(new.sum())
    for max_rows in sorted({rows, rows + 5, max(rows - 3, 0), 0}):
        check_plan(B, past, new, table, free, 0, ps, max_rows, n_pages, in_place=max_rows % 2 == 1)


def test_page_plan_large_cluster(B):
    """Rows enough for every CTA of the cluster, one request much longer than the others."""
    rng = np.random.default_rng(5)
    past, new, table, free, n_pages = plan_case(rng, 300, 40, 500, 16)
    new[17] += 30000
    table = np.concatenate([table, np.full((300, 1900), -7)], 1)
    free = np.arange(n_pages, n_pages + 4000)
    check_plan(B, past, new, table, free, 3, 16, int(new.sum()) + 11, in_place=True)


def test_page_plan_shortage_bounds_and_bad_lengths(B):
    rng = np.random.default_rng(6)
    past, new, table, free, n_pages = plan_case(rng, 20, 60, 200, 8, n_free=11)
    check_plan(B, past, new, table, free, 0, 8, int(new.sum()))           # the list runs out
    check_plan(B, past, new, table, free, 11, 8, int(new.sum()))          # nothing left at all
    check_plan(B, past, new, table, free, 50, 8, int(new.sum()))          # head past the end
    check_plan(B, past, new, table, free, -4, 8, int(new.sum()))
    check_plan(B, past, new, table, free[:0], 0, 8, int(new.sum()))       # an empty list
    check_plan(B, past, new, table[:, :4], free, 0, 8, int(new.sum()))    # requests longer than their row
    check_plan(B, past, new, table, free, 0, 8, int(new.sum()), n_pages=9)  # pages past the pool
    new2 = new.copy()
    new2[[2, 5]] = -3, 0
    past2 = past.copy()
    past2[4] = -9
    check_plan(B, past2, new2, table, free, 0, 8, int(new.sum()))
    # lengths whose sum passes 2^31: rows end at max_rows, lengths saturate
    big = np.array([2 ** 31 - 1, 2 ** 31 - 5, 3])
    check_plan(B, np.array([5, 2 ** 31 - 1, 1]), big, np.full((3, 2), 1), np.arange(9), 0, 64, 100)


@pytest.mark.parametrize("n,new_max", [(5, 3), (1500, 4), (9000, 3), (300, 400)])
@pytest.mark.parametrize("which", ["past", "new"])
def test_page_plan_updates_lengths_in_place(B, n, new_max, which):
    """kv_lens written over the lengths it is made from, by one CTA and by a cluster."""
    import torch
    rng = np.random.default_rng(n)
    past, new, table, free, n_pages = plan_case(rng, n, new_max, 200, 16)
    want = S.page_plan(past, new, table, free, 0, 16, int(new.sum()) + 3, n_pages)
    for _ in range(20):
        lens = dict(past=i32(past), new=i32(new))
        t = i32(table)
        got = B.page_plan(lens["past"], lens["new"], t, i32(free), i32([0]), 16, int(new.sum()) + 3, n_pages=n_pages,
                          kv_lens=lens[which])
        torch.cuda.synchronize()
        for a, b in zip((t, got.cu_seqlens_q, lens[which], got.positions, got.slots, got.free_head), want):
            assert np.array_equal(a.cpu().numpy().reshape(np.shape(b)), b)
        other = "new" if which == "past" else "past"
        assert np.array_equal(lens[other].cpu().numpy(), dict(past=past, new=new)[other])


def test_page_plan_into_a_callers_unaligned_arrays(B):
    """positions and slots that start 4 bytes past a 16-byte boundary, one row more and less than fours."""
    import torch
    rng = np.random.default_rng(3)
    past, new, table, free, n_pages = plan_case(rng, 40, 30, 100, 8)
    for extra in (0, 1, 2, 3):
        rows = int(new.sum()) + extra
        pos, slots = (torch.full((rows + 6,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
        B.page_plan(i32(past), i32(new), i32(table), i32(free), i32([0]), 8, rows, n_pages=n_pages,
                    positions=pos[1:1 + rows], slots=slots[3:3 + rows])
        torch.cuda.synchronize()
        want = S.page_plan(past, new, table, free, 0, 8, rows, n_pages)
        for got, at, w in ((pos, 1, want[3]), (slots, 3, want[4])):
            got = got.cpu().numpy()
            assert np.array_equal(got[at:at + rows], w) and np.all(got[:at] == -9) and np.all(got[at + rows:] == -9)


def test_page_plan_replays_from_a_graph(B):
    """Captured once with the head in place: every replay takes the next pages."""
    import torch
    n, ps, ppr = 5, 4, 40
    past, new = i32(np.arange(n)), i32(np.full(n, 3))
    table, head = i32(np.full((n, ppr), -1)), i32([0])
    free = i32(np.random.default_rng(0).permutation(200))
    outs = dict(cu_seqlens_q=i32(np.zeros(n + 1)), kv_lens=i32(np.zeros(n)), positions=i32(np.zeros(20)),
                slots=i32(np.zeros(20)), shortfall=i32([0]))
    call = lambda: B.page_plan(past, new, table, free, head, ps, 20, free_head_out=head, **outs)  # noqa: E731
    call()                                     # (opts in to shared memory before the capture)
    table.fill_(-1)
    head.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
        past.copy_(outs["kv_lens"])
    t, h, p = np.full((n, ppr), -1), 0, np.arange(n)
    for _ in range(6):
        g.replay()
        torch.cuda.synchronize()
        t, cu, kv, pos, slot, h, short = S.page_plan(p, [3] * n, t, free.cpu().numpy(), h, ps, 20)
        p = kv
        assert np.array_equal(table.cpu().numpy(), t) and int(head) == h
        assert np.array_equal(outs["slots"].cpu().numpy(), slot)
        assert np.array_equal(outs["positions"].cpu().numpy(), pos)


# ------------------------------------------------------------------------------ rotary positions

def half_step(dtype):
    import torch
    return torch.finfo(dtype).eps / 2


# An output is off by its rounding, half a step of itself, and by the fp32 arithmetic: the angle's half
# turns are rounded to 24 bits (2^-25 half turns, 2^-23.3 rad), sincospi is good to 2 ulp, products and the
# sum round three times; each term is at most |a| + |b| of the pair, so 2^-21 (|a| + |b|) m covers them.
def assert_rotated(got, want, pair_sum, dtype, mag):
    g = got.double().cpu().numpy()
    bound = np.abs(want) * half_step(dtype) * (1 + 2.0 ** -10) + 2.0 ** -21 * pair_sum * mag + 2.0 ** -25
    assert np.all(np.abs(g - want) <= bound), np.max(np.abs(g - want) - bound)


def pair_sums(x, rot, offset, interleaved):
    """|a| + |b| of every rotated dim's pair; 0 on the passing dims."""
    s = np.zeros_like(x)
    part = np.abs(x[..., offset:offset + rot])
    if interleaved:
        p = np.repeat(part[..., 0::2] + part[..., 1::2], 2, axis=-1)
    else:
        h = part[..., :rot // 2] + part[..., rot // 2:]
        p = np.concatenate([h, h], -1)
    s[..., offset:offset + rot] = p
    return s


SHAPES = [  # heads, dim, rot, offset
    (1, 64, 64, 0), (3, 128, 128, 0), (6, 256, 256, 0), (2, 256, 64, 192), (8, 576, 64, 512),
    (5, 96, 32, 16), (2, 40, 10, 7), (1, 2, 2, 0), (3, 80, 24, 8), (7, 128, 0, 0)]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("heads,dim,rot,offset", SHAPES)
def test_rope(B, heads, dim, rot, offset, layout, dtype):
    import torch
    dt = getattr(torch, dtype)
    rng = np.random.default_rng(dim + rot)
    table = B.rope_table(max(rot, 2), 10000.0, scaling="yarn", factor=4.0, original_len=4096)
    w, mag = S.rope_frequencies(max(rot, 2), 10000.0, "yarn", 4.0, 4096)
    if rot == 0:
        table, w, mag = B.RopeTable(0, [], 1.0), np.zeros(0), 1.0
    for rows in (1, 2, 33):
        x = torch.from_numpy(rng.standard_normal((rows, heads, dim))).to(dt).cuda()
        pos = rng.integers(0, 1000, rows)
        pos[-1] = 2 ** 31 - 1 if rows > 2 else 131071
        if rows > 2:
            pos[1] = -1
        xs = x.double().cpu().numpy()
        for transpose in (False, True):
            want = S.rope(xs, pos, w, mag, layout == "interleaved", offset, transpose)
            out = torch.full_like(x, 7.0)
            B.rope(x, i32(pos), table, layout=layout, rot_offset=offset, transpose=transpose, out=out)
            torch.cuda.synchronize()
            want[pos < 0] = 7.0                     # rows left out stay as they were
            # the oracle's own angle at position 2^31 is off by 2^31 * 2^-53 * a few
            ps = pair_sums(xs, rot, offset, layout == "interleaved")
            assert_rotated(out, want, ps, dt, mag)
            passing = np.ones(dim, bool)
            passing[offset:offset + rot] = False
            assert np.array_equal(out.double().cpu().numpy()[..., passing], want[..., passing])
        y = x.clone()                               # in place
        B.rope(y, i32(pos), table, layout=layout, rot_offset=offset, out=y)
        full = B.rope(x, i32(np.where(pos < 0, 0, pos)), table, layout=layout, rot_offset=offset)
        keep = torch.from_numpy(pos >= 0).cuda()
        assert torch.equal(y[keep], full[keep]) and torch.equal(y[~keep], x[~keep])


def test_rope_gradient_by_differences(B):
    """<rope(x + h e) - rope(x - h e), g> / 2h = <e, rope^T(g)>, on values that fp16 holds exactly enough:
    with |x|, |e|, |g| <= 4 and h = 1/8 each rotated value rounds by at most 2^-11 * 8, so a sum over n
    products with |g| <= 4 is off by at most n * 2^-8 * 4 / (2 h)."""
    import torch
    rng = np.random.default_rng(3)
    t = B.rope_table(32, 100.0)
    draw = lambda: torch.from_numpy(rng.integers(-16, 17, (4, 2, 48)) / 4.0).half().cuda()  # noqa: E731
    x, e, g, pos = draw(), draw(), draw(), i32([0, 3, 50, 4000])
    for layout in ("half", "interleaved"):
        f = lambda v: B.rope(v, pos, t, layout=layout, rot_offset=16).double()  # noqa: E731
        h = 0.125
        left = ((f(x + h * e) - f(x - h * e)) / (2 * h) * g.double()).sum()
        right = (e.double() * B.rope(g, pos, t, layout=layout, rot_offset=16, transpose=True).double()).sum()
        assert abs(float(left - right)) <= x.numel() * 2.0 ** -8 * 4 / (2 * h)
        # and to the formula: every term of the two sums is bilinear in e and g
        w, mag = S.rope_frequencies(32, 100.0)
        want = (e.double().cpu().numpy() * S.rope(g.double().cpu().numpy(), pos.tolist(), w, mag,
                                                  layout == "interleaved", 16, True)).sum()
        assert abs(float(right) - want) <= x.numel() * 4 * 8 * 2.0 ** -11


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rows,hq,hkv,dim,rot,offset", [
    (1, 6, 1, 256, 256, 0), (45, 24, 2, 256, 64, 0), (300, 4, 4, 64, 32, 16), (9, 3, 3, 50, 20, 5),
    (2000, 1, 1, 128, 128, 0)])
def test_rope_append(B, rows, hq, hkv, dim, rot, offset, layout, dtype):
    """q, k and v as slices of one projected row, some rows left out, some slots outside the cache."""
    import torch
    dt = getattr(torch, dtype)
    rng = np.random.default_rng(rows)
    table = B.rope_table(rot, 10000.0)
    w, mag = S.rope_frequencies(rot, 10000.0)
    qkv = torch.from_numpy(rng.standard_normal((rows, (hq + 2 * hkv) * dim))).to(dt).cuda()
    q, k, v = (t.unflatten(1, (-1, dim)) for t in qkv.split([hq * dim, hkv * dim, hkv * dim], 1))
    n_slots = rows + 3
    pos, slots = rng.integers(0, 5000, rows), rng.permutation(n_slots)[:rows]
    if rows > 3:
        pos[2], slots[0], slots[3] = -1, -1, n_slots
    kc = torch.full((n_slots + 1, hkv, dim), 3.0, dtype=dt, device="cuda")   # one row past n_slots: untouched
    vc = kc.clone()
    q_out = B.rope_append(q, k, v, kc[:n_slots], vc[:n_slots], i32(pos), i32(slots), table, layout=layout,
                          rot_offset=offset, q_out=torch.full((rows, hq, dim), 3.0, dtype=dt, device="cuda"))
    torch.cuda.synchronize()
    inter = layout == "interleaved"
    qs, ks = q.double().cpu().numpy(), k.double().cpu().numpy()
    want = S.rope(qs, pos, w, mag, inter, offset)
    want[pos < 0] = 3.0
    assert_rotated(q_out, want, pair_sums(qs, rot, offset, inter), dt, mag)
    kr = S.rope(ks, pos, w, mag, inter, offset)
    wk, wv = np.full((n_slots + 1, hkv, dim), 3.0), np.full((n_slots + 1, hkv, dim), 3.0)
    sums = np.zeros_like(wk)
    for r in range(rows):
        if pos[r] >= 0 and 0 <= slots[r] < n_slots:
            wk[slots[r]], wv[slots[r]] = kr[r], v[r].double().cpu().numpy()
            sums[slots[r]] = pair_sums(ks[r:r + 1], rot, offset, inter)[0]
    assert_rotated(kc, wk, sums, dt, mag)
    assert np.array_equal(vc.double().cpu().numpy(), wv)


def test_rope_append_latent_rows_and_unaligned_views(B):
    """A cache of latent rows (no V, last 64 of 576 dims turn), and the same call on storage that starts 2
    bytes past a 16-byte boundary: the same values from the other kernel."""
    import torch
    rng = np.random.default_rng(8)
    R, H, D = 21, 8, 576
    t = B.rope_table(64, 10000.0)
    q = torch.from_numpy(rng.standard_normal((R, H, D))).bfloat16().cuda()
    k = torch.from_numpy(rng.standard_normal((R, 1, D))).bfloat16().cuda()
    pos, slots = i32(rng.integers(0, 9000, R)), i32(rng.permutation(40)[:R])
    kw = dict(layout="interleaved", rot_offset=512)
    kc = torch.zeros((40, 1, D), dtype=torch.bfloat16, device="cuda")
    out = B.rope_append(q, k, None, kc, None, pos, slots, t, **kw)
    odd = lambda x: torch.cat([x.new_zeros(1), x.flatten()])[1:].view(x.shape)  # noqa: E731
    kc2 = odd(torch.zeros_like(kc))
    out2 = B.rope_append(odd(q), odd(k), None, kc2, None, pos, slots, t, **kw)
    torch.cuda.synchronize()
    assert out2.data_ptr() % 16 == 0 and kc2.data_ptr() % 16 == 2
    assert torch.equal(out, out2) and torch.equal(kc, kc2)
    w, mag = S.rope_frequencies(64, 10000.0)
    ks = k.double().cpu().numpy()
    want = np.zeros((40, 1, D))
    sums = np.zeros((40, 1, D))
    at = slots.cpu().numpy()
    want[at] = S.rope(ks, pos.tolist(), w, mag, True, 512)
    sums[at] = pair_sums(ks, 64, 512, True)
    assert_rotated(kc, want, sums, torch.bfloat16, mag)


@pytest.mark.parametrize("heads,dim,rot,offset", [(4, 128, 128, 0), (3, 96, 32, 16), (2, 40, 10, 6)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_in_and_out_of_slices(B, heads, dim, rot, offset, layout):
    """Rows inside wider rows, as input, as output and in place: the same values, and nothing beside them."""
    import torch
    t = B.rope_table(rot, 10000.0)
    how = dict(layout=layout, rot_offset=offset)
    R, width = 37, (heads + 3) * dim
    wide = torch.randn((R, width), device="cuda").bfloat16()
    part = lambda w: w[:, dim:dim + heads * dim].unflatten(1, (heads, dim))  # noqa: E731
    pos = i32(np.arange(R) * 97 - 97)                             # the first row is left out
    want = B.rope(part(wide).contiguous(), pos, t, out=part(wide).contiguous(), **how)
    into = wide.clone()
    B.rope(part(wide), pos, t, out=part(into), **how)
    same = wide.clone()
    B.rope(part(same), pos, t, out=part(same), **how)
    torch.cuda.synchronize()
    for got in (into, same):
        assert torch.equal(part(got), want)
        assert torch.equal(got[:, :dim], wide[:, :dim]) and torch.equal(got[:, dim + heads * dim:], wide[:, dim + heads * dim:])


def test_rope_broadcast_rows_empty_calls_and_streams(B):
    import torch
    t = B.rope_table(64, 10000.0)
    row = torch.randn((1, 2, 64), device="cuda").bfloat16()
    pos = i32(np.arange(50))
    wide = row.expand(50, 2, 64)                               # stride 0: one row at 50 positions
    assert torch.equal(B.rope(wide, pos, t), B.rope(wide.contiguous(), pos, t))
    assert B.rope(row[:0], pos[:0], t).shape == (0, 2, 64)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = B.rope(wide, pos, t, stream=s)
    s.synchronize()
    assert torch.equal(a, B.rope(wide, pos, t))
    with torch.cuda.stream(s):
        b = B.rope(wide, pos, t)
    s.synchronize()
    assert torch.equal(a, b)


# ------------------------------------------------------------------------------ 4-bit cache rows

@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("rows,hkv,dim", [(1, 1, 64), (5, 2, 256), (77, 3, 128), (600, 1, 32), (3, 1, 576)])
def test_append_fp4_without_rotation(B, rows, hkv, dim, dtype):
    """Bit for bit: inputs of at most 11 bits, a power-of-two global scale and e4m3 block scales leave no
    quotient so near a border between two codes that fp32 could round it across (a quotient that is not on
    the border is at least 2^-18 away from it, relatively)."""
    import torch
    dt = getattr(torch, dtype)
    rng = np.random.default_rng(dim)
    x = rng.standard_normal((2, rows, hkv, dim)) * np.exp(2 * rng.standard_normal((2, rows, hkv, 1)))
    x[0, 0, 0, :16] = 0.0                                             # an empty block
    x[1, 0, 0, :16] = [6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -5, -2.5, 4, 3, 2, 1]   # ties
    x[1, -1, -1, -16:] *= 1e-6                                        # a scale below e4m3's least
    k, v = (torch.from_numpy(a).to(dt).cuda() for a in x)
    if rows > 3:
        k[3, 0, 16:32] = 60000.0                                      # scale and codes saturate
    n_slots = rows + 2
    slots = rng.permutation(n_slots)[:rows]
    if rows > 2:
        slots[1] = -1
    u8 = lambda w: torch.full((n_slots, hkv, w), 0xAA, dtype=torch.uint8, device="cuda")  # noqa: E731
    kc, vc, ks, vs = u8(dim // 2), u8(dim // 2), u8(dim // 16), u8(dim // 16)
    seen = [torch.full((rows, hkv, dim), 9.0, dtype=dt, device="cuda") for _ in range(2)]
    B.rope_append_fp4(None, k, v, kc, ks, vc, vs, None, i32(slots), None, k_global=0.5, v_global=1.0,
                      k_seen=seen[0], v_seen=seen[1])
    torch.cuda.synchronize()
    for src, c, s, sn, g in ((k, kc, ks, seen[0], 0.5), (v, vc, vs, seen[1], 1.0)):
        codes, sc, values = S.fp4_quantise(src.double().cpu().numpy(), g)
        wc = np.full((n_slots, hkv, dim // 2), 0xAA)
        ws = np.full((n_slots, hkv, dim // 16), 0xAA)
        keep = slots >= 0
        wc[slots[keep]], ws[slots[keep]] = S.fp4_pack(codes)[keep], sc[keep]
        values[~keep] = 9.0
        # a block whose scale is 0 stores code 0, whatever the sign
        got = c.cpu().numpy()
        zero = np.repeat(ws == 0, 8, axis=-1)
        assert np.array_equal(np.where(zero, 0, got), np.where(zero, 0, wc)) and not got[zero].any()
        assert np.array_equal(s.cpu().numpy(), ws)
        # what the cache holds, rounded to the rows' type: exact (6 significant bits)
        want = torch.from_numpy(values).to(dt).double().numpy()
        assert np.array_equal(sn.double().cpu().numpy(), want)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dim,rot,offset", [(256, 256, 0), (128, 64, 32), (64, 32, 0), (96, 64, 32)])
def test_append_fp4_with_rotation(B, dim, rot, offset, layout):
    """A stored value is within half a code step of the rotated one; near the border between two scales or
    two codes either may be taken, so the bound is the largest half step (1 in units of the scale, between
    4 and 6) of the larger neighbouring scale, s (1 + 2^-3)."""
    import torch
    rng = np.random.default_rng(dim)
    rows, hq, hkv = 40, 4, 2
    table = B.rope_table(rot, 10000.0)
    w, mag = S.rope_frequencies(rot, 10000.0)
    q, k, v = (torch.from_numpy(rng.standard_normal((rows, h, dim))).bfloat16().cuda() for h in (hq, hkv, hkv))
    pos, slots = rng.integers(0, 5000, rows), rng.permutation(rows)
    u8 = lambda n: torch.zeros((rows, hkv, n), dtype=torch.uint8, device="cuda")  # noqa: E731
    kc, vc, ks, vs = u8(dim // 2), u8(dim // 2), u8(dim // 16), u8(dim // 16)
    seen = torch.empty_like(k)
    q_out = B.rope_append_fp4(q, k, v, kc, ks, vc, vs, i32(pos), i32(slots), table, k_global=0.25,
                              v_global=0.25, layout=layout, rot_offset=offset, k_seen=seen)
    torch.cuda.synchronize()
    inter = layout == "interleaved"
    kr = S.rope(k.double().cpu().numpy(), pos, w, mag, inter, offset)
    got = S.fp4_values(kc.cpu().numpy(), ks.cpu().numpy(), 0.25)[slots]
    _, sc, values = S.fp4_quantise(kr, 0.25)
    step = np.repeat(S.E4M3[sc], 16, axis=-1) * 0.25 * (1 + 2.0 ** -3)
    assert np.all(np.abs(got - kr) <= step + 2.0 ** -20)
    assert np.mean(got == values) > 0.999                    # and nearly always the very same
    assert np.array_equal(seen.double().cpu().numpy(), got)
    _, scv, vv = S.fp4_quantise(v.double().cpu().numpy(), 0.25)
    assert np.array_equal(S.fp4_values(vc.cpu().numpy(), vs.cpu().numpy(), 0.25)[slots], vv)
    assert torch.equal(q_out, B.rope(q, i32(pos), table, layout=layout, rot_offset=offset))


def test_append_fp4_non_finite_values_saturate(B):
    """Infinities keep their sign at the largest magnitude, NaN takes the largest magnitude too, and the
    other blocks of the row are as they would be."""
    import torch
    k = torch.ones((2, 1, 64), device="cuda").bfloat16()
    k[0, 0, 3], k[0, 0, 20], k[0, 0, 21], k[1, 0, 40] = float("inf"), float("-inf"), 2.0, float("nan")
    u8 = lambda n: torch.zeros((2, 1, n), dtype=torch.uint8, device="cuda")  # noqa: E731
    kc, ks, vc, vs = u8(32), u8(4), u8(32), u8(4)
    seen = torch.empty_like(k)
    B.rope_append_fp4(None, k, k, kc, ks, vc, vs, None, i32([0, 1]), None, k_seen=seen)
    torch.cuda.synchronize()
    got = seen.float().cpu().numpy()[:, 0]
    assert got[0, 3] == 6 * 448 and got[0, 20] == -6 * 448 and np.all(got[0, [0, 1, 2, 21, 22]] == 0)
    assert np.all(got[0, 32:] == got[1, 0]) and abs(got[1, 0] - 1) <= 2 ** -4      # scale e4m3(1 / 6), code 6
    assert abs(got[1, 40]) == 6 * S.E4M3[ks.cpu().numpy()[1, 0, 2]] and np.isfinite(got).all()


@pytest.mark.parametrize("layout", ["half", "interleaved", None])
def test_append_fp4_blocks_of_nan_alone_read_back_as_nan(B, layout):
    """K and V blocks whose values are all NaN get the scale NaN and codes 0, turned or not; a block with a
    number in it stays finite, and the other blocks are what they are without the NaN."""
    import torch
    dim, rot = 128, 64
    rng = np.random.default_rng(2)
    table = None if layout is None else B.rope_table(rot, 10000.0)
    how = {} if layout is None else dict(layout=layout, rot_offset=32)
    pos = None if layout is None else i32([0, 9, 700])
    k, v = (torch.from_numpy(rng.standard_normal((3, 2, dim))).bfloat16().cuda() for _ in range(2))
    # rows 0 and 2: whole rotated part and a passing block; row 1: one value of a passing block
    bad_k, bad_v = k.clone(), v.clone()
    for r, h in ((0, 1), (2, 0)):
        bad_k[r, h, 32:96], bad_k[r, h, :16], bad_v[r, h, 48:80] = float("nan"), float("nan"), float("nan")
    bad_k[1, 0, 100] = float("nan")
    got = []
    for a, b in ((k, v), (bad_k, bad_v)):
        u8 = lambda n: torch.full((3, 2, n), 0xAA, dtype=torch.uint8, device="cuda")  # noqa: E731
        kc, vc, ks, vs = u8(dim // 2), u8(dim // 2), u8(dim // 16), u8(dim // 16)
        seen = [torch.empty_like(k) for _ in range(2)]
        B.rope_append_fp4(None, a, b, kc, ks, vc, vs, pos, i32([0, 1, 2]), table, k_global=0.5, v_global=0.25,
                          k_seen=seen[0], v_seen=seen[1], **how)
        torch.cuda.synchronize()
        got.append([x.cpu() for x in (ks, vs)] + [x.cpu().unflatten(-1, (-1, 8)) for x in (kc, vc)] +
                   [x.float().cpu().unflatten(-1, (-1, 16)) for x in seen])
    for w in (0, 1):
        src = (bad_k, bad_v)[w].float().cpu().unflatten(-1, (-1, 16))
        gone = src.isnan().all(-1)
        assert int(gone.sum()) == (10 if w == 0 else 4)
        scale, codes, seen = got[1][w], got[1][2 + w], got[1][4 + w]
        assert bool((scale[gone] == 0x7F).all()) and not bool(codes[gone].any()) and bool(seen[gone].isnan().all())
        assert bool(seen[~gone].isfinite().all()) and bool((scale[~gone] != 0x7F).all())
        same = ~src.isnan().any(-1)
        for a, b in ((scale, got[0][w]), (codes, got[0][2 + w]), (seen, got[0][4 + w])):
            assert torch.equal(a[same], b[same])


def test_attention_over_a_4_bit_cache_shows_nan_rows(B):
    """A K row of NaN alone, written by the append, makes the rows that see it NaN and no others."""
    import torch
    n, dim = 200, 64
    q, k, v = (torch.randn((n, 1, dim), device="cuda").bfloat16() for _ in range(3))
    k[150] = float("nan")
    u8 = lambda w: torch.zeros((256, 1, w), dtype=torch.uint8, device="cuda")  # noqa: E731
    kc, vc, ks, vs = u8(dim // 2), u8(dim // 2), u8(dim // 16), u8(dim // 16)
    B.rope_append_fp4(None, k, v, kc, ks, vc, vs, None, i32(np.arange(n)), None)
    out, lse = B.window_attention_fp4_paged(q, kc, ks, vc, vs, i32([0, n]), i32([n]), i32([[0, 1, 2, 3]]), 64, 0.125,
                                            window=30)
    torch.cuda.synchronize()
    hit = out.isnan().any(-1)[:, 0].cpu().numpy()
    assert np.array_equal(np.flatnonzero(hit), np.arange(150, 180)) and bool(out[150:180].isnan().all())


@pytest.mark.parametrize("exponent", [-126, -124, -101, -99, 0, 98, 100, 123, 127])
def test_append_fp4_global_scales_at_the_ends_of_the_range(B, exponent):
    """Powers of two from the smallest to the largest: zeros stay zeros and values come out as the oracle's,
    beside the smallest values that a block scale stands for too."""
    import torch
    g = 2.0 ** exponent
    rng = np.random.default_rng(4)
    x = np.clip(rng.standard_normal((4, 1, 64)), -3, 3) * g                # block scales up to 1/2
    x[0, 0, 1:16], x[0, 0, 0] = 0.0, 2.0 ** -7 * g                         # scale 2^-9, all others 0
    x[1, 0, ::3] = 0.0
    k = torch.from_numpy(x).bfloat16().cuda()
    u8 = lambda n: torch.zeros((4, 1, n), dtype=torch.uint8, device="cuda")  # noqa: E731
    kc, vc, ks, vs = u8(32), u8(32), u8(4), u8(4)
    B.rope_append_fp4(None, k, k, kc, ks, vc, vs, None, i32([0, 1, 2, 3]), None, k_global=g, v_global=g)
    torch.cuda.synchronize()
    codes, sc, _ = S.fp4_quantise(k.double().cpu().numpy(), g)
    want = np.where(np.repeat(sc == 0, 8, axis=-1), 0, S.fp4_pack(codes))
    for c, s in ((kc, ks), (vc, vs)):
        assert np.array_equal(s.cpu().numpy(), sc) and np.array_equal(c.cpu().numpy(), want)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("magnitude", [1.0, 1.0 + 2.0 ** -23, 1.0 + 2.0 ** -22, 1.0 - 2.0 ** -24, 1.0 - 2.0 ** -23, 1.3])
@pytest.mark.parametrize("kg,vg", [(0.5, 0.25), (0.1, 0.37), (3.0, 1e-3)])
def test_append_fp4_values_next_to_borders(B, layout, magnitude, kg, vg):
    """Blocks that lie on the borders between codes, and between scales, and one fp32 step beside them.  At
    position 0 a rotated value is its fp32 product with the magnitude (a cos 0 m - b sin 0 m = a m), so the
    rows' exact values are known; x / g is rounded to fp32, and from there on the float64 oracle decides."""
    import torch
    rng = np.random.default_rng(6)
    dim, rows = 128, 60
    t = B.RopeTable(dim, [0] * (dim // 2), magnitude)
    border = np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    x = np.empty((2, rows, 1, dim // 16, 16))
    for w in (0, 1):
        for r in range(rows):
            for b in range(dim // 16):
                i = int(rng.integers(20, 100))                          # scales of all sizes
                s, up = S.E4M3[i], S.E4M3[i + 1]
                x[w, r, 0, b] = rng.choice(border, 16) * rng.choice([-1, 1], 16) * s
                x[w, r, 0, b, rng.integers(16)] = 6 * (s if (r + b) % 2 else (s + up) / 2)
    k, v = (torch.from_numpy(a.reshape(rows, 1, dim)).half().cuda() for a in x)
    u8 = lambda n: torch.zeros((rows, 1, n), dtype=torch.uint8, device="cuda")  # noqa: E731
    kc, vc, ks, vs = u8(dim // 2), u8(dim // 2), u8(dim // 16), u8(dim // 16)
    seen = [torch.empty_like(k) for _ in range(2)]
    B.rope_append_fp4(None, k, v, kc, ks, vc, vs, i32(np.zeros(rows)), i32(np.arange(rows)), t, k_global=kg, v_global=vg,
                      layout=layout, k_seen=seen[0], v_seen=seen[1])
    torch.cuda.synchronize()
    for src, m, g, c, s, sn in ((k, magnitude, kg, kc, ks, seen[0]), (v, 1.0, vg, vc, vs, seen[1])):
        y = src.float().cpu().numpy() * np.float32(m) / np.float32(g)          # fp32, each rounded
        assert y.dtype == np.float32
        codes, sc, values = S.fp4_quantise(y.astype(np.float64), 1.0)
        assert np.array_equal(s.cpu().numpy(), sc)
        # (a block whose scale is 0 stores code 0, whatever the sign)
        want = np.where(np.repeat(sc == 0, 8, axis=-1), 0, S.fp4_pack(codes))
        assert np.array_equal(c.cpu().numpy(), want)
        # values: the scales' product and the code's are rounded to fp32, then to fp16 (half a step, or 2^-25)
        values = values * float(np.float32(g))
        got = sn.double().cpu().numpy()
        assert np.all(np.abs(got - values) <= np.abs(values) * (2.0 ** -11 + 2.0 ** -22) + 2.0 ** -25)
