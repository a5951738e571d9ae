"""The serving-step operators around the paged caches, as cases that can be timed and compared.

One serving step of a paged decoder runs them in this order: the batch's page tables and slot maps
are built from its request lengths ("plan"); q and k are rotated to their positions and the new K/V
rows are written into the cache, as they are ("rope") or in 4 bits ("append4"); and attention reads
the cache through the page tables with a sliding window and a few first tokens that stay visible
("window", and "window4" over the 4-bit cache).

``run`` computes each of them in elementary torch operations; with ``own`` set it makes the calls of
this package that a user makes.
"""
import math
from collections import namedtuple

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # 64 requests in decode, one new token each, contexts up to 8k: the plan of every decode step
        dict(name="plan_decode", op="plan", n_requests=64, new_max=1, past_max=8190, page_size=64,
             pages_per_req=128, pad_rows=0),
        # a full chunked-prefill step: ragged requests, small pages, a padded row array
        dict(name="plan_prefill", op="plan", n_requests=256, new_max=2048, past_max=30000,
             page_size=16, pages_per_req=2048, pad_rows=1000),
        # q and k of an 8192-token prefill, half of each head rotated, positions scaled to 128k
        dict(name="rope_prefill", op="rope", rows=8192, hq=24, hkv=2, dim=256, rot=128, offset=0,
             layout="interleaved", scaling="yarn", base=1000000.0, max_pos=131072, dtype="bf16",
             gradient=False),
        # gradient through the rotation of the 64 rope dims of 576-dim latent queries
        dict(name="rope_mla_grad", op="rope", rows=8192, hq=8, hkv=0, dim=576, rot=64, offset=512,
             layout="interleaved", scaling="none", base=10000.0, max_pos=32768, dtype="bf16",
             gradient=True),
        # 64 decode tokens into the 4-bit cache
        dict(name="append4_decode", op="append4", rows=64, hkv=2, dim=256, dtype="bf16"),
        # an 8192-token prefill into the 4-bit cache
        dict(name="append4_prefill", op="append4", rows=8192, hkv=2, dim=256, dtype="bf16"),
        # one request's decode token at the end of 8k: latency
        dict(name="window_decode_1", op="window", n_requests=1, new_max=1, past_min=8191,
             past_max=8191, hq=6, hkv=1, dim=256, window=4096, sink=4, page_size=64, dtype="bf16"),
        # a decode batch with contexts of 1k to 8k
        dict(name="window_decode_128", op="window", n_requests=128, new_max=1, past_min=1000,
             past_max=8191, hq=24, hkv=2, dim=256, window=4096, sink=4, page_size=64, dtype="bf16"),
        # the last 8192 rows of a 32k prompt
        dict(name="window_prefill_32k", op="window", n_requests=1, new_max=8192, past_min=24576,
             past_max=24576, hq=6, hkv=1, dim=256, window=4096, sink=4, page_size=64, dtype="bf16"),
        # a mixed batch: decode rows and prompt chunks together, small pages, 128-dim heads, fp16
        dict(name="window_mixed", op="window", n_requests=6, new_max=2047, past_min=1,
             past_max=2100, hq=32, hkv=8, dim=128, window=1024, sink=16, page_size=16, dtype="fp16"),
        # decode over a long 4-bit cache, nothing masked by a window
        dict(name="window4_decode_48", op="window4", n_requests=48, new_max=1, past_min=16000,
             past_max=32767, hq=24, hkv=2, dim=256, window=0, sink=0, page_size=64, dtype="bf16"),
        # prompt chunks over a 4-bit cache
        dict(name="window4_chunks", op="window4", n_requests=5, new_max=1000, past_min=100,
             past_max=4000, hq=8, hkv=1, dim=128, window=2048, sink=4, page_size=128, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "rope", "append4", "window", "window", "window4"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "plan":
        page_size = rng.choice([1, 16, 48, 64, 128])
        past_max, new_max = _log(rng, 1, 30000), _log(rng, 1, 2048)
        n = _log(rng, 1, 256)
        return dict(op=op, n_requests=n, new_max=new_max, past_max=past_max, page_size=page_size,
                    pages_per_req=(past_max + new_max) // page_size + rng.randint(1, 20),
                    pad_rows=_log(rng, 1, 1000) - 1)
    if op == "rope":
        hkv = rng.choice([0, 1, 2, 8])
        hq = max(1, hkv) * rng.choice([1, 4, 6, 8])
        dim, rot, offset = rng.choice([(64, 64, 0), (96, 24, 8), (128, 128, 0), (128, 32, 0),
                                       (256, 256, 0), (256, 64, 192), (576, 64, 512)])
        rows = _log(rng, 1, 8192)
        rows = max(1, min(rows, 8192 * 28 * 256 // ((hq + 2 * hkv) * dim)))
        return dict(op=op, rows=rows, hq=hq, hkv=hkv, dim=dim, rot=rot, offset=offset,
                    layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "ntk", "yarn", "turns"]),
                    base=rng.choice([10000.0, 500000.0, 1000000.0]), max_pos=_log(rng, 64, 1000000),
                    dtype=dtype, gradient=hkv == 0)
    if op == "append4":
        return dict(op=op, rows=_log(rng, 1, 8192), hkv=rng.choice([1, 2]),
                    dim=rng.choice([64, 128, 256]), dtype=dtype)
    dim = rng.choice([64, 128, 256])
    hkv = rng.choice([1, 2, 8])
    hq = hkv * rng.choice([1, 3, 4, 6, 8, 12])
    n = _log(rng, 1, 48)
    new_max = 1 if rng.random() < 0.5 else _log(rng, 2, 2000)
    past_max = _log(rng, 1, 16000)
    while n * hq * new_max * (past_max + new_max) > 6e8 or n * hkv * (past_max + new_max) > 4e5:
        n, past_max, new_max = max(1, n // 2), max(1, past_max * 3 // 4), max(1, new_max * 3 // 4)
    return dict(op=op, n_requests=n, new_max=new_max, past_min=max(1, past_max // rng.choice([1, 4, 40])),
                past_max=past_max, hq=hq, hkv=hkv, dim=dim,
                window=rng.choice([0, _log(rng, 1, 4096), _log(rng, 64, 4096)]),
                sink=rng.choice([0, 1, 4, 16, 130]), page_size=rng.choice([1, 16, 48, 64, 128]),
                dtype=dtype)


# ------------------------------------------------------------------------------ inputs

def _spread(n, lo, hi):
    """n lengths spread over lo .. hi on a logarithmic scale; a single one is hi."""
    if n == 1:
        return [hi]
    return [int(round(lo * (hi / lo) ** (i / (n - 1)))) for i in range(n)]


def _lengths(case):
    """The batch's (past, new) lengths.  They follow from the case, so that its work does."""
    n = case["n_requests"]
    news = _spread(n, 1, case["new_max"])
    pasts = _spread(n, case.get("past_min", 1), case["past_max"])
    step = next(s for s in (7, 11, 13, 1) if math.gcd(s, n) == 1)
    return [(pasts[i * step % n], news[i]) for i in range(n)]


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _quantise(x, scale_all):
    """x [..., dim] in 4 bits: e2m1 codes, two in a byte, the even dim in the low half, and an e4m3
    scale for every 16 dims, in units of scale_all."""
    y = x.float().unflatten(-1, (-1, 16)) / scale_all
    s = (y.abs().amax(-1, keepdim=True) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    sf = s.float()
    y = torch.where(sf > 0, y / sf, torch.zeros_like(y)).flatten(-2)
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
            + (a >= 3.5) + (a > 5.0)) | (torch.signbit(y).to(torch.uint8) << 3)
    return code[..., 0::2] | (code[..., 1::2] << 4), s.squeeze(-1)


def _values(code, s, scale_all):
    """The fp32 values of 4-bit rows: e2m1 code times block scale times scale_all."""
    e2m1 = torch.tensor([0., .5, 1., 1.5, 2., 3., 4., 6., -0., -.5, -1., -1.5, -2., -3., -4., -6.],
                        device=code.device)
    x = e2m1[torch.stack((code & 15, code >> 4), -1).flatten(-2).int()]
    return (x.unflatten(-1, (-1, 16)) * (s.float() * scale_all).unsqueeze(-1)).flatten(-2)


def _prepare_plan(case, g):
    n, ps, ppr = case["n_requests"], case["page_size"], case["pages_per_req"]
    lens = _lengths(case)
    order = torch.randperm(n, generator=g, device="cuda").tolist()
    past = [lens[i][0] for i in order]
    new = [lens[i][1] for i in order]
    held = [min(-(-p // ps), ppr) for p in past]
    after = [min(-(-(p + m) // ps), ppr) for p, m in zip(past, new)]
    n_pages = sum(after) + 64
    pages = torch.randperm(n_pages, generator=g, device="cuda").int()
    table = torch.full((n, ppr), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, h in enumerate(held):
        table[i, :h] = pages[at:at + h]
        at += h
    return dict(past=_int32(past), new=_int32(new), table=table, free=pages[at:].contiguous(),
                head=_int32([0]), head_out=_int32([0]), max_rows=sum(new) + case["pad_rows"],
                n_pages=n_pages)


def _scaling(case):
    return dict(base=case["base"], scaling=case["scaling"],
                factor=1.0 if case["scaling"] == "none" else 4.0,
                original_len=max(1, case["max_pos"] // 4))


def _prepare_rope(case, g):
    dt, R, D = _DTYPES[case["dtype"]], case["rows"], case["dim"]
    Hq, Hkv = case["hq"], case["hkv"]
    qkv = torch.randn((R, (Hq + 2 * Hkv) * D), generator=g, device="cuda").to(dt)
    q, k, v = (t.unflatten(1, (-1, D)) if t.shape[1] else None
               for t in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
    st = dict(q=q, k=k, v=v, q_out=torch.empty((R, Hq, D), dtype=dt, device="cuda"),
              positions=torch.randint(0, case["max_pos"], (R,), generator=g, device="cuda").int())
    if Hkv:
        S = R + 64
        st["slots"] = torch.randperm(S, generator=g, device="cuda")[:R].int()
        st["k_cache"] = torch.zeros((S, Hkv, D), dtype=dt, device="cuda")
        st["v_cache"] = torch.zeros((S, Hkv, D), dtype=dt, device="cuda")
    if own:
        from top_sparse_attention_row_gb300 import binding
        s = _scaling(case)
        st["rope"] = binding.rope_table(case["rot"], s.pop("base"), **s)   # kept by a user's model
    return st


def _prepare_append4(case, g):
    dt, R, D, Hkv = _DTYPES[case["dtype"]], case["rows"], case["dim"], case["hkv"]
    S = R + 64
    kv = torch.randn((R, 2, Hkv, D), generator=g, device="cuda")
    kv *= torch.exp(torch.randn((R, 2, Hkv, 1), generator=g, device="cuda"))
    k, v = kv.to(dt).unbind(1)
    z = lambda d: torch.zeros((S, Hkv, d), dtype=torch.uint8, device="cuda")  # noqa: E731
    return dict(k=k, v=v, slots=torch.randperm(S, generator=g, device="cuda")[:R].int(),
                k_cache=z(D // 2), v_cache=z(D // 2), k_scale=z(D // 16), v_scale=z(D // 16),
                k_seen=torch.empty((R, Hkv, D), dtype=dt, device="cuda"),
                v_seen=torch.empty((R, Hkv, D), dtype=dt, device="cuda"), k_all=0.25, v_all=0.125)


def _prepare_window(case, g):
    dt, D, Hq, Hkv = _DTYPES[case["dtype"]], case["dim"], case["hq"], case["hkv"]
    ps = case["page_size"]
    lens = _lengths(case)
    order = torch.randperm(len(lens), generator=g, device="cuda").tolist()
    new = [lens[i][1] for i in order]
    kv = [sum(lens[i]) for i in order]
    ppr = max(-(-x // ps) for x in kv)
    held = [-(-x // ps) for x in kv]
    n_pages = sum(held) + 2
    pages = torch.randperm(n_pages, generator=g, device="cuda").int()
    table = torch.full((len(lens), ppr), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, h in enumerate(held):
        table[i, :h] = pages[at:at + h]
        at += h
    cu = [0]
    for m in new:
        cu.append(cu[-1] + m)
    S, R = n_pages * ps, cu[-1]
    st = dict(q=torch.randn((R, Hq, D), generator=g, device="cuda").to(dt), cu=_int32(cu),
              kv=_int32(kv), table=table, page_size=ps, scale=D ** -0.5, window=case["window"],
              sink=case["sink"], max_new=max(new), max_kv=max(kv), n_pages=n_pages)
    for name in ("k", "v"):
        if case["op"] == "window":
            x = torch.empty((S, Hkv, D), dtype=dt, device="cuda")
            for part in x.split(1 << 18):
                part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
            st[name + "_cache"] = x
        else:
            parts = [_quantise(torch.randn((m, Hkv, D), generator=g, device="cuda"), 0.25)
                     for m in [1 << 18] * (S >> 18) + [S % (1 << 18)] if m]
            st[name + "_cache"] = torch.cat([p[0] for p in parts])
            st[name + "_scale"] = torch.cat([p[1] for p in parts]).view(torch.uint8)
    return st


def prepare(case, seed):
    g = _generator(seed)
    st = {"plan": _prepare_plan, "rope": _prepare_rope, "append4": _prepare_append4,
          "window": _prepare_window, "window4": _prepare_window}[case["op"]](case, g)
    st["case"] = case
    return st


# ------------------------------------------------------------------------------ plain forms

_Plan = namedtuple("_Plan", "cu_seqlens_q kv_lens positions slots free_head shortfall")


def _plan(st):
    ps, table, free = st["case"]["page_size"], st["table"], st["free"]
    n, ppr = table.shape
    past, new = st["past"].long(), st["new"].long()
    cu = torch.nn.functional.pad(new.cumsum(0), (1, 0))
    before = ((past + ps - 1) // ps).clamp(max=ppr)
    after = ((past + new + ps - 1) // ps).clamp(max=ppr)
    need = after - before
    first = st["head"].long() + need.cumsum(0) - need
    col = torch.arange(ppr, device=table.device)
    fresh = (col >= before[:, None]) & (col < after[:, None])
    at = first[:, None] + col - before[:, None]
    page = torch.where(at < free.numel(), free[at.clamp(0, free.numel() - 1)], -1)
    table.copy_(torch.where(fresh, page, table))
    row = torch.arange(st["max_rows"], device=table.device)
    req = torch.searchsorted(cu[1:], row, right=True).clamp(max=n - 1)
    x = past[req] + row - cu[req]
    page = torch.where(x // ps < ppr, table[req, (x // ps).clamp(max=ppr - 1)], -1)
    live = row < cu[n]
    wanted = st["head"].long() + need.sum()
    return _Plan(cu.int(), (past + new).int(), torch.where(live, x, -1).int(),
                 torch.where(live & (page >= 0), page * ps + x % ps, -1).int(),
                 wanted.clamp(max=free.numel()).int(), (wanted - free.numel()).clamp(min=0).int())


def _frequencies(case):
    """Radians per token of every rotated pair, and the factor on the rotated values."""
    s, rot = _scaling(case), case["rot"]
    base, f, L = s["base"], s["factor"], s["original_len"]
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    if s["scaling"] == "ntk":
        return (base * f ** (rot / (rot - 2))) ** (-2 * i / rot), 1.0
    w = base ** (-2 * i / rot)
    if s["scaling"] == "linear":
        return w / f, 1.0
    if s["scaling"] == "turns":       # kept from 32 turns over the original length, stretched below 1
        keep = ((L * w / (2 * math.pi) - 1) / 31).clamp(0, 1)
        return keep * w + (1 - keep) * w / f, 1.0
    if s["scaling"] == "yarn":        # the same ends, and a ramp over the pairs between them
        at = [rot * math.log(L / (2 * math.pi * t)) / (2 * math.log(base)) for t in (32, 1)]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        return (1 - ramp) * w + ramp * w / f, 0.1 * math.log(f) + 1
    return w, 1.0


def _rotated(x, positions, case):
    w, mag = _frequencies(case)
    angle = positions.double()[:, None, None] * w
    cos, sin = (angle.cos() * mag).float(), (angle.sin() * mag).float()
    if case["gradient"]:
        sin = -sin
    rot, off = case["rot"], case["offset"]
    a = x[..., off:off + rot].float()
    if case["layout"] == "half":
        u, v = a[..., :rot // 2], a[..., rot // 2:]
        a = torch.cat((u * cos - v * sin, v * cos + u * sin), -1)
    else:
        u, v = a[..., 0::2], a[..., 1::2]
        a = torch.stack((u * cos - v * sin, v * cos + u * sin), -1).flatten(-2)
    return torch.cat((x[..., :off], a.to(x.dtype), x[..., off + rot:]), -1)


def _rope(st):
    case = st["case"]
    st["q_out"].copy_(_rotated(st["q"], st["positions"], case))
    if st["k"] is None:
        return st["q_out"]
    st["k_cache"][st["slots"].long()] = _rotated(st["k"], st["positions"], case)
    st["v_cache"][st["slots"].long()] = st["v"]
    return st["q_out"], st["k_cache"], st["v_cache"]


def _append4(st):
    at = st["slots"].long()
    for name in ("k", "v"):
        code, s = _quantise(st[name], st[name + "_all"])
        st[name + "_cache"][at] = code
        st[name + "_scale"][at] = s.view(torch.uint8)
        st[name + "_seen"].copy_(_values(code, s, st[name + "_all"]))
    return _append4_outputs(st)


def _append4_outputs(st):
    f8 = torch.float8_e4m3fn
    return (st["k_seen"], st["v_seen"], st["k_cache"], st["v_cache"], st["k_scale"].view(f8),
            st["v_scale"].view(f8))


def _rows(st, name, slots):
    """Cache rows at slots, in fp32."""
    if st["case"]["op"] == "window":
        return st[name + "_cache"][slots].float()
    return _values(st[name + "_cache"][slots], st[name + "_scale"][slots].view(torch.float8_e4m3fn),
                   0.25)


def _window(st):
    q, cu, kv, table, ps = st["q"], st["cu"].long(), st["kv"].long(), st["table"], st["page_size"]
    R, Hq, D = q.shape
    n, Hkv, dev = kv.numel(), st["k_cache"].shape[1], q.device
    new = cu[1:] - cu[:-1]
    t, j = torch.arange(st["max_new"], device=dev), torch.arange(st["max_kv"], device=dev)
    slots = table.long()[:, j // ps].clamp(min=0) * ps + j % ps                  # [n, max_kv]
    k = _rows(st, "k", slots).permute(0, 2, 3, 1)                                # [n, Hkv, D, kv]
    x = q[(cu[:-1, None] + t).clamp(max=R - 1)].float()                          # [n, new, Hq, D]
    x = x.unflatten(2, (Hkv, -1)).permute(0, 2, 3, 1, 4).flatten(2, 3)           # [n, Hkv, g*new, D]
    s = (torch.matmul(x, k) * st["scale"]).unflatten(2, (Hq // Hkv, -1))
    p = (kv - new)[:, None] + t                                                  # [n, new]
    seen = (j <= p[..., None]) & (t < new[:, None])[..., None]
    if st["window"] > 0:
        seen &= (j > p[..., None] - st["window"]) | (j < st["sink"])
    s.masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    s.sub_(m).exp_()
    total = s.sum(-1, keepdim=True)
    v = _rows(st, "v", slots).permute(0, 2, 1, 3)                                # [n, Hkv, kv, D]
    o = torch.matmul(s.flatten(2, 3), v).unflatten(2, s.shape[2:4])              # [n, Hkv, g, new, D]
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (m + total.log()).squeeze(-1)
    row = torch.arange(R, device=dev)
    i = torch.searchsorted(cu[1:], row, right=True)
    o = o.permute(0, 3, 1, 2, 4)[i, row - cu[i]].flatten(1, 2)
    lse = lse.permute(0, 3, 1, 2)[i, row - cu[i]].flatten(1, 2)
    return o.to(q.dtype), lse


# ------------------------------------------------------------------------------ one pass

def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return {"plan": _run_plan, "rope": _rope, "append4": _append4, "window": _window,
                "window4": _window}[op](st)
    from top_sparse_attention_row_gb300 import binding
    if op == "plan":
        plan = binding.page_plan(st["past"], st["new"], st["table"], st["free"], st["head"],
                                 case["page_size"], st["max_rows"], n_pages=st["n_pages"],
                                 free_head_out=st["head_out"])
        return _plan_outputs(plan, st)
    if op == "rope":
        how = dict(layout=case["layout"], rot_offset=case["offset"])
        if st["k"] is None:
            return binding.rope(st["q"], st["positions"], st["rope"], transpose=case["gradient"],
                                out=st["q_out"], **how)
        binding.rope_append(st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"],
                            st["positions"], st["slots"], st["rope"], q_out=st["q_out"], **how)
        return st["q_out"], st["k_cache"], st["v_cache"]
    if op == "append4":
        binding.rope_append_fp4(None, st["k"], st["v"], st["k_cache"], st["k_scale"],
                                st["v_cache"], st["v_scale"], None, st["slots"], None,
                                k_global=st["k_all"], v_global=st["v_all"], k_seen=st["k_seen"],
                                v_seen=st["v_seen"])
        return _append4_outputs(st)
    how = dict(window=st["window"], n_sink=st["sink"])
    if op == "window":
        return binding.window_attention_paged(st["q"], st["k_cache"], st["v_cache"], st["cu"],
                                              st["kv"], st["table"], st["page_size"], st["scale"],
                                              **how)
    return binding.window_attention_fp4_paged(st["q"], st["k_cache"], st["k_scale"], st["v_cache"],
                                              st["v_scale"], st["cu"], st["kv"], st["table"],
                                              st["page_size"], st["scale"], k_global=0.25,
                                              v_global=0.25, **how)


def _run_plan(st):
    return _plan_outputs(_plan(st), st)


def _plan_outputs(plan, st):
    return {"table": st["table"], "cu_seqlens_q": plan.cu_seqlens_q, "kv_lens": plan.kv_lens,
            "positions": plan.positions, "slots": plan.slots, "free_head": plan.free_head.view(1),
            "shortfall": plan.shortfall.view(1)}


# ------------------------------------------------------------------------------ work

def _seen_keys(past, new, window, sink):
    """(pairs of a query row and a key it sees, keys that some row sees) of one request."""
    if window <= 0:
        return new * past + new * (new + 1) // 2, past + new
    pairs = 0
    for t in range(new):
        p = past + t
        lo = max(0, p - window + 1)
        pairs += p + 1 - lo + min(sink, lo)
    lo = max(0, past - window + 1)
    return pairs, past + new - lo + min(sink, lo)


def work(case):
    op = case["op"]
    if op == "plan":
        lens, ps = _lengths(case), case["page_size"]
        rows = sum(m for _, m in lens) + case["pad_rows"]
        fresh = sum(-(-(p + m) // ps) - -(-p // ps) for p, m in lens)
        # lengths in, offsets and lengths out; a free page read and a table entry written for each
        # new page; one held page read per request; position and slot written for each row
        return {"bytes": 4 * (5 * len(lens) + 2 * fresh + 2 * rows), "flops": rows}
    if op == "rope":
        e = case["rows"] * (case["hq"] + 2 * case["hkv"]) * case["dim"]
        turned = case["rows"] * (case["hq"] + case["hkv"]) * case["rot"]
        return {"bytes": 4 * e + 8 * case["rows"], "flops": 3 * turned}
    if op == "append4":
        e = 2 * case["rows"] * case["hkv"] * case["dim"]
        return {"bytes": e * 4 + e // 2 + e // 16 + 4 * case["rows"], "flops": 3 * e}
    D, Hq, Hkv, ps = case["dim"], case["hq"], case["hkv"], case["page_size"]
    per_key = 2 * Hkv * (2 * D if op == "window" else D // 2 + D // 16)
    pairs = keys = rows = 0
    for p, m in _lengths(case):
        a, b = _seen_keys(p, m, case["window"], case["sink"])
        pairs, keys, rows = pairs + a, keys + b, rows + m
    return {"bytes": keys * per_key + rows * Hq * (4 * D + 4) + 4 * (keys // ps),
            "flops": 4 * D * Hq * pairs}


# ------------------------------------------------------------------------------ 64-bit answers

def _exact_rope(case, st):
    rot, off = case["rot"], case["offset"]
    w = [case["base"] ** (-2.0 * i / rot) for i in range(rot // 2)]
    f = 1.0 if case["scaling"] == "none" else 4.0
    L, mag = max(1, case["max_pos"] // 4), 1.0
    if case["scaling"] == "ntk":
        w = [x * f ** (-2.0 * i / (rot - 2)) for i, x in enumerate(w)]
    elif case["scaling"] == "linear":
        w = [x / f for x in w]
    elif case["scaling"] in ("turns", "yarn"):
        pair = lambda t: rot / 2 * math.log(L / (2 * math.pi * t), case["base"])  # noqa: E731
        lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), rot - 1)
        for i, x in enumerate(w):
            if case["scaling"] == "turns":
                short = 1 - min(1.0, max(0.0, (L * x / (2 * math.pi) - 1.0) / 31.0))
            else:
                short = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            w[i] = x + (x / f - x) * short
        if case["scaling"] == "yarn":
            mag = 1 + math.log(f) / 10
    turn = torch.outer(st["positions"].double(), torch.tensor(w, dtype=torch.float64, device="cuda"))
    turn = torch.polar(torch.full_like(turn, mag), -turn if case["gradient"] else turn)[:, None]

    def of(x):
        y = x.double()
        z = y[..., off:off + rot]
        z = z.unflatten(-1, (2, -1)).transpose(-1, -2) if case["layout"] == "half" else z.unflatten(-1, (-1, 2))
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
        z = z.transpose(-1, -2) if case["layout"] == "half" else z
        y[..., off:off + rot] = z.flatten(-2)
        return y

    if st["k"] is None:
        return of(st["q"])
    kc, vc = st["k_cache"].double(), st["v_cache"].double()
    kc[st["slots"].long()], vc[st["slots"].long()] = of(st["k"]), st["v"].double()
    return of(st["q"]), kc, vc


def _exact_append4(st):
    steps = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    e4m3 = torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()

    def nearest(grid, x):       # to the grid's nearest value, ties to the even index
        i = torch.searchsorted(grid, x).clamp(1, grid.numel() - 1)
        low, high = x - grid[i - 1], grid[i] - x
        return torch.where((low < high) | ((low == high) & (i % 2 == 1)), i - 1, i)

    seen, scales = [], []
    for name in ("k", "v"):
        x = st[name].double().unflatten(-1, (-1, 16)) / st[name + "_all"]
        s = e4m3[nearest(e4m3, x.abs().amax(-1) / 6)]
        r = torch.where(s[..., None] > 0, x / s[..., None], 0)
        y = steps[nearest(steps, r.abs())] * r.sign() * s[..., None] * st[name + "_all"]
        seen.append(y.flatten(-2))
        c = st[name + "_scale"].view(torch.float8_e4m3fn).double()
        c[st["slots"].long()] = s
        scales.append(c)
    return (*seen, None, None, *scales)


def _exact_window(case, st):
    q, W, D = st["q"].double(), case["window"], case["dim"]
    R, Hq, Hkv = q.shape[0], case["hq"], case["hkv"]
    o, lse = torch.zeros_like(q), torch.full((R, Hq), -math.inf, dtype=torch.float64, device="cuda")
    cu, kv = st["cu"].tolist(), st["kv"].tolist()
    for i, n in enumerate(kv):
        past = n - (cu[i + 1] - cu[i])
        at = torch.arange(n, device="cuda")
        at = st["table"][i].long()[at // st["page_size"]] * st["page_size"] + at % st["page_size"]
        if case["op"] == "window":
            keys, values = st["k_cache"][at].double(), st["v_cache"][at].double()
        else:
            keys, values = (_values(st[x + "_cache"][at],
                                    st[x + "_scale"][at].view(torch.float8_e4m3fn), 0.25).double()
                            for x in "kv")
        for r0 in range(cu[i], cu[i + 1], 256):
            r1 = min(r0 + 256, cu[i + 1])
            p = torch.arange(r0 - cu[i] + past, r1 - cu[i] + past, device="cuda")
            first = max(0, int(r0 - cu[i] + past) - W + 1) if W > 0 else 0
            js = torch.cat((torch.arange(min(case["sink"], first), device="cuda"),
                            torch.arange(first, r1 - cu[i] + past, device="cuda")))
            ok = js[None] <= p[:, None]
            if W > 0:
                ok &= (js[None] < case["sink"]) | (p[:, None] - js[None] < W)
            for h in range(Hkv):
                hs = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
                s = torch.einsum("rhd,jd->hrj", q[r0:r1, hs], keys[js, h]) / math.sqrt(D)
                s = torch.where(ok, s, -math.inf)
                z = torch.logsumexp(s, -1)
                o[r0:r1, hs] = torch.einsum("hrj,jd->rhd", torch.exp(s - z[..., None]), values[js, h])
                lse[r0:r1, hs] = z.T
    return o, lse


def exact(case, seed):
    if case["op"] == "plan":
        return None                      # whole numbers
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(case, st)
    if case["op"] == "append4":
        return _exact_append4(st)
    return _exact_window(case, st)
