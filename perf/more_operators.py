"""Long contexts over the paged cache: pages chosen by content, and prompts that many requests share,
as cases that can be timed and compared.

A decoder with a long context keeps, for every page of its cache, the smallest and largest value that
each key dim takes there ("bounds").  They bound every logit of the page from above, so a query scores
the pages of its context by them and picks a few ("select"), and attention reads those alone
("selected").  Where requests begin with the same tokens, their page tables name the same pages, and
attention reads these once for all of them ("prefix").

``run`` computes each of them in elementary torch operations; with ``own`` set it makes the calls of
this package that a user makes.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # the pages that 64 requests in decode have just added a token to
        dict(name="bounds_decode", op="bounds", n_requests=64, new_max=1, past_min=1, past_max=8190,
             hkv=2, dim=256, page_size=64, dtype="bf16"),
        # a prefill step of four requests, the longest a whole chunk of 8192
        dict(name="bounds_prefill", op="bounds", n_requests=4, new_max=8192, past_min=1,
             past_max=24576, hkv=2, dim=256, page_size=64, dtype="bf16"),
        # one request's decode token at the end of 32k: latency
        dict(name="select_decode_1", op="select", n_requests=1, new_max=1, past_min=32767,
             past_max=32767, hq=24, hkv=2, dim=256, page_size=64, n_select=32, first=1, last=2,
             dtype="bf16"),
        # a decode batch with contexts of 64k to 128k
        dict(name="select_decode_64", op="select", n_requests=64, new_max=1, past_min=65536,
             past_max=131071, hq=24, hkv=2, dim=256, page_size=64, n_select=32, first=1, last=2,
             dtype="bf16"),
        # the last 8192 rows of a 32k prompt
        dict(name="select_prefill", op="select", n_requests=1, new_max=8192, past_min=24576,
             past_max=24576, hq=24, hkv=2, dim=256, page_size=64, n_select=32, first=1, last=2,
             dtype="bf16"),
        # one request's decode token over 2048 chosen keys: latency
        dict(name="selected_decode_1", op="selected", n_requests=1, new_max=1, past_min=32767,
             past_max=32767, hq=24, hkv=2, dim=256, page_size=64, n_select=32, dtype="bf16"),
        # a decode batch, each request over its own 2048 keys
        dict(name="selected_decode_128", op="selected", n_requests=128, new_max=1, past_min=4000,
             past_max=16383, hq=24, hkv=2, dim=256, page_size=64, n_select=32, dtype="bf16"),
        # the last 8192 rows of a 32k prompt, each row over its own 2048 keys
        dict(name="selected_prefill", op="selected", n_requests=1, new_max=8192, past_min=24576,
             past_max=24576, hq=6, hkv=1, dim=256, page_size=64, n_select=32, dtype="bf16"),
        # a mixed batch: decode rows and prompt chunks together, small pages, 128-dim heads, fp16
        dict(name="selected_mixed", op="selected", n_requests=6, new_max=2047, past_min=1,
             past_max=16000, hq=32, hkv=8, dim=128, page_size=16, n_select=64, dtype="fp16"),
        # four answers to one prompt of 2k: latency
        dict(name="prefix_decode_4", op="prefix", n_requests=4, n_groups=1, new_max=1,
             prefix_min=2048, prefix_max=2048, own_max=100, hq=24, hkv=2, dim=256, page_size=64,
             dtype="bf16"),
        # 64 requests in decode behind one system prompt of 32k
        dict(name="prefix_decode_64", op="prefix", n_requests=64, n_groups=1, new_max=1,
             prefix_min=32768, prefix_max=32768, own_max=1000, hq=24, hkv=2, dim=256, page_size=64,
             dtype="bf16"),
        # four prompts with ten requests each, decode rows and chunks together, small pages, fp16
        dict(name="prefix_groups", op="prefix", n_requests=40, n_groups=4, new_max=200,
             prefix_min=1000, prefix_max=8192, own_max=1000, hq=32, hkv=8, dim=128, page_size=16,
             dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["bounds", "select", "select", "selected", "selected", "prefix", "prefix"])
    dim = rng.choice([64, 128, 256])
    hkv = rng.choice([1, 2, 8])
    c = dict(op=op, hkv=hkv, dim=dim, dtype=rng.choice(["bf16", "fp16"]),
             page_size=rng.choice([8, 16, 48, 64, 128]))
    new_max = 1 if rng.random() < 0.4 else _log(rng, 2, 2048)
    if op == "bounds":
        past_max = _log(rng, 1, 30000)
        return dict(c, n_requests=_log(rng, 1, 64) if new_max == 1 else _log(rng, 1, 8),
                    new_max=new_max, past_min=max(1, past_max // rng.choice([1, 4, 40])),
                    past_max=past_max)
    hq = hkv * rng.choice([1, 3, 4, 6, 8, 12])
    n = _log(rng, 1, 48)
    if op == "prefix":
        prefix_max, own_max = _log(rng, 1, 32768), _log(rng, 1, 2000)
        new_max = min(new_max, 500)
        while n * hq * new_max * (prefix_max + own_max + new_max) > 5e7:
            n, new_max = max(1, n * 3 // 4), max(1, new_max * 3 // 4)
            prefix_max, own_max = max(1, prefix_max * 7 // 8), max(1, own_max * 7 // 8)
        return dict(c, n_requests=n, n_groups=rng.randint(1, min(n, 5)), new_max=new_max,
                    prefix_min=max(1, prefix_max // rng.choice([1, 4])), prefix_max=prefix_max,
                    own_max=own_max, hq=hq)
    past_max = _log(rng, 1, 100000)
    while n * hkv * (past_max + new_max) > 4e5 * 64 / max(dim, 64):
        n, past_max = max(1, n // 2), max(1, past_max * 3 // 4)
    n_select = _log(rng, 4, 64)
    if op == "select":                  # some requests have more pages than are chosen
        n_select = max(4, min(n_select, past_max // (3 * c["page_size"])))
        past_max = max(past_max, 3 * n_select * c["page_size"])
    while n * hq * new_max * n_select * c["page_size"] > 1e8 or \
            op == "select" and n * hq * new_max * (past_max + new_max) // c["page_size"] > 9e7:
        n, new_max, n_select = max(1, n * 3 // 4), max(1, new_max * 3 // 4), max(4, n_select * 7 // 8)
    c.update(n_requests=n, new_max=new_max, past_min=max(1, past_max // rng.choice([1, 4, 40])),
             past_max=past_max, hq=hq, n_select=n_select)
    return dict(c, first=rng.randint(0, 2), last=rng.randint(1, 2)) if op == "select" else c


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
    step = next(s for s in (7, 11, 13, 1) if math.gcd(s, n) == 1)
    if case["op"] == "prefix":
        prefix, cu = _groups(case)
        own_past = [x - 1 for x in _spread(n, 1, case["own_max"])]
        at = [next(g for g in range(len(prefix)) if cu[g + 1] > i) for i in range(n)]
        return [(prefix[at[i]] + own_past[i * step % n], news[i]) for i in range(n)]
    pasts = _spread(n, case["past_min"], case["past_max"])
    return [(pasts[i * step % n], news[i]) for i in range(n)]


def _groups(case):
    """Shared lengths of the groups (whole pages), and the requests they begin with."""
    n, m, ps = case["n_requests"], case["n_groups"], case["page_size"]
    prefix = [-(-x // ps) * ps for x in _spread(m, case["prefix_min"], case["prefix_max"])]
    return prefix, [g * n // m for g in range(m + 1)]


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _normal(shape, g, dt):
    x = torch.empty(shape, dtype=dt, device="cuda")
    for part in x.split(1 << 18):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
    return x


def _batch(case, g):
    """Lengths, and a page table over a pool whose pages are handed out in a random order."""
    ps, lens = case["page_size"], _lengths(case)
    new, kv = [m for _, m in lens], [p + m for p, m in lens]
    held = [-(-x // ps) for x in kv]
    shared = [0] * len(kv)              # pages of a request that its group's first one holds
    first = list(range(len(kv)))
    if case["op"] == "prefix":
        prefix, starts = _groups(case)
        for i in range(len(kv)):
            j = next(j for j in range(len(prefix)) if starts[j + 1] > i)
            first[i] = starts[j]
            shared[i] = 0 if i == starts[j] else prefix[j] // ps
    n_pages = sum(held) - sum(shared) + 2
    pages = torch.randperm(n_pages, generator=g, device="cuda").int()
    table = torch.full((len(kv), max(held)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, h in enumerate(held):
        table[i, :shared[i]] = table[first[i], :shared[i]]
        table[i, shared[i]:h] = pages[at:at + h - shared[i]]
        at += h - shared[i]
    cu = [0]
    for m in new:
        cu.append(cu[-1] + m)
    return dict(cu=_int32(cu), kv=_int32(kv), table=table, page_size=ps, n_pages=n_pages,
                rows=cu[-1], offsets=cu, lens=lens)


def _chosen(case, st, g):
    """Pages of each row and KV head, as a selection by content makes them: the first, the row's own
    and the one before it, and others of the context, of which neighbouring rows share most."""
    ps, H, K = case["page_size"], case["hkv"], case["n_select"]
    out = []
    for past, m in st["lens"]:
        mine = (past + torch.arange(m, device="cuda")) // ps
        moved = (torch.rand((m, H, K), generator=g, device="cuda") < 1 / 16).long().cumsum(0)
        places = torch.rand((m + 1, H, K), generator=g, device="cuda")
        x = (places.gather(0, moved) * (past // ps + 1)).long().clamp(max=past // ps)
        x[..., 0], x[..., 1], x[..., 2] = 0, mine[:, None], (mine[:, None] - 1).clamp(min=0)
        x = x.sort(-1).values
        twice = torch.nn.functional.pad(x[..., 1:] == x[..., :-1], (1, 0))
        x = x.masked_fill(twice, 1 << 40).sort(-1).values
        out.append(torch.where(x < 1 << 40, x, -1).int())
    return torch.cat(out)


def prepare(case, seed):
    g = _generator(seed)
    dt, D, H = _DTYPES[case["dtype"]], case["dim"], case["hkv"]
    st = _batch(case, g)
    st.update(case=case, scale=D ** -0.5)
    S = st["n_pages"] * case["page_size"]
    if case["op"] != "bounds":
        st["q"] = _normal((st["rows"], case["hq"], D), g, dt)
    if case["op"] in ("bounds", "select"):
        # keys of a page lie around a mean of their own; the bounds of the earlier steps are there
        mid = _normal((st["n_pages"], H, D), g, torch.float32) * 0.7
        reach = (2.2 + 0.4 * _normal((st["n_pages"], H, D), g, torch.float32)).abs()
        st["bounds"] = torch.stack((mid - reach, mid + reach), 2).to(dt)
    if case["op"] != "select":
        st["k_cache"] = _normal((S, H, D), g, dt)
    if case["op"] in ("selected", "prefix"):
        st["v_cache"] = _normal((S, H, D), g, dt)
    if case["op"] == "selected":
        st["pages"] = _chosen(case, st, g)
    if case["op"] == "prefix":
        prefix, starts = _groups(case)
        st["prefix"], st["groups"] = _int32(prefix), _int32(starts)
    return st


# ------------------------------------------------------------------------------ plain forms

def _bounds(st):
    ps, bounds, table = st["page_size"], st["bounds"], st["table"]
    pages = st["k_cache"].unflatten(0, (-1, ps))
    at = torch.arange(ps, device=table.device)
    for i, (past, m) in enumerate(st["lens"]):
        if m == 0:
            continue
        e = torch.arange(past // ps, (past + m - 1) // ps + 1, device=table.device)
        x = pages[table[i, e].long()].float()                                    # [e, ps, Hkv, D]
        filled = (e[:, None] * ps + at < past + m)[..., None, None]
        lo = torch.where(filled, x, math.inf).amin(1)
        hi = torch.where(filled, x, -math.inf).amax(1)
        bounds[table[i, e].long()] = torch.stack((lo, hi), 2).to(bounds.dtype)
    return bounds


def _select(st):
    """The scores are in 64 bits: 32 would decide pages next to the last place by their roundings."""
    case, ps, table = st["case"], st["page_size"], st["table"]
    H, K = case["hkv"], case["n_select"]
    out = torch.empty((st["rows"], H, K), dtype=torch.int32, device=table.device)
    for i, (past, m) in enumerate(st["lens"]):
        n = -(-(past + m) // ps)
        e = torch.arange(n, device=table.device)
        lo, hi = st["bounds"][table[i, :n].long()].double().permute(2, 1, 3, 0)  # [Hkv, D, n] each
        for r in range(0, m, 2048):
            rows = slice(st["offsets"][i] + r, st["offsets"][i] + min(r + 2048, m))
            x = st["q"][rows].double().unflatten(1, (H, -1)).transpose(0, 1)     # [Hkv, r, g, D]
            s = torch.matmul(x.clamp(min=0).flatten(1, 2), hi) + torch.matmul(x.clamp(max=0).flatten(1, 2), lo)
            s = s.unflatten(1, x.shape[1:3]).amax(2)                             # [Hkv, r, n]
            mine = (past + r + torch.arange(s.shape[1], device=table.device)) // ps
            mine = mine[:, None]
            s = torch.where((e < case["first"]) | (e > mine - case["last"]), math.inf, s)
            s = torch.where(e <= mine, s, -math.inf)
            s, page = s.sort(dim=-1, descending=True, stable=True)
            page = torch.where(s > -math.inf, page, n)[..., :K].sort(-1).values
            page = torch.nn.functional.pad(page, (0, max(0, K - n)), value=n)
            out[rows] = torch.where(page < n, page, -1).int().transpose(0, 1)
    return out


def _softmax(s, v):
    """Weighted sums of v and the log-sum-exps of s [..., m, n]; rows of -inf give 0 and -inf."""
    m = s.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    s = (s - m).exp()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s, v)
    return torch.where(total > 0, o / total, torch.zeros_like(o)), (m + total.log()).squeeze(-1)


def _selected(st):
    case, ps, table, q = st["case"], st["page_size"], st["table"].long(), st["q"]
    H, dev = case["hkv"], table.device
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=dev)
    head, at = torch.arange(H, device=dev)[:, None], torch.arange(ps, device=dev)
    step = max(1, (1 << 29) // (H * case["n_select"] * ps * case["dim"]))
    for i, (past, m) in enumerate(st["lens"]):
        for r in range(0, m, step):
            rows = slice(st["offsets"][i] + r, st["offsets"][i] + min(r + step, m))
            page = st["pages"][rows].long()                                      # [r, Hkv, K]
            p = past + r + torch.arange(page.shape[0], device=dev)
            j = (page[..., None] * ps + at).flatten(2)                           # [r, Hkv, K ps]
            ok = (page >= 0)[..., None].expand(-1, -1, -1, ps).flatten(2) & (j <= p[:, None, None])
            slot = (table[i, page.clamp(min=0)][..., None] * ps + at).flatten(2)
            x = q[rows].float().unflatten(1, (H, -1))                            # [r, Hkv, g, D]
            s = torch.matmul(x, st["k_cache"][slot, head].float().transpose(2, 3)) * st["scale"]
            s = torch.where(ok[:, :, None], s, -math.inf)
            o, z = _softmax(s, st["v_cache"][slot, head].float())
            out[rows], lse[rows] = o.flatten(1, 2).to(q.dtype), z.flatten(1, 2)
    return out, lse


def _prefix(st):
    case, ps, table, q = st["case"], st["page_size"], st["table"].long(), st["q"]
    H, dev = case["hkv"], table.device
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=dev)
    for i, (past, m) in enumerate(st["lens"]):
        rows = slice(st["offsets"][i], st["offsets"][i] + m)
        j = torch.arange(past + m, device=dev)
        slot = table[i, j // ps] * ps + j % ps
        k, v = (st[x][slot].float().transpose(0, 1)[:, None] for x in ("k_cache", "v_cache"))
        x = q[rows].float().unflatten(1, (H, -1)).permute(1, 2, 0, 3)            # [Hkv, g, m, D]
        s = torch.matmul(x, k.transpose(2, 3)) * st["scale"]
        s = torch.where(j <= past + torch.arange(m, device=dev)[:, None], s, -math.inf)
        o, z = _softmax(s, v)
        out[rows] = o.permute(2, 0, 1, 3).flatten(1, 2).to(q.dtype)
        lse[rows] = z.permute(2, 0, 1).flatten(1, 2)
    return out, lse


# ------------------------------------------------------------------------------ one pass

def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return {"bounds": _bounds, "select": _select, "selected": _selected, "prefix": _prefix}[op](st)
    from top_sparse_attention_row_gb300 import binding
    batch = (st["cu"], st["kv"], st["table"], st["page_size"])
    if op == "bounds":
        return binding.page_bounds(st["k_cache"], *batch, st["bounds"])
    if op == "select":
        return binding.page_select(st["q"], st["bounds"], *batch, case["n_select"],
                                   n_first=case["first"], n_last=case["last"])
    if op == "selected":
        return binding.selected_attention_paged(st["q"], st["k_cache"], st["v_cache"], st["pages"],
                                                *batch, st["scale"])
    return binding.prefix_attention_paged(st["q"], st["k_cache"], st["v_cache"], *batch, st["scale"],
                                          st["groups"], st["prefix"])


# ------------------------------------------------------------------------------ work

def _distinct(n, draws):
    """Expected number of different pages among so many of n."""
    return n * (1 - (1 - 1 / n) ** draws)


def work(case):
    op, ps, H, D = case["op"], case["page_size"], case["hkv"], case["dim"]
    lens = _lengths(case)
    rows = sum(m for _, m in lens)
    if op == "bounds":
        # the filled rows of the pages that new rows lie in, and two rows out for each of them
        pages = keys = 0
        for p, m in lens:
            pages += (p + m - 1) // ps + 1 - p // ps
            keys += p + m - p // ps * ps
        return {"bytes": 2 * H * D * (keys + 2 * pages) + 4 * pages, "flops": 2 * H * D * keys}
    Hq = case["hq"]
    if op == "select":
        # a product over the 2 D bounds of every page up to a row's own, for each of its heads
        K, pages, scored = case["n_select"], 0, 0
        for p, m in lens:
            pages += -(-(p + m) // ps)
            scored += sum((p + t) // ps + 1 for t in range(m))
        return {"bytes": 2 * D * (rows * Hq + 2 * H * pages) + 4 * (pages + rows * H * K),
                "flops": 4 * D * Hq * scored}
    if op == "selected":
        K, keys, pairs = case["n_select"], 0, 0
        for p, m in lens:
            n = p // ps + 1
            each = min(n, _distinct(n, K - 3) + 3) if n > 3 else n
            keys += min(_distinct(n, (K - 3) * (1 + m / 16)) + 3 + m / ps, -(-(p + m) // ps)) * ps
            pairs += m * (each - 0.5) * ps
        return {"bytes": int(4 * H * D * keys + rows * (Hq * (4 * D + 4) + 4 * H * K)),
                "flops": int(4 * D * Hq * pairs)}
    prefix, starts = _groups(case)
    shared = sum(prefix[g] * (starts[g + 1] - starts[g] - 1) for g in range(len(prefix)))
    keys = sum(p + m for p, m in lens) - shared
    pairs = sum(m * p + m * (m + 1) // 2 for p, m in lens)
    return {"bytes": 4 * H * D * keys + rows * Hq * (4 * D + 4) + 4 * (keys // ps),
            "flops": 4 * D * Hq * pairs}


# ------------------------------------------------------------------------------ 64-bit answers

def _exact_bounds(case, st):
    want, ps = st["bounds"].double(), case["page_size"]
    for i, (past, m) in enumerate(st["lens"]):
        for e in range(past // ps, (past + m - 1) // ps + 1):
            page = int(st["table"][i, e])
            keys = st["k_cache"][page * ps:page * ps + min(ps, past + m - e * ps)].double()
            keys = keys.sort(0).values
            want[page] = torch.stack((keys[0], keys[-1]), 1)
    return want


def _attend(q, k, v, seen, scale):
    """q [Hkv, m, D] over k, v [Hkv, n, D] where seen [Hkv or 1, m, n]."""
    s = torch.baddbmm(torch.where(seen, 0.0, -math.inf).double().expand(q.shape[0], -1, -1), q,
                      k.transpose(1, 2), alpha=scale)
    z = torch.logsumexp(s, -1)
    w = torch.exp(s - torch.where(z > -math.inf, z, 0.0)[..., None])
    return torch.bmm(w, v), z


def _exact_selected(case, st):
    ps, H, g, D = case["page_size"], case["hkv"], case["hq"] // case["hkv"], case["dim"]
    o = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(o.shape[:2], dtype=torch.float64, device="cuda")
    K = case["n_select"]
    step = max(1, (1 << 28) // (K * ps * D))
    for i, (past, m) in enumerate(st["lens"]):
        phys = torch.nn.functional.pad(st["table"][i].long(), (0, 1))            # the last: no page
        for h in range(H):
            keys, values = (st[x][:, h].unflatten(0, (-1, ps)) for x in ("k_cache", "v_cache"))
            for t in range(0, m, step):
                n = min(step, m - t)
                r = st["offsets"][i] + t
                at = st["pages"][r:r + n, h].long()
                pos = torch.where(at < 0, 1 << 40, at * ps)[:, :, None] + torch.arange(ps, device="cuda")
                seen = pos.view(n, 1, K * ps) <= torch.arange(past + t, past + t + n, device="cuda").view(n, 1, 1)
                q = st["q"][r:r + n, h * g:(h + 1) * g].double()
                x, z = _attend(q, keys[phys[at]].view(n, K * ps, D).double(),
                               values[phys[at]].view(n, K * ps, D).double(), seen.expand(n, g, -1),
                               1 / math.sqrt(D))
                o[r:r + n, h * g:(h + 1) * g], lse[r:r + n, h * g:(h + 1) * g] = x, z
    return o, lse


def _exact_prefix(case, st):
    ps, H, D = case["page_size"], case["hkv"], case["dim"]
    o = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(o.shape[:2], dtype=torch.float64, device="cuda")
    g = case["hq"] // H
    for i, (past, m) in enumerate(st["lens"]):
        n, r = past + m, st["offsets"][i]
        at = st["table"][i, :-(-n // ps)].long()
        k, v = (st[x].unflatten(0, (-1, ps))[at].flatten(0, 1)[:n].double().permute(1, 0, 2)
                for x in ("k_cache", "v_cache"))
        ahead = torch.arange(n, device="cuda")[None] - torch.arange(past, n, device="cuda")[:, None]
        for h in range(g):                      # the h-th head of every group
            x, z = _attend(st["q"][r:r + m, h::g].double().transpose(0, 1), k, v, (ahead <= 0)[None],
                           1 / math.sqrt(D))
            o[r:r + m, h::g], lse[r:r + m, h::g] = x.transpose(0, 1), z.T
    return o, lse


def exact(case, seed):
    if case["op"] == "select":
        return None                      # whole numbers
    st = prepare(case, seed)
    return {"bounds": _exact_bounds, "selected": _exact_selected, "prefix": _exact_prefix}[case["op"]](case, st)
