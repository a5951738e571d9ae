"""Float64 restatement of the serving-step operators: page plans, rotary positions, 4-bit cache rows
and sliding-window attention over a paged cache.  Test infrastructure; it shares no code with the CUDA
path."""
import math

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _e4m3_values():
    """The 127 non-negative finite e4m3 values in order (codes 0 .. 126)."""
    out = []
    for c in range(127):
        e, m = c >> 3, c & 7
        out.append(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(out)


E4M3 = _e4m3_values()


def page_plan(past, new, table, free, head, page_size, max_rows, n_pages=0):
    """Page by page and row by row: (table, cu, kv_lens, positions, slots, head, shortfall)."""
    table = np.array(table, dtype=np.int64)
    n, ppr = table.shape
    cu, kv, pos, slot = [0], [], [], []
    short, taken = 0, min(max(int(head), 0), len(free))
    for i in range(n):
        p, m = max(int(past[i]), 0), max(int(new[i]), 0)
        have = min(-(-p // page_size), ppr)
        want = min(-(-(p + m) // page_size), ppr)
        for e in range(have, want):
            if taken < len(free):
                table[i, e] = free[taken]
                taken += 1
            else:
                table[i, e] = -1
                short += 1
        for x in range(p, p + m):
            if len(pos) == max_rows:
                break
            e = x // page_size
            page = table[i, e] if e < ppr else -1
            ok = page >= 0 and (n_pages == 0 or page < n_pages)
            pos.append(x)
            slot.append(page * page_size + x % page_size if ok else -1)
        cu.append(min(cu[-1] + m, max_rows))
        kv.append(min(p + m, 2 ** 31 - 1))
    pad = [-1] * (max_rows - len(pos))
    return (table, np.array(cu), np.array(kv), np.array(pos + pad, dtype=np.int64),
            np.array(slot + pad, dtype=np.int64), taken, short)


def rope_frequencies(rot, base, scaling="none", factor=1.0, original_len=0.0, beta_fast=32.0,
                     beta_slow=1.0):
    """Radians per token of every pair, and the magnitude."""
    out, mag = [], 1.0
    for i in range(rot // 2):
        w = base ** (-2.0 * i / rot)
        if scaling == "linear":
            w /= factor
        elif scaling == "ntk":
            w = (base * factor ** (rot / (rot - 2.0))) ** (-2.0 * i / rot)
        elif scaling == "turns":
            t = original_len * w / (2 * math.pi)
            k = min(max((t - beta_slow) / (beta_fast - beta_slow), 0.0), 1.0)
            w = k * w + (1 - k) * w / factor
        elif scaling == "yarn":
            at = lambda t: rot * math.log(original_len / (t * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
            lo, hi = max(math.floor(at(beta_fast)), 0), min(math.ceil(at(beta_slow)), rot - 1)
            r = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            w = (1 - r) * w + r * w / factor
            mag = 0.1 * math.log(factor) + 1 if factor > 1 else 1.0
        out.append(w)
    return np.array(out), mag


def rope(x, positions, freqs, magnitude, interleaved, offset, transpose=False):
    """Rows x [R, H, D] (float64) rotated; rows with a negative position come back unchanged."""
    y = np.array(x, dtype=np.float64)
    half = len(freqs)
    for r, pos in enumerate(positions):
        if pos < 0:
            continue
        for i, w in enumerate(freqs):
            ia = offset + (2 * i if interleaved else i)
            ib = offset + (2 * i + 1 if interleaved else i + half)
            c, s = magnitude * math.cos(pos * w), magnitude * math.sin(pos * w)
            if transpose:
                s = -s
            a, b = np.array(y[r, :, ia]), np.array(y[r, :, ib])
            y[r, :, ia], y[r, :, ib] = a * c - b * s, b * c + a * s
    return y


def _nearest(grid, x):
    """Index of the grid's nearest value, ties to the even index, past the end to the last."""
    i = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    low, high = x - grid[i - 1], grid[i] - x
    return np.where((low < high) | ((low == high) & (i % 2 == 1)), i - 1, i)


def fp4_quantise(x, g):
    """x [..., D] -> (codes [..., D] 0 .. 15, scale codes [..., D / 16], values [..., D])."""
    b = np.asarray(x, dtype=np.float64).reshape(*x.shape[:-1], -1, 16) / g
    sc = _nearest(E4M3, np.abs(b).max(-1) / 6)
    s = E4M3[sc][..., None]
    y = np.divide(b, s, out=np.zeros_like(b), where=s > 0)
    m = _nearest(E2M1, np.abs(y))
    codes = m + 8 * np.signbit(y)
    values = np.where(np.signbit(y), -1.0, 1.0) * E2M1[m] * s * g
    return codes.reshape(x.shape), sc, values.reshape(x.shape)


def fp4_pack(codes):
    codes = codes.astype(np.uint8)
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def fp4_values(packed, scales, g):
    """Values of a packed cache: packed [..., D / 2], scales [..., D / 16] e4m3 bytes."""
    codes = np.stack((packed & 15, packed >> 4), -1).reshape(*packed.shape[:-1], -1).astype(int)
    v = np.where(codes >= 8, -1.0, 1.0) * E2M1[codes & 7]
    return v * np.repeat(E4M3[scales.astype(int)], 16, axis=-1) * g


def window_attention(q, k, v, cu, kv_lens, table, page_size, scale, window=0, n_sink=0, rows=None):
    """q [R, Hq, D], k, v [slots, Hkv, D] in float64.  Row r of request i stands at position p =
    kv_len - new + (r - cu[i]) and sees the positions j <= p of its request that are in the window
    (j > p - window; window 0 = all) or among the first n_sink, on pages that exist.  Rows outside every
    request come back as NaN."""
    R, Hq, D = q.shape
    Hkv = k.shape[1]
    n_pages = k.shape[0] // page_size
    o = np.full((R, Hq, v.shape[2]), np.nan)
    lse = np.full((R, Hq), np.nan)
    wanted = None if rows is None else set(int(r) for r in rows)
    for i, kv in enumerate(kv_lens):
        new = cu[i + 1] - cu[i]
        for t in range(new):
            r = cu[i] + t
            if wanted is not None and r not in wanted:
                continue
            p = kv - new + t
            lo = 0 if window <= 0 else max(0, p - window + 1)
            js = [j for j in range(min(n_sink, lo))] + list(range(lo, p + 1)) if p >= 0 else []
            js = np.array([j for j in js if j < kv and j // page_size < table.shape[1]
                           and 0 <= table[i, j // page_size] < n_pages], dtype=np.int64)
            if len(js) == 0:
                o[r], lse[r] = 0.0, -np.inf
                continue
            at = table[i][js // page_size].astype(np.int64) * page_size + js % page_size
            for h in range(Hq):
                s = k[at, h // (Hq // Hkv)] @ q[r, h] * scale
                m = s.max()
                e = np.exp(s - m)
                o[r, h] = (e / e.sum()) @ v[at, h // (Hq // Hkv)]
                lse[r, h] = m + math.log(e.sum())
    return o, lse


def page_bounds(k, cu, kv_lens, table, page_size, bounds):
    """bounds [n_pages, Hkv, 2, D] with the pages that the new rows reach taken anew from k [slots, Hkv, D]."""
    b = np.array(bounds, dtype=np.float64)
    for i, kv in enumerate(kv_lens):
        new = cu[i + 1] - cu[i]
        if new <= 0 or kv <= 0:
            continue
        for e in range(max(kv - new, 0) // page_size, (kv - 1) // page_size + 1):
            page = table[i, e] if e < table.shape[1] else -1
            if 0 <= page < b.shape[0]:
                rows = k[page * page_size:page * page_size + min(page_size, kv - e * page_size)]
                b[page, :, 0], b[page, :, 1] = rows.min(0), rows.max(0)
    return b


def page_select(q, bounds, cu, kv_lens, table, page_size, n_select, n_first, n_last):
    """Pages [R, Hkv, n_select] of every row and KV head, -1 behind the last; rows outside every request: -2."""
    R, Hq, _ = q.shape
    n_pages, Hkv = bounds.shape[:2]
    out = np.full((R, Hkv, n_select), -2, dtype=np.int64)
    for i, kv in enumerate(kv_lens):
        for r in range(cu[i], cu[i + 1]):
            p = kv - (cu[i + 1] - cu[i]) + (r - cu[i])
            mine = p // page_size if p >= 0 else -1
            for h in range(Hkv):
                ranked = []
                for e in range(min(mine + 1, table.shape[1])):
                    if not 0 <= table[i, e] < n_pages:
                        continue
                    lo, hi = bounds[table[i, e], h]
                    x = q[r, h * (Hq // Hkv):(h + 1) * (Hq // Hkv)]
                    s = np.where(x > 0, x * hi, x * lo).sum(-1).max()
                    taken = e < n_first or e > mine - n_last
                    ranked.append((not taken, not np.isnan(s), 0.0 if np.isnan(s) else -s, e))
                pages = sorted(e for *_, e in sorted(ranked)[:n_select])
                out[r, h] = pages + [-1] * (n_select - len(pages))
    return out


def selected_attention(q, k, v, pages, cu, kv_lens, table, page_size, scale, rows=None):
    """Every row (or those of `rows`) over the positions up to its own whose page is listed for its KV head; rows
    outside every request come back as NaN."""
    R, Hq, _ = q.shape
    Hkv, n_pages = k.shape[1], k.shape[0] // page_size
    o, lse = np.full((R, Hq, v.shape[2]), np.nan), np.full((R, Hq), np.nan)
    wanted = None if rows is None else set(int(r) for r in rows)
    for i, kv in enumerate(kv_lens):
        for r in range(cu[i], cu[i + 1]):
            if wanted is not None and r not in wanted:
                continue
            p = kv - (cu[i + 1] - cu[i]) + (r - cu[i])
            for h in range(Hq):
                g = h // (Hq // Hkv)
                at = [table[i, e] * page_size + j for e in sorted(set(int(x) for x in pages[r, g]))
                      if 0 <= e < table.shape[1] and 0 <= table[i, e] < n_pages
                      for j in range(page_size) if e * page_size + j <= p]
                if not at:
                    o[r, h], lse[r, h] = 0.0, -np.inf
                    continue
                s = k[at, g] @ q[r, h] * scale
                m = s.max()
                e = np.exp(s - m)
                o[r, h] = (e / e.sum()) @ v[at, g]
                lse[r, h] = m + math.log(e.sum())
    return o, lse
