"""Sliding-window attention with sink tokens over paged caches, 16-bit and 4-bit, against its float64
restatement (GPU only)."""
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


class Batch:
    """A ragged batch over a shuffled paged cache: lens = [(kv_len, new rows)]."""

    def __init__(self, lens, hq, hkv, dim, ps, dtype="bfloat16", fp4=False, seed=0, pad_rows=0, spread=1.0):
        import torch
        rng = np.random.default_rng(seed)
        self.dt = getattr(torch, dtype)
        self.ps, self.dim = ps, dim
        self.kv = np.array([a for a, _ in lens])
        self.cu = np.concatenate([[0], np.cumsum([b for _, b in lens])])
        self.R = int(self.cu[-1]) + pad_rows
        ppr = max(1, max(-(-a // ps) for a, _ in lens))
        used = sum(-(-a // ps) for a, _ in lens)
        self.n_pages = used + 3
        pages = rng.permutation(self.n_pages)
        self.table = np.full((len(lens), ppr), -1)
        at = 0
        for i, (a, _) in enumerate(lens):
            n = -(-a // ps)
            self.table[i, :n] = pages[at:at + n]
            at += n
        s = self.n_pages * ps
        to = lambda x: torch.from_numpy(x).to(self.dt).cuda()  # noqa: E731
        self.q = to(rng.standard_normal((self.R, hq, dim)) * spread)
        k, v = rng.standard_normal((2, s, hkv, dim))
        self.fp4 = fp4
        if fp4:
            self.kg, self.vg = 0.25, 0.5
            (kc, ks, k), (vc, vs, v) = S.fp4_quantise(k, self.kg), S.fp4_quantise(v, self.vg)
            u8 = lambda x: torch.from_numpy(x.astype(np.uint8)).cuda()  # noqa: E731
            self.k, self.v = u8(S.fp4_pack(kc)), u8(S.fp4_pack(vc))
            self.ks, self.vs = u8(ks), u8(vs)
            self.k64, self.v64 = k, v
        else:
            self.k, self.v = to(k), to(v)
            self.k64, self.v64 = self.k.double().cpu().numpy(), self.v.double().cpu().numpy()
        self.q64 = self.q.double().cpu().numpy()
        self.scale = dim ** -0.5

    def call(self, B, window, n_sink, **kw):
        common = (i32(self.cu), i32(self.kv), i32(self.table), self.ps, self.scale)
        kw = dict(window=window, n_sink=n_sink, **kw)
        if self.fp4:
            return B.window_attention_fp4_paged(self.q, self.k, self.ks, self.v, self.vs, *common,
                                                k_global=self.kg, v_global=self.vg, **kw)
        return B.window_attention_paged(self.q, self.k, self.v, *common, **kw)

    def check(self, B, window, n_sink, rows=None, **kw):
        import torch
        out, lse = self.call(B, window, n_sink, **kw)
        torch.cuda.synchronize()
        assert B.device_status() == 0
        self.compare(out, lse, window, n_sink, rows)
        return out, lse

    def compare(self, out, lse, window, n_sink, rows=None):
        import torch
        n = int(self.cu[-1])
        rows = np.arange(n) if rows is None else np.asarray(rows)
        args = (self.cu, self.kv, self.table, self.ps, self.scale, window, n_sink, rows)
        o, z = S.window_attention(self.q64, self.k64, self.v64, *args)
        a, _ = S.window_attention(self.q64, self.k64, np.abs(self.v64), *args)
        o, z, a = o[rows], z[rows], a[rows]
        got, zg = out.double().cpu().numpy()[rows], lse.double().cpu().numpy()[rows]
        assert np.array_equal(np.isneginf(zg), np.isneginf(z))
        # Weights and output are rounded to the type's half step u (weights of a 4-bit cache to fp16's);
        # with A = sum w |v| / l: |dO| <= u_w A (numerator) + u |O|.  A logit is a sum of dim products in
        # fp32, off by at most dim 2^-23 sum |q k| scale =: d (for N(0, 1) rows sum |q k| scale is at most
        # about 2 sqrt(dim) spread), which changes a weight by a factor e^d and l likewise: 2 d A.
        u = torch.finfo(self.dt).eps / 2
        uw = 2.0 ** -11 if self.fp4 or self.dt == torch.float16 else u
        spread = max(1.0, float(np.std(self.q64)))
        d = self.dim * 2.0 ** -23 * 2 * np.sqrt(self.dim) * spread + 2.0 ** -20
        if self.fp4 and self.dt == torch.bfloat16:
            pass                       # bf16 q is exact in fp16 above 2^-14
        bound = uw * a + u * np.abs(o) + 2 * d * a + 2.0 ** -24
        worst = np.max(np.abs(got - o) - bound)
        assert worst <= 0, (worst, np.max(np.abs(got - o)))
        fin = np.isfinite(z)
        assert np.all(np.abs(zg[fin] - z[fin]) <= d + 2.0 ** -21 * np.abs(z[fin]) + 2.0 ** -22)


DECODE = [(1, 1), (77, 1), (129, 1), (700, 1), (64, 1)]
MIXED = [(5, 5), (300, 40), (513, 1), (257, 130), (64, 64), (3, 3), (40, 2)]


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window,sink", [(0, 0), (100, 4), (1, 0), (33, 40)])
def test_decode(B, dim, window, sink, fp4):
    Batch(DECODE, 6, 2, dim, 16, fp4=fp4, seed=dim + window).check(B, window, sink)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window,sink", [(0, 0), (64, 3), (200, 130)])
def test_mixed_batch(B, dim, window, sink, dtype, fp4):
    Batch(MIXED, 8, 2, dim, 64, dtype, fp4=fp4, seed=dim + sink).check(B, window, sink)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("ps", [1, 2, 3, 7, 8, 12, 24, 48, 64, 100, 128, 256])
def test_page_sizes(B, ps, fp4):
    Batch([(1000, 30), (129, 1), (40, 40)], 4, 2, 128, ps, fp4=fp4, seed=ps).check(B, 150, 5)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (24, 2), (96, 1), (128, 1), (130, 2), (8, 8), (40, 5)])
def test_head_groups(B, hq, hkv):
    for fp4 in (False, True):
        Batch([(400, 37), (90, 1)], hq, hkv, 64, 16, fp4=fp4, seed=hq).check(B, 90, 2)
