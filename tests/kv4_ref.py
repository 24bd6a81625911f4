"""Plain 64-bit CPU forms of the 4-bit key/value cache and of attention over it, straight from their definitions
(bitnet.h), and the error bounds that the tests hold the kernels to."""
import numpy as np
import torch

PAGE = 64


def quantise(x):
    """Rows x [..., D] fp32 -> (codes uint8, scale f32, minimum f32)."""
    x = np.asarray(x, np.float32)
    lo, hi = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
    span = (hi - lo).astype(np.float32)
    flat = span < np.float32(1e-30)
    d = x.astype(np.float64) - lo
    w = hi.astype(np.float64) - lo
    codes = np.where(flat, 0, np.rint(d * 15.0 / np.where(w > 0, w, 1.0))).astype(np.uint8)
    scale = np.where(flat, np.float32(0), (span / np.float32(15)).astype(np.float32)).astype(np.float32)
    return codes, scale[..., 0], lo[..., 0]


def values(codes, scale, lo):
    return (codes.astype(np.float32) * scale[..., None]).astype(np.float32) + lo[..., None]


def block_parts(cache, D):
    """(k codes, v codes [pages, heads, 64, D], k meta, v meta [pages, heads, 64, 2]) of a cache array (uint8)."""
    P, H, _ = cache.shape
    c = PAGE * D // 2
    out = []
    for i in (0, 1):
        raw = cache[..., i * c:(i + 1) * c].reshape(P, H, PAGE, D // 2)
        codes = np.empty((P, H, PAGE, D), np.uint8)
        codes[..., 0::2], codes[..., 1::2] = raw & 15, raw >> 4
        out.append(codes)
    meta = np.ascontiguousarray(cache[..., 2 * c:]).view(np.float32).reshape(P, H, 2, PAGE, 2)
    return out[0], out[1], meta[:, :, 0], meta[:, :, 1]


def make_block_bytes(kc, vc, km, vm):
    """The inverse of block_parts."""
    P, H = kc.shape[:2]
    parts = [np.ascontiguousarray(c[..., 0::2] | (c[..., 1::2] << 4)).reshape(P, H, -1) for c in (kc, vc)]
    parts += [np.ascontiguousarray(m, np.float32).reshape(P, H, -1).view(np.uint8) for m in (km, vm)]
    return np.concatenate(parts, -1)


class Case:
    """A random cache with its plan: `counts` new rows and `lens` tokens per sequence, pages in random order, the
    table's unused entries -1, and NaN scales in every slot that holds no token."""

    def __init__(self, seed, counts, lens, Hkv, D, spare=2, gain=1.0, most=None):
        r = np.random.default_rng(seed)
        per = [(n + PAGE - 1) // PAGE for n in lens]
        self.counts, self.lens, self.Hkv, self.D = list(counts), list(lens), Hkv, D
        P = sum(per) + spare
        order = r.permutation(P).astype(np.int32)
        table = np.full((len(lens), most or max(max(per), 1)), -1, np.int32)
        at = 0
        for b, n in enumerate(per):
            table[b, :n] = order[at:at + n]
            at += n
        self.table = table
        self.q_start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.T = int(self.q_start[-1])
        rows = (r.standard_normal((2, P, Hkv, PAGE, D)) * gain).astype(np.float32)
        rows[0, ..., :: 17] *= 4
        rows[1] += 0.5
        kc, ks, kl = quantise(rows[0])
        vc, vs, vl = quantise(rows[1])
        km, vm = np.stack([ks, kl], -1), np.stack([vs, vl], -1)
        used = np.zeros((P, PAGE), bool)
        for b, n in enumerate(lens):
            for j in range(n):
                used[table[b, j // PAGE], j % PAGE] = True
        km[np.broadcast_to(~used[:, None, :], km.shape[:3])] = np.nan
        vm[np.broadcast_to(~used[:, None, :], vm.shape[:3])] = np.nan
        self.kc, self.vc, self.km, self.vm = kc, vc, km, vm
        self.cache = make_block_bytes(kc, vc, km, vm)

    def kv(self, b):
        """(K, V) [Hkv, len, D] in float64 of sequence b, and the scales [2, Hkv, len]."""
        n = self.lens[b]
        pg = self.table[b, :(n + PAGE - 1) // PAGE]
        out, sc = [], []
        for c, m in ((self.kc, self.km), (self.vc, self.vm)):
            x = c[pg].astype(np.float64) * m[pg][..., :1] + m[pg][..., 1:]
            out.append(x.transpose(1, 0, 2, 3).reshape(self.Hkv, -1, self.D)[:, :n])
            sc.append(m[pg][..., 0].transpose(1, 0, 2).reshape(self.Hkv, -1)[:, :n])
        return out[0], out[1], np.stack(sc)

    def dev(self):
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        return dict(cache=t(self.cache), q_start=t(self.q_start), kv_lens=t(np.array(self.lens, np.int32)),
                    page_table=t(self.table))


def attention(case, q, scale, causal=True, window=0, skip_pages=()):
    """(out, bound) float64 [T, Hq, D]: the definition, and how far a kernel's fp32 result may be from it.

    Bound: the score of a key is a sum of D products formed from exact integer codes in fp32 (at most 2 D / 16 + 8
    roundings of at most 2^-23 of sum|q| max|k| on the way), so it is off by at most d = |scale| sum|q| max|k|
    (2 D / 16 + 8) 2^-23, plus 2^-22 |score| for its scaling into the exponential and 2^-21 for the exponential itself.
    Probabilities are then off by a factor of 1 +- 2 e, e the sum of these, and the output by 2 e max|v|, plus the fp32
    sums over n keys: (n / 8 + 64) 2^-24 max(|min| + 15 s) (a running sum is split over at least 8 partial sums)."""
    Hq, D = q.shape[1], case.D
    G = Hq // case.Hkv
    out = np.zeros((case.T, Hq, D))
    bound = np.zeros((case.T, Hq, D))
    for b, n in enumerate(case.counts):
        L = case.lens[b]
        if n == 0 or L == 0:
            continue
        K, V, sc = case.kv(b)
        pos = np.arange(L - n, L)[:, None]
        j = np.arange(L)[None, :]
        see = np.ones((n, L), bool)
        if causal:
            see = j <= pos
            if window:
                see &= j > pos - window
        for i in skip_pages:
            see &= ~((j // PAGE) == i)
        t0 = int(case.q_start[b])
        for h in range(Hq):
            kk, vv = K[h // G], V[h // G]
            qq = q[t0:t0 + n, h].astype(np.float64)
            with np.errstate(invalid="ignore"):
                x = np.where(see, qq @ kk.T * scale, -np.inf)
                m = x.max(1, keepdims=True)
                p = np.where(see, np.exp(x - np.where(np.isfinite(m), m, 0)), 0.0)
            l = p.sum(1, keepdims=True)
            o = np.where(l > 0, (p / np.where(l > 0, l, 1)) @ vv, 0.0)
            out[t0:t0 + n, h] = o
            top = np.where(np.isfinite(m), np.abs(np.where(see, x, 0)).max(1, keepdims=True), 0)
            d = abs(scale) * np.abs(qq).sum(1, keepdims=True) * np.abs(kk).max() * (2 * D / 16 + 8) * 2.0 ** -23
            e = d + 2.0 ** -22 * top + 2.0 ** -21
            vmax = np.abs(vv).max()
            s = sc[1][h // G].max()
            bound[t0:t0 + n, h] = 2 * e * vmax + (L / 8 + 64) * 2.0 ** -24 * (vmax + 15 * s)
            case_s = 7.5 * s  # half a row's range: what a rounded probability multiplies
            case.half_range = max(getattr(case, "half_range", 0.0), case_s)
    return out, bound


def bound_for(case, ref, bound, q_dtype, out_dtype):
    """bound plus what 16-bit types may add: probabilities rounded to fp16 (half a step, 2^-11, of at most half a row's
    range around its middle) and one rounding of the output (finfo.eps / 2)."""
    b = bound.copy()
    if q_dtype != torch.float32:
        b += 2.0 ** -11 * case.half_range
    if out_dtype != torch.float32:
        b += torch.finfo(out_dtype).eps / 2 * (np.abs(ref) + b) + torch.finfo(out_dtype).tiny
    return b
