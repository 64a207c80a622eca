"""Plain models of the paged key-value cache and its attention, for the tests: the table as Python
lists, the arithmetic in 64 bits, written from the definitions in include/bwta.h."""
import math

import numpy as np
import torch

BAD, NO_PAGE = 0x8, 0x10


# ------------------------------------------------------------------ table model
class TableModel:
    """What the page calls do to pages / kv_len / refcount (int lists)."""

    def __init__(self, n_slots, max_pages, num_pages, page_size):
        self.pages = [[-1] * max_pages for _ in range(n_slots)]
        self.len = [0] * n_slots
        self.ref = [0] * num_pages
        self.ps, self.max_pages = page_size, max_pages
        self.status = 0

    def need(self, n):
        return -(-n // self.ps)

    def free_list(self):
        return [p for p, r in enumerate(self.ref) if r <= 0]

    def reserve(self, slots, n_new):
        free, left, starved = self.free_list(), None, False
        left = list(free)
        seen = set()
        asked = 0
        for s, g in zip(slots, n_new):
            ok = 0 <= s < len(self.len)
            first = ok and s not in seen
            if ok:
                seen.add(s)
            if not first or g < 0 or self.len[s] < 0 or self.need(self.len[s] + g) > self.max_pages:
                self.status |= BAD
                continue
            want = self.need(self.len[s] + g) - self.need(self.len[s])
            asked += want
            if want and asked > len(free):
                self.status |= NO_PAGE
                continue
            for i in range(want):
                p = left.pop(0)
                self.pages[s][self.need(self.len[s]) + i] = p
                self.ref[p] = 1
            self.len[s] += g

    def free(self, slots):
        for s in slots:
            if not 0 <= s < len(self.len):
                self.status |= BAD
                continue
            n, self.len[s] = self.need(self.len[s]), 0
            for i in range(n):
                p, self.pages[s][i] = self.pages[s][i], -1
                if not 0 <= p < len(self.ref) or self.ref[p] <= 0:
                    self.status |= BAD
                else:
                    self.ref[p] -= 1

    def fork(self, src, dst):
        """Returns the list of (source page, target page) copies."""
        was = list(self.len)
        free, asked, seen, copies, left = self.free_list(), 0, set(), [], None
        left = list(free)
        for s, d in zip(src, dst):
            d_ok = 0 <= d < len(was)
            first = d_ok and d not in seen
            if d_ok:
                seen.add(d)
            if not first or not 0 <= s < len(was) or was[d] != 0 or self.need(was[s]) > self.max_pages:
                self.status |= BAD
                continue
            part = was[s] % self.ps != 0
            asked += part
            if part and asked > len(free):
                self.status |= NO_PAGE
                continue
            full = was[s] // self.ps
            for i in range(full):
                p = self.pages[s][i]
                self.pages[d][i] = p
                if 0 <= p < len(self.ref):
                    self.ref[p] += 1
                else:
                    self.status |= BAD
            if part:
                p = left.pop(0)
                self.ref[p] = 1
                old = self.pages[s][full]
                if 0 <= old < len(self.ref):
                    copies.append((old, p))
                else:
                    self.status |= BAD
                self.pages[d][full] = p
            self.len[d] = was[s]
        return copies

    def compact(self):
        used = [p for p, r in enumerate(self.ref) if r > 0]
        n = len(used)
        moves = list(zip([p for p in used if p >= n], [p for p in self.free_list() if p < n]))
        to = dict(moves)
        for s in range(len(self.len)):
            for i in range(self.need(self.len[s])):
                p = self.pages[s][i]
                if not 0 <= p < len(self.ref) or (p >= n and p not in to):
                    self.status |= BAD
                else:
                    self.pages[s][i] = to.get(p, p)
        for a, b in moves:
            self.ref[b], self.ref[a] = self.ref[a], 0
        return moves, n


# ------------------------------------------------------------------ E4M3 rows
def e4m3_values():
    """The 256 values of E4M3 (NaN at 0x7f and 0xff)."""
    out = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[b] = (-v if b & 128 else v) if (b & 127) != 127 else math.nan
    return out


E4M3 = e4m3_values()


def quantize_rows(x):
    """float64 rows [..., D] -> (bytes, scale), by search over the 127 magnitudes."""
    x = np.asarray(x, np.float64)
    flat = x.reshape(-1, x.shape[-1])
    codes, scales = np.zeros(flat.shape, np.uint8), np.ones(len(flat))
    mags = E4M3[:127]
    for i, row in enumerate(flat):
        top = np.abs(row).max()
        e = 0
        if top > 0:
            e = -15
            while e < 8 and top > 448 * 2.0 ** e:
                e += 1
        lim = 240.0 if e == 8 else 448.0
        y = np.minimum(np.abs(row) / 2.0 ** e, lim)
        hi = np.clip(np.searchsorted(mags, y), 0, 126)      # mags[hi] >= y
        lo = np.maximum(hi - 1, 0)
        dlo, dhi = y - mags[lo], mags[hi] - y
        pick = np.where(dlo < dhi, lo, np.where(dhi < dlo, hi, np.where(lo % 2 == 0, lo, hi)))
        codes[i] = pick | np.where(np.signbit(row), 128, 0).astype(np.int64)
        scales[i] = 2.0 ** e
    return codes.reshape(x.shape), scales.reshape(x.shape[:-1])


# ------------------------------------------------------------------ attention in 64 bits
def attend(q, k, v, pos, scale, window, sinks):
    """q [n, D] at positions pos [n], k, v [t, D] (float64) -> (o [n, D], bound [n, D]).

    bound: how far the kernels' result may be off. With w the weights over their sum and
    A = sum w |v|: the weights are rounded to fp16 (half a step, 2^-11 of each; below 2^-14 of the
    largest half a subnormal step, 2^-25), the scores are fp32 sums of D products (D + 2 roundings
    of 2^-24 of sum |q k|, an absolute error d of the exponent, i.e. a relative one of a weight,
    met by weights and by their sum), exp and the running sums are fp32 (2^-20 covers them for
    these lengths), and the result is rounded to fp16 (2^-11 of it, or 2^-25)."""
    n, t = len(q), len(k)
    o, bound = np.zeros((n, k.shape[1])), np.zeros((n, k.shape[1]))
    for i in range(n):
        p = pos[i]
        if p < 0:
            continue
        j = np.arange(min(t, p + 1))
        if window:
            j = j[(j > p - window) | (j < sinks)]
        x = (k[j] @ q[i]) * scale
        w = np.exp(x - x.max())
        w /= w.sum()
        o[i] = w @ v[j]
        A = w @ np.abs(v[j])
        d = (k.shape[1] + 2) * 2.0 ** -24 * scale * (np.abs(k[j]) @ np.abs(q[i])).max()
        d += 2.0 ** -22 * np.abs(x).max()                   # the exponent's own rounding in fp32
        bound[i] = (2.0 ** -11 * np.abs(o[i]) + 2.0 ** -25 + (2.0 ** -11 + 2 * d + 2.0 ** -20) * A
                    + len(j) * 2.0 ** -25 * np.abs(v[j]).max())
    return o, bound


# ------------------------------------------------------------------ a cache on the GPU
def nan_cache(bt, num_pages, ps, H, D, e4m3, pad=0):
    """A pool whose every value is NaN; `pad` widens the distance of pages."""
    def buf(inner, dtype, fill):
        n = int(np.prod(inner))
        t = torch.full((num_pages, n + pad), fill, dtype=dtype, device="cuda")
        return t[:, :n].unflatten(1, inner) if pad == 0 else t.as_strided(
            (num_pages, *inner), (n + pad, *[int(np.prod(inner[i + 1:])) for i in range(len(inner))]))
    if e4m3:
        return bt.KvCache(buf((H, ps, D), torch.uint8, 0x7f), buf((H, ps, D), torch.uint8, 0xff),
                          buf((H, ps), torch.float32, math.nan), buf((H, ps), torch.float32, math.nan))
    return bt.KvCache(buf((H, ps, D), torch.float16, math.nan), buf((H, ps, D), torch.float16, math.nan))


def cache_values(c):
    """(k, v) of a cache as float64 [pages, heads, page, D]."""
    if c.k.dtype == torch.uint8:
        return tuple(E4M3[x.cpu().numpy()] * s.cpu().numpy().astype(np.float64)[..., None]
                     for x, s in ((c.k, c.k_scale), (c.v, c.v_scale)))
    return c.k.cpu().double().numpy(), c.v.cpu().double().numpy()


class Batch:
    """Sequences of the given lengths on shuffled pages of a pool that is NaN everywhere else."""

    def __init__(self, bt, lens, ps, H, D, e4m3=False, seed=0, pad=0, spare_slots=2, k_scale=1.0):
        r = np.random.default_rng([7, seed])
        self.lens, self.ps, self.H, self.D = list(lens), ps, H, D
        need = [-(-n // ps) for n in self.lens]
        self.num_pages = sum(need) + 3
        self.max_pages = max(need + [1]) + 1
        self.cache = nan_cache(bt, self.num_pages, ps, H, D, e4m3, pad)
        order = r.permutation(self.num_pages)
        n_slots = len(self.lens) + spare_slots
        # sequences sit in slots of a shuffled order
        self.slot_of = r.permutation(n_slots)[:len(self.lens)].astype(np.int32)
        pages = np.full((n_slots, self.max_pages), -1, np.int32)
        kv_len = np.zeros(n_slots, np.int32)
        at = 0
        self.k, self.v = [], []
        ck, cv = self.cache.k, self.cache.v
        for s, n in enumerate(self.lens):
            rows = order[at:at + need[s]]
            at += need[s]
            pages[self.slot_of[s], :need[s]] = rows
            kv_len[self.slot_of[s]] = n
            kk = (r.standard_normal((H, n, D)) * k_scale).astype(np.float16).astype(np.float64)
            vv = (r.standard_normal((H, n, D)) + 0.25).astype(np.float16).astype(np.float64)
            for x, to, sc, keep in ((kk, ck, self.cache.k_scale, self.k), (vv, cv, self.cache.v_scale, self.v)):
                if e4m3:
                    codes, scale = quantize_rows(x)
                    x = E4M3[codes] * scale[..., None]
                keep.append(x)
                for i, p in enumerate(rows):
                    m = min(ps, n - i * ps)
                    sl = slice(i * ps, i * ps + m)
                    if e4m3:
                        to[int(p), :, :m] = torch.from_numpy(codes[:, sl]).cuda()
                        sc[int(p), :, :m] = torch.from_numpy(scale[:, sl].astype(np.float32)).cuda()
                    else:
                        to[int(p), :, :m] = torch.from_numpy(x[:, sl].astype(np.float16)).cuda()
        self.table = bt.KvTable(torch.from_numpy(pages).cuda(), torch.from_numpy(kv_len).cuda(),
                                torch.zeros(self.num_pages, dtype=torch.int32, device="cuda"))
        self.slots = torch.from_numpy(self.slot_of).cuda()

    def queries(self, n_rows, heads, seed=0, size=1.0):
        r = np.random.default_rng([8, seed])
        return (r.standard_normal((n_rows, heads, self.D)) * size).astype(np.float16)

    def check(self, q, out, news, scale, window=0, sinks=0, rows=None):
        """out [rows, heads, D] against 64 bits for sequences with `news` new tokens each."""
        heads = q.shape[1]
        g = heads // self.H
        got = out.detach().cpu().double().numpy()
        at, worst = 0, 0.0
        for s, n in enumerate(news):
            pos = np.arange(n) + self.lens[s] - n
            pick = np.arange(n) if rows is None or n <= rows else np.unique(
                np.concatenate([[0, n - 1], np.linspace(0, n - 1, rows).astype(int)]))
            for h in range(heads):
                o, b = attend(q[at + pick, h].astype(np.float64), self.k[s][h // g], self.v[s][h // g],
                              pos[pick], scale, window, sinks)
                err = np.abs(got[at + pick, h] - o)
                assert not np.isnan(err).any(), (s, h)
                bad = err > b
                assert not bad.any(), (s, h, np.argwhere(bad)[0], err[bad][0], b[bad][0])
                worst = max(worst, float((err / np.maximum(b, 1e-300)).max(initial=0.0)))
            at += n
        return worst
