"""Plain models of the paged 8-bit KV cache for its tests, in 64 bits (or on whole
numbers), written from the definitions in include/cmr_kv8.h."""
import math

import numpy as np
import torch

E4M3_TOP = 448.0


def i32(v, dev):
    return torch.as_tensor(np.asarray(v, dtype=np.int32), device=dev)


def scale_exp(amax):
    """Exponent of the smallest power of two s with amax <= 448 s, within -60 .. 60."""
    if amax == 0:
        return -60
    return max(-60, min(60, math.ceil(math.log2(amax / E4M3_TOP))))


def encode(x, s):
    """Codes (as torch.uint8) of values x under scales s: e4m3, nearest even, beyond
    +-448 saturated, what is not finite as NaN."""
    y = (x.double() / s).clamp(-E4M3_TOP, E4M3_TOP).float()  # exact: s is a power of two
    c = y.to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.where(torch.isfinite(x), c, torch.full_like(c, 0x7F))


class Cache:
    """A pool with its table, its pages handed out in a shuffled order."""

    def __init__(self, dev, counts, L=1, hk=2, D=256, P=64, spare=3, max_pages=None, seed=0,
                 fill=None):
        g = torch.Generator(device=dev).manual_seed(seed)
        pages = sum(counts) + spare
        self.dev, self.L, self.hk, self.D, self.P, self.pages = dev, L, hk, D, P, pages
        shape = (L, pages, hk, P, D)
        if fill is None:  # finite codes: 0x7f and 0xff are NaN
            codes = [torch.randint(0, 0x7F, shape, generator=g, device=dev, dtype=torch.uint8)
                     + 128 * torch.randint(0, 2, shape, generator=g, device=dev,
                                           dtype=torch.uint8) for _ in range(2)]
            exps = [torch.randint(-9, -5, shape[:3], generator=g, device=dev) for _ in range(2)]
        else:
            codes = [torch.full(shape, fill, dtype=torch.uint8, device=dev) for _ in range(2)]
            exps = [torch.zeros(shape[:3], device=dev) for _ in range(2)]
        self.k, self.v = (c.view(torch.float8_e4m3fn) for c in codes)
        self.ks, self.vs = (torch.exp2(e.float()) for e in exps)
        order = np.random.default_rng(seed).permutation(pages)
        cols = max(max(counts, default=1), 1) if max_pages is None else max_pages
        t = np.full((max(len(counts), 1), cols), -1, np.int32)
        at = 0
        for r, c in enumerate(counts):
            t[r, :c] = order[at:at + c]
            at += c
        self.table = torch.from_numpy(t).to(dev)

    def pool(self):
        return self.k, self.v, self.ks, self.vs

    def values(self, which, layer, row, h, n):
        """The first n tokens of a row's K ('k') or V ('v'), in 64 bits."""
        pages = self.table[row, :-(-n // self.P)].long()
        codes, scales = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        c = codes.view(torch.uint8)[layer, pages, h].view(torch.float8_e4m3fn).double()
        return (c * scales[layer, pages, h].double()[:, None, None]).reshape(-1, self.D)[:n]


def attend(q, cache, spans, scale, slot=None):
    """(out, tolerance) of causal attention in 64 bits: spans is (lo, hi, offset) of each
    sequence's packed tokens.

    The tolerance counts the roundings that the kernels' comments name: the result's
    to bf16 (2^-8 |o|), the weights' (2^-9 of sum w |v| / sum w), and what a changed
    score does to a weight (its relative size is the score's change, counted twice: in
    the weight and in the sum): q is off by 2^-10 of a scale s with max |q| > 224 s, and the
    fp32 sums over D dims and n tokens by 2^-23 of the sum of magnitudes per addition.
    Weights under 2^-25 of the largest may vanish."""
    L, N, hq, D = q.shape
    G = hq // cache.hk
    out = torch.zeros_like(q, dtype=torch.float64)
    tol = torch.full_like(out, 1e-30)
    for b, (lo, hi, off) in enumerate(spans):
        row = b if slot is None else slot[b]
        n = min(off + hi - lo, cache.table.shape[1] * cache.P)
        if hi == lo or n <= 0:
            continue
        at = torch.arange(off, off + hi - lo, device=q.device)
        unseen = torch.arange(n, device=q.device)[None] > at[:, None]
        for l in range(L):
            for h in range(cache.hk):
                k, v = (cache.values(w, l, row, h, n) for w in "kv")
                # a NaN among the values reaches the tokens that see it, and no others
                spoilt = ((~unseen).double() @ v.isnan().double()) > 0
                v, kf = v.nan_to_num(0.0), k.nan_to_num(0.0)
                for g in range(G):
                    x = q[l, lo:hi, h * G + g].double()
                    s = (x @ k.T * scale).masked_fill(unseen, -math.inf)
                    w = torch.softmax(s, dim=-1).nan_to_num(0.0) if not s.isnan().any() else \
                        torch.softmax(s, dim=-1)
                    w = torch.where((at >= 0)[:, None], w, torch.zeros_like(w))
                    o = (w @ v).masked_fill(spoilt & (at >= 0)[:, None], math.nan)
                    top = x.abs().amax(dim=-1, keepdim=True)
                    off_q = 2.0 ** -10 / 224 * top * kf.abs().sum(dim=-1)
                    off_s = D * 2.0 ** -23 * (x.abs() @ kf.abs().T)
                    change = (abs(scale) * (off_q + off_s)).masked_fill(unseen, 0).amax(-1)
                    mean = w @ v.abs()
                    out[l, lo:hi, h * G + g] = o
                    tol[l, lo:hi, h * G + g] = 2.0 ** -8 * o.abs() + mean * (
                        2.0 ** -9 + 2 * change[:, None] + n * 2.0 ** -23) + \
                        n * 2.0 ** -25 * v.abs().max() + 1e-30
    return out, tol


def assert_within(got, want, tol, what=""):
    got = got.double()
    assert torch.equal(got.isnan(), want.isnan()), f"{what}: NaN in other places"
    fine = ~want.isnan()
    over = ((got - want).abs() / tol)[fine]
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 1.0, f"{what}: off by {worst:.3g} of the tolerance"


class Pages:
    """Table and counts as the page calls change them."""

    def __init__(self, table, refs, P):
        self.t, self.r, self.P, self.status = table.numpy().copy(), refs.numpy().copy(), P, 0

    def count(self, row):
        c = 0
        while c < self.t.shape[1] and self.t[row, c] >= 0:
            c += 1
        return c

    def free_pages(self):
        return [i for i in range(len(self.r)) if self.r[i] <= 0]

    def known(self, slots):
        seen = set()
        for i, s in enumerate(slots):
            ok = 0 <= s < self.t.shape[0] and s not in seen
            seen.add(s)
            yield i, s, ok

    def extend(self, slots, lens):
        free, stop = self.free_pages(), False
        for i, s, ok in self.known(slots):
            if not ok or lens[i] < 0 or -(-lens[i] // self.P) > self.t.shape[1]:
                self.status |= 2
                continue
            have = self.count(s)
            need = max(0, -(-lens[i] // self.P) - have)
            if need > len(free) or (stop and need):
                self.status |= 8
                stop = True
                continue
            for k in range(need):
                self.t[s, have + k] = free.pop(0)
                self.r[self.t[s, have + k]] = 1

    def fork(self, src, dst, lens):
        free, before = self.free_pages(), self.t.copy()
        refs = self.r.copy()
        jobs = []
        for i, d, ok in self.known(dst):
            s, n = src[i], lens[i]
            need = -(-n // self.P)
            if not ok or not 0 <= s < self.t.shape[0] or s == d or n < 0 or \
                    need > self.t.shape[1] or before[d, 0] >= 0 or \
                    any(before[s, k] < 0 or refs[before[s, k]] <= 0 for k in range(need)):
                self.status |= 2
                continue
            if n % self.P and not free:
                self.status |= 8
                continue
            whole = n // self.P
            self.t[d, :whole] = before[s, :whole]
            for k in range(whole):
                self.r[before[s, k]] += 1
            if n % self.P:
                p = free.pop(0)
                self.t[d, whole] = p
                self.r[p] = 1
                jobs.append((before[s, whole], p, n % self.P))
        return jobs

    def free(self, slots):
        for _, s, ok in self.known(slots):
            if not ok:
                self.status |= 2
                continue
            for k in range(self.count(s)):
                self.r[self.t[s, k]] -= 1
                self.t[s, k] = -1

    def compact(self):
        live = [i for i in range(len(self.r)) if self.r[i] > 0]
        c = len(live)
        moved = [i for i in live if i >= c]
        holes = [i for i in range(c) if self.r[i] <= 0]
        goes = dict(zip(moved, holes))
        for a, b in goes.items():
            self.r[b], self.r[a] = self.r[a], 0
        for idx, v in np.ndenumerate(self.t):
            if v in goes:
                self.t[idx] = goes[v]
        return list(goes.items())
