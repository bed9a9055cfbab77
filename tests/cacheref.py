"""Random packed caches (contiguous or paged, unused slots poisoned) and attention over them in 64 bits,
written from the definitions in include/tq.h (test-side only)."""
import math

import numpy as np

import layout
import oracle

LAYOUTS = {"4": ((128, 4, 4),), "3": ((128, 3, 3),), "3.5": ((64, 4, 4), (64, 3, 3)), "2.5": ((64, 3, 3), (64, 2, 2))}
D = 128


class Cache:
    """Token t of (b, h) in slot[b][h][t]; per group: packed codes, norms and the coordinates they stand for."""

    def __init__(self, rng, kind, B, Hkv, lens, max_len, page=0, poison=True, spread=0.5):
        self.B, self.Hkv, self.lens, self.max_len, self.page = B, Hkv, list(lens), max_len, page
        self.groups = LAYOUTS[kind]
        if page:
            per = max_len // page
            self.pool = B * per + 2
            self.table = rng.permutation(self.pool)[:B * per].astype(np.int32).reshape(B, per)
            slots = self.pool * Hkv * page
        else:
            self.table, slots = None, B * Hkv * max_len
        self.off = [0]
        self.kp, self.vp, self.k, self.v = [], [], [], []
        live = np.zeros(slots, bool)
        for b in range(B):
            for h in range(Hkv):
                live[self.slots(b, h, np.arange(lens[b]))] = True
        for g, (w, kb, vb) in enumerate(self.groups):
            self.off.append(self.off[-1] + w)
            for keys in (True, False):
                bits, seed = (kb, 1000 + 2 * g) if keys else (vb, 1001 + 2 * g)
                p = oracle.make_params(w, bits, seed, 0 if keys else 1)
                k = bits - 1 if keys else bits
                y = rng.standard_normal((slots, w))
                y /= np.linalg.norm(y, axis=1, keepdims=True)
                idx = (y[:, :, None] > p["boundaries"]).sum(-1)
                signs = rng.integers(0, 2, (slots, w)).astype(np.uint8) if keys else None
                norm = (math.sqrt(w) * np.exp(spread * rng.standard_normal(slots))).astype(np.float16)
                rnorm = np.linalg.norm(y - p["centroids"][idx], axis=1).astype(np.float16) if keys else None
                codes = layout.pack(idx, signs, w, k)
                if poison:
                    norm[~live] = np.nan
                    if keys:
                        rnorm[~live] = np.inf
                store = dict(codes=codes, norm=norm, rnorm=rnorm, idx=idx, signs=signs)
                (self.k if keys else self.v).append(store)
                (self.kp if keys else self.vp).append(p)

    def slots(self, b, h, t):
        if self.page:
            return (self.table[b, t // self.page].astype(np.int64) * self.Hkv + h) * self.page + t % self.page
        return (b * self.Hkv + h) * self.max_len + t

    def set_norms(self, b, t, key=None, value=None):
        """Overwrite the norms of one token in every kv head and group."""
        for h in range(self.Hkv):
            s = self.slots(b, h, np.array([t]))
            for kc, vc in zip(self.k, self.v):
                if key is not None:
                    kc["norm"][s] = key
                if value is not None:
                    vc["norm"][s] = value

    def attend(self, b, h, q, tokens, keep, scale, perm=None):
        """q [R, 128] rows over the tokens under keep [R, L] -> (out [R, 128], tolerance [R, 128] without the output's
        rounding).

        Tolerance: keys, queries, levels and their products with norms are carried in 16-bit floats, whose relative
        rounding error is at most 2^-11 and 2e-4 in the mean square; four such factors make 4e-4.  A logit is a sum of
        128 products, so its error is 4e-4 scale |q| |k| / sqrt(128) in the mean square, independent from token to
        token; a weight p_t's relative error e_t is that of its logit.  Channel c of the output then moves by
        sum_t p_t e_t (v_tc - o_c), a sum of independent terms with these known factors: its deviation is the root of
        the sum of their squares, channel by channel (an average over the channels would not do: one token's v_tc - o_c
        is several times its own mean square in some channel).  The weights' own rounding moves it by p_t v_tc 2e-4.
        The values' rounding happens in the rotated coordinates, so it spreads evenly over the channels, as does that of
        the last rotation.  Six standard deviations of each part are allowed."""
        ch = np.arange(D) if perm is None else np.asarray(perm[h])
        s = self.slots(b, h, tokens)
        R, L = keep.shape
        logit, size = np.zeros((R, L)), np.zeros((R, L))
        v = np.zeros((L, D))
        rot = []
        for g, (w, kb, vb) in enumerate(self.groups):
            x = q[:, ch[self.off[g]:self.off[g + 1]]].astype(np.float64)
            kc, p = self.k[g], self.kp[g]
            n, r = kc["norm"][s].astype(np.float64), kc["rnorm"][s].astype(np.float64)
            est = (x @ p["Pi"].T) @ p["centroids"][kc["idx"][s]].T
            est = est + math.sqrt(math.pi / 2) / w * r * ((x @ p["S"].T) @ (2.0 * kc["signs"][s] - 1).T)
            logit += n * est
            size = np.sqrt(size ** 2 + (np.linalg.norm(x, axis=1)[:, None] * n) ** 2 / w)
            vc, p = self.v[g], self.vp[g]
            v[:, self.off[g]:self.off[g + 1]] = vc["norm"][s].astype(np.float64)[:, None] * p["centroids"][vc["idx"][s]]
            rot.append(p["Pi"])
        logit = np.where(keep, logit * scale, -np.inf)
        some = keep.any(1)
        top = np.where(some, logit.max(1, initial=-np.inf), 0.0)
        e = np.where(keep, np.exp(logit - top[:, None]), 0.0)
        p = e / np.where(some, e.sum(1), 1.0)[:, None]
        o = p @ v
        turn = lambda x: np.concatenate([x[:, self.off[g]:self.off[g + 1]] @ rot[g] for g in range(len(rot))], 1)  # noqa: E731
        out, vt = turn(o), turn(v)
        w2 = (p * size * scale) ** 2
        moved = np.maximum(w2 @ vt ** 2 - 2 * out * (w2 @ vt) + out ** 2 * w2.sum(1)[:, None], 0)
        even = np.sqrt((p ** 2 * (v ** 2).sum(1)).sum(1) / D) + np.sqrt((o ** 2).sum(1) / D)
        dev = np.sqrt(moved) + np.sqrt(p ** 2 @ vt ** 2) + even[:, None]
        res = np.zeros_like(out)
        tol = np.zeros_like(out)
        res[:, ch], tol[:, ch] = out, 6 * 4e-4 * dev + 1e-6
        return res, tol


# ------------------------------------------------------------------ the same caches on the GPU
_ctx = {}


def contexts(kind):
    import kv_cache_vector_08_b200 as tq
    if kind not in _ctx:
        _ctx[kind] = ([tq.Context(w, kb, 1000 + 2 * g, tq.MODE_PROD) for g, (w, kb, vb) in enumerate(LAYOUTS[kind])],
                      [tq.Context(w, vb, 1001 + 2 * g, tq.MODE_MSE) for g, (w, kb, vb) in enumerate(LAYOUTS[kind])])
    return _ctx[kind]


def upload(cache, device):
    """(key caches, value caches, block table or None) as the library takes them."""
    import torch
    import kv_cache_vector_08_b200 as tq

    def dev(a):
        return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(device)

    k = [tq.Packed(dev(c["codes"]), dev(c["norm"]), dev(c["rnorm"])) for c in cache.k]
    v = [tq.Packed(dev(c["codes"]), dev(c["norm"]), None) for c in cache.v]
    return k, v, dev(cache.table)


def half_step(dtype):
    import torch
    return torch.finfo(dtype).eps / 2


def check(got, ref, tol, dtype, label=""):
    """got against ref within tol plus the rounding of the output type."""
    g = got.float().cpu().numpy().astype(np.float64)
    err, most = np.abs(g - ref), tol + half_step(dtype) * (np.abs(ref) + tol)
    bad = ~(err <= most)
    assert not bad.any(), "%s: %d of %d outside, worst %.3g at %s (allowed %.3g)" % (
        label, bad.sum(), bad.size, np.nanmax(err), np.argwhere(bad)[0].tolist(), most[bad].min())
