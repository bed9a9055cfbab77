"""Cases for the serving operators around the quantized KV cache, with their plain forms.

Four operators, in the order in which a decode step uses them:

rope    rotary positions applied to queries and keys before they are quantized or scored
bounds  per-page element-wise minimum and maximum of the keys that were appended to a paged cache
sparse  one decode step over the pages that the bounds select for each kv head of each sequence
tree    attention of a tree of drafted tokens over the cache that also holds their keys and values

The plain forms use elementary torch operations in 32 bits (64 where 32 lose what matters: angles
of far positions, page scores next to a border).  The caches are the packed ones of the library:
fp16 norms and P-bit codes of the rotated coordinates, in the record layout of include/tq.h.
"""
import functools
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
# channel groups of a 128-channel head: (width, key bits, value bits) of each group
LAYOUTS = {
    "4": ((128, 4, 4),),
    "3": ((128, 3, 3),),
    "3.5": ((64, 4, 4), (64, 3, 3)),
    "2.5": ((64, 3, 3), (64, 2, 2)),
}
D = 128


# ------------------------------------------------------------------ the cases
def listed():
    llama = dict(Hq=32, Hkv=8)
    return [
        # one new token of each of 64 sequences: q and k of a decode step (latency)
        dict(name="rope step 64", op="rope", n=64, D=128, rot=128, dtype="bf16", inter=False, fused=False, far=8192,
             scaling="bands", **llama),
        # a 32K prompt of the Llama layer, q and k read out of the fused projection's rows
        dict(name="rope prompt 32k", op="rope", n=32768, D=128, rot=128, dtype="bf16", inter=False, fused=True,
             far=32768, scaling="bands", **llama),
        # part of an odd head, interleaved pairs, 32-bit, far positions
        dict(name="rope partial f32", op="rope", n=5001, D=96, rot=40, dtype="f32", inter=True, fused=False, far=131072,
             scaling="yarn", Hq=12, Hkv=3),
        # bounds of the pages that one appended token of each of 64 sequences falls into
        dict(name="bounds step 64", op="bounds", B=64, new=1, ctx=8192, page=64, dtype="bf16", Hkv=8),
        # bounds of a whole 128K prompt
        dict(name="bounds prompt 128k", op="bounds", B=1, new=131072, ctx=131072, page=64, dtype="bf16", Hkv=8),
        # a small odd batch: 7 query heads a kv head, 3-bit cache, fp16 queries
        dict(name="sparse small", op="sparse", B=3, ctx=1500, page=128, select=4, first=1, last=1, layout="3",
             dtype="f16", Hq=28, Hkv=4),
        # the long-context step: 131072 tokens at 2.5 bits, 64 of 2048 pages
        dict(name="sparse long 128k", op="sparse", B=1, ctx=131072, page=64, select=64, first=1, last=2, layout="2.5",
             dtype="bf16", **llama),
        # the serving batch: 64 sequences of up to 8192 tokens at 3.5 bits, 16 of 128 pages
        dict(name="sparse serving", op="sparse", B=64, ctx=8192, page=64, select=16, first=1, last=1, layout="3.5",
             dtype="bf16", **llama),
        # one short conversation with a chain of 5 drafted tokens (latency)
        dict(name="tree small", op="tree", B=1, T=5, ctx=1003, page=0, layout="4", dtype="bf16", **llama),
        # a chat batch, ragged, 23 drafted tokens, one kv head for 7 query heads
        dict(name="tree chat", op="tree", B=16, T=23, ctx=4096, page=128, layout="3", dtype="f16", Hq=28, Hkv=4),
        # the long-context cache with a wide tree
        dict(name="tree long 128k", op="tree", B=1, T=63, ctx=131072, page=64, layout="2.5", dtype="bf16", **llama),
        # the serving batch with 16 drafted tokens a sequence
        dict(name="tree serving", op="tree", B=64, T=16, ctx=8192, page=64, layout="3.5", dtype="bf16", **llama),
    ]


def draw(rng):
    """One more case of the ranges that the listed ones stand for."""
    def size(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))

    heads = rng.choice([(32, 8), (28, 4), (16, 16), (8, 1), (24, 8), (5, 1), (12, 3)])
    c = dict(Hq=heads[0], Hkv=heads[1])
    op = rng.choice(["rope", "bounds", "sparse", "sparse", "tree", "tree"])
    if op == "rope":
        width = rng.choice([64, 80, 96, 128])
        return dict(op=op, n=size(1, 32768), D=width, rot=rng.choice([width, width // 2, 2 * rng.randint(1, width // 2)]),
                    dtype=rng.choice(["bf16", "f16", "f32"]), inter=rng.random() < 0.5, fused=rng.random() < 0.5,
                    far=size(64, 1 << 20), scaling=rng.choice(["none", "linear", "bands", "yarn"]), **c)
    page = rng.choice([64, 128, 256])
    if op == "bounds":
        B = size(1, 64)
        new = size(1, 131072 // B)
        return dict(op=op, B=B, new=new, ctx=new + rng.randint(0, 4096), page=page, dtype=rng.choice(["bf16", "f16", "f32"]),
                    Hkv=c["Hkv"])
    B = size(1, 64)
    if op == "sparse":
        ctx = size(page, min(131072, (64 * 8192 * 8) // (B * c["Hkv"])))
        pages = -(-ctx // page)
        first, last = rng.randint(0, 2), rng.randint(1, 2)
        return dict(op=op, B=B, ctx=ctx, page=page, select=max(first + last, size(1, min(64, 2 * pages))), first=first,
                    last=last, layout=rng.choice(sorted(LAYOUTS)), dtype=rng.choice(["bf16", "f16"]), **c)
    T = size(1, 64)
    most = min(131072, (64 * 8192 * 8) // (B * c["Hkv"]), (64 * 8192 * 16 * 32) // (B * T * c["Hq"]))
    return dict(op=op, B=B, T=T, ctx=size(T + 1, max(T + 1, most)), page=rng.choice([0, page]),
                layout=rng.choice(sorted(LAYOUTS)), dtype=rng.choice(["bf16", "f16"]), **c)


def lengths(case):
    """Cached tokens of every sequence, the drafted or just appended ones among them: ragged, the first one the longest."""
    least = case.get("T", case.get("new", 1))
    return [max(least, case["ctx"] - (b * 977) % (case["ctx"] // 2 + 1)) for b in range(case["B"])]


def drafts(case):
    """Drafted tokens of every sequence (the first has all T)."""
    return [max(1, case["T"] - (b * 5) % (case["T"] // 3 + 1)) for b in range(case["B"])]


def work(case):
    """What one pass cannot do without."""
    if case["op"] == "rope":
        x = case["n"] * (case["Hq"] + case["Hkv"])
        return {"bytes": 2 * x * case["D"] * DTYPES[case["dtype"]].itemsize + 4 * case["n"], "flops": 3 * x * case["rot"]}
    if case["op"] == "bounds":
        es, page = DTYPES[case["dtype"]].itemsize, case["page"]
        rows = case["B"] * case["new"] * case["Hkv"]
        pages = sum(-(-n // page) - (n - case["new"]) // page for n in lengths(case)) * case["Hkv"]
        return {"bytes": (rows + 2 * pages) * D * es, "flops": 2 * rows * D}
    token = sum(w * (kb + vb) // 8 + 6 for w, kb, vb in LAYOUTS[case["layout"]])   # codes and three norms
    if case["op"] == "sparse":
        lens, page = lengths(case), case["page"]
        pages = [-(-n // page) for n in lens]
        tokens = sum(min(n, case["select"] * page) for n in lens) * case["Hkv"]
        rows, rep = case["B"] * case["Hq"], case["Hq"] // case["Hkv"]
        return {"bytes": tokens * token + sum(pages) * case["Hkv"] * 4 * D + rows * 4 * D + case["B"] * case["Hkv"] * 4 * case["select"],
                "flops": tokens * rep * 6 * D + rows * 6 * D * D + sum(pages) * case["Hq"] * 2 * D}
    tokens = sum(lengths(case)) * case["Hkv"]
    rows = sum(drafts(case)) * case["Hq"]
    pairs = sum(n * t for n, t in zip(lengths(case), drafts(case))) * case["Hq"]
    return {"bytes": tokens * token + 2 * case["B"] * case["T"] * case["Hq"] * D * 2 + 8 * case["B"] * case["T"],
            "flops": pairs * 6 * D + rows * sum(6 * w * w for w, _, _ in LAYOUTS[case["layout"]])}


# ------------------------------------------------------------------ parameters of a context
def _normals(seed, n):
    """n standard normals: SplitMix64, 53-bit uniforms, Box-Muller pairs (cos, sin)."""
    with np.errstate(over="ignore"):
        z = np.uint64(seed) + np.arange(1, n + n % 2 + 1, dtype=np.uint64) * np.uint64(0x9E3779B97F4A7C15)
        z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
        z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
        z ^= z >> np.uint64(31)
    u = ((z >> np.uint64(11)).astype(np.float64) + 1.0) * 2.0 ** -53
    r, a = np.sqrt(-2.0 * np.log(u[0::2])), 2.0 * np.pi * u[1::2]
    return np.stack([r * np.cos(a), r * np.sin(a)], 1).reshape(-1)[:n]


@functools.lru_cache(maxsize=None)
def _codebook(d, k):
    """Lloyd-Max levels of the coordinate density (1 - x^2)^((d-3)/2) on [-1, 1]: fixed point of the conditional means."""
    x, w = np.polynomial.legendre.leggauss(96)
    half = 2 ** (k - 1)
    c = (np.arange(half) + 0.5) * 3.0 / (half * math.sqrt(d))     # the positive half: the book is odd
    top = min(1.0, 12.0 / math.sqrt(d))                           # beyond it the density is below 1e-30
    for _ in range(20000):
        t = np.concatenate([[0.0], (c[1:] + c[:-1]) / 2, [top]])
        m, s = (t[1:] + t[:-1]) / 2, (t[1:] - t[:-1]) / 2
        p = m[:, None] + s[:, None] * x
        f = w * np.exp(0.5 * (d - 3) * np.log1p(-p * p))
        new = (f * p).sum(1) / f.sum(1)
        done = np.abs(new - c).max() < 1e-16
        c = new
        if done:
            break
    c = np.concatenate([-c[::-1], c])
    return c, (c[1:] + c[:-1]) / 2


@functools.lru_cache(maxsize=None)
def _params(d, bits, seed, keys):
    """Rotation, sign projection (keys), levels, boundaries and the levels by sign-magnitude code, as a context of this
    seed has them."""
    g = _normals(seed, 2 * d * d if keys else d * d)
    q, r = np.linalg.qr(g[: d * d].reshape(d, d))
    k = bits - 1 if keys else bits
    c, t = _codebook(d, k)
    half = 2 ** (k - 1)
    index = [half - 1 - (i & (half - 1)) if i >> (k - 1) else half + (i & (half - 1)) for i in range(2 * half)]
    if k == 1:
        index = [1, 0]
    dev = lambda a: torch.tensor(np.ascontiguousarray(a), dtype=torch.float64, device="cuda")  # noqa: E731
    return dict(Pi=dev(q * np.sign(np.diag(r))), S=dev(g[d * d:].reshape(d, d)) if keys else None, c=dev(c), t=dev(t),
                by_code=dev(c[index]), code_of=torch.tensor(np.argsort(index), device="cuda"), k=k)


def _bit(P, e, b):
    """Place of code bit b of coordinate e (0..31) of a group: 32 * word + bit."""
    j, s = e % 8, e // 8
    h, t = j // 4, j % 4
    top = 8 * t + 7 - (2 * s + h)
    if P == 1:
        return top
    if P == 4:
        return 32 * s + (4 * j + b if b < 3 else 8 * t + (3 if h else 7))
    if b == P - 1:
        return 32 * (P - 1) + top
    return 4 * j + s if P == 2 else 32 * (s & 1) + 4 * j + 2 * (s >> 1) + b


@functools.lru_cache(maxsize=None)
def _places(d, P):
    """[P, d] places of every code bit in a record."""
    return torch.tensor([[32 * P * (i // 32) + _bit(P, i % 32, b) for i in range(d)] for b in range(P)], device="cuda")


# ------------------------------------------------------------------ inputs
def _pack(code, P):
    """[n, d] codes -> [n, P d / 8] record bytes."""
    n, d = code.shape
    place = _places(d, P).reshape(-1)
    source = torch.argsort(place)                                   # bit of the record -> (plane, coordinate)
    bits = (code[:, source % d] >> (source // d)) & 1
    byte = (bits.reshape(n, P * d // 8, 8) << torch.arange(8, device="cuda")).sum(-1)
    return byte.to(torch.uint8)


def _cache(gen, slots, d, bits, seed, keys):
    """Packed vectors as the quantizer leaves them: directions uniform on the sphere, log-normal lengths."""
    p = _params(d, bits, seed, keys)
    codes = torch.empty(slots, bits * d // 8, dtype=torch.uint8, device="cuda")
    norm = torch.empty(slots, dtype=torch.float16, device="cuda")
    rnorm = torch.empty(slots, dtype=torch.float16, device="cuda") if keys else None
    levels, borders = p["c"].float(), p["t"].float()
    for a in range(0, slots, 1 << 19):
        n = min(1 << 19, slots - a)
        y = torch.randn(n, d, generator=gen, device="cuda")
        y /= y.norm(dim=1, keepdim=True)
        at = torch.bucketize(y, borders)
        code = p["code_of"][at].to(torch.int32)
        if keys:
            rnorm[a:a + n] = (y - levels[at]).norm(dim=1)
            code |= (torch.rand(n, d, generator=gen, device="cuda") < 0.5).to(torch.int32) << p["k"]
        codes[a:a + n] = _pack(code, bits)
        norm[a:a + n] = math.sqrt(d) * torch.exp(0.5 * torch.randn(n, generator=gen, device="cuda"))
    return dict(codes=codes, norm=norm, rnorm=rnorm)


def _frequencies(case):
    """Rotary frequencies of every pair, and the factor on the rotated values, of the usual long-context rules."""
    r = case["rot"]
    f = (500000.0 if case["scaling"] == "bands" else 10000.0) ** (-np.arange(0, r, 2) / r)
    if case["scaling"] == "linear":
        return f / 4.0, 1.0
    if case["scaling"] == "bands":                                   # slow pairs stretched 8 times, a ramp in between
        smooth = np.clip((8192.0 * f / (2 * math.pi) - 1.0) / (4.0 - 1.0), 0, 1)
        return f * (smooth + (1 - smooth) / 8.0), 1.0
    if case["scaling"] == "yarn":
        pair = lambda turns: r * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(10000.0))  # noqa: E731
        lo, hi = max(math.floor(pair(32)), 0), min(math.ceil(pair(1)), r - 1)
        ramp = np.clip((np.arange(r // 2) - lo) / max(hi - lo, 0.001), 0, 1)
        return f / 32.0 * ramp + f * (1 - ramp), 0.1 * math.log(32.0) + 1.0
    return f, 1.0


def _tables(case, gen, max_len):
    """Block table over a shuffled pool with spare pages, and the pool's pages."""
    per = max_len // case["page"]
    pool = case["B"] * per + 3
    return torch.randperm(pool, generator=gen, device="cuda")[: case["B"] * per].to(torch.int32).reshape(case["B"], per), pool


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case=case)
    dt = DTYPES[case["dtype"]]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    if case["op"] == "rope":
        n, w, hq, hk = case["n"], case["D"], case["Hq"], case["Hkv"]
        rows = torch.randn(n, hq + 2 * hk, w, generator=gen, device="cuda").to(dt)
        s["q"], s["k"] = rows[:, :hq], rows[:, hq:hq + hk]
        if not case["fused"]:
            s["q"], s["k"] = s["q"].contiguous(), s["k"].contiguous()
        s["pos"] = torch.randint(0, case["far"], (n,), generator=gen, device="cuda", dtype=torch.int32)
        f, s["factor"] = _frequencies(case)
        s["freq"] = torch.tensor(f, dtype=torch.float64, device="cuda")
        return s
    B, Hkv = case["B"], case["Hkv"]
    page = case["page"]
    lens = lengths(case)
    max_len = -(-max(lens) // page) * page if page else max(lens)
    s["lens"], s["max_len"] = ints(lens), max_len
    if page:
        s["table"], pool = _tables(case, gen, max_len)
    if case["op"] == "bounds":
        s["k"] = torch.randn(B * case["new"], Hkv, D, generator=gen, device="cuda").to(dt)
        s["start"] = ints([n - case["new"] for n in lens])
        s["cu_new"] = ints([case["new"] * b for b in range(B + 1)])
        old = torch.randn(pool, Hkv, 2, D, generator=gen, device="cuda").sort(dim=2).values
        s["bounds"] = old.to(dt)
        return s
    slots = pool * Hkv * page if page else B * Hkv * max_len
    s["groups"] = [(w, kb, vb, 1000 + 2 * g, 1001 + 2 * g) for g, (w, kb, vb) in enumerate(LAYOUTS[case["layout"]])]
    s["kc"] = [_cache(gen, slots, w, kb, sk, True) for w, kb, vb, sk, sv in s["groups"]]
    s["vc"] = [_cache(gen, slots, w, vb, sv, False) for w, kb, vb, sk, sv in s["groups"]]
    s["scale"] = 1.0 / math.sqrt(D)
    if case["op"] == "sparse":
        s["q"] = torch.randn(B, case["Hq"], D, generator=gen, device="cuda").to(dt)
        # bounds as keys of unequal pages leave them
        wide = torch.exp(0.3 * torch.randn(pool, Hkv, 1, 1, generator=gen, device="cuda"))
        mid = 0.5 * torch.randn(pool, Hkv, 1, D, generator=gen, device="cuda")
        half = 2.4 + 0.4 * torch.rand(pool, Hkv, 2, D, generator=gen, device="cuda")
        half[:, :, 0] *= -1
        s["bounds"] = (wide * (mid + half)).to(dt)
    else:
        T = case["T"]
        s["q"] = torch.randn(B, T, case["Hq"], D, generator=gen, device="cuda").to(dt)
        s["drafts"] = ints(drafts(case))
        rng = np.random.RandomState(int(seed) % (1 << 31))
        mask = np.zeros((B, T), dtype=np.uint64)
        for b in range(B):
            for j in range(T):                                        # a random tree: parents come first, -1 is the last cached token
                up = rng.randint(-1, j) if j else -1
                mask[b, j] = (mask[b, up] if up >= 0 else np.uint64(0)) | (np.uint64(1) << np.uint64(j))
        s["mask"] = torch.tensor(mask.view(np.int64), device="cuda").reshape(B, T, 1)
    if own:
        s["plan"] = _plan(s)
    return s


# ------------------------------------------------------------------ plain forms
def _rotated(c, p, key):
    """Stored vectors in the rotated basis, 32 bits: levels times norm and, for keys, signs times both norms."""
    d, P = p["Pi"].shape[0], p["k"] + key
    place = _places(d, P)
    words = c["codes"].view(torch.int32)
    code = (((words[..., place >> 5] >> (place & 31)) & 1) << torch.arange(P, device="cuda", dtype=torch.int32)[:, None]).sum(-2)
    n = c["norm"].float()[..., None]
    level = p["by_code"].float()[code & (2 ** p["k"] - 1)] * n
    return (level, ((code >> p["k"]) * 2 - 1).float() * (c["rnorm"].float()[..., None] * n)) if key else (level, None)


def _attend(s, slots, q, keep):
    """softmax(scale q k) v over the cache's slots [B, Hkv, L]; q [B, Hkv, R, D] in 32 bits, keep [B, 1 or Hkv, 1 or R, L]."""
    logit, off, out = 0.0, 0, []
    take = lambda c: {n: None if x is None else x[slots] for n, x in c.items()}  # noqa: E731
    parts = [(w, _params(w, kb, sk, True), _params(w, vb, sv, False), kc, vc) for (w, kb, vb, sk, sv), kc, vc in zip(s["groups"], s["kc"], s["vc"])]
    for w, pk, pv, kc, vc in parts:
        level, sign = _rotated(take(kc), pk, True)
        x = q[..., off:off + w]
        logit = logit + (x @ pk["Pi"].float().T) @ level.transpose(-1, -2)
        logit = logit + math.sqrt(math.pi / 2) / w * ((x @ pk["S"].float().T) @ sign.transpose(-1, -2))
        off += w
    logit = (logit * s["scale"]).masked_fill_(~keep, -math.inf)
    top = logit.amax(-1, keepdim=True)
    e = torch.exp(logit - torch.where(top == -math.inf, 0.0, top))
    total = e.sum(-1, keepdim=True)
    for w, pk, pv, kc, vc in parts:
        level, _ = _rotated(take(vc), pv, False)
        out.append(torch.where(total > 0, (e @ level) / total, 0.0) @ pv["Pi"].float())
    return torch.cat(out, -1)


def _slots(s, logical):
    """Slots of token numbers [B, Hkv, L] of each sequence."""
    B, Hkv, _ = logical.shape
    b = torch.arange(B, device="cuda")[:, None, None]
    h = torch.arange(Hkv, device="cuda")[None, :, None]
    page = s["case"]["page"]
    if not page:
        return (b * Hkv + h) * s["max_len"] + logical
    return (s["table"].long()[b, logical // page] * Hkv + h) * page + logical % page


def _rope_plain(s):
    a = s["pos"].double()[:, None, None] * s["freq"]
    co, si = (torch.cos(a) * s["factor"]).float(), (torch.sin(a) * s["factor"]).float()
    r = s["case"]["rot"]

    def turned(x):
        v, rest = x[..., :r].float(), x[..., r:]
        if s["case"]["inter"]:
            u, v = v[..., 0::2], v[..., 1::2]
            y = torch.stack([u * co - v * si, v * co + u * si], -1).flatten(-2)
        else:
            u, v = v[..., : r // 2], v[..., r // 2:]
            y = torch.cat([u * co - v * si, v * co + u * si], -1)
        return torch.cat([y.to(x.dtype), rest], -1)

    return turned(s["q"]), turned(s["k"])


def _bounds_plain(s):
    c = s["case"]
    B, new, page = c["B"], c["new"], c["page"]
    t = s["start"].long()[:, None] + torch.arange(new, device="cuda")
    at = torch.gather(s["table"].long(), 1, t // page).reshape(-1)            # physical page of every row
    k = s["k"].float()
    spread = at[:, None, None].expand_as(k)
    old = s["bounds"].float()
    fresh = torch.zeros(old.shape[0], dtype=torch.bool, device="cuda")
    fresh[at[(t % page == 0).reshape(-1)]] = True                             # the page's first token came: what was there is void
    start = torch.where(fresh[:, None, None, None], torch.tensor([math.inf, -math.inf], device="cuda")[:, None], old)
    lo = start[:, :, 0].scatter_reduce(0, spread, k, "amin")
    hi = start[:, :, 1].scatter_reduce(0, spread, k, "amax")
    s["bounds"].copy_(torch.stack([lo, hi], 2))
    return s["bounds"]


def _selected(s):
    """Pages of each (sequence, kv head), ascending, -1 behind the last: the highest sums over the group's query heads of
    sum_c max(q_c lo_c, q_c hi_c), the first and last pages in any case, ties to the lower page."""
    c = s["case"]
    B, Hkv = c["B"], c["Hkv"]
    q = s["q"].double().reshape(B, Hkv, -1, 1, D)
    box = s["bounds"].double()[s["table"].long()].permute(0, 2, 3, 1, 4)      # [B, Hkv, 2, pages, D]
    score = torch.maximum(q * box[:, :, None, 0], q * box[:, :, None, 1]).sum((2, 4))
    n = (s["lens"].long()[:, None, None] + c["page"] - 1) // c["page"]
    p = torch.arange(score.shape[-1], device="cuda")
    score = torch.where((p < c["first"]) | (p >= n - c["last"]), math.inf, score).masked_fill(p >= n, -math.inf)
    order = torch.sort(-score, dim=-1, stable=True).indices[..., : c["select"]]
    order = torch.where(torch.gather((p < n).expand_as(score), -1, order), order, 1 << 30).sort(-1).values
    order = torch.nn.functional.pad(order, (0, c["select"] - order.shape[-1]), value=1 << 30)
    return torch.where(order == 1 << 30, -1, order).to(torch.int32)


def _sparse_plain(s):
    c = s["case"]
    B, Hkv, page = c["B"], c["Hkv"], c["page"]
    chosen = _selected(s)
    token = (chosen.long().clamp(min=0)[..., None] * page + torch.arange(page, device="cuda")).flatten(-2)
    keep = (chosen >= 0).repeat_interleave(page, -1) & (token < s["lens"].long()[:, None, None])
    q = s["q"].float().reshape(B, Hkv, -1, D)
    out = _attend(s, _slots(s, token), q, keep[:, :, None])
    return out.reshape(B, c["Hq"], D).to(s["q"].dtype), chosen


def _tree_plain(s):
    c = s["case"]
    B, T, Hq, Hkv = c["B"], c["T"], c["Hq"], c["Hkv"]
    rep = Hq // Hkv
    t = torch.arange(s["max_len"], device="cuda")
    lens, n = s["lens"].long()[:, None, None], s["drafts"].long()[:, None, None]
    i = t - (lens - n)                                                        # [B, 1, L]: drafted token, negative in the context
    bit = (s["mask"] >> i.clamp(0, 63)) & 1
    keep = (t < lens) & ((i < 0) | (bit == 1)) & (torch.arange(T, device="cuda")[:, None] < n)
    q = s["q"].float().reshape(B, T, Hkv, rep, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * rep, D)
    out = _attend(s, _slots(s, t.expand(B, Hkv, -1)), q, keep.repeat_interleave(rep, 1)[:, None])
    return out.reshape(B, Hkv, T, rep, D).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D).to(s["q"].dtype)


# ------------------------------------------------------------------ the framework's calls
@functools.lru_cache(maxsize=None)
def _context(d, bits, seed, keys):
    import kv_cache_vector_08_b200 as tq
    return tq.Context(d, bits, seed, tq.MODE_PROD if keys else tq.MODE_MSE)


def _plan(s):
    """The plan that a serving loop keeps for its caches."""
    import kv_cache_vector_08_b200 as tq
    c = s["case"]
    kctx = [_context(w, kb, sk, True) for w, kb, vb, sk, sv in s["groups"]]
    vctx = [_context(w, vb, sv, False) for w, kb, vb, sk, sv in s["groups"]]
    kc, vc = ([tq.Packed(x["codes"], x["norm"], x["rnorm"]) for x in s[n]] for n in ("kc", "vc"))
    off = [0] + [w for w, *_ in s["groups"]][:-1] + [D]
    args = (kctx, vctx, off, kc, vc, c["B"])
    paged = dict(block_table=s["table"], page_tokens=c["page"]) if c["page"] else {}
    if c["op"] == "tree":
        return tq.TreePlan(*args, c["T"], c["Hq"], c["Hkv"], D, s["max_len"], **paged)
    return tq.SparsePlan(*args, c["Hq"], c["Hkv"], D, s["max_len"], select=c["select"], first=c["first"], last=c["last"], **paged)


def _call(s):
    import kv_cache_vector_08_b200 as tq
    c = s["case"]
    if c["op"] == "rope":
        return tq.rope(s["q"], s["k"], s["pos"], s["freq"], interleaved=c["inter"], factor=s["factor"])
    if c["op"] == "bounds":
        return tq.page_bounds(s["k"], s["cu_new"], s["start"], s["table"], c["page"], s["bounds"], max_new=c["new"])
    if c["op"] == "sparse":
        return s["plan"](s["q"], s["bounds"], s["lens"], s["scale"])
    return s["plan"](s["q"], s["lens"], s["drafts"], s["mask"], s["scale"])


def run(state):
    if own:
        return _call(state)
    return {"rope": _rope_plain, "bounds": _bounds_plain, "sparse": _sparse_plain, "tree": _tree_plain}[state["case"]["op"]](state)


# ------------------------------------------------------------------ the definitions in 64 bits
def _vectors(c, d, bits, seed, keys, slots):
    """64-bit coordinates of the stored vectors of some slots in the rotated basis, taken bit by bit from the records."""
    p = _params(d, bits, seed, keys)
    byte = c["codes"][slots]
    bits_of = (byte[..., None] >> torch.arange(8, device="cuda", dtype=torch.uint8)) & 1
    bits_of = bits_of.flatten(-2)
    planes = [bits_of[..., _places(d, bits)[b]] for b in range(bits)]
    n = c["norm"][slots].double()[..., None]
    neg = planes[p["k"] - 1].bool()
    rank = sum((planes[b].long() << b for b in range(p["k"] - 1)), torch.zeros_like(neg, dtype=torch.long))
    half = 2 ** (p["k"] - 1)
    value = p["c"][half + rank]
    value = torch.where(neg, -value, value) * n
    if not keys:
        return value
    return value, (planes[p["k"]].double() * 2 - 1) * (c["rnorm"][slots].double()[..., None] * n)


def _exact_attention(s, b, h, slots, q, keep):
    """One kv head of one sequence: q [R, D] in 64 bits over the slots, keep [R, L]."""
    logit = torch.zeros(q.shape[0], slots.shape[0], dtype=torch.float64, device="cuda")
    off = 0
    for (w, kb, vb, sk, sv), kc in zip(s["groups"], s["kc"]):
        p = _params(w, kb, sk, True)
        level, sign = _vectors(kc, w, kb, sk, True, slots)
        x = q[:, off:off + w]
        logit += (x @ p["Pi"].T) @ level.T + math.sqrt(math.pi / 2) / w * (x @ p["S"].T) @ sign.T
        off += w
    logit = torch.where(keep, logit * s["scale"], -math.inf)
    some = keep.any(1, keepdim=True)
    weight = torch.where(some, torch.softmax(torch.where(some, logit, 0.0), 1), 0.0)
    out = []
    for (w, kb, vb, sk, sv), vc in zip(s["groups"], s["vc"]):
        out.append((weight @ _vectors(vc, w, vb, sv, False, slots)) @ _params(w, vb, sv, False)["Pi"])
    return torch.cat(out, 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        r = case["rot"]
        z = torch.polar(torch.full((), float(s["factor"]), dtype=torch.float64, device="cuda"), s["pos"].double()[:, None] * s["freq"])[:, None]

        def turned(x):
            y = x.double().clone()
            i = torch.arange(r // 2, device="cuda")
            a, b = (2 * i, 2 * i + 1) if case["inter"] else (i, i + r // 2)
            w = torch.complex(y[..., a], y[..., b]) * z
            y[..., a], y[..., b] = w.real, w.imag
            return y

        return turned(s["q"]), turned(s["k"])
    lens, page = s["lens"].tolist(), case["page"]
    if case["op"] == "bounds":
        box = s["bounds"].double()
        table, start = s["table"].tolist(), s["start"].tolist()
        for b in range(case["B"]):
            k = s["k"][b * case["new"]:(b + 1) * case["new"]].double()
            for p in range(start[b] // page, -(-lens[b] // page)):
                a = max(p * page, start[b])
                rows = k[a - start[b]:min(lens[b], (p + 1) * page) - start[b]]
                lo, hi = rows.amin(0), rows.amax(0)
                at = table[b][p]
                if a > p * page:
                    lo, hi = torch.minimum(lo, box[at, :, 0]), torch.maximum(hi, box[at, :, 1])
                box[at] = torch.stack([lo, hi], 1)
        return box
    B, Hq, Hkv = case["B"], case["Hq"], case["Hkv"]
    rep = Hq // Hkv
    if case["op"] == "sparse":
        out = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
        for b in range(B):
            pages = -(-lens[b] // page)
            box = s["bounds"][s["table"][b, :pages].long()].double()        # [pages, Hkv, 2, D]
            for h in range(Hkv):
                x = s["q"][b, h * rep:(h + 1) * rep].double()
                score = box[:, h, 1] @ x.clamp(min=0).sum(0) + box[:, h, 0] @ x.clamp(max=0).sum(0)
                score[:case["first"]] = math.inf
                score[max(0, pages - case["last"]):] = math.inf
                best = torch.topk(score, min(case["select"], pages)).indices
                t = (best[:, None] * page + torch.arange(page, device="cuda")).flatten()
                t = t[t < lens[b]]
                slots = (s["table"][b].long()[t // page] * Hkv + h) * page + t % page
                rows = s["q"][b, h * rep:(h + 1) * rep].double()
                out[b, h * rep:(h + 1) * rep] = _exact_attention(s, b, h, slots, rows, torch.ones(rep, t.shape[0], dtype=torch.bool, device="cuda"))
        return out, None
    T = case["T"]
    out = torch.zeros(B, T, Hq, D, dtype=torch.float64, device="cuda")
    place = torch.arange(64, device="cuda")
    for b in range(B):
        n, t = int(s["drafts"][b]), torch.arange(lens[b], device="cuda")
        tree = ((s["mask"][b, :n] >> place[:n]) & 1).bool()                  # [n, n]
        keep = torch.cat([torch.ones(n, lens[b] - n, dtype=torch.bool, device="cuda"), tree], 1).repeat_interleave(rep, 0)
        for h in range(Hkv):
            slots = (s["table"][b].long()[t // page] * Hkv + h) * page + t % page if page else (b * Hkv + h) * s["max_len"] + t
            rows = s["q"][b, :n, h * rep:(h + 1) * rep].double().reshape(n * rep, D)
            out[b, :n, h * rep:(h + 1) * rep] = _exact_attention(s, b, h, slots, rows, keep).reshape(n, rep, D)
    return out
