"""The operators around the paged FP4 cache, as cases to measure.

norm_rope         RMS norm of every head and rotation by position (queries)
norm_rope_append  the same on new key rows, quantised into the cache
chunk_attn        dense attention of new tokens over the paged cache
attn_mass         attention weight that every cached entry has received
evict             the entries kept by that weight, moved to other pages

`own` false: plain torch operations; true: the package's kernels.
"""
import math
from types import SimpleNamespace

import torch

own = False

DEV = "cuda"
KV, IK = 512, 128
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # queries of one decode step: 8 requests, 64 main heads; latency counts
        {"name": "norm_rope_decode_b8", "op": "norm_rope", "n": 8, "H": 64, "D": 512, "rot": 64, "inter": True,
         "src": "bf16", "dst": "bf16", "gap": 0},
        # indexer queries of a prefill chunk, from a fused projection's output (strided), to the indexer's fp32
        {"name": "norm_rope_index_8191", "op": "norm_rope", "n": 8191, "H": 32, "D": 128, "rot": 64, "inter": False,
         "src": "bf16", "dst": "f32", "gap": 640},
        # one new token of each of 64 requests of a ragged serving batch
        {"name": "append_decode_b64", "op": "append", "n": 64, "B": 64, "page": 128, "rot": 64, "inter": True,
         "src": "bf16"},
        # keys of a long prompt's chunk
        {"name": "append_prompt_32765", "op": "append", "n": 32765, "B": 1, "page": 4096, "rot": 64, "inter": True,
         "src": "bf16"},
        # one token of each of 8 requests over 65,536 positions
        {"name": "attn_decode_b8_64k", "op": "attn", "B": 8, "ctx": 65536, "new": 1, "H": 64, "page": 4096,
         "ragged": False, "ratio": 1},
        # two requests with one new token each over short contexts, 16 heads: latency
        {"name": "attn_decode_b2_4k", "op": "attn", "B": 2, "ctx": 4096, "new": 1, "H": 16, "page": 1024,
         "ragged": False, "ratio": 1},
        # mixed batch: chunks of odd lengths, single tokens among them, over odd contexts
        {"name": "attn_ragged_b6", "op": "attn", "B": 6, "ctx": 7001, "new": 333, "H": 32, "page": 256,
         "ragged": True, "ratio": 1},
        # a long prompt's chunk of 1,024 tokens, 64 heads, over 32,768 positions
        {"name": "attn_chunk_1024_32k", "op": "attn", "B": 1, "ctx": 32768, "new": 1024, "H": 64, "page": 4096,
         "ragged": False, "ratio": 1},
        # weight received in a decode step
        {"name": "mass_decode_b8_64k", "op": "mass", "B": 8, "ctx": 65536, "new": 1, "H": 64, "page": 4096,
         "ragged": False, "ratio": 1},
        # weight received from the last chunk of a prompt, two tokens per entry
        {"name": "mass_chunk_512_16k", "op": "mass", "B": 2, "ctx": 16381, "new": 512, "H": 64, "page": 1024,
         "ragged": False, "ratio": 2},
        # 8 requests cut from 65,536 to 16,384 positions
        {"name": "evict_b8_64k_16k", "op": "evict", "B": 8, "ctx": 65536, "page": 4096, "budget": 16384, "sink": 4,
         "recent": 1024, "ragged": False},
        # a ragged serving batch cut to 4,096 positions each, some requests shorter than that
        {"name": "evict_ragged_b64", "op": "evict", "B": 64, "ctx": 98304, "page": 128, "budget": 4096, "sink": 0,
         "recent": 257, "ragged": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "attn", "attn", "mass", "evict"])
    inter = rng.random() < 0.5
    src = rng.choice(["bf16", "f32"])
    if op == "norm_rope":
        D = rng.choice([128, 512])
        H = rng.choice([1, 5, 16, 32, 64])
        n = _log(rng, 1, min(32768, 2 ** 26 // (H * D)))
        return {"op": op, "n": n, "H": H, "D": D, "rot": rng.choice([0, 32, 64, 128]), "inter": inter, "src": src,
                "dst": rng.choice(["bf16", "f32"]), "gap": rng.choice([0, 128, 640])}
    if op == "append":
        B = _log(rng, 1, 64)
        return {"op": op, "n": max(B, _log(rng, 1, 32765)), "B": B, "page": rng.choice([128, 512, 4096]),
                "rot": rng.choice([0, 64, 128]), "inter": inter, "src": src}
    if op == "evict":
        B = _log(rng, 1, 64)
        ctx = _log(rng, 200, min(262144, 6291456 // B))
        budget = max(1, int(ctx * rng.uniform(0.05, 0.9)))
        sink = int(budget * rng.choice([0, 0.01, 0.2]))
        return {"op": op, "B": B, "ctx": ctx, "page": rng.choice([128, 1024]), "budget": budget, "sink": sink,
                "recent": int(budget * rng.choice([0, 0.1, 0.5])), "ragged": rng.random() < 0.6}
    H = rng.choice([16, 32, 64])
    B = _log(rng, 1, 16)
    ctx = _log(rng, 16, 262144 // B)
    most = min(ctx, 2 ** 31 // (B * H * max(ctx, 1024)))
    new = 1 if rng.random() < 0.4 else _log(rng, 1, max(2, most))
    return {"op": op, "B": B, "ctx": ctx, "new": new, "H": H, "page": rng.choice([128, 256, 1024]),
            "ragged": rng.random() < 0.6, "ratio": rng.choice([1, 1, 2])}


# ------------------------------------------------------------------ inputs --

def _lens(case):
    """Lengths (contexts, new tokens) of the requests: host lists, the same for every seed."""
    B, ctx = case["B"], case["ctx"]
    g = torch.Generator()
    g.manual_seed(B * ctx + case.get("new", 1))
    if not case["ragged"]:
        return [ctx] * B, [case.get("new", 1)] * B
    u, v = torch.rand(B, generator=g).tolist(), torch.rand(B, generator=g).tolist()
    lens = [max(1, int(ctx ** (0.5 + 0.5 * x))) for x in u]
    lens[0] = ctx
    new = [max(1, int(case.get("new", 1) * y ** 2)) for y in v]
    new[0] = case.get("new", 1)
    if B > 2:
        new[1], new[2] = 1, 0      # a single token, and a request without new tokens
    return lens, new


def _pages(lens, page, spare, g):
    """Page table (shuffled pages, -1 behind the last) of requests of these lengths; `spare` more pages."""
    per = [-(-n // page) for n in lens]
    ids = torch.randperm(sum(per) + spare, generator=g).tolist()
    width = max(1, max(per))
    table, at = [], 0
    for p in per:
        table.append(ids[at:at + p] + [-1] * (width - p))
        at += p
    return torch.tensor(table, dtype=torch.int32), ids[at:], len(ids)


def _freqs(rot, base=10000.0):
    i = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
    return base ** (-2.0 * i / max(rot, 1))


def _dtype(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _strided(n, width, gap, dtype, g, scale=1.0):
    """n rows of `width` values out of rows of width + gap (a slice of a wider projection)."""
    x = torch.randn(n, width + gap, generator=g, device=DEV) * scale
    return x.to(dtype)[:, :width]


def _kv_rows(rows, c, g):
    """Packed rows of N(0,1) keys with a scale for each channel."""
    codes = torch.empty(rows, KV // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(rows, KV // 16, dtype=torch.uint8, device=DEV)
    step = 65536
    for a in range(0, rows, step):
        x = torch.randn(min(step, rows - a), KV, generator=g, device=DEV) * c
        cd, sc = quantize_fp4(x)
        codes[a:a + step] = cd
        scales[a:a + step] = sc
    return codes, scales


def _handle(s, page, ctx_len):
    """The package's cache over the state's tensors."""
    from kv_cache_decode_index_b200 import csa2
    c = csa2.Cache(1, 128, s.table, ctx_len, device=DEV)
    c.num_pages, c.page_size = s.num_pages, page
    for name in ("kv_codes", "kv_scales", "ik_codes", "ik_exp"):
        if hasattr(s, name):
            setattr(c, name, getattr(s, name))
    return c


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    h = torch.Generator()
    h.manual_seed(seed + 1)
    s = SimpleNamespace(op=case["op"], eps=1e-6)
    op = case["op"]
    if op == "norm_rope":
        n, H, D = case["n"], case["H"], case["D"]
        s.x = _strided(n, H * D, case["gap"], _dtype(case["src"]), g, 3.0).unflatten(1, (H, D))
        s.w = 1.0 + 0.1 * torch.randn(D, generator=g, device=DEV)
        s.pos = torch.randint(0, 1048576, (n,), generator=g, device=DEV, dtype=torch.int32)
        s.freqs, s.inter, s.dst = _freqs(case["rot"]), case["inter"], _dtype(case["dst"])
        if own:
            from kv_cache_decode_index_b200 import csa2
            s.rope = csa2.Rope(s.freqs, s.inter)
        return s
    if op == "append":
        n, B, page = case["n"], case["B"], case["page"]
        per = [n // B + (1 if b < n % B else 0) for b in range(B)]
        place = torch.Generator()                    # where each request stands: the same for every seed
        place.manual_seed(n + B)
        old = torch.randint(0, 2 * page, (B,), generator=place).tolist() if B > 1 else [0] * B
        lens = [o + p for o, p in zip(old, per)]
        s.table, _, s.num_pages = _pages(lens, page, 0, h)
        s.table = s.table.to(DEV)
        rows = s.num_pages * page
        s.kv_codes = torch.zeros(rows, KV // 2, dtype=torch.uint8, device=DEV)
        s.kv_scales = torch.zeros(rows, KV // 16, dtype=torch.uint8, device=DEV)
        s.ik_codes = torch.zeros(rows, IK, dtype=torch.uint8, device=DEV)
        s.ik_exp = torch.zeros(rows, dtype=torch.uint8, device=DEV)
        both = _strided(n, KV + IK, 0, _dtype(case["src"]), g, 2.0)
        s.kv, s.ik = both[:, :KV], both[:, KV:]      # one projection's output
        c = torch.exp(0.5 * torch.randn(KV, generator=g, device=DEV))
        s.kv_w, s.ik_w = c, 1.0 + 0.1 * torch.randn(IK, generator=g, device=DEV)
        s.req = torch.repeat_interleave(torch.arange(B), torch.tensor(per)).to(torch.int32).to(DEV)
        s.pos = torch.cat([torch.arange(o, o + p) for o, p in zip(old, per)]).to(torch.int32).to(DEV)
        s.rope_pos = s.pos + 500000                  # rotated by the token's place in a longer history
        s.freqs, s.inter, s.page = _freqs(case["rot"]), case["inter"], page
        s.lut = torch.tensor([v for b in range(256) for v in (_grid(b & 15), _grid(b >> 4))], dtype=torch.bfloat16,
                             device=DEV).view(256, 2)
        if own:
            from kv_cache_decode_index_b200 import csa2
            s.cache, s.rope = _handle(s, page, lens), csa2.Rope(s.freqs, s.inter)
        return s
    lens, new = _lens(case)
    page = case["page"]
    s.page = page
    if op == "evict":
        B, budget = case["B"], case["budget"]
        moved = [min(n, budget) if n > budget else 0 for n in lens]
        spare = sum(-(-m // page) for m in moved)
        s.table, free, s.num_pages = _pages(lens, page, spare, h)
        s.table = s.table.to(DEV)
        per = [-(-m // page) for m in moved]
        width, at, dst = -(-budget // page), 0, []
        for p in per:
            dst.append(free[at:at + p] + [-1] * (width - p))
            at += p
        s.dst = torch.tensor(dst, dtype=torch.int32, device=DEV)
        rows = s.num_pages * page
        s.kv_codes = torch.randint(0, 256, (rows, KV // 2), generator=g, device=DEV, dtype=torch.uint8)
        s.kv_scales = torch.randint(0, 126, (rows, KV // 16), generator=g, device=DEV, dtype=torch.uint8)
        s.ik_codes = torch.randint(0, 126, (rows, IK), generator=g, device=DEV, dtype=torch.uint8)
        s.ik_exp = torch.randint(100, 130, (rows,), generator=g, device=DEV, dtype=torch.uint8)
        L = s.table.shape[1] * page
        # heavy-tailed weights; many entries never got any (ties)
        u = torch.rand(B, L, generator=g, device=DEV)
        s.mass = torch.where(u < 0.3, torch.zeros_like(u), torch.exp(4.0 * torch.randn(B, L, generator=g, device=DEV)))
        s.ctx_len = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s.budget, s.sink, s.recent, s.L = budget, case["sink"], case["recent"], max(lens)
        s.mass_out = torch.zeros(B, width * page, device=DEV)
        if own:
            from kv_cache_decode_index_b200 import csa2
            s.cache = _handle(s, page, s.ctx_len)
            s.ws = torch.empty(csa2.evict_workspace_bytes(s.cache), dtype=torch.uint8, device=DEV)
        return s
    # attn, mass
    B, H, ratio = case["B"], case["H"], case["ratio"]
    s.H, s.ratio, s.L, s.S = H, ratio, max(lens), max(new)
    s.table, _, s.num_pages = _pages(lens, page, 0, h)
    s.table = s.table.to(DEV)
    c = torch.exp(0.5 * torch.randn(KV, generator=g, device=DEV))
    s.kv_codes, s.kv_scales = _kv_rows(s.num_pages * page, c, g)
    s.ctx_len = torch.tensor(lens, dtype=torch.int32, device=DEV)
    start = [0]
    for x in new:
        start.append(start[-1] + x)
    pad = 3 if case["ragged"] else 0                 # rows behind the last request's
    n = start[-1] + pad
    s.q_start = torch.tensor(start, dtype=torch.int32, device=DEV)
    # the new tokens are the last of their request; with two tokens an entry the first may see no entry yet
    pos = [n_ctx * ratio - x + j for n_ctx, x in zip(lens, new) for j in range(x)] + [0] * pad
    s.q_pos = torch.tensor([max(-1, p) for p in pos], dtype=torch.int32, device=DEV)
    s.q = torch.randn(n, H, KV, generator=g, device=DEV).to(torch.bfloat16)
    s.scale = 1.0 / math.sqrt(KV)
    s.out, s.lse = torch.zeros(n, H, KV, dtype=torch.bfloat16, device=DEV), torch.zeros(n, H, device=DEV)
    if op == "mass":
        sc, _, req, off = _scores(s)
        m, l = _softmax_sums(sc)
        s.lse = torch.where((torch.arange(n, device=DEV) < s.q_start[-1])[:, None], (m + torch.log(l))[req, off],
                            s.lse)
        s.mass = torch.rand(B, s.table.shape[1] * page, generator=g, device=DEV)   # from earlier steps
        del sc, m, l
    if own:
        from kv_cache_decode_index_b200 import csa2
        s.cache = _handle(s, page, s.ctx_len)
        need = csa2.chunk_attn_workspace_bytes if op == "attn" else csa2.attn_mass_workspace_bytes
        s.ws = torch.empty(need(s.cache, n, H), dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------- plain forms --

def _grid(c):
    return (-1.0 if c & 8 else 1.0) * E2M1[c & 7] + 0.0


def e4m3_nearest(r):
    """Nearest E4M3 value of r >= 0 (ties to even, saturating) and its code."""
    e = torch.floor(torch.log2(torch.clamp(r, min=2.0 ** -6)))
    e = torch.where(torch.exp2(e) > r, e - 1, e).clamp(min=-6.0)
    e = torch.where(torch.exp2(e + 1) <= r, e + 1, e)
    v = (torch.round(r / torch.exp2(e - 3)) * torch.exp2(e - 3)).clamp(max=448.0)
    e = torch.where(torch.exp2(e + 1) <= v, e + 1, e)
    sub = v < 2.0 ** -6
    code = torch.where(sub, v * 512.0, (e + 7) * 8 + (v * torch.exp2(-e) - 1) * 8)
    return v, code.to(torch.uint8)


def quantize_fp4(x):
    """Packed E2M1 codes and E4M3 scales of fp32 rows: s = E4M3(amax / 6), codes = E2M1(x / s)."""
    g = x.double().unflatten(-1, (-1, 16))
    s, sc = e4m3_nearest(g.abs().amax(-1) / 6.0)
    r = g.abs() / torch.where(s > 0, s, torch.ones_like(s))[..., None]
    c = (r > 0.25).to(torch.uint8)
    for at, even in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        c += (r >= at) if even else (r > at)
    c = torch.where(s[..., None] > 0, c, torch.zeros_like(c))
    c = torch.where((g < 0) & (c > 0), c | 8, c).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), sc


def quantize_fp8_row(k):
    """E4M3 codes and exponent byte of fp32 rows: sigma = 2^e, e the smallest with 448 * 2^e >= amax."""
    k = k.double()
    a = k.abs().amax(-1)
    e = torch.ceil(torch.log2(torch.clamp(a, min=2.0 ** -140) / 448.0))
    e = torch.where(448.0 * torch.exp2(e - 1) >= a, e - 1, e)
    e = torch.where(448.0 * torch.exp2(e) < a, e + 1, e).clamp(min=-126.0)
    v, code = e4m3_nearest(k.abs() * torch.exp2(-e)[..., None])
    return torch.where((k < 0) & (v > 0), code | 128, code), (e + 127).to(torch.uint8)


def dequantize_fp4(codes, scales):
    """fp32 rows of packed codes and scales."""
    grid = torch.tensor([_grid(c) for c in range(16)], device=codes.device)
    v = grid[torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).int()]
    return (v.unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def rotate(y, pos, freqs, inter):
    """Rotates the last channels of y [n, ..., D] by pos * freqs (angles in 64 bits)."""
    h = freqs.numel()
    a = pos.double()[:, None] * freqs
    shape = (pos.shape[0],) + (1,) * (y.dim() - 2) + (h,)
    cos, sin = torch.cos(a).to(y.dtype).view(shape), torch.sin(a).to(y.dtype).view(shape)
    flat, r = y[..., :y.shape[-1] - 2 * h], y[..., y.shape[-1] - 2 * h:]
    u, v = (r[..., 0::2], r[..., 1::2]) if inter else (r[..., :h], r[..., h:])
    u, v = u * cos - v * sin, u * sin + v * cos
    r = torch.stack([u, v], dim=-1).flatten(-2) if inter else torch.cat([u, v], dim=-1)
    return torch.cat([flat, r], dim=-1)


def _rows(s, L):
    p = torch.arange(L, device=DEV)
    page = s.table[:, p // s.page].clamp(min=0).long()
    return page * s.page + p % s.page


def _scores(s):
    """Scaled scores [B, S, H, L] (-inf where masked), the keys, and each query's place [req, off]."""
    K = dequantize_fp4(*(t[_rows(s, s.L)] for t in (s.kv_codes, s.kv_scales)))
    n, B = s.q.shape[0], s.table.shape[0]
    i = torch.arange(n, device=DEV)
    req = (i[:, None] >= s.q_start[1:]).sum(1).clamp(max=B - 1)
    off = (i - s.q_start[req]).clamp(max=max(s.S - 1, 0))
    at = s.q_start[:-1, None] + torch.arange(s.S, device=DEV)
    there = at < s.q_start[1:, None]
    at = at.clamp(max=n - 1)
    seen = torch.minimum(torch.div(s.q_pos[at].long() + 1, s.ratio, rounding_mode="floor"), s.ctx_len[:, None].long())
    seen = torch.where(there, seen, torch.zeros_like(seen))
    sc = torch.matmul(s.q[at].float().flatten(1, 2), K.transpose(1, 2)).unflatten(1, (s.S, s.H)) * s.scale
    hidden = torch.arange(s.L, device=DEV) >= seen[:, :, None]
    return sc.masked_fill_(hidden[:, :, None, :], -math.inf), K, req, off


def _softmax_sums(sc):
    m = sc.amax(-1)
    base = torch.where(m == -math.inf, torch.zeros_like(m), m)
    return m, torch.exp(sc - base[..., None]).sum(-1)


def _plain_attn(s):
    sc, K, req, off = _scores(s)
    m = sc.amax(-1, keepdim=True)
    p = sc.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(1, 2), K).unflatten(1, (s.S, s.H)) / torch.where(l > 0, l, torch.ones_like(l))
    live = torch.arange(s.q.shape[0], device=DEV) < s.q_start[-1]
    s.out.copy_(torch.where(live[:, None, None], o[req, off].to(torch.bfloat16), s.out))
    s.lse.copy_(torch.where(live[:, None], (m + torch.log(l))[..., 0][req, off], s.lse))
    return s.out, s.lse


def _plain_mass(s):
    sc, _, req, off = _scores(s)
    at = (s.q_start[:-1, None] + torch.arange(s.S, device=DEV)).clamp(max=s.q.shape[0] - 1)
    lse = s.lse[at]
    p = sc.sub_(torch.where(lse == -math.inf, torch.zeros_like(lse), lse)[..., None]).exp_()
    s.mass[:, :s.L] += p.flatten(1, 2).sum(1)
    return s.mass


def _plain_evict(s):
    p = torch.arange(s.L, device=DEV)
    n = s.ctx_len[:, None].long()
    cut = n > s.budget
    # the order of keeping: the first and the last of a request, then by weight, then by position
    w = s.mass[:, :s.L] + 0.0
    w = torch.where((p < s.sink) | (p >= n - s.recent) | ~cut, torch.full_like(w, math.inf), w)
    w = torch.where(p < n, w, torch.full_like(w, -math.inf))
    order = torch.sort(w, dim=1, descending=True, stable=True).indices[:, :s.budget]
    k = torch.sort(torch.where(torch.gather(p < n, 1, order), order, torch.full_like(order, s.L)), dim=1).values
    k = torch.cat([k, k.new_full((k.shape[0], s.budget - k.shape[1]), s.L)], dim=1)
    there = k < n
    kept = torch.where(there, k, torch.full_like(k, -1)).int()
    new_len = torch.minimum(s.ctx_len, torch.full_like(s.ctx_len, s.budget))
    k = torch.where(there, k, torch.zeros_like(k))
    src = torch.gather(_rows(s, s.L), 1, k)
    j = torch.arange(s.budget, device=DEV)
    to = s.dst[:, j // s.page].clamp(min=0).long() * s.page + j % s.page
    to = torch.where(cut & there, to, src)           # what stays is written onto itself
    for t in (s.kv_codes, s.kv_scales, s.ik_codes, s.ik_exp):
        t[to] = t[src]
    got = torch.gather(s.mass, 1, k)
    s.mass_out[:, :s.budget] = torch.where(cut & there, got, s.mass_out[:, :s.budget])
    return kept, new_len


def _append_outputs(s):
    # codes as the values they stand for; scales and indexer keys are E4M3 as they lie
    return {"kv": s.lut[s.kv_codes.int()], "kv_scale": s.kv_scales.view(torch.float8_e4m3fn),
            "ik": s.ik_codes.view(torch.float8_e4m3fn), "ik_exp": s.ik_exp}


def run(s):
    if own:
        from kv_cache_decode_index_b200 import csa2
        if s.op == "norm_rope":
            return csa2.norm_rope(s.x, s.pos, s.rope, weight=s.w, eps=s.eps, out_dtype=s.dst)
        if s.op == "append":
            csa2.norm_rope_append(s.cache, s.kv, s.ik, s.pos, s.rope, s.rope, rope_pos=s.rope_pos, kv_weight=s.kv_w,
                                  ik_weight=s.ik_w, eps=s.eps, req=s.req)
            return _append_outputs(s)
        if s.op == "attn":
            csa2.chunk_attn(s.cache, s.q, s.q_pos, s.q_start, ratio=s.ratio, scale=s.scale, out=s.out, lse=s.lse,
                            workspace=s.ws)
            return s.out, s.lse
        if s.op == "mass":
            return csa2.attn_mass(s.cache, s.q, s.q_pos, s.lse, s.mass, s.q_start, ratio=s.ratio, scale=s.scale,
                                  workspace=s.ws)
        kept, new_len = csa2.evict(s.cache, s.mass, s.budget, s.dst, sink=s.sink, recent=s.recent,
                                   mass_out=s.mass_out, workspace=s.ws)
        return kept, new_len, s.mass_out, s.kv_codes, s.kv_scales, s.ik_codes, s.ik_exp
    if s.op == "norm_rope":
        x = s.x.float()
        y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s.eps) * s.w
        return rotate(y, s.pos, s.freqs, s.inter).to(s.dst)
    if s.op == "append":
        rows = s.table[s.req.long(), s.pos.long() // s.page].long() * s.page + s.pos.long() % s.page

        def normed(x, w):     # in 64 bits: the codes hang on values next to a border
            x = x.double()
            y = x / torch.sqrt(x.square().mean(-1, keepdim=True) + s.eps) * w
            return rotate(y, s.rope_pos, s.freqs, s.inter).float()
        s.kv_codes[rows], s.kv_scales[rows] = quantize_fp4(normed(s.kv, s.kv_w))
        s.ik_codes[rows], s.ik_exp[rows] = quantize_fp8_row(normed(s.ik, s.ik_w))
        return _append_outputs(s)
    if s.op == "attn":
        return _plain_attn(s)
    if s.op == "mass":
        return _plain_mass(s)
    kept, new_len = _plain_evict(s)
    return kept, new_len, s.mass_out, s.kv_codes, s.kv_scales, s.ik_codes, s.ik_exp


# -------------------------------------------------------------------- work --

def work(case):
    op = case["op"]
    size = {"bf16": 2, "f32": 4}
    if op == "norm_rope":
        v = case["n"] * case["H"] * case["D"]
        return {"bytes": v * (size[case["src"]] + size[case["dst"]]), "flops": 4 * v}
    if op == "append":
        return {"bytes": case["n"] * ((KV + IK) * size[case["src"]] + 417), "flops": 8 * case["n"] * (KV + IK)}
    lens, new = _lens(case)
    if op == "evict":
        kept = sum(case["budget"] for n in lens if n > case["budget"])
        return {"bytes": 4 * sum(lens) + (2 * 417 + 4) * kept, "flops": sum(lens)}
    H, ratio = case["H"], case["ratio"]
    pairs = sum(min(n, max(0, (n * ratio - x + j + 1) // ratio)) for n, x in zip(lens, new) for j in range(x))
    cache = 288 * sum(n for n, x in zip(lens, new) if x)
    q = sum(new) * H
    if op == "attn":
        return {"bytes": cache + q * (KV * 4 + 4), "flops": 4 * KV * H * pairs}
    return {"bytes": cache + q * (KV * 2 + 4) + 8 * sum(n for n, x in zip(lens, new) if x), "flops": 2 * KV * H * pairs}


# ------------------------------------------------------------- from 64 bits --

def _exact_rope(x, w, eps, pos, freqs, inter):
    """x [n, ..., D] in 64 bits: normed, weighted, each pair of channels turned as a complex number."""
    x = x.double()
    y = x * w.double() * (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + eps).pow(-0.5)
    h = freqs.numel()
    if h == 0:
        return y
    lo = y.shape[-1] - 2 * h
    i = torch.arange(h, device=DEV)
    a, b = (lo + 2 * i, lo + 2 * i + 1) if inter else (lo + i, lo + h + i)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), pos.double()[:, None] * freqs)
    turn = turn.reshape(turn.shape[0], *([1] * (y.dim() - 2)), h)
    z = torch.complex(y[..., a], y[..., b]) * turn
    y = y.clone()
    y[..., a], y[..., b] = z.real, z.imag
    return y


def _exact_keys(s, b, n):
    """Keys 0 .. n-1 of request b in 64 bits."""
    pages = s.table[b, :-(-n // s.page)].long()
    rows = (pages[:, None] * s.page + torch.arange(s.page, device=DEV)).reshape(-1)[:n]
    codes, e = s.kv_codes[rows].long(), s.kv_scales[rows].long()
    nib = torch.empty(n, KV, dtype=torch.int64, device=DEV)
    nib[:, 0::2], nib[:, 1::2] = codes % 16, codes // 16
    mag, ex = (nib % 2).double(), (nib // 2) % 4
    v = torch.where(ex == 0, 0.5 * mag, (1 + 0.5 * mag) * 2.0 ** (ex.double() - 1)) * (1 - 2 * (nib // 8)).double()
    m, ex = (e % 8).double(), e // 8
    sc = torch.where(ex == 0, m / 512, (1 + m / 8) * 2.0 ** (ex.double() - 7))
    return v * sc.repeat_interleave(16, dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    if s.op == "norm_rope":
        return _exact_rope(s.x, s.w, s.eps, s.pos, s.freqs, s.inter)
    if s.op == "append":
        kv = _exact_rope(s.kv, s.kv_w, s.eps, s.rope_pos, s.freqs, s.inter).float().double()
        ik = _exact_rope(s.ik, s.ik_w, s.eps, s.rope_pos, s.freqs, s.inter).float().double()
        rows = torch.tensor([int(t[p // s.page]) * s.page + p % s.page for t, p in
                             zip(s.table.cpu()[s.req.cpu().long()], s.pos.tolist())], device=DEV)
        e4m3 = torch.arange(127, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn).double()

        def nearest(grid, r):      # index of the nearest value of an ascending grid, ties to the even index
            at = torch.searchsorted(grid, r.contiguous()).clamp(1, len(grid) - 1)
            lo, hi = grid[at - 1], grid[at]
            up = (r - lo > hi - r) | ((r - lo == hi - r) & (at % 2 == 0))
            return torch.where(up, at, at - 1)
        grid = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
        g = kv.reshape(-1, KV // 16, 16)
        sc = e4m3[nearest(e4m3, g.abs().max(dim=-1).values / 6)]
        v = grid[nearest(grid, g.abs() / sc.clamp(min=2.0 ** -10)[..., None])] * torch.sign(g) * (sc > 0)[..., None]
        out = {"kv": torch.zeros(s.kv_codes.shape[0], KV // 2, 2, dtype=torch.float64, device=DEV),
               "kv_scale": torch.zeros(s.kv_scales.shape, dtype=torch.float64, device=DEV),
               "ik": torch.zeros(s.ik_codes.shape, dtype=torch.float64, device=DEV), "ik_exp": None}
        out["kv"][rows] = v.reshape(-1, KV // 2, 2)
        out["kv_scale"][rows] = sc
        two = torch.exp2(torch.arange(-126, 128, dtype=torch.float64, device=DEV))
        sigma = two[torch.searchsorted(448 * two, ik.abs().max(dim=-1).values)]
        r = ik / sigma[:, None]
        out["ik"][rows] = e4m3[nearest(e4m3, r.abs())] * torch.sign(r)
        return out
    if s.op == "evict":
        got = s.mass_out.double()
        for b, n in enumerate(s.ctx_len.tolist()):
            if n <= s.budget:
                continue
            mid = s.mass[b, s.sink:n - s.recent].double()
            m = s.budget - s.sink - s.recent
            best = torch.sort(torch.argsort(-mid, stable=True)[:m]).values + s.sink
            at = torch.cat([torch.arange(s.sink, device=DEV), best, torch.arange(n - s.recent, n, device=DEV)])
            got[b, :s.budget] = s.mass[b].double()[at]
        return None, None, got, None, None, None, None
    start, lens, pos = s.q_start.tolist(), s.ctx_len.tolist(), s.q_pos.tolist()
    out, lse = s.out.double(), s.lse.double()
    mass = s.mass.double() if s.op == "mass" else None
    for b, n in enumerate(lens):
        if start[b] == start[b + 1]:
            continue
        K = _exact_keys(s, b, n)
        step = max(1, 2 ** 28 // (s.H * n))
        for a in range(start[b], start[b + 1], step):
            z = min(start[b + 1], a + step)
            sc = torch.einsum("ihc,ec->ihe", s.q[a:z].double(), K) / math.sqrt(KV)
            seen = torch.tensor([min(n, max(0, (p + 1) // s.ratio)) for p in pos[a:z]], device=DEV)
            sc[(torch.arange(n, device=DEV) >= seen[:, None])[:, None, :].expand(sc.shape)] = -math.inf
            if mass is not None:
                base = s.lse[a:z].double()
                mass[b, :n] += torch.exp(sc - torch.where(base.isinf(), 0.0, base)[..., None]).sum((0, 1))
            else:
                lse[a:z] = torch.logsumexp(sc, dim=-1)
                out[a:z] = torch.einsum("ihe,ec->ihc", torch.softmax(sc, dim=-1).nan_to_num(0.0), K)
    return mass if mass is not None else (out, lse)
