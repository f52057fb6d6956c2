"""The cache operators in the order in which a serving loop uses them: a
ragged prompt (norm and rotation, append, attention, attention weight), an
eviction, and single tokens after it from a captured graph.  Every step is
compared with its float64 formula on the outputs of the steps before it.
Needs a B200 and libcsa2.so."""
import math

import numpy as np
import pytest
import torch

from oracle import formats as F
from tests import ops_util as O
from tests.test_gpu_evict import plain_kept
from tests.test_gpu_norm_rope import _check as check_norm_rope
from tests.test_gpu_norm_rope import csa2  # noqa: F401

pytestmark = pytest.mark.gpu

SCALE = 1 / math.sqrt(512)
ROT = 64


class Layer:
    """Projections' outputs of n tokens (queries, main-KV row, indexer key side
    by side, as one product would give them) and the weights of the norms."""

    def __init__(self, csa2, H, seed):  # noqa: F811
        self.csa2, self.H = csa2, H
        self.rng = np.random.default_rng(seed)
        self.w = [(1 + 0.1 * self.rng.standard_normal(d)).astype(np.float32) for d in (512, 512, 128)]
        self.fr = O.freqs(ROT)
        self.gpu_w = [torch.from_numpy(w).cuda() for w in self.w]
        self.rope = csa2.Rope(torch.from_numpy(self.fr).cuda())

    def draw(self, n):
        x = self.rng.standard_normal((n, self.H * 512 + 640)).astype(np.float32)
        return torch.from_numpy(x).bfloat16().cuda()

    def split(self, x):
        h = self.H * 512
        return x[:, :h].unflatten(1, (self.H, 512)), x[:, h:h + 512], x[:, h + 512:]

    def run(self, cache, k4, x, pos, slot, req, q, out, lse, mass, start=None):
        """The calls of one step; pos: token positions, slot: their cache rows."""
        xq, kv, ik = self.split(x)
        n = slot.shape[0]
        self.csa2.norm_rope(xq, pos, self.rope, weight=self.gpu_w[0], out=q)
        self.csa2.norm_rope_append(cache, kv[:n], ik[:n], slot, self.rope, self.rope, rope_pos=pos[:n],
                                   kv_weight=self.gpu_w[1], ik_weight=self.gpu_w[2], req=req, ik4=k4)
        # the entry of a token is its slot: it sees everything up to that
        self.csa2.chunk_attn(cache, q, self.seen_pos, start, out=out, lse=lse)
        self.csa2.attn_mass(cache, q, self.seen_pos, lse, mass, start)

    def rows(self, x, pos):
        """Codes and scales of the new main-KV rows, indexer codes and exponents."""
        _, kv, ik = (t.double().cpu().numpy() for t in self.split(x))
        n = len(pos)
        eps = np.float32(1e-6)
        y = O.norm_rope(kv[:n], self.w[1], eps, pos, self.fr, True)[0].astype(np.float32)
        z = O.norm_rope(ik[:n], self.w[2], eps, pos, self.fr, True)[0].astype(np.float32)
        return F.quantize_main_kv(y) + F.quantize_indexer(z)

    def check_queries(self, x, pos, q):
        y, spread = O.norm_rope(self.split(x)[0].double().cpu().numpy(), self.w[0], 1e-6, pos, self.fr, True)
        check_norm_rope(q, y, spread, torch.bfloat16, "queries")


def check_attention(q, K, seen, out, lse, mass, before):
    """One request's queries; returns nothing.  Bounds as in the operators' own
    tests: attention_bounds, and for a weight 2 d per term (d of the scores,
    2^-22 for exp2 and the scaling, 2^-23 |lse|) and n rows' sum."""
    q, out, lse = (t.double().cpu().numpy() for t in (q, out, lse))
    ref = O.attention(q, K, seen, SCALE)
    tol, tol_lse = O.attention_bounds(ref, len(K))
    tol = tol + torch.finfo(torch.bfloat16).eps / 2 * (np.abs(ref["out"]) + tol)
    assert (np.abs(out - ref["out"]) <= tol).all()
    assert (np.abs(lse - ref["lse"]) <= tol_lse).all()
    fine = np.isfinite(ref["s"])
    p = np.where(fine, np.exp(np.where(fine, ref["s"] - lse[..., None], 0.0)), 0.0)
    d = (512 + 4) * 2.0 ** -23 * ref["size"] + 2.0 ** -22 + 2.0 ** -23 * np.abs(lse)
    want = p.sum((0, 1))
    bound = (p * 2 * d[..., None]).sum((0, 1)) + (p.shape[0] * p.shape[1] + 4) * 2.0 ** -24 * want
    got, old = mass.double().cpu().numpy(), before.double().cpu().numpy()
    n = len(K)
    assert (np.abs(got[:n] - old[:n] - want) <= bound + 2.0 ** -24 * (np.abs(old[:n]) + want)).all()
    assert (got[n:] == old[n:]).all()


@pytest.mark.parametrize("H,lens,budget", [(16, [300, 170], 129), (64, [257, 90, 140], 130)])
def test_prompt_eviction_and_decode(csa2, H, lens, budget):  # noqa: F811
    B, page, pad, steps = len(lens), 128, 3, 4
    per = 3
    ids = np.random.default_rng(H).permutation(2 * B * per).astype(np.int32)
    table, dst = ids[:B * per].reshape(B, per).copy(), ids[B * per:].reshape(B, per).copy()
    cache = csa2.Cache(2 * B * per, page, table, lens)
    k4 = csa2.Ik4(cache)
    layer = Layer(csa2, H, seed=H)
    c = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()  # noqa: E731

    # ---- the prompts, with rows behind the last one ----
    n = sum(lens)
    start = np.concatenate([[0], np.cumsum(lens)])
    pos = np.concatenate([np.arange(x) for x in lens] + [np.zeros(pad)]).astype(np.int32)
    req = np.repeat(np.arange(B), lens).astype(np.int32)
    x = layer.draw(n + pad)
    q = torch.empty(n + pad, H, 512, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((n + pad, H), 7.0, device="cuda")
    mass = torch.zeros(B, cache.capacity, device="cuda")
    layer.seen_pos = c(pos)
    layer.run(cache, k4, x, c(pos), c(pos[:n]), c(req), q, out, lse, mass, c(start))
    st, word = csa2.get_error(cache)
    assert st == csa2.OK, word
    assert (out[n:] == 7).all() and (lse[n:] == 7).all()
    layer.check_queries(x, pos, q)
    want = layer.rows(x, pos[:n])
    at = table[req, pos[:n] // page].astype(np.int64) * page + pos[:n] % page
    for t, w in zip((cache.kv_codes, cache.kv_scales, cache.ik_codes, cache.ik_exp), want):
        np.testing.assert_array_equal(t.cpu().numpy()[at], w)
    K = F.dequantize_main_kv(want[0], want[1])
    K = [K[a:z] for a, z in zip(start[:-1], start[1:])]
    for b in range(B):
        a, z = start[b], start[b + 1]
        check_attention(q[a:z], K[b], pos[a:z] + 1, out[a:z], lse[a:z], mass[b], torch.zeros_like(mass[b]))

    # ---- the eviction; the caller takes the moved requests' pages and lengths ----
    m = mass.cpu().numpy()
    moved = torch.zeros(B, cache.capacity, device="cuda")
    kept, new_len = csa2.evict(cache, mass, budget, c(dst), sink=4, recent=20, mass_out=moved, ik4=k4)
    lens2 = []
    for b in range(B):
        keep = plain_kept(m[b], lens[b], budget, 4, 20)
        np.testing.assert_array_equal(kept[b].cpu().numpy()[:len(keep)], keep)
        lens2.append(len(keep))
        K[b] = K[b][keep]
        if lens[b] > budget:
            table[b] = dst[b]
            mass[b] = moved[b]
    np.testing.assert_array_equal(new_len.cpu().numpy(), lens2)
    cache.page_table.copy_(c(table))
    cache.ctx_len.copy_(new_len)

    # ---- single tokens: one captured step, replayed with new inputs ----
    x1, q1 = layer.draw(B), torch.empty(B, H, 512, dtype=torch.bfloat16, device="cuda")
    out1, lse1 = torch.empty_like(q1), torch.empty(B, H, device="cuda")
    token, slot = c(lens), cache.ctx_len.clone()        # position in the text, row of the cache
    layer.seen_pos = slot
    warm = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=warm):
        cache.ctx_len.copy_(slot + 1)
        layer.run(cache, k4, x1, token, slot, None, q1, out1, lse1, mass)
    for i in range(steps):
        x1.copy_(layer.draw(B))
        token.copy_(c([v + i for v in lens]))
        slot.copy_(c([v + i for v in lens2]))
        before = mass.clone()
        graph.replay()
        st, word = csa2.get_error(cache)
        assert st == csa2.OK, word
        tpos = token.cpu().numpy()
        layer.check_queries(x1, tpos, q1)
        codes, scales, _, _ = layer.rows(x1, tpos)
        new = F.dequantize_main_kv(codes, scales)
        for b in range(B):
            K[b] = np.concatenate([K[b], new[b:b + 1]])
            check_attention(q1[b:b + 1], K[b], [len(K[b])], out1[b:b + 1], lse1[b:b + 1], mass[b], before[b])
    np.testing.assert_array_equal(cache.ctx_len.cpu().numpy(), [v + steps for v in lens2])


def test_two_streams_and_a_shared_workspace_in_turn(csa2):  # noqa: F811
    """Calls of two streams in flight at once (a workspace each), and two
    graphs that use one workspace one after the other: the bits are those of
    single calls, whatever a workspace held before."""
    H, lens, new = 32, [1500, 700, 2600], [40, 1, 9]
    cache, _, _, _ = O.random_cache(csa2, lens, 128, seed=21)
    rng = np.random.default_rng(22)
    c = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()  # noqa: E731
    start = np.concatenate([[0], np.cumsum(new)])
    cases = []
    for k in range(2):
        pos = c(np.concatenate([rng.integers(0, n, x) for n, x in zip(lens, new)]))
        q = torch.from_numpy(rng.standard_normal((sum(new), H, 512)).astype(np.float32)).bfloat16().cuda() * 0.2
        cases.append((pos, q, torch.empty_like(q), torch.empty(q.shape[:2], device="cuda"),
                      torch.empty(3, cache.capacity, device="cuda"),
                      torch.empty(max(csa2.chunk_attn_workspace_bytes(cache, sum(new), H),
                                      csa2.attn_mass_workspace_bytes(cache, sum(new), H)), dtype=torch.uint8,
                                  device="cuda")))
    st = c(start)

    def run(k, ws):
        pos, q, out, lse, mass, _ = cases[k]
        csa2.chunk_attn(cache, q, pos, st, out=out, lse=lse, workspace=ws)
        mass.zero_()
        csa2.attn_mass(cache, q, pos, lse, mass, st, workspace=ws)

    def results(k):
        return [t.clone() for t in cases[k][2:5]]

    want = []
    for k in range(2):
        run(k, cases[k][5])
        want.append(results(k))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for k in range(2):
            cases[k][2].zero_(), cases[k][3].zero_()
        torch.cuda.synchronize()
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                run(k, cases[k][5])
        torch.cuda.synchronize()
        for k in range(2):
            assert all(torch.equal(a, b) for a, b in zip(want[k], results(k)))
    shared = cases[0][5]
    graphs = []
    for k in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[k]):
            run(k, shared)
    for order in ((0, 1), (1, 0), (1, 1, 0)):
        shared.fill_(0xFF)
        for k in order:
            graphs[k].replay()
        torch.cuda.synchronize()
        for k in range(2):
            assert all(torch.equal(a, b) for a, b in zip(want[k], results(k)))
    status, word = csa2.get_error(cache)
    assert status == csa2.OK, word


def test_rows_behind_32_bit_offsets(csa2):  # noqa: F811
    """A cache of 17.2 million rows (codes behind 2^32 bytes): the bits are
    those of a small cache with the same rows."""
    page, H, lens = 4096, 16, [5000, 130]
    small = csa2.Cache(5, page, [[0, 1], [2, -1]], lens)
    P = 4200
    assert (P - 5) * page * 256 > 2 ** 32
    big = csa2.Cache(P, page, [[P - 1, P - 4], [P - 2, -1]], lens)
    g = torch.Generator(device="cuda").manual_seed(3)
    n = sum(lens)
    x = torch.randn(n, 640, generator=g, device="cuda")
    pos = torch.cat([torch.arange(v) for v in lens]).int().cuda()
    req = torch.repeat_interleave(torch.arange(2), torch.tensor(lens)).int().cuda()
    q = torch.randn(2, H, 512, generator=g, device="cuda").bfloat16()
    qp = torch.tensor(lens).int().cuda() - 1
    rope = csa2.Rope(torch.from_numpy(O.freqs(ROT)).cuda())
    results = []
    for cache, dst in ((small, [[3], [-1]]), (big, [[P - 3], [-1]])):
        k4 = csa2.Ik4(cache)
        csa2.norm_rope_append(cache, x[:, :512], x[:, 512:], pos, rope, rope, req=req, ik4=k4)
        lse = torch.empty(2, H, device="cuda")
        out = csa2.chunk_attn(cache, q, qp, lse=lse)
        mass = csa2.attn_mass(cache, q, qp, lse, torch.zeros(2, cache.capacity, device="cuda"))
        dst = torch.tensor(dst).int().cuda()
        kept, new_len = csa2.evict(cache, mass, 1000, dst, sink=4, recent=16, ik4=k4)
        st, word = csa2.get_error(cache)
        assert st == csa2.OK, word
        row = int(dst[0, 0]) * page
        results.append([out, lse, mass, kept, new_len, cache.kv_codes[row:row + 1000], cache.kv_scales[row:row + 1000],
                        cache.ik_codes[row:row + 1000], cache.ik_exp[row:row + 1000], k4.codes[row:row + 1000],
                        k4.scales[row // 128:row // 128 + 7]])
    assert int(results[0][5].sum()) > 0
    for a, b in zip(*results):
        assert torch.equal(a, b)
