"""Attention weight received by the cached entries (csa2_attn_mass) against its
formula in float64.  Needs a B200 and libcsa2.so."""
import math

import numpy as np
import pytest
import torch

from tests import ops_util as O
from tests.test_gpu_chunk_attn import CASES, _case, csa2  # noqa: F401

pytestmark = pytest.mark.gpu


def _reference(case, lens, ratio, scale):
    """(lse float32 [n, H], weights [batch] of [n_ctx], bounds): a weight's
    terms are each off by e^d - 1 <= 2 d with the scores' d (512 products
    summed in fp32, as in attention_bounds), 2^-21 for exp2 and the product
    with log2 e, and 2^-23 |lse| for the fp32 lse scaled to log2; summing n
    rows adds n 2^-24 of the sum."""
    cache, table, codes, scales, start, pos, q = case
    q64 = q.double().cpu().numpy()
    lse = np.zeros(q.shape[:2], np.float32)
    mass, tol = [], []
    for b, n_ctx in enumerate(lens):
        a, z = int(start[b]), int(start[b + 1])
        seen = np.clip((pos[a:z].astype(np.int64) + 1) // ratio, 0, n_ctx)
        ref = O.attention(q64[a:z], O.keys(table, cache.page_size, codes, scales, b, n_ctx), seen, scale)
        lse[a:z] = ref["lse"]
        l32 = lse[a:z].astype(np.float64)
        fine = np.isfinite(ref["s"])
        with np.errstate(invalid="ignore"):
            p = np.where(fine, np.exp(np.where(fine, ref["s"] - l32[..., None], 0.0)), 0.0)
        d = (512 + 4) * 2.0 ** -23 * ref["size"] + 2.0 ** -22 + 2.0 ** -23 * np.abs(np.where(np.isfinite(l32), l32, 0.0))
        mass.append(p.sum((0, 1)))
        tol.append((p * 2 * d[..., None]).sum((0, 1)) + (p.shape[0] * p.shape[1] + 4) * 2.0 ** -24 * mass[-1])
    return torch.from_numpy(lse).cuda(), mass, tol


def _check(mass, before, want, tol, lens, what=""):
    got, old = mass.double().cpu().numpy(), before.double().cpu().numpy()
    for b, n in enumerate(lens):
        bound = tol[b] + 2.0 ** -24 * (np.abs(old[b, :n]) + want[b])
        err = np.abs(got[b, :n] - old[b, :n] - want[b])
        assert (err <= bound).all(), f"{what} request {b}: off by {err.max():.3e}, {(err / bound).max():.2f} of its bound"
        assert (got[b, n:] == old[b, n:]).all()


@pytest.mark.parametrize("H", [16, 32, 64])
@pytest.mark.parametrize("lens,new,page,ratio", CASES)
def test_attn_mass(csa2, lens, new, page, ratio, H):  # noqa: F811
    case = _case(csa2, lens, new, H, page, ratio, seed=sum(lens) + H, pad=2)
    cache, _, _, _, start, pos, q = case
    lse, want, tol = _reference(case, lens, ratio, 1 / math.sqrt(512))
    lse[-2:] = float("nan")                       # rows behind the last request are not read into anything
    q[-2:] = float("nan")
    before = torch.rand(cache.batch, cache.capacity, generator=torch.Generator().manual_seed(1)).cuda()
    mass = before.clone()
    csa2.attn_mass(cache, q, torch.from_numpy(pos).cuda(), lse, mass, torch.from_numpy(start).cuda(), ratio=ratio)
    st, word = csa2.get_error(cache)
    assert st == csa2.OK, word
    _check(mass, before, want, tol, lens)


@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("lens", [[5000], [1] * 5 + [900] * 8, [30000, 20000]])
def test_attn_mass_single_tokens(csa2, lens, H):  # noqa: F811
    case = _case(csa2, lens, [1] * len(lens), H, 128, seed=len(lens))
    cache, _, _, _, start, pos, q = case
    lse, want, tol = _reference(case, lens, 1, 1 / math.sqrt(512))
    mass = torch.zeros(cache.batch, cache.capacity, device="cuda")
    p = torch.from_numpy(pos).cuda()
    csa2.attn_mass(cache, q, p, lse, mass)
    _check(mass, torch.zeros_like(mass), want, tol, lens)
    again = csa2.attn_mass(cache, q, p, lse, torch.zeros_like(mass))
    assert torch.equal(mass, again)


@pytest.mark.parametrize("H,new", [(16, 300), (32, 129), (64, 700)])
def test_attn_mass_positions_in_any_order(csa2, H, new):  # noqa: F811
    """Shuffled positions (whole items that see nothing of a unit among them),
    units cut over pairs and joined, a negative scale."""
    lens = [777]
    pos = np.random.default_rng(4).integers(-3, 900, new)
    pos[: new // 2] %= 200
    case = _case(csa2, lens, [new], H, 128, seed=9, pos=pos)
    cache, _, _, _, start, p, q = case
    lse, want, tol = _reference(case, lens, 1, -0.03)
    mass = torch.zeros(1, cache.capacity, device="cuda")
    csa2.attn_mass(cache, q, torch.from_numpy(p).cuda(), lse, mass, torch.from_numpy(start).cuda(), scale=-0.03)
    _check(mass, torch.zeros_like(mass), want, tol, lens)


def test_attn_mass_sums_to_the_queries(csa2):  # noqa: F811
    """With chunk_attn's own lse the weights of a request sum to (queries that
    see something) x H."""
    lens, new, H = [2000, 333], [64, 333], 32
    case = _case(csa2, lens, new, H, 128, seed=3)
    cache, _, _, _, start, pos, q = case
    p, s = torch.from_numpy(pos).cuda(), torch.from_numpy(start).cuda()
    lse = torch.empty(q.shape[:2], device="cuda")
    csa2.chunk_attn(cache, q, p, s, lse=lse)
    mass = csa2.attn_mass(cache, q, p, lse, torch.zeros(2, cache.capacity, device="cuda"), s)
    total = mass.double().sum(1).cpu()
    # both sides' scores are off by at most d each (see _reference): 1e-3 here
    assert abs(float(total[0]) - 64 * H) < 2e-3 * 64 * H and abs(float(total[1]) - 333 * H) < 2e-3 * 333 * H


def test_attn_mass_recorded_violations(csa2):  # noqa: F811
    for what in ("page", "ctx", "start"):
        lens, new, H = [300, 200], [70, 3], 32
        case = _case(csa2, lens, new, H, 128, seed=5)
        cache, _, _, _, start, pos, q = case
        lse, want, tol = _reference(case, lens, 1, 1 / math.sqrt(512))
        s = start.copy()
        if what == "page":
            cache.page_table[0, 1] = cache.num_pages
        elif what == "ctx":
            cache.ctx_len[0] = -7
        else:
            s[0] = -4
        mass = torch.zeros(2, cache.capacity, device="cuda")
        csa2.attn_mass(cache, q, torch.from_numpy(pos).cuda(), lse, mass, torch.from_numpy(s).cuda())
        st, word = csa2.get_error(cache)
        assert st == csa2.ERR_DEVICE_BOUNDS and word[2] == 0, (what, word)
        if what == "page":
            assert (mass[0, 128:256] == 0).all() and (mass[0, :128] > 0).all()
        else:
            assert (mass[0] == 0).all()
        _check(mass[1:], torch.zeros_like(mass[1:]), want[1:], tol[1:], lens[1:])


@pytest.mark.parametrize("what", ["large", "tiny", "lse", "scale"])
def test_attn_mass_wide_rows(csa2, what):  # noqa: F811
    """Row tiles that leave the common scale: very large or very small queries,
    log-sum-exps far from the scores, a small scale; an ordinary tile and
    request next to them."""
    lens, new, H = [300, 200], [40, 7], 16
    case = _case(csa2, lens, new, H, 128, seed=8)
    cache, table, codes, scales, start, pos, q = case
    scale = 1 / math.sqrt(512)
    if what == "large":
        q[5, 3] *= 2.0 ** 13                      # scores of thousands: one entry takes all
        q[38] *= 2.0 ** 30
    elif what == "tiny":
        q[5] *= 2.0 ** -40
        q[30] = 0
    elif what == "scale":
        scale = 1e-4
    if what == "large":
        # Rows (5, 3) and 38 have scores up to 10^4 and 10^10.  fp32 holds such an
        # lse to 2^-8 and to 2^9 only, so exp(score - lse) of their largest
        # entries may be off by any factor up to e^(2^9): nothing is asked of the
        # entries whose score lies within the scores' own error d, that spacing
        # and 110 (e^-110 is below fp32) of the largest.  Every other entry gets
        # nothing of these rows, and what the other rows give it.
        lse = torch.empty(q.shape[:2], device="cuda")
        csa2.chunk_attn(cache, q, torch.from_numpy(pos).cuda(), torch.from_numpy(start).cuda(), lse=lse, scale=scale)
        mass = csa2.attn_mass(cache, q, torch.from_numpy(pos).cuda(), lse, torch.zeros(2, cache.capacity, device="cuda"),
                              torch.from_numpy(start).cuda(), scale=scale)
        got = mass.double().cpu().numpy()
        for b, (a, z) in enumerate(((0, 40), (40, 47))):
            K = O.keys(table, 128, codes, scales, b, lens[b])
            seen = pos[a:z] + 1
            q64 = q[a:z].double().cpu().numpy()
            s = np.where(np.arange(lens[b])[None, None] < seen[:, None, None], np.einsum("ihc,ec->ihe", q64, K) * scale, -np.inf)
            size = scale * np.einsum("ihc,ec->ihe", np.abs(q64), np.abs(K)).max(-1)
            l = lse[a:z].double().cpu().numpy()
            d = (512 + 4) * 2.0 ** -23 * size + 2.0 ** -22 + 2.0 ** -23 * np.abs(l)
            d = 2 * d                               # the scores here, and those that the lse was made of
            far = d >= 1.0
            assert far.sum() == (17 if b == 0 else 0)
            near = (far[..., None] & (s >= s.max(-1, keepdims=True) - (110 + 2 * d + 2.0 ** 10)[..., None])).any((0, 1))
            p = np.where(np.isfinite(s) & ~far[..., None], np.exp(np.where(np.isfinite(s), s - l[..., None], 0.0) * ~far[..., None]), 0.0)
            want, tol = p.sum((0, 1)), (p * 2 * np.minimum(d, 1.0)[..., None]).sum((0, 1)) + 700 * 2.0 ** -24 * p.sum((0, 1))
            err = np.abs(got[b, :lens[b]] - want)[~near]
            assert (~near).any() and (err <= tol[~near]).all(), (b, err.max())
        return
    lse, want, tol = _reference(case, lens, 1, scale)
    if what == "lse":                             # as if most of the weight lay elsewhere
        lse[4] += 3.0e4
        lse[20] += 5.0
    mass = torch.zeros(2, cache.capacity, device="cuda")
    csa2.attn_mass(cache, q, torch.from_numpy(pos).cuda(), lse, mass, torch.from_numpy(start).cuda(), scale=scale)
    if what == "lse":
        K = O.keys(table, 128, codes, scales, 0, 300)
        ref = O.attention(q[:40].double().cpu().numpy(), K, pos[:40] + 1, scale)
        l = lse[:40].double().cpu().numpy()
        p = np.where(np.isfinite(ref["s"]), np.exp(np.where(np.isfinite(ref["s"]), ref["s"] - l[..., None], 0.0)), 0.0)
        d = (512 + 4) * 2.0 ** -23 * ref["size"] + 2.0 ** -22 + 2.0 ** -23 * np.abs(l)
        want[0], tol[0] = p.sum((0, 1)), (p * 2 * d[..., None]).sum((0, 1)) + (40 * H + 4) * 2.0 ** -24 * p.sum((0, 1))
    _check(mass, torch.zeros_like(mass), want, tol, lens)


def test_attn_mass_graph(csa2):  # noqa: F811
    lens, new, H = [700, 90], [33, 20], 32
    case = _case(csa2, lens, new, H, 128, seed=15)
    cache, _, _, _, start, pos, q = case
    lse, want, tol = _reference(case, lens, 1, 1 / math.sqrt(512))
    p, s = torch.from_numpy(pos).cuda(), torch.from_numpy(start).cuda()
    ws = torch.empty(csa2.attn_mass_workspace_bytes(cache, q.shape[0], H), dtype=torch.uint8, device="cuda")
    mass = torch.zeros(2, cache.capacity, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        csa2.attn_mass(cache, q, p, lse, mass, s, workspace=ws)
    mass.zero_()
    ws.fill_(0xFF)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    _check(mass, torch.zeros_like(mass), [2 * w for w in want], [2 * t for t in tol], lens)


def test_attn_mass_wait_limit(csa2):  # noqa: F811
    """A wait that runs out is recorded and the launch ends; the next one is
    unharmed."""
    lens, new, H = [700], [300], 64
    case = _case(csa2, lens, new, H, 128, seed=15)
    cache, _, _, _, start, pos, q = case
    lse, want, tol = _reference(case, lens, 1, 1 / math.sqrt(512))
    p, s = torch.from_numpy(pos).cuda(), torch.from_numpy(start).cuda()
    mass = torch.zeros(1, cache.capacity, device="cuda")
    csa2.set_wait_limit_ns(0)
    try:
        csa2.attn_mass(cache, q, p, lse, mass, s)
        st, _ = csa2.get_error(cache)
    finally:
        csa2.set_wait_limit_ns(2_000_000_000)
    assert st == csa2.ERR_TIMEOUT
    cache.err_word.zero_()
    mass.zero_()
    csa2.attn_mass(cache, q, p, lse, mass, s)
    st, word = csa2.get_error(cache)
    assert st == csa2.OK, word
    _check(mass, torch.zeros_like(mass), want, tol, lens)


@pytest.mark.parametrize("H,new", [(16, [0, 12, 1, 0, 0, 3]), (64, [0, 0, 4, 0, 1, 0]), (32, [11, 0, 0, 0, 0, 0])])
def test_attn_mass_few_rows_unevenly(csa2, H, new):  # noqa: F811
    """Few query rows per request on average, most of them one request's."""
    lens = [100, 9000, 2600, 5, 700, 33]
    lens[0] = 8300 if new[0] else 100
    case = _case(csa2, lens, new, H, 128, seed=H, pad=1)
    cache, _, _, _, start, pos, q = case
    assert q.shape[0] * H <= 64 * len(lens)
    lse, want, tol = _reference(case, lens, 1, 1 / math.sqrt(512))
    mass = torch.zeros(cache.batch, cache.capacity, device="cuda")
    csa2.attn_mass(cache, q, torch.from_numpy(pos).cuda(), lse, mass, torch.from_numpy(start).cuda())
    st, word = csa2.get_error(cache)
    assert st == csa2.OK, word
    _check(mass, torch.zeros_like(mass), want, tol, lens)


def test_attn_mass_wait_limit_single_tokens(csa2):  # noqa: F811
    lens = [3000, 200]
    case = _case(csa2, lens, [1, 1], 32, 128, seed=3)
    cache, _, _, _, _, pos, q = case
    lse, want, tol = _reference(case, lens, 1, 1 / math.sqrt(512))
    p = torch.from_numpy(pos).cuda()
    csa2.set_wait_limit_ns(0)
    try:
        csa2.attn_mass(cache, q, p, lse, torch.zeros(2, cache.capacity, device="cuda"))
        st, _ = csa2.get_error(cache)
    finally:
        csa2.set_wait_limit_ns(2_000_000_000)
    assert st == csa2.ERR_TIMEOUT
    cache.err_word.zero_()
    mass = csa2.attn_mass(cache, q, p, lse, torch.zeros(2, cache.capacity, device="cuda"))
    st, word = csa2.get_error(cache)
    assert st == csa2.OK, word
    _check(mass, torch.zeros_like(mass), want, tol, lens)


def test_attn_mass_small_queries_large_scale(csa2):  # noqa: F811
    """Queries times 2^-30 with a scale times 2^30: the weights are those of the
    queries and the scale as they were."""
    lens, new, H = [300, 200], [40, 7], 16
    case = _case(csa2, lens, new, H, 128, seed=8)
    cache, _, _, _, start, pos, q = case
    q.mul_(2.0 ** -30)
    scale = 2.0 ** 30 / math.sqrt(512)
    lse, want, tol = _reference(case, lens, 1, scale)
    mass = torch.zeros(2, cache.capacity, device="cuda")
    csa2.attn_mass(cache, q, torch.from_numpy(pos).cuda(), lse, mass, torch.from_numpy(start).cuda(), scale=scale)
    assert csa2.get_error(cache)[0] == csa2.OK
    _check(mass, torch.zeros_like(mass), want, tol, lens)


@pytest.mark.parametrize("factor", [2.0 ** 4, 2.0 ** 5, 2.0 ** 8, 2.0 ** 20])
def test_attn_mass_scales_on_both_sides_of_the_forms(csa2, factor):  # noqa: F811
    """The same product of queries and scale, split differently."""
    lens, new, H = [300, 200], [40, 7], 16
    case = _case(csa2, lens, new, H, 128, seed=8)
    cache, _, _, _, start, pos, q = case
    q.div_(factor)
    scale = factor / math.sqrt(512)
    lse, want, tol = _reference(case, lens, 1, scale)
    mass = torch.zeros(2, cache.capacity, device="cuda")
    csa2.attn_mass(cache, q, torch.from_numpy(pos).cuda(), lse, mass, torch.from_numpy(start).cuda(), scale=scale)
    _check(mass, torch.zeros_like(mass), want, tol, lens)


def test_attn_mass_many_wide_tiles(csa2):  # noqa: F811
    """Row tiles that all take the wide form, whose CTAs tell each other twice a
    tile, in many launches: no wait runs out, and the bits are the same."""
    lens, new, H = [260, 130], [200, 120], 16
    case = _case(csa2, lens, new, H, 128, seed=11)
    cache, _, _, _, start, pos, q = case
    scale = 1e-4                                  # below the common scale's range
    lse, want, tol = _reference(case, lens, 1, scale)
    p, s = torch.from_numpy(pos).cuda(), torch.from_numpy(start).cuda()
    first = csa2.attn_mass(cache, q, p, lse, torch.zeros(2, cache.capacity, device="cuda"), s, scale=scale)
    _check(first, torch.zeros_like(first), want, tol, lens)
    for _ in range(200):
        again = csa2.attn_mass(cache, q, p, lse, torch.zeros_like(first), s, scale=scale)
        assert torch.equal(first, again)
    assert csa2.get_error(cache)[0] == csa2.OK
