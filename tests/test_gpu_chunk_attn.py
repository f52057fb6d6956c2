"""Dense attention of new tokens over the paged cache (csa2_chunk_attn)
against its formula in float64.  Needs a B200 and libcsa2.so."""
import math

import numpy as np
import pytest
import torch

from tests import ops_util as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def csa2():
    from kv_cache_decode_index_b200 import csa2 as lib
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return lib


def _case(csa2, lens, new, H, page, ratio=1, seed=0, pad=0, q_scale=1.0, pos=None):
    cache, table, codes, scales = O.random_cache(csa2, lens, page, seed)
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    n = int(start[-1]) + pad
    rng = np.random.default_rng(seed + 1)
    if pos is None:
        pos = np.concatenate([np.arange(c * ratio - x, c * ratio) for c, x in zip(lens, new)] + [np.zeros(pad)])
    pos = np.asarray(pos, np.int64).clip(-1).astype(np.int32)
    # E4M3 codes 40 .. 71 are scales of 2^-2 .. 3.75: rows of norm about 100
    q = torch.from_numpy((rng.standard_normal((n, H, 512)) * q_scale * 0.2).astype(np.float32)).bfloat16().cuda()
    return cache, table, codes, scales, start, pos, q


def _check(cache, table, codes, scales, start, pos, q, out, lse, lens, ratio, scale):
    q64 = q.double().cpu().numpy()
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, n_ctx in enumerate(lens):
        a, z = int(start[b]), int(start[b + 1])
        if a == z:
            continue
        seen = np.clip((pos[a:z].astype(np.int64) + 1) // ratio, 0, n_ctx)
        K = O.keys(table, cache.page_size, codes, scales, b, n_ctx)
        ref = O.attention(q64[a:z], K, seen, scale)
        tol, tol_lse = O.attention_bounds(ref, max(n_ctx, 1))
        tol = tol + torch.finfo(torch.bfloat16).eps / 2 * (np.abs(ref["out"]) + tol)
        err = np.abs(got[a:z] - ref["out"])
        assert (err <= tol).all(), f"request {b}: out off by {err.max():.3e}, {(err / np.maximum(tol, 1e-30)).max():.2f} of its bound"
        none = ~np.isfinite(ref["lse"])
        assert (got_lse[a:z][none] == -np.inf).all()
        err = np.abs(got_lse[a:z][~none] - ref["lse"][~none])
        assert (err <= tol_lse[~none]).all(), f"request {b}: lse off by {err.max():.3e}"


CASES = [
    # lens, new, page, ratio
    ([1], [1], 128, 1),
    ([64], [64], 128, 1),
    ([65, 63], [65, 2], 128, 1),
    ([129, 1, 500], [3, 1, 130], 128, 1),
    ([300, 7, 257, 128], [5, 0, 1, 128], 256, 1),
    ([40, 333], [80, 9], 128, 2),          # the first tokens of request 0 see no entry
    ([200], [0], 128, 1),
    ([1, 700], [1, 1], 384, 3),
    ([1000, 33, 2, 515], [70, 33, 2, 1], 128, 1),
]


@pytest.mark.parametrize("H", [16, 32, 64])
@pytest.mark.parametrize("lens,new,page,ratio", CASES)
def test_chunk_attn(csa2, lens, new, page, ratio, H):
    args = _case(csa2, lens, new, H, page, ratio, seed=sum(lens) + H, pad=2)
    cache, _, _, _, start, pos, q = args
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    scale = 1 / math.sqrt(512)
    csa2.chunk_attn(cache, q, torch.from_numpy(pos).cuda(), torch.from_numpy(start).cuda(), ratio=ratio, out=out, lse=lse)
    st, word = csa2.get_error(cache)
    assert st == csa2.OK, word
    assert (out[-2:] == 7.0).all() and (lse[-2:] == 7.0).all()      # rows behind the last request
    _check(*args, out, lse, lens, ratio, scale)


@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("lens", [[5000], [4097, 129, 2000], [1] * 5 + [900] * 8])
def test_chunk_attn_single_tokens(csa2, lens, H):
    """q_start None: one new token per request; long keys are cut and joined.
    Twice the same bits."""
    args = _case(csa2, lens, [1] * len(lens), H, 128, seed=len(lens))
    cache, _, _, _, start, pos, q = args
    lse = torch.empty(q.shape[:2], device="cuda")
    p = torch.from_numpy(pos).cuda()
    out = csa2.chunk_attn(cache, q, p, lse=lse)
    _check(*args, out, lse, lens, 1, 1 / math.sqrt(512))
    assert torch.equal(out, csa2.chunk_attn(cache, q, p))


@pytest.mark.parametrize("H,new", [(16, 300), (32, 129), (64, 70)])
def test_chunk_attn_positions_in_any_order(csa2, H, new):
    """Shuffled positions, some of which see nothing, and a negative scale."""
    rng = np.random.default_rng(4)
    lens = [777]
    pos = rng.integers(-3, 900, new)
    args = _case(csa2, lens, [new], H, 128, seed=9, pos=pos)
    cache, _, _, _, start, p, q = args
    lse = torch.empty(q.shape[:2], device="cuda")
    out = csa2.chunk_attn(cache, q, torch.from_numpy(p).cuda(), torch.from_numpy(start).cuda(), scale=-0.03, lse=lse)
    _check(*args, out, lse, lens, 1, -0.03)


@pytest.mark.parametrize("H", [16, 64])
def test_chunk_attn_peaked(csa2, H):
    """Scores far apart: one key takes nearly all the weight, and the running
    maximum rises by much from step to step."""
    lens, new = [640], [40]
    args = _case(csa2, lens, new, H, 128, seed=21, q_scale=6.0)
    cache, _, _, _, start, pos, q = args
    lse = torch.empty(q.shape[:2], device="cuda")
    out = csa2.chunk_attn(cache, q, torch.from_numpy(pos).cuda(), torch.from_numpy(start).cuda(), lse=lse)
    _check(*args, out, lse, lens, 1, 1 / math.sqrt(512))


def test_chunk_attn_query_sizes(csa2):
    """Rows of very large and very small queries, zeros, and one with a NaN
    and one with an infinity: those rows are NaN, the others are not touched
    by them."""
    lens, new, H = [200], [6], 16
    args = _case(csa2, lens, new, H, 128, seed=2)
    cache, table, codes, scales, start, pos, q = args
    q[0] *= 2.0 ** -90
    q[1] = 0
    q[2, 3, 5] = float("nan")
    q[3, 1, 9] = float("inf")
    lse = torch.empty(q.shape[:2], device="cuda")
    out = csa2.chunk_attn(cache, q, torch.from_numpy(pos).cuda(), torch.from_numpy(start).cuda(), lse=lse)
    assert torch.isnan(out[2, 3]).all() and torch.isnan(out[3, 1]).all()
    bad = torch.zeros(6, H, dtype=torch.bool, device="cuda")
    bad[2, 3] = bad[3, 1] = True
    assert not torch.isnan(out[~bad]).any()
    q[2, 3], q[3, 1] = 0, 0
    again = csa2.chunk_attn(cache, q, torch.from_numpy(pos).cuda(), torch.from_numpy(start).cuda())
    assert torch.equal(out[~bad], again[~bad])
    lse[2, 3], lse[3, 1] = 0, 0
    lse2 = torch.empty_like(lse)
    csa2.chunk_attn(cache, q, torch.from_numpy(pos).cuda(), torch.from_numpy(start).cuda(), lse=lse2)
    _check(*args, again, lse2, lens, 1, 1 / math.sqrt(512))
    big = q.clone()
    big[4] *= 2.0 ** 100
    out = csa2.chunk_attn(cache, big, torch.from_numpy(pos).cuda(), torch.from_numpy(start).cuda())
    assert torch.equal(out[5], again[5]) and torch.isfinite(out[4].float()).all()


def test_chunk_attn_recorded_violations(csa2):
    """Bad pages, lengths and query ranges are recorded; the other requests'
    rows are right and nothing outside is written."""
    lens, new, H = [300, 200], [70, 3], 32
    for what in ("page", "ctx", "start"):
        args = _case(csa2, lens, new, H, 128, seed=5)
        cache, table, codes, scales, start, pos, q = args
        s = start.copy()
        if what == "page":
            cache.page_table[0, 1] = cache.num_pages
        elif what == "ctx":
            cache.ctx_len[0] = 10 ** 6
        else:
            s[0] = -4
        out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
        csa2.chunk_attn(cache, q, torch.from_numpy(pos).cuda(), torch.from_numpy(s).cuda(), out=out, lse=lse)
        st, word = csa2.get_error(cache)
        assert st == csa2.ERR_DEVICE_BOUNDS and word[2] == 0, (what, word)
        if what == "ctx":
            assert (out[:70] == 0).all() and (lse[:70] == -np.inf).all()
        if what == "start":
            assert (out[:70] == 7.0).all()
        _check(cache, table, codes, scales, [70, 70, 73], pos, q, out, lse, lens, 1,
               1 / math.sqrt(512))


def test_chunk_attn_graph_and_stream(csa2):
    """Captured once and replayed on changed inputs; on a side stream."""
    lens, new, H = [700, 90], [33, 20], 32
    args = _case(csa2, lens, new, H, 128, seed=15)
    cache, table, codes, scales, start, pos, q = args
    p, s = torch.from_numpy(pos).cuda(), torch.from_numpy(start).cuda()
    ws = torch.empty(csa2.chunk_attn_workspace_bytes(cache, q.shape[0], H), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        csa2.chunk_attn(cache, q, p, s, out=out, lse=lse, workspace=ws)
    ws.fill_(0xFF)
    q.copy_(q.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    _check(*args, out, lse, lens, 1, 1 / math.sqrt(512))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = csa2.chunk_attn(cache, q, p, s)
    side.synchronize()
    assert torch.equal(other, out)


def test_chunk_attn_offsets_past_32_bits(csa2):
    """Pages whose code bytes lie past 2^31 and 2^32."""
    page, H = 4096, 16
    num = (2 ** 32 // 256) // page + 8
    cache = csa2.Cache(num, page, [[num - 1, num // 2 + 3]], [5000])
    rows = O.rows_of(np.array([[num - 1, num // 2 + 3]]), page, 0, 5000)
    rng = np.random.default_rng(0)
    codes = rng.integers(0, 256, (5000, 256), dtype=np.uint8)
    scales = rng.integers(40, 72, (5000, 32), dtype=np.uint8)
    r = torch.from_numpy(rows).cuda()
    cache.kv_codes[r] = torch.from_numpy(codes).cuda()
    cache.kv_scales[r] = torch.from_numpy(scales).cuda()
    q = (torch.from_numpy(rng.standard_normal((1, H, 512)).astype(np.float32)) * 0.2).bfloat16().cuda()
    pos = np.array([4999], np.int32)
    lse = torch.empty(1, H, device="cuda")
    out = csa2.chunk_attn(cache, q, torch.from_numpy(pos).cuda(), lse=lse)
    small = np.array([[0, 1]], np.int32)      # the same rows in a small table for the reference
    c2, s2 = np.zeros((2 * page, 256), np.uint8), np.zeros((2 * page, 32), np.uint8)
    c2[:5000], s2[:5000] = codes, scales
    _check(cache, small, c2, s2, [0, 1], pos, q, out, lse, [5000], 1, 1 / math.sqrt(512))


def test_chunk_attn_wait_limit(csa2):  # noqa: F811
    """A wait that runs out is recorded and the launch ends; the next one is
    unharmed."""
    args = _case(csa2, [2000, 300], [70, 3], 32, 128, seed=9)
    cache, start, pos, q = args[0], args[4], args[5], args[6]
    p, s = torch.from_numpy(pos).cuda(), torch.from_numpy(start).cuda()
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    csa2.set_wait_limit_ns(0)
    try:
        csa2.chunk_attn(cache, q, p, s, out=out, lse=lse)
        st, _ = csa2.get_error(cache)
    finally:
        csa2.set_wait_limit_ns(2_000_000_000)
    assert st == csa2.ERR_TIMEOUT
    cache.err_word.zero_()
    csa2.chunk_attn(cache, q, p, s, out=out, lse=lse)
    st, word = csa2.get_error(cache)
    assert st == csa2.OK, word
    _check(*args, out, lse, [2000, 300], 1, 1 / math.sqrt(512))


def _without(table, page, n_ctx, bad):
    """Entries of a request that do not lie under the bad page slots."""
    return np.nonzero(~np.isin(np.arange(n_ctx) // page, bad))[0]


@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("q_scale", [1.0, 4.0])
@pytest.mark.parametrize("lens,new,page,bad", [
    ([300, 200], [70, 3], 128, [[1], []]),              # the second half of the first tile
    ([1000, 700], [40, 300], 256, [[0], [2]]),          # a whole tile, the first one; the last entries
    ([900, 130], [1, 130], 384, [[1], [0]]),            # pages that end inside a tile; nothing is left
    ([6000, 200], [1, 1], 128, [list(range(4, 30)), []]),   # ranges of a cut request in which nothing is left
])
def test_chunk_attn_leaves_bad_pages_out(csa2, lens, new, page, bad, q_scale, H):
    """Entries under a page id out of range take no part in the softmax, as if
    they were not there; the weights (attn_mass) of the others sum to the
    queries that see something."""
    args = _case(csa2, lens, new, H, page, seed=7, q_scale=q_scale)
    cache, table, codes, scales, start, pos, q = args
    for b, slots in enumerate(bad):
        for i, s in enumerate(slots):
            cache.page_table[b, s] = (-1, cache.num_pages, -2 ** 31, 2 ** 31 - 1)[i % 4]
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    p, s = torch.from_numpy(pos).cuda(), torch.from_numpy(start).cuda()
    csa2.chunk_attn(cache, q, p, s, out=out, lse=lse)
    st, word = csa2.get_error(cache)
    assert st == csa2.ERR_DEVICE_BOUNDS, word
    mass = csa2.attn_mass(cache, q, p, lse, torch.zeros(2, cache.capacity, device="cuda"), s).double().cpu().numpy()
    scale = 1 / math.sqrt(512)
    for b, n_ctx in enumerate(lens):
        a, z = int(start[b]), int(start[b + 1])
        good = _without(table, page, n_ctx, bad[b])
        seen = np.searchsorted(good, np.clip(pos[a:z].astype(np.int64) + 1, 0, n_ctx))
        K = O.keys(table, page, codes, scales, b, n_ctx)[good]
        ref = O.attention(q[a:z].double().cpu().numpy(), K, seen, scale)
        tol, tol_lse = O.attention_bounds(ref, n_ctx)
        tol = tol + torch.finfo(torch.bfloat16).eps / 2 * (np.abs(ref["out"]) + tol)
        err = np.abs(out[a:z].double().cpu().numpy() - ref["out"])
        assert (err <= tol).all(), f"request {b}: out off by {err.max():.3e}, {(err / np.maximum(tol, 1e-30)).max():.2f} of its bound"
        got, none = lse[a:z].double().cpu().numpy(), ~np.isfinite(ref["lse"])
        assert (got[none] == -np.inf).all()
        err = np.abs(got[~none] - ref["lse"][~none])
        assert (err <= tol_lse[~none]).all(), f"request {b}: lse off by {err.max():.3e}"
        # a row's weights: each off by twice the scores' error and the lse's own; their sum by n 2^-24 more
        d = 2 * ((512 + 4) * 2.0 ** -23 * ref["size"][~none] + 2.0 ** -21 + tol_lse[~none]).sum()
        d += got[~none].size ** 2 * 2.0 ** -24 + n_ctx * 2.0 ** -24 * got[~none].size
        assert abs(mass[b].sum() - got[~none].size) <= d
        assert (mass[b][np.setdiff1d(np.arange(n_ctx), good)] == 0).all()


def test_chunk_attn_maximum_rises_by_one_spacing(csa2):
    """Scores of 2^27 to 2^28 (log2 units), where fp32 values are 16 apart, and a
    maximum that rises by one such step from a tile to the next: the
    probabilities stay inside fp16's range."""
    n, H, new, key = 300, 64, 148, 256
    cache = csa2.Cache(3, 128, [[2, 0, 1]], [n])
    rows = torch.from_numpy(O.rows_of(np.array([[2, 0, 1]]), 128, 0, n)).cuda()
    codes, scales = np.zeros((n, 256), np.uint8), np.full((n, 32), 0x38, np.uint8)     # scales of 1
    scales[:, 0] = 0x58                                # 16
    codes[:, 0] = 6                                    # channel 0: 4 x 16
    codes[:, 8] = 2                                    # channel 16: 1
    codes[key, 16] = 2                                 # channel 32: 1 for one key of the second tile
    codes[:, 24] = 2                                   # channel 48: 1 (no query looks at it)
    cache.kv_codes[rows], cache.kv_scales[rows] = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
    # q . v = 2^27 (1 + j / 128) + 16, and 16 more for that key: odd and even multiples of 16.  fp32's ln 2
    # times its log2 e rounds to 1, so the kernel's scores in log2 units are these numbers.
    scale = float(np.float32(np.log(2.0)))
    assert np.float32(scale) * np.float32(1.4426950408889634) == 1
    q = torch.zeros(new, H, 512)
    j = (torch.arange(new)[:, None] * 7 + torch.arange(H)) % 128
    q[..., 0] = 2.0 ** 21 * (1 + j / 128)
    q[..., 16] = q[..., 32] = 16
    lse = torch.empty(new, H, device="cuda")
    pos, start = torch.full((new,), n - 1, dtype=torch.int32).cuda(), torch.tensor([0, new], dtype=torch.int32).cuda()
    out = csa2.chunk_attn(cache, q.bfloat16().cuda(), pos, start, scale=scale, lse=lse).double().cpu()
    assert csa2.get_error(cache)[0] == csa2.OK
    rest = (n - 1) * 2.0 ** -16                        # the other keys, next to that one
    # P in fp16 (2^-11), the sums (n 2^-23 each), bf16's rounding
    tol = 2.0 ** -11 + 2 * n * 2.0 ** -23 + torch.finfo(torch.bfloat16).eps / 2
    for ch, want in ((48, 1.0), (32, 1 / (1 + rest)), (16, 1.0), (0, 64.0)):
        assert ((out[..., ch] - want).abs() <= 1.01 * tol * want).all(), ch
    want = scale * (2.0 ** 27 * (1 + j.double() / 128) + 32) + math.log(1 + rest)
    assert ((lse.double().cpu() - want).abs() <= 2.0 ** -22 * want).all()


@pytest.mark.parametrize("what", ["inf", "large", "masked"])
def test_chunk_attn_rows_do_not_depend_on_each_other(csa2, what):
    """Every fifth row is changed (an infinity, scores of 10^9, or a position that
    sees a part only): the bits of the others stay."""
    for seed in range(4):
        lens, new, H = [500], [60], 16
        args = _case(csa2, lens, new, H, 128, seed=seed, pos=[499] * 60)
        cache, start, pos, q = args[0], args[4], args[5], args[6]
        s, scale = torch.from_numpy(start).cuda(), 1 / math.sqrt(512)
        lse, lse2 = torch.empty(q.shape[:2], device="cuda"), torch.empty(q.shape[:2], device="cuda")
        out = csa2.chunk_attn(cache, q, torch.from_numpy(pos).cuda(), s, scale=scale, lse=lse)
        change = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
        if what == "masked":
            change[::5] = True
            pos[::5] = np.random.default_rng(seed).integers(0, 499, 12)
        else:
            change.view(-1)[::5] = True
            if what == "inf":
                q.view(-1, 512)[::5, 7] = float("inf")
            else:
                q.view(-1, 512)[::5] *= 2.0 ** 30
        again = csa2.chunk_attn(cache, q, torch.from_numpy(pos).cuda(), s, scale=scale, lse=lse2)
        assert not torch.equal(out[change], again[change])
        assert torch.equal(out[~change], again[~change]) and torch.equal(lse[~change], lse2[~change]), seed


@pytest.mark.parametrize("new", [2, 148])
def test_chunk_attn_long_tail_of_small_weights(csa2, new):
    """One entry 8 to 24 nats above 262,143 equal ones: the tail's weights count
    in the product with V as they do in the sum, in tiles that one range holds
    whole (148 tokens x 64 heads are a tile for each of 74 ranges) and in cut ones.

    Bounds: a score is one exact product, its factor and the reference are off by
    at most 2^-23 of 40 log2 units together, exp2 by 2^-22: 1e-5 for a weight, as
    much for the sum.  P is rounded to fp16 by 2^-11 of itself, or, below
    fp16's normal range, by 2^-25 where the row's largest P is at least 2^7:
    2^-32 of the largest weight for each of the n entries.  O takes 16 keys at a
    time, each sum off by at most 2^-22 of it; the fp32 row sum n / 256 roundings.
    """
    n, H, page = 1 << 18, 64, 4096
    cache = csa2.Cache(n // page, page, np.random.default_rng(3).permutation(n // page).astype(np.int32)[None], [n])
    first = int(cache.page_table[0, 0]) * page
    cache.kv_scales.fill_(0x38)                        # scales of 1
    cache.kv_codes[:, 8] = 2                           # channel 16: 1 for every entry
    cache.kv_codes[:, 16] = 2                          # channel 32: 1 for all but the first
    cache.kv_codes[first, 16] = 0
    cache.kv_codes[first, 0] = 2                       # channel 0: 1 for the first
    q = torch.zeros(new, H, 512)
    q[..., 0] = torch.linspace(8, 24, new * H).view(new, H)
    q = q.bfloat16()
    gap = q[..., 0].double()
    lse = torch.empty(new, H, device="cuda")
    pos, start = torch.full((new,), n - 1, dtype=torch.int32).cuda(), torch.tensor([0, new], dtype=torch.int32).cuda()
    out = csa2.chunk_attn(cache, q.cuda(), pos, start, scale=1.0, lse=lse).double().cpu()
    assert csa2.get_error(cache)[0] == csa2.OK
    tail = (n - 1) * torch.exp(-gap)
    top = 1 / (1 + tail)                               # the first entry's weight
    rel = 2e-5 + 2.0 ** -11 + n / 16 * 2.0 ** -22 + n / 256 * 2.0 ** -24
    for ch, want, low in ((0, top, 0.0), (32, tail * top, 1.0), (16, torch.ones_like(top), 1.0)):
        tol = rel * want + low * n * 2.0 ** -32 * top
        tol = tol + torch.finfo(torch.bfloat16).eps / 2 * (want + tol)
        err = (out[..., ch] - want).abs()
        assert (err <= tol).all(), f"channel {ch}: {float((err / tol).max()):.2f} of its bound, worst at {float(gap.flatten()[(err / tol).argmax()])} nats"
    want = gap + torch.log1p(tail)
    assert ((lse.double().cpu() - want).abs() <= 2e-5 + n / 256 * 2.0 ** -24 + 2.0 ** -23 * want).all()
