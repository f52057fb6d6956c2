"""Eviction by accumulated attention weight (csa2_evict) against a plain
selection.  Needs a B200 and libcsa2.so."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def csa2():
    from kv_cache_decode_index_b200 import csa2 as lib
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return lib


def plain_kept(mass, n, budget, sink, recent):
    """Kept positions of one request: NaN first, then by weight, then by index."""
    if n <= budget:
        return np.arange(n)
    mid = mass[sink:n - recent].astype(np.float64) + 0.0
    mid = np.where(np.isnan(mid), np.inf, mid)
    nan = np.isnan(mass[sink:n - recent])
    order = np.lexsort((np.arange(len(mid)), -mid, ~nan))
    best = np.sort(order[:budget - sink - recent]) + sink
    return np.concatenate([np.arange(sink), best, np.arange(n - recent, n)])


def _setup(csa2, lens, budget, page, seed, ik4=False):
    rng = np.random.default_rng(seed)
    per, need = [-(-n // page) for n in lens], -(-budget // page)
    num = sum(per) + need * len(lens) + 1
    ids = rng.permutation(num).astype(np.int32)
    width = max(1, max(per))
    table = np.full((len(lens), width), -1, np.int32)
    dst = np.full((len(lens), need), -1, np.int32)
    at = 0
    for b, p in enumerate(per):
        table[b, :p] = ids[at:at + p]
        at += p
    for b, n in enumerate(lens):
        if n > budget:
            dst[b] = ids[at:at + need]
            at += need
    cache = csa2.Cache(num, page, table, lens)
    for t in (cache.kv_codes, cache.kv_scales, cache.ik_codes, cache.ik_exp):
        t.copy_(torch.from_numpy(rng.integers(0, 256, tuple(t.shape), dtype=np.uint8)))
    k4 = csa2.Ik4(cache) if ik4 else None
    if ik4:
        for t in (k4.codes, k4.scales):
            t.copy_(torch.from_numpy(rng.integers(0, 256, tuple(t.shape), dtype=np.uint8)))
    return cache, table, dst, k4, rng


def _rows(csa2, cache, k4):
    """Every row's bytes [rows, 417 (+72)]."""
    parts = [cache.kv_codes, cache.kv_scales, cache.ik_codes, cache.ik_exp[:, None]]
    parts = [p.cpu().numpy() for p in parts]
    if k4 is not None:
        rows = cache.kv_codes.shape[0]
        off = np.array([[csa2.ik4_scale_offset(m, g) for g in range(8)] for m in range(128)])
        r = np.arange(rows)
        parts += [k4.codes.cpu().numpy(), k4.scales.cpu().numpy()[(r // 128)[:, None], off[r % 128]]]
    return np.concatenate(parts, axis=1)


def _check(csa2, cache, table, dst, k4, mass, before, kept, new_len, mass_out, lens, budget, sink, recent):
    after = _rows(csa2, cache, k4)
    touched = np.zeros(len(before), bool)
    page = cache.page_size
    for b, n in enumerate(lens):
        want = plain_kept(mass[b], n, budget, sink, recent)
        full = np.full(budget, -1, np.int64)
        full[:len(want)] = want
        np.testing.assert_array_equal(kept[b].cpu().numpy(), full, err_msg=f"request {b}")
        assert int(new_len[b]) == min(n, budget)
        if n <= budget:
            assert (mass_out[b] == 7).all()
            continue
        j = np.arange(budget)
        to = dst[b, j // page].astype(np.int64) * page + j % page
        src = table[b, want // page].astype(np.int64) * page + want % page
        np.testing.assert_array_equal(after[to], before[src], err_msg=f"request {b}")
        touched[to] = True
        got = mass_out[b].cpu().numpy()
        np.testing.assert_array_equal(got[:budget].view(np.int32), mass[b][want].view(np.int32))
        assert (got[budget:] == 7).all()
    np.testing.assert_array_equal(after[~touched], before[~touched])


CASES = [
    # lens, budget, sink, recent, page
    ([300, 40, 128, 129], 64, 4, 16, 128),
    ([1, 2, 3], 2, 0, 1, 128),
    ([5], 1, 0, 0, 128),
    ([5], 1, 1, 0, 128),
    ([5], 1, 0, 1, 128),
    ([1000, 999], 500, 100, 400, 256),        # nothing is left for the weights
    ([5000, 17, 0, 4097], 1000, 0, 0, 128),
    ([70000], 33333, 7, 1001, 4096),
    ([20000, 400], 399, 0, 300, 128),
]


@pytest.mark.parametrize("ik4", [False, True])
@pytest.mark.parametrize("kind", ["normal", "ties", "odd", "narrow"])
@pytest.mark.parametrize("lens,budget,sink,recent,page", CASES)
def test_evict(csa2, lens, budget, sink, recent, page, kind, ik4):
    cache, table, dst, k4, rng = _setup(csa2, lens, budget, page, len(lens) + budget, ik4)
    cap = cache.capacity
    mass = np.exp(3 * rng.standard_normal((len(lens), cap))).astype(np.float32)
    if kind == "ties":
        mass = np.floor(np.log2(mass)).clip(0).astype(np.float32)
    elif kind == "odd":       # negative values, zeros of both signs, infinities, NaN
        mass = (rng.standard_normal(mass.shape) * 2).astype(np.float32)
        pick = rng.random(mass.shape)
        for lo, v in ((0.0, 0.0), (0.1, -0.0), (0.2, np.inf), (0.22, -np.inf), (0.25, np.nan), (0.27, -np.nan), (0.3, 1e-42)):
            mass[(pick >= lo) & (pick < lo + 0.02)] = v
    elif kind == "narrow":    # keys that differ in their last bits alone
        mass = (np.float32(1.0) + rng.integers(0, 40, mass.shape) * np.float32(2.0 ** -23)).astype(np.float32)
    before = _rows(csa2, cache, k4)
    width = dst.shape[1]
    mass_out = torch.full((len(lens), width * page), 7.0).cuda()
    kept, new_len = csa2.evict(cache, torch.from_numpy(mass).cuda(), budget, torch.from_numpy(dst).cuda(), sink=sink,
                               recent=recent, mass_out=mass_out, ik4=k4)
    st, word = csa2.get_error(cache)
    assert st == csa2.OK, word
    _check(csa2, cache, table, dst, k4, mass, before, kept, new_len, mass_out, lens, budget, sink, recent)


def test_evict_shared_pages_stay(csa2):
    """Two requests that share their first page: both are moved, the shared
    page is as before."""
    page, budget = 128, 100
    table = np.array([[0, 1], [0, 2]], np.int32)
    cache = csa2.Cache(6, page, table, [256, 200])
    rng = np.random.default_rng(0)
    for t in (cache.kv_codes, cache.kv_scales, cache.ik_codes, cache.ik_exp):
        t.copy_(torch.from_numpy(rng.integers(0, 256, tuple(t.shape), dtype=np.uint8)))
    before = _rows(csa2, cache, None)
    mass = rng.random((2, 256)).astype(np.float32)
    dst = np.array([[4], [3]], np.int32)
    mass_out = torch.full((2, page), 7.0).cuda()
    kept, new_len = csa2.evict(cache, torch.from_numpy(mass).cuda(), budget, torch.from_numpy(dst).cuda(), mass_out=mass_out)
    assert csa2.get_error(cache)[0] == csa2.OK
    _check(csa2, cache, table, dst, None, mass, before, kept, new_len, mass_out, [256, 200], budget, 0, 0)


@pytest.mark.parametrize("what", ["own", "other", "twice", "range", "source"])
def test_evict_bad_pages(csa2, what):
    """A destination that holds visible entries, is given twice or is out of
    range, and a source page out of range: recorded, and no visible entry
    changes."""
    page, budget = 128, 200
    table = np.array([[0, 1, 2], [3, 4, -1]], np.int32)
    cache = csa2.Cache(10, page, table, [300, 256])
    rng = np.random.default_rng(0)
    for t in (cache.kv_codes, cache.kv_scales, cache.ik_codes, cache.ik_exp):
        t.copy_(torch.from_numpy(rng.integers(0, 256, tuple(t.shape), dtype=np.uint8)))
    before = _rows(csa2, cache, None)
    dst = np.array([[5, 6], [7, 8]], np.int32)
    if what == "source":
        cache.page_table[0, 1] = 10
    else:
        dst[0, 1] = {"own": 2, "other": 4, "twice": 8, "range": -1}[what]
    mass = rng.random((2, 384)).astype(np.float32)
    kept, new_len = csa2.evict(cache, torch.from_numpy(mass).cuda(), budget, torch.from_numpy(dst).cuda())
    st, word = csa2.get_error(cache)
    assert st == csa2.ERR_DEVICE_BOUNDS, word
    after = _rows(csa2, cache, None)
    np.testing.assert_array_equal(after[:5 * page], before[:5 * page])
    np.testing.assert_array_equal(after[9 * page:], before[9 * page:])
    want = plain_kept(mass[0], 300, budget, 0, 0)
    j = np.arange(page if what != "source" else budget)
    ok = np.ones(len(j), bool) if what != "source" else want[j] // page != 1
    to = dst[0, j // page] * page + j % page
    src = table[0, want[j] // page] * page + want[j] % page
    np.testing.assert_array_equal(after[to[ok]], before[src[ok]])
    np.testing.assert_array_equal(after[to[~ok]], before[to[~ok]])


def test_evict_bad_length_and_graph(csa2):
    cache, table, dst, _, rng = _setup(csa2, [300, 500], 100, 128, 3)
    mass = rng.random((2, cache.capacity)).astype(np.float32)
    m, d = torch.from_numpy(mass).cuda(), torch.from_numpy(dst).cuda()
    before = _rows(csa2, cache, None)
    kept = torch.zeros(2, 100, dtype=torch.int32).cuda()
    new_len = torch.zeros(2, dtype=torch.int32).cuda()
    mass_out = torch.full((2, 128), 7.0).cuda()
    ws = torch.empty(csa2.evict_workspace_bytes(cache), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        csa2.evict(cache, m, 100, d, sink=3, recent=20, kept=kept, new_len=new_len, mass_out=mass_out, workspace=ws)
    ws.fill_(0xFF)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    _check(csa2, cache, table, dst, None, mass, before, kept, new_len, mass_out, [300, 500], 100, 3, 20)
    cache.ctx_len[0] = cache.capacity + 1
    kept, new_len = csa2.evict(cache, m, 100, d)
    st, word = csa2.get_error(cache)
    assert st == csa2.ERR_DEVICE_BOUNDS and word[2] == 0
    assert (kept[0] == -1).all() and int(new_len[0]) == 0 and int(new_len[1]) == 100


def test_evict_long_request(csa2):
    """A request of 1,048,576 entries, most without any weight."""
    n, budget, page = 1 << 20, 65536, 4096
    cache = csa2.Cache(n // page + budget // page, page, np.arange(n // page, dtype=np.int32)[None], [n])
    g = torch.Generator(device="cuda").manual_seed(1)
    cache.kv_codes.random_(0, 256, generator=g)
    mass = torch.randn(1, n, device="cuda", generator=g).clamp_(min=0.5).sub_(0.5)
    dst = torch.arange(n // page, n // page + budget // page, dtype=torch.int32, device="cuda")[None]
    kept, new_len = csa2.evict(cache, mass, budget, dst, sink=100, recent=5000)
    assert csa2.get_error(cache)[0] == csa2.OK
    want = plain_kept(mass[0].cpu().numpy(), n, budget, 100, 5000)
    np.testing.assert_array_equal(kept[0].cpu().numpy(), want)
    assert torch.equal(cache.kv_codes[n:], cache.kv_codes[torch.from_numpy(want).cuda()])


def test_evict_many_requests(csa2):
    """40 requests , short and long ones among them."""
    rng = np.random.default_rng(12)
    lens = [int(x) for x in rng.integers(1, 3000, 40)]
    lens[7], lens[30] = 70000, 59000
    budget, page = 700, 128
    cache, table, dst, k4, rng = _setup(csa2, lens, budget, page, 4)
    mass = np.floor(np.exp(3 * rng.standard_normal((40, cache.capacity)))).astype(np.float32)
    before = _rows(csa2, cache, k4)
    mass_out = torch.full((40, dst.shape[1] * page), 7.0).cuda()
    kept, new_len = csa2.evict(cache, torch.from_numpy(mass).cuda(), budget, torch.from_numpy(dst).cuda(), sink=3,
                               recent=99, mass_out=mass_out)
    assert csa2.get_error(cache)[0] == csa2.OK
    _check(csa2, cache, table, dst, k4, mass, before, kept, new_len, mass_out, lens, budget, 3, 99)


def test_evict_neighbouring_buffers(csa2):
    """Inputs and outputs that touch in one buffer, without a gap."""
    budget, page = 100, 128
    cache, table, dst, _, rng = _setup(csa2, [300, 500], budget, page, 3)
    cap, width = cache.capacity, dst.shape[1]
    mass = rng.random((2, cap)).astype(np.float32)
    before = _rows(csa2, cache, None)
    sizes = [2 * cap, 2 * width * page, 2 * budget, 2, 2 * width, 2]
    buf = torch.zeros(sum(sizes), dtype=torch.int32, device="cuda")
    m, mass_out, kept, new_len, pages, ctx = torch.split(buf, sizes)
    m, mass_out, kept = m.view(torch.float32).view(2, cap), mass_out.view(torch.float32).view(2, -1), kept.view(2, budget)
    pages = pages.view(2, width)
    m.copy_(torch.from_numpy(mass))
    mass_out.fill_(7.0)
    pages.copy_(torch.from_numpy(dst))
    ctx.copy_(cache.ctx_len)
    cache.ctx_len = ctx
    csa2.evict(cache, m, budget, pages, sink=3, recent=20, kept=kept, new_len=new_len, mass_out=mass_out)
    assert csa2.get_error(cache)[0] == csa2.OK
    _check(csa2, cache, table, dst, None, mass, before, kept, new_len, mass_out, [300, 500], budget, 3, 20)
