"""Per-head norm with the position rotation (csa2_norm_rope) and the same fused
into quantise-on-append (csa2_norm_rope_append) against their formulas in
float64.  Needs a B200 and libcsa2.so."""
import numpy as np
import pytest
import torch

from oracle import formats as F
from tests import ops_util as O

pytestmark = pytest.mark.gpu

# fp32 arithmetic of norm_rope, in units of 2^-24: a sum of 512 squares held as
# at most 16 terms a lane and 5 shuffle steps (21 roundings, halved by the
# square root), square root, division and the mean's factor (3), two products
# (2), the rotation's product and sum (2); cos and sin are off by at most
# pi * 2^-24 for the angle rounded to fp32 and 2 units for sincosf (5.2).
FP32 = (10.5 + 3 + 2 + 2 + 5.2) * 2.0 ** -24


@pytest.fixture(scope="module")
def csa2():
    from kv_cache_decode_index_b200 import csa2 as lib
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return lib


def _check(got, y, spread, dtype, what):
    tol = FP32 * spread + torch.finfo(dtype).eps / 2 * (np.abs(y) + FP32 * spread)
    err = np.abs(got.double().cpu().numpy() - y)
    assert (err <= tol).all(), f"{what}: worst error {(err - tol).max():.3e} over its bound"


@pytest.mark.parametrize("inter", [True, False])
@pytest.mark.parametrize("rot", [0, 32, 64, 128])
@pytest.mark.parametrize("src,dst", [("bfloat16", "bfloat16"), ("bfloat16", "float32"), ("float32", "bfloat16"),
                                     ("float32", "float32")])
@pytest.mark.parametrize("n,H,D,gap", [(1, 1, 128, 0), (3, 5, 512, 8), (37, 32, 128, 640), (2, 64, 512, 0),
                                       (9, 3, 128, 0), (5, 17, 512, 128)])
def test_norm_rope(csa2, n, H, D, gap, src, dst, rot, inter):
    src, dst = getattr(torch, src), getattr(torch, dst)
    g = torch.Generator().manual_seed(n * 1000 + H + rot)
    wide = (torch.randn(n, H * D + gap, generator=g) * 3).to(src).cuda()
    x = wide[:, :H * D].unflatten(1, (H, D))
    w = (1 + 0.2 * torch.randn(D, generator=g)).cuda()
    pos = torch.randint(0, 2 ** 21, (n,), generator=g, dtype=torch.int32).cuda()
    fr = O.freqs(rot)
    rope = csa2.Rope(torch.from_numpy(fr).cuda() if rot else None, inter)
    got = csa2.norm_rope(x, pos, rope, weight=w, out_dtype=dst)
    assert got.dtype == dst and got.shape == (n, H, D)
    y, spread = O.norm_rope(x.double().cpu().numpy(), w.cpu().numpy(), 1e-6, pos.cpu().numpy(), fr, inter)
    _check(got, y, spread, dst, "norm_rope")


@pytest.mark.parametrize("rot,inter,D", [(512, True, 512), (512, False, 512), (256, False, 512), (96, False, 128)])
def test_norm_rope_wide_rotation(csa2, rot, inter, D):
    g = torch.Generator().manual_seed(rot)
    x = torch.randn(11, 4, D, generator=g).cuda()
    pos = torch.randint(-5, 2 ** 31 - 1, (11,), generator=g, dtype=torch.int32).cuda()
    fr = O.freqs(rot)
    got = csa2.norm_rope(x, pos, csa2.Rope(torch.from_numpy(fr).cuda(), inter))
    y, spread = O.norm_rope(x.double().cpu().numpy(), None, 1e-6, pos.cpu().numpy(), fr, inter)
    _check(got, y, spread, torch.float32, "wide rotation")


def test_norm_rope_extreme_rows(csa2):
    """Zeros, rows whose squares leave fp32's range on either side, and rows
    with a NaN or an infinity, next to an ordinary row."""
    rows = torch.randn(6, 1, 512, generator=torch.Generator().manual_seed(3))
    rows[0] = 0.0
    rows[1] *= 3e37
    rows[2] *= 1e-30
    rows[3, 0, 7] = float("inf")
    rows[4, 0, 500] = float("nan")
    x = rows.cuda()
    pos = torch.arange(6, dtype=torch.int32).cuda() * 100
    fr = O.freqs(64)
    got = csa2.norm_rope(x, pos, csa2.Rope(torch.from_numpy(fr).cuda()))
    fine = [0, 1, 2, 5]
    y, spread = O.norm_rope(rows[fine].double().numpy(), None, 1e-6, pos.cpu().numpy()[fine], fr, True)
    _check(got[fine], y, spread, torch.float32, "extreme rows")
    g3, g4 = got[3, 0].cpu(), got[4, 0].cpu()
    assert torch.isnan(g3[7]) and int(torch.isnan(g3).sum()) == 1 and (g3[~torch.isnan(g3)] == 0).all()
    assert torch.isnan(g4).all()


def test_norm_rope_in_place_stream_and_graph(csa2):
    """out = x, on a side stream, captured and replayed."""
    g = torch.Generator().manual_seed(8)
    x0 = torch.randn(33, 16, 128, generator=g).cuda()
    pos = torch.arange(33, dtype=torch.int32).cuda()
    rope = csa2.Rope(torch.from_numpy(O.freqs(64)).cuda(), False)
    want = csa2.norm_rope(x0, pos, rope)
    x = x0.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        csa2.norm_rope(x, pos, rope, out=x)
    s.synchronize()
    assert torch.equal(x, want)
    y = torch.empty_like(x0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        csa2.norm_rope(x0, pos, rope, out=y)
    x0.mul_(2.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, csa2.norm_rope(x0, pos, rope))


def _cache(csa2, B, pages_per, page, seed=0):
    table = np.random.default_rng(seed).permutation(B * pages_per).astype(np.int32).reshape(B, pages_per)
    return csa2.Cache(B * pages_per, page, table, [0] * B), table


@pytest.mark.parametrize("src", ["bfloat16", "float32"])
@pytest.mark.parametrize("rot_kv,rot_ik,inter", [(64, 64, True), (64, 32, False), (0, 128, True), (512, 0, False),
                                                 (0, 0, True)])
def test_norm_rope_append_bitexact(csa2, src, rot_kv, rot_ik, inter):
    """Codes, scales and exponents of the formula in float64, rounded once to
    fp32; FP4 indexer rows too; rows of requests in shuffled pages."""
    src = getattr(torch, src)
    B, page, n = 3, 128, 61
    cache, table = _cache(csa2, B, 2, page)
    ik4 = csa2.Ik4(cache)
    rng = np.random.default_rng(5)
    both = torch.from_numpy((rng.standard_normal((n, 640)) * np.exp(rng.standard_normal((n, 1)))).astype(np.float32))
    both[3] = 0.0
    both = both.to(src).cuda()
    kv, ik = both[:, :512], both[:, 512:]
    slots = rng.choice(B * 2 * page, n, replace=False)
    req, pos = (slots // (2 * page)).astype(np.int32), (slots % (2 * page)).astype(np.int32)
    rope_pos = rng.integers(0, 2 ** 20, n).astype(np.int32)
    kvw = np.exp(0.5 * rng.standard_normal(512)).astype(np.float32)
    ikw = np.exp(0.2 * rng.standard_normal(128)).astype(np.float32)
    fk, fi = O.freqs(rot_kv), O.freqs(rot_ik, 500.0)
    c = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    csa2.norm_rope_append(cache, kv, ik, c(pos), csa2.Rope(c(fk) if rot_kv else None, inter),
                          csa2.Rope(c(fi) if rot_ik else None, inter), rope_pos=c(rope_pos), kv_weight=c(kvw),
                          ik_weight=c(ikw), req=c(req), ik4=ik4)
    st, word = csa2.get_error(cache)
    assert st == csa2.OK, word
    y = O.norm_rope(kv.double().cpu().numpy(), kvw, np.float32(1e-6), rope_pos, fk, inter)[0].astype(np.float32)
    z = O.norm_rope(ik.double().cpu().numpy(), ikw, np.float32(1e-6), rope_pos, fi, inter)[0].astype(np.float32)
    rows = table[req, pos // page].astype(np.int64) * page + pos % page
    kc, ks = F.quantize_main_kv(y)
    ic, ie = F.quantize_indexer(z)
    np.testing.assert_array_equal(cache.kv_codes.cpu().numpy()[rows], kc)
    np.testing.assert_array_equal(cache.kv_scales.cpu().numpy()[rows], ks)
    np.testing.assert_array_equal(cache.ik_codes.cpu().numpy()[rows], ic)
    np.testing.assert_array_equal(cache.ik_exp.cpu().numpy()[rows], ie)
    c4, s4 = F.quantize_indexer_fp4(z)
    np.testing.assert_array_equal(ik4.codes.cpu().numpy()[rows], c4)
    at = np.array([[csa2.ik4_scale_offset(int(r % 128), g) for g in range(8)] for r in rows])
    np.testing.assert_array_equal(ik4.scales.cpu().numpy()[(rows // 128)[:, None], at], s4)
    rest = np.setdiff1d(np.arange(cache.kv_codes.shape[0]), rows)   # no other row is touched
    assert int(cache.kv_codes[torch.from_numpy(rest).cuda()].sum()) == 0
    assert int(cache.ik_codes[torch.from_numpy(rest).cuda()].sum()) == 0


def test_norm_rope_append_matches_two_steps(csa2):
    """Without rotation, weight 1 and rows of RMS 1 already fp32-exact, it is
    csa2_append_kv of the normed row; req None: row i to request i."""
    B = 4
    a, _ = _cache(csa2, B, 1, 128)
    b, _ = _cache(csa2, B, 1, 128)
    sign = torch.from_numpy(np.random.default_rng(2).choice([-1.0, 1.0], (B, 640)).astype(np.float32)).cuda()
    pos = torch.tensor([0, 5, 127, 64], dtype=torch.int32).cuda()
    none = csa2.Rope()
    csa2.norm_rope_append(a, 2 * sign[:, :512], 2 * sign[:, 512:], pos, none, none, eps=1e-12)
    y = (2 * sign.double() / torch.sqrt(torch.tensor(4.0 + float(np.float32(1e-12)), dtype=torch.float64))).float()
    csa2.append_kv(b, y[:, :512].contiguous(), y[:, 512:].contiguous(), pos)
    for name in ("kv_codes", "kv_scales", "ik_codes", "ik_exp"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name


def test_norm_rope_append_bad_slots(csa2):
    """A slot, a request or a page out of range is recorded and skipped."""
    for what in ("pos", "req", "page"):
        cache, _ = _cache(csa2, 2, 1, 128)
        pos, req = torch.tensor([3, 4], dtype=torch.int32), torch.tensor([0, 1], dtype=torch.int32)
        if what == "pos":
            pos[1] = 128
        elif what == "req":
            req[1] = 2
        else:
            cache.page_table[1, 0] = 2
        x = torch.ones(2, 640).cuda()
        csa2.norm_rope_append(cache, x[:, :512], x[:, 512:], pos.cuda(), csa2.Rope(), csa2.Rope(), req=req.cuda())
        st, word = csa2.get_error(cache)
        assert st == csa2.ERR_DEVICE_BOUNDS, what
        assert int((cache.kv_codes.sum(1) > 0).sum()) == 1


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 3e38])
@pytest.mark.parametrize("where", ["kv_weight", "ik_weight", "kv", "ik"])
def test_norm_rope_append_not_finite(csa2, where, bad):
    """A weight or a value that is not finite (or as large as fp32 goes) is
    stored as csa2_append_kv stores the formula's fp32 row.  Without rotation
    every channel is by itself, so the formula needs no care in float64."""
    B = 2
    a, _ = _cache(csa2, B, 1, 128)
    b, _ = _cache(csa2, B, 1, 128)
    rng = np.random.default_rng(4)
    x = rng.standard_normal((B, 640)).astype(np.float32)
    w = np.ones(640, np.float32)
    if where.endswith("weight"):
        w[37 if where == "kv_weight" else 512 + 37] = bad
    else:
        x[1, 37 if where == "kv" else 512 + 37] = bad
    y = np.empty_like(x)
    with np.errstate(all="ignore"):
        for sl in (slice(0, 512), slice(512, 640)):
            v = x[:, sl].astype(np.float64)
            inv = 1.0 / np.sqrt((v * v).mean(-1, keepdims=True) + np.float64(np.float32(1e-6)))
            y[:, sl] = (v * inv * w[sl].astype(np.float64)).astype(np.float32)
    c = lambda t: torch.from_numpy(np.ascontiguousarray(t)).cuda()  # noqa: E731
    pos = torch.tensor([3, 100], dtype=torch.int32).cuda()
    none = csa2.Rope()
    csa2.norm_rope_append(a, c(x[:, :512]), c(x[:, 512:]), pos, none, none, kv_weight=c(w[:512]), ik_weight=c(w[512:]))
    csa2.append_kv(b, c(y[:, :512]), c(y[:, 512:]), pos)
    for name in ("kv_codes", "kv_scales", "ik_codes", "ik_exp"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name
