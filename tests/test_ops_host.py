"""Refusals of the cache operators (include/csa2_ops.h) on the host: no device
is touched."""
import ctypes
import os
import re

import pytest
import torch

from tests.test_abi import _cache, lib  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F32 = ctypes.c_float


def test_every_operator_is_exported(lib):  # noqa: F811
    text = open(os.path.join(ROOT, "include", "csa2_ops.h")).read()
    names = re.findall(r"CSA2_API\s+[\w\s\*]+?\b(csa2_\w+)\s*\(", text)
    assert names
    so = ctypes.CDLL(lib.LIB_PATH)
    for n in names:
        assert hasattr(so, n), f"{n} missing from libcsa2.so"


def test_norm_rope_refusals(lib):  # noqa: F811
    _, p = _cache(lib)
    P, f = ctypes.c_void_p(p), lib._lib.csa2_norm_rope
    rope = lambda rot=64, fr=p: ctypes.byref(lib.RopeStruct(fr, rot, 1))  # noqa: E731

    def call(n=1, H=2, D=128, x=P, xt=0, stride=256, w=P, eps=1e-6, r=None, pos=P, out=P, ot=0):
        return f(n, H, D, x, xt, stride, w, F32(eps), rope() if r is None else r, pos, out, ot, None)
    assert call(n=-1) == lib.ERR_SHAPE and call(D=256) == lib.ERR_SHAPE and call(H=0) == lib.ERR_SHAPE
    assert call(stride=255) == lib.ERR_SHAPE and call(stride=260) == lib.ERR_SHAPE      # 260 bf16: not 16 bytes
    assert call(xt=2) == lib.ERR_ARG and call(ot=-1) == lib.ERR_ARG
    assert call(eps=0.0) == lib.ERR_SHAPE and call(eps=float("nan")) == lib.ERR_SHAPE
    assert call(r=rope(48)) == lib.ERR_SHAPE and call(r=rope(160)) == lib.ERR_SHAPE
    assert call(r=rope(64, None)) == lib.ERR_ARG and call(r=rope(64, p + 4)) == lib.ERR_ARG
    assert call(x=None) == lib.ERR_ARG and call(out=ctypes.c_void_p(p + 8)) == lib.ERR_ARG
    assert call(pos=None) == lib.ERR_ARG and call(w=ctypes.c_void_p(p + 4)) == lib.ERR_ARG
    assert call(n=0, x=None, out=None, pos=None) == lib.OK


def test_norm_rope_append_refusals(lib):  # noqa: F811
    c, p = _cache(lib)
    P, f = ctypes.c_void_p(p), lib._lib.csa2_norm_rope_append
    good = lib.RopeStruct(p, 64, 1)

    def call(cache=c, ik4=None, n=2, t=1, kv=P, ks=640, ik=P, is_=640, eps=1e-6, kr=good, ir=good, req=P, pos=P):
        return f(ctypes.byref(cache), ik4, n, t, kv, ks, ik, is_, None, None, F32(eps), ctypes.byref(kr),
                 ctypes.byref(ir), None, req, pos, None)
    bad, _ = _cache(lib, page_size=100)
    assert call(cache=bad) == lib.ERR_SHAPE
    assert call(ik4=ctypes.byref(lib.Ik4Struct(None, None))) == lib.ERR_ARG
    assert call(n=-1) == lib.ERR_SHAPE and call(t=5) == lib.ERR_ARG
    assert call(ks=511) == lib.ERR_SHAPE and call(is_=130) == lib.ERR_SHAPE
    assert call(ir=lib.RopeStruct(p, 256, 1)) == lib.ERR_SHAPE and call(eps=2.0) == lib.ERR_SHAPE
    assert call(kv=None) == lib.ERR_ARG and call(ik=ctypes.c_void_p(p + 4)) == lib.ERR_ARG
    assert call(pos=None) == lib.ERR_ARG
    assert call(n=3, req=None) == lib.ERR_SHAPE
    assert call(n=0, kv=None, ik=None, pos=None) == lib.OK


def test_binding_refuses_tensors(lib):  # noqa: F811
    x, pos = torch.zeros(2, 4, 128), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        lib.norm_rope(x, pos, lib.Rope())                      # not on a GPU
    with pytest.raises(ValueError):
        lib.Rope(torch.zeros(32, dtype=torch.float32))
    with pytest.raises(ValueError):
        lib._rows(torch.zeros(2, 4, 128).transpose(1, 2), (2, 128, 4), "x", torch.device("cpu"))


def test_chunk_attn_refusals(lib):  # noqa: F811
    c, p = _cache(lib)
    P, f = ctypes.c_void_p(p), lib._lib.csa2_chunk_attn
    need = lib._lib.csa2_chunk_attn_workspace_bytes(2, 2, 64)
    assert need > 0 and lib._lib.csa2_chunk_attn_workspace_bytes(2, 0, 64) == 0

    def call(cache=c, n=2, start=P, pos=P, ratio=1, q=P, H=64, scale=0.1, out=P, ws=P, size=need):
        return f(ctypes.byref(cache), n, start, pos, ratio, q, H, F32(scale), out, None, ws, size, None)
    bad, _ = _cache(lib, kv_codes=p + 4)
    assert call(cache=bad) == lib.ERR_ARG
    assert call(n=-1) == lib.ERR_SHAPE and call(n=2 ** 20 + 1) == lib.ERR_SHAPE
    assert call(n=3, start=None) == lib.ERR_SHAPE
    assert call(ratio=0) == lib.ERR_SHAPE and call(H=48) == lib.ERR_SHAPE
    assert call(scale=float("inf")) == lib.ERR_ARG and call(scale=float("nan")) == lib.ERR_ARG
    assert call(pos=None) == lib.ERR_ARG and call(q=ctypes.c_void_p(p + 8)) == lib.ERR_ARG and call(out=None) == lib.ERR_ARG
    assert call(ws=None) == lib.ERR_ARG and call(ws=ctypes.c_void_p(p + 8)) == lib.ERR_ARG
    assert call(size=need - 1) == lib.ERR_SHAPE
    assert b"csa2_chunk_attn_workspace_bytes" in lib._lib.csa2_last_error_message()
    assert call(n=0, pos=None, q=None, out=None, ws=None, size=0) == lib.OK


def test_attn_mass_refusals(lib):  # noqa: F811
    c, p = _cache(lib)
    P, f = ctypes.c_void_p(p), lib._lib.csa2_attn_mass
    need = lib._lib.csa2_attn_mass_workspace_bytes(2, 2, 64)
    assert need > 0

    def call(cache=c, n=2, start=P, pos=P, ratio=1, q=P, H=64, scale=0.1, lse=P, mass=P, ws=P, size=need):
        return f(ctypes.byref(cache), n, start, pos, ratio, q, H, F32(scale), lse, mass, ws, size, None)
    assert call(n=-1) == lib.ERR_SHAPE and call(n=3, start=None) == lib.ERR_SHAPE
    assert call(ratio=0) == lib.ERR_SHAPE and call(H=8) == lib.ERR_SHAPE and call(scale=float("nan")) == lib.ERR_ARG
    assert call(q=ctypes.c_void_p(p + 2)) == lib.ERR_ARG and call(lse=None) == lib.ERR_ARG and call(mass=None) == lib.ERR_ARG
    assert call(ws=None) == lib.ERR_ARG and call(size=need - 1) == lib.ERR_SHAPE
    assert call(n=0, pos=None, q=None, lse=None, mass=None, ws=None, size=0) == lib.OK


def test_evict_refusals(lib):  # noqa: F811
    c, p = _cache(lib)
    P, f = ctypes.c_void_p(p), lib._lib.csa2_evict
    Q, R = ctypes.c_void_p(p + 512), ctypes.c_void_p(p + 1024)
    need = lib._lib.csa2_evict_workspace_bytes(4)
    assert need == 16 and lib._lib.csa2_evict_workspace_bytes(0) == 0

    def call(cache=c, ik4=None, mass=P, budget=100, sink=1, recent=9, dst=R, width=1, kept=Q, new_len=Q, out=None, ws=P,
             size=need):
        return f(ctypes.byref(cache), ik4, mass, budget, sink, recent, dst, width, kept, new_len, out, ws, size, None)
    assert call(budget=0) == lib.ERR_SHAPE and call(sink=-1) == lib.ERR_SHAPE and call(recent=100) == lib.ERR_SHAPE
    assert call(sink=2 ** 31 - 1, recent=2 ** 31 - 1) == lib.ERR_SHAPE
    assert call(budget=129) == lib.ERR_SHAPE and call(width=0) == lib.ERR_SHAPE
    assert call(mass=None) == lib.ERR_ARG and call(dst=None) == lib.ERR_ARG and call(kept=None) == lib.ERR_ARG
    assert call(out=P) == lib.ERR_ARG and call(new_len=P) == lib.ERR_ARG and call(dst=P) == lib.ERR_ARG
    assert call(ws=None) == lib.ERR_ARG and call(size=need - 1) == lib.ERR_SHAPE
    assert call(ik4=ctypes.byref(lib.Ik4Struct(None, None))) == lib.ERR_ARG


def test_overlapping_outputs_are_refused(lib):  # noqa: F811
    c, p = _cache(lib)
    V = ctypes.c_void_p
    f = lib._lib.csa2_chunk_attn
    need = lib._lib.csa2_chunk_attn_workspace_bytes(2, 2, 16)
    size = 2 * 16 * 512 * 2
    for out in (p, p + 16, p - 16, p + size - 16, p - size + 16):
        assert f(ctypes.byref(c), 2, V(p), V(p), 1, V(p), 16, F32(0.1), V(out), None, V(p), need, None) == lib.ERR_ARG
        assert b"overlaps" in lib._lib.csa2_last_error_message()
    f, rope = lib._lib.csa2_norm_rope, lib.RopeStruct(p, 64, 1)
    # rows of 2 x 128 bf16, 512 bytes each; x two rows, out bf16 or fp32
    for stride, out, ot in ((264, p, 0), (256, p, 1), (256, p + 16, 0), (256, p - 1008, 0), (256, p - 2032, 1),
                            (264, p + 1024, 0)):
        assert f(2, 2, 128, V(p), 0, stride, None, F32(1e-6), ctypes.byref(rope), V(p), V(out), ot, None) == lib.ERR_ARG
        assert b"overlaps" in lib._lib.csa2_last_error_message()


def test_capacities_above_2_30_are_refused(lib):  # noqa: F811
    """Positions plus a tile or a page would leave 32 bits."""
    V = ctypes.c_void_p
    c, p = _cache(lib, page_size=2 ** 20, num_pages=4, max_pages_per_req=1025)
    need = lib._lib.csa2_chunk_attn_workspace_bytes(2, 2, 16)
    assert lib._lib.csa2_chunk_attn(ctypes.byref(c), 2, V(p), V(p), 1, V(p), 16, F32(0.1), V(p + 2 ** 20), None, V(p), need,
                                    None) == lib.ERR_SHAPE
    need = lib._lib.csa2_attn_mass_workspace_bytes(2, 2, 16)
    assert lib._lib.csa2_attn_mass(ctypes.byref(c), 2, V(p), V(p), 1, V(p), 16, F32(0.1), V(p), V(p), V(p), need,
                                   None) == lib.ERR_SHAPE
    evict = lambda cache, budget: lib._lib.csa2_evict(  # noqa: E731
        ctypes.byref(cache), None, V(p), budget, 1, 9, V(p + 1024), 2047, V(p + 512), V(p + 512), None, V(p), 16, None)
    assert evict(c, 100) == lib.ERR_SHAPE
    assert b"2^30" in lib._lib.csa2_last_error_message()
    c, _ = _cache(lib, page_size=2 ** 20, num_pages=4, max_pages_per_req=1024)
    assert evict(c, 2 ** 30 + 1) == lib.ERR_SHAPE
    assert b"2^30" in lib._lib.csa2_last_error_message()


def test_mass_exchange_is_not_overrun():
    """Every order of steps of attn_mass's exchange() between two CTAs (two warps
    each, four exchanges one after the other), with as many barriers by turns as
    the kernel declares: no barrier completes a second phase while a warp still
    waits for the one before, whose parity it would then miss."""
    text = open(os.path.join(ROOT, "kv_cache_decode_index_b200", "csrc", "k_mass.cu")).read()
    found = re.search(r"uint64_t scale_full(?:\[(\d+)\])?;", text)
    turns, warps, rounds = int(found.group(1) or 1), 2, 4
    # a warp's place: 2 k before its arrival for exchange k, 2 k + 1 before its look at it; the vote
    # lets a warp go on once its CTA's warps have all looked
    start = ((0,) * warps,) * 2
    todo, known = [start], {start}
    while todo:
        state = todo.pop()
        for c in range(2):
            for w in range(warps):
                k, looks = divmod(state[c][w], 2)
                if k == rounds:
                    continue
                if looks:
                    mine = [j for j in range(rounds) if j % turns == k % turns]          # this barrier's exchanges
                    arrived = sum(p > 2 * j for p in state[1 - c] for j in mine)
                    done, phase = arrived // warps, k // turns
                    assert done <= phase + 1, f"exchange {k}: {done} phases are over, {phase} is awaited"
                    if done == phase:
                        continue                      # it waits
                elif any(p < 2 * k for p in state[c]):
                    continue                          # the vote: another warp has not looked yet
                place = tuple(p + (i == w) for i, p in enumerate(state[c]))
                after = (place, state[1]) if c == 0 else (state[0], place)
                if after not in known:
                    known.add(after)
                    todo.append(after)
    assert ((2 * rounds,) * warps,) * 2 in known


def test_evict_refuses_overlaps(lib):  # noqa: F811
    """Outputs and workspace that share bytes with an input or with one another:
    equal, shifted, or by one element.  (Every call is one that is refused.)"""
    _, p = _cache(lib)
    # mass 2 x 256 floats, dst_pages 2 x 1, page_table 2 x 2, ctx_len 2, kept 2 x 100, new_len 2, mass_out 2 x 128 floats
    at = {"mass": p, "dst_pages": p + 4096, "page_table": p + 4112, "ctx_len": p + 4144, "kept": p + 8192,
          "new_len": p + 9216, "mass_out": p + 12288, "workspace": p + 16384}
    size = {"mass": 2048, "dst_pages": 8, "page_table": 16, "ctx_len": 8, "kept": 800, "new_len": 8, "mass_out": 1024,
            "workspace": 16}
    outs, ins = ("kept", "new_len", "mass_out", "workspace"), ("mass", "dst_pages", "page_table", "ctx_len")
    V = ctypes.c_void_p

    def call(places):
        c, _ = _cache(lib, page_table=places["page_table"], ctx_len=places["ctx_len"])
        return lib._lib.csa2_evict(ctypes.byref(c), None, V(places["mass"]), 100, 1, 9, V(places["dst_pages"]), 1,
                                   V(places["kept"]), V(places["new_len"]), V(places["mass_out"]), V(places["workspace"]),
                                   16, None)
    for w in outs:
        for o in ins + outs:
            if o == w:
                continue
            unit = 16 if w == "workspace" else 4
            for where in (at[o], at[o] + (size[o] - 1) // unit * unit, at[o] - (size[w] - 1) // unit * unit):
                assert call({**at, w: where}) == lib.ERR_ARG, (w, o)
                assert b"overlaps" in lib._lib.csa2_last_error_message(), (w, o)


def test_dense_workspaces_hold_what_a_launch_can_touch(lib):  # noqa: F811
    """Two partial results for each of 74 pairs of CTAs, and a record of at most 64
    bytes: 128 rows x (512 sums, reference, sum), or 8,192 weights."""
    for batch, n, H in ((1, 1, 16), (8, 8, 64), (1024, 2 ** 20, 64)):
        assert lib._lib.csa2_chunk_attn_workspace_bytes(batch, n, H) <= 74 * (2 * 128 * 514 * 4 + 64)
        assert lib._lib.csa2_attn_mass_workspace_bytes(batch, n, H) <= 74 * (2 * 8192 * 4 + 64)
