"""Host side of the attention layer's operators (CPU only): the index arithmetic of the paged cache and
of the cut of the work, compiled for the host and compared with enumeration, the refusals of the entry points,
and the fp64 forms that the GPU tests use."""
import ctypes
import os
import random
import subprocess

import numpy as np
import pytest
import torch

import layer_reference as ref
import recsys_context_personalised_b200 as pkg
from recsys_context_personalised_b200 import gdpa as G

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "recsys_context_personalised_b200", "csrc")

HOST = r"""
#include "chunk_plan.cuh"
using namespace gdpa;
extern "C" {
int32_t h_page_of(const int32_t* row, int max_pages, int num_pages, int shift, int64_t pos) {
  return page_of(row, max_pages, num_pages, shift, pos);
}
int64_t h_cache_row(int32_t id, int head, int hk, int shift, int row, int dh) {
  return cache_row(id, head, hk, shift, row, dh);
}
int32_t h_blocks(int n, int ctx, int window, int rt, int shift, int tile) {
  return ChunkSample{n, ctx, window, rt, shift}.blocks(tile);
}
int32_t h_first(int n, int ctx, int window, int rt, int shift, int tile) {
  return ChunkSample{n, ctx, window, rt, shift}.first_block(tile);
}
int64_t h_before(int n, int ctx, int window, int rt, int shift, int tile) {
  return ChunkSample{n, ctx, window, rt, shift}.blocks_before(tile);
}
void h_place(int n, int ctx, int window, int rt, int shift, int64_t x, int32_t* out) {
  const ChunkPlace p = place_of(ChunkSample{n, ctx, window, rt, shift}, x);
  out[0] = p.head; out[1] = p.tile; out[2] = p.block;
}
int64_t h_part(int64_t total, int workers, int w) { return part_start(total, workers, w); }
}
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "host.cpp").write_text(HOST)
    so = str(d / "libplan.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-x", "c++",
                    "-fsanitize=undefined", "-fno-sanitize-recover=all",
                    "-I", CSRC, str(d / "host.cpp"), "-o", so], check=True)
    lib = ctypes.CDLL(so)
    i32, i64, p = ctypes.c_int32, ctypes.c_int64, ctypes.POINTER(ctypes.c_int32)
    lib.h_page_of.argtypes = [p, i32, i32, i32, i64]
    lib.h_cache_row.argtypes, lib.h_cache_row.restype = [i32] * 6, i64
    for f in ("h_blocks", "h_first", "h_before"):
        getattr(lib, f).argtypes = [i32] * 6
    lib.h_before.restype = i64
    lib.h_place.argtypes, lib.h_place.restype = [i32] * 5 + [i64, p], None
    lib.h_part.argtypes, lib.h_part.restype = [i64, i32, i32], i64
    return lib


def test_pages(host):
    row = (ctypes.c_int32 * 3)(5, -1, 9)
    assert host.h_page_of(row, 3, 10, 4, 0) == 5 and host.h_page_of(row, 3, 10, 4, 15) == 5
    assert host.h_page_of(row, 3, 10, 4, 16) == -1            # no page
    assert host.h_page_of(row, 3, 10, 4, 47) == 9
    assert host.h_page_of(row, 3, 9, 4, 47) == -1             # id past the cache
    assert host.h_page_of(row, 3, 10, 4, 48) == -1            # past the table
    assert host.h_page_of(row, 3, 10, 4, -1) == -1
    # offsets past 32 bits
    assert host.h_cache_row(40_000_000, 3, 8, 7, 127, 128) == ((40_000_000 * 8 + 3) * 128 + 127) * 128


def _blocks(n, ctx, window, rt, bn, tile):
    """(first block, blocks) of a tile by enumeration of what its rows see."""
    seen = [p for i in range(tile * rt, min(n, (tile + 1) * rt))
            for p in (max(0, ctx + i - window + 1), ctx + i) if ctx + i >= 0]
    return (min(seen) // bn, max(seen) // bn - min(seen) // bn + 1) if seen else (0, 1)


@pytest.mark.parametrize("seed", range(60))
def test_cut_matches_enumeration(host, seed):
    r = random.Random(seed)
    n, rt, shift = r.randint(1, 900), r.choice([1, 2, 3, 5, 16, 21, 32, 42, 64, 128]), r.choice([6, 7, 8])
    ctx = r.choice([0, r.randint(0, 3000), -r.randint(1, 2 * n), -n])
    window = r.choice([1, r.randint(1, 500), 2**31 - 1])
    tiles = -(-n // rt)
    total, places = 0, []
    for t in range(tiles):
        first, cnt = _blocks(n, ctx, window, rt, 1 << shift, t)
        args = (n, ctx, window, rt, shift, t)
        assert host.h_before(*args) == total
        assert host.h_blocks(*args) == cnt
        assert ctx + min(n, (t + 1) * rt) <= 0 or host.h_first(*args) == first
        places += [(t, j) for j in range(cnt)]
        total += cnt
    assert host.h_before(n, ctx, window, rt, shift, tiles) == total
    out = (ctypes.c_int32 * 3)()
    for x in [0, total - 1, total, 2 * total - 1] + [r.randrange(3 * total) for _ in range(20)]:
        host.h_place(n, ctx, window, rt, shift, x, out)
        assert (out[0], out[1], out[2]) == (x // total, *places[x % total])


def test_cut_of_long_lengths(host):
    """Closed form at lengths whose sums pass 32 bits, against the sum over tiles."""
    n, ctx, window, rt, shift = 1_000_000, 2_000_000_000 - 1_000_000, 2**31 - 1, 7, 6
    tiles = -(-n // rt)
    got = host.h_before(n, ctx, window, rt, shift, tiles)
    u = np.arange(tiles, dtype=np.int64)
    last = (ctx + np.minimum(n, (u + 1) * rt) - 1) >> shift
    assert got == int((last + 1).sum()) and got > 2**31


@pytest.mark.parametrize("total,workers", [(0, 296), (5, 296), (296, 296), (10**12 + 7, 148), (1000, 7)])
def test_parts_cover_the_line(host, total, workers):
    cut = [host.h_part(total, workers, w) for w in range(workers + 1)]
    size = np.diff(cut)
    assert cut[0] == 0 and cut[-1] == total and size.min() >= 0 and size.max() - size.min() <= 1
    assert (np.diff(size) <= 0).all()         # no empty part between two that hold blocks


# ------------------------------------------------------------------------- refusals
P = 4096     # a plausible pointer: validation fails before anything reads it


def _rot(**kw):
    d = dict(rot=64, base=10000.0, interleaved=False)
    d.update(kw)
    return G.rotary_spec(**d)


def _rotary(spec=None, dtype=1, B=2, h=4, dh=64, T=10, off=P, kv=None, pos=None, x=P, xs=256, y=P,
            ys=256):
    return G.load().gdpa_rotary(ctypes.byref(spec or _rot()), dtype, B, h, dh, T, off, kv, pos, x,
                                xs, y, ys, 0, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), 1), (dict(h=0), 1), (dict(T=-1), 1), (dict(dh=48), 2), (dict(off=None), 1),
    (dict(x=None), 1), (dict(x=P + 8), 1), (dict(xs=255), 1), (dict(xs=260), 1), (dict(ys=128), 1),
    (dict(ys=264), 1), (dict(kv=P, pos=P), 1), (dict(kv=P + 2), 1), (dict(B=0), 1),
    (dict(h=1 << 15, xs=1 << 21, ys=1 << 21), 2),
])
def test_rotary_refusals(kw, code):
    assert _rotary(**kw) == code


@pytest.mark.parametrize("kw", [
    dict(rot=0), dict(rot=63), dict(rot=66), dict(base=0.5), dict(base=float("nan")),
    dict(factor=0.5), dict(factor=float("inf")), dict(mscale=float("nan")), dict(trained_len=-1),
    dict(trained_len=100, low=4.0, high=4.0),
])
def test_rotary_spec_refusals(kw):
    assert _rotary(spec=_rot(**kw)) == 1


def _cache(**kw):
    d = dict(k=P, v=P, page_table=P, num_pages=8, max_pages=4, page=16, hk=2, dh=64, reserved=0)
    d.update(kw)
    return G.Cache(*[d[f[0]] for f in G.Cache._fields_])


BAD_CACHES = [(dict(k=None), 1), (dict(v=P + 8), 1), (dict(page_table=None), 1), (dict(num_pages=0), 1),
              (dict(max_pages=0), 1), (dict(page=8), 2), (dict(page=48), 2), (dict(page=2048), 2),
              (dict(dh=96), 2), (dict(hk=0), 1), (dict(max_pages=1 << 28), 2)]


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_cache_refusals(kw, code):
    lib, c, n = G.load(), _cache(**kw), ctypes.c_size_t()
    assert lib.gdpa_chunk_workspace_size(ctypes.byref(c), 2, 4, 10, 8, ctypes.byref(n)) == code
    assert lib.gdpa_cache_append(None, ctypes.byref(c), 2, 0, 10, P, P, None, 0, None, P, 128, P,
                                 128, None, None) == code


def test_append_refusals():
    lib, c = G.load(), _cache()

    def call(r=None, B=2, hq=0, T=10, off=P, kv=P, q=None, qs=0, qo=None, k=P, ks=128, v=P, vs=128,
             ws=None):
        return lib.gdpa_cache_append(r, ctypes.byref(c), B, hq, T, off, kv, q, qs, qo, k, ks, v, vs,
                                     ws, None)
    for kw in (dict(off=None), dict(kv=None), dict(k=None), dict(ks=120), dict(vs=132), dict(q=P),
               dict(q=P, qo=P, hq=0), dict(q=P, qo=P, hq=2, qs=64), dict(T=-1), dict(B=0),
               dict(r=ctypes.byref(_rot(rot=128))), dict(q=P, qo=P, hq=2, qs=256)):
        assert call(**kw) == 1, kw
    assert call(ws=P + 64) == 5


def test_chunk_refusals():
    lib, c, n = G.load(), _cache(), ctypes.c_size_t()
    size = lib.gdpa_chunk_workspace_size
    assert size(ctypes.byref(c), 2, 3, 10, 8, ctypes.byref(n)) == 1          # 3 heads on 2
    assert size(ctypes.byref(c), 2, 4, 17, 8, ctypes.byref(n)) == 1          # T > B * max_n
    assert size(ctypes.byref(c), 2, 258, 10, 8, ctypes.byref(n)) == 2        # 129 heads on one
    assert size(ctypes.byref(c), 2, 4, 10, 8, ctypes.byref(n)) == 0 and n.value % 256 == 0

    def call(window=8, scale=1.0, q=P, off=P, kv=P, o=P, lse=None, ws=P, nbytes=1 << 40):
        return lib.gdpa_chunk_fwd(ctypes.byref(c), 2, 4, 10, 8, window, scale, q, off, kv, o, lse,
                                  ws, nbytes, None)
    for kw in (dict(window=0), dict(scale=float("nan")), dict(scale=float("inf")), dict(q=None),
               dict(o=P + 8), dict(off=None), dict(kv=None), dict(lse=P + 2)):
        assert call(**kw) == 1, kw
    assert call(ws=None) == 5 and call(ws=P + 128) == 5 and call(nbytes=n.value - 1) == 5


def _norm(**kw):
    d = dict(T=10, d=64, dtype=1, gate=0, sigmoid=0, B=0, alpha=1.0, eps=1e-6, reserved=0)
    d.update(kw)
    return G.BlockNorm(*[d[f[0]] for f in G.BlockNorm._fields_])


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(d=0), 1), (dict(d=8193), 2), (dict(dtype=3), 1), (dict(gate=3), 1),
    (dict(gate=2), 1), (dict(alpha=float("inf")), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
])
def test_norm_refusals(kw, code):
    lib, p, n = G.load(), _norm(**kw), ctypes.c_size_t()
    assert lib.gdpa_block_norm_bwd_workspace_size(ctypes.byref(p), ctypes.byref(n)) == code
    assert lib.gdpa_block_norm_fwd(ctypes.byref(p), P, P, P, P, P, P, P, P, None) == code


def test_norm_operand_refusals():
    lib, p, g = G.load(), _norm(), _norm(gate=1)

    def fwd(p=p, off=None, x=P, f=P, gate=None, wq=P, wp=P, y=P, n=P):
        return lib.gdpa_block_norm_fwd(ctypes.byref(p), off, x, f, gate, wq, wp, y, n, None)
    for kw in (dict(x=None), dict(y=None), dict(n=None), dict(wp=None), dict(f=None), dict(p=g),
               dict(gate=P), dict(x=P + 8), dict(wq=P + 4), dict(p=_norm(gate=2, B=2), gate=P),
               dict(f=None, wq=None, y=None, wp=None, n=None)):
        assert fwd(**kw) == 1, kw
    n = ctypes.c_size_t()
    assert lib.gdpa_block_norm_bwd_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0

    def bwd(p=p, off=None, y=P, f=P, gate=None, wq=P, wp=P, dy=P, dn=P, dx=P, df=P, dg=None, dwq=P,
            dwp=P, ws=P, size=1 << 40):
        return lib.gdpa_block_norm_bwd(ctypes.byref(p), off, y, f, gate, wq, wp, dy, dn, dx, df, dg,
                                       dwq, dwp, ws, size, None)
    for kw in (dict(y=None), dict(dn=None), dict(dx=None), dict(df=None), dict(dwq=None),
               dict(dwp=None), dict(p=g, gate=P), dict(wp=None, dwp=None, dn=None, dy=None)):
        assert bwd(**kw) == 1, kw
    assert bwd(ws=None) == 5 and bwd(size=n.value - 1) == 5


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    off = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(G.GdpaError) as e:
        pkg.gdpa.rotary(_rot(), x, offsets=off)
    assert e.value.code == 1
    with pytest.raises(G.GdpaError):
        pkg.gdpa.block_norm_fwd(torch.zeros(4, 8), w_pre=torch.ones(8))


# ------------------------------------------------------- the fp64 forms of the GPU tests
@pytest.mark.parametrize("gate", [None, "token", "sample"])
@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False)])
def test_norm_formulas_against_autograd_and_differences(gate, post, pre):
    g = torch.Generator().manual_seed(4)
    T, d, B = 7, 12, 3
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)       # noqa: E731
    sample = torch.tensor([0, 0, 1, 1, 1, 2, 2]) if gate == "sample" else None
    leaves = dict(x=rnd(T, d), f=rnd(T, d),
                  gate=None if gate is None else rnd(B if gate == "sample" else T, d),
                  w_post=rnd(d) if post else None, w_pre=rnd(d) if pre else None)
    kw = dict(alpha=0.7, eps=1e-6, sigmoid=True, sample=sample)
    dy, dn = rnd(T, d), rnd(T, d) if pre else None

    def loss(v):
        y, n = ref.block_norm(**v, **kw)
        return (y * dy).sum() + (0 if n is None else (n * dn).sum())
    live = {k: v.clone().requires_grad_() for k, v in leaves.items() if v is not None}
    auto = dict(zip(live, torch.autograd.grad(loss({**leaves, **live}), live.values())))
    y, _ = ref.block_norm(**leaves, **kw)
    got = ref.block_norm_grads(y, leaves["f"], leaves["gate"], leaves["w_post"], leaves["w_pre"], dy,
                               dn, B=B, **kw)
    for name, key in (("x", "dx"), ("f", "df"), ("gate", "dgate"), ("w_post", "dw_post"),
                      ("w_pre", "dw_pre")):
        if name not in auto:
            continue
        assert torch.allclose(got[key][0], auto[name], rtol=1e-11, atol=1e-11), name
        flat, h = leaves[name].reshape(-1), 1e-6
        for i in range(0, flat.numel(), max(1, flat.numel() // 9)):
            side = []
            for s in (h, -h):
                v = flat.clone()
                v[i] += s
                side.append(loss({**leaves, name: v.view_as(leaves[name])}))
            # central differences: truncation h^2 and rounding 1e-16 / h, both far below 1e-6
            assert abs((side[0] - side[1]) / (2 * h) - auto[name].reshape(-1)[i]) < 1e-6


def test_rotary_form_is_orthogonal():
    r = np.random.default_rng(0)
    x, g = r.normal(size=(5, 2, 32)), r.normal(size=(5, 2, 32))
    kw = dict(pos=np.array([0, 1, -3, 1000, 2**31 - 1]), rot=24, interleaved=True, factor=4.0,
              trained_len=256)
    y, _ = ref.rotary(x, **kw)
    dx, _ = ref.rotary(g, inverse=True, **kw)
    assert abs((y * g).sum() - (x * dx).sum()) < 1e-12
    assert np.allclose((y * y).sum(-1), (x * x).sum(-1))
