"""The attention layer's operators on the GPU against their plain fp64 forms (layer_reference), element
by element.

Tolerances.  A result rounded to bf16 / fp32 is off by half a step, HALF[dtype] of its value.
  rotary   each element is two products of an fp32 (cos, sin) with relative error below 4 * 2^-24
           (sincospif 2 ulp, the angle 2^-26 turns, mscale) and three fp32 roundings: 8 * 2^-24 of |a| + |b|.
  chunk    P is rounded to bf16 before PV: 2^-8 of sum p|v|.  A logit's fp32 sum of dh products is off by
           at most (dh + 4) 2^-24 of sum |q||k| (times scale), and ex2.approx by 2^-22; both move p relatively,
           in the numerator and the denominator.
  norm     fp32 sums over a row: at most 16 terms in a thread, 9 levels of a tree and 16 warps, so 2^-24 * 48
           relative; with the exponential's 2^-21 and the products around them 2^-18 of the terms' absolute sum.
           Sums over rows add one 2^-24 per row of a group and per group."""
import numpy as np
import pytest
import torch

import layer_reference as ref
import recsys_context_personalised_b200 as pkg
from recsys_context_personalised_b200 import gdpa as G

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _np(t):
    return t.detach().double().cpu().numpy()


def _offsets(n):
    off = np.concatenate([[0], np.cumsum(n)]).astype(int)
    return [int(x) for x in off], torch.tensor(off, dtype=torch.int32, device=DEV)


def _near(got, want, tol, what=""):
    err = np.abs(_np(got) - want)
    assert np.isfinite(_np(got)).all(), what
    assert (err <= tol).all(), (what, float((err - tol).max()), float(err.max()))


def _int32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------------------ rotary
ROT = [dict(rot=64), dict(rot=64, interleaved=True), dict(rot=32), dict(rot=30, interleaved=True),
       dict(rot=22), dict(rot=2), dict(rot=64, factor=4.0),
       dict(rot=48, factor=8.0, trained_len=2048, mscale=1.2, interleaved=True)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kw", ROT, ids=str)
@pytest.mark.parametrize("inverse", [False, True])
def test_rotary(kw, dtype, inverse):
    n, h, dh = [1, 0, 37, 5, 0, 64], 3, 64
    off, offd = _offsets(n)
    x = torch.randn(off[-1], h, dh, generator=torch.Generator().manual_seed(1)).to(dtype)
    kv = [1, 7, 1000, 2**31 - 1, 3, 500000]
    y = G.rotary(G.rotary_spec(**kw), x.to(DEV), offsets=offd, kv_len=_int32(kv), inverse=inverse)
    want, mag = ref.rotary(_np(x), ref.positions(off, kv), inverse=inverse, **kw)
    _near(y, want, HALF[dtype] * np.abs(want) + 8 * 2.0 ** -24 * mag)


@pytest.mark.parametrize("dh", [32, 64, 128])
@pytest.mark.parametrize("h", [1, 5])
@pytest.mark.parametrize("T", [1, 17, 20000])
def test_rotary_of_strided_heads_in_place(T, h, dh):
    """Heads 1 .. h of a wider fused tensor, turned in place by given positions (negative ones too); the heads
    around them stay."""
    g = torch.Generator().manual_seed(T + dh)
    wide = torch.randn(T, h + 3, dh, generator=g).bfloat16()
    pos = torch.randint(-5, 100000, (T,), generator=g, dtype=torch.int32)
    w = wide.to(DEV)
    part = w[:, 1:1 + h]
    spec = dict(rot=dh // 2 + 2, interleaved=bool(T % 2))
    out = G.rotary(G.rotary_spec(**spec), part, positions=pos.to(DEV), out=part)
    assert out.data_ptr() == part.data_ptr()
    want, mag = ref.rotary(_np(wide[:, 1:1 + h]), pos.numpy(), **spec)
    _near(part, want, HALF[torch.bfloat16] * np.abs(want) + 8 * 2.0 ** -24 * mag)
    assert torch.equal(w[:, :1].cpu(), wide[:, :1]) and torch.equal(w[:, 1 + h:].cpu(), wide[:, 1 + h:])


def test_rotary_leaves_rows_behind_the_last_sample():
    off, offd = _offsets([3, 0, 5])
    x = torch.randn(20, 2, 32, device=DEV)
    out = torch.full_like(x, 7.0)
    G.rotary(G.rotary_spec(32), x, offsets=offd, out=out)
    assert (out[8:] == 7.0).all() and (out[:8] != 7.0).all()
    want, mag = ref.rotary(_np(x[:8]), ref.positions(off), rot=32)
    _near(out[:8], want, 2.0 ** -24 * (np.abs(want) + 8 * mag))
    empty = G.rotary(G.rotary_spec(32), x[:0], offsets=_int32([0, 0]))
    assert empty.shape == (0, 2, 32)


def test_rotary_places_tokens_of_many_samples():
    """Every token finds its sample among 1, 31, 32, 33, 1000 and 5000 samples, empty ones among them."""
    for B in (1, 31, 32, 33, 1000, 5000):
        r = np.random.default_rng(B)
        n = r.integers(0, 4, B)
        n[0] = 2
        off, offd = _offsets(n)
        x = torch.randn(off[-1], 1, 32, device=DEV)
        y = G.rotary(G.rotary_spec(32), x, offsets=offd)
        want, mag = ref.rotary(_np(x), ref.positions(off), rot=32)
        _near(y, want, 2.0 ** -24 * (np.abs(want) + 8 * mag), B)


def test_rotary_gradient_is_the_transpose():
    """<R x, g> = <x, R^T g> in fp32: the two sums of 64 * 40 * 2 products of O(1) terms differ by their
    elements' errors only, 10 * 2^-24 of the sum of |x||g|-sized terms."""
    g = torch.Generator(device=DEV).manual_seed(3)
    x, dy = (torch.randn(40, 2, 64, generator=g, device=DEV) for _ in range(2))
    off = _int32([0, 15, 40])
    spec = G.rotary_spec(56, interleaved=True, factor=2.0, trained_len=512, mscale=1.1)
    y = G.rotary(spec, x, offsets=off)
    dx = G.rotary(spec, dy, offsets=off, inverse=True)
    a, b = (y.double() * dy.double()).sum(), (x.double() * dx.double()).sum()
    size = 2 * 1.1 * (x.abs().sum(-1) * dy.abs().sum(-1)).double().sum()
    assert abs(a - b) <= 10 * 2.0 ** -24 * size


# ------------------------------------------------------------------------------ cache
def _paged(kv, page, hk, dh, seed, spare=2, width=0, fill=float("nan")):
    """A shuffled page table and caches for samples of kv[b] tokens; rows without a token hold `fill`."""
    r = np.random.default_rng(seed)
    need = [-(-max(k, 0) // page) for k in kv]
    P = sum(need) + spare
    order = r.permutation(P)
    table = np.full((len(kv), max(width, 1, *need)), -1, dtype=np.int32)
    ck = torch.full((P, hk, page, dh), fill, dtype=torch.bfloat16)
    cv = ck.clone()
    g = torch.Generator().manual_seed(seed)
    at = 0
    for b, c in enumerate(need):
        for j in range(c):
            table[b, j] = order[at]
            rows = min(page, kv[b] - j * page)
            for cache in (ck, cv):
                cache[order[at], :, :rows] = torch.randn(hk, rows, dh, generator=g).bfloat16()
            at += 1
    return table, ck, cv


@pytest.mark.parametrize("page", [16, 64, 1024])
@pytest.mark.parametrize("dh,spec", [(64, dict(rot=64)), (128, dict(rot=100, interleaved=True)),
                                     (32, None), (64, dict(rot=18, factor=2.0))])
def test_append(page, dh, spec):
    """Ragged chunks at odd places of the pages, an empty sample, one whose first tokens lie before position 0
    (left padding), rows behind the last sample; everything that is not appended keeps its bits."""
    n, kv, hq, hk = [5, 0, 70, 1, 9], [5, 40, 85, 33, 4], 6, 2
    off, offd = _offsets(n)
    T = off[-1] + 3
    table, ck, cv = _paged(kv, page, hk, dh, 1, fill=3.0)
    g = torch.Generator().manual_seed(2)
    qkv = torch.randn(T, hq + 2 * hk, dh, generator=g).bfloat16()
    d = qkv.to(DEV)
    dk, dv = ck.to(DEV), cv.to(DEV)
    q_out = torch.full((T, hq, dh), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = G.workspace(256, DEV)
    q = G.cache_append(d[:, hq:hq + hk], d[:, hq + hk:], offd, _int32(kv), _int32(table), dk, dv,
                       spec=None if spec is None else G.rotary_spec(**spec), q=d[:, :hq],
                       q_out=q_out, status_ws=ws)
    assert q is q_out and G.workspace_status(ws) == 0
    pos = ref.positions(off, kv)
    T0 = off[-1]

    def turned(x):
        x = _np(x[:T0])
        return ref.rotary(x, pos, **spec) if spec else (x, 0 * x)
    want, mag = turned(qkv[:, :hq])
    _near(q_out[:T0], want, HALF[torch.bfloat16] * np.abs(want) + 8 * 2.0 ** -24 * mag)
    assert (q_out[T0:] == 7.0).all()
    want, mag = turned(qkv[:, hq:hq + hk])
    mine = torch.zeros(ck.shape[0], page, dtype=torch.bool)
    for b in range(len(n)):
        for t in range(off[b], off[b + 1]):
            if pos[t] < 0:
                continue
            pg, row = int(table[b, pos[t] // page]), int(pos[t] % page)
            mine[pg, row] = True
            _near(dk[pg, :, row], want[t],
                  HALF[torch.bfloat16] * np.abs(want[t]) + 8 * 2.0 ** -24 * mag[t])
            assert torch.equal(dv[pg, :, row].cpu(), qkv[t, hq + hk:])
    keep = ~mine[:, None, :, None].expand_as(ck)
    assert torch.equal(dk.cpu()[keep], ck[keep]) and torch.equal(dv.cpu()[keep], cv[keep])


def test_append_reports_bad_pages_and_skips_them():
    table, ck, cv = _paged([20, 20], 16, 1, 32, 5, fill=0.0)
    table[0, 1] = ck.shape[0]                 # past the cache
    _, off = _offsets([20, 21])               # sample 1: position 20 lies in page 1, 32 tokens would not fit
    k = torch.ones(41, 1, 32, dtype=torch.bfloat16, device=DEV)
    dk, dv = torch.zeros_like(ck).to(DEV), torch.zeros_like(cv).to(DEV)
    ws = G.workspace(256, DEV)
    G.cache_append(k, k, off, _int32([20, 21]), _int32(table), dk, dv, status_ws=ws)
    assert G.workspace_status(ws) == 1
    assert int((dv[:, 0, :, 0] == 1).sum()) == 16 + 21
    G.cache_append(k[:20], k[:20], _int32([0, 0, 20]), _int32([20, 40]), _int32(table), dk, dv,
                   status_ws=ws)              # positions 20 .. 39: past the table of two pages
    assert G.workspace_status(ws) == 1
    G.cache_append(k[:20], k[:20], _int32([0, 0, 20]), _int32([20, 20]), _int32(table), dk, dv,
                   status_ws=ws)
    assert G.workspace_status(ws) == 0


# ------------------------------------------------------------------------------ chunk attention
def _chunk_case(n, kv, hq, hk, dh, page, seed, window=None, scale=None, evict=False, pad=0, std=1.5):
    off, offd = _offsets(n)
    table, ck, cv = _paged(kv, page, hk, dh, seed)
    if evict and window:                      # pages behind every window are gone
        for b in range(len(n)):
            for j in range(table.shape[1]):
                if (j + 1) * page <= kv[b] - n[b] - window + 1:
                    table[b, j] = -7
    g = torch.Generator().manual_seed(seed + 1)
    q = std * torch.randn(off[-1] + pad, hq, dh, generator=g).bfloat16()
    scale = dh ** -0.5 if scale is None else scale
    return off, offd, table, ck, cv, q.bfloat16(), scale


def _check_chunk(n, kv, hq, hk, dh, page, seed=0, window=None, scale=None, evict=False, max_n=None,
                 std=1.5):
    off, offd, table, ck, cv, q, scale = _chunk_case(n, kv, hq, hk, dh, page, seed, window, scale,
                                                     evict, std=std)
    max_n = max_n or max(n)
    c = G.Cache(0, 0, 0, *([1] * 6))
    ws = None
    dk, dv, dq, dt = ck.to(DEV), cv.to(DEV), q.to(DEV), _int32(table)
    c = G._cache("t", dk, dv, dt, len(n))
    ws = G.workspace(G.chunk_workspace_bytes(c, len(n), hq, off[-1], max_n), DEV)
    ws.fill_(0x5a)                            # a workspace needs no preparation
    o, lse = G.chunk_fwd(dq, offd, _int32(kv), dt, dk, dv, scale, max_n=max_n, window=window, ws=ws)
    assert G.workspace_status(ws) == 0
    want, wl, mag, size = ref.chunk(_np(q), off, kv, table, ck.float().numpy(), cv.float().numpy(),
                                    scale, window)
    delta = (dh + 4) * 2.0 ** -24 * size + 2.0 ** -21
    tol = 2.0 ** -8 * (mag + np.abs(want)) + 2 * delta.T[:, :, None] * mag
    _near(o, want, tol * 1.001, "o")
    got = lse.double().cpu().numpy()
    none = np.isinf(wl)
    assert np.array_equal(np.isneginf(got), none)
    # the logarithm and the max add two fp32 roundings of the result
    tol = delta + 2.0 ** -22 * (1 + np.abs(np.where(none, 0, wl)))
    assert (np.abs(got[~none] - wl[~none]) <= tol[~none]).all()
    return o, lse


@pytest.mark.parametrize("dh", [32, 64, 128])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("hq,hk", [(4, 4), (8, 2), (3, 1)])
def test_decode(dh, page, hq, hk):
    """One token per sample (some with none), lengths around a page's and a block's end."""
    kv = [1, 16, 17, 63, 64, 65, 300, 5, 128]
    n = [1, 1, 1, 1, 1, 1, 1, 0, 1]
    _check_chunk(n, kv, hq, hk, dh, page, seed=dh + page)


@pytest.mark.parametrize("window", [None, 1, 7, 64, 100])
@pytest.mark.parametrize("page", [16, 32, 128])
def test_ragged_chunks(window, page):
    """Chunks of every length beside each other, at odd starts; tokens without any position; windows that
    begin inside a page, with the pages behind them gone."""
    n = [3, 0, 40, 1, 17, 130, 9]
    kv = [3, 50, 77, 200, 17, 301, 4]
    _check_chunk(n, kv, 4, 2, 64, page, seed=page, window=window, evict=True)


@pytest.mark.parametrize("dh", [32, 64, 128])
@pytest.mark.parametrize("hq,hk,nmax", [(1, 1, 300), (6, 2, 150), (24, 2, 40), (40, 1, 20), (128, 1, 5)])
def test_many_rows(dh, hq, hk, nmax):
    """Head groups from 1 to 128 on a kv head, chunks of many row tiles, fresh and late in a context."""
    n, kv = [nmax, 1, nmax // 2 + 1], [nmax, 130, nmax // 2 + 400]
    _check_chunk(n, kv, hq, hk, dh, 32, seed=hq + nmax)


def test_one_long_context_is_cut_among_all_workers():
    _check_chunk([1], [9000], 2, 1, 64, 64, seed=3)
    _check_chunk([2, 1], [7003, 1], 8, 1, 128, 16, seed=4)
    _check_chunk([150], [4000], 1, 1, 64, 64, seed=5)


def test_bound_above_the_lengths():
    """max_n may exceed every length: few tokens through the kernel for many rows."""
    _check_chunk([1, 3, 2], [70, 3, 500], 4, 2, 64, 16, seed=6, max_n=1000)
    _check_chunk([1, 3, 2], [70, 3, 500], 4, 2, 128, 32, seed=7, max_n=1000, window=50, evict=True)


@pytest.mark.parametrize("n,max_n", [([1, 2], 2), ([200, 3], 200)])
@pytest.mark.parametrize("scale", [0.0, -0.2, 2.0])
def test_scales(scale, n, max_n):
    """A zero, a negative and a large scale (sharp softmax)."""
    _check_chunk(n, [90, 300], 4, 2, 64, 16, seed=9, scale=scale)


@pytest.mark.parametrize("n", [[1, 1], [150, 4]])
def test_tokens_without_positions(n):
    """kv_len 0, and chunks that begin before position 0: those rows are 0 and -inf."""
    o, lse = _check_chunk(n, [0, 3], 4, 2, 64, 16, seed=10)
    assert (o[:n[0]] == 0).all() and torch.isneginf(lse[:, :n[0]]).all()


@pytest.mark.parametrize("n", [[1, 1, 1], [130, 60, 2]])
def test_rows_behind_the_last_sample_and_guards(n):
    off, offd, table, ck, cv, q, scale = _chunk_case(n, [150, 61, 30], 4, 2, 64, 16, 11, pad=5)
    T = q.shape[0]
    big = torch.full((T + 64, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((4, T), 7.0, device=DEV)
    args = (offd, _int32([150, 61, 30]), _int32(table), ck.to(DEV), cv.to(DEV), scale)
    G.chunk_fwd(q.to(DEV), *args, max_n=max(max(n), 3), o=big[32:32 + T], lse=lse)
    assert (big[:32] == 7.0).all() and (big[32 + off[-1]:] == 7.0).all()
    assert (lse[:, off[-1]:] == 7.0).all() and torch.isfinite(big[32:32 + off[-1]]).all()


@pytest.mark.parametrize("max_n", [4, 300])
def test_bad_offsets_lengths_and_pages_are_reported(max_n):
    off, offd, table, ck, cv, q, scale = _chunk_case([2, 3, 4], [40, 50, 60], 4, 2, 64, 16, 12)
    dq, dk, dv = q.to(DEV), ck.to(DEV), cv.to(DEV)
    ws = G.workspace(64 << 20, DEV)

    def status(o=offd, kv=(40, 50, 60), t=table):
        out, _ = G.chunk_fwd(dq, o, _int32(list(kv)), _int32(t), dk, dv, scale, max_n=max_n, ws=ws)
        return G.workspace_status(ws), out
    ok, good = status()
    assert ok == 0
    assert status(o=_int32([0, 2, 1, 9]))[0] == 1
    assert status(o=_int32([0, 2, 5, 90]))[0] == 1
    assert status(kv=(40, 50, 65))[0] == 1 and status(kv=(40, -1, 60))[0] == 1
    bad = table.copy()
    bad[1, 2] = ck.shape[0]
    code, out = status(t=bad)
    assert code == 1 and torch.equal(out[:2], good[:2]) and torch.equal(out[5:], good[5:])
    bad[1, 2] = -1
    assert status(t=bad)[0] == 1
    assert status()[0] == 0


def test_same_bits_again_and_beside_another_call():
    """Two calls on two streams with workspaces of their own give the bits of a call alone."""
    for n, kv, dh in (([1] * 20, list(range(50, 1050, 50)), 128), ([300, 20], [2000, 500], 64),
                      ([130, 0, 7, 301, 64], [900, 5, 7, 1000, 3000], 32),
                      ([33, 700, 1, 90], [500, 700, 2000, 91], 128)):
        off, offd, table, ck, cv, q, scale = _chunk_case(n, kv, 8, 2, dh, 16, 13)
        args = (q.to(DEV), offd, _int32(kv), _int32(table), ck.to(DEV), cv.to(DEV), scale)
        want, wl = G.chunk_fwd(*args, max_n=max(n))
        torch.cuda.synchronize()
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        outs = []
        for _ in range(5):
            outs += [G.chunk_fwd(*args, max_n=max(n), stream=s) for s in (s1, s2)]
        torch.cuda.synchronize()
        for o, lse in outs:
            assert torch.equal(o, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("n", [[1, 1, 1], [40, 3, 100]])
def test_shared_pages_and_no_lse(n):
    """Samples that begin with the same pages (a common prefix), and a call that asks for no LSE."""
    kv = [200, 150, 130]
    off, offd, table, ck, cv, q, scale = _chunk_case(n, kv, 4, 2, 64, 16, 17)
    table[1, :4], table[2, :4] = table[0, :4], table[0, :4]
    args = (q.to(DEV), offd, _int32(kv), _int32(table), ck.to(DEV), cv.to(DEV), scale)
    o, lse = G.chunk_fwd(*args, max_n=max(n), want_lse=False)
    assert lse is None
    want, _, mag, size = ref.chunk(_np(q), off, kv, table, ck.float().numpy(), cv.float().numpy(), scale)
    delta = 68 * 2.0 ** -24 * size + 2.0 ** -21
    _near(o, want, 1.001 * (2.0 ** -8 * (mag + np.abs(want)) + 2 * delta.T[:, :, None] * mag))


def test_cache_offsets_past_32_bits():
    """Pages whose elements lie beyond 2^31 in the cache: written by the append, read by both attention
    kernels; and rows beyond 2^31 elements in a strided rotation."""
    hk, page, dh, P = 8, 128, 128, 16500
    ck, cv = (torch.empty(P, hk, page, dh, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    assert ck.numel() > 2 ** 31
    g = torch.Generator(device=DEV).manual_seed(18)
    for n in (200, 1):
        table = _int32([[P - 1, P - 3]])
        k, v, q = (torch.randn(m, h, dh, generator=g, device=DEV).bfloat16()
                   for m, h in ((200, hk), (200, hk), (n, hk)))
        G.cache_append(k, v, _int32([0, 200]), _int32([200]), table, ck, cv)
        o, _ = G.chunk_fwd(q, _int32([0, n]), _int32([200]), table, ck, cv, 0.1, max_n=n)
        want, _, mag, size = ref.chunk(_np(q), [0, n], [200], np.array([[1, 0]]),
                                       *(torch.cat([torch.nn.functional.pad(x[128:], (0, 0, 0, 0, 0, 56)),
                                                    x[:128]]).view(2, page, hk, dh).transpose(1, 2)
                                         .float().cpu().numpy() for x in (k, v)), 0.1)
        delta = 132 * 2.0 ** -24 * size + 2.0 ** -21
        _near(o, want, 1.001 * (2.0 ** -8 * (mag + np.abs(want)) + 2 * delta.T[:, :, None] * mag))
    del cv
    rows = ck.view(P, hk * page * dh)
    assert (P - 1) * rows.stride(0) > 2 ** 31
    rows[-1, :256] = torch.randn(256, generator=g, device=DEV).bfloat16()
    x = rows[:, :256].unflatten(1, (2, 128))
    y = G.rotary(G.rotary_spec(128), x, positions=torch.arange(P, dtype=torch.int32, device=DEV))
    want, mag = ref.rotary(_np(x[-1:]), np.array([P - 1]), rot=128)
    _near(y[-1:], want, HALF[torch.bfloat16] * np.abs(want) + 8 * 2.0 ** -24 * mag)


def test_calls_on_another_stream():
    """`stream` as a torch stream and as a raw handle: the call and what it allocates belong to that stream."""
    off, offd, table, ck, cv, q, scale = _chunk_case([2, 3], [40, 50], 4, 2, 64, 16, 19)
    args = (q.to(DEV), offd, _int32([40, 50]), _int32(table), ck.to(DEV), cv.to(DEV), scale)
    x, w = torch.randn(30, 96, device=DEV), torch.ones(96, device=DEV)
    want, wl = G.chunk_fwd(*args, max_n=3)
    _, wn = G.block_norm_fwd(x, w_pre=w)
    wr = G.rotary(G.rotary_spec(64), args[0], offsets=offd)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for st in (s, s.cuda_stream):
        o, lse = G.chunk_fwd(*args, max_n=3, stream=st)
        _, n = G.block_norm_fwd(x, w_pre=w, stream=st)
        r = G.rotary(G.rotary_spec(64), args[0], offsets=offd, stream=st)
        s.synchronize()
        assert torch.equal(o, want) and torch.equal(lse, wl) and torch.equal(n, wn) and torch.equal(r, wr)
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    # inputs that are dropped right behind the call live on until the stream has read them
    big = torch.randn(1 << 20, 96, device=DEV)
    want = G.block_norm_fwd(big, w_pre=w)[1]
    copy = big.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
    _, n = G.block_norm_fwd(copy, w_pre=w, stream=s)
    del copy
    torch.zeros(1 << 20, 96, device=DEV)
    s.synchronize()
    assert torch.equal(n, want)


def test_empty_batch():
    table, ck, cv = _paged([10], 16, 1, 64, 14)
    ws = G.workspace(64 << 20, DEV)
    q = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    o, lse = G.chunk_fwd(q, _int32([0, 0]), _int32([10]), _int32(table), ck.to(DEV), cv.to(DEV), 1.0,
                         max_n=0, ws=ws)
    assert o.shape == (0, 2, 64) and G.workspace_status(ws) == 0


def test_window_attention_in_chunks():
    """A history served in chunks gives what the training form gives on the whole history, both within
    their own roundings of the same fp64 result (2^-8 of sum p|v| twice over)."""
    n, h, dh, w = 300, 2, 64, 100
    g = torch.Generator().manual_seed(15)
    q, k, v = (torch.randn(n, h, dh, generator=g).bfloat16().to(DEV) for _ in range(3))
    whole, _ = G.window_fwd(q, _int32([0, n]), k, v, w, 0.125, [0, n])
    table = torch.randperm(19, generator=g).to(torch.int32)[None].to(DEV)
    ck, cv = (torch.full((19, h, 16, dh), float("nan"), dtype=torch.bfloat16, device=DEV)
              for _ in range(2))
    at, outs = 0, []
    for step in (1, 1, 7, 129, 1, 100, 61):
        off, kv = _int32([0, step]), _int32([at + step])
        G.cache_append(k[at:at + step], v[at:at + step], off, kv, table, ck, cv)
        o, _ = G.chunk_fwd(q[at:at + step], off, kv, table, ck, cv, 0.125, max_n=step, window=w)
        outs.append(o)
        at += step
    assert at == n
    _, _, mag, _ = ref.chunk(_np(q), [0, n], [n], table.cpu().numpy(), ck.float().cpu().numpy(),
                             cv.float().cpu().numpy(), 0.125, w)
    got = torch.cat(outs)
    _near(got, _np(whole), 2 * 2.0 ** -8 * (mag + np.abs(_np(whole))) + 1e-4)


# ------------------------------------------------------------------------------ block norm
def _norm_case(T, d, dtype, gate, post, pre, seed, B=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)                # noqa: E731
    t = dict(x=(std * rnd(T, d)).to(dtype), f=(std * rnd(T, d)).to(dtype),
             gate=None if gate is None else rnd(B if gate == "sample" else T, d).to(dtype),
             w_post=1 + 0.3 * rnd(d) if post else None, w_pre=1 + 0.3 * rnd(d) if pre else None)
    return t, rnd


def _dev(t):
    return None if t is None else t.to(DEV)


def _dbl(t):
    return None if t is None else t.double()


def _check_norm(n, d, dtype, gate="token", post=True, pre=True, sigmoid=True, alpha=0.7, seed=0,
                pad=0, std=1.0):
    off, offd = _offsets(n)
    T, B = off[-1], len(n)
    t, rnd = _norm_case(T + pad, d, dtype, gate, post, pre, seed, B, std)
    sample = torch.repeat_interleave(torch.arange(B), torch.tensor(n)) if gate == "sample" else None
    kw = dict(alpha=alpha, eps=1e-5, sigmoid=sigmoid)
    offs = offd if gate == "sample" else None
    dev = {k: _dev(v) for k, v in t.items()}
    y0 = torch.full((T + pad, d), 7.0, dtype=dtype, device=DEV)
    n0 = y0.clone() if pre else None
    y, nn = G.block_norm_fwd(**dev, offsets=offs, y=y0, n=n0, **kw)
    cut = {k: _dbl(v if k in ("w_post", "w_pre") or (k == "gate" and sample is not None) else
                   None if v is None else v[:T]) for k, v in t.items()}
    wy, wn = ref.block_norm(**cut, sample=sample, **kw)
    terms = cut["x"].abs() + (wy - cut["x"]).abs()
    _near(y[:T], wy.numpy(), (HALF[dtype] * wy.abs() + 2.0 ** -18 * terms).numpy(), "y")
    if pre:
        r = 1 / torch.sqrt((wy * wy).mean(-1, keepdim=True) + 1e-5)
        _near(nn[:T], wn.numpy(), (HALF[dtype] * wn.abs() + 2.0 ** -17 * (wn.abs() + (
            cut["w_pre"].abs() * r) * terms)).numpy(), "n")
    if pad:
        assert (y[T:] == 7.0).all() and (nn is None or (nn[T:] == 7.0).all())

    # backward, for the y that a training step keeps
    yk = wy.to(dtype)
    if pad:
        yk = torch.cat([yk, torch.full((pad, d), 5.0, dtype=dtype)])
    dy, dn = rnd(T + pad, d).to(dtype), rnd(T + pad, d).to(dtype) if pre else None
    outs = {k: torch.full((T + pad, d), 7.0, dtype=dtype, device=DEV) for k in ("dx", "df")}
    got = G.block_norm_bwd(yk.to(DEV), dev["f"], dev["gate"], dev["w_post"], dev["w_pre"], _dev(dy),
                           _dev(dn), offsets=offs, **outs, **kw)
    want = ref.block_norm_grads(yk[:T].double(), cut["f"], cut["gate"], cut["w_post"], cut["w_pre"],
                                dy[:T].double(), None if dn is None else dn[:T].double(),
                                sample=sample, B=B, **kw)
    for name, out in zip(("dx", "df", "dgate", "dw_post", "dw_pre"), got):
        if name not in want:
            assert out is None
            continue
        v, mag = want[name]
        half = HALF[out.dtype]
        extra = 2.0 ** -16 if name in ("df", "dgate", "dw_post") else 2.0 ** -17
        if name in ("dw_post", "dw_pre") or (name == "dgate" and sample is not None):
            extra += 2.0 ** -24 * (T + 300)
        if pad and name in ("dx", "df") or (pad and name == "dgate" and sample is None):
            if name != "dgate":
                assert (out[T:] == 7.0).all()
            out = out[:T]
        _near(out, v.numpy(), (half * v.abs() + extra * mag).numpy(), name)
    return got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [1, 7, 8, 64, 100, 256, 1000, 1001, 1024, 2048, 5000, 8190, 8192])
def test_norm_widths(d, dtype):
    _check_norm([5, 0, 30], d, dtype, seed=d)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate", [None, "token", "sample"])
@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False), (False, False)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_norm_forms(gate, post, pre, sigmoid, dtype):
    _check_norm([1, 0, 4, 20, 0, 3], 96, dtype, gate, post, pre, sigmoid, seed=2)


@pytest.mark.parametrize("n", [[1], [3000], [0, 0, 2500, 1, 0], [700] * 9, [1] * 1500, [5000, 3, 5000]])
@pytest.mark.parametrize("d", [40, 136, 1024])
def test_norm_shared_gates(n, d):
    """A sample's gate gradient sums rows of one group, of many groups, and of none; rows behind the last sample
    take no part."""
    _check_norm(n, d, torch.bfloat16, "sample", seed=len(n) + d, pad=6)


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 256), (torch.bfloat16, 776), (torch.bfloat16, 1024),
                                     (torch.bfloat16, 2056), (torch.bfloat16, 5000), (torch.bfloat16, 8192),
                                     (torch.float32, 128), (torch.float32, 1000), (torch.float32, 1540),
                                     (torch.float32, 4096), (torch.bfloat16, 257), (torch.bfloat16, 1001),
                                     (torch.bfloat16, 2053), (torch.float32, 130), (torch.float32, 1001),
                                     (torch.float32, 2047)])
@pytest.mark.parametrize("gate,post,pre", [("token", True, True), ("sample", True, True), (None, False, True),
                                           ("sample", False, False), (None, True, False)])
def test_norm_streamed_rows(dtype, d, gate, post, pre):
    """Enough rows for every group of warps to walk a range: rows of one to sixteen warps, whole and cut last
    segments, rows that start anywhere, samples that span several groups, rows behind the last sample."""
    _check_norm([2000, 0, 1, 2900], d, dtype, gate, post, pre, seed=d, pad=7 if gate == "sample" else 0)


@pytest.mark.parametrize("n,d,dtype", [([9000, 0, 3], 7, torch.bfloat16), ([4500, 4501], 64, torch.bfloat16),
                                       ([9001], 100, torch.float32), ([300, 0, 400], 4100, torch.float32),
                                       ([300, 0, 400], 8191, torch.float32)])
@pytest.mark.parametrize("gate", ["token", "sample"])
def test_norm_rows_in_registers(n, d, dtype, gate):
    """Many narrow rows and very wide ones, several to a group of threads."""
    _check_norm(n, d, dtype, gate, seed=d, pad=3 if gate == "sample" else 0)


@pytest.mark.parametrize("std", [0.0, 1e-6, 1e6])
def test_norm_scales(std):
    """Rows of zeros (the root holds eps alone), tiny and huge rows."""
    _check_norm([6, 5], 72, torch.float32, std=std, seed=4)


@pytest.mark.parametrize("T,d", [(40, 72), (40, 71), (5000, 520), (5000, 519)])
@pytest.mark.parametrize("gate", ["token", "sample"])
def test_norm_saturated_gates(T, d, gate):
    """Gates from -12 to 12: the slope act (1 - act) keeps its relative precision on both sides."""
    t, rnd = _norm_case(T, d, torch.float32, gate, True, False, 9, B=2)
    t["gate"] = torch.linspace(-12, 12, t["gate"].numel()).view_as(t["gate"])
    dy = rnd(T, d)
    off, sample = (None, None) if gate == "token" else (_int32([0, 7, T]), (torch.arange(T) >= 7).long())
    got = G.block_norm_bwd(t["x"].to(DEV), t["f"].to(DEV), t["gate"].to(DEV), t["w_post"].to(DEV), None,
                           dy.to(DEV), offsets=off, sigmoid=True)[2]
    v, mag = ref.block_norm_grads(_dbl(t["x"]), _dbl(t["f"]), _dbl(t["gate"]), _dbl(t["w_post"]), None, _dbl(dy),
                                  None, sample=sample, B=2, sigmoid=True)["dgate"]
    extra = 2.0 ** -16 + (2.0 ** -24 * (T + 300) if sample is not None else 0)
    _near(got, v.numpy(), (HALF[torch.float32] * v.abs() + extra * mag).numpy())


def test_norm_without_a_block():
    t, rnd = _norm_case(33, 200, torch.bfloat16, None, False, True, 5)
    x, w = t["x"].to(DEV), t["w_pre"].to(DEV)
    same, n = G.block_norm_fwd(x, w_pre=w)
    assert same is x
    _, want = ref.block_norm(t["x"].double(), w_pre=t["w_pre"].double())
    _near(n, want.numpy(), ((HALF[torch.bfloat16] + 2.0 ** -18) * want.abs()).numpy())
    dn = rnd(33, 200).bfloat16()
    dx, df, dg, dq, dw = G.block_norm_bwd(x, w_pre=w, dn=dn.to(DEV))
    assert df is None and dg is None and dq is None
    want = ref.block_norm_grads(t["x"].double(), None, None, None, t["w_pre"].double(), None,
                                dn.double())
    for got, key in ((dx, "dx"), (dw, "dw_pre")):
        v, mag = want[key]
        _near(got, v.numpy(), (HALF[got.dtype] * v.abs() + 2.0 ** -17 * mag).numpy(), key)


def test_norm_in_place_and_empty():
    t, _ = _norm_case(50, 128, torch.float32, "token", True, True, 6)
    dev = {k: _dev(v) for k, v in t.items()}
    y, n = G.block_norm_fwd(**dev)
    x2 = dev["x"].clone()
    y2, n2 = G.block_norm_fwd(**{**dev, "x": x2}, y=x2)
    assert y2 is x2 and torch.equal(y, y2) and torch.equal(n, n2)
    z = torch.empty(0, 128, device=DEV)
    _, _, dg, dq, dw = G.block_norm_bwd(z, z, torch.ones(2, 128, device=DEV), dev["w_post"],
                                        dev["w_pre"], z, z, offsets=_int32([0, 0, 0]))
    assert (dg == 0).all() and (dq == 0).all() and (dw == 0).all()


def test_norm_gradient_against_differences():
    """The kernel's forward in fp32, moved by +-h along a direction of all inputs: the difference of the loss
    (summed in fp64) is off by h^2 and by the outputs' 2^-18 / h, against the kernel's gradients."""
    T, d = 12, 64
    t, rnd = _norm_case(T, d, torch.float32, "token", True, True, 7)
    dy, dn = rnd(T, d), rnd(T, d)
    way = {k: rnd(*v.shape) for k, v in t.items()}
    kw = dict(alpha=0.7, sigmoid=True)

    def loss(s):
        y, n = G.block_norm_fwd(**{k: (v + s * way[k]).to(DEV) for k, v in t.items()}, **kw)
        return float((_dbl(y.cpu()) * dy).sum() + (_dbl(n.cpu()) * dn).sum())
    h = 2.0 ** -7
    slope = (loss(h) - loss(-h)) / (2 * h)
    y, _ = G.block_norm_fwd(**{k: v.to(DEV) for k, v in t.items()}, **kw)
    dx, df, dg, dq, dw = G.block_norm_bwd(y, t["f"].to(DEV), t["gate"].to(DEV), t["w_post"].to(DEV),
                                          t["w_pre"].to(DEV), dy.to(DEV), dn.to(DEV), **kw)
    want = sum(float((_dbl(g.cpu()) * way[k]).sum())
               for g, k in zip((dx, df, dg, dq, dw), ("x", "f", "gate", "w_post", "w_pre")))
    size = sum(float((_dbl(g.cpu()).abs() * way[k].abs()).sum())
               for g, k in zip((dx, df, dg, dq, dw), ("x", "f", "gate", "w_post", "w_pre")))
    assert abs(slope - want) <= size * (8 * h * h)


def test_norm_same_bits_again():
    t, rnd = _norm_case(3001, 512, torch.bfloat16, "sample", True, True, 8, B=3)
    dev = {k: _dev(v) for k, v in t.items()}
    off, dy, dn = _int32([0, 1500, 1500, 3001]), *(rnd(3001, 512).bfloat16().to(DEV) for _ in "ab")
    runs = [G.block_norm_bwd(dev["x"], dev["f"], dev["gate"], dev["w_post"], dev["w_pre"], dy, dn,
                             offsets=off) for _ in range(3)]
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


# ------------------------------------------------------------------------------ together
def _served_layer(x, f_w, o_w, norms, spec, state, off, kv, max_n, h, hk, dh, w):
    """One layer of a serving step: norm, projection, append, attention, projection, gated residual."""
    _, n = G.block_norm_fwd(x, w_pre=norms["pre"])
    qkv = (n.float() @ f_w).bfloat16().view(-1, h + 2 * hk, dh)
    q = G.cache_append(qkv[:, h:h + hk], qkv[:, h + hk:], off, kv, state["table"], state["k"],
                       state["v"], spec=spec, q=qkv[:, :h])
    o, _ = G.chunk_fwd(q, off, kv, state["table"], state["k"], state["v"], dh ** -0.5, max_n=max_n,
                       window=w)
    f = (o.flatten(1).float() @ o_w).bfloat16()
    return G.block_norm_fwd(x, f, gate=norms["gate"], offsets=off, w_post=norms["post"],
                            w_pre=norms["next"], sigmoid=True)


def _layer(seed=21, h=4, hk=2, dh=64, B=3, page=16, pages=40):
    g = torch.Generator(device=DEV).manual_seed(seed)
    d = h * dh
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)    # noqa: E731
    f_w, o_w = rnd(d, (h + 2 * hk) * dh) / d ** 0.5, rnd(d, d) / d ** 0.5
    norms = dict(pre=1 + 0.1 * rnd(d), post=1 + 0.1 * rnd(d), next=1 + 0.1 * rnd(d),
                 gate=rnd(B, d).bfloat16())
    state = dict(table=torch.randperm(pages, generator=g, device=DEV).to(torch.int32)[:B * 10].view(B, 10)
                 .contiguous(), k=rnd(pages, hk, page, dh).bfloat16(), v=rnd(pages, hk, page, dh).bfloat16())
    return f_w, o_w, norms, state, rnd, d


def test_a_served_layer_step_by_step_equals_one_chunk():
    """A history of three users through the layer in one chunk, and token by token: the same rows up to the
    roundings of bf16 activations (each path rounds q, k, v, o and f at 2^-8; a few of them add up)."""
    f_w, o_w, norms, state, rnd, d = _layer()
    n, spec, w = [12, 5, 9], G.rotary_spec(32, interleaved=True), 6
    off, offd = _offsets(n)
    x = rnd(off[-1], d).bfloat16()
    kw = dict(h=4, hk=2, dh=64, w=w)
    y1, n1 = _served_layer(x, f_w, o_w, norms, spec, state, offd, _int32(n), max(n), **kw)
    state2 = {k: v.clone() for k, v in state.items()}
    y2, n2 = torch.zeros_like(y1), torch.zeros_like(n1)
    for i in range(max(n)):
        step = [1 if i < c else 0 for c in n]
        rows = [off[b] + i for b in range(3) if i < n[b]]
        o2, od2 = _offsets(step)
        kv = [min(i + 1, c) for c in n]
        y, nn = _served_layer(x[rows].contiguous(), f_w, o_w, norms, spec, state2, od2, _int32(kv), 1, **kw)
        y2[rows], n2[rows] = y, nn
    for a, b in ((y1, y2), (n1, n2)):
        err = (a.float() - b.float()).norm() / b.float().norm()
        assert err <= 8 * 2.0 ** -8, float(err)


def test_a_served_step_captured_and_replayed():
    """The step in a CUDA graph: replays with other inputs in the same buffers give what eager calls give."""
    f_w, o_w, norms, state, rnd, d = _layer(seed=22)
    spec, off = G.rotary_spec(64), _int32([0, 1, 2, 3])
    x, kv = rnd(3, d).bfloat16(), _int32([5, 1, 100])
    kw = dict(h=4, hk=2, dh=64, w=50)
    keep = {k: v.clone() for k, v in state.items()}

    def step():
        return _served_layer(x, f_w, o_w, norms, spec, state, off, kv, 1, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph, graph2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, n = step()
    with torch.cuda.graph(graph2):
        y2, n2 = step()
    for k in state:
        state[k].copy_(keep[k])
    for lens in ([5, 1, 100], [6, 2, 101], [150, 33, 16]):
        x.copy_(rnd(3, d).bfloat16())
        kv.copy_(_int32(lens))
        before = {k: v.clone() for k, v in state.items()}
        graph.replay()
        graph2.replay()
        torch.cuda.synchronize()
        for k in state:
            state[k].copy_(before[k])
        ey, en = step()
        torch.cuda.synchronize()
        assert torch.equal(y, ey) and torch.equal(n, en) and torch.equal(y2, ey) and torch.equal(n2, en)


@pytest.mark.parametrize("d", [96, 512])
def test_training_operators_captured_and_replayed(d):
    """Rotary and its gradient, block norm and its gradient in two graphs that are replayed in turn with
    other inputs and other offsets in the same buffers: the bits of eager calls."""
    B, T, spec = 4, 300, G.rotary_spec(32, base=1e4)
    dev = {k: _dev(v) for k, v in _norm_case(T, d, torch.bfloat16, "sample", True, True, 31, B=B)[0].items()}
    off = _int32([0, 100, 100, 170, 300])
    gen = torch.Generator(device=DEV).manual_seed(32)

    def fill():
        for k in ("x", "f", "gate"):
            dev[k].normal_(generator=gen)
    dn = torch.randn(T, d, device=DEV, generator=gen).bfloat16()

    def step():
        x = G.rotary(spec, dev["x"].view(T, d // 32, 32), offsets=off).view(T, d)
        y, n = G.block_norm_fwd(x, dev["f"], dev["gate"], dev["w_post"], dev["w_pre"], off, sigmoid=True)
        g = G.block_norm_bwd(y, dev["f"], dev["gate"], dev["w_post"], dev["w_pre"], n, dn, off, sigmoid=True)
        back = G.rotary(spec, g[0].view(T, d // 32, 32), offsets=off, inverse=True)
        return (x, y, n, back, *g)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    outs = []
    for graph in graphs:
        with torch.cuda.graph(graph):
            outs.append(step())
    for places in ([0, 100, 100, 170, 300], [0, 0, 1, 299, 300], [0, 300, 300, 300, 300]):
        fill()
        off.copy_(_int32(places))
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        for out in outs:
            assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_a_training_layer_and_its_gradient():
    """norm -> rotary -> window attention -> gated residual and back: the gradient of the residual stream
    against fp64 autograd of the same layer (dense causal window), within the bf16 activations' roundings."""
    g = torch.Generator().manual_seed(23)
    n, h, dh, w = [40, 0, 23], 2, 64, 16
    off, offd = _offsets(n)
    T, d = off[-1], h * dh
    x, dy = (torch.randn(T, d, generator=g).bfloat16() for _ in range(2))
    gate = torch.randn(T, d, generator=g).bfloat16()
    w_pre, w_post = (1 + 0.1 * torch.randn(d, generator=g) for _ in range(2))
    spec, sd = G.rotary_spec(64), dict(rot=64)
    scale = dh ** -0.5
    xd, gd, pre, post = x.to(DEV), gate.to(DEV), w_pre.to(DEV), w_post.to(DEV)
    _, nn = G.block_norm_fwd(xd, w_pre=pre)
    v = nn.view(T, h, dh)
    qk = G.rotary(spec, v, offsets=offd)
    o, lse = G.window_fwd(qk, offd, qk, v, w, scale, off)
    y, _ = G.block_norm_fwd(xd, o.view(T, d), gate=gd, w_post=post, sigmoid=True)
    dx, df, _, _, _ = G.block_norm_bwd(y, o.view(T, d), gd, post, None, dy.to(DEV), sigmoid=True)
    dq, dk, dv = G.window_bwd(qk, offd, qk, v, o, lse, df.view(T, h, dh), w, scale, off)
    dn = dv.float() + G.rotary(spec, dq, offsets=offd, inverse=True).float() + \
        G.rotary(spec, dk, offsets=offd, inverse=True).float()
    got, _, _, _, _ = G.block_norm_bwd(xd, w_pre=pre, dy=dx, dn=dn.view(T, d).bfloat16())

    lx = x.double().requires_grad_()
    _, rn = ref.block_norm(lx, w_pre=w_pre.double())
    rv = rn.view(T, h, dh)
    pos = ref.positions(off)
    t = torch.tensor(pos, dtype=torch.float64)[:, None] * torch.tensor(
        ref.frequencies(64, 10000.0, 1.0, 0, 1.0, 32.0))
    c, s = t.cos()[:, None], t.sin()[:, None]
    a, b = rv[..., :32], rv[..., 32:]
    rq = torch.cat([a * c - b * s, a * s + b * c], -1)
    sample = torch.repeat_interleave(torch.arange(len(n)), torch.tensor(n))
    tt = torch.arange(T)
    see = (sample[:, None] == sample) & (tt[:, None] >= tt) & (tt[:, None] - tt < w)
    logits = torch.einsum("thd,shd->hts", rq, rq) * scale
    p = torch.softmax(logits.masked_fill(~see, -float("inf")), -1)
    ro = torch.einsum("hts,shd->thd", p, rv).reshape(T, d)
    ry, _ = ref.block_norm(lx, ro, gate.double(), w_post.double(), sigmoid=True)
    want, = torch.autograd.grad((ry * dy.double()).sum(), lx)
    assert (y.cpu().double() - ry.detach()).norm() / ry.norm() <= 8 * 2.0 ** -8
    assert (got.cpu().double() - want).norm() / want.norm() <= 8 * 2.0 ** -8
