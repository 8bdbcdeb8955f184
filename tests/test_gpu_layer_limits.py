"""The attention layer's operators at the edges of their calls, on the GPU: rows of a tile that no token
owns, padded batches, waits that run out, whole numbers beyond 32 bits,
values that are not finite.  Helpers: test_gpu_layer."""
import ctypes

import numpy as np
import pytest
import torch

from recsys_context_personalised_b200 import gdpa as G
from test_gpu_layer import DEV, _chunk_case, _int32, _norm_case

pytestmark = pytest.mark.gpu


def _fill_tiles(dh, heads, size):
    """Leaves queries of that size in every row of the tiles of the kernel for few rows: `heads` on one kv head
    fill a tile, and 8 x 6000 positions give every worker some of them."""
    n, kv = [1] * 8, [6000] * 8
    _, off, table, ck, cv, q, scale = _chunk_case(n, kv, heads * 2, 2, dh, 64, 41)
    G.chunk_fwd(size * torch.ones_like(q).to(DEV), off, _int32(kv), _int32(table), ck.to(DEV), cv.to(DEV), scale,
                max_n=1)


# (heads on a kv head, new tokens, dh, heads that fill the tile): 16 and 32 rows that the heads do not divide
@pytest.mark.parametrize("group,n,dh,full", [(3, [1] * 4, 64, 16), (5, [2, 0, 3, 1], 64, 16),
                                             (12, [1] * 4, 128, 16), (3, [5, 4, 1], 128, 16),
                                             (7, [2, 1], 32, 16), (7, [4, 3, 2], 64, 32), (19, [1] * 3, 32, 32),
                                             (16, [1] * 4, 64, 16)])
def test_rows_that_no_token_owns_change_no_bits(group, n, dh, full):
    """What an earlier call left in the rest of a tile takes no part: the same call behind one with queries of
    zero and behind one with large queries gives the same bits."""
    kv = [3000, 700, 1500, 4000][:len(n)]
    _, off, table, ck, cv, q, scale = _chunk_case(n, kv, group * 2, 2, dh, 64, 42)
    args = (q.to(DEV), off, _int32(kv), _int32(table), ck.to(DEV), cv.to(DEV), scale)
    outs = []
    for size in (0.0, 40.0, -40.0):
        _fill_tiles(dh, full, size)
        outs.append(G.chunk_fwd(*args, max_n=max(n)))
    for o, lse in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(lse, outs[0][1])


@pytest.mark.parametrize("group,n,dh", [(1, [1, 1, 1], 64), (4, [1, 3, 1], 128), (2, [3, 8, 1], 32),
                                        (8, [1, 4, 2], 64), (1, [140, 3, 200], 64)])
def test_a_sample_keeps_its_bits_beside_other_neighbours(group, n, dh):
    """Queries of the samples behind it, whose rows are loaded with a sample's last tile, take no part in its
    results."""
    kv = [3000, 2000, 2500]
    off, offd, table, ck, cv, q, scale = _chunk_case(n, kv, group * 2, 2, dh, 64, 43)
    args = (offd, _int32(kv), _int32(table), ck.to(DEV), cv.to(DEV), scale)
    want, wl = G.chunk_fwd(q.to(DEV), *args, max_n=max(n))
    for keep in (1, 2):                       # the samples before `keep` stay, the others' queries grow
        loud = q.clone()
        loud[off[keep]:] *= 40
        o, lse = G.chunk_fwd(loud.to(DEV), *args, max_n=max(n))
        assert torch.equal(o[:off[keep]], want[:off[keep]]) and torch.equal(lse[:, :off[keep]], wl[:, :off[keep]])


def _padded_call(off, kv, table, ck, cv, q, scale, max_n, hq):
    """chunk_fwd into outputs full of 7: (o, lse, status)."""
    T, dh = q.shape[0], q.shape[2]
    args = (_int32(off), _int32(kv), _int32(table), ck.to(DEV), cv.to(DEV))
    o = torch.full((T, hq, dh), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((hq, T), 7.0, device=DEV)
    c = G._cache("t", args[3], args[4], args[2], len(kv))
    ws = G.workspace(G.chunk_workspace_bytes(c, len(kv), hq, T, max_n), DEV)
    G.chunk_fwd(q.to(DEV), *args, scale, max_n=max_n, o=o, lse=lse, ws=ws)
    return o, lse, G.workspace_status(ws)


@pytest.mark.parametrize("dh,hq,hk", [(64, 4, 2), (128, 8, 1), (32, 40, 1)])
@pytest.mark.parametrize("n", [[1, 1, 1], [0, 1, 0], [2, 0, 3]])
@pytest.mark.parametrize("before,behind", [(0, 61), (5, 0), (3, 200)])
def test_a_padded_batch(n, dh, hq, hk, before, behind):
    """Few tokens in many rows, with the true bound of the lengths: the bits of the call without the padding,
    whose rows stay as they were."""
    kv = [300, 61, 1200]
    off, _, table, ck, cv, q, scale = _chunk_case(n, kv, hq, hk, dh, 16, 44)
    want, wl, _ = _padded_call(off, kv, table, ck, cv, q, scale, max(n), hq)
    T = off[-1]
    pads = [torch.full((m, hq, dh), float("nan"), dtype=q.dtype) for m in (before, behind)]
    wide = torch.cat([pads[0], q, pads[1]])
    o, lse, status = _padded_call([before + x for x in off], kv, table, ck, cv, wide, scale, max(n), hq)
    assert status == 0
    mine = slice(before, before + T)
    assert torch.equal(o[mine], want) and torch.equal(lse[:, mine], wl)
    o[mine], lse[:, mine] = 7.0, 7.0
    assert (o == 7.0).all() and (lse == 7.0).all()


@pytest.mark.parametrize("hq", [1, 20, 128])
def test_a_batch_of_padding_alone(hq):
    """No sample has a token and max_n says so: nothing is written; a sample with a token is then reported."""
    off, _, table, ck, cv, q, scale = _chunk_case([0, 0], [40, 0], hq, 1, 64, 16, 45, pad=9)
    o, lse, status = _padded_call(off, [40, 0], table, ck, cv, q, scale, 0, hq)
    assert status == 0 and (o == 7.0).all() and (lse == 7.0).all()
    o, lse, status = _padded_call([0, 1, 1], [40, 0], table, ck, cv, q, scale, 0, hq)
    assert status == 1 and (o == 7.0).all() and (lse == 7.0).all()


# ------------------------------------------------------------------------------ waits of the streamed norm
def _lose(row, us=3000):
    fn = G.load().gdpa_selftest_norm_wait
    fn.argtypes, fn.restype = [ctypes.c_int64, ctypes.c_uint32], ctypes.c_int
    assert fn(row, us) == 0


def _right_or_nan(got, want, what):
    """Every element is the healthy call's or NaN; returns where it is NaN."""
    nan = torch.isnan(got)
    assert torch.equal(got[~nan], want[~nan]), what
    return nan


NORM_WAITS = [(torch.bfloat16, 200, "token", True, True), (torch.bfloat16, 2048, "sample", True, True),
              (torch.float32, 1001, "token", True, True), (torch.bfloat16, 1001, "sample", True, False),
              (torch.bfloat16, 8192, None, True, True), (torch.float32, 1024, None, False, True),
              (torch.bfloat16, 5000, "token", True, False), (torch.bfloat16, 512, "token", False, False)]


@pytest.mark.parametrize("dtype,d,gate,post,pre", NORM_WAITS)
@pytest.mark.parametrize("T,row", [(1500, 0), (1500, 777), (3, 2)])
def test_a_row_that_never_arrives(T, row, dtype, d, gate, post, pre):
    """A wait that runs out ends the call with NaN in the row and no wrong number anywhere, the backward with a
    status; the next call is whole."""
    t, rnd = _norm_case(T, d, dtype, gate, post, pre, 46, B=2)
    dev = {k: None if v is None else v.to(DEV) for k, v in t.items()}
    kw = dict(offsets=_int32([0, T // 2, T]) if gate == "sample" else None, sigmoid=True)

    def forward():
        return G.block_norm_fwd(**dev, **kw)
    y, n = forward()
    _lose(row)
    by, bn = forward()
    nan = _right_or_nan(by, y, "y")
    first = int(nan.any(1).nonzero()[0])      # the row that did not arrive, the first of those around `row`
    assert first <= row and nan[first, 0] and (nan[first].all() or not post)
    assert nan[row, 0] and (nan[row].all() or not post)
    if pre:
        assert _right_or_nan(bn, n, "n")[row].all()
    assert all(a is None or torch.equal(a, b) for a, b in zip(forward(), (y, n)))

    dy, dn = rnd(T, d).to(dtype).to(DEV), rnd(T, d).to(dtype).to(DEV) if pre else None
    ws = G.workspace(64 << 20, DEV)
    ws.fill_(0x5a)

    def backward():
        return G.block_norm_bwd(y, dev["f"], dev["gate"], dev["w_post"], dev["w_pre"], dy, dn, ws=ws, **kw)
    want = backward()
    assert G.workspace_status(ws) == 0
    _lose(row)
    got = backward()
    assert G.workspace_status(ws) == 4
    for name, a, b in zip(("dx", "df", "dgate", "dw_post", "dw_pre"), got, want):
        if a is None:
            continue
        nan = _right_or_nan(a, b, name)
        if name in ("dx", "df"):
            assert nan[row, 0] and (nan[row].all() or not (post if name == "df" else pre)), name
        elif name.startswith("dw"):
            assert nan[0], name
    again = backward()
    assert G.workspace_status(ws) == 0
    assert all(a is None or torch.equal(a, b) for a, b in zip(again, want))


@pytest.mark.parametrize("T,d,dtype", [(0, 64, torch.float32), (9000, 64, torch.bfloat16), (40, 5000, torch.float32),
                                       (40, 512, torch.bfloat16)])
@pytest.mark.parametrize("post,pre", [(True, True), (False, False)])
def test_the_norms_status_word(T, d, dtype, post, pre):
    """Set by every form: no rows, rows in registers, streamed rows; with gradients to join and without."""
    t, rnd = _norm_case(T, d, dtype, "token", post, pre, 47)
    dev = {k: None if v is None else v.to(DEV) for k, v in t.items()}
    dy = rnd(T, d).to(dtype).to(DEV)
    ws = G.workspace(64 << 20, DEV)
    ws.fill_(0x5a)
    G.block_norm_bwd(dev["x"], dev["f"], dev["gate"], dev["w_post"], dev["w_pre"], dy, dy if pre else None, ws=ws)
    assert G.workspace_status(ws) == 0


# ------------------------------------------------------------------------------ whole numbers beyond 32 bits
@pytest.mark.parametrize("n", [[1, 2], [140, 3]])
def test_windows_and_bounds_beyond_32_bits(n):
    """A window as long as any history is plain causal attention, whatever its lower 32 bits are; numpy's whole
    numbers are taken like Python's."""
    kv = [300, 150]
    off, offd, table, ck, cv, q, scale = _chunk_case(n, kv, 4, 2, 64, 16, 48)
    args = (q.to(DEV), offd, _int32(kv), _int32(table), ck.to(DEV), cv.to(DEV), scale)
    want, wl = G.chunk_fwd(*args, max_n=max(n))
    for window in (2**31 - 1, 2**31, 2**32, 2**32 + 5, 2**63 - 1):
        o, lse = G.chunk_fwd(*args, max_n=max(n), window=window)
        assert torch.equal(o, want) and torch.equal(lse, wl), window
    for window in (0, -1, -2**32 + 5):
        with pytest.raises(G.GdpaError):
            G.chunk_fwd(*args, max_n=max(n), window=window)
    for max_n in (-1, 2**32 + max(n)):
        with pytest.raises(G.GdpaError):
            G.chunk_fwd(*args, max_n=max_n)
    o, _ = G.chunk_fwd(*args, max_n=np.int64(max(n)), window=np.int32(7))
    assert torch.equal(o, G.chunk_fwd(*args, max_n=max(n), window=7)[0])


# ------------------------------------------------------------------------------ values that are not finite
@pytest.mark.parametrize("hq,hk,dh", [(2, 2, 64), (6, 2, 128), (40, 2, 32)])
@pytest.mark.parametrize("n,at", [([4, 1], 2), ([200, 3], 130)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_values_that_are_not_finite(hq, hk, dh, n, at, value):
    """In the key row of a new token they reach the tokens that see it and no other; in its value row they may
    reach the sample's other tokens (0 times infinity), and no other sample or kv head."""
    kv = [n[0] + 300, 150]
    off, offd, table, ck, cv, q, scale = _chunk_case(n, kv, hq, hk, dh, 16, 49)
    pos, group = kv[0] - n[0] + at, hq // hk
    place = (int(table[0, pos // 16]), 0, pos % 16)

    def call(k, v):
        return G.chunk_fwd(q.to(DEV), offd, _int32(kv), _int32(table), k.to(DEV), v.to(DEV), scale, max_n=max(n))
    want, wl = call(ck, cv)
    bad = ck.clone()
    bad[place] = value
    o, lse = call(bad, cv)
    mine = torch.zeros(off[-1], hq, dtype=torch.bool, device=DEV)
    mine[at:n[0], :group] = True              # what sees the row
    assert torch.equal(o[~mine], want[~mine]) and torch.equal(lse.T[~mine], wl.T[~mine])
    if value != value:
        assert not torch.isfinite(o[mine]).any()
    bad = cv.clone()
    bad[place] = value
    o, lse = call(ck, bad)
    assert not torch.isfinite(o[mine]).any()
    mine[:n[0], :group] = True                # the sample's tokens with the heads of the kv head
    assert torch.equal(o[~mine], want[~mine]) and torch.equal(lse, wl)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("d", [64, 1001, 4096])
def test_a_norm_keeps_a_row_that_is_not_finite_to_itself(d, value):
    """Other rows' results and their gate's gradient keep their bits."""
    t, rnd = _norm_case(600, d, torch.float32, "token", True, True, 50)
    dy, dn = rnd(600, d).to(DEV), rnd(600, d).to(DEV)

    def both(f):
        a = {k: v.to(DEV) for k, v in t.items()}
        a["f"] = f.to(DEV)
        y, n = G.block_norm_fwd(**a, sigmoid=True)
        return y, n, *G.block_norm_bwd(y, a["f"], a["gate"], a["w_post"], a["w_pre"], dy, dn, sigmoid=True)[:3]
    want = both(t["f"])
    bad = t["f"].clone()
    bad[300, d // 2] = value
    keep = torch.arange(600, device=DEV) != 300
    for a, b in zip(both(bad), want):
        assert torch.equal(a[keep], b[keep]) and not torch.isfinite(a[300]).all()
