"""The attention layer's operators at the edges of their calls, on the GPU: rows of a tile that no token
owns, padded batches.  Helpers: test_gpu_layer."""
import pytest
import torch

from recsys_context_personalised_b200 import gdpa as G
from test_gpu_layer import DEV, _chunk_case, _int32

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
