"""The attention layer's operators at the edges of their calls, on the GPU: rows of a tile that no token
owns.  Helpers: test_gpu_layer."""
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
