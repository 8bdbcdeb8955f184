"""The attention layer's operators at the edges of their calls: what the host accepts and refuses (CPU only: no call
here reaches a kernel launch)."""
import ctypes
import importlib
import types

import pytest
import torch

from recsys_context_personalised_b200 import gdpa as G
from test_layer_plan import P, _cache


@pytest.mark.parametrize("B,T,max_n", [(3, 64, 1), (1, 1000, 4), (2, 10, 0)])
def test_a_padded_batch_is_not_refused(B, T, max_n):
    """Rows behind the last sample do not count against max_n, the bound of a sample's tokens: the call goes on
    to its workspace (5: too small), whose size does not depend on them."""
    lib, c = G.load(), _cache()
    assert lib.gdpa_chunk_fwd(ctypes.byref(c), B, 4, T, max_n, 8, 1.0, P, P, P, P, None, P, 0, None) == 5
    assert G.chunk_workspace_bytes(c, B, 4, T, max_n) == G.chunk_workspace_bytes(c, B, 4, 0, max_n)
    for bad in (dict(T=-1), dict(T=1 << 31), dict(max_n=-1), dict(B=0)):
        kw = {**dict(B=B, T=T, max_n=max_n), **bad}
        assert lib.gdpa_chunk_fwd(ctypes.byref(c), kw["B"], 4, kw["T"], kw["max_n"], 8, 1.0, P, P, P, P, None, P,
                                  1 << 40, None) == 1
        if kw["T"] < 1 << 31:
            with pytest.raises(G.GdpaError):
                G.chunk_workspace_bytes(c, kw["B"], 4, kw["T"], kw["max_n"])


@pytest.mark.parametrize("group", [1, 16, 17, 40, 128])
def test_a_bound_of_zero_takes_the_workspace_of_one(group):
    lib, c, n = G.load(), _cache(hk=1), [ctypes.c_size_t(), ctypes.c_size_t()]
    for max_n in (0, 1):
        assert lib.gdpa_chunk_workspace_size(ctypes.byref(c), 2, group, 0, max_n, ctypes.byref(n[max_n])) == 0
    assert n[0].value == n[1].value


@pytest.mark.parametrize("kernel", ["gdpa_fwd_sm100", "gdpa_bwd_sm100"])
def test_the_recorded_traffic_belongs_to_the_present_sources(kernel):
    """The bench reports a kernel's DRAM bytes while the sources that they were captured with are unchanged: what
    other operators share stands in headers that these kernels do not include."""
    bench = importlib.import_module("bench")
    for workload, (per_unit, _) in bench.TRAFFIC_PER_UNIT[kernel].items():
        assert bench.traffic_for(kernel, workload, 2.0) == 2.0 * per_unit


def test_the_self_test_of_the_norms_waits_refuses():
    lib = G.load()
    fn = lib.gdpa_selftest_norm_wait
    fn.argtypes, fn.restype = [ctypes.c_int64, ctypes.c_uint32], ctypes.c_int
    for row, us in ((-1, 10), (0, 0), (0, 5000001)):
        assert fn(row, us) == 1


def test_the_norms_workspace_has_room_for_a_status():
    """256 bytes of header for gdpa_workspace_status, and a word for every block, before anything else."""
    lib, n = G.load(), ctypes.c_size_t()
    for d in (8, 1024):
        p = G.BlockNorm(1, d, 1, 0, 0, 0, 1.0, 1e-6, 0)
        assert lib.gdpa_block_norm_bwd_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0
        assert n.value >= 512 + 2 * 4 * d and n.value % 256 == 0


@pytest.mark.parametrize("kw", [dict(rot=2**32 + 64), dict(rot=64, trained_len=2**32 + 2048),
                                dict(rot=64, trained_len=-2**32)])
def test_rotary_settings_beyond_32_bits_are_refused(kw):
    """A whole number that 32 bits do not hold is not cut to the ones that they do."""
    with pytest.raises(G.GdpaError) as e:
        G.rotary_spec(**kw)
    assert e.value.code == 1


def test_a_bound_beyond_32_bits_is_refused():
    with pytest.raises(G.GdpaError) as e:
        G.chunk_workspace_bytes(_cache(), 2, 4, 10, 2**32 + 8)
    assert e.value.code == 1


def test_a_stream_of_another_device_is_refused():
    """(A stand-in for a stream: there is no device here.)"""
    other = types.SimpleNamespace(cuda_stream=1 << 20, device=torch.device("cuda", 1))
    with pytest.raises(G.GdpaError) as e:
        G._On(0, other, ())
    assert e.value.code == 1
