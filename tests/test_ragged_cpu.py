"""Refusals of the ragged append and single-token attention that need no GPU:
argument errors are found on the host before any launch."""
import ctypes

import pytest
import torch

import paged_kv_chunk_query_b200 as pk
import paged_kv_chunk_query_b200._lib as L


@pytest.fixture
def pool():
    h = L.pool_create(8, 16, 2, 64, L.LOC_HOST, True, 0)
    yield h
    L.pool_destroy(h)


def test_calls_refuse_host_pools_and_null(pool):
    lib = L.load()
    rope, dec = L.RopeArgs(), L.DecodeArgs()
    for fn in (lib.oomb_kv_append_rope, lib.oomb_kv_append_rope_bwd):
        assert fn(pool, ctypes.byref(rope), None) == L.ERR_INVALID_ARG
        assert fn(None, ctypes.byref(rope), None) == L.ERR_INVALID_ARG
        assert fn(pool, None, None) == L.ERR_INVALID_ARG
    assert lib.oomb_decode_attn(pool, ctypes.byref(dec), None) == L.ERR_INVALID_ARG
    assert lib.oomb_decode_attn(None, ctypes.byref(dec), None) == L.ERR_INVALID_ARG
    assert lib.oomb_decode_attn(pool, None, None) == L.ERR_INVALID_ARG


def test_binding_refuses_cpu_tensors(pool):
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        pk.kv_append_rope(pool, k, k, i, i[:1], i[None], i, torch.zeros(32))
    with pytest.raises(TypeError):
        pk.kv_append_rope_bwd(pool, k, k, i, i[:1], i[None], i, torch.zeros(32))
    with pytest.raises(TypeError):
        pk.decode_attn(pool, k, k, i[None], i, 1.0, torch.zeros(16, dtype=torch.uint8))


def test_workspace_size_of_refused_shapes_is_zero():
    f = L.load().oomb_decode_attn_workspace_size
    for bad in ((-1, 4, 2, 64, 0), (65536, 4, 2, 64, 0), (4, 3, 2, 64, 0), (4, 4, 0, 64, 0),
                (4, 0, 2, 64, 0), (4, 4, 2, 96, 0), (4, 4, 2, 64, 5), (4, 4, 2, 64, -1)):
        assert f(*bad) == 0, bad
        with pytest.raises(ValueError):
            pk.decode_attn_workspace_size(*bad)
    small, more = f(1, 28, 4, 128, 0), f(256, 28, 4, 128, 0)
    assert 0 < small <= more <= f(256, 28, 4, 128, 256)


def test_packed_arguments_have_the_structures_layout():
    for cls, pack in ((L.RopeArgs, L._ROPE_PACK), (L.DecodeArgs, L._DECODE_PACK)):
        values = [i + 1 for i in range(len(cls._fields_))]
        raw = cls.from_buffer_copy(pack.pack(*values).ljust(ctypes.sizeof(cls), b"\0"))
        assert [getattr(raw, n) or 0 for n, _ in cls._fields_] == values
        assert ctypes.sizeof(cls) - pack.size in (0, 4)  # padding behind the last field
