"""CPU checks of what the 8-bit cache's binding reads from a Dims, and of what its handles let a caller change."""
import ctypes
import types

import pytest
import torch

import learned_sparse_kv_decode_b200 as lsa
from learned_sparse_kv_decode_b200 import abi, kv8


def ragged():
    return lsa.Dims(3, 1, 128, 16, 64, chunk_offsets=[0, 5, 9, 20], k_per_seq=[2, 3, 4])


def test_sizes_follow_a_dims_that_is_changed_in_place():
    d = ragged()
    assert (kv8._shape(d).chunks, kv8._shape(d).kept) == (20, 9)
    assert kv8._shape(d) is kv8._shape(d)
    d.c.k_per_seq[1] = 30
    assert kv8._shape(d).kept == 36
    d.c.chunk_offsets[3] = 50
    assert kv8._shape(d).chunks == 50
    d.c.B = 2
    assert (kv8._shape(d).B, kv8._shape(d).chunks, kv8._shape(d).kept) == (2, 9, 32)
    d.c.H, d.c.kv_dtype, d.c.chunk_len = 32, lsa.LSA_F32, 128
    s = kv8._shape(d)
    assert (s.H, s.dtype, s.C) == (32, torch.float32, 128)
    other = (ctypes.c_int32 * 2)(1, 1)
    d.c.k_per_seq = ctypes.cast(other, ctypes.POINTER(ctypes.c_int32))
    assert kv8._shape(d).kept == 2
    other[0] = 7
    assert kv8._shape(d).kept == 8
    d.c.B = 0
    with pytest.raises(lsa.LsaError):
        kv8._shape(d)


def test_sizes_of_a_uniform_dims_follow_it_too():
    d = lsa.Dims(2, 1, 128, 16, 64, N=100, k=10)
    assert (kv8._shape(d).chunks, kv8._shape(d).kept) == (200, 20)
    d.c.k, d.c.N = 11, 90
    assert (kv8._shape(d).chunks, kv8._shape(d).kept) == (180, 22)
    d.c = ragged().c  # its arrays are kept alive only by their Dims, and not read here
    d.c.chunk_offsets = d.c.k_per_seq = None
    d.c.N = d.c.k = 1
    assert (kv8._shape(d).B, kv8._shape(d).chunks) == (3, 3)
    assert ctypes.addressof(kv8._shape(d).ptr._obj) == ctypes.addressof(d.c)


def test_a_call_on_changed_dims_is_refused(monkeypatch):
    """The kept ids of a call are checked against what the C side is about to read."""
    d = ragged()
    cache = types.SimpleNamespace(check=lambda s: -1, ptr=None, n_kv_heads=4)
    q, out = torch.zeros(3, 16, 128, dtype=torch.bfloat16), torch.zeros(3, 16, 128)
    ws, ids = torch.zeros(64, dtype=torch.uint8), torch.zeros(9, dtype=torch.int32)
    made = []
    monkeypatch.setattr(kv8, "_check", lambda *a: made.append(a))
    monkeypatch.setattr(kv8, "_stream", lambda *a: None)
    monkeypatch.setattr(kv8, "lib", types.SimpleNamespace(lsa_kv8_decode_attn=lambda *a: abi.LSA_OK))
    lsa.lsa_kv8_decode_attn(d, cache, q, ids, None, None, out, None, ws)
    assert len(made) == 1
    d.c.k_per_seq[0] = 5
    with pytest.raises(ValueError, match="12 elements, got 9"):
        lsa.lsa_kv8_decode_attn(d, cache, q, ids, None, None, out, None, ws)
    assert len(made) == 1


def test_handles_refuse_another_value(monkeypatch):
    """A tensor that replaced a handle's own would leave the struct with the address of freed memory."""
    prep = lsa.QkPrep(0, eps=1e-5)
    with pytest.raises(AttributeError, match="make a new QkPrep"):
        prep.c = kv8._Prep()
    with pytest.raises(AttributeError, match="make a new QkPrep"):
        prep.tensors = (None, None, None)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)  # stands for tensors on a GPU
    codes = torch.zeros(20, 4, 64, 128, dtype=torch.uint8)
    scales = torch.zeros(20, 4, 1)
    cache = lsa.Kv8Cache(ragged(), 4, 64, codes, codes.clone(), scales, scales.clone())
    for name in ("K8", "V8", "k_scale", "v_scale", "n_kv_heads", "scale_block", "chunks", "C", "c", "ptr"):
        with pytest.raises(AttributeError, match="make a new Kv8Cache"):
            setattr(cache, name, getattr(cache, name))
    assert cache.K8 is codes and cache.c.K8 == codes.data_ptr()
    cache.K8[0] = 1  # what they hold may change
