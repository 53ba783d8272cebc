"""CPU checks of the 8-bit cache's C ABI and binding: exports, refusals on the host before any CUDA call, and the
definitions that the GPU tests compare with."""
import ctypes
import types

import numpy as np
import pytest
import torch

import learned_sparse_kv_decode_b200 as lsa
from learned_sparse_kv_decode_b200 import abi, kv8
from tests import _kv8 as R

P = 0x10000  # an aligned address that no call may follow: every case here is refused before a launch


def dims(**kw):
    base = dict(B=2, Q=1, E=128, H=16, chunk_len=64, N=100, k=10)
    base.update(kw)
    return lsa.Dims(**base)


def cache(hkv=4, sb=64, K8=P, V8=P, ks=P, vs=P):
    return kv8._Cache(hkv, sb, K8, V8, ks, vs)


def prep(rot=128, inter=0, eps=1e-6, inv=P, qw=None, kw=None):
    return kv8._Prep(rot, inter, eps, inv, qw, kw)


def ref(x):
    return None if x is None else ctypes.byref(x)


def test_exports_every_header_symbol():
    names = lsa.kv8_header_symbols()
    assert len(names) == 6
    for n in names:
        assert hasattr(abi.lib, n) and hasattr(lsa, n), n


INV, UNS = lsa.LSA_ERR_INVALID_ARG, lsa.LSA_ERR_UNSUPPORTED


@pytest.mark.parametrize("d,c,expect", [
    (dict(), None, INV),
    (dict(B=0), dict(), INV),
    (dict(), dict(hkv=0), UNS),
    (dict(), dict(hkv=3), UNS),
    (dict(), dict(hkv=32), UNS),          # more than the query heads
    (dict(), dict(sb=4), UNS),
    (dict(), dict(sb=128), UNS),
    (dict(), dict(sb=24), UNS),
    (dict(chunk_len=32), dict(sb=64), UNS),
])
def test_cache_shapes_refused(d, c, expect):
    n = ctypes.c_size_t(0)
    cc = None if c is None else cache(**c)
    assert abi.lib.lsa_kv8_workspace_size(dims(**d).ptr, ref(cc), ctypes.byref(n)) == expect


def test_workspace_size_needs_a_place_for_the_answer():
    assert abi.lib.lsa_kv8_workspace_size(dims().ptr, ref(cache()), None) == INV


BIG = 1 << 40


@pytest.mark.parametrize("kw", [
    dict(K8=None), dict(V8=None), dict(ks=None), dict(vs=None), dict(K8=P + 8), dict(V8=P + 4), dict(ks=P + 2),
    dict(vs=P + 1),
])
def test_cache_pointers_refused(kw):
    c = cache(**kw)
    d = dims()
    lib = abi.lib
    assert lib.lsa_kv8_append(d.ptr, ref(c), None, 1, P, 512, P, 512, P, None, P, BIG, None) == INV
    assert lib.lsa_kv8_gather(d.ptr, ref(c), P, None, P, P, P, BIG, None) == INV
    assert lib.lsa_kv8_decode_attn(d.ptr, ref(c), P, P, None, None, P, P, P, BIG, None) == INV
    assert lib.lsa_decode_step_kv8(d.ptr, ref(c), None, P, P, P, 2048, None, 0, None, 0, None, P, P, P, P, BIG,
                                   None) == INV


def test_null_dims_and_workspace_refused():
    d, c, lib = dims(), cache(), abi.lib
    assert lib.lsa_kv8_append(None, ref(c), None, 1, P, 512, P, 512, P, None, P, BIG, None) == INV
    assert lib.lsa_kv8_append(d.ptr, ref(c), None, 1, P, 512, P, 512, P, None, None, BIG, None) == INV
    assert lib.lsa_kv8_gather(d.ptr, ref(c), P, None, P, P, P + 8, BIG, None) == INV
    assert lib.lsa_kv8_decode_attn(d.ptr, None, P, P, None, None, P, P, P, BIG, None) == INV


@pytest.mark.parametrize("kw,expect", [
    (dict(p=None), INV),
    (dict(p=prep(rot=-16)), INV), (dict(p=prep(rot=144)), INV), (dict(p=prep(rot=24)), UNS),
    (dict(p=prep(inter=2)), INV), (dict(p=prep(eps=-1.0)), INV), (dict(p=prep(eps=float("nan"))), INV),
    (dict(p=prep(eps=float("inf"))), INV), (dict(p=prep(inv=None)), INV), (dict(p=prep(inv=P + 2)), INV),
    (dict(p=prep(qw=P + 4)), INV), (dict(p=prep(kw=P + 8)), INV),
    (dict(n=-1), INV), (dict(hkv=3), UNS), (dict(hkv=32), UNS), (dict(pos=None), INV), (dict(pos=P + 2), INV),
    (dict(q=None), INV), (dict(qo=None), INV), (dict(k=None), INV), (dict(q=None, qo=None, k=None, ko=None), INV),
    (dict(q=P + 8), INV), (dict(ko=P + 8), INV), (dict(qs=2040), INV), (dict(qs=2049), INV), (dict(kos=511), INV),
    (dict(ks=1 << 41), INV), (dict(qo=P, q=P, qs=2048, qos=4096), INV),
])
def test_norm_rope_arguments_refused(kw, expect):
    a = dict(hkv=4, p=prep(), n=5, pos=P, q=P, qs=2048, k=P, ks=512, qo=2 * P, qos=2048, ko=2 * P, kos=512)
    a.update(kw)
    assert abi.lib.lsa_qk_norm_rope(dims().ptr, a["hkv"], ref(a["p"]), a["n"], a["pos"], a["q"], a["qs"], a["k"],
                                    a["ks"], a["qo"], a["qos"], a["ko"], a["kos"], None) == expect


def test_norm_rope_of_no_tokens_is_nothing():
    for q in (P, None):  # an empty tensor's pointer may be null
        assert abi.lib.lsa_qk_norm_rope(dims().ptr, 4, ref(prep()), 0, None, q, 2048, q, 512, q, 2048, q, 512,
                                        None) == lsa.LSA_OK


@pytest.mark.parametrize("kw,expect", [
    (dict(n=0), INV), (dict(n=-3), INV), (dict(k=None), INV), (dict(v=P + 8), INV), (dict(ks=504), INV),
    (dict(vs=516), INV), (dict(start=P + 2), INV), (dict(count=P + 1), INV), (dict(p=prep(rot=8)), UNS),
])
def test_append_arguments_refused(kw, expect):
    a = dict(p=None, n=1, k=P, ks=512, v=P, vs=512, start=P, count=None, size=BIG)
    a.update(kw)
    assert abi.lib.lsa_kv8_append(dims().ptr, ref(cache()), ref(a["p"]), a["n"], a["k"], a["ks"], a["v"], a["vs"],
                                  a["start"], a["count"], P, a["size"], None) == expect


def test_gather_and_attention_arguments_refused():
    d, c, lib = dims(), ref(cache()), abi.lib
    for args in ((P + 2, None, P, P), (P, P + 1, P, P), (P, None, None, P), (P, None, P, P + 8)):
        assert lib.lsa_kv8_gather(d.ptr, c, *args, P, BIG, None) == INV
    for args in ((None, P, None, None, P, P), (P, P + 2, None, None, P, P), (P, P, P + 2, None, P, P),
                 (P, P, None, P + 2, P, P), (P, P, None, None, None, P), (P, P, None, None, P, P + 2)):
        assert lib.lsa_kv8_decode_attn(d.ptr, c, *args, P, BIG, None) == INV
    big = dims(B=1, N=1 << 21, k=1, chunk_len=1024)  # 2^31 tokens of one sequence
    assert lib.lsa_kv8_decode_attn(big.ptr, c, P, None, None, None, P, P, P, 1 << 60, None) == UNS


@pytest.mark.parametrize("kw,expect", [
    (dict(k=None), INV), (dict(v=None), INV), (dict(len=None), INV),
    (dict(len=None, k=None, v=None, p=prep()), INV), (dict(qs=4096), INV), (dict(qs=2044, p=prep()), INV),
    (dict(ks=500), INV), (dict(q=None), INV), (dict(ids=None), INV), (dict(out=None), INV),
    (dict(p=prep(eps=-1.0)), INV),
])
def test_step_arguments_refused(kw, expect):
    a = dict(p=None, q=P, qs=2048, k=P, ks=512, v=P, vs=512, len=P, ids=P, out=P)
    a.update(kw)
    assert abi.lib.lsa_decode_step_kv8(dims().ptr, ref(cache()), ref(a["p"]), P, P, a["q"], a["qs"], a["k"], a["ks"],
                                       a["v"], a["vs"], a["len"], a["ids"], a["out"], P, P, BIG, None) == expect


@pytest.mark.gpu
def test_short_workspace_refused():
    d, c, lib = dims(), ref(cache()), abi.lib
    n = ctypes.c_size_t(0)
    assert lib.lsa_kv8_workspace_size(d.ptr, c, ctypes.byref(n)) == lsa.LSA_OK
    assert n.value >= lsa.lsa_workspace_size(d)
    short, want = n.value - 1, lsa.LSA_ERR_WORKSPACE
    assert lib.lsa_kv8_append(d.ptr, c, None, 1, P, 512, P, 512, P, None, P, short, None) == want
    assert lib.lsa_kv8_gather(d.ptr, c, P, None, P, P, P, short, None) == want
    assert lib.lsa_kv8_decode_attn(d.ptr, c, P, P, None, None, P, P, P, short, None) == want
    assert lib.lsa_decode_step_kv8(d.ptr, c, None, P, P, P, 2048, None, 0, None, 0, None, P, P, P, P, short,
                                   None) == want


# ---------------------------------------------------------------- the binding
def test_binding_refuses_host_tensors():
    d = dims(B=1, N=2, k=1)
    z = torch.zeros(2, 4, 64, 128, dtype=torch.uint8)
    s = torch.zeros(2, 4, 1)
    with pytest.raises(ValueError, match="CUDA"):
        lsa.Kv8Cache(d, 4, 64, z, z, s, s)
    with pytest.raises(ValueError, match="CUDA"):
        lsa.QkPrep(128, torch.zeros(64))
    with pytest.raises(ValueError, match="CUDA"):
        lsa.lsa_qk_norm_rope(d, lsa.QkPrep(0), torch.zeros(1, dtype=torch.int32), None, None, None, None)


def test_binding_checks_types_shapes_and_devices():
    cpu = -1  # a CPU tensor's device index
    x = torch.zeros(6, 4)
    with pytest.raises(TypeError, match="float32"):
        kv8._ptr(x.half(), "x", torch.float32, 24, cpu)
    with pytest.raises(ValueError, match="elements"):
        kv8._ptr(x, "x", torch.float32, 25, cpu)
    with pytest.raises(ValueError, match="contiguous"):
        kv8._ptr(x.t(), "x", torch.float32, 24, cpu)
    with pytest.raises(ValueError, match="cuda:1"):
        kv8._ptr(x, "x", torch.float32, 24, 1)
    with pytest.raises(ValueError, match="cuda:1"):
        kv8._rows(x.view(1, 6, 4), "x", torch.float32, 1, 6, 1)
    with pytest.raises(ValueError, match="cuda:1"):
        kv8._ws(x, 1)
    assert kv8._opt(None, "x", torch.float32, 24, cpu) is None


def test_binding_refuses_another_device(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    there = types.SimpleNamespace(get_device=lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        kv8._device(there)


def test_binding_row_strides():
    f32, cpu = torch.float32, -1
    qkv = torch.zeros(3, 5, 12, 128)  # [B][n][heads]
    assert kv8._rows(qkv[:, :, 4:8], "k", f32, 15, 4, cpu)[1] == 12 * 128
    assert kv8._rows(qkv[:1, :, 4:8], "k", f32, 5, 4, cpu)[1] == 12 * 128
    assert kv8._rows(qkv[:, :1, 4:8], "k", f32, 3, 4, cpu)[1] == 5 * 12 * 128
    assert kv8._rows(qkv[:1, :1, 4:8], "k", f32, 1, 4, cpu)[1] == 4 * 128
    assert kv8._rows(qkv[0, :, 4:5], "k", f32, 5, 1, cpu)[1] == 12 * 128
    for bad in (qkv[:, :3, 4:8], qkv[..., :64], qkv.transpose(-1, -2), qkv[:, :, ::2]):
        with pytest.raises(ValueError):
            kv8._rows(bad, "k", f32, bad.shape[0] * bad.shape[1], 4 if bad is not qkv else 12, cpu)
    with pytest.raises(ValueError):
        kv8._rows(qkv[:, :, ::3], "k", f32, 15, 4, cpu)
    with pytest.raises(TypeError):
        kv8._rows(qkv.half(), "k", f32, 15, 12, cpu)


# ---------------------------------------------------------------- the definitions
def test_e4m3_definition_agrees_with_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    v = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v, R.VALUES, equal_nan=True)
    x = np.concatenate([np.linspace(-448, 448, 20011), np.exp2(np.linspace(-14, 8.8, 4001)), R.VALUES[:127],
                        (R.VALUES[:126] + R.VALUES[1:127]) / 2])  # the midpoints: ties
    t = torch.from_numpy(x).float()
    assert np.array_equal(R.e4m3_round(t.double().numpy()), t.to(torch.float8_e4m3fn).double().numpy())


@pytest.mark.parametrize("amax,e", [(448.0, 0), (448.0000001, 1), (224.0, -1), (1.75, -8), (1.7500001, -7), (1.0, -8),
                                    (0.0, -120), (1e-45, -120), (3.4e38, 120), (2.0 ** -112 * 1.75, -120)])
def test_scale_definition(amax, e):
    assert R.scale_of(amax) == 2.0 ** e


def test_append_definition_by_hand():
    """Two blocks of 8: a first row of 448 sets scale 1, a later one of 1792 makes it 4 and the old codes are rounded
    again; the second block starts afresh."""
    vals, scales = np.zeros((1, 1, 16, R.DH)), np.zeros((1, 1, 2))
    rows = np.full((1, 1, R.DH), 448.0)
    rows[0, 0, 1] = 13.0
    R.append(vals, scales, rows, 0, 1, 16, 8, 0)
    assert scales[0, 0].tolist() == [1.0, 0.0] and vals[0, 0, 0, :2].tolist() == [448.0, 13.0]
    R.append(vals, scales, np.full((1, 1, R.DH), 1792.0), 0, 1, 16, 8, 1)
    assert scales[0, 0, 0] == 4.0 and vals[0, 0, 0, :2].tolist() == [112.0, 3.25] and vals[0, 0, 1, 0] == 448.0
    R.append(vals, scales, np.full((7, 1, R.DH), 7.0), 0, 1, 16, 8, 8)
    assert scales[0, 0].tolist() == [4.0, 2.0 ** -6] and vals[0, 0, 8, 0] == 448.0 and vals[0, 0, 15, 0] == 0.0
