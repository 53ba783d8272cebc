"""GPU tests that queries and keys which are not finite give NaN, in every attention over the 16- and 32-bit caches: a
softmax over such logits is NaN, and an output of zeros would say that there was nothing to attend to."""
import numpy as np
import pytest
import torch

import datagen
from tests import _gpu as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lsa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import learned_sparse_kv_decode_b200 as m
    return m


def kept(w, seed):
    r = np.random.default_rng(seed)
    return torch.from_numpy(np.concatenate(
        [np.sort(r.permutation(n)[:k]) for n, k in zip(w.N, w.k)]).astype(np.int32)).cuda()


def check(call, q, out, lse, out0, lse0, b, h, value):
    """`call(q)` with `value` in one row of q: that row's output is NaN, the others keep their bits."""
    bad = q.clone()
    bad[b, h, 77] = value
    out.fill_(7.0)
    lse.fill_(7.0)
    call(bad)
    assert bool(torch.isnan(out[b, h]).all()) and bool(torch.isnan(lse[b, h]).all())
    rest = torch.ones(lse.shape, dtype=torch.bool, device="cuda")
    rest[b, h] = False
    assert torch.equal(out[rest], out0[rest]) and torch.equal(lse[rest], lse0[rest])


VALUES = [float("nan"), float("inf"), float("-inf")]


@pytest.mark.parametrize("kv_dtype,H", [("bf16", 16), ("bf16", 128), ("f32", 8), ("bf16", 1)])
def test_sparse_attention(lsa, kv_dtype, H):
    w = datagen.small_workload(B=3, N=(40, 9, 200), k=(11, 9, 200), C=64, E=64, H=H, kv_dtype=kv_dtype, seed=71)
    dw = G.DeviceWorkload(w, lsa)
    ids = kept(w, 1)
    counts = torch.tensor([7, 0, 200], dtype=torch.int32, device="cuda")
    calls = {
        "ids": lambda q: lsa.lsa_sparse_decode_attn(dw.dims, q, dw.K, dw.V, ids, dw.out, dw.lse, dw.ws),
        "counts": lambda q: lsa.lsa_sparse_decode_attn_counts(dw.dims, q, dw.K, dw.V, ids, counts, dw.out, dw.lse, dw.ws),
        "noalloc": lambda q: lsa.lsa_sparse_decode_attn_noalloc(dw.dims, q, dw.K, dw.V, ids, dw.out, dw.lse),
    }
    if H == 128:  # more partials than the library's fixed scratch holds
        with pytest.raises(lsa.LsaError):
            calls.pop("noalloc")(dw.q)
    for name, call in calls.items():
        call(dw.q)
        out0, lse0 = dw.out.clone(), dw.lse.clone()
        for b, h, value in zip((0, 2, 2), (0, H - 1, H // 2), VALUES):
            check(call, dw.q, dw.out, dw.lse, out0, lse0, b, h, value)
        if name == "counts":
            assert bool((dw.out[1] == 0).all()) and bool((dw.lse[1] == -np.inf).all())
    dw.K[int(w.chunk_offsets[1]) * w.C:int(w.chunk_offsets[2]) * w.C, 0] = float("nan")  # all keys of one sequence
    calls["ids"](dw.q)
    assert bool(torch.isnan(dw.out[1, 0]).all()) and bool(torch.isfinite(dw.out[[0, 2]]).all())


@pytest.mark.parametrize("B,N,k,C,H,kv_dtype", [(1, 64, 8, 64, 8, "f32"), (2, 20, 3, 8, 4, "bf16"), (1, 40, 1, 16, 2, "f32"),
                                                (2, 50, 20, 32, 4, "bf16")])
def test_one_launch_step(lsa, B, N, k, C, H, kv_dtype):
    w = datagen.small_workload(B=B, N=(N,) * B, k=(k,) * B, C=C, E=64, H=H, kv_dtype=kv_dtype, seed=72)
    dw = G.DeviceWorkload(w, lsa)

    def call(q):
        lsa.lsa_decode_step(dw.dims, dw.q_emb, dw.chunk_emb, q, dw.K, dw.V, dw.ids, dw.out, dw.lse, dw.ws)

    call(dw.q)
    out0, lse0 = dw.out.clone(), dw.lse.clone()
    for h, value in zip((0, H - 1, H // 2), VALUES):
        check(call, dw.q, dw.out, dw.lse, out0, lse0, B - 1, h, value)
    first = int(dw.ids[0])
    dw.K[first * C + 3, 0, 5] = float("nan")  # one key of one head
    call(dw.q)
    assert bool(torch.isnan(dw.out[0, 0]).all()) and bool(torch.isnan(dw.lse[0, 0]))
    assert torch.equal(dw.out[0, 1:], out0[0, 1:])
    assert lsa.lsa_get_device_status(dw.ws) == lsa.LSA_OK


@pytest.mark.parametrize("B,N,k,C,Q,H", [(2, (40, 72), (5, 9), 64, 64, 4), (1, (9,), (1,), 64, 64, 1),
                                         (1, (600,), (600,), 64, 7, 1), (3, (30, 50, 8), (7, 3, 8), 16, 33, 2)])
def test_lookahead_attention(lsa, B, N, k, C, Q, H):
    w = datagen.small_workload(B=B, N=N, k=k, C=C, Q=Q, E=64, H=H, kv_dtype="bf16", seed=73)
    dw = G.DeviceWorkload(w, lsa)
    q = G.to_device(datagen.make_lookahead_queries(w), "bf16").view(B, Q * H, w.Dh)
    out, lse = torch.empty(B, Q * H, w.Dh, device="cuda"), torch.empty(B, Q * H, device="cuda")
    ids = kept(w, 2)

    def call(x):
        lsa.lsa_sparse_decode_attn_lookahead(dw.dims, x, dw.K, dw.V, ids, out, lse, dw.ws)

    call(q)
    out0, lse0 = out.clone(), lse.clone()
    assert bool(torch.isfinite(out0).all())
    for row, value in zip((0, Q * H - 1, Q * H // 2), VALUES):
        check(call, q, out, lse, out0, lse0, B - 1, row, value)
    dw.K[int(w.chunk_offsets[B - 1]) * C + int(ids[-1]) * C + 2, 0, 5] = float("nan")
    call(q)
    nan = torch.isnan(out.view(B, Q, H, w.Dh))
    assert bool(nan[B - 1, :, 0].all()) and not bool(nan[:, :, 1:].any()) and not bool(nan[:B - 1].any())
    assert lsa.lsa_get_device_status(dw.ws) == lsa.LSA_OK


def test_merge_of_partials(lsa):
    """A rank's NaN reaches the merged output; a rank that kept nothing (lse = -inf) does not take part, whatever it holds."""
    G_, B, H, Dh = 3, 2, 4, 128
    gen = torch.Generator(device="cuda").manual_seed(5)
    outs = torch.randn(G_, B, H, Dh, generator=gen, device="cuda")
    lses = torch.randn(G_, B, H, generator=gen, device="cuda")
    lses[1, 0, 1], outs[1, 0, 1] = -np.inf, 0.0
    lses[:, 1, 2], outs[:, 1, 2] = -np.inf, 0.0
    out, lse = torch.empty(B, H, Dh, device="cuda"), torch.empty(B, H, device="cuda")
    lsa.lsa_merge_partials(G_, B, H, outs, lses, out, lse)
    out0, lse0 = out.clone(), lse.clone()
    assert bool(torch.isfinite(out0).all()) and bool((out0[1, 2] == 0).all()) and float(lse0[1, 2]) == -np.inf
    p = torch.softmax(lses.double(), 0)
    want = (p[..., None] * outs.double()).sum(0)
    ok = torch.ones(B, H, dtype=torch.bool, device="cuda")
    ok[1, 2] = False
    torch.testing.assert_close(out0[ok].double(), want[ok], rtol=0, atol=1e-5)
    nan = float("nan")
    lses[2, 0, 0], outs[2, 0, 0] = nan, nan                 # one rank of three
    lses[:, 0, 3], outs[:, 0, 3] = nan, nan                 # every rank
    lses[0, 1, 2], outs[0, 1, 2] = nan, nan                 # the others kept nothing
    lsa.lsa_merge_partials(G_, B, H, outs, lses, out, lse)
    hit = torch.zeros(B, H, dtype=torch.bool, device="cuda")
    hit[0, 0] = hit[0, 3] = hit[1, 2] = True
    assert bool(torch.isnan(out[hit]).all()) and bool(torch.isnan(lse[hit]).all())
    assert torch.equal(out[~hit], out0[~hit]) and torch.equal(lse[~hit], lse0[~hit])
