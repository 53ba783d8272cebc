"""GPU tests of the 8-bit K/V cache at values and sizes where a kernel's own number format, split or plan could show:
non-finite queries."""
import numpy as np
import pytest
import torch

from tests import _kv8 as R
from tests.test_gpu_kv8 import attn_inputs, i32

pytestmark = pytest.mark.gpu
DH = R.DH


@pytest.fixture(scope="module")
def lsa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import learned_sparse_kv_decode_b200 as m
    return m


# ---------------------------------------------------------------- non-finite values
# n_b, C, H, Hkv, sb: runs of one part (a few tokens), and runs that are cut into parts and joined
RUNS = [([4], 16, 4, 4, 16), ([4, 2], 16, 16, 1, 8), ([1500], 64, 1, 1, 64), ([1500], 64, 2, 1, 64),
        ([700, 3], 32, 16, 2, 32), ([300], 64, 64, 4, 64), ([60, 50], 64, 8, 8, 64)]


@pytest.mark.parametrize("n_b,C,H,Hkv,sb", RUNS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_query_that_is_not_finite_makes_its_own_head_nan(lsa, n_b, C, H, Hkv, sb, dtype):
    """All logits of such a head are NaN or infinite, and so its softmax is NaN however the run is cut; the other heads
    keep their bits."""
    dims, cache, q = attn_inputs(lsa, n_b, C, H, Hkv, sb, dtype, None, "append", 40, n_b)
    ws = lsa.alloc_workspace(dims, kv8=cache)
    B = len(n_b)
    out0, lse0, out, lse = (torch.empty(B, H, *x, device="cuda") for x in ((DH,), (), (DH,), ()))
    lsa.lsa_kv8_decode_attn(dims, cache, q, None, None, None, out0, lse0, ws)
    assert bool(torch.isfinite(out0).all())
    for value, h in ((float("nan"), 0), (float("inf"), H - 1), (float("-inf"), H // 2)):
        bad = q.clone()
        bad[0, h, 77] = value
        lsa.lsa_kv8_decode_attn(dims, cache, bad, None, None, None, out, lse, ws)
        assert bool(torch.isnan(out[0, h]).all()) and bool(torch.isnan(lse[0, h]))
        rest = torch.ones(B, H, dtype=torch.bool, device="cuda")
        rest[0, h] = False
        assert torch.equal(out[rest], out0[rest]) and torch.equal(lse[rest], lse0[rest])


@pytest.mark.parametrize("H,Hkv", [(2, 2), (16, 2)])
def test_keys_that_are_nan_over_whole_parts_make_their_head_nan(lsa, H, Hkv):
    """NaN from chunk `a` to the end of a run that is cut into parts of fewer than 64 chunks (a tile each): for some of
    64 successive `a` no part holds other scores beside them."""
    n_b, C, sb = [1500], 32, 32
    dims, cache, q = attn_inputs(lsa, n_b, C, H, Hkv, sb, "bf16", None, "append", 41, n_b)
    ws = lsa.alloc_workspace(dims, kv8=cache)
    out0, out = (torch.empty(1, H, DH, device="cuda") for _ in range(2))
    lsa.lsa_kv8_decode_attn(dims, cache, q, None, None, None, out0, None, ws)
    g = H // Hkv
    for a in range(1063, 999, -1):
        cache.K8.view(torch.uint8)[a:, 1] = 0x7F
        lsa.lsa_kv8_decode_attn(dims, cache, q, None, None, None, out, None, ws)
        assert bool(torch.isnan(out[0, g:]).all()) and torch.equal(out[0, :g], out0[0, :g]), a
