"""GPU tests of the 8-bit K/V cache's operators against their definitions in 64 bits (tests/_kv8.py)."""
import numpy as np
import pytest
import torch

import datagen
from tests import _gpu as G
from tests import _kv8 as R
from tests.test_gpu_canary import Guards

pytestmark = pytest.mark.gpu
DH = R.DH


@pytest.fixture(scope="module")
def lsa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import learned_sparse_kv_decode_b200 as m
    return m


def make_dims(lsa, n_b, k_b, C, H, dtype="bf16", E=128, Q=1):
    off = np.concatenate([[0], np.cumsum(n_b)]).tolist()
    return lsa.Dims(len(n_b), Q, E, H, C, chunk_offsets=off, k_per_seq=list(k_b), emb_dtype=dtype, kv_dtype=dtype)


def tensor(x, dtype):
    return torch.from_numpy(np.asarray(x)).to(G.tdtype(dtype)).cuda()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


HALF = {"bf16": 2.0 ** -9, "f32": 2.0 ** -24}  # half a step, relative to the next power of two below


# ---------------------------------------------------------------- norm and rotation
PREP = [
    # T, H, Hkv, dtype, rot, interleaved, norm, positions up to
    (1, 8, 8, "bf16", 128, False, True, 1 << 20),
    (1, 1, 1, "f32", 128, True, True, 7),
    (3, 16, 2, "bf16", 64, True, True, 1 << 20),
    (37, 4, 1, "f32", 32, False, True, 1 << 20),
    (5, 32, 8, "bf16", 112, False, False, 1000),
    (129, 2, 2, "f32", 96, True, False, 1 << 30),
    (64, 128, 16, "bf16", 16, True, True, 100),
    (2, 8, 4, "bf16", 0, False, True, 100),
    (5000, 8, 2, "bf16", 128, False, True, 1 << 20),
    (14211, 4, 1, "bf16", 64, True, True, 1 << 20),   # four tokens to a warp, the last warp with three
    (14209, 1, 1, "f32", 128, False, True, 1 << 20),
    (14210, 2, 2, "f32", 32, True, False, 1 << 20),
]


def prep_inputs(T, H, Hkv, dtype, rot, norm, far, seed):
    r = np.random.default_rng(seed)
    qkv = tensor(r.normal(0, 2, (T, H + 2 * Hkv, DH)), dtype)
    pos = i32(r.integers(0, far, T))
    inv = torch.from_numpy((10000.0 ** (-2.0 * np.arange(rot // 2) / max(rot, 1))).astype(np.float32)).cuda()
    w = [torch.from_numpy(r.normal(1, 0.3, DH).astype(np.float32)).cuda() if norm else None for _ in range(2)]
    return qkv, pos, inv, w


def check_prep(got, x, pos, inv, w, rot, inter, dtype, eps=1e-6):
    """Each value of a pair (or alone) carries the norm's and the rotation's fp32 errors: the sum of squares (16 terms a
    lane, 3 joins: 20 u), its root, two products, and sine and cosine within 2 u: 40 u of the pair's size together,
    u = 2^-24; then the rounding to the row's type."""
    y = R.norm_rope(R.f64(x), pos.cpu().numpy(), inv.cpu().numpy(), None if w is None else R.f64(w), rot, inter, eps)
    n = np.array(R.norm_rope(R.f64(x), pos.cpu().numpy(), np.zeros(rot // 2), None if w is None else R.f64(w), rot,
                             inter, eps))
    size = np.abs(n)
    for i in range(rot // 2):
        p, r = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
        size[..., p] = size[..., r] = np.hypot(n[..., p], n[..., r])
    tol = size * 40 * 2.0 ** -24
    tol = tol + (np.abs(y) + tol) * (2 * HALF[dtype]) + 1e-30
    assert np.all(np.abs(R.f64(got) - y) <= tol), np.max(np.abs(R.f64(got) - y) / tol)


@pytest.mark.parametrize("T,H,Hkv,dtype,rot,inter,norm,far", PREP)
def test_norm_rope(lsa, T, H, Hkv, dtype, rot, inter, norm, far):
    qkv, pos, inv, w = prep_inputs(T, H, Hkv, dtype, rot, norm, far, T + H)
    q, k = qkv[:, :H], qkv[:, H:H + Hkv]
    d = lsa.Dims(1, 1, 128, H, 64, N=1, k=1, kv_dtype=dtype)
    prep = lsa.QkPrep(rot, inv if rot else None, *w, eps=1e-6, interleaved=inter)
    g = Guards()
    qo, ko = g((T, H, DH), q.dtype), g((T, Hkv, DH), q.dtype)
    lsa.lsa_qk_norm_rope(d, prep, pos, q, k, qo, ko)
    g.check()
    check_prep(qo, q, pos, inv, w[0], rot, inter, dtype)
    check_prep(ko, k, pos, inv, w[1], rot, inter, dtype)
    # one of the two alone, and in place inside the packed rows: the same bits, the rest untouched
    k1 = torch.empty_like(ko)
    lsa.lsa_qk_norm_rope(d, prep, pos, None, k, None, k1)
    assert torch.equal(k1, ko)
    both = qkv.clone()
    lsa.lsa_qk_norm_rope(d, prep, pos, both[:, :H], both[:, H:H + Hkv], both[:, :H], both[:, H:H + Hkv])
    assert torch.equal(both[:, :H], qo) and torch.equal(both[:, H:H + Hkv], ko)
    assert torch.equal(both[:, H + Hkv:], qkv[:, H + Hkv:])


def test_norm_rope_of_no_tokens(lsa):
    d = lsa.Dims(1, 1, 128, 4, 64, N=1, k=1, kv_dtype="f32")
    x = torch.empty(0, 4, DH, device="cuda")
    lsa.lsa_qk_norm_rope(d, lsa.QkPrep(0), i32([]), x, x[:, :2], x, x[:, :2])


def test_norm_rope_infinities_stay_in_their_pairs(lsa):
    """Without a norm, an infinity reaches its own pair and no other value; with one its row, and no other row."""
    d = lsa.Dims(1, 1, 128, 2, 64, N=1, k=1, kv_dtype="f32")
    inv = torch.linspace(1.0, 0.001, 32, device="cuda")
    for inter in (False, True):
        x = torch.randn(3, 2, DH, device="cuda")
        x[1, 0, 5] = float("inf")    # rotated
        x[1, 1, 70] = float("-inf")  # not rotated: rot_dim 64
        o = torch.empty_like(x)
        lsa.lsa_qk_norm_rope(d, lsa.QkPrep(64, inv, None, None, 1e-6, inter), i32([3, 4, 5]), x, None, o, None)
        bad = ~torch.isfinite(o)
        assert bad[1, 0].nonzero().view(-1).tolist() == ([4, 5] if inter else [5, 37])
        assert bad[1, 1].nonzero().view(-1).tolist() == [70] and not bool(bad[[0, 2]].any())
        lsa.lsa_qk_norm_rope(d, lsa.QkPrep(64, inv, torch.ones(DH, device="cuda"), None, 1e-6, inter), i32([3, 4, 5]),
                             x, None, o, None)
        assert bool(torch.isfinite(o[[0, 2]]).all())


def test_norm_rope_zero_rows_and_negative_positions(lsa):
    d = lsa.Dims(1, 1, 128, 2, 64, N=1, k=1, kv_dtype="f32")
    x = torch.zeros(2, 2, DH, device="cuda")
    x[1] = torch.randn(2, DH, device="cuda")
    inv = torch.linspace(1.0, 0.001, 64, device="cuda")
    pos = i32([5, -70001])
    w = torch.ones(DH, device="cuda")
    o = torch.full_like(x, 9.0)
    lsa.lsa_qk_norm_rope(d, lsa.QkPrep(128, inv, w, None, 1e-6), pos, x, None, o, None)
    assert bool((o[0] == 0).all())
    check_prep(o[1:], x[1:], pos[1:], inv, w, 128, False, "f32")


# ---------------------------------------------------------------- the quantising write
APPEND = [
    # chunks per sequence, C, Hkv, sb, dtype, n_new, starts, counts, values' size
    ([2], 8, 1, 8, "bf16", 1, [0], None, 1.0),
    ([3, 2], 16, 2, 8, "f32", 5, [13, 31], None, 1.0),            # the second overruns by 4 rows
    ([4, 4, 4], 64, 4, 64, "bf16", 1, [63, 64, 200], None, 1.0),
    ([4, 4, 4], 64, 4, 16, "f32", 130, [1, 0, 120], [130, 0, 77], 3.0),
    ([9, 1], 32, 16, 32, "bf16", 100, [60, 0], [99, 31], 1.0),
    ([2, 2], 1024, 1, 64, "bf16", 1000, [1000, 24], None, 1e-3),
    ([30], 8, 8, 8, "f32", 239, [1], None, 100.0),
    ([5, 7], 16, 2, 16, "bf16", 64, [0, 16], None, 1.0),
    ([3], 128, 2, 32, "f32", 65, [63], None, 1e30),
    ([3], 128, 2, 32, "f32", 65, [63], None, 1e-40),
]


def append_case(lsa, n_b, C, Hkv, sb, dtype, n, seed, size, scales="append"):
    r = np.random.default_rng(seed)
    B = len(n_b)
    dims = make_dims(lsa, n_b, [1] * B, C, max(Hkv, 2), dtype)
    t = R.make_cache(lsa, sum(n_b), Hkv, C, sb, r, scales)
    rows = r.normal(0, size, (B, n, 3 * Hkv, DH)) * np.exp(r.normal(0, 1, (B, n, 3 * Hkv, 1)))
    qkv = tensor(rows, dtype)
    return dims, t, qkv[:, :, Hkv:2 * Hkv], qkv[:, :, 2 * Hkv:]


def guarded_cache(lsa, g, dims, Hkv, sb, t):
    u = {n: g(tuple(x.shape), torch.uint8 if x.dtype == torch.float8_e4m3fn else x.dtype) for n, x in t.items()}
    for n in u:
        u[n].copy_(t[n].view(u[n].dtype))
    return lsa.Kv8Cache(dims, Hkv, sb, u["K8"], u["V8"], u["k_scale"], u["v_scale"]), u


def check_append(before, after, x, n_b, C, sb, starts, counts, name):
    vals, sc = R.decode(before[name + "8"]), R.f64(before[name.lower() + "_scale"])
    off = np.concatenate([[0], np.cumsum(n_b)])
    for b in range(len(n_b)):
        n = x.shape[1] if counts is None else max(0, min(x.shape[1], counts[b]))
        R.append(vals, sc, x[b, :n], int(off[b]), n_b[b], C, sb, starts[b])
    assert np.array_equal(R.f64(after[name.lower() + "_scale"]), sc, equal_nan=True)  # untouched blocks may hold NaN
    assert np.array_equal(R.decode(after[name + "8"]), vals, equal_nan=True)


@pytest.mark.parametrize("n_b,C,Hkv,sb,dtype,n,starts,counts,size", APPEND)
@pytest.mark.parametrize("scales", ["append", "free"])
def test_append(lsa, n_b, C, Hkv, sb, dtype, n, starts, counts, size, scales):
    dims, t, k, v = append_case(lsa, n_b, C, Hkv, sb, dtype, n, 5 + C + n, size, scales)
    if scales == "free":
        # a block that came with another scale: compare where no quotient lies within the divisions' rounding of a
        # border, by making every value and scale an integer times a power of two with few bits
        for s in ("k_scale", "v_scale"):
            t[s].copy_(torch.exp2(torch.floor(torch.log2(t[s]))) * 1.5)
    g = Guards()
    cache, u = guarded_cache(lsa, g, dims, Hkv, sb, t)
    ws = g(lsa.lsa_kv8_workspace_size(dims, cache), torch.uint8)
    lsa.lsa_workspace_init(ws)
    lsa.lsa_kv8_append(dims, cache, None, k, v, i32(starts), None if counts is None else i32(counts), ws)
    g.check()
    if scales == "append":
        check_append(t, u, R.f64(k), n_b, C, sb, starts, counts, "K")
        check_append(t, u, R.f64(v), n_b, C, sb, starts, counts, "V")
    else:
        for name, x in (("K", k), ("V", v)):
            vals, sc = R.decode(t[name + "8"]), R.f64(t[name.lower() + "_scale"])
            off = np.concatenate([[0], np.cumsum(n_b)])
            for b in range(len(n_b)):
                m = n if counts is None else counts[b]
                R.append(vals, sc, R.f64(x)[b, :m], int(off[b]), n_b[b], C, sb, starts[b])
            assert np.array_equal(R.f64(u[name.lower() + "_scale"]), sc)
            got = R.decode(u[name + "8"])
            # a quotient by 1.5 2^e that is rounded to fp32 first may cross a border: one e4m3 step (2^-3) at most,
            # and hardly ever
            assert np.all(np.abs(got - vals) <= np.maximum(np.abs(vals), 2.0 ** -6) * 2.0 ** -3 * 1.01)
            assert np.mean(got != vals) < 1e-3
    over = any(s + (n if counts is None else counts[i]) > n_b[i] * C for i, s in enumerate(starts))
    assert lsa.lsa_get_device_status(ws) == (lsa.LSA_ERR_BAD_ID if over else lsa.LSA_OK)


def test_append_token_by_token_equals_definition(lsa):
    """A block filled a token at a time, whose scale grows on the way, in a captured and replayed step."""
    n_b, C, Hkv, sb = [2, 3], 16, 2, 16
    dims = make_dims(lsa, n_b, [1, 1], C, 2, "f32")
    r = np.random.default_rng(3)
    t = R.make_cache(lsa, 5, Hkv, C, sb, r)
    before = {n: x.clone() for n, x in t.items()}
    cache = lsa.Kv8Cache(dims, Hkv, sb, t["K8"], t["V8"], t["k_scale"], t["v_scale"])
    ws = lsa.alloc_workspace(dims, kv8=cache)
    rows = (r.normal(0, 1, (30, 2, 1, 2 * Hkv, DH)) * np.exp2(np.arange(30) % 16 / 2.0)[:, None, None, None, None])
    kv = torch.zeros(2, 1, 2 * Hkv, DH, device="cuda")
    start = i32([0, 3])
    lsa.lsa_kv8_append(dims, cache, None, kv[:, :, :Hkv], kv[:, :, Hkv:], start, None, ws)  # warm-up, rewritten below
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lsa.lsa_kv8_append(dims, cache, None, kv[:, :, :Hkv], kv[:, :, Hkv:], start, None, ws)
    for n, x in t.items():
        x.copy_(before[n])
    vals = {n: R.decode(before[n + "8"]) for n in "KV"}
    sc = {n: R.f64(before[n.lower() + "_scale"]) for n in "KV"}
    x32 = torch.from_numpy(rows).float()
    for i in range(30):
        kv.copy_(x32[i])
        graph.replay()
        start += 1
        for b in range(2):
            for n, j in (("K", 0), ("V", Hkv)):
                R.append(vals[n], sc[n], x32[i, b, :, j:j + Hkv].double().numpy(), [0, 2][b], n_b[b], C, sb, [0, 3][b] + i)
    for n in "KV":
        assert np.array_equal(R.f64(t[n.lower() + "_scale"]), sc[n])
        assert np.array_equal(R.decode(t[n + "8"]), vals[n])
    assert lsa.lsa_get_device_status(ws) == lsa.LSA_OK


@pytest.mark.parametrize("starts,counts,status", [
    ([-1, 3], None, "BAD_ID"), ([40, 0], None, "BAD_ID"), ([33, 0], [-5, 99], "OK"), ([2 ** 31 - 1, 1], None, "BAD_ID"),
    ([-2 ** 31, 1], [1, 1], "BAD_ID"), ([32, 0], [0, 0], "OK"),
])
def test_append_odd_starts_and_counts(lsa, starts, counts, status):
    n_b, C, Hkv, sb, n = [2, 2], 16, 2, 8, 7
    dims, t, k, v = append_case(lsa, n_b, C, Hkv, sb, "bf16", n, 11, 1.0)
    g = Guards()
    cache, u = guarded_cache(lsa, g, dims, Hkv, sb, t)
    ws = lsa.alloc_workspace(dims, kv8=cache)
    lsa.lsa_kv8_append(dims, cache, None, k, v, i32(starts), None if counts is None else i32(counts), ws)
    g.check()
    c = None if counts is None else [max(0, min(n, x)) for x in counts]
    check_append(t, u, R.f64(k), n_b, C, sb, starts, c, "K")
    check_append(t, u, R.f64(v), n_b, C, sb, starts, c, "V")
    assert lsa.lsa_get_device_status(ws) == getattr(lsa, "LSA_OK" if status == "OK" else "LSA_ERR_" + status)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_non_finite_rows(lsa, dtype):
    """An infinity is stored as the largest code, a NaN as NaN; neither makes the scale."""
    n_b, C, Hkv, sb, n = [1], 16, 2, 8, 16
    dims, t, k, v = append_case(lsa, n_b, C, Hkv, sb, dtype, n, 12, 1.0)
    k, v = k.clone(), v.clone()
    k[0, 3, 0, 5], k[0, 9, 1, 127], v[0, 0, 0, 0], v[0, 15, 1, 64] = float("inf"), float("nan"), float("-inf"), float("nan")
    v[0, 4, 0] = float("nan")
    cache = lsa.Kv8Cache(dims, Hkv, sb, t["K8"].clone(), t["V8"].clone(), t["k_scale"].clone(), t["v_scale"].clone())
    ws = lsa.alloc_workspace(dims, kv8=cache)
    lsa.lsa_kv8_append(dims, cache, None, k, v, None, None, ws)
    u = {"K8": cache.K8, "V8": cache.V8, "k_scale": cache.k_scale, "v_scale": cache.v_scale}
    check_append(t, u, R.f64(k), n_b, C, sb, [0], None, "K")
    check_append(t, u, R.f64(v), n_b, C, sb, [0], None, "V")
    assert lsa.lsa_get_device_status(ws) == lsa.LSA_ERR_NONFINITE


@pytest.mark.parametrize("dtype,rot,inter,norm,n", [
    ("bf16", 128, False, True, 70), ("f32", 64, True, True, 9), ("bf16", 32, False, False, 1), ("f32", 0, False, True, 130),
    ("bf16", 96, True, True, 300),
])
def test_append_prepares_as_the_separate_call(lsa, dtype, rot, inter, norm, n):
    """K prepared in the same pass: bit for bit what lsa_qk_norm_rope followed by a plain append gives."""
    n_b, C, Hkv, sb = [6, 6], 64, 8, 32
    starts, counts = [37, 0], [n, max(1, n - 3)]
    dims, t, k, v = append_case(lsa, n_b, C, Hkv, sb, dtype, n, 13, 2.0)
    _, _, inv, w = prep_inputs(1, 1, 1, dtype, rot, norm, 2, 14)
    prep = lsa.QkPrep(rot, inv if rot else None, None, w[1], 1e-5, inter)
    a, b = ({m: x.clone() for m, x in t.items()} for _ in range(2))
    ca, cb = (lsa.Kv8Cache(dims, Hkv, sb, y["K8"], y["V8"], y["k_scale"], y["v_scale"]) for y in (a, b))
    ws = lsa.alloc_workspace(dims, kv8=ca)
    lsa.lsa_kv8_append(dims, ca, prep, k, v, i32(starts), i32(counts), ws)
    pos = (torch.tensor(starts)[:, None] + torch.arange(n)).to(torch.int32).cuda()
    kp = torch.empty((2, n, Hkv, DH), dtype=k.dtype, device="cuda")
    lsa.lsa_qk_norm_rope(dims, prep, pos.view(-1), None, k.contiguous().view(-1, Hkv, DH), None, kp.view(-1, Hkv, DH))
    lsa.lsa_kv8_append(dims, cb, None, kp, v, i32(starts), i32(counts), ws)
    for m in a:
        assert torch.equal(a[m].view(torch.uint8), b[m].view(torch.uint8)), m
    assert lsa.lsa_get_device_status(ws) == lsa.LSA_OK


@pytest.mark.parametrize("dtype,B,n", [("bf16", 4, 700), ("f32", 4, 700), ("bf16", 32, 200), ("f32", 32, 200)])
@pytest.mark.parametrize("inter", [False, True])
def test_append_of_many_rows_walks_several_heads(lsa, dtype, B, n, inter):
    """Calls long enough that a CTA takes three to eight heads one after the other: plain rows against the definition,
    prepared rows bit for bit against the two separate calls."""
    C, Hkv, sb = 64, 16, 32
    n_b = [n // C + 2 + b % 3 for b in range(B)]
    starts, counts = [(29 * b) % 65 for b in range(B)], [n - 13 * (b % 4) for b in range(B)]
    dims, t, k, v = append_case(lsa, n_b, C, Hkv, sb, dtype, n, 50 + B, 1.5)
    caches = [{m: x.clone() for m, x in t.items()} for _ in range(3)]
    ca, cb, cc = (lsa.Kv8Cache(dims, Hkv, sb, y["K8"], y["V8"], y["k_scale"], y["v_scale"]) for y in caches)
    ws = lsa.alloc_workspace(dims, kv8=ca)
    lsa.lsa_kv8_append(dims, ca, None, k, v, i32(starts), i32(counts), ws)
    check_append(t, caches[0], R.f64(k), n_b, C, sb, starts, counts, "K")
    check_append(t, caches[0], R.f64(v), n_b, C, sb, starts, counts, "V")
    _, _, inv, w = prep_inputs(1, 1, 1, dtype, 128, True, 2, 14)
    prep = lsa.QkPrep(128, inv, None, w[1], 1e-5, inter)
    lsa.lsa_kv8_append(dims, cb, prep, k, v, i32(starts), i32(counts), ws)
    pos = (torch.tensor(starts)[:, None] + torch.arange(n)).to(torch.int32).cuda()
    kp = torch.empty((B, n, Hkv, DH), dtype=k.dtype, device="cuda")
    lsa.lsa_qk_norm_rope(dims, prep, pos.view(-1), None, k.contiguous().view(-1, Hkv, DH), None, kp.view(-1, Hkv, DH))
    lsa.lsa_kv8_append(dims, cc, None, kp, v, i32(starts), i32(counts), ws)
    for m in t:
        assert torch.equal(caches[1][m].view(torch.uint8), caches[2][m].view(torch.uint8)), m
    assert lsa.lsa_get_device_status(ws) == lsa.LSA_OK


# ---------------------------------------------------------------- reading back
GATHER = [
    # n_b, k_b, C, Hkv, sb, dtype, lengths
    ([1], [1], 8, 1, 8, "f32", None),
    ([5, 9], [2, 9], 8, 2, 8, "bf16", None),
    ([20, 3, 7], [6, 1, 7], 64, 16, 64, "bf16", [1279, 0, 400]),
    ([4], [3], 1024, 4, 64, "f32", [3000]),
    ([11, 2], [5, 2], 32, 8, 16, "f32", [1, 64]),
    ([6, 6], [4, 4], 128, 1, 8, "bf16", [-4, 10 ** 9]),
]


def kept_ids(n_b, k_b, seed):
    r = np.random.default_rng(seed)
    return [np.sort(r.permutation(n)[:k]) for n, k in zip(n_b, k_b)]


@pytest.mark.parametrize("n_b,k_b,C,Hkv,sb,dtype,lens", GATHER)
@pytest.mark.parametrize("whole", [False, True])
@pytest.mark.parametrize("scales", ["append", "free"])
@pytest.mark.parametrize("shift", [0, 16])
def test_gather(lsa, n_b, k_b, C, Hkv, sb, dtype, lens, whole, scales, shift):
    r = np.random.default_rng(C + Hkv)
    dims = make_dims(lsa, n_b, k_b, C, max(2, Hkv), dtype)
    t = R.make_cache(lsa, sum(n_b), Hkv, C, sb, r, scales)
    cache = lsa.Kv8Cache(dims, Hkv, sb, t["K8"], t["V8"], t["k_scale"], t["v_scale"])
    ws = lsa.alloc_workspace(dims, kv8=cache)
    ids = kept_ids(n_b, k_b, 1) if not whole else [np.arange(n) for n in n_b]
    rows = sum(len(x) for x in ids) * C
    g = Guards()
    es = 2 if dtype == "bf16" else 4
    bufs = []
    for _ in range(2):  # `shift` bytes behind the allocator's alignment: 16-byte aligned, not 32
        raw = g((rows * Hkv * DH + shift // es,), G.tdtype(dtype))
        raw.fill_(7.0)
        bufs.append(raw[shift // es:].view(rows, Hkv, DH))
    lsa.lsa_kv8_gather(dims, cache, None if whole else i32(np.concatenate(ids)), None if lens is None else i32(lens),
                       bufs[0], bufs[1], ws)
    g.check()
    off, j = np.concatenate([[0], np.cumsum(n_b)]), 0
    for name, got in (("K", bufs[0]), ("V", bufs[1])):
        x = R.decode(t[name + "8"]) * np.repeat(R.f64(t[name.lower() + "_scale"]), sb, -1)[..., None]
        want = np.full((rows, Hkv, DH), 7.0)
        j = 0
        for b, kept in enumerate(ids):
            for i in kept:
                n = C if lens is None else int(np.clip(lens[b] - i * C, 0, C))
                want[j * C:j * C + n] = x[off[b] + i].transpose(1, 0, 2)[:n]
                j += 1
        # code * scale is exact in fp32 for a power of two and within half an fp32 step otherwise
        want = torch.from_numpy(want).float().to(got.dtype)
        assert torch.equal(got.cpu(), want)
    assert lsa.lsa_get_device_status(ws) == lsa.LSA_OK


def test_gather_bad_ids(lsa):
    n_b, k_b, C, Hkv, sb = [4, 4], [3, 2], 16, 2, 16
    r = np.random.default_rng(0)
    dims = make_dims(lsa, n_b, k_b, C, 2, "f32")
    t = R.make_cache(lsa, 8, Hkv, C, sb, r)
    cache = lsa.Kv8Cache(dims, Hkv, sb, t["K8"], t["V8"], t["k_scale"], t["v_scale"])
    ws = lsa.alloc_workspace(dims, kv8=cache)
    K, V = (torch.full((5 * C, Hkv, DH), 7.0, device="cuda") for _ in range(2))
    lsa.lsa_kv8_gather(dims, cache, i32([0, 4, 2, -1, 3]), None, K, V, ws)
    x = R.decode(t["K8"]) * R.f64(t["k_scale"])[..., None]
    for j, c in enumerate([0, None, 2, None, 7]):
        want = np.full((C, Hkv, DH), 7.0) if c is None else x[c].transpose(1, 0, 2)
        assert np.array_equal(R.f64(K[j * C:(j + 1) * C]), want)
    assert lsa.lsa_get_device_status(ws) == lsa.LSA_ERR_BAD_ID
    assert lsa.lsa_get_device_status(ws) == lsa.LSA_OK


# ---------------------------------------------------------------- attention
ATTN = [
    # n_b, k_b, C, H, Hkv, sb, dtype, lengths, scales
    ([1], [1], 8, 1, 1, 8, "f32", None, "append"),
    ([1], [1], 8, 1, 1, 8, "bf16", [1], "append"),
    ([64], [8], 64, 8, 8, 64, "f32", None, "append"),
    ([3, 5], [3, 4], 8, 4, 2, 8, "bf16", None, "free"),                # an odd number of 8-token chunks
    ([30, 1, 7], [9, 1, 7], 16, 8, 2, 8, "f32", [480, 3, 100], "free"),
    ([30, 1, 7], [9, 1, 7], 16, 16, 2, 16, "bf16", [471, 0, 112], "wide"),
    ([40, 60], [33, 60], 64, 16, 1, 32, "f32", [2551, 3840], "free"),  # 16 query heads on one K/V head
    ([12], [12], 64, 128, 4, 64, "bf16", [700], "append"),             # 32 query heads on one
    ([300], [211], 32, 8, 8, 32, "bf16", None, "free"),
    ([20, 9], [20, 3], 32, 128, 1, 8, "f32", [633, 280], "wide"),      # 128 query heads on one
    ([5, 4], [5, 2], 1024, 8, 4, 64, "f32", [5000, 1025], "wide"),
    ([1500], [1500], 64, 1, 1, 64, "bf16", None, "append"),            # one run across every CTA
    ([900, 700], [800, 5], 64, 8, 1, 64, "f32", [57600, 44799], "free"),
    (list(range(1, 61)), [max(1, n // 2) for n in range(1, 61)], 16, 4, 4, 16, "bf16",
     [max(0, 16 * n - n % 17) for n in range(1, 61)], "free"),
    ([2] * 256, [1] * 256, 8, 2, 2, 8, "f32", [(7 * i) % 17 for i in range(256)], "append"),
]


def attn_inputs(lsa, n_b, C, H, Hkv, sb, dtype, lens, scales, seed, k_b):
    r = np.random.default_rng(seed)
    dims = make_dims(lsa, n_b, k_b, C, H, dtype)
    t = R.make_cache(lsa, sum(n_b), Hkv, C, sb, r, scales)
    off = np.concatenate([[0], np.cumsum(n_b)])
    if lens is not None:  # rows and blocks behind the sequences hold NaN
        for b, n in enumerate(n_b):
            first = int(np.clip(lens[b], 0, n * C))
            for name in ("K", "V"):
                codes = t[name + "8"].view(torch.uint8)[off[b]:off[b + 1]]
                sc = t[name.lower() + "_scale"][off[b]:off[b + 1]]
                ch, wi = first // C, first % C
                codes[ch + 1:], sc[ch + 1:] = 0x7F, float("nan")
                if ch < n:
                    codes[ch, :, wi:] = 0x7F
                    sc[ch, :, -(-wi // sb):] = float("nan")
    q = tensor(r.normal(0, 1.5, (len(n_b), H, DH)), dtype)
    cache = lsa.Kv8Cache(dims, Hkv, sb, t["K8"], t["V8"], t["k_scale"], t["v_scale"])
    return dims, cache, q


def tokens_of(ids, C, n, length):
    return [(i, w) for i in ids if 0 <= i < n for w in range(C) if i * C + w < length]


def check_attn(out, lse, q, cache, n_b, C, ids, lens, H, q_err=0.0):
    off = np.concatenate([[0], np.cumsum(n_b)])
    K, V = R.decode(cache.K8), R.decode(cache.V8)
    ks, vs = R.f64(cache.k_scale), R.f64(cache.v_scale)
    for b, n in enumerate(n_b):
        s = slice(off[b], off[b + 1])
        tok = tokens_of(ids[b], C, n, n * C if lens is None else lens[b])
        o, l, A, top = R.attention(R.f64(q[b]), K[s], ks[s], V[s], vs[s], tok)
        to, tl = R.attn_tolerance(A, top, len(tok), q_err)
        if not tok:
            assert bool((out[b] == 0).all()) and bool((lse[b] == -np.inf).all())
            continue
        err = np.abs(R.f64(out[b]) - o).max(-1)
        assert np.all(err <= to), (b, np.max(err / to))
        el = np.abs(R.f64(lse[b]) - l)
        assert np.all(el <= tl + np.abs(l) * 2.0 ** -22), (b, np.max(el / tl))


@pytest.mark.parametrize("n_b,k_b,C,H,Hkv,sb,dtype,lens,scales", ATTN)
@pytest.mark.parametrize("whole", [False, True])
def test_attention(lsa, n_b, k_b, C, H, Hkv, sb, dtype, lens, scales, whole):
    dims, cache, q = attn_inputs(lsa, n_b, C, H, Hkv, sb, dtype, lens, scales, 7 + C + H, k_b)
    ids = [np.arange(n) for n in n_b] if whole else kept_ids(n_b, k_b, 2)
    g = Guards()
    out, lse = g((len(n_b), H, DH), torch.float32), g((len(n_b), H), torch.float32)
    ws = g(lsa.lsa_kv8_workspace_size(dims, cache), torch.uint8)
    lsa.lsa_workspace_init(ws)
    sl = None if lens is None else i32(lens)
    di = None if whole else i32(np.concatenate(ids))
    lsa.lsa_kv8_decode_attn(dims, cache, q, di, None, sl, out, lse, ws)
    g.check()
    check_attn(out, lse, q, cache, n_b, C, ids, lens, H)
    assert lsa.lsa_get_device_status(ws) == lsa.LSA_OK
    again = torch.empty_like(out)
    lsa.lsa_kv8_decode_attn(dims, cache, q, di, None, sl, again, None, ws)
    assert torch.equal(again, out)  # the joins' order is fixed


@pytest.mark.parametrize("H,Hkv", [(4, 4), (16, 2)])
def test_attention_counts_and_bad_ids(lsa, H, Hkv):
    n_b, k_b, C, sb = [9, 9, 9, 9], [5, 5, 5, 5], 16, 16
    dims, cache, q = attn_inputs(lsa, n_b, C, H, Hkv, sb, "f32", None, "free", 3, k_b)
    ws = lsa.alloc_workspace(dims, kv8=cache)
    out, lse = torch.empty(4, H, DH, device="cuda"), torch.empty(4, H, device="cuda")
    ids = [[0, 2, 4, 6, 8], [1, 9, 3, -1, 5], [7, 100, 2 ** 31 - 1, -2 ** 31, -5], [3, 3, 3, 1, 2]]  # a chunk may recur
    counts = [0, 5, 99, -3]
    lsa.lsa_kv8_decode_attn(dims, cache, q, i32(np.concatenate(ids)), i32(counts), None, out, lse, ws)
    used = [ids[b][:max(0, min(5, c))] for b, c in enumerate(counts)]
    check_attn(out, lse, q, cache, n_b, C, used, None, H)
    assert lsa.lsa_get_device_status(ws) == lsa.LSA_ERR_BAD_ID
    lsa.lsa_kv8_decode_attn(dims, cache, q, i32([0, 2, 4, 6, 8] * 4), i32([1, 2, 3, 4]), i32([1, 144, 33, 0]), out, lse, ws)
    check_attn(out, lse, q, cache, n_b, C, [[0, 2, 4, 6, 8][:c] for c in (1, 2, 3, 4)], [1, 144, 33, 0], H)
    lsa.lsa_kv8_decode_attn(dims, cache, q, None, i32([1, 9, 0, 4]), None, out, lse, ws)
    check_attn(out, lse, q, cache, n_b, C, [range(1), range(9), [], range(4)], None, H)
    assert lsa.lsa_get_device_status(ws) == lsa.LSA_OK


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_sharp_and_huge_logits(lsa, dtype):
    """One key that takes nearly all the weight, keys whose logits differ by thousands, a zero query, and queries of very
    unlike size: no overflow, and the tolerance still holds."""
    n_b, C, H, Hkv, sb = [6, 6], 64, 8, 2, 64
    dims, cache, q = attn_inputs(lsa, n_b, C, H, Hkv, sb, dtype, None, "wide", 5, [6, 6])
    q[0, 0] *= 300.0
    q[0, 1] = 0.0
    q[0, 2] *= 1e-20
    q[1, 3] *= 1e4
    q[1, 4, ::2] *= 1e-6
    ws = lsa.alloc_workspace(dims, kv8=cache)
    out, lse = torch.empty(2, H, DH, device="cuda"), torch.empty(2, H, device="cuda")
    lsa.lsa_kv8_decode_attn(dims, cache, q, None, None, None, out, lse, ws)
    off = [0, 6, 12]
    K, V, ks, vs = R.decode(cache.K8), R.decode(cache.V8), R.f64(cache.k_scale), R.f64(cache.v_scale)
    for b in range(2):
        s = slice(off[b], off[b + 1])
        tok = tokens_of(range(6), C, 6, 6 * C)
        o, l, A, top = R.attention(R.f64(q[b]), K[s], ks[s], V[s], vs[s], tok)
        to, tl = R.attn_tolerance(A, top, len(tok))
        # the weights' relative error is at most e^(2 delta) - 1 with delta the logits': where A is large the linear
        # bound does not hold and the sharp softmax's own (max |v| times 2) takes its place
        assert np.all(np.abs(R.f64(out[b]) - o).max(-1) <= np.minimum(2 * top, np.where(A * 2.0 ** -18 < 0.05, 1.1 * to, 2 * top)))
        assert np.all(np.abs(R.f64(lse[b]) - l) <= tl + np.abs(l) * 2.0 ** -22)
    assert bool(torch.isfinite(out).all())


def test_attention_nan_in_used_rows_stays_in_its_head(lsa):
    n_b, C, H, Hkv, sb = [4], 16, 4, 4, 16
    dims, cache, q = attn_inputs(lsa, n_b, C, H, Hkv, sb, "bf16", None, "append", 5, [4])
    ws = lsa.alloc_workspace(dims, kv8=cache)
    out0, out1 = (torch.empty(1, H, DH, device="cuda") for _ in range(2))
    lsa.lsa_kv8_decode_attn(dims, cache, q, None, None, None, out0, None, ws)
    cache.V8.view(torch.uint8)[2, 1, 3, 5] = 0x7F
    cache.K8.view(torch.uint8)[2, 3, 3, 5] = 0xFF
    lsa.lsa_kv8_decode_attn(dims, cache, q, None, None, None, out1, None, ws)
    nan = torch.isnan(out1[0])
    assert bool(nan[1, 5]) and int(nan[1].sum()) == 1 and bool(nan[3].all()) and not bool(nan[[0, 2]].any())
    assert torch.equal(out1[0][[0, 2]], out0[0][[0, 2]])


def test_attention_agrees_with_the_wide_cache(lsa):
    """Read back to fp32, the chunks give the same attention through lsa_sparse_decode_attn."""
    n_b, k_b, C, H, sb = [40, 25], [11, 25], 64, 8, 32
    dims, cache, q = attn_inputs(lsa, n_b, C, H, H, sb, "f32", None, "append", 6, k_b)
    ws = lsa.alloc_workspace(dims, kv8=cache)
    ids = i32(np.concatenate(kept_ids(n_b, k_b, 4)))
    K, V = (torch.empty(36 * C, H, DH, device="cuda") for _ in range(2))
    lsa.lsa_kv8_gather(dims, cache, ids, None, K, V, ws)
    a, b, la, lb = (torch.empty(2, H, *x, device="cuda") for x in ((DH,), (DH,), (), ()))
    lsa.lsa_sparse_decode_attn(dims, q, K, V, None, a, la, ws)
    lsa.lsa_kv8_decode_attn(dims, cache, q, ids, None, None, b, lb, ws)
    top = float(V.abs().max())
    assert float((a - b).abs().max()) <= 2.0 ** -14 * top and float((la - lb).abs().max()) <= 1e-4


def test_two_graphs_share_a_workspace(lsa):
    """Two captured attentions of unlike shapes on one workspace, replayed in turn: each gives what it gives alone."""
    n_b, k_b, C, H, Hkv, sb = [200, 90], [100, 90], 64, 8, 2, 64
    dims, cache, q = attn_inputs(lsa, n_b, C, H, Hkv, sb, "bf16", None, "free", 8, k_b)
    ids = i32(np.concatenate(kept_ids(n_b, k_b, 5)))
    ws = lsa.alloc_workspace(dims, kv8=cache)
    outs = [torch.empty(2, H, DH, device="cuda") for _ in range(4)]
    lsa.lsa_kv8_decode_attn(dims, cache, q, ids, None, None, outs[0], None, ws)
    lsa.lsa_kv8_decode_attn(dims, cache, q, None, None, None, outs[1], None, ws)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    with torch.cuda.graph(graphs[0]):
        lsa.lsa_kv8_decode_attn(dims, cache, q, ids, None, None, outs[2], None, ws)
    with torch.cuda.graph(graphs[1]):
        lsa.lsa_kv8_decode_attn(dims, cache, q, None, None, None, outs[3], None, ws)
    for _ in range(3):
        graphs[0].replay()
        graphs[1].replay()
    assert torch.equal(outs[2], outs[0]) and torch.equal(outs[3], outs[1])


def test_calls_on_another_stream(lsa):
    n_b, k_b, C, H, Hkv, sb = [50], [20], 64, 8, 8, 64
    dims, cache, q = attn_inputs(lsa, n_b, C, H, Hkv, sb, "bf16", None, "free", 9, k_b)
    ids = i32(np.concatenate(kept_ids(n_b, k_b, 5)))
    ws = lsa.alloc_workspace(dims, kv8=cache)
    a, b = (torch.empty(1, H, DH, device="cuda") for _ in range(2))
    lsa.lsa_kv8_decode_attn(dims, cache, q, ids, None, None, a, None, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    big = torch.randn(4096, 4096, device="cuda")
    with torch.cuda.stream(side):
        for _ in range(4):
            big = big @ big * 1e-4
        q2 = q * 2
        lsa.lsa_kv8_decode_attn(dims, cache, q2, ids, None, None, b, None, ws)  # after its input, on the same stream
    torch.cuda.synchronize()
    lsa.lsa_kv8_decode_attn(dims, cache, q * 2, ids, None, None, a, None, ws)
    assert torch.equal(a, b)


def test_ids_in_any_order_and_twice(lsa):
    """Kept chunks need not be sorted, and one that is named twice counts twice."""
    n_b, k_b, C, H, Hkv, sb = [12, 5], [6, 4], 16, 8, 2, 8
    lens = [190, 70]
    dims, cache, q = attn_inputs(lsa, n_b, C, H, Hkv, sb, "bf16", lens, "free", 31, k_b)
    ids = [[11, 3, 3, 0, 11, 7], [4, 4, 4, 4]]
    ws = lsa.alloc_workspace(dims, kv8=cache)
    out, lse = torch.empty(2, H, DH, device="cuda"), torch.empty(2, H, device="cuda")
    lsa.lsa_kv8_decode_attn(dims, cache, q, i32(sum(ids, [])), None, i32(lens), out, lse, ws)
    check_attn(out, lse, q, cache, n_b, C, ids, lens, H)
    K, V = (torch.zeros(sum(k_b) * C, Hkv, DH, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lsa.lsa_kv8_gather(dims, cache, i32(sum(ids, [])), i32(lens), K, V, ws)
    assert torch.equal(K[C:2 * C], K[2 * C:3 * C]) and torch.equal(V[:6 * C][:C], V[4 * C:5 * C])
    assert lsa.lsa_get_device_status(ws) == lsa.LSA_OK


def test_offsets_past_32_bits(lsa):
    """A cache whose codes pass 2^32 bytes: its last chunks written, read back and attended to, as those of a small one."""
    C, H, Hkv, sb, far = 64, 32, 16, 64, 33000  # 128 KB a chunk: 4.3 GB each of K and V
    n_b, k_b = [far, 3], [4, 3]
    dims = make_dims(lsa, n_b, k_b, C, H, "bf16")
    small = make_dims(lsa, [4, 3], k_b, C, H, "bf16")
    big, ref = lsa.alloc_kv8_cache(dims, Hkv, sb), lsa.alloc_kv8_cache(small, Hkv, sb)
    assert big.K8.numel() > 2 ** 32
    r = np.random.default_rng(6)
    rows = tensor(r.normal(0, 1, (2, 250, 2 * Hkv, DH)), "bf16")
    q = tensor(r.normal(0, 1, (2, H, DH)), "bf16")
    ids, lens = np.arange(4), [4 * C - 1, 150]
    got = []
    for d, cache, first in ((dims, big, far - 4), (small, ref, 0)):
        ws = lsa.alloc_workspace(d, kv8=cache)
        lsa.lsa_kv8_append(d, cache, None, rows[:, :, :Hkv], rows[:, :, Hkv:], i32([first * C + 5, 1]), i32([250, 149]), ws)
        di, sl = i32(np.concatenate([first + ids, np.arange(3)])), i32([first * C + lens[0], lens[1]])
        out, lse = torch.empty(2, H, DH, device="cuda"), torch.empty(2, H, device="cuda")
        lsa.lsa_kv8_decode_attn(d, cache, q, di, None, sl, out, lse, ws)
        K, V = (torch.zeros(7 * C, Hkv, DH, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        lsa.lsa_kv8_gather(d, cache, di, sl, K, V, ws)
        assert lsa.lsa_get_device_status(ws) == lsa.LSA_OK
        got.append((out, lse, K, V, cache.K8[first:].view(torch.uint8), cache.v_scale[first:]))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    check_attn(got[1][0], got[1][1], q, ref, [4, 3], C, [ids, np.arange(3)], lens, H)
    assert not bool(big.K8.view(torch.uint8)[:far - 4].any())


def test_two_streams_at_once(lsa):
    """Two streams, each with its workspace, over one cache: attention of the one beside the read-back of the other."""
    n_b, k_b, C, H, Hkv, sb = [400, 300], [300, 300], 64, 8, 8, 64
    dims, cache, q = attn_inputs(lsa, n_b, C, H, Hkv, sb, "bf16", None, "free", 19, k_b)
    ids = i32(np.concatenate(kept_ids(n_b, k_b, 5)))
    streams = [torch.cuda.Stream() for _ in range(2)]
    wss = [lsa.alloc_workspace(dims, kv8=cache) for _ in range(2)]
    rows = sum(k_b) * C

    def calls(which, ws):
        out, lse = torch.empty(2, H, DH, device="cuda"), torch.empty(2, H, device="cuda")
        K, V = (torch.empty(rows, Hkv, DH, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        for _ in range(5):
            lsa.lsa_kv8_decode_attn(dims, cache, q * (1 + which), ids if which else None, None, None, out, lse, ws)
            lsa.lsa_kv8_gather(dims, cache, ids, None, K, V, ws)
        return out, lse, K, V

    want = [calls(i, wss[0]) for i in range(2)]
    torch.cuda.synchronize()
    got = []
    for i in range(2):
        with torch.cuda.stream(streams[i]):
            got.append(calls(i, wss[i]))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


# ---------------------------------------------------------------- the whole step
def step_inputs(lsa, dtype, H, Hkv, seed, B=3, Q=1):
    r = np.random.default_rng(seed)
    n_b, k_b, C, sb, E = [30, 12, 41][:B], [7, 12, 5][:B], 32, 16, 64
    dims = make_dims(lsa, n_b, k_b, C, H, dtype, E=E, Q=Q)
    t = R.make_cache(lsa, sum(n_b), Hkv, C, sb, r)
    cache = lsa.Kv8Cache(dims, Hkv, sb, t["K8"], t["V8"], t["k_scale"], t["v_scale"])
    emb, qe = tensor(r.normal(0, 1, (sum(n_b), E)), dtype), tensor(r.normal(0, 1, (B, Q, E)), dtype)
    qkv = tensor(r.normal(0, 1.5, (B, H + 2 * Hkv, DH)), dtype)
    lens = i32([n * C - 1 - 5 * i for i, n in enumerate(n_b)])
    return n_b, k_b, C, sb, dims, t, cache, emb, qe, qkv, lens


@pytest.mark.parametrize("dtype,H,Hkv,rot,Q", [("bf16", 16, 2, 128, 1), ("f32", 4, 4, 64, 1), ("bf16", 8, 8, 32, 64)])
@pytest.mark.parametrize("with_prep", [True, False])
def test_step_is_its_parts(lsa, dtype, H, Hkv, rot, Q, with_prep):
    """The fused step over several tokens, each compared bit for bit with the calls it is made of."""
    n_b, k_b, C, sb, dims, t, cache, emb, qe, qkv, lens = step_inputs(lsa, dtype, H, Hkv, 21, Q=Q)
    _, _, inv, w = prep_inputs(1, 1, 1, dtype, rot, True, 2, 15)
    prep = lsa.QkPrep(rot, inv, *w, eps=1e-6) if with_prep else None
    twin = lsa.Kv8Cache(dims, Hkv, sb, *(t[n].clone() for n in ("K8", "V8", "k_scale", "v_scale")))
    ws, ws2 = lsa.alloc_workspace(dims, kv8=cache), lsa.alloc_workspace(dims, kv8=cache)
    kept = sum(k_b)
    ids, ids2 = (torch.empty(kept, dtype=torch.int32, device="cuda") for _ in range(2))
    out, out2 = (torch.empty(3, H, DH, device="cuda") for _ in range(2))
    lse, lse2 = (torch.empty(3, H, device="cuda") for _ in range(2))
    scores = torch.empty(sum(n_b), device="cuda")
    for step in range(7):  # the second sequence reaches its end on the way
        x = qkv * (1.0 + step)
        q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
        qs = q if with_prep else q.contiguous()
        lsa.lsa_decode_step_kv8(dims, cache, prep, qe, emb, qs, k, v, lens, ids, out, lse, ws)
        lsa.lsa_kv8_append(dims, twin, prep, k[:, None], v[:, None], lens, None, ws2)
        qp = q.contiguous()
        if with_prep:
            lsa.lsa_qk_norm_rope(dims, prep, lens, qp, None, qp, None)
        lsa.lsa_score_chunks(dims, qe, emb, scores, ws2)
        lsa.lsa_topk_select(dims, scores, ids2, ws2)
        lens += 1
        lsa.lsa_kv8_decode_attn(dims, twin, qp, ids2, None, lens, out2, lse2, ws2)
        assert torch.equal(ids, ids2) and torch.equal(out, out2) and torch.equal(lse, lse2)
        for n in ("K8", "V8", "k_scale", "v_scale"):
            assert torch.equal(getattr(cache, n).view(torch.uint8), getattr(twin, n).view(torch.uint8)), n
        s = lsa.lsa_get_device_status(ws)
        assert s == lsa.lsa_get_device_status(ws2)
        assert s == (lsa.LSA_ERR_BAD_ID if step >= 1 else lsa.LSA_OK)  # the first sequence is full after one token


def test_step_against_the_definitions(lsa):
    """Prepare, write, select and attend, against the 64-bit forms of each; then without new rows."""
    n_b, k_b, C, sb, dims, t, cache, emb, qe, qkv, lens = step_inputs(lsa, "f32", 8, 4, 22)
    H, Hkv, rot = 8, 4, 128
    _, _, inv, w = prep_inputs(1, 1, 1, "f32", rot, True, 2, 16)
    ws = lsa.alloc_workspace(dims, kv8=cache)
    ids = torch.empty(sum(k_b), dtype=torch.int32, device="cuda")
    out, lse = torch.empty(3, H, DH, device="cuda"), torch.empty(3, H, device="cuda")
    q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    before = {n: x.clone() for n, x in t.items()}
    lsa.lsa_decode_step_kv8(dims, cache, lsa.QkPrep(rot, inv, *w, eps=1e-6), qe, emb, q, k, v, lens, ids, out, lse, ws)
    pos = lens.cpu().numpy()
    kp = R.norm_rope(R.f64(k), pos, R.f64(inv), R.f64(w[1]), rot, False, 1e-6)
    off = np.concatenate([[0], np.cumsum(n_b)])
    for name, rows in (("K", kp), ("V", R.f64(v))):
        vals, sc = R.decode(before[name + "8"]), R.f64(before[name.lower() + "_scale"])
        for b in range(3):
            R.append(vals, sc, rows[b][None], int(off[b]), n_b[b], C, sb, int(pos[b]))
        assert np.array_equal(R.f64(getattr(cache, name.lower() + "_scale")), sc)
        got = R.decode(getattr(cache, name + "8"))
        # a prepared key is off by fp32 rounding, which may cross a border of e4m3: one step, hardly ever
        assert np.all(np.abs(got - vals) <= np.maximum(np.abs(vals), 2.0 ** -6) * 2.0 ** -3 * 1.01)
        assert np.mean(got != vals) < 1e-4
    qp = R.norm_rope(R.f64(q), pos, R.f64(inv), R.f64(w[0]), rot, False, 1e-6)
    kept = np.split(ids.cpu().numpy(), np.cumsum(k_b)[:-1])
    for b in range(3):
        s = R.f64(emb)[off[b]:off[b + 1]] @ R.f64(qe)[b, 0]
        G.check_ids(kept[b], np.sort(np.lexsort((np.arange(n_b[b]), -s))[:k_b[b]]), s, k_b[b])
    check_attn(out, lse, torch.from_numpy(qp), cache, n_b, C, kept, [int(x) + 1 for x in pos], H, 40 * 2.0 ** -24)
    lsa.lsa_decode_step_kv8(dims, cache, None, qe, emb, q.contiguous(), None, None, lens, ids, out, lse, ws)
    check_attn(out, lse, q, cache, n_b, C, np.split(ids.cpu().numpy(), np.cumsum(k_b)[:-1]), pos.tolist(), H)
    assert lsa.lsa_get_device_status(ws) == lsa.LSA_OK


def test_decode_loop_in_a_graph(lsa):
    """A captured step replayed for a run of tokens: the cache, lengths and outputs of eager steps."""
    n_b, k_b, C, sb, dims, t, cache, emb, qe, qkv, lens = step_inputs(lsa, "bf16", 8, 2, 23)
    H, Hkv = 8, 2
    lens = i32([40, 0, 900])
    _, _, inv, w = prep_inputs(1, 1, 1, "bf16", 128, True, 2, 17)
    prep = lsa.QkPrep(128, inv, *w, eps=1e-6)
    start = {n: x.clone() for n, x in t.items()}
    ws = lsa.alloc_workspace(dims, kv8=cache)
    ids = torch.empty(sum(k_b), dtype=torch.int32, device="cuda")
    out, lse = torch.empty(3, H, DH, device="cuda"), torch.empty(3, H, device="cuda")
    x = torch.empty_like(qkv)

    def step():
        lsa.lsa_decode_step_kv8(dims, cache, prep, qe, emb, x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:], lens, ids, out,
                                lse, ws)
        lens.add_(1)

    def loop(one):
        for n in t:
            t[n].copy_(start[n])
        lens.copy_(i32([40, 0, 900]))
        got = []
        for i in range(40):
            x.copy_(qkv * (0.2 + 0.1 * i))
            one()
            got.append((out.clone(), lse.clone()))
        return got, {n: y.clone() for n, y in t.items()}

    a, ca = loop(step)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    b, cb = loop(graph.replay)
    for (o, l), (p, m) in zip(a, b):
        assert torch.equal(o, p) and torch.equal(l, m)
    for n in ca:
        assert torch.equal(ca[n].view(torch.uint8), cb[n].view(torch.uint8))
    assert lsa.lsa_get_device_status(ws) == lsa.LSA_OK


def test_random_shapes(lsa):
    """Seeded random batches through write, read-back and attention."""
    for seed in range(30):
        r = np.random.default_rng(1000 + seed)
        C = int(r.choice([8, 16, 32, 64, 128]))
        sb = int(r.choice([s for s in (8, 16, 32, 64) if s <= C]))
        Hkv = int(r.choice([1, 2, 4, 8]))
        H = Hkv * int(r.choice([1, 2, 4, 8, 16]))
        B = int(r.integers(1, 6))
        n_b = r.integers(1, 40, B).tolist()
        k_b = [int(r.integers(1, n + 1)) for n in n_b]
        dtype = ["bf16", "f32"][seed % 2]
        lens = [int(r.integers(0, n * C + 1)) for n in n_b]
        dims, cache, q = attn_inputs(lsa, n_b, C, H, Hkv, sb, dtype, lens, "append", seed, k_b)
        ws = lsa.alloc_workspace(dims, kv8=cache)
        before = {n: getattr(cache, n).clone() for n in ("K8", "V8", "k_scale", "v_scale")}
        n = int(r.integers(1, 90))
        counts = [int(min(r.integers(0, n + 1), m * C - x)) for m, x in zip(n_b, lens)]
        rows = tensor(r.normal(0, 1, (B, n, 2 * Hkv, DH)), dtype)
        lsa.lsa_kv8_append(dims, cache, None, rows[:, :, :Hkv], rows[:, :, Hkv:], i32(lens), i32(counts), ws)
        after = {m: getattr(cache, m) for m in before}
        check_append(before, after, R.f64(rows[:, :, :Hkv]), n_b, C, sb, lens, counts, "K")
        check_append(before, after, R.f64(rows[:, :, Hkv:]), n_b, C, sb, lens, counts, "V")
        lens = [x + c for x, c in zip(lens, counts)]
        ids = kept_ids(n_b, k_b, seed)
        out, lse = torch.empty(B, H, DH, device="cuda"), torch.empty(B, H, device="cuda")
        lsa.lsa_kv8_decode_attn(dims, cache, q, i32(np.concatenate(ids)), None, i32(lens), out, lse, ws)
        check_attn(out, lse, q, cache, n_b, C, ids, lens, H)
        assert lsa.lsa_get_device_status(ws) == lsa.LSA_OK
