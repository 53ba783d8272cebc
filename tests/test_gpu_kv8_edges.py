"""GPU tests of the 8-bit K/V cache at values and sizes where a kernel's own number format, split or plan could show:
non-finite queries, V scales of very unlike size, scales at the ends of the range under new rows, chunks
that hold no token yet, one key that takes all the weight, many K/V heads."""
import numpy as np
import pytest
import torch

from tests import _kv8 as R
from tests.test_gpu_kv8 import append_case, attn_inputs, check_append, i32, kept_ids, make_dims, prep_inputs, tensor

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


# ---------------------------------------------------------------- V's scales
def attention_and_bounds(q, K, V, ks, vs):
    """One sequence over all its tokens in 64 bits. q [H][128]; K, V code values [n][Hkv][C][128]; scales
    [n][Hkv][C/sb]. -> out, lse and their bounds, out's for each value.

    With u = 2^-24 and p the normalised weights: a logit is off by delta = 2^-18 (A_t + A_max), A_t = sum |q k| / sqrt(128)
    of its token and A_max of the one with the largest logit (q's halves 2^-22 of sum |q k|, fp32 sums that truncate
    2^-20, scales and differences 4 u), which changes p_t v_t in the sum over tokens and p_t in the one that divides it.
    Weights, their f16 halves and the joins: 2^-20 each at most, 2^-18 together. Sums with truncation: 2^-23 for each
    of at most n / 16 steps, and 64 for the joins, in both sums. All of these are relative to sum p |v| of the value's
    own column. What is not: the low f16 half ends at 2^-24, half a step of it is 2^-25, and products p vs are brought
    to 2^13 at least, so a token's is off by up to 2^-38 of the largest, times a code of up to 448. And a weight below
    2^-125 of the largest may count as 0."""
    H, Hkv, C = q.shape[0], K.shape[1], K.shape[2]
    sb = C // ks.shape[2]
    out, lse, tol, tol_l = np.zeros((H, DH)), np.zeros(H), np.zeros((H, DH)), np.zeros(H)
    for h in range(H):
        kv = h // (H // Hkv)
        s = np.repeat(vs[:, kv], sb, -1).reshape(-1)
        k = K[:, kv].reshape(-1, DH) * np.repeat(ks[:, kv], sb, -1).reshape(-1, 1)
        v = V[:, kv].reshape(-1, DH) * s[:, None]
        n = len(k)
        logit = k @ q[h] / np.sqrt(DH)
        A = np.abs(k) @ np.abs(q[h]) / np.sqrt(DH)
        top = logit.argmax()
        p = np.exp(logit - logit[top])
        total = p.sum()
        lse[h], p = logit[top] + np.log(total), p / total
        out[h], size = p @ v, p @ np.abs(v)
        delta = np.expm1(2.0 ** -18 * (A + A[top]))
        steps = (n / 16 + 64) * 2.0 ** -23
        lost = p < 2.0 ** -125 * p[top]
        tol[h] = ((p * delta) @ np.abs(v) + size * (p @ delta) + size * (2.0 ** -18 + 2 * steps)
                  + n * 2.0 ** -38 * 448 * (p * s).max() + p[lost] @ np.abs(v[lost]))
        tol_l[h] = p @ delta + 2.0 ** -18 * (1 + A[top]) + steps + 2.0 ** -22 * abs(lse[h])
    return out, lse, tol, tol_l


def scaled_cache(lsa, n, C, H, Hkv, sb, dtype, exponents, seed, low=()):
    """One sequence whose K are N(0, 1) and whose V codes are random, with V's scales 2^exponents [n][Hkv][C/sb]. The keys
    of the chunks `low`, {chunk: logit}, give about that logit with the queries, which are multiples of one row."""
    r = np.random.default_rng(seed)
    dims = make_dims(lsa, [n], [n], C, H, dtype)
    base = r.normal(0, 1.5, DH)
    q = tensor((base * (1 + 0.01 * np.arange(H))[:, None])[None], dtype)
    K = r.normal(0, 1, (n, Hkv, C, DH))
    for c, logit in dict(low).items():
        K[c] = base * (logit * np.sqrt(DH) / (base @ base)) * r.uniform(0.97, 1.03, (Hkv, C, 1))
    ks = np.exp2(np.ceil(np.log2(np.maximum(np.abs(K).reshape(n, Hkv, C // sb, -1).max(-1), 1e-3) / 448)))
    k8 = torch.from_numpy(K / np.repeat(ks, sb, -1)[..., None]).float().cuda().to(torch.float8_e4m3fn)
    c = r.integers(0, 256, (n, Hkv, C, DH), dtype=np.uint8)
    c[(c & 127) == 127] = 0x30
    f32 = [torch.from_numpy(x.astype(np.float32)).cuda() for x in (ks, np.exp2(exponents))]
    cache = lsa.Kv8Cache(dims, Hkv, sb, k8, torch.from_numpy(c).cuda(), *f32)
    return dims, cache, q


def check_scaled(lsa, dims, cache, q):
    H = q.shape[1]
    out, lse = torch.empty(1, H, DH, device="cuda"), torch.empty(1, H, device="cuda")
    ws = lsa.alloc_workspace(dims, kv8=cache)
    lsa.lsa_kv8_decode_attn(dims, cache, q, None, None, None, out, lse, ws)
    o, l, to, tl = attention_and_bounds(R.f64(q[0]), R.decode(cache.K8), R.decode(cache.V8), R.f64(cache.k_scale),
                                        R.f64(cache.v_scale))
    assert np.all(np.abs(o).max(-1) > 50 * to.max(-1))  # no output of zeros, or of a few bits, is within the bounds
    assert np.all(np.abs(R.f64(out[0]) - o) <= to), np.max(np.abs(R.f64(out[0]) - o) / to)
    assert np.all(np.abs(R.f64(lse[0]) - l) <= tl), np.max(np.abs(R.f64(lse[0]) - l) / tl)


# chunks, C, H, Hkv, sb, dtype: one part and cut runs, every grouping of heads
SHAPES = [(6, 64, 4, 4, 64, "f32"), (30, 16, 8, 1, 16, "bf16"), (600, 32, 2, 1, 32, "bf16"), (600, 32, 16, 1, 8, "f32"),
          (90, 64, 32, 8, 64, "bf16")]


@pytest.mark.parametrize("n,C,H,Hkv,sb,dtype", SHAPES)
@pytest.mark.parametrize("e", [20, 30, 40, 70, 100])
@pytest.mark.parametrize("where", [0.0, 0.5, 1.0])
def test_a_block_of_large_v_that_is_hardly_attended(lsa, n, C, H, Hkv, sb, dtype, e, where):
    """A chunk whose V are 2^e times larger and whose weights are 2^-e e^-8 of the others': it adds little, and takes no
    bits from the rest."""
    at = int(where * (n - 1))
    exps = np.full((n, Hkv, C // sb), -6.0)
    exps[at] += e
    check_scaled(lsa, *scaled_cache(lsa, n, C, H, Hkv, sb, dtype, exps, 50 + e, {at: -e * np.log(2) - 8}))


@pytest.mark.parametrize("n,C,H,Hkv,sb,dtype", SHAPES)
@pytest.mark.parametrize("kind", ["rising", "falling", "random", "least", "largest"])
def test_v_scales_of_all_sizes(lsa, n, C, H, Hkv, sb, dtype, kind):
    """Scales from 2^-120 to 2^110 over the sequence, in order and in none, and all of them at an end of the range."""
    m = n * (C // sb)
    e = {"rising": np.linspace(-120, 110, m), "falling": np.linspace(110, -120, m),
         "random": np.random.default_rng(9).uniform(-120, 110, m), "least": np.full(m, -120.0),
         "largest": np.full(m, 110.0)}[kind]
    exps = np.round(e).reshape(n, 1, C // sb).repeat(Hkv, 1)
    check_scaled(lsa, *scaled_cache(lsa, n, C, H, Hkv, sb, dtype, exps, 60))


@pytest.mark.parametrize("n,C,H,Hkv,sb,dtype", SHAPES)
def test_logits_that_rise_while_v_scales_fall(lsa, n, C, H, Hkv, sb, dtype):
    """Each chunk's weights are up to 2^90 times the first's and its scales as many times smaller, so that all of them
    count: the carried output is rescaled at every step, by weights and by scales in turn."""
    bits = np.round(np.linspace(0, 90, n))
    exps = (20 - bits)[:, None, None].repeat(Hkv, 1).repeat(C // sb, 2)
    check_scaled(lsa, *scaled_cache(lsa, n, C, H, Hkv, sb, dtype, exps, 61,
                                    {c: (bits[c] - 90) * np.log(2) for c in range(n)}))


# ---------------------------------------------------------------- the write
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("e", [-126, -121, -120, 0, 119, 120, 121, 126, 127])
def test_append_to_blocks_whose_scale_is_at_an_end_of_the_range(lsa, dtype, e):
    """Rows of all sizes written behind older tokens, in blocks that came with a scale of 2^e: quotients by a power of two
    are exact, so the codes are those of the definition."""
    n_b, C, Hkv, sb, n, start = [2], 32, 2, 16, 20, 5
    dims = make_dims(lsa, n_b, [1], C, 2, dtype)
    r = np.random.default_rng(70)
    t = R.make_cache(lsa, 2, Hkv, C, sb, r)
    for name in ("k_scale", "v_scale"):
        t[name].fill_(2.0 ** e)
    size = np.exp2(np.where(np.arange(n) % 3 == 0, 126.0, r.uniform(-130, 126, n)))[None, :, None, None]
    size[:, :11] *= 1.0 if e >= 0 else 2.0 ** -240  # below 0 the first block's scale stays as it is
    x = np.clip(r.normal(0, 1, (1, n, 2 * Hkv, DH)) * size, -3.3e38, 3.3e38)
    x[0, 3, :, :8] = 3.0 * 2.0 ** np.clip(np.arange(8) + e - 9.0, -149, 126)  # in and out of the codes' subnormals
    rows = tensor(x.astype(np.float32), dtype)
    before = {m: y.clone() for m, y in t.items()}
    cache = lsa.Kv8Cache(dims, Hkv, sb, t["K8"], t["V8"], t["k_scale"], t["v_scale"])
    ws = lsa.alloc_workspace(dims, kv8=cache)
    lsa.lsa_kv8_append(dims, cache, None, rows[:, :, :Hkv], rows[:, :, Hkv:], i32([start]), None, ws)
    check_append(before, t, R.f64(rows[:, :, :Hkv]), n_b, C, sb, [start], None, "K")
    check_append(before, t, R.f64(rows[:, :, Hkv:]), n_b, C, sb, [start], None, "V")
    assert lsa.lsa_get_device_status(ws) == lsa.LSA_OK
    if e == 127:  # not all of them round to 0
        assert bool((R.decode(t["K8"])[0, :, start:sb] != 0).any())


# ---------------------------------------------------------------- the step's selection
@pytest.mark.parametrize("N,k", [(12, 5), (12, 12), (300, 40), (1000, 7), (5000, 300), (33000, 64), (400000, 33)])
def test_the_step_keeps_chunks_that_hold_tokens(lsa, N, k):
    """Chunks behind a sequence's length have embeddings that would win, lose or be NaN, and are named only where too few
    others are left. Sizes for every form of the selection."""
    C, H, Hkv, E = 8, 2, 1, 4
    lens = [N * C - 1, 0, 3 * C, 3 * C - 1, N * C // 2, (N - 1) * C]
    B = len(lens) if N < 100000 else 2
    lens = lens[:B] if N < 100000 else [N * C // 3, 5 * C + 1]
    r = np.random.default_rng(N)
    dims = make_dims(lsa, [N] * B, [k] * B, C, H, "f32", E=E)
    cache = lsa.alloc_kv8_cache(dims, Hkv, 8)
    cache.k_scale.fill_(2.0 ** -6)
    cache.v_scale.fill_(2.0 ** -6)
    for c in (cache.K8, cache.V8):
        c.view(torch.uint8).random_(0, 126)
    scores = -r.permutation(B * N).astype(np.float64) - 1
    emb = np.zeros((B * N, E), dtype=np.float32)
    emb[:, 0] = scores
    empty = np.arange(N) >= -(-(np.asarray(lens)[:, None] + 1) // C)  # once the new token is there
    fill = np.array([0.0, np.nan, np.inf, -np.inf, 1e30, -1e30], dtype=np.float32)
    emb[empty.reshape(-1)] = fill[np.arange(empty.sum()) % 6][:, None]
    emb[0, 1:] = 0.0
    qe = np.zeros((B, 1, E), dtype=np.float32)
    qe[:, :, 0] = 1.0
    emb, qe = tensor(emb, "f32"), tensor(qe, "f32")
    qkv = tensor(r.normal(0, 1, (B, H + 2 * Hkv, DH)), "f32")
    q, kk, v = qkv[:, :H].contiguous(), qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    ws = lsa.alloc_workspace(dims, kv8=cache)
    ids = torch.full((B * k,), -7, dtype=torch.int32, device="cuda")
    out, out2, lse, lse2 = (torch.empty(B, H, *x, device="cuda") for x in ((DH,), (DH,), (), ()))
    for write in (True, False):
        live = [-(-(n + write) // C) for n in lens]
        lsa.lsa_decode_step_kv8(dims, cache, None, qe, emb, q, kk if write else None, v if write else None, i32(lens), ids,
                                out, lse, ws)
        got = ids.view(B, k).cpu().numpy()
        for b, n in enumerate(live):
            s = scores[b * N:b * N + n]
            want = np.sort(np.argsort(-s, kind="stable")[:k])
            want = np.concatenate([want, np.arange(n, n + max(0, k - n))])
            assert np.array_equal(got[b], want), (b, n)
        lsa.lsa_kv8_decode_attn(dims, cache, q, ids, None, i32([n + write for n in lens]), out2, lse2, ws)
        assert torch.equal(out, out2) and torch.equal(lse, lse2)
        assert lsa.lsa_get_device_status(ws) == lsa.LSA_OK


# ---------------------------------------------------------------- sharp softmax
@pytest.mark.parametrize("n,C,H,Hkv,sb,dtype", SHAPES)
@pytest.mark.parametrize("at", [0, 17, -1])
def test_one_key_that_takes_all_the_weight(lsa, n, C, H, Hkv, sb, dtype, at):
    """Queries of sizes 1 to 10000 and a key whose logit is 40 and more above all others: the output is that token's V. Its
    own weight cancels in the quotient, so what is left is the halves and sums (2^-18 and 2^-23 a step, relative), the
    low halves' end, 2^-38 of its scale times the largest code for each token, and what the other tokens weigh."""
    r = np.random.default_rng(80 + n)
    at = at % (n * C)
    exps = r.integers(-10, -2, (n, Hkv, C // sb)).astype(np.float64)
    dims, cache, q = scaled_cache(lsa, n, C, H, Hkv, sb, dtype, exps, 81)
    q = (q.double() * torch.logspace(0, 4, H, dtype=torch.float64, device="cuda")[:, None]).to(q.dtype)
    base = R.f64(q[0, 0])
    key = torch.from_numpy(2.0 * base / 2.0 ** -5).float().cuda().to(torch.float8_e4m3fn)  # its block's scale becomes 2^-5
    cache.k_scale[at // C, :, at % C // sb] = 2.0 ** -5
    cache.K8[at // C, :, at % C] = key
    K, V, ks, vs = R.decode(cache.K8), R.decode(cache.V8), R.f64(cache.k_scale), R.f64(cache.v_scale)
    out, lse = torch.empty(1, H, DH, device="cuda"), torch.empty(1, H, device="cuda")
    lsa.lsa_kv8_decode_attn(dims, cache, q, None, None, None, out, lse, lsa.alloc_workspace(dims, kv8=cache))
    for h in range(H):
        kv, x = h // (H // Hkv), R.f64(q[0, h])
        k = K[:, kv].reshape(-1, DH) * np.repeat(ks[:, kv], sb, -1).reshape(-1, 1)
        logit = k @ x / np.sqrt(DH)
        A = np.abs(k) @ np.abs(x) / np.sqrt(DH)
        assert logit.argmax() == at
        gap = (logit[at] - logit - 2.0 ** -18 * (A + A[at]))[np.arange(len(logit)) != at].min()
        assert gap > 30.0  # 40 and more, but for what the logits may be off
        s = vs[at // C, kv, at % C // sb]
        v = V[at // C, kv, at % C] * s
        steps = (len(logit) / 16 + 64) * 2.0 ** -23
        rest = len(logit) * np.exp(-gap) * 448 * vs.max()
        tol = np.abs(v) * (2.0 ** -18 + 2 * steps) + len(logit) * 448 * 2.0 ** -38 * s + 2 * rest
        assert np.all(np.abs(R.f64(out[0, h]) - v) <= tol), (h, np.max(np.abs(R.f64(out[0, h]) - v) / tol))
        tol = 2.0 ** -18 * A[at] + 2.0 ** -18 + steps + 2 * len(logit) * np.exp(-gap) + 2.0 ** -22 * abs(logit[at])
        assert abs(float(lse[0, h]) - logit[at]) <= tol


# ---------------------------------------------------------------- many K/V heads
@pytest.mark.parametrize("Hkv", [32, 64, 128])
@pytest.mark.parametrize("dtype,B,n", [("bf16", 1, 1), ("f32", 2, 1), ("bf16", 3, 70), ("f32", 2, 130), ("bf16", 6, 300)])
def test_append_of_many_heads(lsa, dtype, B, n, Hkv):
    """Rows as they are against the definition, prepared ones against the two separate calls."""
    C, sb = 64, 32
    n_b = [n // C + 2 + b % 2 for b in range(B)]
    starts, counts = [(29 * b + 5) % 65 for b in range(B)], [max(1, n - 13 * b) for b in range(B)]
    dims, t, k, v = append_case(lsa, n_b, C, Hkv, sb, dtype, n, 90 + B, 1.5)
    got = [{m: x.clone() for m, x in t.items()} for _ in range(3)]
    ca, cb, cc = (lsa.Kv8Cache(dims, Hkv, sb, y["K8"], y["V8"], y["k_scale"], y["v_scale"]) for y in got)
    ws = lsa.alloc_workspace(dims, kv8=ca)
    lsa.lsa_kv8_append(dims, ca, None, k, v, i32(starts), i32(counts), ws)
    check_append(t, got[0], R.f64(k), n_b, C, sb, starts, counts, "K")
    check_append(t, got[0], R.f64(v), n_b, C, sb, starts, counts, "V")
    _, _, inv, w = prep_inputs(1, 1, 1, dtype, 128, True, 2, 14)
    for inter in (False, True):
        prep = lsa.QkPrep(128, inv, None, w[1], 1e-5, inter)
        for c in got[1:]:
            for m in t:
                c[m].copy_(t[m])
        lsa.lsa_kv8_append(dims, cb, prep, k, v, i32(starts), i32(counts), ws)
        pos = (torch.tensor(starts)[:, None] + torch.arange(n)).to(torch.int32).cuda()
        kp = torch.empty((B, n, Hkv, DH), dtype=k.dtype, device="cuda")
        lsa.lsa_qk_norm_rope(dims, prep, pos.view(-1), None, k.contiguous().view(-1, Hkv, DH), None, kp.view(-1, Hkv, DH))
        lsa.lsa_kv8_append(dims, cc, None, kp, v, i32(starts), i32(counts), ws)
        for m in t:
            assert torch.equal(got[1][m].view(torch.uint8), got[2][m].view(torch.uint8)), m
    assert lsa.lsa_get_device_status(ws) == lsa.LSA_OK


@pytest.mark.parametrize("H,Hkv", [(32, 32), (64, 32), (64, 64), (128, 64), (128, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_and_read_back_of_many_heads(lsa, H, Hkv, dtype):
    n_b, k_b, C, sb = [30, 4], [21, 4], 32, 16
    lens = [30 * 32 - 9, 70]
    dims, cache, q = attn_inputs(lsa, n_b, C, H, Hkv, sb, dtype, lens, "append", 91, k_b)
    q *= 0.02  # codes of up to 448 times 2^-6: keeps the logits within tens
    ids = kept_ids(n_b, k_b, 3)
    ws = lsa.alloc_workspace(dims, kv8=cache)
    out, lse = torch.empty(2, H, DH, device="cuda"), torch.empty(2, H, device="cuda")
    lsa.lsa_kv8_decode_attn(dims, cache, q, i32(np.concatenate(ids)), None, i32(lens), out, lse, ws)
    K, V = (torch.full((sum(k_b) * C, Hkv, DH), 7.0, dtype=q.dtype, device="cuda") for _ in range(2))
    lsa.lsa_kv8_gather(dims, cache, i32(np.concatenate(ids)), i32(lens), K, V, ws)
    at, off = 0, 0
    for b, kept in enumerate(ids):
        pos = (kept[:, None] * C + np.arange(C)).reshape(-1)
        ok = pos < lens[b]
        chunk, within = off + pos[ok] // C, pos[ok] % C
        rows = [R.decode(c)[chunk, :, within] * R.f64(sc)[chunk, :, within // sb][..., None]
                for c, sc in ((cache.K8, cache.k_scale), (cache.V8, cache.v_scale))]
        for got, want in zip((K, V), rows):
            mine = got[at:at + len(pos)]
            assert torch.equal(mine[torch.from_numpy(ok)].cpu(), torch.from_numpy(want).to(q.dtype))
            assert bool((mine[torch.from_numpy(~ok)] == 7.0).all())
        k, v = (x.transpose(1, 0, 2)[:, None] for x in rows)  # [Hkv][1][n][128]: one chunk of all the tokens
        one = np.ones((1, Hkv, 1))
        vs = R.f64(cache.v_scale)[chunk, :, within // sb]     # and the codes' scales, for the bound
        o, l, to, tl = attention_and_bounds(R.f64(q[b]), k.transpose(1, 0, 2, 3), v.transpose(1, 0, 2, 3), one, one)
        to = to + len(chunk) * 2.0 ** -38 * 448 * vs.max()
        assert np.all(np.abs(o).max(-1) > 50 * to.max(-1))
        assert np.all(np.abs(R.f64(out[b]) - o) <= to) and np.all(np.abs(R.f64(lse[b]) - l) <= tl)
        at, off = at + len(pos), off + n_b[b]
    assert lsa.lsa_get_device_status(ws) == lsa.LSA_OK


@pytest.mark.parametrize("T,H,Hkv,rot,inter", [(1, 128, 128, 128, False), (5, 64, 64, 64, True), (2500, 32, 32, 128, False),
                                               (14211, 2, 2, 128, True)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_rope_is_off_by_half_a_step_and_fp32s_own_errors(lsa, T, H, Hkv, rot, inter, dtype):
    """Before the rounding to the row's type, fp32: the sum of squares (16 terms a lane, 3 joins: 20 u), its root, two
    products, and sine and cosine within 2 u: 40 u of the pair's size, u = 2^-24. The rounding adds half a step of the
    value, eps / 2 relative."""
    qkv, pos, inv, w = prep_inputs(T, H, Hkv, dtype, rot, True, 1 << 20, T + H)
    d = lsa.Dims(1, 1, 128, H, 64, N=1, k=1, kv_dtype=dtype)
    q, k = qkv[:, :H], qkv[:, H:H + Hkv]
    qo, ko = torch.empty_like(q.contiguous()), torch.empty_like(k.contiguous())
    lsa.lsa_qk_norm_rope(d, lsa.QkPrep(rot, inv, *w, eps=1e-6, interleaved=inter), pos, q, k, qo, ko)
    half = torch.finfo(q.dtype).eps / 2
    pick = np.random.default_rng(1).permutation(T)[:400]
    for got, x, wt in ((qo, q, w[0]), (ko, k, w[1])):
        args = R.f64(x)[pick], pos.cpu().numpy()[pick]
        y = R.norm_rope(*args, inv.cpu().numpy(), R.f64(wt), rot, inter, 1e-6)
        n = np.abs(R.norm_rope(*args, np.zeros(rot // 2), R.f64(wt), rot, inter, 1e-6))
        size = n.copy()
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
            size[..., a] = size[..., b] = np.hypot(n[..., a], n[..., b])
        tol = size * 40 * 2.0 ** -24
        tol = tol + (np.abs(y) + tol) * half
        assert np.all(np.abs(R.f64(got)[pick] - y) <= tol), np.max(np.abs(R.f64(got)[pick] - y) / tol)
