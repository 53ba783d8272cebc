"""The 8-bit K/V cache's operators written out from their definitions in 64 bits (plain loops and numpy on the
CPU), the inputs of their tests, and the tolerances."""
import math

import numpy as np
import torch

DH = 128
E4M3_MAX = 448.0
MIN_EXP = -120


# ---------------------------------------------------------------- e4m3
def e4m3_values():
    """The value of each of the 256 codes (S.EEEE.MMM, bias 7, 0x7F and 0xFF NaN)."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = math.nan if (c & 127) == 127 else (-x if c & 128 else x)
    return v


VALUES = e4m3_values()


def e4m3_round(y):
    """Nearest e4m3 value, ties to even, +-448 beyond the range; NaN stays."""
    y = np.asarray(y, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        a = np.minimum(np.abs(y), E4M3_MAX)
        step = np.exp2(np.maximum(np.frexp(np.where(np.isfinite(a), a, 1.0))[1] - 1, -6) - 3)
        return np.copysign(np.round(a / step) * step, y)


def scale_of(amax):
    """The least power of two >= 2^-120 with amax <= 448 * scale."""
    e = MIN_EXP
    if amax > 0:
        e = max(MIN_EXP, math.floor(math.log2(amax / E4M3_MAX)) - 2)
        while amax > E4M3_MAX * 2.0 ** e:
            e += 1
    return 2.0 ** e


def decode(codes):
    """float64 values of a tensor of e4m3 bytes."""
    return VALUES[codes.view(torch.uint8).cpu().numpy()]


# ---------------------------------------------------------------- the operators
def norm_rope(x, pos, inv_freq, w, rot, interleaved, eps):
    """x float64 [T][heads][128], pos int [T] -> float64, not rounded."""
    y = np.array(x, dtype=np.float64)
    if w is not None:
        y = y / np.sqrt((y ** 2).mean(-1, keepdims=True) + eps) * np.asarray(w, dtype=np.float64)
    z = y.copy()
    for i in range(rot // 2):
        a = np.asarray(pos, dtype=np.float64) * float(inv_freq[i])
        c, s = np.cos(a)[:, None], np.sin(a)[:, None]
        p, r = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        z[..., p] = y[..., p] * c - y[..., r] * s
        z[..., r] = y[..., r] * c + y[..., p] * s
    return z


def append(vals, scales, rows, chunk0, n_chunks, C, sb, start):
    """Write rows float64 [n][Hkv][128] at token `start` of a sequence into vals float64 [chunks][Hkv][C][128]
    (code values) and scales [chunks][Hkv][C/sb], in place."""
    end = min(start + len(rows), n_chunks * C)
    if start < 0:
        return
    for blk in range(start // sb, -(-end // sb) if end > start else 0):
        lo, hi = max(blk * sb, start), min(blk * sb + sb, end)
        chunk, w0 = chunk0 + blk * sb // C, blk * sb % C
        for h in range(vals.shape[1]):
            r = rows[lo - start:hi - start, h]
            fin = np.abs(r[np.isfinite(r)])
            s = scale_of(fin.max() if fin.size else 0.0)
            if lo > blk * sb:
                was = scales[chunk, h, w0 // sb]
                s = max(s, was)
                if s > was:
                    j = slice(w0, w0 + lo - blk * sb)
                    vals[chunk, h, j] = e4m3_round(vals[chunk, h, j] * (was / s))
            scales[chunk, h, w0 // sb] = s
            vals[chunk, h, w0 + lo - blk * sb:w0 + hi - blk * sb] = e4m3_round(r / s)


def attention(q, vals_k, ks, vals_v, vs, tokens):
    """One sequence: q [H][128]; vals [n][Hkv][C][128] code values of its chunks, scales [n][Hkv][C/sb]; tokens: the
    (chunk, within) pairs that are attended. -> out [H][128], lse [H], bound on |logit| sums A [H], max|v| [H]."""
    H, Hkv, C = q.shape[0], vals_k.shape[1], vals_k.shape[2]
    sb = C // ks.shape[2]
    out, lse = np.zeros((H, DH)), np.full(H, -np.inf)
    A, top = np.zeros(H), np.zeros(H)
    if len(tokens):
        ch, wi = np.asarray(tokens).T
        for h in range(H):
            kv = h // (H // Hkv)
            k = vals_k[ch, kv, wi] * ks[ch, kv, wi // sb][:, None]
            v = vals_v[ch, kv, wi] * vs[ch, kv, wi // sb][:, None]
            l = k @ q[h] / math.sqrt(DH)
            m = l.max()
            p = np.exp(l - m)
            lse[h] = m + math.log(p.sum())
            out[h] = (p / p.sum()) @ v
            A[h] = (np.abs(k) @ np.abs(q[h])).max() / math.sqrt(DH)
            top[h] = np.abs(v).max()
    return out, lse, A, top


def attn_tolerance(A, top, n_tokens, q_err=0.0):
    """(out, lse) bounds per head. With u = 2^-24: q as two f16 halves is off by 2^-22 of its row's largest, a product
    of 128 terms accumulated in fp32 in 8 steps, each truncating, by 2^-20 of sum |q k|; scale factors and the
    exponent's argument by 4 u of a logit's size, which A bounds too: 2^-18 A together, twice over in the weights'
    quotient. The exponential, the weights' halves and the joins: 2^-20 each at most. Sums of up to n weights or
    products, in fp32 with truncation: 2^-23 a step, at most n / 16 steps plus 64 for the joins. q_err:
    how far the queries themselves may be off, relative to their pairs' size."""
    steps = (n_tokens / 16 + 64) * 2.0 ** -23
    u = 2.0 ** -18 + 2 * q_err
    return top * (2 * u * A + 2.0 ** -18 + 2 * steps) + 1e-37, u * A + 2.0 ** -20 + steps + 2.0 ** -20


# ---------------------------------------------------------------- inputs
def make_cache(lsa, chunks, Hkv, C, sb, rng, scales="append"):
    """Random code bytes (no NaN) and scales on the device; `scales`: as the append writes them (powers of two), any
    ("free"), or powers of two of all sizes ("wide")."""
    t = {}
    for name in ("K", "V"):
        c = rng.integers(0, 256, (chunks, Hkv, C, DH), dtype=np.uint8)
        c[(c & 127) == 127] = 0x30
        if scales == "free":
            s = np.exp(rng.normal(-3, 1, (chunks, Hkv, C // sb)))
        elif scales == "wide":
            s = np.exp2(rng.integers(-14, 5, (chunks, Hkv, C // sb)))
        else:
            s = np.exp2(rng.integers(-9, -5, (chunks, Hkv, C // sb)))
        t[name + "8"] = torch.from_numpy(c).cuda().view(torch.float8_e4m3fn)
        t[name.lower() + "_scale"] = torch.from_numpy(s.astype(np.float32)).cuda()
    return t


def f64(t):
    return t.detach().double().cpu().numpy()
