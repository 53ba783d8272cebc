// kv8.cuh - pieces that the kernels of the 8-bit K/V cache share: the cache's geometry as a kernel
// parameter, the head row split over eight lanes, RMS norm and rotation, e4m3 conversion.
#pragma once

#include "../../include/lsa_kv8.h"
#include "lsa_device.cuh"

namespace lsa {

constexpr float kE4m3Max = 448.f;
constexpr int kKv8MinExp = -120;  // exponent of the least scale that is written

// Geometry of one call, passed by value.
struct Kv8Geom {
    int32_t Hkv;       // a power of two
    int32_t h_log2;    // log2(Hkv)
    int32_t sb_log2;   // log2(scale_block)
    int32_t c_log2;    // log2(chunk_len)
    int32_t spc;       // scales per (chunk, head) = chunk_len / scale_block
};

// Preparation of q/k rows as a kernel parameter.
struct PrepParams {
    const float* inv_freq;
    const float* q_weight;
    const float* k_weight;
    float eps;
    int32_t ho;           // rot_dim / 16: pairs of octets that are rotated
    int32_t interleaved;
};

// A truth value as a type, for lambdas that are compiled for both.
template <bool V>
struct Const {
    static constexpr bool value = V;
};

// ---------------------------------------------------------------- pairs of floats
// Two floats in a register pair; one instruction works on both, each rounded as the scalar one would.
struct F2 {
    unsigned long long v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 f2_floats(F2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 f2_add(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// ---------------------------------------------------------------- e4m3
// Two floats -> two e4m3 (x in the low byte), to nearest even, saturating at +-448, NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2(float x, float y) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(y), "f"(x));
    return r;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}

// Two e4m3 in the low (or high) half of a word -> f16x2, exact.
__device__ __forceinline__ uint32_t e4m3lo_f16x2(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t e4m3hi_f16x2(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
    return r;
}

__device__ __forceinline__ float2 f16x2_floats(uint32_t w) {
    float2 f;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(f.x), "=f"(f.y)
        : "r"(w));
    return f;
}

// Four e4m3 of a word -> four floats, exact.
__device__ __forceinline__ void e4m3x4_floats(uint32_t w, float* x) {
    const float2 a = f16x2_floats(e4m3lo_f16x2(w)), b = f16x2_floats(e4m3hi_f16x2(w));
    x[0] = a.x;
    x[1] = a.y;
    x[2] = b.x;
    x[3] = b.y;
}

// The least power of two >= 2^kKv8MinExp that brings amax (finite, >= 0) to 448 or less: with
// amax = m 2^e, 1 <= m < 2, that is 2^(e-8) while m <= 1.75 = 448 / 256, and 2^(e-7) above.
__device__ __forceinline__ float kv8_scale_of(float amax) {
    const uint32_t bits = __float_as_uint(amax);
    int e = (int)(bits >> 23) - 127 - ((bits & 0x7FFFFFu) <= 0x600000u ? 8 : 7);
    e = e < kKv8MinExp ? kKv8MinExp : e;
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// ---------------------------------------------------------------- head rows on eight lanes
// A row of Dh = 128 values is 16 octets (8 values). Lane `sub` of the row's eight holds two of them,
// a and b, such that every rotated pair lies within one lane: with half-split pairs the octets sub and
// sub + ho (ho = rot_dim / 16) while sub < ho, else 2 sub and 2 sub + 1; with interleaved pairs, or no
// rotation, always 2 sub and 2 sub + 1. In both forms the lane's eight angles are 8 sub .. 8 sub + 7.
__device__ __forceinline__ void row_octets(int sub, int ho, int interleaved, int* a, int* b) {
    const bool split = sub < ho && !interleaved;
    *a = split ? sub : 2 * sub;
    *b = split ? sub + ho : 2 * sub + 1;
}

template <bool BF16>
struct OctetRaw;  // eight values as loaded
template <>
struct OctetRaw<true> {
    uint4 v;
};
template <>
struct OctetRaw<false> {
    uint4 v, w;
};

template <bool BF16>
__device__ __forceinline__ OctetRaw<BF16> octet_load(const void* row, int o) {
    OctetRaw<BF16> r;
    const uint8_t* p = static_cast<const uint8_t*>(row) + o * (BF16 ? 16 : 32);
    r.v = *reinterpret_cast<const uint4*>(p);
    if constexpr (!BF16) r.w = *reinterpret_cast<const uint4*>(p + 16);
    return r;
}

template <bool BF16>
__device__ __forceinline__ void octet_floats(const OctetRaw<BF16>& r, float* x) {
    if constexpr (BF16) {
        x[0] = bf16lo(r.v.x); x[1] = bf16hi(r.v.x); x[2] = bf16lo(r.v.y); x[3] = bf16hi(r.v.y);
        x[4] = bf16lo(r.v.z); x[5] = bf16hi(r.v.z); x[6] = bf16lo(r.v.w); x[7] = bf16hi(r.v.w);
    } else {
        x[0] = __uint_as_float(r.v.x); x[1] = __uint_as_float(r.v.y);
        x[2] = __uint_as_float(r.v.z); x[3] = __uint_as_float(r.v.w);
        x[4] = __uint_as_float(r.w.x); x[5] = __uint_as_float(r.w.y);
        x[6] = __uint_as_float(r.w.z); x[7] = __uint_as_float(r.w.w);
    }
}

__device__ __forceinline__ uint32_t bf16x2_rn(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Eight floats rounded to the row's type.
template <bool BF16>
__device__ __forceinline__ OctetRaw<BF16> octet_pack(const float* x) {
    OctetRaw<BF16> r;
    if constexpr (BF16) {
        r.v = make_uint4(bf16x2_rn(x[0], x[1]), bf16x2_rn(x[2], x[3]), bf16x2_rn(x[4], x[5]), bf16x2_rn(x[6], x[7]));
    } else {
        r.v = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
        r.w = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
    }
    return r;
}

template <bool BF16>
__device__ __forceinline__ void octet_store(void* row, int o, const OctetRaw<BF16>& r) {
    uint8_t* p = static_cast<uint8_t*>(row) + o * (BF16 ? 16 : 32);
    reinterpret_cast<uint4*>(p)[0] = r.v;
    if constexpr (!BF16) reinterpret_cast<uint4*>(p)[1] = r.w;
}

__device__ __forceinline__ void load8(const float* p, float* w) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
}

// Cosine and sine of position * f. The product and its reduction to within an eighth of a turn are in 64 bits
// (positions of a long context make angles of 2^20 rad and more, where 32 bits are off by tenths); from there
// the Taylor series about 0 suffice in 32: on [-pi/4, pi/4] the first omitted terms, x^11 / 11! and x^12 / 12!,
// are below 2e-9, and the result is within 2^-23.
__device__ __forceinline__ void angle_cs(int32_t position, float f, float* c, float* s) {
    double t = (double)position * (double)f * 0.63661977236758134;  // 2 / pi: quarter turns
    t = fma(-4.0, rint(t * 0.25), t);                                 // whole turns off: [-2, 2]
    const double q = rint(t);
    const float x = (float)(t - q) * 1.5707963267948966f, x2 = x * x;
    const int quarter = (int)(float)q;
    float si = fmaf(x2, 1.f / 362880, -1.f / 5040);
    si = fmaf(x2, si, 1.f / 120);
    si = fmaf(x2, si, -1.f / 6);
    si = fmaf(x * x2, si, x);
    float co = fmaf(x2, -1.f / 3628800, 1.f / 40320);
    co = fmaf(x2, co, -1.f / 720);
    co = fmaf(x2, co, 1.f / 24);
    co = fmaf(x2, co, -0.5f);
    co = fmaf(x2, co, 1.f);
    // turned by `quarter` quarters
    const float u = quarter & 1 ? si : co, v = quarter & 1 ? co : si;
    *c = (quarter + 1) & 2 ? -u : u;
    *s = quarter & 2 ? -v : v;
}

// The 16 values of a lane as eight pairs (p, q) that a rotation mixes: p and q are the octets a and b, or
// (INTER) the even and the odd values of both. Two pairs lie in each F2 of p and of q.
struct RowPairs {
    F2 p[4], q[4];
};

template <bool BF16, bool INTER>
__device__ __forceinline__ RowPairs row_pairs(const OctetRaw<BF16>& a, const OctetRaw<BF16>& b) {
    float x[8], y[8];
    octet_floats<BF16>(a, x);
    octet_floats<BF16>(b, y);
    RowPairs r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (INTER) {
            const float* v = j < 2 ? x + 4 * j : y + 4 * (j - 2);
            r.p[j] = f2(v[0], v[2]);
            r.q[j] = f2(v[1], v[3]);
        } else {
            r.p[j] = f2(x[2 * j], x[2 * j + 1]);
            r.q[j] = f2(y[2 * j], y[2 * j + 1]);
        }
    }
    return r;
}

// Back to octets, rounded to the row's type.
template <bool BF16, bool INTER>
__device__ __forceinline__ void row_octets_of(const RowPairs& r, OctetRaw<BF16>* a, OctetRaw<BF16>* b) {
    float x[8], y[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 p = f2_floats(r.p[j]), q = f2_floats(r.q[j]);
        if constexpr (INTER) {
            float* v = j < 2 ? x + 4 * j : y + 4 * (j - 2);
            v[0] = p.x; v[1] = q.x; v[2] = p.y; v[3] = q.y;
        } else {
            x[2 * j] = p.x; x[2 * j + 1] = p.y;
            y[2 * j] = q.x; y[2 * j + 1] = q.y;
        }
    }
    *a = octet_pack<BF16>(x);
    *b = octet_pack<BF16>(y);
}

// 1 / sqrt(mean(x^2) + eps) of a row, from its lanes' values.
__device__ __forceinline__ float row_rms(const RowPairs& r, float eps) {
    F2 s = f2_mul(r.p[0], r.p[0]);
#pragma unroll
    for (int j = 1; j < 4; ++j) s = f2_fma(r.p[j], r.p[j], s);
#pragma unroll
    for (int j = 0; j < 4; ++j) s = f2_fma(r.q[j], r.q[j], s);
    const float2 h = f2_floats(s);
    float ss = h.x + h.y;
    ss += __shfl_xor_sync(0xffffffffu, ss, 1);
    ss += __shfl_xor_sync(0xffffffffu, ss, 2);
    ss += __shfl_xor_sync(0xffffffffu, ss, 4);
    return rsqrtf(fmaf(ss, 1.f / kDh, eps));
}

// Weight and rotation are one linear map of a pair, the same for every head of a token:
//     p <- p w_p cos - q w_q sin,   q <- q w_q cos + p w_p sin.
// The coefficients of a lane's eight pairs, from its weights (null: 1) and its eight angles, lie in shared
// memory as eight float4, `stride` float4 apart: of p by p, of q by q, of p by q, of q by p, each two. A lane
// that is not rotated has only the weights.
template <bool INTER>
__device__ __forceinline__ void row_coefs(float4* k, int stride, const float* weight, int oa, int ob, bool rot,
                                          const float* c, const float* s) {
    float w[16], a[8][4];
#pragma unroll
    for (int e = 0; e < 16; ++e) w[e] = 1.f;
    if (weight != nullptr) {
        load8(weight + oa * 8, w);
        load8(weight + ob * 8, w + 8);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float wp = w[INTER ? 2 * e : e], wq = w[INTER ? 2 * e + 1 : 8 + e];
        a[e >> 2][e & 3] = rot ? wp * c[e] : wp;
        a[2 + (e >> 2)][e & 3] = rot ? wq * c[e] : wq;
        a[4 + (e >> 2)][e & 3] = rot ? -wq * s[e] : 0.f;
        a[6 + (e >> 2)][e & 3] = rot ? wp * s[e] : 0.f;
    }
#pragma unroll
    for (int f = 0; f < 8; ++f) k[f * stride] = make_float4(a[f][0], a[f][1], a[f][2], a[f][3]);
}

// A lane's values normed by r, weighted and rotated. `full`: every lane of the row is rotated (uniform).
// Otherwise a lane that is not takes no part of its partner, not even 0 times infinity.
__device__ __forceinline__ void row_apply(RowPairs& v, float r, bool rot, bool full, const float4* k, int stride) {
    const F2 r2 = f2(r, r);
    auto apply = [&](auto all) {
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            const float4 pp = k[f * stride], qq = k[(2 + f) * stride], pq = k[(4 + f) * stride], qp = k[(6 + f) * stride];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const F2 p = f2_mul(v.p[2 * f + i], r2), q = f2_mul(v.q[2 * f + i], r2);
                F2 s = f2_mul(q, i ? f2(pq.z, pq.w) : f2(pq.x, pq.y)), t = f2_mul(p, i ? f2(qp.z, qp.w) : f2(qp.x, qp.y));
                if constexpr (!decltype(all)::value) {
                    s.v = rot ? s.v : 0ull;
                    t.v = rot ? t.v : 0ull;
                }
                v.p[2 * f + i] = f2_fma(p, i ? f2(pp.z, pp.w) : f2(pp.x, pp.y), s);
                v.q[2 * f + i] = f2_fma(q, i ? f2(qq.z, qq.w) : f2(qq.x, qq.y), t);
            }
        }
    };
    if (full) apply(Const<true>{}); else apply(Const<false>{});
}

}  // namespace lsa
