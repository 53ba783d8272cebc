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

// The same, stored at octet o.
template <bool BF16>
__device__ __forceinline__ void octet_store(void* row, int o, const float* x) {
    uint8_t* p = static_cast<uint8_t*>(row) + o * (BF16 ? 16 : 32);
    const OctetRaw<BF16> r = octet_pack<BF16>(x);
    reinterpret_cast<uint4*>(p)[0] = r.v;
    if constexpr (!BF16) reinterpret_cast<uint4*>(p)[1] = r.w;
}

__device__ __forceinline__ void load8(const float* p, float* w) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
}

// Cosine and sine of position * f: the product and its reduction to a turn in 64 bits (positions of a
// long context make angles of 2^20 rad and more, where 32 bits are off by tenths), the fraction in 32.
// FAST, for rows that are rounded to bf16 (2^-9): the hardware's sine and cosine, within 2^-21 on [-pi, pi];
// otherwise within 2 ulp, at four times the instructions.
template <bool FAST>
__device__ __forceinline__ void angle_cs(int32_t position, float f, float* c, float* s) {
    double t = (double)position * (double)f * 0.15915494309189534;  // 1 / (2 pi)
    t -= rint(t);
    if constexpr (FAST) {
        const float a = (float)t * 6.2831853071795865f;
        *s = __sinf(a);
        *c = __cosf(a);
    } else {
        sincospif((float)(2.0 * t), s, c);
    }
}

// 1 / sqrt(mean(x^2) + eps) of a row, from its lanes' values x[0..7] (octet a) and y[0..7] (octet b).
__device__ __forceinline__ float row_rms(const float* x, const float* y, float eps) {
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], fmaf(y[e], y[e], ss));
    ss += __shfl_xor_sync(0xffffffffu, ss, 1);
    ss += __shfl_xor_sync(0xffffffffu, ss, 2);
    ss += __shfl_xor_sync(0xffffffffu, ss, 4);
    return rsqrtf(fmaf(ss, 1.f / kDh, eps));
}

// Weight and rotation are one linear map of a pair, the same for every head of a token: value v becomes
// v a + partner b. The coefficients of a lane's 16 values (octet a, octet b), from its weights (null: 1) and
// its eight angles, lie in shared memory as eight float4, a[16] then b[16], `stride` float4 apart; a lane
// that is not rotated has only a.
template <bool INTER>
__device__ __forceinline__ void row_coefs(float4* k, int stride, const float* weight, int oa, int ob, bool rot,
                                          const float* c, const float* s) {
    float w[16], a[16], b[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) w[e] = 1.f;
    if (weight != nullptr) {
        load8(weight + oa * 8, w);
        load8(weight + ob * 8, w + 8);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        // the e-th pair: (octet a, octet b) at e, or two neighbours of one octet
        const int p = INTER ? 2 * e : e, q = INTER ? 2 * e + 1 : 8 + e;
        a[p] = rot ? w[p] * c[e] : w[p];
        a[q] = rot ? w[q] * c[e] : w[q];
        b[p] = rot ? -w[q] * s[e] : 0.f;
        b[q] = rot ? w[p] * s[e] : 0.f;
    }
#pragma unroll
    for (int f = 0; f < 4; ++f) {
        k[f * stride] = make_float4(a[4 * f], a[4 * f + 1], a[4 * f + 2], a[4 * f + 3]);
        k[(4 + f) * stride] = make_float4(b[4 * f], b[4 * f + 1], b[4 * f + 2], b[4 * f + 3]);
    }
}

// A lane's values (x: octet a, y: octet b) normed by r, weighted and rotated. `full`: every lane of the row is
// rotated (uniform). Otherwise a lane that is not takes no part of its neighbour, not even 0 times infinity.
template <bool INTER>
__device__ __forceinline__ void row_apply(float* x, float* y, float r, bool rot, bool full, const float4* k,
                                          int stride) {
    auto apply = [&](auto all) {
        auto pair = [&](float& u, float& v, float au, float av, float bu, float bv) {
            const float p = u * r, q = v * r;
            float s = q * bu, t = p * bv;
            if constexpr (!decltype(all)::value) {
                s = rot ? s : 0.f;
                t = rot ? t : 0.f;
            }
            u = fmaf(p, au, s);
            v = fmaf(q, av, t);
        };
#pragma unroll
        for (int f = 0; f < (INTER ? 4 : 2); ++f) {
            if constexpr (INTER) {
                const float4 a = k[f * stride], b = k[(4 + f) * stride];
                float* v = (f < 2 ? x : y) + 4 * (f & 1);
                pair(v[0], v[1], a.x, a.y, b.x, b.y);
                pair(v[2], v[3], a.z, a.w, b.z, b.w);
            } else {
                const float4 au = k[f * stride], av = k[(2 + f) * stride], bu = k[(4 + f) * stride], bv = k[(6 + f) * stride];
                pair(x[4 * f], y[4 * f], au.x, av.x, bu.x, bv.x);
                pair(x[4 * f + 1], y[4 * f + 1], au.y, av.y, bu.y, bv.y);
                pair(x[4 * f + 2], y[4 * f + 2], au.z, av.z, bu.z, bv.z);
                pair(x[4 * f + 3], y[4 * f + 3], au.w, av.w, bu.w, bv.w);
            }
        }
    };
    if (full) apply(Const<true>{}); else apply(Const<false>{});
}

}  // namespace lsa
