// kv8_write.cu - what a new token's rows go through before the attention reads them: RMS norm and
// rotation of queries and keys, and the quantising write to the 8-bit cache.
//
//   k_qk_norm_rope   q, k rows -> normed, rotated rows          (read once, written once)
//   k_kv8_append     k, v rows -> e4m3 codes and their scales   (2 or 4 bytes in, 1 byte out a value)
//
// Both are bound by memory on long runs and by launch latency on single tokens; neither has a product
// for the tensor cores. A row of 128 values lies on eight lanes (kv8.cuh), 16 values to a lane: the
// norm is three shuffles, and a rotated pair never leaves its lane.
#include "kv8.cuh"

namespace lsa {

// ---------------------------------------------------------------- norm and rotation
// A token's angles cost as much as a few of its rows, and weight and rotation become coefficients that serve
// all its heads from shared memory (in registers they would halve the warps in flight). Two forms:
//   a warp per (token, slice of heads): its lanes share the angles, two each, and it walks four heads at a
//   time, in 1 KB runs (bf16) of the token's row;
//   (MANY) with four heads or fewer and tokens enough, a warp per four tokens, eight lanes to a token, each with
//   its own eight angles: a quarter of the coefficients' work.
// In both the next rows are loaded while the ones before are worked on. 16384 tokens of 32 + 8 heads, 336 MB,
// take 61 us in the first form (5.5 TB/s) and 78 to 84 in the second (four rows far apart at a time), 27011 of
// 2 + 1 heads 25 and 14.
constexpr int kPrepThreads = 128;

struct PrepRows {
    const uint8_t *q, *k;
    uint8_t *qo, *ko;
    int64_t q_stride, k_stride, qo_stride, ko_stride;  // bytes from one token to the next
    int32_t H, Hkv;        // 0 where q or k is absent
    int64_t n_tok;
    int32_t slices;        // warps per token, or per four
    int32_t q_per, k_per;  // heads per slice
};

// Heads h, h + step, ... below h1 of a token, n steps (uniform in the warp: the norm's shuffles need every lane).
template <bool BF16, bool INTER, bool MANY>
__device__ __forceinline__ void prep_heads(const uint8_t* src, uint8_t* dst, int h, int h1, int n, int oa, int ob,
                                           bool norm, float eps, bool rot, bool full, const float4* k) {
    constexpr int kRow = kDh * (BF16 ? 2 : 4), step = MANY ? 1 : 4;
    src += (int64_t)h * kRow;
    dst += (int64_t)h * kRow;
    OctetRaw<BF16> ra{}, rb{};
    if (h < h1) {
        ra = octet_load<BF16>(src, oa);
        rb = octet_load<BF16>(src, ob);
    }
    for (int u = 0; u < n; ++u) {
        RowPairs v = row_pairs<BF16, INTER>(ra, rb);
        src += step * kRow;
        if (h + step < h1) {
            ra = octet_load<BF16>(src, oa);
            rb = octet_load<BF16>(src, ob);
        }
        row_apply(v, norm ? row_rms(v, eps) : 1.f, rot, full, k, MANY ? 32 : 8);
        if (h < h1) {
            OctetRaw<BF16> xa, xb;
            row_octets_of<BF16, INTER>(v, &xa, &xb);
            octet_store<BF16>(dst, oa, xa);
            octet_store<BF16>(dst, ob, xb);
        }
        dst += step * kRow;
        h += step;
    }
}

template <bool BF16, bool INTER, bool MANY>
__global__ void __launch_bounds__(kPrepThreads, BF16 ? 8 : 6)
k_qk_norm_rope(const PrepRows r, const PrepParams pp, const int32_t* __restrict__ positions) {
    constexpr int kLanes = MANY ? 32 : 8;
    __shared__ float4 s_coef[kPrepThreads / 32][8][kLanes];  // [warp][which][lane of the row (MANY: and token)]
    pdl_trigger();
    const int lane = threadIdx.x & 31, sub = lane & 7, grp = lane >> 3;
    const int64_t w = (int64_t)blockIdx.x * (kPrepThreads / 32) + (threadIdx.x >> 5);
    const int64_t cell = r.slices == 1 ? w : w / r.slices;
    const int slice = (int)(w - cell * r.slices);
    const int64_t tok = MANY ? 4 * cell + grp : cell;
    if (cell * (MANY ? 4 : 1) < r.n_tok) {
        const bool on = tok < r.n_tok;
        const int q0 = slice * r.q_per, q1 = min(r.H, q0 + r.q_per), k0 = slice * r.k_per, k1 = min(r.Hkv, k0 + r.k_per);
        const uint8_t *q = r.q + tok * r.q_stride, *kk = r.k + tok * r.k_stride;
        const bool rot = sub < pp.ho, full = pp.ho == 8;
        // MANY: the lane's eight angles; else two of the token's, handed round when coefficients are made
        float c2[MANY ? 8 : 2], s2[MANY ? 8 : 2];
        if (MANY ? on && rot : pp.ho > 0) {
            const int32_t pos = positions[tok];
#pragma unroll
            for (int j = 0; j < (MANY ? 8 : 2); ++j) {
                const int a = MANY ? 8 * sub + j : 2 * lane + j;
                if (MANY || a < pp.ho * 8) angle_cs(pos, pp.inv_freq[a], &c2[j], &s2[j]);
            }
        }
        int oa, ob;
        row_octets(sub, pp.ho, INTER, &oa, &ob);
        float4* k = &s_coef[threadIdx.x >> 5][0][MANY ? lane : sub];
        auto heads = [&](const uint8_t* src, uint8_t* dst, int h0, int h1, const float* weight) {
            if (h0 >= h1) return;
            float c[8], s[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                c[e] = MANY ? c2[MANY ? e : 0] : __shfl_sync(0xffffffffu, c2[e & 1], sub * 4 + (e >> 1));
                s[e] = MANY ? s2[MANY ? e : 0] : __shfl_sync(0xffffffffu, s2[e & 1], sub * 4 + (e >> 1));
            }
            __syncwarp();  // the queries' coefficients are done with
            if (MANY || grp == 0) row_coefs<INTER>(k, kLanes, weight, oa, ob, rot, c, s);
            __syncwarp();
            prep_heads<BF16, INTER, MANY>(src, dst, MANY ? h0 : h0 + grp, on ? h1 : h0, MANY ? h1 - h0 : (h1 - h0 + 3) >> 2,
                                          oa, ob, weight != nullptr, pp.eps, rot, full, k);
        };
        heads(q, r.qo + tok * r.qo_stride, q0, q1, pp.q_weight);
        heads(kk, r.ko + tok * r.ko_stride, k0, k1, pp.k_weight);
    }
    pdl_wait();  // launched early, nothing above depends on the kernel before; the one after does
}

// ---------------------------------------------------------------- quantising write
// One CTA per (64-token window of a sequence, K or V, slice of heads): window rows are aligned to 64 tokens of
// the sequence, eight lanes to a row, so that every block of 8..64 tokens lies inside one CTA and its largest
// magnitude is a reduction in the warp (four rows) and a look at scale_block / 4 warps' words.
//
// Measured (B200, 16 heads, bf16, in a graph): 4 x 8192 tokens, 403 MB, 65 us, 6.2 TB/s; with K prepared 90 us,
// 4.5 TB/s, where no one thing binds: the SMs issue in 62% of the cycles, the integer pipe is busy in 51%, and the
// angles alone cost 4 us, the weights and rotations 13. fp32: 109 us (6.2 TB/s) and 152. 4 x 256 tokens prepared
// 8.6 us; one token for each of 8 sequences 4.7, unprepared 3. Tried and slower (when the whole took 94): a head's rows per warp in shared
// memory without barriers (123 us), asynchronous copies three heads ahead (104 us).
constexpr int kAppendThreads = 512;
constexpr int kAppendRows = kAppendThreads / 8;
constexpr int kAppendCoefBytes = 8 * kAppendThreads * 16;

struct AppendParams {
    Kv8Geom g;
    const uint8_t *k, *v;
    int64_t k_stride, v_stride;  // bytes from one row to the next
    uint8_t *K8, *V8;
    float *k_scale, *v_scale;
    const int32_t *start, *new_count;
    int32_t n_new;
    int32_t windows;       // per sequence
    int32_t slices, per;   // slices of heads per window, heads per slice
    uint32_t turn;         // even
};

// A lane's codes of one row: eight bytes at each of its octets. Usually the scale is 2^e, and multiplying by
// 1 / 2^e is the division, exactly: in bf16 pairs too, as what falls below bf16's range is below e4m3's.
template <bool BF16>
__device__ __forceinline__ void store_codes(uint8_t* row, int oa, int ob, OctetRaw<BF16> a, OctetRaw<BF16> b,
                                            float scale, bool power_of_two) {
    float x[8], y[8];
    // 2^-e of a scale 2^e; that of 2^127, which only an older block can have, is subnormal
    const float inv = __uint_as_float(max((254u << 23) - __float_as_uint(scale), 1u << 22));
    if (BF16 && power_of_two) {
        const uint32_t w = __float_as_uint(inv), i2 = (w & 0xFFFF0000u) | w >> 16;
        auto mul = [i2](uint32_t& v) { asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(v) : "r"(i2)); };
        mul(a.v.x); mul(a.v.y); mul(a.v.z); mul(a.v.w);
        mul(b.v.x); mul(b.v.y); mul(b.v.z); mul(b.v.w);
        octet_floats<BF16>(a, x);
        octet_floats<BF16>(b, y);
    } else {
        octet_floats<BF16>(a, x);
        octet_floats<BF16>(b, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[e] = power_of_two ? x[e] * inv : x[e] / scale;  // else: a block that came with another scale
            y[e] = power_of_two ? y[e] * inv : y[e] / scale;
        }
    }
    uint32_t c[4];
    c[0] = e4m3x4(x[0], x[1], x[2], x[3]);
    c[1] = e4m3x4(x[4], x[5], x[6], x[7]);
    c[2] = e4m3x4(y[0], y[1], y[2], y[3]);
    c[3] = e4m3x4(y[4], y[5], y[6], y[7]);
    if (ob == oa + 1) {
        *reinterpret_cast<uint4*>(row + oa * 8) = make_uint4(c[0], c[1], c[2], c[3]);
    } else {
        *reinterpret_cast<uint2*>(row + oa * 8) = make_uint2(c[0], c[1]);
        *reinterpret_cast<uint2*>(row + ob * 8) = make_uint2(c[2], c[3]);
    }
}

// Bits of the largest magnitude of a lane's 16 values, as they lie in the row's type (bf16 in the low half);
// what is not finite is above the rest. bf16 by the paired maximum of magnitudes that passes a NaN on (its
// sign bit is then masked), fp32 as integers once the sign is off.
template <bool BF16>
__device__ __forceinline__ uint32_t top_bits(const OctetRaw<BF16>& a, const OctetRaw<BF16>& b) {
    if constexpr (BF16) {
        auto mx = [](uint32_t x, uint32_t y) {
            uint32_t r;
            asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
            return r;
        };
        const uint32_t z = mx(mx(mx(a.v.x, a.v.y), mx(a.v.z, a.v.w)), mx(mx(b.v.x, b.v.y), mx(b.v.z, b.v.w))) & 0x7FFF7FFFu;
        return max(z & 0xFFFFu, z >> 16);
    } else {
        const uint32_t m = 0x7FFFFFFFu;
        const uint32_t x = max(max(a.v.x & m, a.v.y & m), max(a.v.z & m, a.v.w & m));
        const uint32_t y = max(max(a.w.x & m, a.w.y & m), max(a.w.z & m, a.w.w & m));
        const uint32_t z = max(max(b.v.x & m, b.v.y & m), max(b.v.z & m, b.v.w & m));
        const uint32_t w = max(max(b.w.x & m, b.w.y & m), max(b.w.z & m, b.w.w & m));
        return max(max(x, y), max(z, w));
    }
}

// The warp's largest finite magnitude as fp32 bits, and the error where there were others.
template <bool BF16>
__device__ __forceinline__ uint32_t warp_amax(const OctetRaw<BF16>& a, const OctetRaw<BF16>& b, uint32_t* err) {
    uint32_t top = __reduce_max_sync(0xffffffffu, top_bits<BF16>(a, b));
    if (top >= (BF16 ? 0x7F80u : 0x7F800000u)) {  // rare: look at the finite ones alone
        if ((threadIdx.x & 31) == 0) set_error(err, kErrNonFinite);
        float x[16], m = 0.f;
        octet_floats<BF16>(a, x);
        octet_floats<BF16>(b, x + 8);
        for (int e = 0; e < 16; ++e) m = fmaxf(m, fabsf(x[e]) < INFINITY ? fabsf(x[e]) : 0.f);
        return __reduce_max_sync(0xffffffffu, __float_as_uint(m));
    }
    return BF16 ? top << 16 : top;
}

// Requantise a lane's 16 older codes of a row whose scale grows.
__device__ __forceinline__ void rescale_codes(uint8_t* row, int sub, float ratio) {
    uint4 v = *reinterpret_cast<const uint4*>(row + sub * 16);
    uint32_t* w = &v.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float x[4];
        e4m3x4_floats(w[i], x);
        w[i] = e4m3x4(x[0] * ratio, x[1] * ratio, x[2] * ratio, x[3] * ratio);
    }
    *reinterpret_cast<uint4*>(row + sub * 16) = v;
}

// What the lanes of one row know of it.
struct AppendRow {
    const uint8_t* src;   // the row in the input, head h0
    uint8_t* dst;         // and in the cache
    float* scale;         // its block's
    int64_t dst_step;     // bytes from one head to the next in the cache
    int32_t scale_step;
    int32_t n_h;          // heads
    int32_t pos;
    bool fresh, older, has_old, touched, writer;
};

// The heads of one window. ALL: every row of it is written and none of its blocks is older, as in all but a
// call's first and last windows. PREP: 0 none, 1 half-split pairs, 2 interleaved pairs.
template <bool BF16, int PREP, bool ALL>
__device__ __forceinline__ void append_heads(AppendRow w, const PrepParams& pp, int amax_at,
                                             uint32_t (*s_amax)[kAppendRows / 4], float4* coef, uint32_t* err) {
    constexpr int kRow = kDh * (BF16 ? 2 : 4);
    constexpr bool INTER = PREP == 2;
    const int sub = threadIdx.x & 7;
    int oa, ob;
    row_octets(sub, PREP ? pp.ho : 0, INTER, &oa, &ob);
    OctetRaw<BF16> na{}, nb{};
    const uint8_t *pa = w.src + oa * (kRow / 16), *pb = w.src + ob * (kRow / 16);
    if (ALL || w.fresh) {
        na = octet_load<BF16>(pa, 0);
        nb = octet_load<BF16>(pb, 0);
    }
    const bool rot = PREP != 0 && sub < pp.ho, full = PREP != 0 && pp.ho == 8, norm = PREP != 0 && pp.k_weight != nullptr;
    const float eps = pp.eps;
    if constexpr (PREP != 0) {
        if (ALL || w.fresh) {
            float c[8], s[8];
            if (rot) {
#pragma unroll
                for (int e = 0; e < 8; ++e) angle_cs(w.pos, pp.inv_freq[sub * 8 + e], &c[e], &s[e]);
            }
            row_coefs<INTER>(coef, kAppendThreads, pp.k_weight, oa, ob, rot, c, s);
        }
    }
#pragma unroll (BF16 && ALL ? 2 : 1)
    for (int i = 0; i < w.n_h; ++i) {
        OctetRaw<BF16> xa, xb;
        auto next = [&] {
            pa += kRow;
            pb += kRow;
            if ((ALL || w.fresh) && i + 1 < w.n_h) {
                na = octet_load<BF16>(pa, 0);
                nb = octet_load<BF16>(pb, 0);
            }
        };
        const float was = !ALL && w.has_old ? *w.scale : 0.f;  // read before the barrier, written after it
        if constexpr (PREP != 0) {
            RowPairs v = row_pairs<BF16, INTER>(na, nb);
            next();
            const float rms = norm ? row_rms(v, eps) : 1.f;
            if (ALL || w.fresh) row_apply(v, rms, rot, full, coef, kAppendThreads);
            row_octets_of<BF16, INTER>(v, &xa, &xb);  // what lsa_qk_norm_rope would have stored
        } else {
            xa = na;
            xb = nb;
            next();
        }
        uint32_t top = warp_amax<BF16>(xa, xb, err);
        if ((threadIdx.x & 31) == 0) s_amax[i & 1][threadIdx.x >> 5] = top;
        __syncthreads();  // the other parity's words are free again after the next one
        if (ALL || w.touched) {
            top = __reduce_max_sync(0xffffffffu, s_amax[i & 1][amax_at]);
            const float need = kv8_scale_of(__uint_as_float(top)), sc = ALL ? need : fmaxf(need, was);
            if (ALL || w.fresh) {
                store_codes<BF16>(w.dst, oa, ob, xa, xb, sc, ALL || (__float_as_uint(sc) & 0x807FFFFFu) == 0);
            } else if (w.older && sc > was) {
                rescale_codes(w.dst, sub, was / sc);
            }
            if (w.writer) *w.scale = sc;
        }
        w.dst += w.dst_step;
        w.scale += w.scale_step;
    }
}

// K and V go to CTAs of their own (even, odd): the less a lane holds, the more rows are in flight. A
// bf16 row's values stay packed until they are written, a head's rows are loaded while the one before it is
// worked on, and the coefficients of weight and rotation (computed once for the slice's heads) wait in shared
// memory, where each lane keeps its own. PREP is of K.
template <bool BF16, int PREP>
__global__ void __launch_bounds__(kAppendThreads, BF16 || PREP == 0 ? 2 : 1)
k_kv8_append(const AppendParams ap, const PrepParams pp, const SeqTable tab, uint32_t* err) {
    constexpr int kRow = kDh * (BF16 ? 2 : 4);
    extern __shared__ float4 s_coef[];  // PREP: [8][thread]
    __shared__ uint32_t s_amax[2][kAppendRows / 4];  // [head parity][warp], fp32 bits
    pdl_trigger();
    const int tid = threadIdx.x, r = tid >> 3, warp = tid >> 5, lane = tid & 31;
    // CTA pairs (c, c ^ 1) are K and V of one cell; which is which alternates (bf16) every `turn` CTAs.
    const bool is_v = (BF16 ? blockIdx.x ^ blockIdx.x / ap.turn : blockIdx.x) & 1;
    const int cell = blockIdx.x >> 1;
    const int slice = cell % ap.slices, win = cell / ap.slices % ap.windows, b = cell / ap.slices / ap.windows;

    const int64_t L = (int64_t)(tab.chunk_off[b + 1] - tab.chunk_off[b]) << ap.g.c_log2;
    const int64_t start = ap.start != nullptr ? ap.start[b] : 0;
    int count = ap.new_count != nullptr ? ap.new_count[b] : ap.n_new;
    count = count < 0 ? 0 : count > ap.n_new ? ap.n_new : count;
    int64_t end = start + count;
    if (count > 0 && (start < 0 || end > L)) {
        if (tid == 0 && slice == 0 && win == 0) set_error(err, kErrBadId);
        if (start < 0) end = start;
    }
    end = end < L ? end : L;
    const int64_t w0 = ((start >> 6) + win) << 6;  // first token of the window
    if (w0 < end && w0 + kAppendRows > start && start >= 0) {
        const int64_t pos = w0 + r;
        const int64_t blk0 = pos >> ap.g.sb_log2 << ap.g.sb_log2;  // the row's block
        const int64_t lo = blk0 > start ? blk0 : start;
        const int64_t hi = blk0 + (1 << ap.g.sb_log2) < end ? blk0 + (1 << ap.g.sb_log2) : end;
        AppendRow w;
        w.touched = lo < hi;  // uniform in a warp: its four rows share a block
        w.fresh = pos >= start && pos < end;
        w.older = w.touched && pos < start;
        w.has_old = w.touched && blk0 < start;
        w.writer = w.touched && r % (1 << ap.g.sb_log2) == 0 && (tid & 7) == 0;
        const int h0 = slice * ap.per;
        w.n_h = min(ap.g.Hkv - h0, ap.per);
        w.pos = (int32_t)pos;
        const int64_t row_in = (int64_t)b * ap.n_new + (pos - start);
        w.src = (is_v ? ap.v + row_in * ap.v_stride : ap.k + row_in * ap.k_stride) + (int64_t)h0 * kRow;
        // A head's rows are short runs far apart: the slice's heads of a row, which follow one another, are
        // brought to L2 in one request (8% of the largest prepared append's time).
        if (w.n_h > 1 && w.fresh && (tid & 7) == 0)
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(w.src), "r"(w.n_h * kRow) : "memory");
        const int within = (int)(pos & ((1 << ap.g.c_log2) - 1));
        const int64_t ch0 = (tab.chunk_off[b] + (pos >> ap.g.c_log2)) * ap.g.Hkv + h0;
        w.dst = (is_v ? ap.V8 : ap.K8) + ((ch0 << ap.g.c_log2) + within) * kDh;
        w.dst_step = (int64_t)kDh << ap.g.c_log2;
        w.scale = (is_v ? ap.v_scale : ap.k_scale) + ch0 * ap.g.spc + (within >> ap.g.sb_log2);
        w.scale_step = ap.g.spc;
        const int nw = 1 << (ap.g.sb_log2 - 2);  // a block's warps
        const int amax_at = (warp & ~(nw - 1)) + (lane & (nw - 1));
        const bool all = w0 >= start && w0 + kAppendRows <= end;
        if (PREP != 0 && !is_v) {
            if (all) append_heads<BF16, PREP, true>(w, pp, amax_at, s_amax, s_coef + tid, err);
            else append_heads<BF16, PREP, false>(w, pp, amax_at, s_amax, s_coef + tid, err);
        } else {
            if (all) append_heads<BF16, 0, true>(w, pp, amax_at, s_amax, nullptr, err);
            else append_heads<BF16, 0, false>(w, pp, amax_at, s_amax, nullptr, err);
        }
    }
    pdl_wait();  // as in k_qk_norm_rope
}

// ------------------------------------------------------------------ host side
static PrepParams prep_params(const lsa_qk_prep* p) {
    PrepParams pp = {};
    if (p != nullptr) {
        pp.inv_freq = p->inv_freq;
        pp.q_weight = p->q_weight;
        pp.k_weight = p->k_weight;
        pp.eps = p->eps;
        pp.ho = p->rot_dim / 16;
        pp.interleaved = p->interleaved;
    }
    return pp;
}

cudaError_t launch_qk_norm_rope(const lsa_dims& d, int n_kv_heads, const lsa_qk_prep& prep, int64_t n_tok,
                                const int32_t* positions, const void* q, int64_t q_stride, const void* k,
                                int64_t k_stride, void* q_out, int64_t qo_stride, void* k_out, int64_t ko_stride,
                                int num_sms, cudaStream_t stream, bool pdl) {
    const int es = d.kv_dtype == LSA_BF16 ? 2 : 4;
    PrepRows r = {};
    r.q = (const uint8_t*)q;
    r.k = (const uint8_t*)k;
    r.qo = (uint8_t*)q_out;
    r.ko = (uint8_t*)k_out;
    r.q_stride = q_stride * es;
    r.k_stride = k_stride * es;
    r.qo_stride = qo_stride * es;
    r.ko_stride = ko_stride * es;
    r.H = q != nullptr ? d.H : 0;
    r.Hkv = k != nullptr ? n_kv_heads : 0;
    r.n_tok = n_tok;
    // A warp to a token (or, with few heads, to four) where there are tokens enough to fill the SMs, else the
    // heads of a token are spread, four to a warp at the least.
    const bool many = r.H <= 4 && r.Hkv <= 4 && n_tok >= (int64_t)num_sms * 4 * 24;
    const int64_t cells = many ? (n_tok + 3) / 4 : n_tok, want = (int64_t)num_sms * 24;
    const int unit = many ? 1 : 4, qu = (r.H + unit - 1) / unit, ku = (r.Hkv + unit - 1) / unit, most = qu > ku ? qu : ku;
    int64_t slices = cells >= want ? 1 : (want + cells - 1) / cells;
    if (slices > most) slices = most;
    r.slices = (int)slices;
    r.q_per = (int)((qu + slices - 1) / slices) * unit;
    r.k_per = (int)((ku + slices - 1) / slices) * unit;
    const int64_t warps = cells * r.slices;
    const int64_t ctas = (warps + kPrepThreads / 32 - 1) / (kPrepThreads / 32);
    if (ctas > 0x7fffffffll) return cudaErrorInvalidValue;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    cfg.gridDim = dim3((unsigned)ctas, 1, 1);
    cfg.blockDim = dim3(kPrepThreads, 1, 1);
    const PrepParams pp = prep_params(&prep);
    auto launch = [&](auto bf, auto inter, auto form) {
        return cudaLaunchKernelEx(&cfg,
                                  k_qk_norm_rope<decltype(bf)::value, decltype(inter)::value, decltype(form)::value>,
                                  r, pp, positions);
    };
    auto by_form = [&](auto bf, auto inter) {
        return many ? launch(bf, inter, Const<true>{}) : launch(bf, inter, Const<false>{});
    };
    if (d.kv_dtype == LSA_BF16)
        return pp.interleaved ? by_form(Const<true>{}, Const<true>{}) : by_form(Const<true>{}, Const<false>{});
    return pp.interleaved ? by_form(Const<false>{}, Const<true>{}) : by_form(Const<false>{}, Const<false>{});
}

cudaError_t launch_kv8_append(const lsa_dims& d, const SeqTable& tab, const lsa_kv8_cache& cache, const Kv8Geom& g,
                              const lsa_qk_prep* prep, int n_new, const void* k, int64_t k_stride, const void* v,
                              int64_t v_stride, const int32_t* start, const int32_t* new_count, uint32_t* err,
                              int num_sms, cudaStream_t stream, bool pdl) {
    const int es = d.kv_dtype == LSA_BF16 ? 2 : 4;
    AppendParams ap = {};
    ap.g = g;
    ap.k = (const uint8_t*)k;
    ap.v = (const uint8_t*)v;
    ap.k_stride = k_stride * es;
    ap.v_stride = v_stride * es;
    ap.K8 = (uint8_t*)cache.K8;
    ap.V8 = (uint8_t*)cache.V8;
    ap.k_scale = cache.k_scale;
    ap.v_scale = cache.v_scale;
    ap.start = start;
    ap.new_count = new_count;
    ap.n_new = n_new;
    // a run of n tokens touches at most (n + 62) / 64 + 1 aligned windows (one token: one)
    ap.windows = (int)(((int64_t)n_new + 62) / 64 + 1);
    // Slices of heads. A row's heads follow one another in memory, and K's angles are computed once for a slice,
    // so slices are long, but the calls are bound by what an SM works through: as many as make one round of CTAs
    // (two to an SM, prepared fp32 one; two rounds of fp32 that is not prepared, whose heads are mostly loads; no
    // more than one CTA to an SM where that leaves two heads or fewer), and of `most` heads at most where there are
    // several rounds. Measured with 16 heads, bf16, in 1, 2, 3, 4, 8, 16 slices: 4 x 8192 tokens prepared 101, 89,
    // 95, 102, 138, 222 us, not prepared 85, 72, 65, 69, 90, 139; 4 x 1021 prepared 22.2, 15.3, 19.1, 18.7, 22.6,
    // 32.5; 4 x 256: 21.3, 12.6, 10.4, 9.3, 10.4, 11.9 (8.7 in 6); 8 x 1, not prepared: 7.9, 5.0, 4.7, 3.7, 3.1,
    // 3.6; fp32 4 x 8192, not prepared: 152, 128, 109, 111, 127, 162, 4 x 1021: 30, 23, 25, 22, 21, 25.
    const bool bf16 = d.kv_dtype == LSA_BF16;
    const int64_t cells = (int64_t)ap.windows * d.B * 2;
    const int64_t round = (int64_t)num_sms * (bf16 ? 2 : prep != nullptr ? 1 : 4);
    const int most = prep != nullptr ? 8 : 6;
    int64_t slices = num_sms / cells;
    if (2 * slices < g.Hkv) slices = round / cells;
    if (slices * most < g.Hkv) slices = (g.Hkv + most - 1) / most;
    if (slices > g.Hkv) slices = g.Hkv;
    // Two CTAs that share an SM are a round of CTAs apart: one of K and one of V (K's take longer): 15.3 us
    // instead of 19.7 for 4 x 1021. In fp32 one fits an SM, and this gains nothing (4 x 4096: 87 instead of 84).
    ap.turn = num_sms > 1 ? num_sms & ~1 : 2;
    ap.per = (int)((g.Hkv + slices - 1) / slices);
    ap.slices = (g.Hkv + ap.per - 1) / ap.per;
    const int64_t ctas = (int64_t)ap.windows * d.B * ap.slices * 2;
    if (ctas > 0x7fffffffll) return cudaErrorInvalidValue;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    cfg.gridDim = dim3((unsigned)ctas, 1, 1);
    cfg.blockDim = dim3(kAppendThreads, 1, 1);
    const PrepParams pp = prep_params(prep);
    const int form = prep == nullptr ? 0 : prep->interleaved ? 2 : 1;
    cfg.dynamicSmemBytes = form != 0 ? kAppendCoefBytes : 0;
    if (d.kv_dtype == LSA_BF16)
        return form == 0   ? cudaLaunchKernelEx(&cfg, k_kv8_append<true, 0>, ap, pp, tab, err)
               : form == 1 ? cudaLaunchKernelEx(&cfg, k_kv8_append<true, 1>, ap, pp, tab, err)
                           : cudaLaunchKernelEx(&cfg, k_kv8_append<true, 2>, ap, pp, tab, err);
    return form == 0   ? cudaLaunchKernelEx(&cfg, k_kv8_append<false, 0>, ap, pp, tab, err)
           : form == 1 ? cudaLaunchKernelEx(&cfg, k_kv8_append<false, 1>, ap, pp, tab, err)
                       : cudaLaunchKernelEx(&cfg, k_kv8_append<false, 2>, ap, pp, tab, err);
}

cudaError_t kv8_write_init_attrs() {
    cudaError_t e = set_smem_attrs(k_kv8_append<true, 1>, kAppendCoefBytes);
    if (e == cudaSuccess) e = set_smem_attrs(k_kv8_append<true, 2>, kAppendCoefBytes);
    if (e == cudaSuccess) e = set_smem_attrs(k_kv8_append<false, 1>, kAppendCoefBytes);
    if (e == cudaSuccess) e = set_smem_attrs(k_kv8_append<false, 2>, kAppendCoefBytes);
    return e;
}

}  // namespace lsa
