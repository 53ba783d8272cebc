// kv8_attn.cu - split-K flash-decode attention over the kept chunks of the 8-bit K/V cache.
//
//     l_t = (q . k8_t) ks_t / sqrt(Dh),   out = sum_t softmax(l)_t vs_t v8_t
//
// for one decode query per sequence, H query heads sharing Hkv K/V heads in groups of H / Hkv.
//
// What bounds it: reading 2 Dh bytes a token and K/V head, as long as the instructions spent on them
// stay few. On the CUDA cores a byte would cost a conversion and a multiply-add; both products
// therefore run on the tensor cores. They are one group of query heads wide, far from what fills a
// tcgen05 tile, so they use the warp-level instructions, whose operands come from registers.
//
//  * Both products run in f16 (m16n8k16) with fp32 accumulation: an e4m3 code is an f16 number exactly,
//    and one conversion unpacks two. (The e4m3 form of the instruction is no cheaper: by the counters of
//    executed instructions it costs conversions and f16 products too, and 96 instructions a tile more.)
//  * Full precision from f16 operands. A row of q, scaled by a power of two, is split into f16 hi + lo; lo
//    lies in the eight rows of the 16-row operand that a group of up to 8 heads leaves free. The weights
//    P are split in the same way: with 4 heads or fewer, lo takes the free half of the 8 columns, with 8
//    heads a second product.
//  * The reduction index of a product may be permuted as long as both operands agree, so each lane uses
//    whole 16-byte pieces as they come. Lane (g, t) of a warp (g = lane / 4, t = lane % 4) takes bytes
//    32 t .. 32 t + 31 of token g's row of K (four to a step of 16 dims), and bytes 16 g .. 16 g + 15 of
//    tokens 2 t and 2 t + 1 of V, whose bytes a permute interleaves into pairs along the tokens. S leaves
//    its scores exactly where the second product wants P, so nothing is exchanged between them.
//  * V's scale multiplies the weight, times a power of two that brings the largest such product that the
//    row has met to 2^13..2^15, so that they fit f16 whatever the scales are; the running output carries
//    that power of two. A product keeps 22 bits down to 2^-16 of the row's largest, and what is below
//    2^-38 of it is lost, as it would be in an fp32 sum. (A power of two for all rows, from the scales
//    alone, would let a block of large scale that a row hardly attends to take that row's bits.)
//  * The tensor cores truncate when they accumulate: each tile's product starts from zero and is added
//    to the running output in fp32, rounded to nearest, by the multiply-add that also rescales it.
//  * A warp streams tiles of 32 tokens of one (sequence, K/V head) run through its own 4 KB of K and 4 KB
//    of V in shared memory, filled by asynchronous copies (no barrier between warps). Each part is
//    refilled for the next tile as soon as it is read: with 16 warps on an SM a warp's step takes longer
//    than memory does, so one tile ahead is enough, and few registers (128) matter more. What a warp has
//    to know of a tile (chunk id, row, scales, how many tokens exist) its lanes work out side by side for
//    32 groups of 8 tokens ("octets") at a time.
//  * Every run is cut into equal parts, one to a CTA, so that the CTAs fit the device at once; a CTA joins
//    its warps in shared memory, and the parts of a run are joined by k_kv8_attn_merge. Runs of one part
//    are written at once.
//
// Measured (B200, bf16 queries, calls captured in a graph): 256 of 2048 chunks x 8 sequences, 16 heads, 538 MB:
// 82 us, 6.5 TB/s (a plain copy moves 6.47); 819 of 8192 x 4, 32 heads on 8, 430 MB: 70 us, 6.1 TB/s. What is
// left above the bytes is 8 to 10 us a call to start, fill and join. 32 ragged sequences with groups of 8, 355 MB:
// 66 us, 5.4 TB/s. 8 chunks of one sequence: 6.3 us.
#include <algorithm>

#include "kv8.cuh"

namespace lsa {

constexpr int kKv8Tile = 32;       // tokens per tile: 4 octets
constexpr int kKv8Batch = 8;       // tiles whose 32 octets the lanes hold
constexpr int kKv8MaxRows = 8;     // query heads per run
constexpr float kKv8Top = 14.f;    // weights times V's scales are brought to about 2^14
constexpr float kKv8MinD = -112.f; // and the factor for that stays within fp32
constexpr int kKv8SlotV = kKv8Tile * kDh;          // a warp's shared memory: K rows, V rows,
constexpr int kKv8Meta = 2 * kKv8Tile * kDh;       // two batches of ks[32], vs[32], n[32], vs's exponents[32]
constexpr int kKv8MetaBytes = 4 * 32 * 4;
constexpr int kKv8WarpBytes = kKv8Meta + 2 * kKv8MetaBytes;
constexpr int kKv8JoinBytes = kKv8MaxRows * (kDh + 2) * 4;  // of a warp; takes the tiles' place
static_assert(kKv8JoinBytes <= kKv8WarpBytes, "the join's buffers lie where the tiles were");
__host__ __device__ constexpr int kv8_smem(int warps) { return warps * kKv8WarpBytes + 8 * 32 * 16; }

// Prefix tables of one call: the kept (or all) chunks, and the CTAs (all heads' parts).
struct Kv8Tab {
    int32_t B;
    int32_t chunk_off[kMaxB + 1];
    int32_t kept_off[kMaxB + 1];
    int32_t cta_off[kMaxB + 1];  // by place: sequences ordered by the length of their parts, longest first
    uint8_t seq_at[kMaxB], place_of[kMaxB];
};
static_assert(kMaxB <= 256, "places fit in a byte");

struct Kv8AttnParams {
    Kv8Geom g;
    const uint8_t *q, *K8, *V8;
    const float *k_scale, *v_scale;
    const int32_t *ids, *counts, *seq_len;  // nullable
    float *out, *lse, *part_o, *part_ml;    // lse nullable
    int32_t H;
    int32_t rows;       // query heads per run: min(group, 8)
    int32_t rts;        // runs per K/V head: group / rows
    int32_t runs_log2;  // log2 of a sequence's runs, Hkv * rts
    int32_t len_add;    // added to seq_len
    int32_t num_sms;
    float qscale;       // log2(e) / sqrt(Dh)
};

// 2^x by the hardware's approximation (relative error ~2^-22; 2^-inf = 0).
__device__ __forceinline__ float kv8_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The exponent of the power of two that brings 2^d to 2^13..2^14, as an integer in the low bits of a float: adding
// 1.5 2^23 rounds 13.5 - d to it.
__device__ __forceinline__ float kv8_up(float d) { return (kKv8Top - 0.5f - d) + 12582912.f; }
// That power of two (sign 1), or its inverse (-1): the shift leaves the exponent's bits alone.
__device__ __forceinline__ float kv8_pow2(float up, int sign) {
    return __uint_as_float((127u << 23) + (uint32_t)sign * (__float_as_uint(up) << 23));
}
// x, the largest finite number in place of an infinity; NaN stays.
__device__ __forceinline__ float kv8_finite(float x) {
    float y;
    asm("min.NaN.f32 %0, %1, 0f7F7FFFFF;" : "=f"(y) : "f"(x));
    return y;
}

// d = a b + c; c may be zeros, which cost no registers.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1, const float (&c)[4]) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

__device__ __forceinline__ uint32_t f16x2_rn(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
template <typename T>
__device__ __forceinline__ void kv8_sts(uint32_t addr, T v) {
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(*reinterpret_cast<const uint32_t*>(&v)) : "memory");
}
__device__ __forceinline__ uint32_t kv8_lds(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint4 kv8_lds16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

// The place of the sequence whose CTAs hold CTA c.
__device__ __forceinline__ int kv8_place_of(const Kv8Tab& tab, int c) {
    int lo = 0, hi = tab.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tab.cta_off[mid] <= c) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// The part that a CTA takes. Of the CTAs that share an SM from the start (a round apart), every other full round
// is turned about, so that long parts (they come first) meet short ones. 32 ragged sequences, 4 runs each: 71 -> 67
// us; 250: 70 -> 63.
template <int WARPS>
__device__ __forceinline__ int kv8_cta(int num_sms) {
    const int c = blockIdx.x, round = c / num_sms;
    const bool turned = (round & 1) && round < 16 / WARPS && (round + 1) * num_sms <= (int)gridDim.x;
    return turned ? (2 * round + 1) * num_sms - 1 - c : c;
}

// Grid: all parts of all runs; WARPS * 32 threads. BF16: the type of q; PLO: groups of 8 (a second product
// for P's low halves).
template <bool BF16, bool PLO, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 16 / WARPS)
k_kv8_attn(const Kv8AttnParams p, const Kv8Tab tab, uint32_t* err) {
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int c_log2 = p.g.c_log2;
    pdl_trigger();

    // ---- this CTA's part: a sequence's CTAs are ordered by part, then run
    const int cta = kv8_cta<WARPS>(p.num_sms);
    const int place = kv8_place_of(tab, cta), b = tab.seq_at[place];
    const int idx = cta - tab.cta_off[place], run = idx & ((1 << p.runs_log2) - 1), part = idx >> p.runs_log2;
    const int parts = (tab.cta_off[place + 1] - tab.cta_off[place]) >> p.runs_log2;
    const int h = run / p.rts;
    const int qrow0 = b * p.H + run * p.rows;
    __shared__ int s_part[3];  // for the end: registers are short in between
    if (tid == 0) {
        s_part[0] = cta;
        s_part[1] = parts;
        s_part[2] = qrow0;
    }
    int tile0, tile1;
    {
        const int tokens = (tab.kept_off[b + 1] - tab.kept_off[b]) << c_log2;
        const int tiles = (tokens + kKv8Tile - 1) / kKv8Tile, per = tiles / parts, more = tiles - per * parts;
        tile0 = part * per + min(part, more);
        tile1 = tile0 + per + (part < more ? 1 : 0);
    }
    pdl_wait();
    // chunks and tokens that take part (both fit in 31 bits)
    int kept = tab.kept_off[b + 1] - tab.kept_off[b];
    int len = (tab.chunk_off[b + 1] - tab.chunk_off[b]) << c_log2;
    if (p.counts != nullptr) kept = max(0, min(kept, p.counts[b]));
    if (p.seq_len != nullptr) {
        const int n = p.seq_len[b];  // + len_add may pass 2^31 - 1
        len = n >= len ? len : max(0, min(len, n + p.len_add));
    }
    if (p.ids == nullptr) kept = min(kept, (len + (1 << c_log2) - 1) >> c_log2);
    // This warp's tiles are tile0 + warp + WARPS * i, i < n_it, as far as there are tokens.
    const int first = tile0 + warp;
    const int n_it = (max(min(tile1, ((kept << c_log2) + kKv8Tile - 1) / kKv8Tile) - first, 0) + WARPS - 1) / WARPS;

    // ---- addresses in shared memory. A row's 16-byte units are XOR-swizzled by the row: the copies' and
    // both fragments' accesses are free of bank conflicts.
    const uint32_t slot = smem_u32(smem) + warp * kKv8WarpBytes, meta = slot + kKv8Meta + 4 * lane;
    const uint32_t cp0 = slot + (lane >> 3) * kDh + (((lane & 7) ^ (lane >> 3)) << 4);
    const uint32_t cp1 = slot + ((lane >> 3) + 4) * kDh + (((lane & 7) ^ ((lane >> 3) + 4)) << 4);
    const uint32_t ka0 = slot + g * kDh + ((2 * t ^ g) << 4), ka1 = ka0 ^ 16;
    const uint32_t va0 = slot + kKv8SlotV + 2 * t * kDh + ((g ^ 2 * t) << 4);
    const uint32_t va1 = slot + kKv8SlotV + (2 * t + 1) * kDh + ((g ^ (2 * t + 1)) << 4);
    const uint32_t qs = smem_u32(smem) + WARPS * kKv8WarpBytes + lane * 16;  // q's halves: [step][lane]

    // ---- what the lanes know of the octets being copied: lane L has octet L % 4 of tile (batch) + L / 4.
    // Its first row in the cache stays in a register; its scales and its count of tokens that take part go
    // to the batch's place in shared memory, for when the batch is read.
    uint32_t row = 0;
    uint32_t nz = 0;  // octets (lanes) with tokens
    int id_next = 0;
    auto token_of = [&](int i) {  // first token of this lane's octet in the batch of tile i
        return (first + WARPS * (i + (lane >> 2))) * kKv8Tile + 8 * (lane & 3);
    };
    auto fetch_id = [&](int i) {
        const int j = token_of(i) >> c_log2;
        id_next = j >= kept ? -1 : p.ids != nullptr ? p.ids[tab.kept_off[b] + j] : j;
    };
    auto next_batch = [&](int i) {
        const int tk = token_of(i), w = tk & ((1 << c_log2) - 1), id = id_next;
        const uint32_t m = meta + (i & kKv8Batch ? kKv8MetaBytes : 0);
        int n = 0;
        if (tk >> c_log2 < kept && i + (lane >> 2) < n_it) {
            if (id >= 0 && id < tab.chunk_off[b + 1] - tab.chunk_off[b]) {
                n = min(max(len - ((id << c_log2) + w), 0), 8);
                const uint32_t ch = (uint32_t)(tab.chunk_off[b] + id) * p.g.Hkv + h;
                row = (ch << c_log2) + w;
                if (n > 0) {
                    const uint32_t si = ch * p.g.spc + (w >> p.g.sb_log2);
                    cp_async4(m, p.k_scale + si);
                    cp_async4(m + 128, p.v_scale + si);
                }
            } else {
                set_error(err, kErrBadId);
            }
        }
        if (n == 0) {
            kv8_sts(m, 0.f);
            kv8_sts(m + 128, 0.f);
        }
        kv8_sts(m + 256, n);
        nz = __ballot_sync(0xffffffffu, n > 0);
        fetch_id(i + kKv8Batch);
    };
    // Copies of tile i's K or V rows (`off` into the warp's tile), one group for each (empty past the end).
    // Octets without tokens are not copied; of the others all 8 rows are (they lie in the cache).
    auto copy = [&](int i, const uint8_t* base, uint32_t off) {
        if (i < n_it) {
            const int l0 = 4 * (i & (kKv8Batch - 1));
            if (c_log2 >= 5) {  // the octets follow one another; if the first has no tokens, nor have the others
                const uint32_t r = __shfl_sync(0xffffffffu, row, l0);
                if (nz >> l0 & 1) {
                    const uint8_t* src = base + (uint64_t)r * kDh + lane * 16;
#pragma unroll
                    for (int o = 0; o < 4; ++o) {
                        cp_async16(cp0 + off + o * 8 * kDh, src + o * 8 * kDh);
                        cp_async16(cp1 + off + o * 8 * kDh, src + o * 8 * kDh + 4 * kDh);
                    }
                }
            } else {
#pragma unroll
                for (int o = 0; o < 4; ++o) {
                    const uint32_t r = __shfl_sync(0xffffffffu, row, l0 + o);
                    if (nz >> (l0 + o) & 1) {
                        const uint8_t* src = base + (uint64_t)r * kDh + lane * 16;
                        cp_async16(cp0 + off + o * 8 * kDh, src);
                        cp_async16(cp1 + off + o * 8 * kDh, src + 4 * kDh);
                    }
                }
            }
        }
        cp_async_commit();
    };

    fetch_id(0);
    next_batch(0);
    copy(0, p.K8, 0);
    copy(0, p.V8, kKv8SlotV);

    // ---- q: rows scaled to stay below 2^15, as f16 hi + lo. A warp splits a row at a time: a lane's four values
    // are one step's share of lane (row, lane / 8) in the 16-row operand, hi in rows 0..7 and lo in rows 8..15.
    // With fewer than 8 heads the rows recur.
    __shared__ float s_qmul[kKv8MaxRows];
    for (int c = warp; c < kKv8MaxRows; c += WARPS) {
        const int r = c & (p.rows - 1);
        float x[4];
        if constexpr (BF16) {
            const uint2 v = reinterpret_cast<const uint2*>(p.q)[(int64_t)(qrow0 + r) * 32 + lane];
            x[0] = bf16lo(v.x); x[1] = bf16hi(v.x); x[2] = bf16lo(v.y); x[3] = bf16hi(v.y);
        } else {
            const float4 v = reinterpret_cast<const float4*>(p.q)[(int64_t)(qrow0 + r) * 32 + lane];
            x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
        }
        // the largest magnitude's bits; what is not finite is above the rest
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(top, __float_as_uint(x[e]) & 0x7FFFFFFFu);
        top = __reduce_max_sync(0xffffffffu, top);
        // top < 2^(ex + 1): times 2^(14 - ex) it stays below 2^15. The factor is kept within fp32.
        int ex = (int)(top >> 23) - 127;
        ex = ex < -110 ? -110 : ex;
        const float up = __uint_as_float((uint32_t)(14 - ex + 127) << 23);
        uint32_t a[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float x0 = x[2 * j] * up, x1 = x[2 * j + 1] * up;
            a[2 * j] = f16x2_rn(x0, x1);
            const float2 f = f16x2_floats(a[2 * j]);
            a[2 * j + 1] = f16x2_rn(x0 - f.x, x1 - f.y);
        }
        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::
                     "r"(qs - 16 * lane + (lane & 7) * 512 + (4 * c + (lane >> 3)) * 16),
                     "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3])
                     : "memory");
        // a row with an infinity or a NaN has no finite scores
        if (lane == 0)
            s_qmul[c] = top < 0x7F800000u ? p.qscale * __uint_as_float((uint32_t)(ex - 14 + 127) << 23)
                                          : __uint_as_float(0x7FC00000u);
    }
    __syncthreads();
    const float qmul = s_qmul[g];

    // of the lane's row: running maximum and sum, and log2 of its largest weight times a V scale (the scale's
    // power of two) relative to that maximum
    float o[8][4], m = -INFINITY, l = 0.f, d = kKv8MinD;
    const float zero[4] = {0.f, 0.f, 0.f, 0.f};
    const bool one = p.g.sb_log2 >= 5;  // a tile lies in one block
    uint32_t full = 0;  // octets of the batch in use whose 8 tokens all take part
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;

    for (int it = 0; it < n_it; ++it) {
        const int l0 = 4 * (it & (kKv8Batch - 1));
        const uint32_t mt = meta + (it & kKv8Batch ? kKv8MetaBytes : 0);  // this batch's, at this lane
        cp_async_wait<1>();
        __syncwarp();  // every lane's copies of K have landed
        if (l0 == 0) {  // a new batch
            full = __ballot_sync(0xffffffffu, kv8_lds(mt + 256) == 8);
            kv8_sts(mt + 384, (float)((int)(kv8_lds(mt + 128) >> 23) - 127));  // read behind the next barrier
        }
        const bool whole = (full >> l0 & 15u) == 15u;
        const uint32_t mb = mt - 4 * lane + 4 * l0;  // of the tile's four octets

        // ---- S: the halves of q against the tile's tokens
        float sc[8];
        {
            uint32_t kw[4][8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 ka = kv8_lds16(ka0 + i * 8 * kDh), kb = kv8_lds16(ka1 + i * 8 * kDh);
                kw[i][0] = ka.x; kw[i][1] = ka.y; kw[i][2] = ka.z; kw[i][3] = ka.w;
                kw[i][4] = kb.x; kw[i][5] = kb.y; kw[i][6] = kb.z; kw[i][7] = kb.w;
            }
            float c[4][4];
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                const uint4 a = kv8_lds16(qs + s * 512);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t b0 = e4m3lo_f16x2(kw[i][s]), b1 = e4m3hi_f16x2(kw[i][s]);
                    if (s == 0) mma_f16(c[i], a.x, a.y, a.z, a.w, b0, b1, zero);
                    else mma_f16(c[i], a.x, a.y, a.z, a.w, b0, b1, c[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sc[2 * i] = c[i][0] + c[i][2];
                sc[2 * i + 1] = c[i][1] + c[i][3];
            }
            const uint4 k4 = kv8_lds16(mb);
            const uint32_t ks[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float f = qmul * __uint_as_float(ks[i]);
                sc[2 * i] *= f;
                sc[2 * i + 1] *= f;
            }
        }
        if (!whole) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int n = (int)kv8_lds(mb + 256 + 4 * i);
                if (2 * t >= n) sc[2 * i] = -INFINITY;
                if (2 * t + 1 >= n) sc[2 * i + 1] = -INFINITY;
            }
        }
        __syncwarp();  // the K rows are read
        if ((it + 1) % kKv8Batch == 0) next_batch(it + 1);
        copy(it + 1, p.K8, 0);

        // ---- running maximum of the lane's row of q, with and without V's scales
        float two[4], mx, mv;
#pragma unroll
        for (int i = 0; i < 4; ++i) two[i] = fmaxf(sc[2 * i], sc[2 * i + 1]);
        mx = fmaxf(fmaxf(two[0], two[1]), fmaxf(two[2], two[3]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        if (one) {
            mv = mx + __uint_as_float(kv8_lds(mb + 384));
        } else {
            const uint4 e4 = kv8_lds16(mb + 384);
            mv = fmaxf(fmaxf(two[0] + __uint_as_float(e4.x), two[1] + __uint_as_float(e4.y)),
                       fmaxf(two[2] + __uint_as_float(e4.z), two[3] + __uint_as_float(e4.w)));
            mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, 1));
            mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, 2));
        }
        mx = fmaxf(mx, m);
        const float ref = mx == -INFINITY ? 0.f : mx, dm = m - ref;
        const float was = kv8_up(d);
        d = fmaxf(fmaxf(d + dm, mv - ref), kKv8MinD);
        const float up = kv8_up(d);
        const float al = kv8_ex2(dm), ao = kv8_ex2(dm + (up - was));
        m = mx;
        const float a0 = __shfl_sync(0xffffffffu, ao, 8 * t);  // of columns 2 t and 2 t + 1
        const float a1 = __shfl_sync(0xffffffffu, ao, 8 * t + 4);
        // ---- weights, and the f16 halves of their products with V's scales
        uint32_t ph[4], pl[PLO ? 4 : 1];
        {
            // a scale that leaves fp32 here is one of weights below 2^-100
            const float c = kv8_pow2(up, 1);
            const uint4 r4 = kv8_lds16(mb + 128);
            float v[4];
            v[0] = v[1] = v[2] = v[3] = kv8_finite(__uint_as_float(r4.x) * c);
            if (!one) {
                v[1] = kv8_finite(__uint_as_float(r4.y) * c);
                v[2] = kv8_finite(__uint_as_float(r4.z) * c);
                v[3] = kv8_finite(__uint_as_float(r4.w) * c);
            }
            float ls = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float p0 = kv8_ex2(sc[2 * i] - ref), p1 = kv8_ex2(sc[2 * i + 1] - ref);
                ls += p0 + p1;
                const float w0 = p0 * v[i], w1 = p1 * v[i];
                ph[i] = f16x2_rn(w0, w1);
                const float2 f = f16x2_floats(ph[i]);
                const uint32_t low = f16x2_rn(w0 - f.x, w1 - f.y);
                if constexpr (PLO) pl[i] = low;
                else ph[i] = g >= 4 ? low : ph[i];  // columns 4..7 carry the low halves of columns 0..3
            }
            l = fmaf(l, al, ls);
        }

        // ---- O^T = O^T alpha + V^T P^T
        cp_async_wait<1>();
        __syncwarp();  // every lane's copies of V have landed
        // PLO: 16 tokens at a time, each added to the output on its own, for the low halves' registers
        constexpr int HALVES = PLO ? 2 : 1, NE = 2 / HALVES;
#pragma unroll
        for (int half = 0; half < HALVES; ++half) {
            uint4 vv[4 * NE];
#pragma unroll
            for (int i = 0; i < 2 * NE; ++i) {
                vv[2 * i] = kv8_lds16(va0 + (2 * half + i) * 8 * kDh);
                vv[2 * i + 1] = kv8_lds16(va1 + (2 * half + i) * 8 * kDh);
            }
            if (!whole) {  // rows behind the sequence may hold anything: a weight of 0 does not undo a NaN
#pragma unroll
                for (int i = 0; i < 2 * NE; ++i) {
                    const int n = (int)kv8_lds(mb + 256 + 4 * (2 * half + i));
                    if (2 * t >= n) vv[2 * i] = make_uint4(0, 0, 0, 0);
                    if (2 * t + 1 >= n) vv[2 * i + 1] = make_uint4(0, 0, 0, 0);
                }
            }
            if (half == HALVES - 1) {
                __syncwarp();  // the V rows are read
                copy(it + 1, p.V8, kKv8SlotV);
            }
#pragma unroll
            for (int w = 0; w < 4; ++w) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float c[4];
#pragma unroll
                    for (int e = 0; e < NE; ++e) {  // 16 tokens
                        const int k = 2 * (half + e);
                        const uint32_t y0 = __byte_perm((&vv[4 * e].x)[w], (&vv[4 * e + 1].x)[w], i ? 0x7362 : 0x5140);
                        const uint32_t y1 = __byte_perm((&vv[4 * e + 2].x)[w], (&vv[4 * e + 3].x)[w], i ? 0x7362 : 0x5140);
                        const uint32_t b0 = e4m3lo_f16x2(y0), b1 = e4m3hi_f16x2(y0);
                        const uint32_t b2 = e4m3lo_f16x2(y1), b3 = e4m3hi_f16x2(y1);
                        if (e == 0) mma_f16(c, b0, b1, b2, b3, ph[k], ph[k + 1], zero);
                        else mma_f16(c, b0, b1, b2, b3, ph[k], ph[k + 1], c);
                        if constexpr (PLO) mma_f16(c, b0, b1, b2, b3, pl[k], pl[k + 1], c);
                    }
                    float(&oo)[4] = o[2 * w + i];
                    if (half == 0) {
                        oo[0] = fmaf(oo[0], a0, c[0]);
                        oo[1] = fmaf(oo[1], a1, c[1]);
                        oo[2] = fmaf(oo[2], a0, c[2]);
                        oo[3] = fmaf(oo[3], a1, c[3]);
                    } else {
                        oo[0] += c[0];
                        oo[1] += c[1];
                        oo[2] += c[2];
                        oo[3] += c[3];
                    }
                }
            }
        }
    }

    // ---- join the warps
    float(*s_o)[kKv8MaxRows][kDh] = reinterpret_cast<float(*)[kKv8MaxRows][kDh]>(smem);
    float(*s_ml)[kKv8MaxRows][2] = reinterpret_cast<float(*)[kKv8MaxRows][2]>(smem + WARPS * kKv8MaxRows * kDh * 4);
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    const float down = kv8_pow2(kv8_up(d), -1);  // of the lane's row; of columns 2 t and 2 t + 1:
    const float downs[2] = {__shfl_sync(0xffffffffu, down, 8 * t), __shfl_sync(0xffffffffu, down, 8 * t + 4)};
    if constexpr (!PLO) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][e] += __shfl_xor_sync(0xffffffffu, o[j][e], 2);
    }
    cp_async_wait<0>();
    __syncthreads();  // the tiles are done with
    const int my_cta = s_part[0], my_parts = s_part[1], my_row = s_part[2];
    if (t == 0 && g < p.rows) {
        s_ml[warp][g][0] = m;
        s_ml[warp][g][1] = l;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int r = 2 * t + e;
        if (r < p.rows) {
#pragma unroll
            for (int w = 0; w < 4; ++w)
                *reinterpret_cast<float4*>(&s_o[warp][r][16 * g + 4 * w]) =
                    make_float4(o[2 * w][e] * downs[e], o[2 * w][2 + e] * downs[e], o[2 * w + 1][e] * downs[e],
                                o[2 * w + 1][2 + e] * downs[e]);
        }
    }
    __syncthreads();
    // Each thread sums four columns of a row over the warps. A row's maximum, sum and factors: with one or two
    // rows every thread works them out for itself, with more a warp does it for all.
    const bool shared_factors = p.rows > 2;
    if (shared_factors) {
        for (int r = warp; r < p.rows; r += WARPS) {
            const float mw = lane < WARPS ? s_ml[lane & (WARPS - 1)][r][0] : -INFINITY;
            float M = mw;
#pragma unroll
            for (int k = 1; k < WARPS; k <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, k));
            const float f = mw == -INFINITY ? 0.f : kv8_ex2(mw - M);
            float L = lane < WARPS ? f * s_ml[lane & (WARPS - 1)][r][1] : 0.f;
#pragma unroll
            for (int k = 1; k < WARPS; k <<= 1) L += __shfl_xor_sync(0xffffffffu, L, k);
            __syncwarp();
            if (lane < WARPS) s_ml[lane][r][0] = f;
            if (lane == 0) {
                s_ml[0][r][1] = L;
                s_qmul[r] = M;
            }
        }
        __syncthreads();
    }
    for (int i = tid; i < p.rows * (kDh / 4); i += WARPS * 32) {
        const int r = i >> 5, d = (i & 31) * 4;
        float M = -INFINITY, L = 0.f;
        if (shared_factors) {
            M = s_qmul[r];
            L = s_ml[0][r][1];
        } else {
#pragma unroll
            for (int w = 0; w < WARPS; ++w) M = fmaxf(M, s_ml[w][r][0]);
        }
        float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            float f = s_ml[w][r][0];
            if (!shared_factors) {
                f = f == -INFINITY ? 0.f : kv8_ex2(f - M);
                L = fmaf(f, s_ml[w][r][1], L);
            }
            const float4 v = *reinterpret_cast<const float4*>(&s_o[w][r][d]);
            A.x = fmaf(f, v.x, A.x); A.y = fmaf(f, v.y, A.y);
            A.z = fmaf(f, v.z, A.z); A.w = fmaf(f, v.w, A.w);
        }
        if (my_parts == 1) {
            *reinterpret_cast<float4*>(p.out + (int64_t)(my_row + r) * kDh + d) =
                L == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(A.x / L, A.y / L, A.z / L, A.w / L);
            if (d == 0 && p.lse != nullptr)
                p.lse[my_row + r] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
        } else {
            const int64_t at = (int64_t)my_cta * kKv8MaxRows + r;
            *reinterpret_cast<float4*>(p.part_o + at * kDh + d) = A;
            if (d == 0) {
                // The join takes a maximum of -inf for a part without tokens. Scores that are all NaN leave it so
                // too (a maximum passes NaN over), with a sum that is NaN: any finite maximum carries that on.
                p.part_ml[at * 2] = M == -INFINITY && L != 0.f ? 0.f : M;
                p.part_ml[at * 2 + 1] = L;
            }
        }
    }
}

// Join of the runs that were cut: `wpr` warps to a row (a query head), a lane owns four of its Dh columns.
constexpr int kKv8MergeU = 8;  // partials in flight per lane

__global__ void __launch_bounds__(1024)
k_kv8_attn_merge(const Kv8AttnParams p, const Kv8Tab tab, int wpr) {
    extern __shared__ __align__(16) float s_join[];  // [warp][Dh + 4]: columns, m, l
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
    const int r = (blockIdx.x * (blockDim.x >> 5) + wp) / wpr;  // row of out
    const int sub = wp & (wpr - 1);
    const int b = r / p.H, run = (r - b * p.H) / p.rows, row = r & (p.rows - 1);
    int parts = 0, cta = 0;
    if (b < tab.B) {
        const int place = tab.place_of[b];
        parts = (tab.cta_off[place + 1] - tab.cta_off[place]) >> p.runs_log2;
        cta = tab.cta_off[place] + run;
    }
    pdl_wait();
    // parts == 1: written by the CTA that held the run
    float m = -INFINITY, l = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    if (parts > 1) {
        for (int i0 = sub; i0 < parts; i0 += wpr * kKv8MergeU) {
            float4 v[kKv8MergeU];
            float2 ml[kKv8MergeU];
#pragma unroll
            for (int k = 0; k < kKv8MergeU; ++k) {
                const int i = i0 + k * wpr;
                v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                ml[k] = make_float2(-INFINITY, 0.f);
                if (i < parts) {
                    const int64_t at = (int64_t)(cta + (i << p.runs_log2)) * kKv8MaxRows + row;
                    v[k] = *reinterpret_cast<const float4*>(p.part_o + at * kDh + lane * 4);
                    ml[k] = *reinterpret_cast<const float2*>(p.part_ml + at * 2);
                }
            }
            float mc = m;
#pragma unroll
            for (int k = 0; k < kKv8MergeU; ++k) mc = fmaxf(mc, ml[k].x);
            if (mc == -INFINITY) continue;
            const float f = m == -INFINITY ? 0.f : kv8_ex2(m - mc);
            l *= f;
            a.x *= f; a.y *= f; a.z *= f; a.w *= f;
#pragma unroll
            for (int k = 0; k < kKv8MergeU; ++k) {
                if (ml[k].x != -INFINITY) {
                    const float w = kv8_ex2(ml[k].x - mc);
                    l = fmaf(w, ml[k].y, l);
                    a.x = fmaf(w, v[k].x, a.x); a.y = fmaf(w, v[k].y, a.y);
                    a.z = fmaf(w, v[k].z, a.z); a.w = fmaf(w, v[k].w, a.w);
                }
            }
            m = mc;
        }
    }
    if (wpr > 1) {
        float* mine = s_join + wp * (kDh + 4);
        *reinterpret_cast<float4*>(mine + lane * 4) = a;
        if (lane == 0) {
            mine[kDh] = m;
            mine[kDh + 1] = l;
        }
        __syncthreads();
        if (sub != 0) return;
        m = -INFINITY;
        l = 0.f;
        a = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < wpr; ++k) m = fmaxf(m, mine[k * (kDh + 4) + kDh]);
        for (int k = 0; k < wpr; ++k) {
            const float* o = mine + k * (kDh + 4);
            if (o[kDh] == -INFINITY) continue;
            const float w = kv8_ex2(o[kDh] - m);
            const float4 v = *reinterpret_cast<const float4*>(o + lane * 4);
            l = fmaf(w, o[kDh + 1], l);
            a.x = fmaf(w, v.x, a.x); a.y = fmaf(w, v.y, a.y);
            a.z = fmaf(w, v.z, a.z); a.w = fmaf(w, v.w, a.w);
        }
    }
    if (parts > 1) {
        const float4 y = l == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(a.x / l, a.y / l, a.z / l, a.w / l);
        *reinterpret_cast<float4*>(p.out + (int64_t)r * kDh + lane * 4) = y;
        if (lane == 0 && p.lse != nullptr) p.lse[r] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
    }
}

// ------------------------------------------------------------------ host side
template <bool BF16, bool PLO, int WARPS>
static cudaError_t kv8_set_attrs(int* least) {
    const cudaError_t e = set_smem_attrs(k_kv8_attn<BF16, PLO, WARPS>, kv8_smem(WARPS));
    if (e != cudaSuccess) return e;
    int n = 0;
    const cudaError_t f = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, k_kv8_attn<BF16, PLO, WARPS>, WARPS * 32,
                                                                        kv8_smem(WARPS));
    if (n * WARPS < *least) *least = n * WARPS;
    return f;
}

template <int WARPS>
static cudaError_t kv8_set_all(int* least) {
    cudaError_t e = kv8_set_attrs<true, false, WARPS>(least);
    if (e == cudaSuccess) e = kv8_set_attrs<true, true, WARPS>(least);
    if (e == cudaSuccess) e = kv8_set_attrs<false, false, WARPS>(least);
    if (e == cudaSuccess) e = kv8_set_attrs<false, true, WARPS>(least);
    return e;
}

// Kernel attributes; every variant has to reach 16 warps an SM, which the plan counts on.
cudaError_t kv8_init_attrs() {
    int least = 16;
    cudaError_t e = kv8_set_all<4>(&least);
    if (e == cudaSuccess) e = kv8_set_all<8>(&least);
    if (e == cudaSuccess) e = kv8_set_all<16>(&least);
    return e == cudaSuccess && least < 16 ? cudaErrorLaunchOutOfResources : e;
}

// Most CTAs that a call with cut runs launches: four of four warps an SM.
static int kv8_max_ctas(int num_sms) { return 4 * num_sms; }
size_t kv8_part_o_bytes(int num_sms) { return (size_t)kv8_max_ctas(num_sms) * kKv8MaxRows * kDh * 4; }
size_t kv8_part_ml_bytes(int num_sms) { return (size_t)kv8_max_ctas(num_sms) * kKv8MaxRows * 2 * 4; }

// The least tiles per CTA (at least `least`) with which all runs' parts are `slots` CTAs or fewer; if there
// are more runs than that, what leaves every run whole. `all`: the tiles of all runs, `most` of the longest.
static int kv8_part_tiles(const int* tiles, int B, int64_t runs_b, int64_t slots, int least, int most, int64_t all) {
    const int64_t runs = runs_b * B;
    if (runs >= slots || most <= least) return most > least ? most : least;
    // the parts are at least all / T and less than all / T + runs
    int64_t lo = (all + slots - 1) / slots, hi = (all + slots - runs - 1) / (slots - runs);
    lo = lo < least ? least : lo;
    hi = hi > most ? most : hi;
    while (lo < hi) {
        const int mid = (int)(lo + (hi - lo) / 2);
        int64_t n = 0;
        for (int b = 0; b < B; ++b) n += runs_b * ((tiles[b] + mid - 1) / mid);
        if (n <= slots) hi = mid; else lo = mid + 1;
    }
    return (int)lo;
}

// Microseconds that the runs take in parts of `per` tiles, `slots` CTAs at a time: the larger of what the
// fullest SM computes (0.2 a tile while its 16 warps have one each, 0.137 from then on; 3.3 for a round of
// CTAs to start and to join its warps) and what memory reads (8 KB a tile at 7 TB/s), and, where runs are left
// to be joined, 2 for that and 0.8 for the host to launch it. Measured (bf16): 8 runs of 8 tiles 4.6 us as 8
// CTAs of 8 warps, 5.3 as 16 of 4; of 16 tiles 6.0 as 8 of 16 warps, 5.8 as 32 of 4; of 32 tiles 6.0 as 64 of 4;
// 128 runs of 16 tiles 6.8 as 128 of 16 warps, 9.0 as 512 of 4.
static double kv8_estimate(const int* tiles, int B, int64_t runs_b, int per, int64_t all, int num_sms, int64_t slots) {
    int64_t ctas = 0;
    for (int b = 0; b < B; ++b) ctas += runs_b * ((tiles[b] + per - 1) / per);
    const int64_t rounds = (ctas + slots - 1) / slots, per_sm = (ctas + num_sms - 1) / num_sms, full = slots / num_sms;
    const double load = (double)per * (double)(per_sm < full ? per_sm : full);
    const double compute = load < 16. ? 0.2 * load : 1. + 0.137 * load;
    const double memory = 3.3 + 0.00117 * (double)all, busy = (double)rounds * (3.3 + compute);
    return (busy > memory ? busy : memory) + (ctas > runs_b * B ? 2.8 : 0.);
}

template <bool BF16, bool PLO>
static cudaError_t kv8_launch(cudaLaunchConfig_t& cfg, int warps, const Kv8AttnParams& p, const Kv8Tab& kt,
                              uint32_t* err) {
    cfg.blockDim = dim3(warps * 32, 1, 1);
    cfg.dynamicSmemBytes = kv8_smem(warps);
    return warps == 4   ? cudaLaunchKernelEx(&cfg, k_kv8_attn<BF16, PLO, 4>, p, kt, err)
           : warps == 8 ? cudaLaunchKernelEx(&cfg, k_kv8_attn<BF16, PLO, 8>, p, kt, err)
                        : cudaLaunchKernelEx(&cfg, k_kv8_attn<BF16, PLO, 16>, p, kt, err);
}

// `tab`: the kept chunks of each sequence, or all of them where ids is null.
cudaError_t launch_kv8_attn(const lsa_dims& d, const SeqTable& tab, const lsa_kv8_cache& cache, const Kv8Geom& g,
                            int num_sms, const void* q, const int32_t* ids, const int32_t* counts,
                            const int32_t* seq_len, int len_add, float* part_o, float* part_ml, float* out,
                            float* lse, uint32_t* err, cudaStream_t stream, bool pdl) {
    Kv8AttnParams p = {};
    p.g = g;
    p.q = (const uint8_t*)q;
    p.K8 = (const uint8_t*)cache.K8;
    p.V8 = (const uint8_t*)cache.V8;
    p.k_scale = cache.k_scale;
    p.v_scale = cache.v_scale;
    p.ids = ids;
    p.counts = counts;
    p.seq_len = seq_len;
    p.out = out;
    p.lse = lse;
    p.part_o = part_o;
    p.part_ml = part_ml;
    p.H = d.H;
    const int group = d.H / g.Hkv;
    p.rows = group < kKv8MaxRows ? group : kKv8MaxRows;
    p.rts = group / p.rows;
    const int runs_b = g.Hkv * p.rts;
    while ((1 << p.runs_log2) < runs_b) ++p.runs_log2;
    p.len_add = len_add;
    p.num_sms = num_sms;
    p.qscale = 1.4426950408889634f / sqrtf((float)kDh);

    Kv8Tab kt;
    kt.B = tab.B;
    for (int b = 0; b <= tab.B; ++b) {
        kt.chunk_off[b] = tab.chunk_off[b];
        kt.kept_off[b] = tab.kept_off[b];
    }
    int tiles[kMaxB], most = 0;  // of a sequence's runs, and of the longest run
    int64_t all = 0;
    for (int b = 0; b < tab.B; ++b) {
        tiles[b] = (int)((((int64_t)(tab.kept_off[b + 1] - tab.kept_off[b]) << g.c_log2) + kKv8Tile - 1) / kKv8Tile);
        most = tiles[b] > most ? tiles[b] : most;
        all += (int64_t)tiles[b] * runs_b;
    }
    // 16 warps to an SM, as CTAs of 16, 8 or 4. Wide CTAs leave less to join but cut the work in lumps, and
    // idle warps where runs are short; the form with the least estimated time is taken, the wider one where
    // it hardly matters.
    int warps = 0, per = 0;
    double best = 0.;
    for (int w = 16; w >= 4; w >>= 1) {
        const int64_t slots = (int64_t)num_sms * (16 / w);
        const int n = kv8_part_tiles(tiles, tab.B, runs_b, slots, w, most, all);
        const double t = kv8_estimate(tiles, tab.B, runs_b, n, all, num_sms, slots);
        if (warps == 0 || t < 0.98 * best) {
            warps = w;
            per = n;
            best = t;
        }
    }
    // Places: the sequences by the length of their longest parts, longest first.
    int part_len[kMaxB], order[kMaxB];
    for (int b = 0; b < tab.B; ++b) {
        const int parts = (tiles[b] + per - 1) / per;
        part_len[b] = (tiles[b] + parts - 1) / parts;
        order[b] = b;
    }
    std::sort(order, order + tab.B,
              [&](int x, int y) { return part_len[x] > part_len[y] || (part_len[x] == part_len[y] && x < y); });
    int64_t ctas = 0;
    bool cut = false;
    for (int i = 0; i < tab.B; ++i) {
        const int b = order[i], parts = (tiles[b] + per - 1) / per;
        kt.seq_at[i] = (uint8_t)b;
        kt.place_of[b] = (uint8_t)i;
        kt.cta_off[i] = (int32_t)ctas;
        ctas += (int64_t)parts * runs_b;
        cut |= parts > 1;
    }
    kt.cta_off[tab.B] = (int32_t)ctas;

    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    cfg.gridDim = dim3((unsigned)ctas, 1, 1);
    const bool plo = p.rows > 4;
    cudaError_t e = d.kv_dtype == LSA_BF16 ? (plo ? kv8_launch<true, true>(cfg, warps, p, kt, err)
                                                  : kv8_launch<true, false>(cfg, warps, p, kt, err))
                                           : (plo ? kv8_launch<false, true>(cfg, warps, p, kt, err)
                                                  : kv8_launch<false, false>(cfg, warps, p, kt, err));
    if (e != cudaSuccess || !cut) return e;
    // One warp to a row where a run has few parts; eight, and 32 (a block), where it has many.
    const int64_t rows = (int64_t)d.B * d.H;
    const int64_t span = ctas / ((int64_t)runs_b * tab.B);
    const int wpr = span <= 8 ? 1 : span <= 64 ? 8 : 32;
    const int threads = wpr == 32 ? 1024 : 256;
    cfg.numAttrs = 1;  // the join always follows the split kernel: overlap its launch
    cfg.gridDim = dim3((unsigned)((rows * wpr * 32 + threads - 1) / threads), 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = wpr == 1 ? 0 : threads / 32 * (kDh + 4) * 4;
    return cudaLaunchKernelEx(&cfg, k_kv8_attn_merge, p, kt, wpr);
}

// Whether the kept tokens of one head and the rows of the cache are few enough for 32-bit counts
// (2^31 rows of K8 are 256 GiB). A lane looks up to two batches past its warp's last tile.
bool kv8_attn_fits(const SeqTable& tab, const Kv8Geom& g) {
    const int64_t slack = ((int64_t)tab.B + 2 * kKv8Batch * 16) * kKv8Tile;
    return ((int64_t)tab.kept_off[tab.B] << g.c_log2) + slack < (1ll << 31) &&
           ((int64_t)tab.chunk_off[tab.B] << (g.c_log2 + g.h_log2)) < (1ll << 31);
}

}  // namespace lsa
