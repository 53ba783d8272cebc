// kv8_attn.cu - split-K flash-decode attention over the kept chunks of the 8-bit K/V cache.
//
//     l_t = (q . k8_t) ks_t / sqrt(Dh),   out = sum_t softmax(l)_t vs_t v8_t
//
// for one decode query per sequence, H query heads sharing Hkv K/V heads in groups of H / Hkv.
//
// What bounds it: reading 2 Dh bytes a token and K/V head. Converting 8-bit codes and multiplying them
// on the CUDA cores would take several instructions a byte, so both products run on the tensor cores
// in f16 (m16n8k16): an e4m3 code is an f16 number exactly, and one conversion unpacks two. The
// products are a few rows wide (one group of query heads), far from what fills a tcgen05 tile; the
// warp-level instruction takes its operands from registers, where the loads put them.
//
//  * Fragments straight from memory. The reduction index of a product may be permuted as long as both
//    operands agree, so each lane loads whole 16- or 32-byte pieces and uses them as they come:
//      S = q K^T   lane (g, t) of a warp (g = lane / 4, t = lane % 4) holds bytes 32 t .. 32 t + 31 of
//                  token g's row: step s of the 8 steps over Dh takes its bytes 4 s .. 4 s + 3;
//      O^T = V^T P^T  lane (g, t) holds bytes 16 g .. 16 g + 15 of tokens 2 t and 2 t + 1: interleaving
//                  the two tokens' bytes (one byte permute per four) gives the pairs along the tokens.
//    S leaves its scores exactly where the second product wants P, so nothing is exchanged between.
//  * Full precision from f16 operands. A row of q is scaled by a power of two and, for fp32 queries,
//    split into the f16 numbers hi + lo; lo sits in the eight rows of the 16-row operand that a group
//    of up to 8 heads leaves free. The weights P, at most 2^14, are split in the same way: with 4 heads
//    or fewer, lo takes the free half of the 8 columns (no extra product), with 8 heads a second
//    product. Weights keep 22 bits down to 2^-28 of the largest and reach down to 2^-39.
//  * V's scale multiplies the weight, relative to the largest scale seen (vref), which the running
//    output carries, so that the products stay within f16's range whatever the scales are.
//  * The cache's (chunk, head) runs are contiguous; each warp streams tiles of 16 tokens of one
//    (sequence, K/V head) run, with its own running maximum, sum and output. The tiles of all runs form
//    one list that is split evenly over the CTAs; a CTA joins its warps in shared memory, and a run that
//    spans CTAs is joined by k_kv8_attn_merge. Runs that one CTA holds whole are written at once.
#include "kv8.cuh"

namespace lsa {

constexpr int kKv8Warps = 4;
constexpr int kKv8Threads = kKv8Warps * 32;
constexpr int kKv8CtasPerSm = 3;
constexpr int kKv8Stages = 4;      // tiles of a warp's ring
constexpr int kKv8Tile = 16;       // tokens per tile
constexpr int kKv8MaxRows = 8;     // query heads per run
constexpr float kKv8PShift = 14.f; // weights are at most 2^14

// Prefix tables of one call: the kept (or all) chunks and their tiles.
struct Kv8Tab {
    int32_t B;
    int32_t chunk_off[kMaxB + 1];
    int32_t kept_off[kMaxB + 1];
    int32_t tile_off[kMaxB + 1];  // prefix of the tiles of one (sequence, head) run
};

struct Kv8AttnParams {
    Kv8Geom g;
    const uint8_t *q, *K8, *V8;
    const float *k_scale, *v_scale;
    const int32_t *ids, *counts, *seq_len;  // nullable
    float *out, *lse, *part_o, *part_ml;    // lse nullable
    int32_t H;
    int32_t rows;       // query heads per run: min(group, 8)
    int32_t rts;        // runs per K/V head: group / rows
    int32_t len_add;    // added to seq_len
    int32_t G;          // CTAs
    int64_t F;          // tiles of all runs
    float qscale;       // log2(e) / sqrt(Dh)
};

// 2^x by the hardware's approximation (relative error ~2^-22; 2^-inf = 0).
__device__ __forceinline__ float kv8_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t f16x2_rn(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// ---------------------------------------------------------------- a warp's ring of tiles
// One slot: 16 rows of K, 16 rows of V (128 bytes each), then the tile's scales and token counts. A
// row's 16-byte units are XOR-swizzled by the row, so that both fragment reads are free of conflicts.
constexpr int kKv8SlotK = 0;
constexpr int kKv8SlotV = kKv8Tile * kDh;
constexpr int kKv8SlotMeta = 2 * kKv8Tile * kDh;  // ks[2], vs[2] (float), n[2] (int)
constexpr int kKv8SlotBytes = kKv8SlotMeta + 32;
constexpr int kKv8WarpBytes = kKv8Stages * kKv8SlotBytes;
constexpr int kKv8JoinBytes = kKv8Warps * kKv8MaxRows * (kDh + 2) * 4;
constexpr int kKv8Smem = kKv8Warps * kKv8WarpBytes > kKv8JoinBytes ? kKv8Warps * kKv8WarpBytes : kKv8JoinBytes;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 kv8_lds16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

// The run that a warp streams.
struct Kv8Run {
    int64_t chunk0;      // first chunk of the sequence
    int64_t len;         // tokens of the sequence that exist
    const int32_t* ids;  // nullable
    int n_b, kept, h;
};

// Start the copies of one tile into `slot`: first token t0 within the run, the ids of its two octets'
// chunks. The counts n are what the consumer goes by: an octet without tokens is not copied.
__device__ __forceinline__ void kv8_issue(uint32_t slot, const Kv8AttnParams& p, const Kv8Run& r, int t0, int id0,
                                          int id1, int lane, uint32_t* err) {
    const int cm = (1 << p.g.c_log2) - 1;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int tk = t0 + 8 * i, id = i ? id1 : id0;
        const int j = tk >> p.g.c_log2, w = tk & cm;
        int n = 0;
        if (j < r.kept) {
            if (id >= 0 && id < r.n_b) {
                const int64_t left = r.len - (((int64_t)id << p.g.c_log2) + w);
                n = left >= 8 ? 8 : left > 0 ? (int)left : 0;
            } else if (lane == 0) {
                set_error(err, kErrBadId);
            }
        }
        if (n > 0) {  // the whole octet lies in the cache, even where only part of it is used
            const int64_t ch = (r.chunk0 + id) * p.g.Hkv + r.h;
            const int64_t at = ((ch << p.g.c_log2) + w) * kDh + lane * 16;
            const int row = lane >> 3, unit = lane & 7;
            const uint32_t d0 = slot + (8 * i + row) * kDh + ((unit ^ row) << 4);
            const uint32_t d1 = slot + (8 * i + row + 4) * kDh + ((unit ^ (row + 4)) << 4);
            cp_async16(d0 + kKv8SlotK, p.K8 + at);
            cp_async16(d1 + kKv8SlotK, p.K8 + at + 512);
            cp_async16(d0 + kKv8SlotV, p.V8 + at);
            cp_async16(d1 + kKv8SlotV, p.V8 + at + 512);
            const int64_t si = ch * p.g.spc + (w >> p.g.sb_log2);
            if (lane < 2) cp_async4(slot + kKv8SlotMeta + 8 * lane + 4 * i, (lane ? p.v_scale : p.k_scale) + si);
        }
        if (lane == 0)
            asm volatile("st.shared.s32 [%0], %1;" ::"r"(slot + kKv8SlotMeta + 16 + 4 * i), "r"(n) : "memory");
    }
}

// grid G, kKv8Threads threads. QLO: fp32 queries (hi + lo); PLO: groups of 8 (a second product for lo).
template <bool QLO, bool PLO>
__global__ void __launch_bounds__(kKv8Threads, kKv8CtasPerSm)
k_kv8_attn(const Kv8AttnParams p, const Kv8Tab tab, uint32_t* err) {
    extern __shared__ __align__(128) uint8_t smem[];
    // the join's buffers take the ring's place once a run's tiles are done
    float(*s_o)[kKv8MaxRows][kDh] = reinterpret_cast<float(*)[kKv8MaxRows][kDh]>(smem);
    float(*s_ml)[kKv8MaxRows][2] =
        reinterpret_cast<float(*)[kKv8MaxRows][2]>(smem + kKv8Warps * kKv8MaxRows * kDh * 4);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int64_t u0 = (int64_t)blockIdx.x * p.F / p.G, u1 = ((int64_t)blockIdx.x + 1) * p.F / p.G;
    const int runs_b = p.g.Hkv * p.rts;
    const int my_row = g & (p.rows - 1);
    const uint32_t ring = smem_u32(smem) + warp * kKv8WarpBytes;
    // byte offsets of this lane's fragments in a slot (second octet: + 8 rows)
    const uint32_t k_at0 = g * kDh + ((2 * t ^ g) << 4), k_at1 = g * kDh + (((2 * t + 1) ^ g) << 4);
    const uint32_t v_at0 = kKv8SlotV + 2 * t * kDh + ((g ^ 2 * t) << 4);
    const uint32_t v_at1 = kKv8SlotV + (2 * t + 1) * kDh + ((g ^ (2 * t + 1)) << 4);
    pdl_trigger();
    pdl_wait();

    int b = 0;
    {
        int lo = 0, hi = tab.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((int64_t)tab.tile_off[mid] * runs_b <= u0) lo = mid; else hi = mid - 1;
        }
        b = lo;
    }
    for (int64_t u = u0; u < u1;) {
        // ---- the run that holds unit u
        while (u >= (int64_t)tab.tile_off[b + 1] * runs_b) ++b;
        const int tiles = tab.tile_off[b + 1] - tab.tile_off[b];
        const int64_t rel = u - (int64_t)tab.tile_off[b] * runs_b;
        const int run = (int)(rel / tiles);
        const int tile0 = (int)(rel - (int64_t)run * tiles);
        const int tile1 = (int)min((int64_t)tiles, tile0 + (u1 - u));
        const int h = run / p.rts, rt = run - h * p.rts;
        Kv8Run r;
        r.h = h;
        r.n_b = tab.chunk_off[b + 1] - tab.chunk_off[b];
        r.chunk0 = tab.chunk_off[b];
        r.kept = tab.kept_off[b + 1] - tab.kept_off[b];
        r.ids = p.ids != nullptr ? p.ids + tab.kept_off[b] : nullptr;
        if (p.counts != nullptr) r.kept = max(0, min(r.kept, p.counts[b]));
        r.len = (int64_t)r.n_b << p.g.c_log2;
        if (p.seq_len != nullptr) r.len = min(r.len, (int64_t)p.seq_len[b] + p.len_add);
        const int qrow0 = b * p.H + (h * p.rts + rt) * p.rows;

        // ---- q: 32 values of row my_row, scaled by a power of two, as f16 operands
        uint32_t qa[8][2], ql[QLO ? 8 : 1][2];
        float qmul;
        {
            float x[32], top = 0.f;
            const int64_t at = (int64_t)(qrow0 + my_row) * kDh + t * 32;
            if constexpr (QLO) {
                const float4* src = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p.q) + at);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float4 f = src[e];
                    x[4 * e] = f.x; x[4 * e + 1] = f.y; x[4 * e + 2] = f.z; x[4 * e + 3] = f.w;
                }
            } else {
                const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.q) + at);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint4 f = src[e];
                    x[8 * e] = bf16lo(f.x); x[8 * e + 1] = bf16hi(f.x);
                    x[8 * e + 2] = bf16lo(f.y); x[8 * e + 3] = bf16hi(f.y);
                    x[8 * e + 4] = bf16lo(f.z); x[8 * e + 5] = bf16hi(f.z);
                    x[8 * e + 6] = bf16lo(f.w); x[8 * e + 7] = bf16hi(f.w);
                }
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) top = fmaxf(top, fabsf(x[e]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // top < 2^(ex + 1): times 2^(14 - ex) it stays below 2^15. The factor is kept within fp32.
            int ex = (int)(__float_as_uint(top) >> 23) - 127;
            ex = ex < -100 ? -100 : ex > 127 ? 127 : ex;
            const float up = __uint_as_float((uint32_t)(14 - ex + 127) << 23);
            qmul = p.qscale * __uint_as_float((uint32_t)(ex - 14 + 127) << 23);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float a = x[4 * e + 2 * i] * up, c = x[4 * e + 2 * i + 1] * up;
                    qa[e][i] = f16x2_rn(a, c);
                    if constexpr (QLO) {
                        const float2 f = f16x2_floats(qa[e][i]);
                        ql[e][i] = f16x2_rn(a - f.x, c - f.y);
                    }
                }
            }
        }

        float o[8][4], m = -INFINITY, l = 0.f, vref = 0.f, inv_vref = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;

        // This warp's tiles are tile0 + warp + 4 i, i < n_it. Lane i holds the chunk ids of its tiles i,
        // i + 32, ...: one load serves 32 tiles.
        const int n_it = (tile1 - tile0 - warp + kKv8Warps - 1) / kKv8Warps;
        int idv0 = 0, idv1 = 0;
        auto issue = [&](int i) {
            if (i < n_it) {
                const int first = tile0 + warp + kKv8Warps * i;
                if ((i & 31) == 0) {
                    const int64_t tk = (int64_t)(first + kKv8Warps * lane) * kKv8Tile;
                    const int64_t j0 = tk >> p.g.c_log2, j1 = (tk + 8) >> p.g.c_log2;
                    idv0 = j0 >= r.kept ? -1 : r.ids != nullptr ? r.ids[j0] : (int)j0;
                    idv1 = j1 >= r.kept ? -1 : r.ids != nullptr ? r.ids[j1] : (int)j1;
                }
                const int id0 = __shfl_sync(0xffffffffu, idv0, i & 31), id1 = __shfl_sync(0xffffffffu, idv1, i & 31);
                kv8_issue(ring + (i % kKv8Stages) * kKv8SlotBytes, p, r, first * kKv8Tile, id0, id1, lane, err);
            }
            cp_async_commit();  // one group per tile, empty past the end
        };
#pragma unroll
        for (int i = 0; i < kKv8Stages - 1; ++i) issue(i);

        for (int it = 0; it < n_it; ++it) {
            cp_async_wait<kKv8Stages - 2>();
            __syncwarp();  // every lane's copies of this tile have landed, and the last tile's reads are done
            issue(it + kKv8Stages - 1);
            const uint32_t slot = ring + (it % kKv8Stages) * kKv8SlotBytes;
            int n[2];
            float ks[2], vs[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                asm volatile("ld.shared.s32 %0, [%1];" : "=r"(n[i]) : "r"(slot + kKv8SlotMeta + 16 + 4 * i));
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(ks[i]) : "r"(slot + kKv8SlotMeta + 4 * i));
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(vs[i]) : "r"(slot + kKv8SlotMeta + 8 + 4 * i));
                if (n[i] == 0) vs[i] = 0.f;
            }
            if (n[0] + n[1] == 0) continue;  // uniform in the warp

            // ---- S: rows of q against the tile's tokens, in two chains of four products
            float sc[4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint4 ka = kv8_lds16(slot + k_at0 + 8 * i * kDh), kb = kv8_lds16(slot + k_at1 + 8 * i * kDh);
                const uint32_t kw[8] = {ka.x, ka.y, ka.z, ka.w, kb.x, kb.y, kb.z, kb.w};
                float c[4] = {0.f, 0.f, 0.f, 0.f}, e[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    mma_f16(s < 4 ? c : e, qa[s][0], QLO ? ql[QLO ? s : 0][0] : 0u, qa[s][1],
                            QLO ? ql[QLO ? s : 0][1] : 0u, e4m3lo_f16x2(kw[s]), e4m3hi_f16x2(kw[s]));
                const float f = qmul * ks[i];
                const float s0 = QLO ? (c[0] + e[0]) + (c[2] + e[2]) : c[0] + e[0];
                const float s1 = QLO ? (c[1] + e[1]) + (c[3] + e[3]) : c[1] + e[1];
                sc[2 * i] = 2 * t < n[i] ? s0 * f : -INFINITY;
                sc[2 * i + 1] = 2 * t + 1 < n[i] ? s1 * f : -INFINITY;
            }
            // ---- running maximum of row my_row, and V's reference scale
            float mx = fmaxf(fmaxf(sc[0], sc[1]), fmaxf(sc[2], sc[3]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float vtop = fmaxf(vs[0], vs[1]);
            if (__any_sync(0xffffffffu, mx > m) || vtop > vref) {
                const float mn = fmaxf(m, mx);
                const float al = mn == -INFINITY ? 1.f : kv8_ex2(m - mn);
                m = mn;
                l *= al;
                float a0 = __shfl_sync(0xffffffffu, al, 8 * t), a1 = __shfl_sync(0xffffffffu, al, 8 * t + 4);
                if (vtop > vref && vtop >= 1.17549435e-38f) {
                    const float f = vref / vtop;
                    a0 *= f;
                    a1 *= f;
                    vref = vtop;
                    inv_vref = 1.f / vtop;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    o[j][0] *= a0;
                    o[j][1] *= a1;
                    o[j][2] *= a0;
                    o[j][3] *= a1;
                }
            }
            // ---- weights (times 2^14, which out = O / l cancels) and their f16 halves
            const float ms = m == -INFINITY ? 0.f : m - kKv8PShift;
            uint32_t ph[2], pl[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float p0 = kv8_ex2(sc[2 * i] - ms), p1 = kv8_ex2(sc[2 * i + 1] - ms);
                l += p0 + p1;
                const float rv = vs[i] * inv_vref;
                const float w0 = p0 * rv, w1 = p1 * rv;
                ph[i] = f16x2_rn(w0, w1);
                const float2 f = f16x2_floats(ph[i]);
                pl[i] = f16x2_rn(w0 - f.x, w1 - f.y);
                if (!PLO && g >= 4) ph[i] = pl[i];  // columns 4..7 carry the low halves of columns 0..3
            }
            // ---- O^T += V^T P^T
            uint4 vv[4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                vv[2 * i] = kv8_lds16(slot + v_at0 + 8 * i * kDh);
                vv[2 * i + 1] = kv8_lds16(slot + v_at1 + 8 * i * kDh);
                if (n[i] < 8) {  // rows behind the sequence may hold anything: a weight of 0 does not undo a NaN
                    if (2 * t >= n[i]) vv[2 * i] = make_uint4(0, 0, 0, 0);
                    if (2 * t + 1 >= n[i]) vv[2 * i + 1] = make_uint4(0, 0, 0, 0);
                }
            }
            const uint32_t *v0 = &vv[0].x, *v1 = &vv[1].x, *v2 = &vv[2].x, *v3 = &vv[3].x;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t y0 = __byte_perm(v0[w], v1[w], i ? 0x7362 : 0x5140);
                    const uint32_t y1 = __byte_perm(v2[w], v3[w], i ? 0x7362 : 0x5140);
                    const uint32_t a0 = e4m3lo_f16x2(y0), a1 = e4m3hi_f16x2(y0);
                    const uint32_t a2 = e4m3lo_f16x2(y1), a3 = e4m3hi_f16x2(y1);
                    mma_f16(o[2 * w + i], a0, a1, a2, a3, ph[0], ph[1]);
                    if constexpr (PLO) mma_f16(o[2 * w + i], a0, a1, a2, a3, pl[0], pl[1]);
                }
            }
        }

        // ---- join the warps
        cp_async_wait<0>();
        __syncthreads();  // the rings are done with
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if constexpr (!PLO) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[j][e] += __shfl_xor_sync(0xffffffffu, o[j][e], 2);
        }
        if (t == 0 && g < p.rows) {
            s_ml[warp][g][0] = m == -INFINITY ? -INFINITY : m - kKv8PShift;
            s_ml[warp][g][1] = l;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int row = 2 * t + e;
            if (row < p.rows) {
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    *reinterpret_cast<float4*>(&s_o[warp][row][16 * g + 4 * w]) =
                        make_float4(o[2 * w][e] * vref, o[2 * w][2 + e] * vref, o[2 * w + 1][e] * vref,
                                    o[2 * w + 1][2 + e] * vref);
            }
        }
        __syncthreads();
        const bool whole = tile0 == 0 && tile1 == tiles;
        const int64_t slot = 2 * (int64_t)blockIdx.x + (u == u0 ? 0 : 1);
        for (int i = tid; i < p.rows * kDh; i += kKv8Threads) {
            const int row = i >> 7, d = i & (kDh - 1);
            float M = -INFINITY, A = 0.f, L = 0.f;
#pragma unroll
            for (int w = 0; w < kKv8Warps; ++w) M = fmaxf(M, s_ml[w][row][0]);
#pragma unroll
            for (int w = 0; w < kKv8Warps; ++w) {
                const float mw = s_ml[w][row][0];
                const float f = mw == -INFINITY ? 0.f : kv8_ex2(mw - M);
                A = fmaf(f, s_o[w][row][d], A);
                L = fmaf(f, s_ml[w][row][1], L);
            }
            if (whole) {
                p.out[(int64_t)(qrow0 + row) * kDh + d] = M == -INFINITY ? 0.f : A / L;
                if (d == 0 && p.lse != nullptr)
                    p.lse[qrow0 + row] = M == -INFINITY ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
            } else {
                p.part_o[(slot * kKv8MaxRows + row) * kDh + d] = A;
                if (d == 0) {
                    p.part_ml[(slot * kKv8MaxRows + row) * 2] = M;
                    p.part_ml[(slot * kKv8MaxRows + row) * 2 + 1] = L;
                }
            }
        }
        __syncthreads();  // the shared partials are free for the next run
        u += tile1 - tile0;
    }
}

// Join of the runs that span CTAs. grid (G, rows, 4): CTA c takes the run that begins in range c and
// reaches past it (there is at most one), one of its rows, and 32 of the Dh columns. Warp k takes the
// spanned CTAs k, k + 8, ...; a lane owns a column.
constexpr int kKv8MergeThreads = 256;
constexpr int kKv8MergeWarps = kKv8MergeThreads / 32;
constexpr int kKv8MergeU = 8;  // partials in flight per lane

__device__ __forceinline__ int kv8_cta_of(int64_t u, int64_t F, int G) { return (int)(((u + 1) * G + F - 1) / F - 1); }

__global__ void __launch_bounds__(kKv8MergeThreads)
k_kv8_attn_merge(const Kv8AttnParams p, const Kv8Tab tab) {
    __shared__ float s_m[kKv8MergeWarps], s_l[kKv8MergeWarps], s_a[kKv8MergeWarps][32];
    const int c = blockIdx.x, row = blockIdx.y, lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
    const int runs_b = p.g.Hkv * p.rts;
    const int64_t u0 = (int64_t)c * p.F / p.G, u1 = ((int64_t)c + 1) * p.F / p.G;
    pdl_wait();
    if (u1 == u0) return;
    int lo = 0, hi = tab.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((int64_t)tab.tile_off[mid] * runs_b <= u1 - 1) lo = mid; else hi = mid - 1;
    }
    const int b = lo, tiles = tab.tile_off[b + 1] - tab.tile_off[b];
    const int64_t base = (int64_t)tab.tile_off[b] * runs_b;
    const int run = (int)((u1 - 1 - base) / tiles);
    const int64_t r0 = base + (int64_t)run * tiles, r1 = r0 + tiles;  // the run's units
    if (r0 < u0 || r1 <= u1) return;
    const int ns = kv8_cta_of(r1 - 1, p.F, p.G) - c + 1;
    const int d = blockIdx.z * 32 + lane;

    float m = -INFINITY, l = 0.f, a = 0.f;
    for (int i0 = wp; i0 < ns; i0 += kKv8MergeWarps * kKv8MergeU) {
        float v[kKv8MergeU], mu[kKv8MergeU], lu[kKv8MergeU];
#pragma unroll
        for (int k = 0; k < kKv8MergeU; ++k) {  // past the last: reload it with no weight
            const int i = i0 + k * kKv8MergeWarps, ic = i < ns ? i : ns - 1;
            const int64_t slot = 2 * (int64_t)(c + ic) + (ic == 0 && r0 > u0 ? 1 : 0);
            v[k] = p.part_o[(slot * kKv8MaxRows + row) * kDh + d];
            const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + (slot * kKv8MaxRows + row) * 2);
            mu[k] = i < ns ? ml.x : -INFINITY;
            lu[k] = ml.y;
        }
        float mc = m;
#pragma unroll
        for (int k = 0; k < kKv8MergeU; ++k) mc = fmaxf(mc, mu[k]);
        if (mc == -INFINITY) continue;
        const float f = m == -INFINITY ? 0.f : kv8_ex2(m - mc);
        l *= f;
        a *= f;
#pragma unroll
        for (int k = 0; k < kKv8MergeU; ++k) {
            const float w = mu[k] == -INFINITY ? 0.f : kv8_ex2(mu[k] - mc);
            if (w > 0.f) {
                l = fmaf(w, lu[k], l);
                a = fmaf(w, v[k], a);
            }
        }
        m = mc;
    }
    if (lane == 0) {
        s_m[wp] = m;
        s_l[wp] = l;
    }
    s_a[wp][lane] = a;
    __syncthreads();
    if (wp != 0) return;
    float M = -INFINITY, A = 0.f, L = 0.f;
#pragma unroll
    for (int k = 0; k < kKv8MergeWarps; ++k) M = fmaxf(M, s_m[k]);
#pragma unroll
    for (int k = 0; k < kKv8MergeWarps; ++k) {
        const float w = s_m[k] == -INFINITY ? 0.f : kv8_ex2(s_m[k] - M);
        A = fmaf(w, s_a[k][lane], A);
        L = fmaf(w, s_l[k], L);
    }
    const int h = run / p.rts, rt = run - h * p.rts;
    const int q = b * p.H + (h * p.rts + rt) * p.rows + row;
    p.out[(int64_t)q * kDh + d] = M == -INFINITY ? 0.f : A / L;
    if (d == 0 && p.lse != nullptr) p.lse[q] = M == -INFINITY ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
}

// ------------------------------------------------------------------ host side
cudaError_t kv8_init_attrs(int num_sms, int* ctas) {
    int occ = 0;  // the least of the variants': one split serves them all
    const void* kernels[4] = {(const void*)k_kv8_attn<false, false>, (const void*)k_kv8_attn<false, true>,
                              (const void*)k_kv8_attn<true, false>, (const void*)k_kv8_attn<true, true>};
    for (const void* k : kernels) {
        int n = 0;
        cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kKv8Smem);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout,
                                     (int)cudaSharedmemCarveoutMaxShared);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, k, kKv8Threads, kKv8Smem);
        if (e != cudaSuccess) return e;
        if (occ == 0 || n < occ) occ = n;
    }
    *ctas = (occ < 1 ? 1 : occ) * num_sms;
    return cudaSuccess;
}

size_t kv8_part_o_bytes(int ctas) { return (size_t)2 * ctas * kKv8MaxRows * kDh * 4; }
size_t kv8_part_ml_bytes(int ctas) { return (size_t)2 * ctas * kKv8MaxRows * 2 * 4; }

// Whether some run spans two CTAs of the even split.
static bool kv8_splits(const Kv8Tab& tab, int runs_b, int64_t F, int G) {
    int b = 0;
    for (int c = 1; c < G; ++c) {
        const int64_t u = (int64_t)c * F / G;
        while (u >= (int64_t)tab.tile_off[b + 1] * runs_b) ++b;
        if ((u - (int64_t)tab.tile_off[b] * runs_b) % (tab.tile_off[b + 1] - tab.tile_off[b]) != 0) return true;
    }
    return false;
}

// `tab`: the kept chunks of each sequence, or all of them where ids is null.
cudaError_t launch_kv8_attn(const lsa_dims& d, const SeqTable& tab, const lsa_kv8_cache& cache, const Kv8Geom& g,
                            int max_ctas, const void* q, const int32_t* ids, const int32_t* counts,
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
    p.len_add = len_add;
    p.qscale = 1.4426950408889634f / sqrtf((float)kDh);

    Kv8Tab kt;
    kt.B = tab.B;
    int64_t tiles = 0;
    for (int b = 0; b <= tab.B; ++b) {
        kt.chunk_off[b] = tab.chunk_off[b];
        kt.kept_off[b] = tab.kept_off[b];
        kt.tile_off[b] = (int32_t)tiles;
        if (b < tab.B)
            tiles += (((int64_t)(tab.kept_off[b + 1] - tab.kept_off[b]) << g.c_log2) + kKv8Tile - 1) / kKv8Tile;
    }
    const int runs_b = g.Hkv * p.rts;
    const int64_t runs = (int64_t)runs_b * tab.B;
    p.F = tiles * runs_b;
    // Few tiles: at least four to a warp, one CTA to a run if that is enough, so that nothing is left
    // to join; many: every resident CTA an equal share.
    int64_t G = (p.F + 4 * kKv8Warps - 1) / (4 * kKv8Warps);
    if (G < runs) G = runs;
    if (G > max_ctas) G = max_ctas;
    if (G > p.F) G = p.F;
    p.G = (int)G;

    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    cfg.gridDim = dim3(p.G, 1, 1);
    cfg.blockDim = dim3(kKv8Threads, 1, 1);
    cfg.dynamicSmemBytes = kKv8Smem;
    const bool qlo = d.kv_dtype != LSA_BF16, plo = p.rows > 4;
    cudaError_t e = qlo ? (plo ? cudaLaunchKernelEx(&cfg, k_kv8_attn<true, true>, p, kt, err)
                               : cudaLaunchKernelEx(&cfg, k_kv8_attn<true, false>, p, kt, err))
                        : (plo ? cudaLaunchKernelEx(&cfg, k_kv8_attn<false, true>, p, kt, err)
                               : cudaLaunchKernelEx(&cfg, k_kv8_attn<false, false>, p, kt, err));
    if (e != cudaSuccess || !kv8_splits(kt, runs_b, p.F, p.G)) return e;
    cfg.numAttrs = 1;  // the merge always follows the split kernel: overlap its launch
    cfg.gridDim = dim3(p.G, p.rows, 4);
    cfg.blockDim = dim3(kKv8MergeThreads, 1, 1);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, k_kv8_attn_merge, p, kt);
}

// Whether the tokens of one head are few enough to be counted in 32 bits.
bool kv8_attn_fits(const SeqTable& tab, int c_log2) {
    return ((int64_t)tab.kept_off[tab.B] << c_log2) + (int64_t)tab.B * kKv8Tile < (1ll << 31);
}

}  // namespace lsa
