// kv8_gather.cu - chunks of the 8-bit K/V cache read back into resident buffers of the 16- or 32-bit
// layout: x = code * scale in fp32 (exact for a power-of-two scale, and then exact in bf16 too), rounded
// to bf16 where that is the layout's type.
//
// Pure streaming: 1 byte read and 2 or 4 written a value. Eight lanes convert a row of 128 codes, 16
// bytes to a lane; consecutive rows of a CTA are the heads of one token, so that its stores are one
// contiguous run of the output and its loads whole 128-byte rows.
//
// Measured (B200, in a graph): 256 of 2048 chunks x 8 sequences, 16 heads, to bf16, 1.61 GB: 241 us, 6.7 TB/s (a
// plain copy moves 6.47); 8 chunks of 8 heads to fp32, 5.2 MB: 3.3 us, a launch.
#include "kv8.cuh"

namespace lsa {

constexpr int kKv8GatherThreads = 256;
constexpr int kKv8GatherUnroll = 4;
constexpr int kKv8GatherRows = kKv8GatherThreads / 8 * kKv8GatherUnroll;  // rows per CTA

struct Kv8GatherParams {
    Kv8Geom g;
    const uint8_t *K8, *V8;
    const float *k_scale, *v_scale;
    uint8_t *K_res, *V_res;
    const int32_t *ids, *seq_len;  // nullable
    int32_t pieces;                // CTAs per chunk
    int32_t wide;                  // K_res and V_res are 32-byte aligned
};

// 32 bytes to global memory: one store where the buffers are 32-byte aligned, else two of 16.
__device__ __forceinline__ void st_32(void* p, const uint32_t* w, bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        static_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        static_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// grid (chunks * pieces, 2): blockIdx.y selects K (0) or V (1). `tab` has the chunks that are read as
// its kept chunks (all of them where ids is null).
template <bool BF16>
__global__ void __launch_bounds__(kKv8GatherThreads)
k_kv8_gather(const Kv8GatherParams gp, const SeqTable tab, uint32_t* err) {
    const int64_t j = blockIdx.x / gp.pieces;
    const int piece = blockIdx.x % gp.pieces;
    const int b = seq_of(tab.kept_off, tab.B, j);
    const int n_b = tab.chunk_off[b + 1] - tab.chunk_off[b];
    const int id = gp.ids != nullptr ? gp.ids[j] : (int)(j - tab.kept_off[b]);
    if (id < 0 || id >= n_b) {
        if (threadIdx.x == 0) set_error(err, kErrBadId);
        return;
    }
    const int C = 1 << gp.g.c_log2;
    int64_t left = ((int64_t)n_b - id) << gp.g.c_log2;
    if (gp.seq_len != nullptr) left = min(left, gp.seq_len[b] - ((int64_t)id << gp.g.c_log2));
    const int valid = (int)(left < 0 ? 0 : left > C ? C : left);  // tokens of the chunk that exist
    const uint8_t* codes = blockIdx.y ? gp.V8 : gp.K8;
    const float* scales = blockIdx.y ? gp.v_scale : gp.k_scale;
    uint8_t* res = blockIdx.y ? gp.V_res : gp.K_res;
    const int64_t ch0 = (int64_t)(tab.chunk_off[b] + id) * gp.g.Hkv;
    const int sub = threadIdx.x & 7;
    const int row0 = piece * kKv8GatherRows + (threadIdx.x >> 3);
    const int rows = valid * gp.g.Hkv;

    uint4 w[kKv8GatherUnroll];
    float sc[kKv8GatherUnroll];
#pragma unroll
    for (int u = 0; u < kKv8GatherUnroll; ++u) {
        const int row = row0 + u * (kKv8GatherThreads / 8);
        if (row < rows) {
            const int t = row >> gp.g.h_log2, h = row & (gp.g.Hkv - 1);
            w[u] = ld_stream16(codes + (((ch0 + h) << gp.g.c_log2) + t) * kDh + sub * 16);
            sc[u] = __ldg(scales + (ch0 + h) * gp.g.spc + (t >> gp.g.sb_log2));
        }
    }
#pragma unroll
    for (int u = 0; u < kKv8GatherUnroll; ++u) {
        const int row = row0 + u * (kKv8GatherThreads / 8);
        if (row < rows) {
            const uint32_t* cw = &w[u].x;
            float x[16];
#pragma unroll
            for (int i = 0; i < 4; ++i) e4m3x4_floats(cw[i], x + 4 * i);
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] *= sc[u];
            uint8_t* dst = res + (((j << gp.g.c_log2) * gp.g.Hkv + row) * 8 + sub) * (BF16 ? 32 : 64);
            uint32_t o[BF16 ? 8 : 16];
            if constexpr (BF16) {
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = bf16x2_rn(x[2 * e], x[2 * e + 1]);
                st_32(dst, o, gp.wide);
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(x[e]);
                st_32(dst, o, gp.wide);
                st_32(dst + 32, o + 8, gp.wide);
            }
        }
    }
}

cudaError_t launch_kv8_gather(const lsa_dims& d, const SeqTable& tab, const lsa_kv8_cache& cache, const Kv8Geom& g,
                              const int32_t* ids, const int32_t* seq_len, void* K_res, void* V_res, uint32_t* err,
                              cudaStream_t stream) {
    Kv8GatherParams gp = {};
    gp.g = g;
    gp.K8 = (const uint8_t*)cache.K8;
    gp.V8 = (const uint8_t*)cache.V8;
    gp.k_scale = cache.k_scale;
    gp.v_scale = cache.v_scale;
    gp.K_res = (uint8_t*)K_res;
    gp.V_res = (uint8_t*)V_res;
    gp.ids = ids;
    gp.seq_len = seq_len;
    gp.wide = ((reinterpret_cast<uintptr_t>(K_res) | reinterpret_cast<uintptr_t>(V_res)) & 31u) == 0;
    gp.pieces = (d.chunk_len * g.Hkv + kKv8GatherRows - 1) / kKv8GatherRows;
    const int64_t ctas = (int64_t)tab.kept_off[d.B] * gp.pieces;
    if (ctas > 0x7fffffffll) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cfg.gridDim = dim3((unsigned)ctas, 2, 1);
    cfg.blockDim = dim3(kKv8GatherThreads, 1, 1);
    return d.kv_dtype == LSA_BF16 ? cudaLaunchKernelEx(&cfg, k_kv8_gather<true>, gp, tab, err)
                                  : cudaLaunchKernelEx(&cfg, k_kv8_gather<false>, gp, tab, err);
}

}  // namespace lsa
