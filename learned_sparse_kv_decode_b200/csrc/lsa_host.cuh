// lsa_host.cuh - host-side helpers that the C entry points share: per-device facts, validation of the
// shape, the workspace layout (defined in lsa_api.cu).
#pragma once

#include "lsa_device.cuh"

namespace lsa {

struct DeviceInfo {
    bool ready;
    int sms;
    int attn_ctas[2];  // per kv dtype (LSA_F32, LSA_BF16)
    int la_ctas;       // CTAs of the lookahead-window attention
    bool kv8;          // the 8-bit cache's kernels can run as planned
};

// Facts of the current device, computed once per device.
lsa_status device_info(DeviceInfo* out);

struct Prepared {
    SeqTable tab;
    int max_n;
    int64_t total_chunks;
    int64_t total_kept;
};

// Validate the shape and build the per-sequence table.
lsa_status prepare(const lsa_dims* d, Prepared* p);

struct WsLayout {
    size_t scores, part_o, part_ml, ids, copy_src, copy_dst, copy_count, la_o, la_ml, small, total;
};

WsLayout ws_layout(const lsa_dims* d, const Prepared& p, const DeviceInfo& di);

inline bool is_pow2(int64_t x) { return x > 0 && (x & (x - 1)) == 0; }
inline bool aligned16(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }  // or null
inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
inline uint8_t* at(void* ws, size_t off) { return static_cast<uint8_t*>(ws) + off; }
inline lsa_status cuda_status(cudaError_t e) { return e == cudaSuccess ? LSA_OK : LSA_ERR_CUDA; }

}  // namespace lsa
