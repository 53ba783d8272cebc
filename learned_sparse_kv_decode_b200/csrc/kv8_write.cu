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
// One warp per (token, slice of heads). The token's 64 angles are computed once per warp, two to a
// lane (the 64-bit reduction and sincospi cost as much as a dozen rows), and handed round by
// shuffles; the warp then walks its slice four heads at a time, eight lanes to a head, so that a
// warp's loads and stores are 1 KB runs (bf16) of the token's row.
constexpr int kPrepThreads = 256;

struct PrepRows {
    const uint8_t *q, *k;
    uint8_t *qo, *ko;
    int64_t q_stride, k_stride, qo_stride, ko_stride;  // bytes from one token to the next
    int32_t H, Hkv;        // 0 where q or k is absent
    int64_t n_tok;
    int32_t slices;        // warps per token
    int32_t units, per;    // four-head units per token, units per slice
};

template <bool BF16>
__global__ void __launch_bounds__(kPrepThreads)
k_qk_norm_rope(const PrepRows r, const PrepParams pp, const int32_t* __restrict__ positions) {
    constexpr int kRow = kDh * (BF16 ? 2 : 4);
    pdl_trigger();
    const int lane = threadIdx.x & 31, sub = lane & 7, grp = lane >> 3;
    const int64_t w = (int64_t)blockIdx.x * (kPrepThreads / 32) + (threadIdx.x >> 5);
    const int64_t tok = w / r.slices;
    if (tok < r.n_tok) {
        const int slice = (int)(w - tok * r.slices);
        float c[8], s[8];
        if (pp.ho > 0) {
            const int32_t pos = positions[tok];
            float c2[2] = {1.f, 1.f}, s2[2] = {0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (2 * lane + j < pp.ho * 8) angle_cs(pos, pp.inv_freq[2 * lane + j], &c2[j], &s2[j]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                c[e] = __shfl_sync(0xffffffffu, c2[e & 1], sub * 4 + (e >> 1));
                s[e] = __shfl_sync(0xffffffffu, s2[e & 1], sub * 4 + (e >> 1));
            }
        }
        int oa, ob;
        row_octets(sub, pp.ho, pp.interleaved, &oa, &ob);
        const int qu = (r.H + 3) >> 2;  // units of queries come first
        float wa[8], wb[8];
        int have = -1;  // whose weights are loaded: 0 queries, 1 keys
        const int u1 = min(r.units, (slice + 1) * r.per);
        OctetRaw<BF16> ra, rb;
        auto load = [&](int u) {  // a unit ahead of its use, so that a warp has two in flight
            const int part = u >= qu, h = ((part ? u - qu : u) << 2) + grp;
            if (u < u1 && h < (part ? r.Hkv : r.H)) {
                const uint8_t* src = (part ? r.k + tok * r.k_stride : r.q + tok * r.q_stride) + (int64_t)h * kRow;
                ra = octet_load<BF16>(src, oa);
                rb = octet_load<BF16>(src, ob);
            }
        };
        ra = rb = OctetRaw<BF16>{};
        load(slice * r.per);
        for (int u = slice * r.per; u < u1; ++u) {
            const int part = u >= qu, h = ((part ? u - qu : u) << 2) + grp;
            const float* weight = part ? pp.k_weight : pp.q_weight;
            float x[8], y[8];
            octet_floats<BF16>(ra, x);
            octet_floats<BF16>(rb, y);
            load(u + 1);
            if (part != have && weight != nullptr) {
                load8(weight + oa * 8, wa);
                load8(weight + ob * 8, wb);
            }
            have = part;
            if (weight != nullptr) row_norm(x, y, wa, wb, pp.eps);
            if (sub < pp.ho) row_rotate(x, y, c, s, pp.interleaved);
            if (h < (part ? r.Hkv : r.H)) {
                uint8_t* dst = (part ? r.ko + tok * r.ko_stride : r.qo + tok * r.qo_stride) + (int64_t)h * kRow;
                octet_store<BF16>(dst, oa, x);
                octet_store<BF16>(dst, ob, y);
            }
        }
    }
    pdl_wait();  // launched early, nothing above depends on the kernel before; the one after does
}

// ---------------------------------------------------------------- quantising write
// One CTA per (64-token window of a sequence, slice of heads): window rows are aligned to 64 tokens of
// the sequence, eight lanes to a row, so that every block of 8..64 tokens lies inside one CTA and its
// amax is a shuffle inside the warp (four rows) and a look at scale_block / 4 warps' words.
constexpr int kAppendThreads = 512;
constexpr int kAppendRows = kAppendThreads / 8;
constexpr int kAppendCtas = 8;  // CTAs per SM that a long call is cut into

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
};

// A lane's codes of one row: eight bytes at each of its octets.
__device__ __forceinline__ void store_codes(uint8_t* row, int oa, int ob, const float* x, const float* y,
                                            float scale) {
    uint32_t c[4];
    const bool p2 = (__float_as_uint(scale) & 0x807FFFFFu) == 0;
    if (p2) {  // the usual case: multiplying by 1 / 2^e is the division, exactly
        const float inv = 1.f / scale;
        c[0] = e4m3x4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
        c[1] = e4m3x4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv);
        c[2] = e4m3x4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
        c[3] = e4m3x4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv);
    } else {  // a block that came with another scale
        c[0] = e4m3x4(x[0] / scale, x[1] / scale, x[2] / scale, x[3] / scale);
        c[1] = e4m3x4(x[4] / scale, x[5] / scale, x[6] / scale, x[7] / scale);
        c[2] = e4m3x4(y[0] / scale, y[1] / scale, y[2] / scale, y[3] / scale);
        c[3] = e4m3x4(y[4] / scale, y[5] / scale, y[6] / scale, y[7] / scale);
    }
    if (ob == oa + 1) {
        *reinterpret_cast<uint4*>(row + oa * 8) = make_uint4(c[0], c[1], c[2], c[3]);
    } else {
        *reinterpret_cast<uint2*>(row + oa * 8) = make_uint2(c[0], c[1]);
        *reinterpret_cast<uint2*>(row + ob * 8) = make_uint2(c[2], c[3]);
    }
}

// Largest finite magnitude of a lane's 16 values; sets *bad if one is not finite.
__device__ __forceinline__ float amax16(const float* x, const float* y, bool* bad) {
    float a = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float p = fabsf(x[e]), q = fabsf(y[e]);
        const bool fp = p < INFINITY, fq = q < INFINITY;
        *bad |= !(fp && fq);
        a = fmaxf(a, fmaxf(fp ? p : 0.f, fq ? q : 0.f));
    }
    return a;
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

// Registers are what keeps loads in flight here: a bf16 row's values stay packed until they are written, a
// head's rows are loaded while the one before it is worked on, and the angles (PREP; computed once for the
// slice's heads) wait in shared memory, where each lane keeps its own.
template <bool BF16, bool PREP>
__global__ void __launch_bounds__(kAppendThreads, BF16 ? 2 : 1)
k_kv8_append(const AppendParams ap, const PrepParams pp, const SeqTable tab, uint32_t* err) {
    constexpr int kRow = kDh * (BF16 ? 2 : 4);
    __shared__ float s_amax[2][2][kAppendRows / 4];  // [head parity][K, V][warp]
    __shared__ float4 s_angle[PREP ? 4 : 1][PREP ? kAppendThreads : 1];  // cosines 0-3, 4-7, sines 0-3, 4-7
    pdl_trigger();
    const int tid = threadIdx.x, sub = tid & 7, r = tid >> 3, warp = tid >> 5;
    const int slice = blockIdx.x % ap.slices;
    const int win = (blockIdx.x / ap.slices) % ap.windows;
    const int b = blockIdx.x / ap.slices / ap.windows;

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
        const bool touched = lo < hi;             // uniform in a warp: its four rows share a block
        const bool fresh = pos >= start && pos < end;
        const bool older = touched && pos < start;
        const bool has_old = touched && blk0 < start;
        const int64_t row_in = (int64_t)b * ap.n_new + (pos - start);
        const int h0 = slice * ap.per, h1 = min(ap.g.Hkv, h0 + ap.per);
        // this row's place in the cache, of head h0: element offset and scale index (a head on: + C rows, + spc)
        const int64_t ch0 = (tab.chunk_off[b] + (pos >> ap.g.c_log2)) * ap.g.Hkv + h0;
        const int within = (int)(pos & ((1 << ap.g.c_log2) - 1));
        const bool writer = touched && r % (1 << ap.g.sb_log2) == 0 && sub == 0;

        int oa, ob;
        row_octets(sub, PREP ? pp.ho : 0, PREP ? pp.interleaved : 0, &oa, &ob);
        const uint8_t* kr = ap.k + row_in * ap.k_stride + (int64_t)h0 * kRow;
        const uint8_t* vr = ap.v + row_in * ap.v_stride + (int64_t)h0 * kRow;
        OctetRaw<BF16> nka{}, nkb{}, nva{}, nvb{};
        auto load = [&]() {
            if (fresh) {
                nka = octet_load<BF16>(kr, oa);
                nkb = octet_load<BF16>(kr, ob);
                nva = octet_load<BF16>(vr, 2 * sub);
                nvb = octet_load<BF16>(vr, 2 * sub + 1);
            }
            kr += kRow;
            vr += kRow;
        };
        load();
        if constexpr (PREP) {
            if (fresh && sub < pp.ho) {
                float c[8], s[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) angle_cs((int32_t)pos, pp.inv_freq[sub * 8 + e], &c[e], &s[e]);
                s_angle[0][tid] = make_float4(c[0], c[1], c[2], c[3]);
                s_angle[1][tid] = make_float4(c[4], c[5], c[6], c[7]);
                s_angle[2][tid] = make_float4(s[0], s[1], s[2], s[3]);
                s_angle[3][tid] = make_float4(s[4], s[5], s[6], s[7]);
            }
        }
        for (int h = h0; h < h1; ++h) {
            OctetRaw<BF16> ka = nka, kb = nkb;
            const OctetRaw<BF16> va = nva, vb = nvb;
            if (h + 1 < h1) load();
            // the block's scales so far (read before the barrier, written after it)
            const int64_t ch = ch0 + (h - h0);
            const int64_t si = ch * ap.g.spc + (within >> ap.g.sb_log2);
            float was_k = 0.f, was_v = 0.f;
            if (has_old) {
                was_k = ap.k_scale[si];
                was_v = ap.v_scale[si];
            }
            bool bad = false;
            float ak, av;
            {
                float x[8], y[8];
                octet_floats<BF16>(ka, x);
                octet_floats<BF16>(kb, y);
                if constexpr (PREP) {
                    if (pp.k_weight != nullptr) {
                        float wa[8], wb[8];
                        load8(pp.k_weight + oa * 8, wa);
                        load8(pp.k_weight + ob * 8, wb);
                        row_norm(x, y, wa, wb, pp.eps);
                    }
                    if (fresh && sub < pp.ho) {
                        const float4 c0 = s_angle[0][tid], c1 = s_angle[1][tid], s0 = s_angle[2][tid], s1 = s_angle[3][tid];
                        const float c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
                        const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
                        row_rotate(x, y, c, s, pp.interleaved);
                    }
                    // what lsa_qk_norm_rope would have stored
                    ka = octet_pack<BF16>(x);
                    kb = octet_pack<BF16>(y);
                    octet_floats<BF16>(ka, x);
                    octet_floats<BF16>(kb, y);
                }
                ak = amax16(x, y, &bad);
                octet_floats<BF16>(va, x);
                octet_floats<BF16>(vb, y);
                av = amax16(x, y, &bad);
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                ak = fmaxf(ak, __shfl_xor_sync(0xffffffffu, ak, o));
                av = fmaxf(av, __shfl_xor_sync(0xffffffffu, av, o));
            }
            if (bad) set_error(err, kErrNonFinite);
            if ((tid & 31) == 0) {
                s_amax[h & 1][0][warp] = ak;
                s_amax[h & 1][1][warp] = av;
            }
            __syncthreads();  // the other parity's words are free again after the next one
            if (touched) {
                const int nw = 1 << (ap.g.sb_log2 - 2), wfirst = warp & ~(nw - 1);
                for (int i = 0; i < nw; ++i) {
                    ak = fmaxf(ak, s_amax[h & 1][0][wfirst + i]);
                    av = fmaxf(av, s_amax[h & 1][1][wfirst + i]);
                }
                const float sk = fmaxf(kv8_scale_of(ak), was_k), sv = fmaxf(kv8_scale_of(av), was_v);
                uint8_t* kd = ap.K8 + ((ch << ap.g.c_log2) + within) * kDh;
                uint8_t* vd = ap.V8 + ((ch << ap.g.c_log2) + within) * kDh;
                if (fresh) {
                    float x[8], y[8];
                    octet_floats<BF16>(ka, x);
                    octet_floats<BF16>(kb, y);
                    store_codes(kd, oa, ob, x, y, sk);
                    octet_floats<BF16>(va, x);
                    octet_floats<BF16>(vb, y);
                    store_codes(vd, 2 * sub, 2 * sub + 1, x, y, sv);
                } else if (older) {
                    if (sk > was_k) rescale_codes(kd, sub, was_k / sk);
                    if (sv > was_v) rescale_codes(vd, sub, was_v / sv);
                }
                if (writer) {
                    ap.k_scale[si] = sk;
                    ap.v_scale[si] = sv;
                }
            }
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
    r.units = (r.H + 3) / 4 + (r.Hkv + 3) / 4;
    // a warp per token where there are tokens enough to fill the SMs, else the heads are split
    const int64_t want = (int64_t)num_sms * 32;
    int64_t slices = n_tok >= want ? 1 : (want + n_tok - 1) / n_tok;
    if (slices > r.units) slices = r.units;
    r.per = (int)((r.units + slices - 1) / slices);
    r.slices = (r.units + r.per - 1) / r.per;
    const int64_t warps = n_tok * r.slices;
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
    return d.kv_dtype == LSA_BF16 ? cudaLaunchKernelEx(&cfg, k_qk_norm_rope<true>, r, pp, positions)
                                  : cudaLaunchKernelEx(&cfg, k_qk_norm_rope<false>, r, pp, positions);
}

// CTAs of an append, or 0 where they pass a grid's limit.
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
    // Long slices while there are CTAs enough: the angles are computed once for a slice's heads, and a head's
    // rows are loaded during the one before.
    const int64_t cells = (int64_t)ap.windows * d.B, want = (int64_t)num_sms * kAppendCtas;
    int64_t slices = cells >= want ? 1 : (want + cells - 1) / cells;
    if (slices > g.Hkv) slices = g.Hkv;
    ap.per = (int)((g.Hkv + slices - 1) / slices);
    ap.slices = (g.Hkv + ap.per - 1) / ap.per;
    const int64_t ctas = (int64_t)ap.windows * d.B * ap.slices;
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
    const bool bf = d.kv_dtype == LSA_BF16;
    if (prep != nullptr)
        return bf ? cudaLaunchKernelEx(&cfg, k_kv8_append<true, true>, ap, pp, tab, err)
                  : cudaLaunchKernelEx(&cfg, k_kv8_append<false, true>, ap, pp, tab, err);
    return bf ? cudaLaunchKernelEx(&cfg, k_kv8_append<true, false>, ap, pp, tab, err)
              : cudaLaunchKernelEx(&cfg, k_kv8_append<false, false>, ap, pp, tab, err);
}

}  // namespace lsa
