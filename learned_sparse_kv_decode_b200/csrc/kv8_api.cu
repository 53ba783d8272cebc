// kv8_api.cu - the C ABI of the 8-bit K/V cache (include/lsa_kv8.h): host-side validation and launches.
#include <cmath>
#include <cstring>

#include "kv8.cuh"
#include "lsa_host.cuh"

namespace lsa {
cudaError_t launch_score(const lsa_dims& d, const SeqTable& tab, int max_n, const void* q_emb,
                         const void* chunk_emb, float* scores, uint32_t* err, int num_sms,
                         cudaStream_t stream, bool pdl);
cudaError_t launch_topk_live(const lsa_dims& d, const SeqTable& tab, int max_n, const float* scores,
                             const int32_t* seq_len, int len_add, int32_t* ids, uint32_t* err, cudaStream_t stream,
                             bool pdl);
cudaError_t launch_qk_norm_rope(const lsa_dims& d, int n_kv_heads, const lsa_qk_prep& prep, int64_t n_tok,
                                const int32_t* positions, const void* q, int64_t q_stride, const void* k,
                                int64_t k_stride, void* q_out, int64_t qo_stride, void* k_out, int64_t ko_stride,
                                int num_sms, cudaStream_t stream, bool pdl);
cudaError_t launch_kv8_append(const lsa_dims& d, const SeqTable& tab, const lsa_kv8_cache& cache, const Kv8Geom& g,
                              const lsa_qk_prep* prep, int n_new, const void* k, int64_t k_stride, const void* v,
                              int64_t v_stride, const int32_t* start, const int32_t* new_count, uint32_t* err,
                              int num_sms, cudaStream_t stream, bool pdl);
cudaError_t launch_kv8_gather(const lsa_dims& d, const SeqTable& tab, const lsa_kv8_cache& cache, const Kv8Geom& g,
                              const int32_t* ids, const int32_t* seq_len, void* K_res, void* V_res, uint32_t* err,
                              cudaStream_t stream);
bool kv8_attn_fits(const SeqTable& tab, const Kv8Geom& g);
size_t kv8_part_o_bytes(int num_sms);
size_t kv8_part_ml_bytes(int num_sms);
cudaError_t launch_kv8_attn(const lsa_dims& d, const SeqTable& tab, const lsa_kv8_cache& cache, const Kv8Geom& g,
                            int num_sms, const void* q, const int32_t* ids, const int32_t* counts,
                            const int32_t* seq_len, int len_add, float* part_o, float* part_ml, float* out,
                            float* lse, uint32_t* err, cudaStream_t stream, bool pdl);
}  // namespace lsa

using namespace lsa;

namespace {

int log2_of(int x) {
    int n = 0;
    while ((1 << n) < x) ++n;
    return n;
}

// Shape of the cache (its pointers are checked by the calls that use them).
lsa_status cache_geom(const lsa_dims* d, const lsa_kv8_cache* c, Kv8Geom* g) {
    if (c == nullptr) return LSA_ERR_INVALID_ARG;
    if (!is_pow2(c->n_kv_heads) || c->n_kv_heads > d->H) return LSA_ERR_UNSUPPORTED;  // powers of two: it divides H
    if (!is_pow2(c->scale_block) || c->scale_block < 8 || c->scale_block > 64) return LSA_ERR_UNSUPPORTED;
    if (c->scale_block > d->chunk_len) return LSA_ERR_UNSUPPORTED;
    g->Hkv = c->n_kv_heads;
    g->h_log2 = log2_of(c->n_kv_heads);
    g->sb_log2 = log2_of(c->scale_block);
    g->c_log2 = log2_of(d->chunk_len);
    g->spc = d->chunk_len / c->scale_block;
    return LSA_OK;
}

struct Kv8Ws {
    WsLayout base;
    size_t part_o, part_ml, q, total;
};

// The workspace of lsa.h's calls, then: split partials | prepared queries of the step.
Kv8Ws kv8_layout(const lsa_dims* d, const Prepared& p, const DeviceInfo& di) {
    Kv8Ws w;
    w.base = ws_layout(d, p, di);
    w.part_o = w.base.total;
    w.part_ml = align256(w.part_o + kv8_part_o_bytes(di.sms));
    w.q = align256(w.part_ml + kv8_part_ml_bytes(di.sms));
    w.total = align256(w.q + (size_t)d->B * d->H * LSA_HEAD_DIM * (d->kv_dtype == LSA_BF16 ? 2 : 4));
    return w;
}

struct Kv8Call {
    Prepared p;
    DeviceInfo di;
    Kv8Geom g;
    Kv8Ws w;
};

// Shape and pointers that every call on a cache takes; no CUDA call.
lsa_status kv8_check(const lsa_dims* d, const lsa_kv8_cache* c, void* ws, Kv8Call* k) {
    lsa_status s = prepare(d, &k->p);
    if (s != LSA_OK) return s;
    s = cache_geom(d, c, &k->g);
    if (s != LSA_OK) return s;
    if (!aligned16(c->K8) || !aligned16(c->V8)) return LSA_ERR_INVALID_ARG;
    if (c->k_scale == nullptr || c->v_scale == nullptr || !aligned4(c->k_scale) || !aligned4(c->v_scale))
        return LSA_ERR_INVALID_ARG;
    return aligned16(ws) ? LSA_OK : LSA_ERR_INVALID_ARG;
}

// The device's facts and the workspace, once the arguments are known to be good.
lsa_status kv8_device(const lsa_dims* d, size_t ws_bytes, Kv8Call* k) {
    const lsa_status s = device_info(&k->di);
    if (s != LSA_OK) return s;
    if (!k->di.kv8) return LSA_ERR_CUDA;
    k->w = kv8_layout(d, k->p, k->di);
    if (ws_bytes < k->w.total) return LSA_ERR_WORKSPACE;
    return LSA_OK;
}

lsa_status prep_check(const lsa_qk_prep* p) {
    if (p == nullptr) return LSA_ERR_INVALID_ARG;
    if (p->rot_dim < 0 || p->rot_dim > LSA_HEAD_DIM) return LSA_ERR_INVALID_ARG;
    if (p->rot_dim % 16 != 0) return LSA_ERR_UNSUPPORTED;
    if (p->interleaved != 0 && p->interleaved != 1) return LSA_ERR_INVALID_ARG;
    if (!std::isfinite(p->eps) || p->eps < 0.f) return LSA_ERR_INVALID_ARG;
    if (p->rot_dim > 0 && p->inv_freq == nullptr) return LSA_ERR_INVALID_ARG;
    if (!aligned4(p->inv_freq)) return LSA_ERR_INVALID_ARG;
    if (p->q_weight != nullptr && !aligned16(p->q_weight)) return LSA_ERR_INVALID_ARG;
    if (p->k_weight != nullptr && !aligned16(p->k_weight)) return LSA_ERR_INVALID_ARG;
    return LSA_OK;
}

// Distance between rows of `heads` heads: a row at least, a multiple of 16 bytes, within 64-bit bytes.
bool stride_ok(const lsa_dims* d, int heads, int64_t stride) {
    const int per16 = d->kv_dtype == LSA_BF16 ? 8 : 4;
    return stride >= (int64_t)heads * LSA_HEAD_DIM && stride % per16 == 0 && stride < (1ll << 40);
}

// The kept chunks of the call: all of them where there are no ids.
void keep_all(SeqTable* t) { std::memcpy(t->kept_off, t->chunk_off, sizeof(t->kept_off)); }

}  // namespace

extern "C" {

lsa_status lsa_kv8_workspace_size(const lsa_dims* dims, const lsa_kv8_cache* cache, size_t* bytes) {
    if (bytes == nullptr) return LSA_ERR_INVALID_ARG;
    Prepared p;
    lsa_status s = prepare(dims, &p);
    if (s != LSA_OK) return s;
    Kv8Geom g;
    s = cache_geom(dims, cache, &g);
    if (s != LSA_OK) return s;
    DeviceInfo di;
    s = device_info(&di);
    if (s != LSA_OK) return s;
    *bytes = kv8_layout(dims, p, di).total;
    return LSA_OK;
}

lsa_status lsa_qk_norm_rope(const lsa_dims* dims, int32_t n_kv_heads, const lsa_qk_prep* prep, int64_t n_tok,
                            const int32_t* positions, const void* q, int64_t q_stride, const void* k,
                            int64_t k_stride, void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                            void* stream) {
    Prepared p;
    lsa_status s = prepare(dims, &p);
    if (s != LSA_OK) return s;
    s = prep_check(prep);
    if (s != LSA_OK) return s;
    if (n_tok < 0 || n_tok > (1ll << 31)) return LSA_ERR_INVALID_ARG;
    if (!is_pow2(n_kv_heads) || n_kv_heads > dims->H) return LSA_ERR_UNSUPPORTED;
    if (n_tok == 0) return LSA_OK;
    if ((q == nullptr) != (q_out == nullptr) || (k == nullptr) != (k_out == nullptr)) return LSA_ERR_INVALID_ARG;
    if (q == nullptr && k == nullptr) return LSA_ERR_INVALID_ARG;
    if (positions == nullptr || !aligned4(positions)) return LSA_ERR_INVALID_ARG;
    if (q != nullptr && (!aligned16(q) || !aligned16(q_out) || !stride_ok(dims, dims->H, q_stride) ||
                         !stride_ok(dims, dims->H, q_out_stride) || (q == q_out && q_stride != q_out_stride)))
        return LSA_ERR_INVALID_ARG;
    if (k != nullptr && (!aligned16(k) || !aligned16(k_out) || !stride_ok(dims, n_kv_heads, k_stride) ||
                         !stride_ok(dims, n_kv_heads, k_out_stride) || (k == k_out && k_stride != k_out_stride)))
        return LSA_ERR_INVALID_ARG;
    DeviceInfo di;
    s = device_info(&di);
    if (s != LSA_OK) return s;
    if (!di.kv8) return LSA_ERR_CUDA;
    return cuda_status(launch_qk_norm_rope(*dims, n_kv_heads, *prep, n_tok, positions, q, q_stride, k, k_stride,
                                           q_out, q_out_stride, k_out, k_out_stride, di.sms,
                                           static_cast<cudaStream_t>(stream), false));
}

lsa_status lsa_kv8_append(const lsa_dims* dims, const lsa_kv8_cache* cache, const lsa_qk_prep* prep, int32_t n_new,
                          const void* k, int64_t k_stride, const void* v, int64_t v_stride, const int32_t* start,
                          const int32_t* new_count, void* ws, size_t ws_bytes, void* stream) {
    Kv8Call c;
    lsa_status s = kv8_check(dims, cache, ws, &c);
    if (s != LSA_OK) return s;
    if (prep != nullptr) {
        s = prep_check(prep);
        if (s != LSA_OK) return s;
    }
    if (n_new < 1) return LSA_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v) || !stride_ok(dims, c.g.Hkv, k_stride) || !stride_ok(dims, c.g.Hkv, v_stride))
        return LSA_ERR_INVALID_ARG;
    if (!aligned4(start) || !aligned4(new_count)) return LSA_ERR_INVALID_ARG;
    s = kv8_device(dims, ws_bytes, &c);
    if (s != LSA_OK) return s;
    return cuda_status(launch_kv8_append(*dims, c.p.tab, *cache, c.g, prep, n_new, k, k_stride, v, v_stride, start,
                                         new_count, reinterpret_cast<uint32_t*>(ws), c.di.sms,
                                         static_cast<cudaStream_t>(stream), false));
}

lsa_status lsa_kv8_gather(const lsa_dims* dims, const lsa_kv8_cache* cache, const int32_t* chunk_ids,
                          const int32_t* seq_len, void* K_res, void* V_res, void* ws, size_t ws_bytes,
                          void* stream) {
    Kv8Call c;
    lsa_status s = kv8_check(dims, cache, ws, &c);
    if (s != LSA_OK) return s;
    if (!aligned16(K_res) || !aligned16(V_res) || !aligned4(chunk_ids) || !aligned4(seq_len))
        return LSA_ERR_INVALID_ARG;
    if (chunk_ids == nullptr) keep_all(&c.p.tab);
    s = kv8_device(dims, ws_bytes, &c);
    if (s != LSA_OK) return s;
    return cuda_status(launch_kv8_gather(*dims, c.p.tab, *cache, c.g, chunk_ids, seq_len, K_res, V_res,
                                         reinterpret_cast<uint32_t*>(ws), static_cast<cudaStream_t>(stream)));
}

lsa_status lsa_kv8_decode_attn(const lsa_dims* dims, const lsa_kv8_cache* cache, const void* q,
                               const int32_t* chunk_ids, const int32_t* kept_count, const int32_t* seq_len,
                               float* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
    Kv8Call c;
    lsa_status s = kv8_check(dims, cache, ws, &c);
    if (s != LSA_OK) return s;
    if (!aligned16(q) || !aligned16(out) || !aligned4(chunk_ids) || !aligned4(kept_count) || !aligned4(seq_len) ||
        !aligned4(lse))
        return LSA_ERR_INVALID_ARG;
    if (chunk_ids == nullptr) keep_all(&c.p.tab);
    if (!kv8_attn_fits(c.p.tab, c.g)) return LSA_ERR_UNSUPPORTED;
    s = kv8_device(dims, ws_bytes, &c);
    if (s != LSA_OK) return s;
    return cuda_status(launch_kv8_attn(*dims, c.p.tab, *cache, c.g, c.di.sms, q, chunk_ids, kept_count, seq_len,
                                       0, reinterpret_cast<float*>(at(ws, c.w.part_o)),
                                       reinterpret_cast<float*>(at(ws, c.w.part_ml)), out, lse,
                                       reinterpret_cast<uint32_t*>(ws), static_cast<cudaStream_t>(stream), false));
}

lsa_status lsa_decode_step_kv8(const lsa_dims* dims, const lsa_kv8_cache* cache, const lsa_qk_prep* prep,
                               const void* q_emb, const void* chunk_emb, const void* q, int64_t q_stride,
                               const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                               const int32_t* seq_len, int32_t* chunk_ids_out, float* out, float* lse, void* ws,
                               size_t ws_bytes, void* stream) {
    Kv8Call c;
    lsa_status s = kv8_check(dims, cache, ws, &c);
    if (s != LSA_OK) return s;
    if (prep != nullptr) {
        s = prep_check(prep);
        if (s != LSA_OK) return s;
    }
    if ((k == nullptr) != (v == nullptr)) return LSA_ERR_INVALID_ARG;
    if (seq_len == nullptr && (k != nullptr || prep != nullptr)) return LSA_ERR_INVALID_ARG;
    if (!aligned16(q_emb) || !aligned16(chunk_emb) || !aligned16(q) || !aligned16(chunk_ids_out) || !aligned16(out) ||
        !aligned4(seq_len) || !aligned4(lse))
        return LSA_ERR_INVALID_ARG;
    if (!stride_ok(dims, dims->H, q_stride)) return LSA_ERR_INVALID_ARG;
    if (prep == nullptr && q_stride != (int64_t)dims->H * LSA_HEAD_DIM) return LSA_ERR_INVALID_ARG;
    if (k != nullptr && (!aligned16(k) || !aligned16(v) || !stride_ok(dims, c.g.Hkv, k_stride) ||
                         !stride_ok(dims, c.g.Hkv, v_stride)))
        return LSA_ERR_INVALID_ARG;
    if (!kv8_attn_fits(c.p.tab, c.g)) return LSA_ERR_UNSUPPORTED;
    s = kv8_device(dims, ws_bytes, &c);
    if (s != LSA_OK) return s;

    cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint32_t* err = reinterpret_cast<uint32_t*>(ws);
    float* scores = reinterpret_cast<float*>(at(ws, c.w.base.scores));
    cudaError_t e = launch_score(*dims, c.p.tab, c.p.max_n, q_emb, chunk_emb, scores, err, c.di.sms, st, false);
    const int len_add = k != nullptr ? 1 : 0;  // the new token counts
    if (e == cudaSuccess)
        e = launch_topk_live(*dims, c.p.tab, c.p.max_n, scores, seq_len, len_add, chunk_ids_out, err, st, true);
    // The write and the queries depend on neither: launched early, they run beside the top-k. Each waits
    // for the kernel before it at its end, so that the attention still follows all of them.
    if (e == cudaSuccess && k != nullptr)
        e = launch_kv8_append(*dims, c.p.tab, *cache, c.g, prep, 1, k, k_stride, v, v_stride, seq_len, nullptr, err,
                              c.di.sms, st, true);
    const void* qr = q;
    if (e == cudaSuccess && prep != nullptr) {
        void* qw = at(ws, c.w.q);
        e = launch_qk_norm_rope(*dims, c.g.Hkv, *prep, dims->B, seq_len, q, q_stride, nullptr, 0, qw,
                                (int64_t)dims->H * LSA_HEAD_DIM, nullptr, 0, c.di.sms, st, true);
        qr = qw;
    }
    if (e == cudaSuccess)
        e = launch_kv8_attn(*dims, c.p.tab, *cache, c.g, c.di.sms, qr, chunk_ids_out, nullptr, seq_len,
                            len_add, reinterpret_cast<float*>(at(ws, c.w.part_o)),
                            reinterpret_cast<float*>(at(ws, c.w.part_ml)), out, lse, err, st, true);
    return cuda_status(e);
}

}  // extern "C"
