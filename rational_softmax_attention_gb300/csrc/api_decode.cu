// The C ABI of the position and serving operators (declared in include/raattn.h): argument
// validation and dispatch.  Nothing here allocates device memory.
#include <climits>
#include <cmath>

#include "kernels.cuh"

namespace raattn {
namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool dtype_ok(ra_dtype_t t) { return t == RA_F32 || t == RA_BF16; }
bool head_dim_ok(int D) { return D == 16 || D == 32 || D == 64 || D == 128; }

// Sizes whose row counts fit 32 bits; elements are addressed in 64.
bool rows_ok(int64_t a, int64_t b, int64_t c) { return a * b <= INT_MAX && a * b * c <= INT_MAX; }

// Loops over a cache's slots step by up to 8192 in 32 bits.
constexpr int kMostKeys = INT_MAX - 16384;

// Offsets within a token are formed in 32 bits, up to 256 heads of 128 past its last one.
constexpr int kMostTokenElements = INT_MAX - 256 * 128;

ra_status_t norm_rope_shape(NormRopeShape* a, const void* qkv, int64_t batch_stride, int64_t token_stride,
                            const void* qw, const void* qb, const void* kw, const void* kb, ra_norm_t norm, float eps,
                            const double* freq, const int32_t* pos, int64_t pos_axis_stride, int64_t pos_batch_stride,
                            const int32_t* sections, int axes, int interleaved, int B, int N, int Hq, int Hkv, int D,
                            ra_dtype_t dtype) {
  if (!qkv || !aligned(qkv, 16) || !dtype_ok(dtype)) return RA_ERR_ARG;
  if (B < 1 || N < 1 || Hq < 1 || Hkv < 1 || D < 1 || axes < 0 || (axes > 0 && !sections)) return RA_ERR_ARG;
  if (Hq > INT_MAX / 4 || Hkv > INT_MAX / 4 || !rows_ok(B, N, Hq + 2 * Hkv)) return RA_ERR_ARG;
  if (static_cast<int64_t>(Hq + 2 * Hkv) * D > kMostTokenElements) return RA_ERR_ARG;
  if (norm != RA_NORM_NONE && norm != RA_NORM_LAYER && norm != RA_NORM_RMS) return RA_ERR_ARG;
  if (norm == RA_NORM_NONE ? (qw || qb || kw || kb) : (!qw || !kw)) return RA_ERR_ARG;
  if (norm == RA_NORM_RMS && (qb || kb)) return RA_ERR_ARG;
  if (norm != RA_NORM_NONE && !(eps >= 0.0f && std::isfinite(eps))) return RA_ERR_ARG;
  for (const void* p : {qw, qb, kw, kb})
    if (!aligned(p, 16)) return RA_ERR_ARG;
  const int vec = dtype == RA_BF16 ? 8 : 4;
  if (batch_stride % vec || token_stride % vec) return RA_ERR_ARG;
  int64_t pairs = 0;
  a->end[0] = a->end[1] = a->end[2] = INT_MAX;
  for (int i = 0; i < axes; ++i) {
    if (sections[i] < 1) return RA_ERR_ARG;
    pairs += sections[i];
    if (i < 3) a->end[i] = static_cast<int>(pairs < INT_MAX ? pairs : INT_MAX);
  }
  if (2 * pairs > D) return RA_ERR_ARG;
  if (axes > 0 && (!freq || !pos || !aligned(freq, 8) || !aligned(pos, 4))) return RA_ERR_ARG;
  if (axes > 4 || !head_dim_ok(D) || (!interleaved && pairs % 8)) return RA_ERR_UNSUPPORTED;
  a->qkv = qkv;
  a->batch_stride = batch_stride;
  a->token_stride = token_stride;
  a->qw = qw;
  a->qb = qb;
  a->kw = kw;
  a->kb = kb;
  a->freq = freq;
  a->pos = pos;
  a->pos_axis_stride = pos_axis_stride;
  a->pos_batch_stride = pos_batch_stride;
  a->pairs = static_cast<int>(pairs);
  a->interleaved = interleaved ? 1 : 0;
  a->B = B;
  a->N = N;
  a->Hq = Hq;
  a->Hkv = Hkv;
  a->D = D;
  a->norm = norm;
  a->eps = eps;
  return RA_OK;
}

ra_status_t decode_shape(DecodeArgs* a, int B, int Hq, int Hkv, int C, int P, int D) {
  if (B < 1 || Hq < 1 || Hkv < 1 || C < 1 || P < 0 || D < 1 || Hq % Hkv) return RA_ERR_ARG;
  if (!rows_ok(B, Hq, 1) || C > kMostKeys || P > kMostKeys) return RA_ERR_ARG;
  if (!rows_ok(B, Hkv, C) || !rows_ok(Hkv, P, 1)) return RA_ERR_ARG;
  if (!head_dim_ok(D) || B > kDecodeMaxBatch || Hq / Hkv > 1024) return RA_ERR_UNSUPPORTED;
  a->B = B;
  a->Hq = Hq;
  a->Hkv = Hkv;
  a->C = C;
  a->P = P;
  a->D = D;
  return RA_OK;
}

}  // namespace
}  // namespace raattn

using namespace raattn;

extern "C" {

ra_status_t ra_qk_norm_rope_fwd(const void* qkv, int64_t batch_stride, int64_t token_stride, const void* q_weight,
                                const void* q_bias, const void* k_weight, const void* k_bias, ra_norm_t norm,
                                float eps, const double* frequencies, const int32_t* positions,
                                int64_t pos_axis_stride, int64_t pos_batch_stride, const int32_t* sections, int axes,
                                int interleaved, void* q, void* k, void* v, const int32_t* start,
                                const int32_t* count, int capacity, int B, int N, int H_Q, int H_KV, int D,
                                ra_dtype_t dtype, void* stream) {
  NormRopeShape a;
  const ra_status_t s = norm_rope_shape(&a, qkv, batch_stride, token_stride, q_weight, q_bias, k_weight, k_bias, norm,
                                        eps, frequencies, positions, pos_axis_stride, pos_batch_stride, sections,
                                        axes, interleaved, B, N, H_Q, H_KV, D, dtype);
  if (s == RA_ERR_ARG) return s;
  if (!q || !k || !v || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16)) return RA_ERR_ARG;
  if (!aligned(start, 4) || !aligned(count, 4) || (!start && count)) return RA_ERR_ARG;
  if (start ? capacity < 1 || !rows_ok(B, H_KV, capacity) : capacity != 0) return RA_ERR_ARG;
  if (s != RA_OK) return s;
  const NormRopeFwd io{q, k, v, start, count, start ? capacity : N};
  return launch_norm_rope_fwd(a, io, dtype == RA_BF16, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? RA_OK
             : RA_ERR_LAUNCH;
}

size_t ra_qk_norm_rope_bwd_workspace_size(int D) {
  return head_dim_ok(D) ? static_cast<size_t>(norm_rope_bwd_ctas()) * 2 * D * sizeof(float) : 0;
}

ra_status_t ra_qk_norm_rope_bwd(const void* qkv, int64_t batch_stride, int64_t token_stride, const void* q_weight,
                                const void* q_bias, const void* k_weight, const void* k_bias, ra_norm_t norm,
                                float eps, const double* frequencies, const int32_t* positions,
                                int64_t pos_axis_stride, int64_t pos_batch_stride, const int32_t* sections, int axes,
                                int interleaved, const void* dq, const void* dk, const void* dv, void* dqkv,
                                float* dparams, void* workspace, int B, int N, int H_Q, int H_KV, int D,
                                ra_dtype_t dtype, void* stream) {
  NormRopeShape a;
  const ra_status_t s = norm_rope_shape(&a, qkv, batch_stride, token_stride, q_weight, q_bias, k_weight, k_bias, norm,
                                        eps, frequencies, positions, pos_axis_stride, pos_batch_stride, sections,
                                        axes, interleaved, B, N, H_Q, H_KV, D, dtype);
  if (s == RA_ERR_ARG) return s;
  if (!dq || !dk || !dv || !dqkv) return RA_ERR_ARG;
  for (const void* p : {dq, dk, dv, static_cast<const void*>(dqkv), static_cast<const void*>(dparams),
                        static_cast<const void*>(workspace)})
    if (!aligned(p, 16)) return RA_ERR_ARG;
  if (norm != RA_NORM_NONE && (!dparams || !workspace)) return RA_ERR_ARG;
  if (s != RA_OK) return s;
  const NormRopeBwd io{dq, dk, dv, dqkv, dparams, static_cast<float*>(workspace)};
  return launch_norm_rope_bwd(a, io, dtype == RA_BF16, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? RA_OK
             : RA_ERR_LAUNCH;
}

size_t ra_attention_decode_workspace_size(int B, int H_Q, int H_KV, int C, int P, int D, ra_dtype_t dtype) {
  DecodeArgs a{};
  if (!dtype_ok(dtype) || decode_shape(&a, B, H_Q, H_KV, C, P, D) != RA_OK) return 0;
  return plan_decode(&a, dtype == RA_BF16, nullptr);
}

ra_status_t ra_attention_decode(const void* q, const void* k, const void* v, const int32_t* length,
                                const void* prefix_k, const void* prefix_v, void* o, float* weight, void* workspace,
                                int B, int H_Q, int H_KV, int C, int P, int D, float scale, ra_dtype_t dtype,
                                void* stream) {
  if (!q || !k || !v || !length || !o || !workspace || !dtype_ok(dtype)) return RA_ERR_ARG;
  DecodeArgs a{};
  const ra_status_t s = decode_shape(&a, B, H_Q, H_KV, C, P, D);
  if (s == RA_ERR_ARG) return s;
  if (P > 0 ? !prefix_k || !prefix_v : prefix_k || prefix_v) return RA_ERR_ARG;
  for (const void* p : {q, k, v, prefix_k, prefix_v, static_cast<const void*>(o), static_cast<const void*>(workspace)})
    if (!aligned(p, 16)) return RA_ERR_ARG;
  if (!aligned(length, 4) || !aligned(weight, 4)) return RA_ERR_ARG;
  if (!(scale > 0.0f)) scale = 1.0f / std::sqrt(static_cast<float>(D));
  if (!std::isfinite(scale)) return RA_ERR_ARG;
  if (s != RA_OK) return s;
  if (dtype == RA_BF16 && D < 64) return RA_ERR_UNSUPPORTED;
  a.q = q;
  a.k = k;
  a.v = v;
  a.pk = prefix_k;
  a.pv = prefix_v;
  a.length = length;
  a.weight = weight;
  a.o = o;
  a.scale = scale;
  if (plan_decode(&a, dtype == RA_BF16, static_cast<char*>(workspace)) == 0) return RA_ERR_UNSUPPORTED;
  PrefixMaps maps;
  LaunchCtx ctx;
  if (a.tc && (launch_context(&ctx) != RA_OK || !tensor_map_bf16(&maps.k, prefix_k, H_KV, P, D) ||
               !tensor_map_bf16(&maps.v, prefix_v, H_KV, P, D)))
    return RA_ERR_LAUNCH;
  return launch_decode(a, dtype == RA_BF16, maps, ctx, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? RA_OK
             : RA_ERR_LAUNCH;
}

ra_status_t ra_cache_evict(const void* k, const void* v, const float* weight, const int32_t* length, void* k_out,
                           void* v_out, float* weight_out, int32_t* length_out, int32_t* index, int B, int H_KV,
                           int C, int C_out, int D, int keep, int recent, ra_dtype_t dtype, void* stream) {
  if (!k || !v || !weight || !length || !k_out || !v_out || !weight_out || !length_out || !index || !dtype_ok(dtype))
    return RA_ERR_ARG;
  if (B < 1 || H_KV < 1 || C < 1 || C_out < 1 || D < 1 || keep < 1 || keep > C_out || recent < 0 || recent > keep)
    return RA_ERR_ARG;
  if (!rows_ok(B, H_KV, C) || !rows_ok(B, H_KV, C_out) || C > kMostKeys || C_out > kMostKeys || D > (1 << 20))
    return RA_ERR_ARG;
  for (const void* p : {k, v, static_cast<const void*>(k_out), static_cast<const void*>(v_out)})
    if (!aligned(p, 16)) return RA_ERR_ARG;
  for (const void* p : {static_cast<const void*>(weight), static_cast<const void*>(length),
                        static_cast<const void*>(weight_out), static_cast<const void*>(length_out),
                        static_cast<const void*>(index)})
    if (!aligned(p, 4)) return RA_ERR_ARG;
  if (k == k_out || k == v_out || v == k_out || v == v_out || k_out == v_out || weight == weight_out ||
      length == length_out)
    return RA_ERR_ARG;
  const int row_bytes = D * (dtype == RA_BF16 ? 2 : 4);
  if (row_bytes % 16) return RA_ERR_UNSUPPORTED;
  const EvictArgs a{k, v, weight, length, k_out, v_out, weight_out, length_out, index, B, H_KV, C, C_out, row_bytes,
                    keep, recent};
  return launch_evict(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? RA_OK : RA_ERR_LAUNCH;
}

}  // extern "C"
