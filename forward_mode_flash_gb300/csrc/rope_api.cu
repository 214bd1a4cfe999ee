// rope_api.cu -- entry points of the norms and rotation of queries and keys:
// on dense tensors, and on their way into a paged cache.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "serve_checks.h"

namespace jvp {
namespace {

jvp_status_t check_rope(const jvp_rope_t* r, int64_t D, RopeParams* p) {
  if (!r) return api_fail(JVP_ERR_INVALID_ARG, "rope is NULL");
  if (D <= 0) return api_fail(JVP_ERR_INVALID_ARG, "D must be positive");
  if (D > 128) return api_fail(JVP_ERR_UNSUPPORTED, "D > 128 is not supported");
  if (r->dim < 0 || r->dim > D || r->dim % 2 != 0)
    return api_fail(JVP_ERR_INVALID_ARG, "the rotated columns must be an even number of at most D");
  if (r->rows < 0) return api_fail(JVP_ERR_INVALID_ARG, "negative number of table rows");
  if (r->rows > kMax) return api_fail(JVP_ERR_UNSUPPORTED, "the table has more than 2^31 - 1 rows");
  if (r->interleaved != 0 && r->interleaved != 1)
    return api_fail(JVP_ERR_INVALID_ARG, "interleaved must be 0 or 1");
  if (r->dim > 0 && r->rows > 0 && !r->table)
    return api_fail(JVP_ERR_INVALID_ARG, "the table of angles is NULL");
  if (!aligned_to(r->table, 4))
    return api_fail(JVP_ERR_ALIGNMENT, "the table of angles is not 4-byte aligned");
  if (!r->q_weight != !r->k_weight)
    return api_fail(JVP_ERR_INVALID_ARG, "q_weight and k_weight go together");
  if (r->dim == 0 && !r->q_weight)
    return api_fail(JVP_ERR_INVALID_ARG, "neither angles nor norm weights are given");
  if (r->q_weight) {
    if (!tensor_type(r->weight_dtype))
      return api_fail(JVP_ERR_INVALID_ARG, "unknown dtype of the norm weights");
    if (!aligned_to(r->q_weight, elem_bytes(r->weight_dtype)) ||
        !aligned_to(r->k_weight, elem_bytes(r->weight_dtype)))
      return api_fail(JVP_ERR_ALIGNMENT, "norm weights not aligned to their element size");
    if (!std::isfinite(r->eps) || r->eps < 0.f)
      return api_fail(JVP_ERR_INVALID_ARG, "eps must be finite and not negative");
  }
  *p = RopeParams{};
  p->D = static_cast<int>(D), p->rot = static_cast<int>(r->dim);
  p->interleaved = r->interleaved;
  p->table_rows = static_cast<int>(r->rows), p->table = r->table;
  p->wq = r->q_weight, p->wk = r->k_weight, p->weight_type = r->weight_dtype;
  p->eps = r->eps, p->inv_d = 1.f / static_cast<float>(D);
  return JVP_OK;
}

// Rows of whole 16-byte pieces whose rotated pairs lie in a lane's two pieces
// (or, neighbours, in one).
bool pieces(const RopeParams& p, int64_t elem) {
  const int n = static_cast<int>(16 / elem);
  return p.D % n == 0 && p.rot % (p.interleaved ? n : 2 * n) == 0 && aligned_to(p.table, 8);
}

// Blocks that leave sums of the weights' gradients, at most.
size_t sums_bytes(int64_t D, int num_sms) {
  return static_cast<size_t>(num_sms) * rope_blocks_per_sm() * 2 * static_cast<size_t>(D) * 4;
}

jvp_status_t norm_rope(bool bwd, const jvp_shape_t* shape, jvp_dtype_t dtype, const jvp_rope_t* rope,
                       const int32_t* positions, int64_t positions_stride, const void* const (&x)[8],
                       const jvp_strides_t* in, void* const (&y)[4], const jvp_strides_t* out,
                       float* gwq, float* gwk, void* workspace, size_t workspace_bytes,
                       void* stream) {
  api_set_path(0);
  if (!shape) return api_fail(JVP_ERR_INVALID_ARG, "shape is NULL");
  const int64_t B = shape->B, H = shape->H, N = shape->Nq, D = shape->D, Hkv = shape->Hkv;
  if (B < 0 || H < 0 || N < 0 || Hkv < 0) return api_fail(JVP_ERR_INVALID_ARG, "negative size");
  if (shape->Nk != N) return api_fail(JVP_ERR_INVALID_ARG, "Nk must equal Nq");
  if (!tensor_type(dtype)) return api_fail(JVP_ERR_INVALID_ARG, "unknown dtype");
  RopeDense d{};
  jvp_status_t st = check_rope(rope, D, &d.r);
  if (st != JVP_OK) return st;
  if (!in || !out) return api_fail(JVP_ERR_INVALID_ARG, "strides are NULL");
  if (B > kMax || H > kMax || N > kMax || Hkv > kMax || (N > 0 && B > kMax / N) ||
      (B * N > 0 && H + Hkv > kMax / (B * N)))
    return api_fail(JVP_ERR_UNSUPPORTED, "problem too large for one launch");
  const bool norm = d.r.wq != nullptr;
  const bool tangents = x[2] || x[3] || (bwd && !norm && (x[6] || x[7]));
  const int sides[4] = {0, 1, 2, 3};
  // (without norms the gradients do not depend on the rows)
  const int first = bwd && !norm ? 4 : 0, inputs = bwd ? 8 : 4;
  for (int i = first; i < inputs; ++i) {
    if ((i & 2) && !tangents) continue;
    st = check_strides(in[i], "innermost (d) stride must be 1", "negative stride");
    if (st != JVP_OK) return st;
  }
  for (int i : sides) {
    if ((i & 2) && !tangents) continue;
    st = check_strides(out[i], "innermost (d) stride must be 1", "negative stride");
    if (st != JVP_OK) return st;
    const int64_t heads = (i & 1) ? Hkv : H;
    if ((B > 1 && out[i].b == 0) || (heads > 1 && out[i].h == 0) || (N > 1 && out[i].n == 0))
      return api_fail(JVP_ERR_INVALID_ARG, "an output must not have a stride of 0");
  }
  if (positions && positions_stride < 0)
    return api_fail(JVP_ERR_INVALID_ARG, "negative stride of positions");
  if (!positions && d.r.rot > 0 && N > d.r.table_rows)
    return api_fail(JVP_ERR_INVALID_ARG, "the table of angles has fewer rows than there are tokens");
  if (!aligned_to(positions, 4))
    return api_fail(JVP_ERR_ALIGNMENT, "positions not 4-byte aligned");
  // (without tokens or heads the weights' gradients are still written: zeros)
  const bool empty = B * N == 0 || H + Hkv == 0;
  if (empty && !(bwd && norm)) return api_ok();
  const int64_t e = elem_bytes(dtype);
  bool vec = pieces(d.r, e);
  if (!empty) {
    for (int i = first; i < inputs; ++i) {
      const int64_t heads = (i & 1) ? Hkv : H;
      if (((i & 2) && !tangents) || heads == 0) continue;
      if (!x[i]) return api_fail(JVP_ERR_INVALID_ARG, "an input is NULL");
      if (!aligned_to(x[i], e))
        return api_fail(JVP_ERR_ALIGNMENT, "an input is not aligned to its element size");
      d.x[i] = x[i], d.in[i] = used(in[i], B, heads, N);
      vec = vec && aligned_to(x[i], 16) && multiple(d.in[i], 16 / e);
    }
    for (int i : sides) {
      const int64_t heads = (i & 1) ? Hkv : H;
      if (((i & 2) && !tangents) || heads == 0) continue;
      if (!y[i]) return api_fail(JVP_ERR_INVALID_ARG, "an output is NULL");
      if (!aligned_to(y[i], e))
        return api_fail(JVP_ERR_ALIGNMENT, "an output is not aligned to its element size");
      d.y[i] = y[i], d.out[i] = used(out[i], B, heads, N);
      vec = vec && aligned_to(y[i], 16) && multiple(d.out[i], 16 / e);
    }
  }
  if (bwd && norm) {
    if (!gwq || !gwk)
      return api_fail(JVP_ERR_INVALID_ARG, "an output of the weights' gradients is NULL");
    if (!aligned_to(gwq, 4) || !aligned_to(gwk, 4) || !aligned_to(workspace, 4))
      return api_fail(JVP_ERR_ALIGNMENT, "weights' gradients or workspace not 4-byte aligned");
  }
  int sms = 0;
  st = api_device(&sms, &d.r.status);
  if (st != JVP_OK) return st;
  if (bwd && norm && (!workspace || workspace_bytes < sums_bytes(D, sms)))
    return api_fail(JVP_ERR_WORKSPACE,
                    "workspace is NULL or smaller than jvp_attn_norm_rope_bwd_workspace_size()");
  d.tokens = B * N, d.N = static_cast<int>(N);
  d.H = static_cast<int>(H), d.Hkv = static_cast<int>(Hkv);
  d.positions = positions, d.positions_stride = B > 1 ? positions_stride : 0;
  d.ws = static_cast<float*>(workspace), d.gwq = gwq, d.gwk = gwk;
  if (bwd && !norm) {  // the rotation of the cotangents the other way
    d.back = 1;
    for (int i : sides) d.x[i] = d.x[4 + i], d.in[i] = d.in[4 + i];
  }
  const cudaError_t err = launch_norm_rope(static_cast<DType>(dtype), vec, bwd, d, sms,
                                           static_cast<cudaStream_t>(stream));
  if (err != cudaSuccess) return api_cuda_fail(err);
  api_set_path(2);
  return api_ok();
}

}  // namespace
}  // namespace jvp

extern "C" {

jvp_status_t jvp_attn_norm_rope(const jvp_shape_t* shape, jvp_dtype_t dtype, const jvp_rope_t* rope,
                                const int32_t* positions, int64_t positions_stride, const void* q,
                                const void* k, const void* dq, const void* dk,
                                const jvp_strides_t* in_strides, void* q_out, void* k_out,
                                void* dq_out, void* dk_out, const jvp_strides_t* out_strides,
                                void* stream) {
  return jvp::norm_rope(false, shape, dtype, rope, positions, positions_stride,
                        {q, k, dq, dk, nullptr, nullptr, nullptr, nullptr}, in_strides,
                        {q_out, k_out, dq_out, dk_out}, out_strides, nullptr, nullptr, nullptr, 0,
                        stream);
}

jvp_status_t jvp_attn_norm_rope_bwd(const jvp_shape_t* shape, jvp_dtype_t dtype,
                                    const jvp_rope_t* rope, const int32_t* positions,
                                    int64_t positions_stride, const void* q, const void* k,
                                    const void* dq, const void* dk, const void* g_q,
                                    const void* g_k, const void* g_dq, const void* g_dk,
                                    const jvp_strides_t* in_strides, void* gq_out, void* gk_out,
                                    void* gdq_out, void* gdk_out, const jvp_strides_t* out_strides,
                                    float* g_q_weight, float* g_k_weight, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  return jvp::norm_rope(true, shape, dtype, rope, positions, positions_stride,
                        {q, k, dq, dk, g_q, g_k, g_dq, g_dk}, in_strides,
                        {gq_out, gk_out, gdq_out, gdk_out}, out_strides, g_q_weight, g_k_weight,
                        workspace, workspace_bytes, stream);
}

size_t jvp_attn_norm_rope_bwd_workspace_size(int64_t D) {
  int sms = 0;
  unsigned int* status = nullptr;
  if (D <= 0 || D > 128 || jvp::api_device(&sms, &status) != JVP_OK) return 0;
  return jvp::sums_bytes(D, sms);
}

jvp_status_t jvp_attn_cache_append(const jvp_cache_t* cache, int64_t H, jvp_dtype_t dtype, int64_t T,
                                   const void* q, const void* k, const void* v,
                                   const jvp_strides_t* in_strides, const jvp_rope_t* rope,
                                   const int32_t* block_table, const int32_t* start_pos,
                                   const int32_t* cu_seqlens, void* q_out,
                                   const jvp_strides_t* q_out_strides, void* k_cache, void* v_cache,
                                   uint8_t* k_scale, uint8_t* v_scale, void* stream) {
  using namespace jvp;
  api_set_path(0);
  jvp_status_t st = check_cache(cache, true);
  if (st != JVP_OK) return st;
  if (!tensor_type(dtype)) return api_fail(JVP_ERR_INVALID_ARG, "unknown dtype");
  if (cache->dtype != JVP_E4M3 && cache->dtype != dtype)
    return api_fail(JVP_ERR_INVALID_ARG, "the rows must have the cache's dtype (or the cache e4m3)");
  if (T < 0 || H < 0) return api_fail(JVP_ERR_INVALID_ARG, "negative T or H");
  AppendParams a{};
  st = check_rope(rope, cache->D, &a.r);
  if (st != JVP_OK) return st;
  const int64_t Hkv = cache->Hkv;
  if (T > kMax || H > kMax || Hkv > kMax / 4 || H + 2 * Hkv > kMax / (T > 0 ? T : 1))
    return api_fail(JVP_ERR_UNSUPPORTED, "problem too large for one launch");
  if (!cu_seqlens && T != cache->B)
    return api_fail(JVP_ERR_INVALID_ARG, "without cu_seqlens there must be one row per sequence");
  if (!in_strides || !q_out_strides) return api_fail(JVP_ERR_INVALID_ARG, "strides are NULL");
  for (int i = 0; i < 4; ++i) {
    st = check_strides(i < 3 ? in_strides[i] : *q_out_strides, "innermost (d) stride must be 1",
                       "negative stride");
    if (st != JVP_OK) return st;
  }
  if ((T > 1 && q_out_strides->n == 0) || (H > 1 && q_out_strides->h == 0))
    return api_fail(JVP_ERR_INVALID_ARG, "an output must not have a stride of 0");
  if (T == 0 || cache->B == 0 || H + Hkv == 0) return api_ok();
  if ((H > 0 && (!q || !q_out)) || (Hkv > 0 && (!k || !v)))
    return api_fail(JVP_ERR_INVALID_ARG, "q, k, v or q_out is NULL");
  const int64_t e = elem_bytes(dtype), ce = elem_bytes(cache->dtype);
  if (!aligned_to(q, e) || !aligned_to(k, e) || !aligned_to(v, e) || !aligned_to(q_out, e))
    return api_fail(JVP_ERR_ALIGNMENT, "q, k, v or q_out not aligned to its element size");
  if (!aligned_to(start_pos, 4) || !aligned_to(cu_seqlens, 4))
    return api_fail(JVP_ERR_ALIGNMENT, "start_pos or cu_seqlens not 4-byte aligned");
  st = check_cache_ptrs(cache, k_cache, v_cache, k_scale, v_scale, block_table);
  if (st != JVP_OK) return st;
  int sms = 0;
  st = api_device(&sms, &a.r.status);
  if (st != JVP_OK) return st;
  a.c = describe(cache, k_cache, v_cache, k_scale, v_scale, block_table, a.r.status);
  a.T = T, a.H = static_cast<int>(H);
  a.cu = cu_seqlens, a.start = start_pos;
  a.x[0] = q, a.x[1] = k, a.x[2] = v, a.q_out = q_out;
  for (int i = 0; i < 3; ++i) a.in[i] = used(in_strides[i], 0, i ? Hkv : H, T);
  a.sq_out = used(*q_out_strides, 0, H, T);
  const int64_t n = 16 / e;
  bool vec = pieces(a.r, e) && aligned_to(q, 16) && aligned_to(k, 16) && aligned_to(v, 16) &&
             aligned_to(q_out, 16) && multiple(a.sq_out, n) && aligned_to(k_cache, n * ce) &&
             aligned_to(v_cache, n * ce) && multiple(a.c.sk, n) && multiple(a.c.sv, n);
  for (int i = 0; i < 3; ++i) vec = vec && multiple(a.in[i], n);
  const cudaError_t err = launch_cache_append(static_cast<DType>(dtype), cache->dtype == JVP_E4M3,
                                              vec, a, sms, static_cast<cudaStream_t>(stream));
  if (err != cudaSuccess) return api_cuda_fail(err);
  api_set_path(2);
  return api_ok();
}

}  // extern "C"
