// Expert routing over all experts, and the gradient of the logits
// (segtopk_route and segtopk_route_backward in include/segtopk.h).
#include "route.cuh"

namespace segtopk {
namespace {

// The gradient of the logits, dense: with u_i the weight before the scale c
// and h_i = c g_i,
//   softmax, renormalised  d_i = u_i (h_i - sum_j u_j h_j)       else 0
//   softmax                d_e = s_e (h_e [e chosen] - sum_j s_j h_j)
//   sigmoid, renormalised  d_i = u_i (1 - s_i) (h_i - sum_j u_j h_j)  else 0
//   sigmoid                d_i = h_i s_i (1 - s_i)               else 0
// Only the plain softmax reads the whole row of logits. The row is put
// together in shared memory and written once.
template <class T, int NV, bool VECTOR, bool SIGMOID>
__global__ void __launch_bounds__(kWarps * 32)
route_backward_kernel(const float* grad, const T* logits, uint32_t tokens, int experts, int64_t stride, int k,
                      const int32_t* ids, bool renormalize, float scale, T* out)
{
  __shared__ Vec<float, NV> rows_sh[kWarps][32];
  wait_for_previous();
  allow_next();
  const int lane = threadIdx.x & 31;
  const uint32_t t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= tokens)
    return;
  float* d = reinterpret_cast<float*>(rows_sh[threadIdx.x >> 5]);
  const T* row = logits + (int64_t)t * stride;
  const int first = lane * NV;
  // all loads that wait for none
  float x[NV] = {};
  if (!SIGMOID && !renormalize)
    load_share<T, NV, VECTOR>(x, row, first, experts);
  const int id = lane < k ? ids[(int64_t)t * k + lane] : -1;
  const float weight_grad = lane < k ? grad[(int64_t)t * k + lane] : 0.0f;
  const bool on = id >= 0 && id < experts;
  const float l = on ? to_f32(row[id]) : 0.0f;
  const float g = on ? scale * weight_grad : 0.0f;
  float top = 0, sum = 1;
  if (!SIGMOID && !renormalize) {
    top = warp_max_nan(max_of(x));
#pragma unroll
    for (int i = 0; i < NV; ++i)
      x[i] = expf(x[i] - top); // each is a result's factor
    sum = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      sum += x[i];
    sum = warp_sum(sum);
  }
  const float u = chosen_weight<SIGMOID>(l, on, renormalize, top, sum);
  float dot = 0, part = u;
  if (renormalize || !SIGMOID)
    dot = warp_sum(on ? u * g : 0.0f);
  if (SIGMOID)
    part *= sigmoid(-l); // 1 - sigmoid(l)
  part *= renormalize ? g - dot : g;
  if (!SIGMOID && !renormalize) {
    // a token without choices gets zeros, whatever its logits are
    const bool any = __any_sync(kAll, on);
    const float c = -dot / sum;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      x[i] = any ? x[i] * c : 0.0f;
  }
  store_f32<float, NV>(d + first, x);
  __syncwarp();
  if (on)
    d[id] += part; // ids of a token are distinct
  __syncwarp();
  T* to = out + (int64_t)t * experts;
  if constexpr (VECTOR) {
    constexpr int V = NV * (int)sizeof(T) > 16 ? 16 / (int)sizeof(T) : NV;
#pragma unroll
    for (int e = 0; e < NV; e += V)
      if (first + e < experts) {
        const Vec<float, V> v = load<float, V>(d + first + e);
        float y[V];
#pragma unroll
        for (int i = 0; i < V; ++i)
          y[i] = v.f32(i);
        store_f32<T, V>(to + first + e, y);
      }
  } else {
    for (int e = lane; e < experts; e += 32)
      to[e] = from_f32<T>(d[e]);
  }
}

} // namespace
} // namespace segtopk

using namespace segtopk;

extern "C" int segtopk_route(segtopk_dtype dtype, const void* logits, int64_t tokens, int32_t experts,
                             int64_t row_stride, int32_t k, segtopk_score score, int renormalize, float scale,
                             const float* bias, int32_t* expert_ids, float* weights, void* stream)
{
  record_launch_count(0);
  return route<false>(dtype, logits, tokens, experts, row_stride, k, {}, score, renormalize, scale, bias, expert_ids,
                      weights, stream);
}

extern "C" int segtopk_route_backward(segtopk_dtype dtype, const float* grad_weights, const void* logits,
                                      int64_t tokens, int32_t experts, int64_t row_stride, int32_t k,
                                      const int32_t* expert_ids, segtopk_score score, int renormalize, float scale,
                                      void* grad_logits, void* stream)
{
  record_launch_count(0);
  int rc = check(dtype, logits, tokens, experts, row_stride, k, score, renormalize);
  if (rc != SEGTOPK_SUCCESS)
    return rc;
  if (tokens == 0)
    return SEGTOPK_SUCCESS;
  if (!grad_weights || !expert_ids || !grad_logits)
    return SEGTOPK_ERROR_INVALID_VALUE;
  if (!aligned(expert_ids, 4) || !aligned(grad_weights, 4) || !aligned(grad_logits, dtype == SEGTOPK_F32 ? 4 : 2))
    return SEGTOPK_ERROR_MISALIGNED;
  int sms;
  if ((rc = check_device(&sms)) != SEGTOPK_SUCCESS)
    return rc;
  return with_float_type(dtype, [&](auto zero) {
    using T = decltype(zero);
    const int n = std::min<int>(share_of(experts), 16 / (int)sizeof(T));
    const bool vector = rows_fit(logits, row_stride, experts, sizeof(T), n) &&
                        rows_fit(grad_logits, experts, experts, sizeof(T), n);
    return finish(with_share(experts, vector, [&](auto nv, auto vec) {
      constexpr int NV = decltype(nv)::value;
      constexpr bool V = decltype(vec)::value;
      auto kernel =
        score == SEGTOPK_SIGMOID ? route_backward_kernel<T, NV, V, true> : route_backward_kernel<T, NV, V, false>;
      return launch(kernel, dim3((unsigned)((tokens + kWarps - 1) / kWarps)), kWarps * 32, 0, (cudaStream_t)stream,
                    grad_weights, (const T*)logits, (uint32_t)tokens, experts, row_stride, k, expert_ids,
                    renormalize != 0, scale, (T*)grad_logits);
    }), 1);
  });
}
