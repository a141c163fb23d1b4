// Expert routing: the k best experts of each token from its router logits,
// their weights, and the logits' gradient (segtopk_route and
// segtopk_route_backward in include/segtopk.h).
//
// Scores of the logits l of one token: softmax s_e = exp(l_e - m) / sum, or
// sigmoid s_e = 1 / (1 + exp(-l_e)). Chosen: the k best by (s_e + b_e
// descending, e ascending); without a bias b the logits themselves are
// compared, which order alike and, unlike scores rounded to 32 bits, make no
// new ties. Weights: c s_i, or c s_i / (sum of the chosen scores).
//
// One warp serves a token: its lanes hold the row in registers (NV
// consecutive logits each), so the row is read once. 65536 rows of 256 in
// f32, k = 8, weights from the full softmax: 25.5 us, 10.5 at the copy rate;
// bound by issue (385 instructions a row, 83 % of the issue slots), which is
// why the k best are not searched for one after the other, see choose(). A
// warp that fetches its next row ahead, or blocks that stay, were slower (28
// to 30 us): the registers cost more warps than the loads cost time. The
// backward pass reads the row again and writes it: 24.5 us, 20.4 at the copy
// rate, bound by memory; in bf16 19.5, 10.4 at the copy rate.
#include "rows.cuh"

namespace segtopk {
namespace {
using namespace rows;

constexpr int kWarps = 8; // tokens of a block

// Order-preserving code of a score: larger is better; +-0 equal; any NaN
// above +inf; kNone and below for -inf and for places past the row's end,
// which are never chosen.
constexpr uint32_t kNone = 0x007fffffu; // code of -inf
__device__ __forceinline__ uint32_t code_of(float x)
{
  const uint32_t b = __float_as_uint(x + 0.0f); // -0 + 0 = +0
  const uint32_t c = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
  return isnan(x) ? 0xffffffffu : c;
}

__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    x += __shfl_xor_sync(kAll, x, o);
  return x;
}
// The largest of x and y, or of all lanes' x; NaN if any is.
__device__ __forceinline__ float max_nan(float x, float y)
{
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(x), "f"(y));
  return m;
}
__device__ __forceinline__ float warp_max_nan(float x)
{
  float m;
  asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
  return m;
}
template <int NV>
__device__ __forceinline__ float max_of(const float (&x)[NV])
{
  float m = x[0];
#pragma unroll
  for (int i = 1; i < NV; ++i)
    m = max_nan(m, x[i]);
  return m;
}

// 1 / (1 + e^-x), by the exponential that does not overflow, so that scores
// below the normal numbers stay apart: e^-90 is not 0, 1 / (1 + e^90) is.
__device__ __forceinline__ float sigmoid(float x)
{
  const float e = expf(-fabsf(x));
  return (x < 0 ? e : 1.0f) / (1.0f + e);
}

// NV consecutive logits of a lane, in 32 bits; -inf past the row's end.
template <class T, int NV, bool VECTOR>
__device__ __forceinline__ void load_share(float (&x)[NV], const T* row, int first, int experts)
{
  if constexpr (VECTOR) {
    constexpr int V = NV * (int)sizeof(T) > 16 ? 16 / (int)sizeof(T) : NV;
#pragma unroll
    for (int v = 0; v < NV; v += V) {
      if (first + v < experts) { // experts is a multiple of V
        const Vec<T, V> got = load<T, V>(row + first + v);
#pragma unroll
        for (int i = 0; i < V; ++i)
          x[v + i] = got.f32(i);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
          x[v + i] = -INFINITY;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      x[i] = first + i < experts ? to_f32(row[first + i]) : -INFINITY;
  }
}

// exp(d) for the terms of a softmax's sum: 2^(d log2 e) by the special
// function unit, d at most 0. A term is off by 2^-22 and |d| 2^-24 of its
// value (by as much again where d itself was rounded) and zero below 2^-126.
// The terms' mean |d|, weighted by themselves, is at most the entropy's ln E,
// so the sum, which is at least 1, is off by 2^-22 + 2.25 ln(E) 2^-24 of its
// value, beside its additions' roundings. expf would leave out 1.25 ln(E)
// 2^-24 of that and takes 27.6 us instead of 25.4 (65536 rows of 256 in f32,
// k = 8). For the sum only: where a single term is a result or decides, expf.
__device__ __forceinline__ float fast_exp(float d)
{
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(d * 1.44269504f));
  return y;
}

// The sum of exp(x_i - top) over the row. NaN or +inf among the logits give
// NaN, as the formula does; a row of -inf alone has no weights and its sum no
// use.
template <bool FAST, int NV>
__device__ __forceinline__ float softmax_sum(const float (&x)[NV], float top)
{
  float s = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    s += FAST ? fast_exp(x[i] - top) : expf(x[i] - top);
  return warp_sum(s);
}

// The weights of the chosen logits, one per lane (`on`: this lane has one),
// before the scale. Renormalised sigmoids are taken relative to the largest
// chosen one when all are small, s_i / s = e^(l_i - h) / (1 + e^(l_i)) with
// h = min(0, largest l), so that they neither vanish nor divide by zero.
template <bool SIGMOID>
__device__ __forceinline__ float chosen_weight(float l, bool on, bool renormalize, float top, float sum)
{
  if (!renormalize)
    return !on ? 0.0f : SIGMOID ? sigmoid(l) : expf(l - top) / sum;
  const float most = warp_max_nan(on ? l : -INFINITY);
  float s;
  if (SIGMOID)
    s = l > 0 ? 1.0f / (1.0f + expf(-l)) : expf(l - fminf(most, 0.0f)) / (1.0f + expf(l));
  else
    s = expf(l - most);
  s = on ? s : 0.0f;
  const float total = warp_sum(s);
  return on ? s / total : 0.0f;
}

// The k best keys of a row that are above -inf: lane j's result is the j-th
// one's expert, or -1. `largest` is the largest key of this lane, `top` that
// of all (NaN if any is); key_at(e) gives expert e's key again.
//
// The k-th best of the lanes' largest keys is a bound: k keys are at or above
// it, so nothing below it is chosen. About k + k^2 / 64 keys are not below
// it; their experts go to a list in shared memory, one a lane, and each lane
// counts the entries ahead of its own. The rounds (k times: find the best,
// take it out) are left for k above 16, where the list overflows, for rows
// that overflow it by ties at the bound or hold NaN, and for the shares
// where they are as fast. 65536 rows of 256, k = 8, on GB300: 50 us by rounds,
// 24 with the list; k = 2: 22 and 19; rows of 64, k = 6: 17.3 and 18.7.
constexpr int kListCap = 32;
struct Choice {
  uint64_t ranked[kListCap]; // code, and ~expert: larger is ahead, ties go to the lower expert
  int list[kListCap];
};
template <int NV, class F>
__device__ __forceinline__ int choose(const float (&key)[NV], float largest, float top, int k, Choice& sh, F&& key_at)
{
  const int lane = threadIdx.x & 31;
  const int first = lane * NV;
  if (k <= 16 && k * NV > 12 && top == top) {
    // lanes with equal largest keys leave together: the bound is then lower,
    // and only the list longer
    float bound = top;
    for (int j = 1; j < k; ++j) {
      largest = largest == bound ? -INFINITY : largest;
      bound = warp_max_nan(largest);
    }
    bound = fmaxf(bound, -3.402823466e38f);
    unsigned mine = 0; // places of this lane's keys at or above the bound
#pragma unroll
    for (int i = 0; i < NV; ++i)
      mine |= key[i] >= bound ? 1u << i : 0u;
    int n = 0;
    for (unsigned in; (in = __ballot_sync(kAll, mine != 0)) != 0; mine &= mine - 1) {
      const int at = n + __popc(in & ((1u << lane) - 1));
      if (mine != 0 && at < kListCap)
        sh.list[at] = first + __ffs(mine) - 1;
      n += __popc(in);
    }
    __syncwarp();
    if (n <= kListCap) {
      const int e = lane < n ? sh.list[lane] : -1;
      const uint64_t own = e >= 0 ? (uint64_t)code_of(key_at(e)) << 32 | (uint32_t)~e : 0;
      sh.ranked[lane] = own;
      __syncwarp();
      sh.list[lane] = -1;
      int ahead = 0;
      for (int j = 0; j < n; j += 4)
#pragma unroll
        for (int u = 0; u < 4; ++u) // entries past the n-th are 0
          ahead += sh.ranked[j + u] > own;
      __syncwarp();
      if (e >= 0 && ahead < k)
        sh.list[ahead] = e;
      __syncwarp();
      return sh.list[lane];
    }
  }
  uint32_t code[NV], best = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    code[i] = code_of(key[i]);
    best = max(best, code[i]);
  }
  // the lowest lane that holds the best code and there the lowest place,
  // since lanes hold consecutive experts in order
  int id = -1;
  for (int j = 0; j < k; ++j) {
    const uint32_t m = __reduce_max_sync(kAll, best);
    if (m <= kNone)
      break; // the same for all lanes
    const int src = __ffs(__ballot_sync(kAll, best == m)) - 1;
    int at = 0;
    if (lane == src) {
#pragma unroll
      for (int i = NV - 1; i >= 0; --i)
        at = code[i] == m ? i : at;
      best = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        code[i] = i == at ? 0 : code[i];
        best = max(best, code[i]);
      }
    }
    const int e = __shfl_sync(kAll, first + at, src);
    if (lane == j)
      id = e;
  }
  return id;
}

template <class T, int NV, bool VECTOR, bool SIGMOID>
__global__ void __launch_bounds__(kWarps * 32)
route_kernel(const T* logits, uint32_t tokens, int experts, int64_t stride, int k, bool renormalize, float scale,
             const float* bias, int32_t* ids, float* weights)
{
  __shared__ Choice choices[kWarps];
  wait_for_previous();
  allow_next();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t t = blockIdx.x * kWarps + warp;
  if (t >= tokens)
    return;
  const T* row = logits + (int64_t)t * stride;
  const int first = lane * NV;
  float x[NV];
  load_share<T, NV, VECTOR>(x, row, first, experts);
  float largest = max_of(x);
  const float top = warp_max_nan(largest);
  float sum = 1;
  int id;
  if (bias) {
    // Scores by expf, their sum too: a single one decides here, however small
    // it is. 65536 rows of 256 in f32, k = 8: 34 us, sigmoids 39.
    if (!SIGMOID)
      sum = softmax_sum<false>(x, top);
    const float part = 1.0f / sum;
    auto key_at = [&](int e, float l) {
      const float b = bias[e]; // -inf takes an expert out, NaN scores or not
      return b == -INFINITY ? b : (SIGMOID ? sigmoid(l) : expf(l - top) * part) + b;
    };
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (x[i] != -INFINITY) // which those past the row's end are
        x[i] = key_at(first + i, x[i]);
    largest = max_of(x);
    id = choose<NV>(x, largest, warp_max_nan(largest), k, choices[warp],
                    [&](int e) { return key_at(e, to_f32(row[e])); });
  } else {
    if (!SIGMOID && !renormalize)
      sum = softmax_sum<true>(x, top);
    id = choose<NV>(x, largest, top, k, choices[warp], [&](int e) { return to_f32(row[e]); });
  }
  const bool on = id >= 0;
  const float w = chosen_weight<SIGMOID>(on ? to_f32(row[id]) : 0.0f, on, renormalize, top, sum);
  if (lane < k) {
    ids[(int64_t)t * k + lane] = id;
    weights[(int64_t)t * k + lane] = on ? scale * w : 0.0f;
  }
}

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

int check(segtopk_dtype dtype, const void* logits, int64_t tokens, int32_t experts, int64_t stride, int32_t k,
          int score, int renormalize)
{
  if (dtype < SEGTOPK_F16 || dtype > SEGTOPK_I32 || (score != SEGTOPK_SOFTMAX && score != SEGTOPK_SIGMOID) ||
      (renormalize != 0 && renormalize != 1) || tokens < 0 || experts < 1 || k < 1 || k > experts ||
      stride < 0)
    return SEGTOPK_ERROR_INVALID_VALUE;
  if ((dtype != SEGTOPK_F16 && dtype != SEGTOPK_BF16 && dtype != SEGTOPK_F32) || experts > SEGTOPK_MAX_EXPERTS ||
      k > SEGTOPK_ROUTE_MAX_K || tokens > 2147483647LL / k)
    return SEGTOPK_ERROR_NOT_SUPPORTED;
  if (tokens > 0) {
    if (!logits)
      return SEGTOPK_ERROR_INVALID_VALUE;
    if (!aligned(logits, dtype == SEGTOPK_F32 ? 4 : 2))
      return SEGTOPK_ERROR_MISALIGNED;
  }
  return SEGTOPK_SUCCESS;
}

// Calls f with the share of a lane (a power of two) and whether rows move as
// vectors.
template <class F>
cudaError_t with_share(int experts, bool vector, F&& f)
{
  auto one = [&](auto nv) {
    return vector ? f(nv, std::true_type{}) : f(nv, std::false_type{});
  };
  if (experts <= 32)
    return one(std::integral_constant<int, 1>{});
  if (experts <= 64)
    return one(std::integral_constant<int, 2>{});
  if (experts <= 128)
    return one(std::integral_constant<int, 4>{});
  if (experts <= 256)
    return one(std::integral_constant<int, 8>{});
  if (experts <= 512)
    return one(std::integral_constant<int, 16>{});
  return one(std::integral_constant<int, 32>{});
}

int share_of(int experts)
{
  int nv = 1;
  while (nv * 32 < experts)
    nv *= 2;
  return nv;
}

} // namespace
} // namespace segtopk

using namespace segtopk;

extern "C" int segtopk_route(segtopk_dtype dtype, const void* logits, int64_t tokens, int32_t experts,
                             int64_t row_stride, int32_t k, segtopk_score score, int renormalize, float scale,
                             const float* bias, int32_t* expert_ids, float* weights, void* stream)
{
  record_launch_count(0);
  int rc = check(dtype, logits, tokens, experts, row_stride, k, score, renormalize);
  if (rc != SEGTOPK_SUCCESS)
    return rc;
  if (tokens == 0)
    return SEGTOPK_SUCCESS;
  if (!expert_ids || !weights)
    return SEGTOPK_ERROR_INVALID_VALUE;
  if (!aligned(expert_ids, 4) || !aligned(weights, 4) || !aligned(bias, 4))
    return SEGTOPK_ERROR_MISALIGNED;
  int sms;
  if ((rc = check_device(&sms)) != SEGTOPK_SUCCESS)
    return rc;
  return with_float_type(dtype, [&](auto zero) {
    using T = decltype(zero);
    const int n = std::min<int>(share_of(experts), 16 / (int)sizeof(T));
    const bool vector = rows_fit(logits, row_stride, experts, sizeof(T), n);
    return finish(with_share(experts, vector, [&](auto nv, auto vec) {
      constexpr int NV = decltype(nv)::value;
      constexpr bool V = decltype(vec)::value;
      auto kernel = score == SEGTOPK_SIGMOID ? route_kernel<T, NV, V, true> : route_kernel<T, NV, V, false>;
      return launch(kernel, dim3((unsigned)((tokens + kWarps - 1) / kWarps)), kWarps * 32, 0, (cudaStream_t)stream,
                    (const T*)logits, (uint32_t)tokens, experts, row_stride, k, renormalize != 0, scale, bias,
                    expert_ids, weights);
    }), 1);
  });
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
