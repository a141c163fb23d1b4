// Layer norm of rows and its gradients, and rows in 8 bits with a scale for
// each block of 128 (segtopk_layer_norm, segtopk_layer_norm_backward and
// segtopk_quantize_rows in include/segtopk.h).
//
// A row x of n values: m = mean(x), r = 1 / sqrt(mean((x - m)^2) + eps), h =
// (x - m) r, y = h w + b. With g the gradient of y:
//   of x  r (g w - mean(g w) - h mean(g w h))
//   of w  the sum over the rows of g h,  of b  that of g
//
// All are bound by memory: a group of threads holds a row in registers, so
// that it is read once, and its sums go through shuffles and, where the group
// is more than a warp, shared memory. The gradient of w and b takes two
// kernels: the first keeps each thread's columns' sums in registers over all
// the rows of its block and leaves one row of sums a block, the second adds
// those up in order. So the sums do not depend on timing.
#include "rows.cuh"

namespace segtopk {
namespace {
using namespace rows;

constexpr int kThreads = 256; // of a block where a warp serves a row
constexpr int kSmWarps = 16;  // of the blocks that an SM holds at once, backward pass
constexpr int threads_of(int warps) { return warps == 1 ? kThreads : warps * 32; }
constexpr int groups_of(int warps) { return warps == 1 ? kThreads / 32 : 1; }
constexpr int kMaxNormWidth = SEGTOPK_MAX_NORM_WIDTH;

__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    x += __shfl_xor_sync(kAll, x, o);
  return x;
}

// The sums of x and y over the group: a warp, or all of the block's WARPS.
// Two buffers in turn, so that one barrier a sum is enough.
template <int WARPS>
struct Sums {
  float2 part[2][WARPS];
};
template <int WARPS>
__device__ __forceinline__ float2 group_sum(float2 v, Sums<WARPS>& sh, int& turn)
{
  v.x = warp_sum(v.x);
  v.y = warp_sum(v.y);
  if constexpr (WARPS == 1) {
    return v;
  } else {
    float2* part = sh.part[turn];
    turn ^= 1;
    if ((threadIdx.x & 31) == 0)
      part[threadIdx.x / 32] = v;
    __syncthreads();
    const float2 p = (threadIdx.x & 31) < WARPS ? part[threadIdx.x & 31] : float2{};
    return make_float2(warp_sum(p.x), warp_sum(p.y));
  }
}

// A thread's part of a row: PARTS times kPart<N> columns, a step of the group's
// threads apart; zeros past the row's end, where nothing is read.
template <class T, int N, int PARTS>
struct Share {
  Part<T, N> part[PARTS];
};
template <class T, int N, int PARTS>
__device__ __forceinline__ void load_row(Share<T, N, PARTS>& s, const T* row, int lane, int lanes, int width)
{
#pragma unroll
  for (int i = 0; i < PARTS; ++i) {
    const int at = part_start<N>(lane) + i * lanes * kPart<N>;
    if (at < width)
      s.part[i] = load_part<T, N>(row + at, lanes, width - at);
    else
      s.part[i] = {};
  }
}
// Whether place j of part i is in the row.
template <int N>
__device__ __forceinline__ bool in_row(int lane, int lanes, int width, int i, int j)
{
  const int at = part_start<N>(lane) + i * lanes * kPart<N>;
  return N > 1 ? at < width : at + j * lanes < width;
}

// Parts of a row a thread has against warps that wait for one another: rows of
// 4096 in bf16 (65536 of them) took 205 us with 2 parts and 8 warps, 172 with 4
// and 4, 178 with 8 and 2, 200 with 16 and one; of 2048 199, 170 (4 and 2) and
// 158 (8 and one). A row read ahead into registers, or several into shared
// memory, cost more warps than it hid latency. At 80 registers 8 parts in 16
// bits spill 8 to 64 bytes a thread, which the figures above include.
template <class T, class W, int N, int PARTS, int WARPS>
__global__ void __launch_bounds__(threads_of(WARPS), std::max(1, (WARPS == 1 ? 768 : PARTS == 4 ? 1024 : 768) / threads_of(WARPS)))
norm_kernel(const T* x, int64_t x_stride, uint32_t rows, int width, const W* weight, const W* bias, float eps, T* out,
            float* means, float* rstds)
{
  __shared__ float2 part[WARPS];
  wait_for_previous();
  allow_next();
  constexpr int kLanes = WARPS * 32;
  const int lane = threadIdx.x % kLanes, warp = lane / 32;
  const float part_of = 1.0f / (float)width;
  // values that this warp, and each warp, has
  auto values_of = [&](int w) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
      if constexpr (N > 1) {
        n += max(0, min(32 * N, width - (i * kLanes + w * 32) * N));
      } else {
#pragma unroll
        for (int j = 0; j < kLoose; ++j)
          n += max(0, min(32, width - (i * kLoose + j) * kLanes - w * 32));
      }
    }
    return (float)n;
  };
  const float mine = values_of(warp);
  const float other = WARPS > 1 && (threadIdx.x & 31) < WARPS ? values_of(threadIdx.x & 31) : 0.0f;
  const uint32_t r = blockIdx.x * (blockDim.x / kLanes) + threadIdx.x / kLanes;
  if (r < rows) { // the same for all of a group
    Share<T, N, PARTS> s;
    load_row(s, x + (int64_t)r * x_stride, lane, kLanes, width);
    // the warp's mean and its values' squares about it, then those of the row:
    // n var = sum over the warps of theirs + n_w (mean_w - mean)^2, which needs
    // one barrier and does not cancel
    float sum = 0;
#pragma unroll
    for (int i = 0; i < PARTS; ++i)
#pragma unroll
      for (int j = 0; j < kPart<N>; ++j)
        sum += s.part[i].f32(j);
    float mean = mine > 0 ? warp_sum(sum) / mine : 0.0f;
    float square = 0;
#pragma unroll
    for (int i = 0; i < PARTS; ++i)
#pragma unroll
      for (int j = 0; j < kPart<N>; ++j) {
        const float d = in_row<N>(lane, kLanes, width, i, j) ? s.part[i].f32(j) - mean : 0.0f;
        square = fmaf(d, d, square);
      }
    square = warp_sum(square);
    if constexpr (WARPS > 1) {
      if ((threadIdx.x & 31) == 0)
        part[warp] = make_float2(mean, square);
      __syncthreads();
      const float2 p = other > 0 ? part[threadIdx.x & 31] : float2{};
      mean = warp_sum(p.x * other) * part_of;
      const float d = p.x - mean;
      square = warp_sum(fmaf(d * d, other, p.y));
    }
    const float rstd = 1.0f / sqrtf(square * part_of + eps);
    if (lane == 0) {
      means[r] = mean;
      rstds[r] = rstd;
    }
    T* const to = out + (int64_t)r * width;
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
      const int at = part_start<N>(lane) + i * kLanes * kPart<N>;
      if (at < width) {
        const Part<W, N> w = load_part<W, N>(weight + at, kLanes, width - at);
        float y[kPart<N>];
        if (bias) {
          const Part<W, N> b = load_part<W, N>(bias + at, kLanes, width - at);
#pragma unroll
          for (int j = 0; j < kPart<N>; ++j)
            y[j] = fmaf((s.part[i].f32(j) - mean) * rstd, w.f32(j), b.f32(j));
        } else {
#pragma unroll
          for (int j = 0; j < kPart<N>; ++j)
            y[j] = (s.part[i].f32(j) - mean) * rstd * w.f32(j);
        }
        store_part<T, N>(to + at, y, kLanes, width - at);
      }
    }
  }
}

// Rows' gradients, and a row of the sums of g h and of g for each block.
//
// Where a group is a large block, whose warps wait for one another at every
// row, it loads its next row while it works on one: 65536 rows of 4096 in
// bf16 283 us, 315 without; with 4 parts and 4 warps 294. Groups of two warps
// and single ones do not: rows of 2048 278 us, 354 with a row ahead.
// Rows over 8192 values take a block of 32 warps, whose 64 registers a thread
// spill 120 to 576 bytes: 16384 rows of 16384 in bf16 436 us, 237 at the copy
// rate, in f32 1202 and 474.
constexpr bool ahead(int warps) { return warps >= 8; }

template <class T, class W, int N, int PARTS, int WARPS>
__global__ void __launch_bounds__(threads_of(WARPS), std::max(1, kSmWarps / (threads_of(WARPS) / 32)))
norm_backward_kernel(const T* grad, int64_t grad_stride, const T* x, int64_t x_stride, uint32_t rows, int width,
                     const W* weight, const float* means, const float* rstds, T* grad_x, float* sums)
{
  __shared__ Sums<WARPS> sh;
  constexpr int kLanes = WARPS * 32, kGroups = WARPS == 1 ? kThreads / 32 : 1;
  __shared__ float joined[kGroups > 1 ? (kGroups / 2) * 32 * kPart<N> : 1];
  wait_for_previous();
  allow_next();
  const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  const uint32_t step = gridDim.x * kGroups;
  int turn = 0;
  const float part_of = 1.0f / (float)width;
  float sum_w[PARTS][kPart<N>] = {}, sum_b[PARTS][kPart<N>] = {};
  struct Row {
    Share<T, N, PARTS> g, x;
    float mean, rstd;
  };
  auto get = [&](Row& row, uint32_t r) {
    load_row(row.g, grad + (int64_t)r * grad_stride, lane, kLanes, width);
    load_row(row.x, x + (int64_t)r * x_stride, lane, kLanes, width);
    row.mean = means[r];
    row.rstd = rstds[r];
  };
  Row next;
  uint32_t r = blockIdx.x * kGroups + group;
  if (ahead(WARPS) && r < rows)
    get(next, r);
  for (; r < rows; r += step) { // rows + step is below 2^32
    Row row;
    if constexpr (ahead(WARPS)) {
      row = next;
      if (step < rows - r)
        get(next, r + step);
    } else {
      get(row, r);
    }
    const Share<T, N, PARTS>&sx = row.x, &sg = row.g;
    const float mean = row.mean, rstd = row.rstd;
    float2 inner = {};
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
      const int at = part_start<N>(lane) + i * kLanes * kPart<N>;
      if (at < width) {
        const Part<W, N> w = load_part<W, N>(weight + at, kLanes, width - at);
#pragma unroll
        for (int j = 0; j < kPart<N>; ++j) {
          // past the row's end g is 0, and x may be anything finite
          const float g = sg.part[i].f32(j), h = (sx.part[i].f32(j) - mean) * rstd;
          const bool in = N > 1 || in_row<N>(lane, kLanes, width, i, j);
          sum_w[i][j] += in ? g * h : 0.0f;
          sum_b[i][j] += in ? g : 0.0f;
          const float gw = in ? g * w.f32(j) : 0.0f;
          inner.x += gw;
          inner.y = fmaf(gw, in ? h : 0.0f, inner.y);
        }
      }
    }
    inner = group_sum<WARPS>(inner, sh, turn);
    const float a = inner.x * part_of, b = inner.y * part_of;
    T* const to = grad_x + (int64_t)r * width;
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
      const int at = part_start<N>(lane) + i * kLanes * kPart<N>;
      if (at < width) {
        const Part<W, N> w = load_part<W, N>(weight + at, kLanes, width - at);
        float y[kPart<N>];
#pragma unroll
        for (int j = 0; j < kPart<N>; ++j) {
          const float h = (sx.part[i].f32(j) - mean) * rstd;
          y[j] = rstd * (fmaf(sg.part[i].f32(j), w.f32(j), -a) - h * b);
        }
        store_part<T, N>(to + at, y, kLanes, width - at);
      }
    }
  }
  // one row of sums a block, [2][width]
  float* const to = sums + (int64_t)blockIdx.x * 2 * width;
#pragma unroll
  for (int i = 0; i < PARTS; ++i) {
    const int at = part_start<N>(lane) + i * kLanes * kPart<N>;
    for (int which = 0; which < 2; ++which) {
      float v[kPart<N>];
#pragma unroll
      for (int j = 0; j < kPart<N>; ++j)
        v[j] = which ? sum_b[i][j] : sum_w[i][j];
      if constexpr (kGroups > 1) {
        // the upper half of the groups to the lower, until one is left
#pragma unroll
        for (int n = kGroups / 2; n > 0; n /= 2) {
          __syncthreads();
          if (group >= n && group < 2 * n)
#pragma unroll
            for (int j = 0; j < kPart<N>; ++j)
              joined[((group - n) * kPart<N> + j) * 32 + lane] = v[j];
          __syncthreads();
          if (group < n)
#pragma unroll
            for (int j = 0; j < kPart<N>; ++j)
              v[j] += joined[(group * kPart<N> + j) * 32 + lane];
        }
      }
      if (group == 0 && at < width)
        store_part<float, N>(to + which * width + at, v, kLanes, width - at);
    }
  }
}

// Adds up the blocks' rows of sums: a block for 32 columns of either, each
// warp an equal run of the rows, the warps in order.
constexpr int kJoinWarps = 16;
template <class W>
__global__ void __launch_bounds__(kJoinWarps * 32)
norm_join_kernel(const float* sums, int blocks, int width, W* grad_weight, W* grad_bias)
{
  __shared__ float part[kJoinWarps][33];
  wait_for_previous();
  allow_next();
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane; // of 2 * width
  float sum = 0;
  if (c < 2 * (int64_t)width) {
    const float* at = sums + c;
    const int each = (blocks + kJoinWarps - 1) / kJoinWarps;
    const int end = min(blocks, (warp + 1) * each);
#pragma unroll 16
    for (int b = warp * each; b < end; ++b)
      sum += at[(int64_t)b * 2 * width];
  }
  part[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && c < 2 * (int64_t)width) {
    sum = 0;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w)
      sum += part[w][lane];
    if (c < width)
      grad_weight[c] = from_f32<W>(sum);
    else
      grad_bias[c - width] = from_f32<W>(sum);
  }
}

// ---------------------------------------------------------------------------
// Rows in 8 bits
// ---------------------------------------------------------------------------
constexpr int kBlock = 128;              // values of a scale
constexpr float kLargest = 448.0f;       // of e4m3
constexpr float kSmallest = 0x1p-100f;   // below it a block's largest value counts as this

__device__ __forceinline__ uint32_t to_e4m3(float a, float b, float c, float d) // to nearest, ties to even
{
  uint16_t low, high;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(low) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(high) : "f"(d), "f"(c));
  return low | (uint32_t)high << 16;
}
__device__ __forceinline__ float max_nan(float x, float y)
{
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(x), "f"(y));
  return m;
}

// Eight values a thread, 16 threads a block of values. STEPS of them are read
// before the first is used and stay in the type they came in until then.
// 131072 rows of 4096 in bf16: 260 us, 240 at the copy rate; 282 when all were
// widened to 32 bits at once.
template <class T, bool VECTOR, int STEPS>
__global__ void __launch_bounds__(kThreads)
quantize_kernel(const T* x, int64_t x_stride, uint32_t blocks, uint32_t per_row, float per_row_inverse, int width,
                uint8_t* values, float* scales)
{
  wait_for_previous();
  allow_next();
  constexpr int kGroups = kThreads / 16;
  const int lane = threadIdx.x & 15;
  const uint32_t first = blockIdx.x * (kGroups * STEPS) + threadIdx.x / 16;
  struct Eight {
    T v[8];
  };
  std::conditional_t<VECTOR, Vec<T, 8>, Eight> got[STEPS];
  uint32_t row[STEPS];
  int at[STEPS];
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const uint32_t b = first + i * kGroups;
    // b / per_row: by a product, at most one off below 2^22, and a step
    uint32_t r = b >> 22 ? b / per_row : (uint32_t)((float)b * per_row_inverse);
    const int32_t rest = (int32_t)(b - r * per_row);
    r += rest < 0 ? -1 : rest >= (int32_t)per_row ? 1 : 0;
    row[i] = r;
    at[i] = (int)(b - r * per_row) * kBlock + (VECTOR ? lane * 8 : lane); // then 16 apart, side by side in a warp
    const bool in = b < blocks;
    const T* from = x + (int64_t)r * x_stride + at[i];
    if constexpr (VECTOR) {
      got[i] = {};
      if (in && at[i] < width) // width is a multiple of 8
        got[i] = load<T, 8>(from);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        got[i].v[j] = in && at[i] + 16 * j < width ? from[16 * j] : from_f32<T>(0.0f);
    }
  }
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (VECTOR)
        v[j] = got[i].f32(j);
      else
        v[j] = to_f32(got[i].v[j]);
    }
    float most = fabsf(v[0]);
#pragma unroll
    for (int j = 1; j < 8; ++j)
      most = max_nan(most, fabsf(v[j]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
      most = max_nan(most, __shfl_xor_sync(kAll, most, o));
    most = max_nan(most, kSmallest);
    const float by = kLargest / most;
    const uint2 q = {to_e4m3(v[0] * by, v[1] * by, v[2] * by, v[3] * by), to_e4m3(v[4] * by, v[5] * by, v[6] * by, v[7] * by)};
    const uint32_t b = first + i * kGroups;
    if (b < blocks) {
      if (lane == 0)
        scales[b] = most / kLargest;
      uint8_t* to = values + (int64_t)row[i] * width + at[i];
      if constexpr (VECTOR) {
        if (at[i] < width)
          *reinterpret_cast<uint2*>(to) = q;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (at[i] + 16 * j < width)
            to[16 * j] = (uint8_t)((j < 4 ? q.x : q.y) >> (8 * (j & 3)));
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
// Calls f with the parts that a thread holds of a row and the warps of a group
// (measured at the kernels).
#define SEGTOPK_GROUP(P, WARPS) return f(std::integral_constant<int, P>{}, std::integral_constant<int, WARPS>{})
template <class F>
cudaError_t with_group(int64_t parts, F&& f)
{
  if (parts <= 64)
    SEGTOPK_GROUP(2, 1);
  if (parts <= 128)
    SEGTOPK_GROUP(4, 1);
  if (parts <= 256)
    SEGTOPK_GROUP(8, 1);
  if (parts <= 512)
    SEGTOPK_GROUP(4, 4);
  if (parts <= 1024)
    SEGTOPK_GROUP(8, 4);
  if (parts <= 2048)
    SEGTOPK_GROUP(8, 8);
  SEGTOPK_GROUP(8, 16);
}
template <int N, class F>
cudaError_t with_backward_group(int64_t parts, int64_t rows, F&& f)
{
  if (parts <= 64)
    SEGTOPK_GROUP(2, 1);
  // with few rows more warps for each: 1237 of 1001 in f32 8.3 us, 13.0 by (4, 2); measured at that size alone
  const bool few = rows <= 152 * 16;
  if (parts <= 128 && !few)
    SEGTOPK_GROUP(4, 1);
  if (parts <= 256) {
    if (few)
      SEGTOPK_GROUP(1, 8);
    SEGTOPK_GROUP(4, 2);
  }
  if (parts <= 512)
    SEGTOPK_GROUP(2, 8);
  if (parts <= 1024)
    SEGTOPK_GROUP(2, 16);
  if constexpr (kMaxNormWidth / kPart<N> > 2048)
    if (parts > 2048)
      SEGTOPK_GROUP(4, 32);
  SEGTOPK_GROUP(2, 32);
}
#undef SEGTOPK_GROUP

// Blocks of the backward pass stay and take row after row; each leaves 2 *
// width sums, so a group has four rows at least where that leaves no SM idle
// (1237 rows of 1001 in f32: 14.1 us with one row each, 1216 blocks).
constexpr int64_t kSms = 152;
constexpr int64_t kMostBlocks = kSms * (kSmWarps / 2);
int64_t blocks_for(int64_t rows, int warps)
{
  const int64_t resident = kSms * std::max(1, kSmWarps / (threads_of(warps) / 32));
  const int64_t each = groups_of(warps), most = (rows + each - 1) / each;
  return std::max<int64_t>(1, std::min({most, std::max(kSms, most / 4), resident}));
}

int check(segtopk_dtype dtype, segtopk_dtype weight_dtype, int64_t rows, int64_t width)
{
  if (dtype < SEGTOPK_F16 || dtype > SEGTOPK_I32 || weight_dtype < SEGTOPK_F16 || weight_dtype > SEGTOPK_I32 || rows < 0 ||
      width < 1)
    return SEGTOPK_ERROR_INVALID_VALUE;
  auto is_float = [](int t) { return t == SEGTOPK_F16 || t == SEGTOPK_BF16 || t == SEGTOPK_F32; };
  if (!is_float(dtype) || (weight_dtype != dtype && weight_dtype != SEGTOPK_F32) || rows > 2147483647LL ||
      width > kMaxNormWidth)
    return SEGTOPK_ERROR_NOT_SUPPORTED;
  return SEGTOPK_SUCCESS;
}
size_t size_of(int dtype) { return dtype == SEGTOPK_F32 ? 4 : 2; }

// Calls f with values of the rows' and the weight's type.
template <class F>
int with_types(segtopk_dtype dtype, segtopk_dtype weight_dtype, F&& f)
{
  return with_float_type(dtype, [&](auto x) { return weight_dtype == dtype ? f(x, x) : f(x, float{}); });
}

} // namespace
} // namespace segtopk

using namespace segtopk;

extern "C" int segtopk_layer_norm(segtopk_dtype dtype, const void* x, int64_t num_rows, int64_t width, int64_t row_stride,
                                  segtopk_dtype weight_dtype, const void* weight, const void* bias, float eps, void* out,
                                  float* mean, float* rstd, void* stream)
{
  record_launch_count(0);
  int rc = check(dtype, weight_dtype, num_rows, width);
  if (rc != SEGTOPK_SUCCESS)
    return rc;
  if (row_stride < 0 || !(eps >= 0))
    return SEGTOPK_ERROR_INVALID_VALUE;
  if (num_rows == 0)
    return SEGTOPK_SUCCESS;
  if (!x || !weight || !out || !mean || !rstd)
    return SEGTOPK_ERROR_INVALID_VALUE;
  if (!aligned(x, size_of(dtype)) || !aligned(out, size_of(dtype)) || !aligned(weight, size_of(weight_dtype)) ||
      !aligned(bias, size_of(weight_dtype)) || !aligned(mean, 4) || !aligned(rstd, 4))
    return SEGTOPK_ERROR_MISALIGNED;
  int sms;
  if ((rc = check_device(&sms)) != SEGTOPK_SUCCESS)
    return rc;
  return with_types(dtype, weight_dtype, [&](auto tx, auto tw) {
    using T = decltype(tx);
    using W = decltype(tw);
    constexpr int N = 16 / (int)sizeof(T);
    const bool vector = rows_fit(x, row_stride, width, sizeof(T), N) && rows_fit(out, width, width, sizeof(T), N) &&
                        rows_fit(weight, width, width, sizeof(W), N) && rows_fit(bias, width, width, sizeof(W), N);
    auto go = [&](auto n) {
      constexpr int V = decltype(n)::value;
      return with_group(parts_of(width, V), [&](auto parts, auto warps) {
        constexpr int G = decltype(warps)::value;
        const int64_t blocks = (num_rows + groups_of(G) - 1) / groups_of(G);
        return launch(norm_kernel<T, W, V, decltype(parts)::value, G>, dim3((unsigned)blocks),
                      threads_of(G), 0, (cudaStream_t)stream, (const T*)x, row_stride, (uint32_t)num_rows, (int)width,
                      (const W*)weight, (const W*)bias, eps, (T*)out, mean, rstd);
      });
    };
    return finish(vector ? go(std::integral_constant<int, N>{}) : go(std::integral_constant<int, 1>{}), 1);
  });
}

extern "C" size_t segtopk_layer_norm_backward_workspace_bytes(int64_t num_rows, int64_t width)
{
  if (num_rows < 1 || num_rows > 2147483647LL || width < 1 || width > kMaxNormWidth)
    return 0;
  return (size_t)std::min(num_rows, kMostBlocks) * 2 * width * sizeof(float);
}

extern "C" int segtopk_layer_norm_backward(segtopk_dtype dtype, const void* grad_out, int64_t grad_stride, const void* x,
                                           int64_t num_rows, int64_t width, int64_t row_stride,
                                           segtopk_dtype weight_dtype, const void* weight, const float* mean,
                                           const float* rstd, void* grad_x, void* grad_weight, void* grad_bias,
                                           void* workspace, size_t workspace_bytes, void* stream)
{
  record_launch_count(0);
  int rc = check(dtype, weight_dtype, num_rows, width);
  if (rc != SEGTOPK_SUCCESS)
    return rc;
  if (row_stride < 0 || grad_stride < 0 || !grad_weight || !grad_bias)
    return SEGTOPK_ERROR_INVALID_VALUE;
  if (!aligned(grad_weight, size_of(weight_dtype)) || !aligned(grad_bias, size_of(weight_dtype)))
    return SEGTOPK_ERROR_MISALIGNED;
  if (num_rows > 0) {
    if (!grad_out || !x || !weight || !mean || !rstd || !grad_x || !workspace ||
        workspace_bytes < segtopk_layer_norm_backward_workspace_bytes(num_rows, width))
      return SEGTOPK_ERROR_INVALID_VALUE;
    if (!aligned(x, size_of(dtype)) || !aligned(grad_out, size_of(dtype)) || !aligned(grad_x, size_of(dtype)) ||
        !aligned(weight, size_of(weight_dtype)) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(workspace, 16))
      return SEGTOPK_ERROR_MISALIGNED;
  }
  int sms;
  if ((rc = check_device(&sms)) != SEGTOPK_SUCCESS)
    return rc;
  return with_types(dtype, weight_dtype, [&](auto tx, auto tw) {
    using T = decltype(tx);
    using W = decltype(tw);
    constexpr int N = 16 / (int)sizeof(T);
    int blocks = 0;
    cudaError_t e = cudaSuccess;
    if (num_rows > 0) {
      const bool vector = rows_fit(x, row_stride, width, sizeof(T), N) &&
                          rows_fit(grad_out, grad_stride, width, sizeof(T), N) &&
                          rows_fit(grad_x, width, width, sizeof(T), N) && rows_fit(weight, width, width, sizeof(W), N);
      auto go = [&](auto n) {
        constexpr int V = decltype(n)::value;
        return with_backward_group<V>(parts_of(width, V), num_rows, [&](auto parts, auto warps) {
          constexpr int G = decltype(warps)::value;
          blocks = (int)blocks_for(num_rows, G);
          return launch(norm_backward_kernel<T, W, V, decltype(parts)::value, G>, dim3((unsigned)blocks), threads_of(G), 0,
                        (cudaStream_t)stream, (const T*)grad_out, grad_stride, (const T*)x, row_stride,
                        (uint32_t)num_rows, (int)width, (const W*)weight, mean, rstd, (T*)grad_x, (float*)workspace);
        });
      };
      e = vector ? go(std::integral_constant<int, N>{}) : go(std::integral_constant<int, 1>{});
    }
    if (e == cudaSuccess)
      e = launch(norm_join_kernel<W>, dim3((unsigned)((2 * width + 31) / 32)), kJoinWarps * 32, 0, (cudaStream_t)stream,
                 (const float*)workspace, blocks, (int)width, (W*)grad_weight, (W*)grad_bias);
    return finish(e, num_rows > 0 ? 2 : 1);
  });
}

extern "C" int segtopk_quantize_rows(segtopk_dtype dtype, const void* x, int64_t num_rows, int64_t width,
                                     int64_t row_stride, void* values, float* scales, void* stream)
{
  record_launch_count(0);
  if (dtype < SEGTOPK_F16 || dtype > SEGTOPK_I32 || num_rows < 0 || width < 1 || row_stride < 0)
    return SEGTOPK_ERROR_INVALID_VALUE;
  if ((dtype != SEGTOPK_F16 && dtype != SEGTOPK_BF16 && dtype != SEGTOPK_F32) || num_rows > 2147483647LL ||
      width > (1 << 20) || num_rows * ((width + kBlock - 1) / kBlock) > 2147483647LL)
    return SEGTOPK_ERROR_NOT_SUPPORTED;
  if (num_rows == 0)
    return SEGTOPK_SUCCESS;
  if (!x || !values || !scales)
    return SEGTOPK_ERROR_INVALID_VALUE;
  if (!aligned(x, size_of(dtype)) || !aligned(scales, 4))
    return SEGTOPK_ERROR_MISALIGNED;
  int sms;
  const int rc = check_device(&sms);
  if (rc != SEGTOPK_SUCCESS)
    return rc;
  return with_float_type(dtype, [&](auto zero) {
    using T = decltype(zero);
    const uint32_t per_row = (uint32_t)((width + kBlock - 1) / kBlock);
    const int64_t blocks = num_rows * per_row;
    const bool vector = width % 8 == 0 && rows_fit(x, row_stride, width, sizeof(T), 16 / (int)sizeof(T)) &&
                        aligned(values, 8);
    // several blocks a group where the GPU has enough of them anyway
    const bool few = blocks < (int64_t)sms * 2048 / 16;
    auto go = [&](auto vec, auto steps) {
      constexpr int S = decltype(steps)::value;
      const int64_t each = kThreads / 16 * S;
      return launch(quantize_kernel<T, decltype(vec)::value, S>, dim3((unsigned)((blocks + each - 1) / each)), kThreads, 0,
                    (cudaStream_t)stream, (const T*)x, row_stride, (uint32_t)blocks, per_row, 1.0f / (float)per_row, (int)width, (uint8_t*)values, scales);
    };
    auto by = [&](auto vec) {
      return few ? go(vec, std::integral_constant<int, 1>{}) : go(vec, std::integral_constant<int, 4>{});
    };
    return finish(vector ? by(std::true_type{}) : by(std::false_type{}), 1);
  });
}
