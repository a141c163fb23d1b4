// Shared pieces of the row operators (routing, sorting tokens by expert,
// embedding): element types, vectors of them held in 32 bits, launches.
#pragma once

#include <algorithm>
#include <cstdint>
#include <type_traits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/segtopk.h"
#include "entry.h"

namespace segtopk {
namespace rows {

constexpr uint32_t kAll = 0xffffffffu;

// ---------------------------------------------------------------------------
// Launch order
// ---------------------------------------------------------------------------
// Every row kernel is launched as a programmatic dependent of the kernel
// before it on its stream: its blocks may be scheduled while that kernel
// drains, and wait_for_previous() (before any access to global memory, but
// for the one kernel that says otherwise) holds them until that kernel has
// completed and its writes are visible. A chain of such kernels stays in
// order, since none completes before its own wait has ended. allow_next()
// lets the next kernel's blocks be scheduled once all blocks have called it
// or ended; it promises nothing about memory.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void allow_next() { asm volatile("griddepcontrol.launch_dependents;"); }

template <class... P, class... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream, A... args)
{
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// ---------------------------------------------------------------------------
// Elements
// ---------------------------------------------------------------------------
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
// rounded to nearest, ties to even
template <class T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// N consecutive elements, moved as one access where N * sizeof(T) is 2, 4, 8
// or 16 bytes (32 bytes: two), from an address aligned to that size (16 at
// most). They are kept as the 32-bit words they came in, two 16-bit elements
// to a register, until each is used: held as elements, a vector of eight
// takes eight registers, and kernels that keep eight vectors in flight had
// 100 registers a thread and half the occupancy.
template <class T, int N>
struct alignas(sizeof(T) * N > 16 ? 16 : sizeof(T) * N) Vec {
  static constexpr int kWords = (int)sizeof(T) * N / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ float f32(int i) const // i known when compiling
  {
    if constexpr (sizeof(T) == 4)
      return __uint_as_float(w[i]);
    else if constexpr (std::is_same_v<T, __nv_bfloat16>)
      return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    else
      return __half2float(__ushort_as_half((unsigned short)(w[i / 2] >> (16 * (i & 1)))));
  }
  __device__ __forceinline__ void set(const float (&x)[N])
  {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (sizeof(T) == 4) {
        w[i] = __float_as_uint(x[i]);
      } else if constexpr (std::is_same_v<T, __nv_bfloat16>) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
  }
};
template <class T>
struct Vec<T, 1> {
  T one;
  __device__ __forceinline__ float f32(int) const { return to_f32(one); }
  __device__ __forceinline__ void set(const float (&x)[1]) { one = from_f32<T>(x[0]); }
};

template <class T, int N>
__device__ __forceinline__ Vec<T, N> load(const T* p)
{
  Vec<T, N> v;
  if constexpr (sizeof(v) % 16 == 0) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(v) / 16; ++i)
      reinterpret_cast<uint4*>(&v)[i] = reinterpret_cast<const uint4*>(p)[i];
  } else {
    v = *reinterpret_cast<const Vec<T, N>*>(p);
  }
  return v;
}
template <class T, int N>
__device__ __forceinline__ void store(T* p, const Vec<T, N>& v)
{
  if constexpr (sizeof(v) % 16 == 0) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(v) / 16; ++i)
      reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(&v)[i];
  } else {
    *reinterpret_cast<Vec<T, N>*>(p) = v;
  }
}
template <class T, int N>
__device__ __forceinline__ void store_f32(T* p, const float (&x)[N])
{
  Vec<T, N> v;
  v.set(x);
  store<T, N>(p, v);
}

// What a thread moves of a row at a time. Where rows start and end on whole
// vectors, N > 1 consecutive elements. Otherwise (N = 1) kLoose single ones, a
// group's threads apart, so that a warp still reads consecutive addresses and
// a thread has as many loads under way: 8192 rows of 2047 in bf16, summed four
// by four, took 139 us one element at a time.
constexpr int kLoose = 4;
template <class T>
struct Loose {
  T at[kLoose];
  __device__ __forceinline__ float f32(int i) const { return to_f32(at[i]); }
};
template <class T, int N>
using Part = std::conditional_t<(N > 1), Vec<T, N>, Loose<T>>;
template <int N>
constexpr int kPart = N > 1 ? N : kLoose; // its elements

// Where a lane's first part of a row begins; `lanes` parts make a step of
// lanes * kPart<N> columns.
template <int N>
__device__ __forceinline__ int part_start(int lane)
{
  return N > 1 ? lane * N : lane;
}
// p: the part's first element; left: columns of the row from there on (none
// are read or written past them).
template <class T, int N>
__device__ __forceinline__ Part<T, N> load_part(const T* p, int lanes, int64_t left)
{
  if constexpr (N > 1) {
    return load<T, N>(p);
  } else {
    Loose<T> v = {};
#pragma unroll
    for (int i = 0; i < kLoose; ++i)
      if (i * lanes < left)
        v.at[i] = p[i * lanes];
    return v;
  }
}
template <class T, int N>
__device__ __forceinline__ void store_part(T* p, const float (&x)[kPart<N>], int lanes, int64_t left)
{
  if constexpr (N > 1) {
    store_f32<T, N>(p, x);
  } else {
#pragma unroll
    for (int i = 0; i < kLoose; ++i)
      if (i * lanes < left)
        p[i * lanes] = from_f32<T>(x[i]);
  }
}

// ---------------------------------------------------------------------------
// Asynchronous copies of a thread's own
// ---------------------------------------------------------------------------
// A kernel that gathers rows is bound by their latency unless enough of them
// are under way. Copied into shared memory ahead of their use they take no
// registers, and where a thread reads only what it copied itself, no barrier.
constexpr int kRingBytes = 48 << 10; // of a block: no opt-in, four blocks an SM

template <int BYTES>
__device__ __forceinline__ void copy_async(void* to, const void* from)
{
  const uint32_t at = (uint32_t)__cvta_generic_to_shared(to);
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(at), "l"(from), "n"(BYTES) : "memory");
}
// Copies since the last call become a group (an empty one without any).
__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_for_copies() // all but the last N groups
{
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ---------------------------------------------------------------------------
// Host helpers
// ---------------------------------------------------------------------------
// Calls f with a value of the element type of `dtype`; NOT_SUPPORTED for a
// type the row operators do not take.
template <class F>
int with_float_type(int dtype, F&& f)
{
  switch (dtype) {
  case SEGTOPK_F16: return f(__half{});
  case SEGTOPK_BF16: return f(__nv_bfloat16{});
  case SEGTOPK_F32: return f(float{});
  case SEGTOPK_F64:
  case SEGTOPK_U32:
  case SEGTOPK_I32: return SEGTOPK_ERROR_NOT_SUPPORTED;
  default: return SEGTOPK_ERROR_INVALID_VALUE;
  }
}

inline bool aligned(const void* p, size_t bytes) { return ((uintptr_t)p & (bytes - 1)) == 0; }

// Whether rows of `width` elements of `size` bytes, `stride` elements apart
// from p on, can be moved as vectors of `n` elements.
inline bool rows_fit(const void* p, int64_t stride, int64_t width, size_t size, int n)
{
  const size_t bytes = std::min<size_t>(16, size * (size_t)n);
  return width % n == 0 && aligned(p, bytes) && ((size_t)stride * size) % bytes == 0;
}

// Parts of a row of `width` columns.
inline int64_t parts_of(int64_t width, int n)
{
  const int part = n > 1 ? n : kLoose;
  return (width + part - 1) / part;
}

// Threads that share one row: the smallest power of two that covers `vectors`
// (at least 1), up to `most`.
inline int lanes_for(int64_t vectors, int most)
{
  int l = 1;
  while (l < most && l < vectors)
    l *= 2;
  return l;
}

inline int finish(cudaError_t e, int launches)
{
  if (e != cudaSuccess)
    return record_cuda_error(e);
  record_launch_count(launches);
  return SEGTOPK_SUCCESS;
}

} // namespace rows
} // namespace segtopk
