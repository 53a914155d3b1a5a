// What the norms' kernels share: statistics of a row, columns in registers, copies
// ahead into shared memory.
#pragma once

#include "ops_internal.cuh"

namespace ar {
namespace {

constexpr int kAnyThreads = 256;

template <class E>
__device__ __forceinline__ float value(const void* p, int64_t i) {
  return E::to_f32(ld_elem<E::kBytes>(static_cast<const char*>(p) + i * E::kBytes));
}
template <class E>
__device__ __forceinline__ void put(void* p, int64_t i, float v) {
  st_elem<E::kBytes>(static_cast<char*>(p) + i * E::kBytes, E::from_f32(v));
}

// The sums of v over the CTA's threads, in a fixed order; `room` is free again
// once every thread has called this for another room.
template <int N>
__device__ __forceinline__ void cta_sums(float (&v)[N], float (*room)[32]) {
#pragma unroll
  for (int k = 0; k < N; ++k)
#pragma unroll
    for (int o = 16; o; o >>= 1) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], o);
  const int warps = (int)blockDim.x >> 5, lane = threadIdx.x & 31;
  if (warps == 1) return;
  if (lane == 0)
#pragma unroll
    for (int k = 0; k < N; ++k) room[k][threadIdx.x >> 5] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    v[k] = lane < warps ? room[k][lane] : 0.0f;
#pragma unroll
    for (int o = 16; o; o >>= 1) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], o);
  }
}

// A row's mean (0 for the root mean square) and the factor 1 / sqrt(mean square + eps).
struct Stats {
  float mean, factor;
};

// Statistics of the row whose element c is get(c), by passes over it.
template <class F>
__device__ __forceinline__ Stats stats_any(F get, int64_t cols, int layer, float eps, float (*room)[32]) {
  Stats s = {0.0f, 0.0f};
  float v[1];
  if (layer) {
    v[0] = 0.0f;
    for (int64_t c = threadIdx.x; c < cols; c += kAnyThreads) v[0] += get(c);
    cta_sums<1>(v, room);
    s.mean = v[0] / (float)cols;
  }
  v[0] = 0.0f;
  for (int64_t c = threadIdx.x; c < cols; c += kAnyThreads) {
    const float d = get(c) - s.mean;
    v[0] = __fmaf_rn(d, d, v[0]);
  }
  cta_sums<1>(v, room + 1);
  s.factor = 1.0f / sqrtf(v[0] / (float)cols + eps);
  return s;
}

// ---------------------------------------------------------------------------
// Rows that a CTA (or a warp) holds in registers.

// The columns of thread t of the T that share a row, N of them.  VEC (every row
// and vector starts on 16 bytes): 16 bytes at a time; else one by one, so that neighbouring
// threads read neighbouring elements.
template <class E, int N, bool VEC>
struct Columns {
  static constexpr int G = E::kGroup, B = E::kBytes;
  int t, T, cols;

  __device__ __forceinline__ int at(int i) const { return VEC ? (t + i / G * T) * G + i % G : t + i * T; }
  __device__ __forceinline__ bool has(int i) const { return at(i) < cols; }
  // Columns past the last are 0.
  __device__ __forceinline__ void load(const void* p, int64_t first, float (&v)[N]) const {
    const char* row = static_cast<const char*>(p) + first * B;
    if (VEC) {
#pragma unroll
      for (int i = 0; i < N; i += G) {
        Acc<E> a;
        a.set(at(i) < cols ? load_group<E>(row, at(i) / G, min(cols - at(i), G), true) : make_uint4(0, 0, 0, 0));
#pragma unroll
        for (int k = 0; k < G; ++k) v[i + k] = a.v[k];
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = has(i) ? E::to_f32(ld_elem<B>(row + (int64_t)at(i) * B)) : 0.0f;
    }
  }
  // The same of what other rows' threads read too.
  __device__ __forceinline__ void load_shared(const void* p, int64_t first, float (&v)[N]) const {
    if (!VEC) return load(p, first, v);
    const char* row = static_cast<const char*>(p) + first * B;
#pragma unroll
    for (int i = 0; i < N; i += G) {
      Acc<E> a;
      const int left = cols - at(i);
      a.set(left >= G   ? *reinterpret_cast<const uint4*>(row + at(i) * B)
            : left > 0 ? load_group<E>(row, at(i) / G, left, false)
                       : make_uint4(0, 0, 0, 0));
#pragma unroll
      for (int k = 0; k < G; ++k) v[i + k] = a.v[k];
    }
  }
  __device__ __forceinline__ void store(void* p, int64_t first, const float (&v)[N]) const {
    char* row = static_cast<char*>(p) + first * B;
    if (VEC) {
#pragma unroll
      for (int i = 0; i < N; i += G) {
        Acc<E> a;
#pragma unroll
        for (int k = 0; k < G; ++k) a.v[k] = v[i + k];
        if (at(i) < cols) store_group<E>(row, at(i) / G, a.round(), min(cols - at(i), G), true);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (has(i)) st_elem<B>(row + (int64_t)at(i) * B, E::from_f32(v[i]));
    }
  }
};

__device__ __forceinline__ void copy_async16(uint32_t to, const char* from, int bytes) {  // the rest of the 16 is zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

// Whether a vector, or every row of a matrix, starts on 16 bytes; absent ones do.
bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
template <class E>
bool on16(const void* p, int64_t ld, int64_t rows) {
  return !p || (on16(p) && (rows == 1 || ld % E::kGroup == 0));
}

}  // namespace
}  // namespace ar
