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

// How a kernel finds its rows.  kAligned: every row and vector starts on 16 bytes.  kShifted: a piece of 16 bytes is
// read as the two aligned ones around it, shifted into place, and written as the aligned one that
// it begins in, with the end of the neighbouring lane's piece before it.  kElements: one by one,
// neighbouring threads having neighbouring elements.
enum Layout { kAligned, kShifted, kElements };

// The columns of thread t of the T that share a row, N of them, 16 bytes at a time (kElements: one).
template <class E, int N, Layout L>
struct Columns {
  static constexpr int G = E::kGroup, B = E::kBytes;
  static constexpr bool VEC = L == kAligned;
  int t, T, cols;

  __device__ __forceinline__ int at(int i) const { return L == kElements ? t + i * T : (t + i / G * T) * G + i % G; }
  __device__ __forceinline__ bool has(int i) const { return at(i) < cols; }
  static __device__ __forceinline__ void put(uint4 x, float* v) {
    Acc<E> a;
    a.set(x);
#pragma unroll
    for (int k = 0; k < G; ++k) v[k] = a.v[k];
  }
  static __device__ __forceinline__ uint4 get(const float* v) {
    Acc<E> a;
#pragma unroll
    for (int k = 0; k < G; ++k) a.v[k] = v[k];
    return a.round();
  }
  // The row that begins at element `first` of a matrix of `extent` elements; columns past the last are 0.
  __device__ __forceinline__ void load(const void* p, int64_t first, int64_t extent, float (&v)[N]) const {
    const char *begin = static_cast<const char*>(p), *row = begin + first * B;
    if (L == kElements) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = has(i) ? E::to_f32(ld_elem<B>(row + (int64_t)at(i) * B)) : 0.0f;
      return;
    }
#pragma unroll
    for (int i = 0; i < N; i += G) {
      const int left = cols - at(i);
      uint4 x = make_uint4(0, 0, 0, 0);
      if (VEC) {
        if (left > 0) x = load_group<E>(row, at(i) / G, min(left, G), true);
      } else {
        x = load_anywhere<B>(row + (int64_t)at(i) * B, left * B, begin, begin + extent * B);
      }
      put(x, v + i);
    }
  }
  // The same of what other rows' threads read too.
  __device__ __forceinline__ void load_shared(const void* p, int64_t first, int64_t extent, float (&v)[N]) const {
    if (L == kElements) return load(p, first, extent, v);
    const char *begin = static_cast<const char*>(p), *row = begin + first * B;
#pragma unroll
    for (int i = 0; i < N; i += G) {
      const int left = cols - at(i);
      uint4 x = make_uint4(0, 0, 0, 0);
      if (!VEC)
        x = load_anywhere<B>(row + (int64_t)at(i) * B, left * B, begin, begin + extent * B);
      else if (left >= G)
        x = *reinterpret_cast<const uint4*>(row + at(i) * B);
      else if (left > 0)
        x = load_group<E>(row, at(i) / G, left, false);
      put(x, v + i);
    }
  }
  // All lanes of a warp together.
  __device__ __forceinline__ void store(void* p, int64_t first, const float (&v)[N]) const {
    char* row = static_cast<char*>(p) + first * B;
    if (L == kElements) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (has(i)) st_elem<B>(row + (int64_t)at(i) * B, E::from_f32(v[i]));
      return;
    }
    const uint32_t o = VEC ? 0 : (uint32_t)(reinterpret_cast<uintptr_t>(row) & 15u);
#pragma unroll
    for (int i = 0; i < N; i += G) {
      const uint4 x = get(v + i);
      const int left = cols - at(i);
      char* to = row + (int64_t)at(i) * B;
      if (o == 0) {
        if (left >= G)
          st_v4_stream(to, x);
        else if (left > 0)
          store_group<E>(to, 0, x, left, false);
        continue;
      }
      const int lane = threadIdx.x & 31, head = (16 - (int)o) / B;  // elements before the next multiple of 16
      uint4 before;
      before.x = __shfl_up_sync(0xFFFFFFFFu, x.x, 1), before.y = __shfl_up_sync(0xFFFFFFFFu, x.y, 1);
      before.z = __shfl_up_sync(0xFFFFFFFFu, x.z, 1), before.w = __shfl_up_sync(0xFFFFFFFFu, x.w, 1);
      const bool joined = lane > 0 && left >= head, next_joined = lane < 31 && left - G >= head;
      if (joined) st_v4_stream(to - o, shift_window(before, x, 16 - o));
      if (!joined || !next_joined) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int k = 0; k < G; ++k)
          if (k < left && (k < head ? !joined : !next_joined)) st_elem<B>(to + k * B, B == 4 ? w[k & 3] : w[k / 2] >> (16 * (k & 1)));
      }
    }
  }
};

__device__ __forceinline__ void copy_async16(uint32_t to, const char* from, int bytes) {  // the rest of the 16 is zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

// A row on its way through shared memory, in pieces of 16 bytes, one behind the other.  VEC: a thread copies
// the pieces that it will read.  Else the row begins somewhere in the first piece, and what a thread reads lies in
// pieces that its neighbours copied: the threads that share the row meet between waiting for their copies
// and reading.
template <class E, int N, bool VEC>
struct Staged {
  static constexpr int G = E::kGroup, B = E::kBytes, kPieces = N / G;
  Columns<E, N, VEC ? kAligned : kShifted> c;

  static __host__ __device__ constexpr int bytes(int T) { return (T * kPieces + (VEC ? 0 : 1)) * 16; }

  // The row at `row` of a matrix between begin and end, to shared memory at `to`.
  __device__ __forceinline__ void fetch(uint32_t to, const char* row, const char* begin, const char* end) const {
    if (VEC) {
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        const int at = c.at(p * G) * B, left = min(max(c.cols * B - at, 0), 16);
        copy_async16(to + (c.t + p * c.T) * 16, left ? row + at : row, left);
      }
    } else {
      const int o = (int)(reinterpret_cast<uintptr_t>(row) & 15u), total = o + c.cols * B;
      const char* base = row - o;
#pragma unroll
      for (int p = 0; p <= kPieces; ++p) {
        const int piece = c.t + p * c.T;
        if (piece * 16 >= total || (p == kPieces && c.t > 0)) continue;
        const char* from = base + piece * 16;
        if (from >= begin) {
          copy_async16(to + piece * 16, from, (int)min(end - from, (int64_t)16));
        } else {  // the matrix begins inside this piece
          for (int k = o; k < 16 && k < total; k += B) {
            const uint32_t v = ld_elem<B>(from + k);
            if (B == 2)
              asm volatile("st.shared.u16 [%0], %1;" ::"r"(to + piece * 16 + k), "h"((unsigned short)v) : "memory");
            else
              asm volatile("st.shared.u32 [%0], %1;" ::"r"(to + piece * 16 + k), "r"(v) : "memory");
          }
        }
      }
    }
  }
  static __device__ __forceinline__ uint4 piece(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
  }
  // This thread's columns of the row that was copied to `from`; o: where it begins in its first piece.
  __device__ __forceinline__ void read(uint32_t from, int o, float (&v)[N]) const {
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
      const uint32_t at = from + (c.t + p * c.T) * 16;
      const int left = c.cols - c.at(p * G);
      uint4 x;
      if (VEC) {
        x = piece(at);  // what the copy did not bring is zeros
      } else {
        x = make_uint4(0, 0, 0, 0);
        if (left > 0) x = o ? shift_window(piece(at), piece(at + 16), (uint32_t)o) : piece(at);
        if (left > 0 && left < G) {
          uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int there = left * B - 4 * i;
            w[i] = there >= 4 ? w[i] : there == 2 ? w[i] & 0xFFFFu : 0;
          }
          x = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      c.put(x, v + p * G);
    }
  }
};

// Whether a vector, or every row of a matrix, starts on 16 bytes; absent ones do.
bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
template <class E>
bool on16(const void* p, int64_t ld, int64_t rows) {
  return !p || (on16(p) && (rows == 1 || ld % E::kGroup == 0));
}

}  // namespace
}  // namespace ar
