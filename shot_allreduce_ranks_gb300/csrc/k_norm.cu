// Norms before and after a block with its gate and the residual, and their
// gradients (formulas in include/ar.h).
#include <stdlib.h>

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

// Any row: a CTA a row, which it reads again for every statistic.
template <class E>
__global__ void __launch_bounds__(kAnyThreads) k_norm_any(NormArgs a) {
  __shared__ float room[4][32];
  pdl_enter();
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const int64_t gate = a.gate ? row / a.gate_run * a.ldg : 0;
    Stats sx = {0.0f, 1.0f}, sr = {0.0f, 1.0f};
    const auto x = [&](int64_t c) { return value<E>(a.x, row * a.ldx + c); };
    if (a.after_weight) sx = stats_any(x, a.cols, a.layer, a.eps, room);
    const auto r = [&](int64_t c) {
      float z = x(c);
      if (a.after_weight) {
        z = (z - sx.mean) * sx.factor * (a.offset + value<E>(a.after_weight, c));
        if (a.after_bias) z += value<E>(a.after_bias, c);
      }
      if (a.gate) z *= value<E>(a.gate, gate + c);
      return a.residual ? __fmaf_rn(a.alpha, value<E>(a.residual, row * a.ldres + c), z) : z;
    };
    if (a.weight) sr = stats_any(r, a.cols, a.layer, a.eps, room + 2);
    for (int64_t c = threadIdx.x; c < a.cols; c += kAnyThreads) {
      const float v = r(c);
      if (a.r) put<E>(a.r, row * a.ldr + c, v);
      if (a.weight) {
        float y = (v - sr.mean) * sr.factor * (a.offset + value<E>(a.weight, c));
        if (a.bias) y += value<E>(a.bias, c);
        put<E>(a.y, row * a.ldy + c, y);
      }
    }
    __syncthreads();
  }
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

template <int N, bool WARP>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*room)[32]) {
  if (!WARP) {
    cta_sums<N>(v, room);
    return;
  }
#pragma unroll
  for (int k = 0; k < N; ++k)
#pragma unroll
    for (int o = 16; o; o >>= 1) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], o);
}

// The row in v: its statistics; room holds two rows.
template <bool WARP, class C, int N>
__device__ __forceinline__ Stats stats_of(const C& c, const float (&v)[N], int layer, float eps, float (*room)[32]) {
  Stats s = {0.0f, 0.0f};
  float sum[1];
  if (layer) {
    sum[0] = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) sum[0] += v[i];
    row_sums<1, WARP>(sum, room);
    s.mean = sum[0] / (float)c.cols;
  }
  sum[0] = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float d = layer ? (c.has(i) ? v[i] - s.mean : 0.0f) : v[i];
    sum[0] = __fmaf_rn(d, d, sum[0]);
  }
  row_sums<1, WARP>(sum, room + 1);
  s.factor = 1.0f / sqrtf(sum[0] / (float)c.cols + eps);
  return s;
}

// One row, x in v and the residual in q: r and y are stored.  room holds four rows.
template <class E, int N, bool VEC, bool WARP>
__device__ __forceinline__ void norm_row(const NormArgs& a, const Columns<E, N, VEC>& c, int64_t row, float (&v)[N], const float (&q)[N],
                                         float (*room)[32]) {
  float w[N];
  if (a.after_weight) {
    c.load_shared(a.after_weight, 0, w);
    const Stats s = stats_of<WARP>(c, v, a.layer, a.eps, room);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = (v[i] - s.mean) * s.factor * (a.offset + w[i]);
    if (a.after_bias) {
      c.load_shared(a.after_bias, 0, w);
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += w[i];
    }
  }
  if (a.gate) {
    c.load_shared(a.gate, row / a.gate_run * a.ldg, w);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] *= w[i];
  }
  if (a.residual) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __fmaf_rn(a.alpha, q[i], v[i]);
  }
  if (a.weight) c.load_shared(a.weight, 0, w);
  if (a.r) c.store(a.r, row * a.ldr, v);
  if (!a.weight) return;
  // Columns past the last hold what biases left there, which the norm must not see.
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = c.has(i) ? v[i] : 0.0f;
  const Stats s = stats_of<WARP>(c, v, a.layer, a.eps, room + 2);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = (v[i] - s.mean) * s.factor * (a.offset + w[i]);
  if (a.bias) {
    c.load_shared(a.bias, 0, w);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += w[i];
  }
  c.store(a.y, row * a.ldy, v);
}

// A row a CTA, or (WARP) a row a warp, read once and held in registers, N columns a thread.
template <class E, int N, bool VEC, bool WARP>
__global__ void __launch_bounds__(1024) k_norm_rows(NormArgs a) {
  __shared__ float room[4][32];
  pdl_enter();
  const int64_t row = WARP ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
  if (WARP && row >= a.rows) return;
  const Columns<E, N, VEC> c = {WARP ? (int)(threadIdx.x & 31) : (int)threadIdx.x, WARP ? 32 : (int)blockDim.x, (int)a.cols};
  float v[N], q[N];
  c.load(a.x, row * a.ldx, v);
  if (a.residual) c.load(a.residual, row * a.ldres, q);
  norm_row<E, N, VEC, WARP>(a, c, row, v, q, room);
}

__device__ __forceinline__ void copy_async16(uint32_t to, const char* from, int bytes) {  // the rest of the 16 is zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

// Many rows: a CTA (or warp) takes every gridDim-th and copies the next ones into shared
// memory meanwhile, kStages - 1 of them; a thread copies what it will read itself, so only its own
// copies have to be waited for.
constexpr int kStages = 3;
template <class E, int N, bool WARP>
__global__ void __launch_bounds__(1024) k_norm_stream(NormArgs a) {
  extern __shared__ __align__(16) char smem[];
  __shared__ float room[8][32];
  constexpr int G = E::kGroup, kPieces = N / G;
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const Columns<E, N, true> c = {WARP ? lane : (int)threadIdx.x, WARP ? 32 : (int)blockDim.x, (int)a.cols};
  const int64_t first = WARP ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
  const int64_t step = WARP ? (int64_t)gridDim.x * (blockDim.x >> 5) : (int64_t)gridDim.x;
  // Piece p of matrix m of a stage, one thread's after the other's.
  const auto slot = [&](int stage, int m, int p) {
    return smem + (((stage * 2 + m) * kPieces + p) * (int)blockDim.x + (int)threadIdx.x) * 16;
  };
  const auto fetch = [&](int64_t row, int stage) {
    if (row < a.rows) {
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        if (m == 1 && !a.residual) continue;
        const char* from = static_cast<const char*>(m ? a.residual : a.x) + row * (m ? a.ldres : a.ldx) * E::kBytes;
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
          const int at = c.at(p * G), left = min(max(c.cols - at, 0), G) * E::kBytes;
          copy_async16((uint32_t)__cvta_generic_to_shared(slot(stage, m, p)), from + (left ? at * E::kBytes : 0), left);
        }
      }
    }
    copies_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(first + i * step, i);
  int stage = 0, parity = 0;
  for (int64_t row = first; row < a.rows; row += step) {
    fetch(row + (kStages - 1) * step, stage == 0 ? kStages - 1 : stage - 1);
    copies_wait<kStages - 1>();
    float v[N], q[N];
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
      Acc<E> x, y;
      x.set(*reinterpret_cast<const uint4*>(slot(stage, 0, p)));
      if (a.residual) y.set(*reinterpret_cast<const uint4*>(slot(stage, 1, p)));
#pragma unroll
      for (int k = 0; k < G; ++k) {
        v[p * G + k] = x.v[k];
        q[p * G + k] = a.residual ? y.v[k] : 0.0f;
      }
    }
    // The next row's sums go to the other half of the room: a warp may be a row ahead.
    norm_row<E, N, true, WARP>(a, c, row, v, q, room + 4 * parity);
    parity ^= 1;
    stage = stage == kStages - 1 ? 0 : stage + 1;
  }
}

// The rows of a CTA, all of one gate row where split > 0.
__device__ __forceinline__ void rows_of(const NormGradArgs& a, int64_t cta, int64_t& first, int64_t& last) {
  if (a.split) {
    const int64_t g = cta / a.split, j = cta % a.split;
    first = g * a.gate_run + min(j * a.chunk, a.gate_run);
    last = g * a.gate_run + min((j + 1) * a.chunk, a.gate_run);
  } else {
    first = cta * a.gate_rows / a.ctas * a.gate_run;
    last = (cta + 1) * a.gate_rows / a.ctas * a.gate_run;
  }
}

// Any row: a CTA takes its rows one after the other, reads each again for every
// statistic and adds to its own row of the parts, a thread to its own columns.
template <class E>
__global__ void __launch_bounds__(kAnyThreads) k_norm_grad_any(NormGradArgs a) {
  __shared__ float room[8][32];
  pdl_enter();
  const int64_t cta = blockIdx.x;
  int64_t first, last;
  rows_of(a, cta, first, last);
  const auto add = [&](int k, int64_t c, bool start, float v) {
    float* p = a.part[k] + cta * a.cols + c;
    *p = start ? v : *p + v;
  };
  for (int64_t row = first; row < last; ++row) {
    const int64_t gate_row = row / a.gate_run;
    Stats sr = {0.0f, 1.0f}, sx = {0.0f, 1.0f};
    float m[2] = {0.0f, 0.0f};  // means of d and d * N(r), d the gradient of N(r)
    const auto r_hat = [&](int64_t c) { return (value<E>(a.r, row * a.ldr + c) - sr.mean) * sr.factor; };
    const auto d_hat = [&](int64_t c) { return value<E>(a.dy, row * a.lddy + c) * (a.offset + value<E>(a.weight, c)); };
    if (a.weight) {
      sr = stats_any([&](int64_t c) { return value<E>(a.r, row * a.ldr + c); }, a.cols, a.layer, a.eps, room);
      for (int64_t c = threadIdx.x; c < a.cols; c += kAnyThreads) {
        const float d = d_hat(c);
        m[0] += d;
        m[1] = __fmaf_rn(d, r_hat(c), m[1]);
      }
      cta_sums<2>(m, room + 2);
      m[0] = a.layer ? m[0] / (float)a.cols : 0.0f;
      m[1] /= (float)a.cols;
    }
    const auto g = [&](int64_t c) {
      float v = a.dr ? value<E>(a.dr, row * a.lddr + c) : 0.0f;
      if (a.weight) v = __fmaf_rn(sr.factor, d_hat(c) - m[0] - r_hat(c) * m[1], v);
      return v;
    };
    const auto x_hat = [&](int64_t c) { return (value<E>(a.x, row * a.ldx + c) - sx.mean) * sx.factor; };
    const auto dz = [&](int64_t c) { return a.gate ? g(c) * value<E>(a.gate, gate_row * a.ldg + c) : g(c); };
    float n[2] = {0.0f, 0.0f};  // likewise of the norm after the block
    if (a.after_weight) {
      sx = stats_any([&](int64_t c) { return value<E>(a.x, row * a.ldx + c); }, a.cols, a.layer, a.eps, room + 4);
      for (int64_t c = threadIdx.x; c < a.cols; c += kAnyThreads) {
        const float d = dz(c) * (a.offset + value<E>(a.after_weight, c));
        n[0] += d;
        n[1] = __fmaf_rn(d, x_hat(c), n[1]);
      }
      cta_sums<2>(n, room + 6);
      n[0] = a.layer ? n[0] / (float)a.cols : 0.0f;
      n[1] /= (float)a.cols;
    }
    const bool gate_done = a.split == 0 && (row + 1) % a.gate_run == 0;
    for (int64_t c = threadIdx.x; c < a.cols; c += kAnyThreads) {
      const float gv = g(c), dzv = dz(c), hat = a.after_weight ? x_hat(c) : 0.0f;
      if (a.sum[kSumWeight]) add(kSumWeight, c, row == first, value<E>(a.dy, row * a.lddy + c) * r_hat(c));
      if (a.sum[kSumBias]) add(kSumBias, c, row == first, value<E>(a.dy, row * a.lddy + c));
      if (a.sum[kSumAfterWeight]) add(kSumAfterWeight, c, row == first, dzv * hat);
      if (a.sum[kSumAfterBias]) add(kSumAfterBias, c, row == first, dzv);
      if (a.sum[kSumGate]) {
        float z = a.after_weight ? hat * (a.offset + value<E>(a.after_weight, c)) : value<E>(a.x, row * a.ldx + c);
        if (a.after_bias) z += value<E>(a.after_bias, c);
        add(kSumGate, c, row % a.gate_run == 0 || row == first, gv * z);
        if (gate_done) put<E>(a.sum[kSumGate], gate_row * a.lddg + c, a.part[kSumGate][cta * a.cols + c]);
      }
      if (a.dresidual) put<E>(a.dresidual, row * a.lddres + c, a.alpha * gv);
      if (a.dx)
        put<E>(a.dx, row * a.lddx + c,
               a.after_weight ? sx.factor * (dzv * (a.offset + value<E>(a.after_weight, c)) - n[0] - hat * n[1]) : dzv);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Gradients of rows that T threads hold in registers and shared memory.
//
// The columns' sums over rows stay in a thread's registers while its CTA walks
// its rows; a CTA of short rows has several groups of T threads, each with rows of
// its own.  A row's statistics and the two means that the gradient wants come out of one
// joint sum (mean square) or two (differences from the mean), and one more for the norm
// after the block.  VEC: the next row is copied to shared memory meanwhile; a
// thread reads what it copied itself.
constexpr int kGroupThreads = 256;  // of a CTA of short rows

__host__ __device__ constexpr int row_threads(int64_t cols, int n) { return (int)((cols + 32 * n - 1) / (32 * n) * 32); }
__host__ __device__ constexpr int row_groups(int threads) { return threads < kGroupThreads ? kGroupThreads / threads : 1; }

// Sums of up to four values over a warp: at the first steps a lane gives away the
// values that its half (or quarter) does not finish, so that N values cost about
// as many shuffles as one (the SM does one of them a clock).  Lane 32 / P * k
// and the ones after it end with value k, P = N rounded up to a power of two.
template <int N>
__device__ __forceinline__ float spread_sums(const float (&v)[N], int lane) {
  constexpr int P = N == 1 ? 1 : N == 2 ? 2 : 4;
  float a = v[0];
  if (P == 2) {
    const bool high = lane & 16;
    a = (high ? v[N > 1 ? 1 : 0] : v[0]) + __shfl_xor_sync(0xFFFFFFFFu, high ? v[0] : v[N > 1 ? 1 : 0], 16);
  }
  if (P == 4) {
    const bool high = lane & 16, odd = lane & 8;
    const float v1 = v[N > 1 ? 1 : 0], v2 = v[N > 2 ? 2 : 0], v3 = N > 3 ? v[N - 1] : 0.0f;
    const float b0 = (high ? v2 : v[0]) + __shfl_xor_sync(0xFFFFFFFFu, high ? v[0] : v2, 16);
    const float b1 = (high ? v3 : v1) + __shfl_xor_sync(0xFFFFFFFFu, high ? v1 : v3, 16);
    a = (odd ? b1 : b0) + __shfl_xor_sync(0xFFFFFFFFu, odd ? b0 : b1, 8);
  }
#pragma unroll
  for (int o = 16 / P; o; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
  return a;
}

// Sums over the T threads of a group, which has its own barrier; room: a row of 32 for each value.
template <int N>
__device__ __forceinline__ void group_sums(float (&v)[N], float (*room)[32], int group, int T) {
  constexpr int P = N == 1 ? 1 : N == 2 ? 2 : 4, kSpan = 32 / P;
  const int lane = threadIdx.x & 31, k = lane / kSpan, in = lane % kSpan;
  float a = spread_sums<N>(v, lane);
  if (T > 32) {
    const int warp = (threadIdx.x >> 5) - group * (T >> 5), warps = T >> 5;
    if (in == 0 && k < N) room[k][warp] = a;
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(T) : "memory");
    a = 0.0f;
    if (k < N) {
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (in + kSpan * i < warps) a += room[k][in + kSpan * i];
    }
#pragma unroll
    for (int o = kSpan / 2; o; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = P == 1 ? a : __shfl_sync(0xFFFFFFFFu, a, kSpan * i);
}

enum { kDy = 0, kDr, kR, kX };  // the matrices that are read

// FULL: a norm after the block or a gate; BIAS: dbias is wanted (FULL has it always).
template <class E, int N, int MAXT, int MINB, bool VEC, bool LAYER, bool FULL, bool BIAS>
__global__ void __launch_bounds__(MAXT, MINB) k_norm_grad_rows(NormGradArgs a, int T, int stages) {
  constexpr int G = E::kGroup, kPieces = N / G, kMats = FULL ? 4 : 3;
  extern __shared__ __align__(16) char smem[];
  __shared__ float rooms[MAXT > kGroupThreads ? 1 : 4][2][8][32];  // groups of one warp use none
  pdl_enter();
  const int groups = (int)blockDim.x / T, group = (int)threadIdx.x / T;
  const Columns<E, N, VEC> c = {(int)threadIdx.x - group * T, T, (int)a.cols};
  const float inv = 1.0f / (float)a.cols;
  int64_t first, last, step;
  if (a.split) {
    rows_of(a, blockIdx.x, first, last);
    first += group, step = groups;
  } else {
    const int64_t unit = (int64_t)blockIdx.x * groups + group, units = a.ctas * groups;
    first = unit * a.gate_rows / units * a.gate_run, last = (unit + 1) * a.gate_rows / units * a.gate_run, step = 1;
  }
  const void* const mats[4] = {a.dy, a.dr, a.weight ? a.r : nullptr, FULL ? a.x : nullptr};
  const int64_t lds[4] = {a.lddy, a.lddr, a.ldr, a.ldx};
  const auto slot = [&](int stage, int m, int p) {
    return smem + (((stage * kMats + m) * kPieces + p) * (int)blockDim.x + (int)threadIdx.x) * 16;
  };
  const auto fetch = [&](int64_t row, int stage) {
    if (row < last) {
#pragma unroll
      for (int m = 0; m < kMats; ++m) {
        if (!mats[m]) continue;
        const char* from = static_cast<const char*>(mats[m]) + row * lds[m] * E::kBytes;
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
          const int at = c.at(p * G), left = min(max(c.cols - at, 0), G) * E::kBytes;
          copy_async16((uint32_t)__cvta_generic_to_shared(slot(stage, m, p)), from + (left ? at * E::kBytes : 0), left);
        }
      }
    }
    copies_commit();
  };
  // The row's part of matrix m in v.
  const auto get = [&](int m, int64_t row, int stage, float(&v)[N]) {
    if (VEC) {
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        Acc<E> x;
        x.set(*reinterpret_cast<const uint4*>(slot(stage, m, p)));
#pragma unroll
        for (int k = 0; k < G; ++k) v[p * G + k] = x.v[k];
      }
    } else {
      c.load(mats[m], row * lds[m], v);
    }
  };

  float dw[N] = {}, db[BIAS ? N : 1] = {}, daw[FULL ? N : 1] = {}, dab[FULL ? N : 1] = {}, dgate[FULL ? N : 1] = {};
  if (VEC)
    for (int i = 0; i < stages - 1; ++i) fetch(first + i * step, i);
  int stage = 0, parity = 0;
  for (int64_t row = first; row < last; row += step) {
    if (VEC) {
      const int to = stage == 0 ? stages - 1 : stage - 1;
      fetch(row + (stages - 1) * step, to);
      if (stages == 4)
        copies_wait<3>();
      else if (stages == 3)
        copies_wait<2>();
      else if (stages == 2)
        copies_wait<1>();
      else
        copies_wait<0>();
    }
    float(*room)[32] = rooms[group][parity];
    float r[N], d[N], w[N];
    float rmean = 0.0f, rfactor = 1.0f, xmean = 0.0f, xfactor = 1.0f, m0 = 0.0f, m1 = 0.0f;
    if (a.weight) {
      c.load_shared(a.weight, 0, w);
      get(kR, row, stage, r);
      get(kDy, row, stage, d);
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] += a.offset;  // past the last column d is 0
    }
    float x[FULL ? N : 1];
    if constexpr (FULL) get(kX, row, stage, x);
    // Two sums of the norm before the next block, and one of that after this one.
    constexpr int kSums = FULL ? 3 : 2;
    const auto centred = [&](float v, float mean, int i) { return LAYER ? (c.has(i) ? v - mean : 0.0f) : v; };
    if (LAYER) {
      float s[kSums] = {};
      if (a.weight) {
#pragma unroll
        for (int i = 0; i < N; ++i) s[0] += r[i], s[1] = __fmaf_rn(d[i], w[i], s[1]);
      }
      if constexpr (FULL) {
#pragma unroll
        for (int i = 0; i < N; ++i) s[2] += x[i];
        group_sums<kSums>(s, room, group, T);
        xmean = s[2] * inv;
      } else {
        group_sums<kSums>(s, room, group, T);
      }
      rmean = s[0] * inv, m0 = s[1] * inv;
    }
    {
      float s[kSums] = {};
      if (a.weight) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float v = centred(r[i], rmean, i);
          s[0] = __fmaf_rn(v, v, s[0]);
          s[1] = __fmaf_rn(d[i] * w[i], v, s[1]);
        }
      }
      if constexpr (FULL) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float v = centred(x[i], xmean, i);
          s[2] = __fmaf_rn(v, v, s[2]);
        }
      }
      group_sums<kSums>(s, room + 3, group, T);
      if (a.weight) {
        rfactor = 1.0f / sqrtf(s[0] * inv + a.eps);
        m1 = s[1] * inv * rfactor;
      }
      if constexpr (FULL) {
        if (a.after_weight) xfactor = 1.0f / sqrtf(s[2] * inv + a.eps);
      }
    }
    float g[N];
    if (a.dr) {
      get(kDr, row, stage, g);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) g[i] = 0.0f;
    }
    if (a.weight) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float hat = (LAYER ? r[i] - rmean : r[i]) * rfactor, t = LAYER ? __fmaf_rn(d[i], w[i], -m0) : d[i] * w[i];
        g[i] = __fmaf_rn(rfactor, __fmaf_rn(-hat, m1, t), g[i]);
        dw[i] = __fmaf_rn(d[i], hat, dw[i]);
        if constexpr (BIAS) db[i] += d[i];
      }
    }
    if (a.dresidual) {
#pragma unroll
      for (int i = 0; i < N; ++i) r[i] = a.alpha * g[i];
      c.store(a.dresidual, row * a.lddres, r);
    }
    if constexpr (FULL) {
      const int64_t gate_row = row / a.gate_run;
      if (a.gate) {
        c.load_shared(a.gate, gate_row * a.ldg, w);
        float ab[N];
        if (a.after_weight) {
          c.load_shared(a.after_weight, 0, d);
          if (a.after_bias) c.load_shared(a.after_bias, 0, ab);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
          float z = x[i];
          if (a.after_weight) {
            z = (LAYER ? x[i] - xmean : x[i]) * xfactor * (a.offset + d[i]);
            if (a.after_bias) z += ab[i];
          }
          dgate[i] = __fmaf_rn(g[i], z, dgate[i]);
          g[i] *= w[i];
        }
        if (!a.split && (row + 1) % a.gate_run == 0) {
          if (a.sum[kSumGate]) c.store(a.sum[kSumGate], gate_row * a.lddg, dgate);
#pragma unroll
          for (int i = 0; i < N; ++i) dgate[i] = 0.0f;
        }
      }
      if (a.after_weight) {
        c.load_shared(a.after_weight, 0, w);
        float s[2] = {};
#pragma unroll
        for (int i = 0; i < N; ++i) {
          w[i] += a.offset;
          const float hat = centred(x[i], xmean, i) * xfactor;
          daw[i] = __fmaf_rn(g[i], hat, daw[i]);
          dab[i] += g[i];
          if (LAYER) s[0] += c.has(i) ? g[i] * w[i] : 0.0f;
          s[1] = __fmaf_rn(g[i] * w[i], hat, s[1]);
        }
        group_sums<2>(s, room + 6, group, T);
        const float n0 = LAYER ? s[0] * inv : 0.0f, n1 = s[1] * inv;
#pragma unroll
        for (int i = 0; i < N; ++i) g[i] = xfactor * __fmaf_rn(LAYER ? xmean - x[i] : -x[i], xfactor * n1, LAYER ? __fmaf_rn(g[i], w[i], -n0) : g[i] * w[i]);
      }
    }
    if (a.dx) c.store(a.dx, row * a.lddx, g);
    parity ^= 1;
    stage = stage == stages - 1 ? 0 : stage + 1;
  }

  // The groups' sums are joined in their order, through shared memory, and stored as the CTA's part.
  if (VEC) copies_wait<0>();
  float* sum = reinterpret_cast<float*>(smem);
  const auto finish = [&](int k, const float(&v)[N]) {
    if (!a.sum[k] || (k == kSumGate && !a.split)) return;
    for (int q = 0; q < groups; ++q) {
      if (groups > 1) __syncthreads();
      if (q != group) continue;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (!c.has(i)) continue;
        const float t = q ? sum[c.at(i)] + v[i] : v[i];
        if (q == groups - 1)
          a.part[k][(int64_t)blockIdx.x * a.cols + c.at(i)] = t;
        else
          sum[c.at(i)] = t;
      }
    }
  };
  finish(kSumWeight, dw);
  if constexpr (BIAS) finish(kSumBias, db);
  if constexpr (FULL) {
    finish(kSumAfterWeight, daw);
    finish(kSumAfterBias, dab);
    finish(kSumGate, dgate);
  }
}

// The CTAs' parts joined: output row blockIdx.z of sum blockIdx.y.  32 columns a
// CTA; its warps take turns at the parts and are joined in their order.
struct JoinArgs {
  const float* part[kNormSums];
  void* sum[kNormSums];
  int64_t count[kNormSums], rows[kNormSums], ld[kNormSums];  // parts of an output row; output rows
  int64_t cols;
};
constexpr int kJoinWarps = 8;

template <class E>
__global__ void __launch_bounds__(32 * kJoinWarps) k_norm_join(JoinArgs a) {
  __shared__ float room[kJoinWarps][32];
  pdl_enter();
  const int k = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = blockIdx.z, c = (int64_t)blockIdx.x * 32 + lane;
  if (row >= a.rows[k]) return;
  const float* p = a.part[k] + row * a.count[k] * a.cols;
  float v = 0.0f;
  if (c < a.cols) {
#pragma unroll 8
    for (int64_t i = warp; i < a.count[k]; i += kJoinWarps) v += p[i * a.cols + c];
  }
  room[warp][lane] = v;
  __syncthreads();
  if (warp || c >= a.cols) return;
  v = 0.0f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) v += room[w][lane];
  put<E>(a.sum[k], row * a.ld[k] + c, v);
}

// Whether a vector, or every row of a matrix, starts on 16 bytes; absent ones do.
bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
template <class E>
bool on16(const void* p, int64_t ld, int64_t rows) {
  return !p || (on16(p) && (rows == 1 || ld % E::kGroup == 0));
}

template <class E, int N, bool VEC>
cudaError_t norm_rows(const NormArgs& a, cudaStream_t s) {
  const int64_t threads = (a.cols + 32 * N - 1) / (32 * N) * 32;
  if (threads == 32) {
    const int64_t grid = (a.rows + 3) / 4;
    return launch_op(k_norm_rows<E, N, VEC, true>, dim3((unsigned)grid), 128, 0, 1, s, a);
  }
  return launch_op(k_norm_rows<E, N, VEC, false>, dim3((unsigned)a.rows), (int)threads, 0, 1, s, a);
}

template <class E>
cudaError_t norm(const NormArgs& a, int num_sms, cudaStream_t s) {
  const bool vec = on16<E>(a.x, a.ldx, a.rows) && on16<E>(a.residual, a.ldres, a.rows) && on16<E>(a.r, a.ldr, a.rows) &&
                   on16<E>(a.y, a.ldy, a.rows) && on16<E>(a.gate, a.ldg, a.rows / a.gate_run) && on16(a.after_weight) &&
                   on16(a.after_bias) && on16(a.weight) && on16(a.bias);
  static const int force = getenv("NORM_N") ? atoi(getenv("NORM_N")) : 0;
  static const int stream = getenv("NORM_S") ? atoi(getenv("NORM_S")) : 0;
  constexpr int NS = 2 * E::kGroup;
  if (stream && vec && a.cols <= 1024 * NS) {
    const int64_t threads = (a.cols + 32 * NS - 1) / (32 * NS) * 32;
    const int cta = threads == 32 ? 128 : (int)threads, rows = threads == 32 ? 4 : 1;
    const size_t smem = (size_t)kStages * 2 * 32 * cta;
    int64_t per_sm = 1024 / cta;
    const int64_t grid = (a.rows + rows - 1) / rows;
    auto* k = threads == 32 ? k_norm_stream<E, NS, true> : k_norm_stream<E, NS, false>;
    cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    return launch_op(k, dim3((unsigned)(grid < per_sm * num_sms ? grid : per_sm * num_sms)), cta, smem, 1, s, a);
  }
  const bool wide = force ? force == 16 : a.cols > 8192;
  if (a.cols <= 16384 && a.rows <= 0x7FFFFFFF) {
    if (wide) return vec ? norm_rows<E, 16, true>(a, s) : norm_rows<E, 16, false>(a, s);
    return vec ? norm_rows<E, 8, true>(a, s) : norm_rows<E, 8, false>(a, s);
  }
  const int64_t most = (int64_t)num_sms * 8;
  return launch_op(k_norm_any<E>, dim3((unsigned)(a.rows < most ? a.rows : most)), kAnyThreads, 0, 1, s, a);
}

// The rows dealt out to at most `want` CTAs: where there are fewer gate rows each is
// split among as many CTAs; where there are more, a CTA takes several whole ones.
void deal(NormGradArgs& a, int64_t want) {
  if (a.gate_rows <= want) {
    const int64_t parts = want / a.gate_rows;
    a.chunk = (a.gate_run + parts - 1) / parts;
    a.split = (a.gate_run + a.chunk - 1) / a.chunk;
    a.ctas = a.gate_rows * a.split;
  } else {
    a.split = a.chunk = 0;
    a.ctas = want;
  }
}

template <class E, int N, bool VEC, bool LAYER, bool FULL, bool BIAS>
cudaError_t norm_grad_rows_kind(NormGradArgs& a, int num_sms, cudaStream_t s) {
  constexpr int kMats = FULL ? 4 : 3;
  const int T = row_threads(a.cols, N), cta = T < kGroupThreads ? T * row_groups(T) : T;
  // 64 registers a thread, or 128 where the sums need them, and as many stages as fit beside one another.
  const int per_sm = cta > 512 || (FULL && cta > 256) ? 1 : FULL ? 512 / cta : 1024 / cta;
  const int64_t stage = (int64_t)kMats * N * E::kBytes * cta, room = (228 * 1024) / per_sm - 1024 - (cta > kGroupThreads ? 2048 : 8192);
  const int stages = !VEC ? 0 : room >= 4 * stage ? 4 : room >= 3 * stage ? 3 : room >= 2 * stage ? 2 : 1;
  int64_t smem = stages * stage;
  if (smem < a.cols * 4 && cta > T) smem = a.cols * 4;
  int64_t want = (int64_t)per_sm * num_sms;
  const int64_t most = norm_parts(a.rows, a.cols);
  deal(a, want < most ? want : most);
  const auto go = [&](auto* k) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    return e != cudaSuccess ? e : launch_op(k, dim3((unsigned)a.ctas), cta, (size_t)smem, 1, s, a, T, stages);
  };
  if constexpr (N == 8) {
    if (cta <= 256) return go(k_norm_grad_rows<E, N, 256, FULL ? 2 : 4, VEC, LAYER, FULL, BIAS>);
    if (cta <= 512) return go(k_norm_grad_rows<E, N, 512, FULL ? 1 : 2, VEC, LAYER, FULL, BIAS>);
    if (FULL && cta <= 768) return go(k_norm_grad_rows<E, N, 768, 1, VEC, LAYER, FULL, BIAS>);
  }
  return go(k_norm_grad_rows<E, N, 1024, 1, VEC, LAYER, FULL, BIAS>);
}

template <class E, int N, bool VEC, bool FULL, bool BIAS>
cudaError_t norm_grad_rows(NormGradArgs& a, int num_sms, cudaStream_t s) {
  return a.layer ? norm_grad_rows_kind<E, N, VEC, true, FULL, BIAS>(a, num_sms, s)
                 : norm_grad_rows_kind<E, N, VEC, false, FULL, BIAS>(a, num_sms, s);
}

template <class E>
cudaError_t norm_grad(NormGradArgs& a, int num_sms, cudaStream_t s) {
  const bool full = a.gate || a.after_weight;
  const bool vec = on16<E>(a.dy, a.lddy, a.rows) && on16<E>(a.dr, a.lddr, a.rows) && on16<E>(a.r, a.ldr, a.rows) &&
                   on16<E>(a.x, a.ldx, a.rows) && on16<E>(a.dx, a.lddx, a.rows) && on16<E>(a.dresidual, a.lddres, a.rows) &&
                   on16<E>(a.gate, a.ldg, a.gate_rows) && on16<E>(a.sum[kSumGate], a.lddg, a.gate_rows) && on16(a.after_weight) &&
                   on16(a.after_bias) && on16(a.weight);
  cudaError_t e;
  if (a.cols <= 8192) {
    e = vec ? (full              ? norm_grad_rows<E, 8, true, true, true>(a, num_sms, s)
               : a.sum[kSumBias] ? norm_grad_rows<E, 8, true, false, true>(a, num_sms, s)
                                 : norm_grad_rows<E, 8, true, false, false>(a, num_sms, s))
            : (full              ? norm_grad_rows<E, 8, false, true, true>(a, num_sms, s)
               : a.sum[kSumBias] ? norm_grad_rows<E, 8, false, false, true>(a, num_sms, s)
                                 : norm_grad_rows<E, 8, false, false, false>(a, num_sms, s));
  } else if (a.cols <= 16384 && vec && !full && E::kBytes == 2) {
    e = norm_grad_rows<E, 16, true, false, true>(a, num_sms, s);
  } else {
    const int64_t want = 2 * (int64_t)num_sms, most = norm_parts(a.rows, a.cols);
    deal(a, want < most ? want : most);
    e = launch_op(k_norm_grad_any<E>, dim3((unsigned)a.ctas), kAnyThreads, 0, 1, s, a);
  }
  if (e != cudaSuccess) return e;
  JoinArgs j = {};
  j.cols = a.cols;
  int n = 0;
  int64_t deepest = 1;
  for (int k = 0; k < kNormSums; ++k) {
    if (!a.sum[k] || (k == kSumGate && !a.split)) continue;  // those gates are whole already
    const bool gate = k == kSumGate;
    j.part[n] = a.part[k], j.sum[n] = a.sum[k];
    j.count[n] = gate ? a.split : a.ctas, j.rows[n] = gate ? a.gate_rows : 1, j.ld[n] = gate ? a.lddg : 0;
    deepest = j.rows[n] > deepest ? j.rows[n] : deepest;
    ++n;
  }
  if (!n) return cudaSuccess;
  return launch_op(k_norm_join<E>, dim3((unsigned)((a.cols + 31) / 32), (unsigned)n, (unsigned)deepest), 32 * kJoinWarps, 0, 1, s, j);
}

}  // namespace

cudaError_t launch_norm(int dtype, const NormArgs& a, int num_sms, cudaStream_t s) {
  switch (dtype) {
    case AR_BF16: return norm<Bf16>(a, num_sms, s);
    case AR_FP16: return norm<F16>(a, num_sms, s);
    default: return norm<F32>(a, num_sms, s);
  }
}

int64_t norm_parts(int64_t rows, int64_t cols) {
  const int64_t most = cols <= 4096 ? 4 * kMostSms : cols <= 8192 ? 2 * kMostSms : kMostSms;
  return rows < most ? rows : most;
}

cudaError_t launch_norm_grad(int dtype, NormGradArgs& a, int num_sms, cudaStream_t s) {
  switch (dtype) {
    case AR_BF16: return norm_grad<Bf16>(a, num_sms, s);
    case AR_FP16: return norm_grad<F16>(a, num_sms, s);
    default: return norm_grad<F32>(a, num_sms, s);
  }
}

}  // namespace ar
