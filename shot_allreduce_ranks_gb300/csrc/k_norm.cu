// Norms before and after a block with its gate and the residual, and their
// gradients (formulas in include/ar.h).
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
  if (c < a.cols)
    for (int64_t i = warp; i < a.count[k]; i += kJoinWarps) v += p[i * a.cols + c];
  room[warp][lane] = v;
  __syncthreads();
  if (warp || c >= a.cols) return;
  v = 0.0f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) v += room[w][lane];
  put<E>(a.sum[k], row * a.ld[k] + c, v);
}

template <class E>
cudaError_t norm(const NormArgs& a, int num_sms, cudaStream_t s) {
  const int64_t most = (int64_t)num_sms * 8;
  return launch_op(k_norm_any<E>, dim3((unsigned)(a.rows < most ? a.rows : most)), kAnyThreads, 0, 1, s, a);
}

template <class E>
cudaError_t norm_grad(const NormGradArgs& a, cudaStream_t s) {
  cudaError_t e = launch_op(k_norm_grad_any<E>, dim3((unsigned)a.ctas), kAnyThreads, 0, 1, s, a);
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

cudaError_t launch_norm_grad(int dtype, NormGradArgs& a, int num_sms, cudaStream_t s) {
  // Up to two CTAs an SM.  Where there are fewer gate rows than CTAs each is split
  // among as many; where there are more, a CTA takes several whole ones.
  const int64_t want = 2 * (int64_t)num_sms < kNormMaxCtas ? 2 * (int64_t)num_sms : kNormMaxCtas;
  if (a.gate_rows <= want) {
    const int64_t parts = want / a.gate_rows;
    a.chunk = (a.gate_run + parts - 1) / parts;
    a.split = (a.gate_run + a.chunk - 1) / a.chunk;
    a.ctas = a.gate_rows * a.split;
  } else {
    a.split = a.chunk = 0;
    a.ctas = want;
  }
  switch (dtype) {
    case AR_BF16: return norm_grad<Bf16>(a, s);
    case AR_FP16: return norm_grad<F16>(a, s);
    default: return norm_grad<F32>(a, s);
  }
}

}  // namespace ar
