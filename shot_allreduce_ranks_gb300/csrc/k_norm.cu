// Norms before and after a block with its gate and the residual (formulas in
// include/ar.h): x and the residual are read once, r and y written once, and memory
// bounds it.  A row stays in its threads' registers between its statistics and its
// results; the mean square is that of the differences from the mean.  1 / sqrt is the
// hardware's reciprocal root, good to 2^-22.9 (the kernel for any row divides by the root: two roundings, 2^-23).
//
// Measured on one GB300 in a replayed graph: 16384 x 8192 bf16 with the residual 177-182 us (1.07
// GB: 87-89% of the copy rate), 8192 x 8192 fp32 154, 440 x 5120 with both norms 4.7, one row 2.3; rows of
// odd length 8192 x 4095 bf16 107 (2.7 times the floor: shifting pieces and storing
// across lanes takes the issue slots).
#include "norm_device.cuh"

namespace ar {
namespace {

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
  s.factor = rsqrtf(sum[0] / (float)c.cols + eps);
  return s;
}

// One row, x in v and the residual in q: r and y are stored.  room holds four rows.
template <class E, int N, Layout L, bool WARP>
__device__ __forceinline__ void norm_row(const NormArgs& a, const Columns<E, N, L>& c, int64_t row, float (&v)[N], const float (&q)[N],
                                         float (*room)[32]) {
  float w[N];
  if (a.after_weight) {
    c.load_shared(a.after_weight, 0, a.cols, w);
    const Stats s = stats_of<WARP>(c, v, a.layer, a.eps, room);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = (v[i] - s.mean) * s.factor * (a.offset + w[i]);
    if (a.after_bias) {
      c.load_shared(a.after_bias, 0, a.cols, w);
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += w[i];
    }
  }
  if (a.gate) {
    c.load_shared(a.gate, row / a.gate_run * a.ldg, a.gate_extent, w);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] *= w[i];
  }
  if (a.residual) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __fmaf_rn(a.alpha, q[i], v[i]);
  }
  if (a.weight) c.load_shared(a.weight, 0, a.cols, w);
  if (a.r) c.store(a.r, row * a.ldr, v);
  if (!a.weight) return;
  // Columns past the last hold what biases left there, which the norm must not see.
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = c.has(i) ? v[i] : 0.0f;
  const Stats s = stats_of<WARP>(c, v, a.layer, a.eps, room + 2);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = (v[i] - s.mean) * s.factor * (a.offset + w[i]);
  if (a.bias) {
    c.load_shared(a.bias, 0, a.cols, w);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += w[i];
  }
  c.store(a.y, row * a.ldy, v);
}

// A row a CTA, or (WARP) a row a warp, read once and held in registers, N columns a thread.
template <class E, int N, Layout L, bool WARP>
__global__ void __launch_bounds__(1024) k_norm_rows(NormArgs a) {
  __shared__ float room[4][32];
  pdl_enter();
  const int64_t row = WARP ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
  if (WARP && row >= a.rows) return;
  const Columns<E, N, L> c = {WARP ? (int)(threadIdx.x & 31) : (int)threadIdx.x, WARP ? 32 : (int)blockDim.x, (int)a.cols};
  float v[N], q[N];
  c.load(a.x, row * a.ldx, (a.rows - 1) * a.ldx + a.cols, v);
  if (a.residual) c.load(a.residual, row * a.ldres, (a.rows - 1) * a.ldres + a.cols, q);
  norm_row<E, N, L, WARP>(a, c, row, v, q, room);
}

// Many rows: a CTA (or warp) takes every gridDim-th and copies the next ones into shared
// memory meanwhile, kStages - 1 of them (128 KB an SM in flight); a thread copies what it will read itself, so only
// its own copies have to be waited for.
constexpr int kStages = 3;
template <class E, int N, bool WARP>
__global__ void __launch_bounds__(1024) k_norm_stream(NormArgs a) {
  extern __shared__ __align__(16) char smem[];
  __shared__ float room[8][32];
  constexpr int G = E::kGroup, kPieces = N / G;
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const Columns<E, N, kAligned> c = {WARP ? lane : (int)threadIdx.x, WARP ? 32 : (int)blockDim.x, (int)a.cols};
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
    norm_row<E, N, kAligned, WARP>(a, c, row, v, q, room + 4 * parity);
    parity ^= 1;
    stage = stage == kStages - 1 ? 0 : stage + 1;
  }
}

template <class E, int N, Layout L>
cudaError_t norm_rows(const NormArgs& a, cudaStream_t s) {
  const int64_t threads = (a.cols + 32 * N - 1) / (32 * N) * 32;
  if (threads == 32) {
    const int64_t grid = (a.rows + 3) / 4;
    return launch_op(k_norm_rows<E, N, L, true>, dim3((unsigned)grid), 128, 0, 1, s, a);
  }
  return launch_op(k_norm_rows<E, N, L, false>, dim3((unsigned)a.rows), (int)threads, 0, 1, s, a);
}

template <class E>
cudaError_t norm_stream(const NormArgs& a, int num_sms, cudaStream_t s) {
  constexpr int N = 16;
  const int64_t threads = (a.cols + 32 * N - 1) / (32 * N) * 32;
  const int cta = threads == 32 ? 128 : (int)threads, rows = threads == 32 ? 4 : 1;
  const size_t smem = (size_t)kStages * 2 * N * E::kBytes * cta;
  const int64_t want = (a.rows + rows - 1) / rows, most = 1024 / cta * (int64_t)num_sms;
  const dim3 grid((unsigned)(want < most ? want : most));
  return threads == 32 ? launch_raised<k_norm_stream<E, N, true>>(grid, cta, smem, s, a)
                       : launch_raised<k_norm_stream<E, N, false>>(grid, cta, smem, s, a);
}

template <class E>
cudaError_t norm(const NormArgs& a, int num_sms, cudaStream_t s) {
  const bool vec = on16<E>(a.x, a.ldx, a.rows) && on16<E>(a.residual, a.ldres, a.rows) && on16<E>(a.r, a.ldr, a.rows) &&
                   on16<E>(a.y, a.ldy, a.rows) && on16<E>(a.gate, a.ldg, a.rows / a.gate_run) && on16(a.after_weight) &&
                   on16(a.after_bias) && on16(a.weight) && on16(a.bias);
  if (a.cols > 16384 || a.rows > 0x7FFFFFFF) {
    const int64_t most = (int64_t)num_sms * 8;
    return launch_op(k_norm_any<E>, dim3((unsigned)(a.rows < most ? a.rows : most)), kAnyThreads, 0, 1, s, a);
  }
  // Rows that start anywhere: 16-bit ones by shifted pieces, fp32 by elements (8192 x 4095 bf16 108 and 110 us,
  // 2048 x 5121 fp32 73 and 50).
  constexpr Layout kAny = E::kBytes == 2 ? kShifted : kElements;
  if (!vec) return a.cols <= 8192 ? norm_rows<E, 8, kAny>(a, s) : norm_rows<E, 16, kAny>(a, s);
  // Eight columns a thread where no SM gets a second row (1 x 5120 bf16 2.3 us, sixteen 2.7);
  // above, sixteen, whose loads in flight keep fp32 at the copy rate (8192 x 8192: 154 us, copied ahead 179);
  // 16-bit rows of half the bytes are copied ahead from three rows an SM on (440 x 8192 bf16 6.4 us,
  // copied ahead 7.1; 1000 x 8192 16.1 and 14.5; 16384 x 8192 232 and 177).
  if (a.rows <= num_sms && a.cols <= 8192) return norm_rows<E, 8, kAligned>(a, s);
  if constexpr (E::kBytes == 2)
    if (a.rows > 3 * (int64_t)num_sms) return norm_stream<E>(a, num_sms, s);
  return norm_rows<E, 16, kAligned>(a, s);
}

}  // namespace

cudaError_t launch_norm(int dtype, const NormArgs& a, int num_sms, cudaStream_t s) {
  switch (dtype) {
    case AR_BF16: return norm<Bf16>(a, num_sms, s);
    case AR_FP16: return norm<F16>(a, num_sms, s);
    default: return norm<F32>(a, num_sms, s);
  }
}

}  // namespace ar
