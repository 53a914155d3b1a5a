// The operators' matrix products for operands of any alignment and stride:
// rows of odd length, views that begin at an odd element.
//
// C[m, n] = sum_k A(m, k) B(n, k) in fp32 on mma.sync m16n8k16.  A CTA of four
// warps makes a 64 x 64 tile; in the gated product its 64 columns are 32 of
// the gate and the same 32 of the up projection, so that one thread holds both
// pre-activations of an element.  Elements are loaded one at a time, along
// the contiguous axis, into registers while the tile before is multiplied.
// 8-bit integers become fp16 on the way into shared memory: fp16 holds them
// exactly, their products are exact in fp32, and so are the sums while they
// stay below 2^24 (always so for K <= 1024).
//
// It makes what the tensor-map kernels cannot read and the caller gave no scratch
// to lay out for them.  Measured on one GB300: 46 TFLOP/s on large sizes, a
// thirtieth of theirs (gradients at 1001 x 1031 -> 777: 153 us, 23 with scratch);
// bound by its element loads.
#include "ops_internal.cuh"

namespace ar {
namespace {

constexpr int kTile = 64, kDepth = 32, kThreadsAny = 128;
constexpr int kPitch = kDepth + 8;  // 80 bytes: the fragments' 32-bit loads hit 32 banks
constexpr int kPer = kTile * kDepth / kThreadsAny;

__device__ __forceinline__ uint32_t load_bits(const uint16_t* p) { return *p; }
__device__ __forceinline__ uint32_t load_bits(const int8_t* p) {
  return cvt_rn_f16x2((float)*p, 0.0f) & 0xFFFFu;
}

// One tile of an operand into registers.  KMAJOR: element (row, k) at
// p[row * ld + k], else at p[k * ld + row].  Outside `rows` x `depth`: 0.
template <bool KMAJOR, class S>
__device__ __forceinline__ void load_tile(uint32_t (&r)[kPer], const S* p, int64_t ld, int64_t row0,
                                          int64_t rows, int64_t k0, int64_t depth, int tid) {
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid + i * kThreadsAny;
    const int64_t row = row0 + (KMAJOR ? e / kDepth : e % kTile);
    const int64_t k = k0 + (KMAJOR ? e % kDepth : e / kTile);
    r[i] = row < rows && k < depth ? load_bits(p + (KMAJOR ? row * ld + k : k * ld + row)) : 0u;
  }
}

template <bool KMAJOR>
__device__ __forceinline__ void store_tile(uint16_t (*s)[kPitch], const uint32_t (&r)[kPer], int tid) {
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid + i * kThreadsAny;
    s[KMAJOR ? e / kDepth : e % kTile][KMAJOR ? e % kDepth : e / kTile] = (uint16_t)r[i];
  }
}

template <int MODE, class E, int ACT>
__global__ void __launch_bounds__(kThreadsAny) k_gemm_any(GemmArgs g, int64_t tiles_n) {
  using S = typename std::conditional<MODE == kGemmI8, int8_t, uint16_t>::type;
  using F = typename std::conditional<MODE == kGemmI8, F16, E>::type;  // type that is multiplied
  constexpr bool kAK = MODE != kGemmDw, kBK = MODE == kGemmGated || MODE == kGemmI8;
  constexpr int kCols = MODE == kGemmGated ? kTile / 2 : kTile;  // output columns of a tile
  __shared__ uint16_t sa[kTile][kPitch], sb[kTile][kPitch];
  pdl_enter();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int wm = warp >> 1, wn = warp & 1, g4 = lane >> 2, t4 = lane & 3;
  const int64_t m0 = (int64_t)(blockIdx.x / tiles_n) * kTile;
  const int64_t n0 = (int64_t)(blockIdx.x % tiles_n) * kCols;
  const bool second = blockIdx.y != 0;  // kGemmDw: the up projection's gradient
  const int64_t steps = (g.K + kDepth - 1) / kDepth;
  const int64_t total = MODE == kGemmDx ? 2 * steps : steps;

  float acc[2][4][4] = {};
  uint32_t ra[kPer], rb[kPer];
  auto fetch = [&](int64_t step) {
    const bool up = MODE == kGemmDx ? step >= steps : second;
    const int64_t k0 = (up && MODE == kGemmDx ? step - steps : step) * kDepth;
    load_tile<kAK>(ra, static_cast<const S*>(up ? g.a1 : g.a0), g.lda, m0, g.M, k0, g.K, tid);
    if (MODE == kGemmGated) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {  // rows 0..31 of the tile: gate, 32..63: up
        const int e = tid + i * kThreadsAny, row = e / kDepth;
        const int64_t n = n0 + (row & 31), k = k0 + e % kDepth;
        const S* p = static_cast<const S*>(row < 32 ? g.b0 : g.b1);
        rb[i] = n < g.N && k < g.K ? load_bits(p + n * (row < 32 ? g.ldb : g.ldb1) + k) : 0u;
      }
    } else {
      const bool b1 = MODE == kGemmDx && up;
      load_tile<kBK>(rb, static_cast<const S*>(b1 ? g.b1 : g.b0), b1 ? g.ldb1 : g.ldb, n0, g.N, k0, g.K, tid);
    }
  };
  fetch(0);
  for (int64_t step = 0; step < total; ++step) {
    __syncthreads();
    store_tile<kAK>(sa, ra, tid);
    store_tile<kBK>(sb, rb, tid);
    __syncthreads();
    if (step + 1 < total) fetch(step + 1);
#pragma unroll
    for (int kk = 0; kk < kDepth; kk += 16) {
      uint32_t a[2][4], b[4][2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = wm * 32 + i * 16 + g4, c = kk + 2 * t4;
        a[i][0] = *reinterpret_cast<const uint32_t*>(&sa[r][c]);
        a[i][1] = *reinterpret_cast<const uint32_t*>(&sa[r + 8][c]);
        a[i][2] = *reinterpret_cast<const uint32_t*>(&sa[r][c + 8]);
        a[i][3] = *reinterpret_cast<const uint32_t*>(&sa[r + 8][c + 8]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // gated: columns 0, 8 of this warp's 16 of the gate, then of the up
        const int r = (MODE == kGemmGated ? (j >> 1) * 32 + wn * 16 + (j & 1) * 8 : wn * 32 + j * 8) + g4;
        b[j][0] = *reinterpret_cast<const uint32_t*>(&sb[r][kk + 2 * t4]);
        b[j][1] = *reinterpret_cast<const uint32_t*>(&sb[r][kk + 2 * t4 + 8]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) mma_16816<F>(acc[i][j], a[i], b[j]);
    }
  }

#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < (MODE == kGemmGated ? 2 : 4); ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t m = m0 + wm * 32 + i * 16 + g4 + (e >> 1) * 8;
        const int64_t n = n0 + wn * (kCols / 2) + j * 8 + 2 * t4 + (e & 1);
        if (m >= g.M || n >= g.N) continue;
        const int64_t at = m * g.ldc + n;
        const float v = acc[i][j][e];
        if (MODE == kGemmGated) {
          const float u = acc[i][j + 2][e];
          static_cast<uint16_t*>(g.c0)[at] = (uint16_t)E::from_f32(act_value<ACT>(v) * u);
          if (g.c1) {
            static_cast<uint16_t*>(g.c1)[at] = (uint16_t)E::from_f32(v);
            static_cast<uint16_t*>(g.c2)[at] = (uint16_t)E::from_f32(u);
          }
        } else if (MODE == kGemmI8) {
          static_cast<uint16_t*>(g.c0)[at] = (uint16_t)E::from_f32(v * g.sm[m] * g.sn[n]);
        } else {
          static_cast<uint16_t*>(second ? g.c1 : g.c0)[at] = (uint16_t)E::from_f32(v);
        }
      }
}

template <int MODE, class E, int ACT>
cudaError_t launch(const GemmArgs& g, cudaStream_t s) {
  const int64_t cols = MODE == kGemmGated ? kTile / 2 : kTile;
  const int64_t tn = (g.N + cols - 1) / cols, tm = (g.M + kTile - 1) / kTile;
  if (tn * tm > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)(tn * tm), MODE == kGemmDw ? 2 : 1);
  return launch_op(k_gemm_any<MODE, E, ACT>, grid, kThreadsAny, 0, 1, s, g, tn);
}

template <class E>
cudaError_t launch_type(int mode, const GemmArgs& g, cudaStream_t s) {
  switch (mode) {
    case kGemmGated:
      return g.act == AR_ACT_SILU ? launch<kGemmGated, E, AR_ACT_SILU>(g, s)
                                  : launch<kGemmGated, E, AR_ACT_GELU_TANH>(g, s);
    case kGemmDx: return launch<kGemmDx, E, 0>(g, s);
    case kGemmDw: return launch<kGemmDw, E, 0>(g, s);
    default: return launch<kGemmI8, E, 0>(g, s);
  }
}

}  // namespace

cudaError_t launch_gemm_any(int mode, int dtype, const GemmArgs& g, cudaStream_t s) {
  return dtype == AR_BF16 ? launch_type<Bf16>(mode, g, s) : launch_type<F16>(mode, g, s);
}

}  // namespace ar
