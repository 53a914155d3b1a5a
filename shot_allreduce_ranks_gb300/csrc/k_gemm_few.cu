// The gated product and the 8-bit product for a few tokens (a decoding step):
// the weights are streamed once and memory bounds it.
//
// A CTA makes a strip of 16 weight rows (8 of the gate and the same 8 of the up
// projection, or 16 channels) for all tokens, its eight warps taking turns along
// k.  The rows stand for the 16 rows of mma.sync m16n8k16 and the tokens for its
// eight columns.  Which k an instruction's k slots stand for is free as long
// as both operands agree, so a lane loads 16 contiguous bytes of its rows
// and of its token and uses them as they come: no shared memory, no shuffles.
// The gate's and the up projection's sums of one output land in one lane.  The
// warps' sums are joined in shared memory in a fixed order.
//
// Measured on one GB300: one token 8192 -> 3584 (117 MB of weights) 18.8-20 us,
// 5.9-6.2 TB/s, 87-92% of a copy's rate; 8 tokens 21.6 us; 8-bit, one token 3584
// -> 8192 (29 MB) 8.6 us; rows that begin anywhere, read by pairs of aligned
// pieces and shifted: 8001 -> 3500 40 us (62 by laying them out first).  Four-warp CTAs, and register limits for four CTAs an
// SM, were slower at most sizes (24.5 and 24.6 against 20.4 us for the first).
#include "ops_internal.cuh"

namespace ar {
namespace {

constexpr int kFewWarps = 8, kFewThreads = kFewWarps * 32;

// 16 bytes of a row at p, of which `left` may be read (the rest zero); VEC: rows
// start on 16 bytes.
template <bool VEC, int B>
__device__ __forceinline__ uint4 load_piece(const char* p, int64_t left, const char* begin, const char* end) {
  if (VEC && left >= 16) return ld_v4_stream(p);
  return load_anywhere<B>(p, left, begin, end);
}

__device__ __forceinline__ uint32_t offset_of(const char* row) {
  return (uint32_t)(reinterpret_cast<uintptr_t>(row) & 15u);  // of its pieces too: they lie 16 bytes apart
}

// Whether the aligned windows of a row's pieces k0 .. k1 lie within the matrix.
__device__ __forceinline__ bool within(const char* row, int64_t k0, int64_t k1, const char* begin, const char* end) {
  const char* base = row - offset_of(row);
  return base + k0 >= begin && base + k1 + 32 <= end;
}

__device__ __forceinline__ void load_window(const char* p, uint4& u, uint4& v) {
  const uint4* base = reinterpret_cast<const uint4*>(p - offset_of(p));
  u = __ldg(base);
  v = __ldg(base + 1);
}

template <int MODE, class E, int ACT, int NT, bool VEC>
__global__ void __launch_bounds__(kFewThreads) k_gemm_few(GemmArgs g) {
  constexpr int B = MODE == kGemmI8 ? 1 : 2;  // bytes of an element
  // 64-byte pieces of each row in flight a warp; rows that begin anywhere take two
  // loads a piece.
  constexpr int kUnroll = VEC ? (NT > 2 ? 2 : 4) : (NT > 2 ? 1 : 2);
  constexpr int kRows = MODE == kGemmI8 ? 16 : 8;
  using F = typename std::conditional<MODE == kGemmI8, F16, E>::type;
  __shared__ float4 part[kFewWarps][NT][32];
  pdl_enter();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g8 = lane >> 2, t4 = lane & 3;
  const int64_t n0 = (int64_t)blockIdx.x * kRows;
  // Rows past the last are read as the last one; their results are dropped.
  const int64_t ra = min(n0 + g8, g.N - 1), rb = MODE == kGemmI8 ? min(n0 + g8 + 8, g.N - 1) : ra;
  const int64_t bytes = g.K * B;
  const char* wa = static_cast<const char*>(g.b0) + ra * g.ldb * B;
  const char* wb = static_cast<const char*>(MODE == kGemmI8 ? g.b0 : g.b1) + rb * (MODE == kGemmI8 ? g.ldb : g.ldb1) * B;
  // Where the matrices begin and end.
  const char *begin_a = static_cast<const char*>(g.b0), *begin_b = static_cast<const char*>(MODE == kGemmI8 ? g.b0 : g.b1),
             *begin_x = static_cast<const char*>(g.a0);
  const char* end_a = begin_a + ((g.N - 1) * g.ldb + g.K) * B;
  const char* end_b = MODE == kGemmI8 ? end_a : begin_b + ((g.N - 1) * g.ldb1 + g.K) * B;
  const char* end_x = begin_x + ((g.M - 1) * g.lda + g.K) * B;
  const char* xs[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) xs[j] = static_cast<const char*>(g.a0) + min((int64_t)(8 * j + g8), g.M - 1) * g.lda * B;

  float acc[NT][4] = {};
  constexpr int kUnit = 64 * kUnroll;  // bytes of a row that a warp takes at a time
  for (int64_t at = (int64_t)warp * kUnit; at < bytes; at += kFewWarps * kUnit) {
    uint4 a[kUnroll], b[kUnroll], x[NT][kUnroll];
    // Inside the matrices, the windows around all pieces are loaded before the
    // first is shifted.
    const int64_t k0 = at + 16 * t4, k1 = k0 + 64 * (kUnroll - 1);
    bool inside = !VEC && k1 + 16 <= bytes && within(wa, k0, k1, begin_a, end_a) && within(wb, k0, k1, begin_b, end_b);
#pragma unroll
    for (int j = 0; j < NT; ++j) inside = inside && within(xs[j], k0, k1, begin_x, end_x);
    if (inside) {
      uint4 av[kUnroll], bv[kUnroll], xv[NT][kUnroll];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        load_window(wa + k0 + 64 * i, a[i], av[i]);
        load_window(wb + k0 + 64 * i, b[i], bv[i]);
#pragma unroll
        for (int j = 0; j < NT; ++j) load_window(xs[j] + k0 + 64 * i, x[j][i], xv[j][i]);
      }
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        a[i] = shift_window(a[i], av[i], offset_of(wa));
        b[i] = shift_window(b[i], bv[i], offset_of(wb));
#pragma unroll
        for (int j = 0; j < NT; ++j)
          x[j][i] = 8 * j + g8 < g.M ? shift_window(x[j][i], xv[j][i], offset_of(xs[j])) : make_uint4(0, 0, 0, 0);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int64_t k = k0 + 64 * i;
        a[i] = load_piece<VEC, B>(wa + k, bytes - k, begin_a, end_a);
        b[i] = load_piece<VEC, B>(wb + k, bytes - k, begin_b, end_b);
#pragma unroll
        for (int j = 0; j < NT; ++j)
          x[j][i] = 8 * j + g8 < g.M ? load_piece<VEC, B>(xs[j] + k, bytes - k, begin_x, end_x) : make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const uint32_t aw[4] = {a[i].x, a[i].y, a[i].z, a[i].w}, bw[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
      if (MODE == kGemmI8) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t f[4];
          i8_to_f16(aw[w], f[0], f[2]);
          i8_to_f16(bw[w], f[1], f[3]);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const uint32_t xw[4] = {x[j][i].x, x[j][i].y, x[j][i].z, x[j][i].w};
            uint32_t y[2];
            i8_to_f16(xw[w], y[0], y[1]);
            mma_16816<F>(acc[j], f, y);
          }
        }
      } else {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const uint32_t f[4] = {aw[2 * w], bw[2 * w], aw[2 * w + 1], bw[2 * w + 1]};
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const uint32_t xw[4] = {x[j][i].x, x[j][i].y, x[j][i].z, x[j][i].w};
            const uint32_t y[2] = {xw[2 * w], xw[2 * w + 1]};
            mma_16816<F>(acc[j], f, y);
          }
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) part[warp][j][lane] = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
  __syncthreads();
  if (threadIdx.x >= NT * 32) return;
  const int j = warp;  // the eight tokens that this warp finishes
  float s[4] = {};
#pragma unroll
  for (int w = 0; w < kFewWarps; ++w) {
    const float4 p = part[w][j][lane];
    s[0] += p.x, s[1] += p.y, s[2] += p.z, s[3] += p.w;
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int64_t m = 8 * j + 2 * t4 + e;
    if (m >= g.M) continue;
    if (MODE == kGemmGated) {
      const int64_t n = n0 + g8, at = m * g.ldc + n;
      if (n >= g.N) continue;
      static_cast<uint16_t*>(g.c0)[at] = (uint16_t)E::from_f32(act_value<ACT>(s[e]) * s[e + 2]);
      if (g.c1) {
        static_cast<uint16_t*>(g.c1)[at] = (uint16_t)E::from_f32(s[e]);
        static_cast<uint16_t*>(g.c2)[at] = (uint16_t)E::from_f32(s[e + 2]);
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t n = n0 + g8 + 8 * h;
        if (n < g.N)
          static_cast<uint16_t*>(g.c0)[m * g.ldc + n] = (uint16_t)E::from_f32(s[2 * h + e] * g.sm[m] * g.sn[n]);
      }
    }
  }
}

template <int MODE, class E, int ACT, bool VEC>
cudaError_t launch(const GemmArgs& g, cudaStream_t s) {
  constexpr int kRows = MODE == kGemmI8 ? 16 : 8;
  const int64_t grid = (g.N + kRows - 1) / kRows;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  auto* k = g.M <= 8    ? k_gemm_few<MODE, E, ACT, 1, VEC>
            : g.M <= 16 ? k_gemm_few<MODE, E, ACT, 2, VEC>
                        : k_gemm_few<MODE, E, ACT, 4, VEC>;
  return launch_op(k, dim3((unsigned)grid), kFewThreads, 0, 1, s, g);
}

template <int MODE, class E, int ACT>
cudaError_t launch_align(const GemmArgs& g, cudaStream_t s) {
  const int64_t unit = MODE == kGemmI8 ? 16 : 8;
  const bool vec = ((reinterpret_cast<uintptr_t>(g.a0) | reinterpret_cast<uintptr_t>(g.b0) |
                     reinterpret_cast<uintptr_t>(g.b1)) & 15u) == 0 && g.lda % unit == 0 && g.ldb % unit == 0 &&
                   g.ldb1 % unit == 0;
  return vec ? launch<MODE, E, ACT, true>(g, s) : launch<MODE, E, ACT, false>(g, s);
}

template <class E>
cudaError_t launch_type(int mode, const GemmArgs& g, cudaStream_t s) {
  if (mode == kGemmI8) return launch_align<kGemmI8, E, 0>(g, s);
  return g.act == AR_ACT_SILU ? launch_align<kGemmGated, E, AR_ACT_SILU>(g, s)
                              : launch_align<kGemmGated, E, AR_ACT_GELU_TANH>(g, s);
}

}  // namespace

bool gemm_few_takes(int mode, const GemmArgs& g) {
  return (mode == kGemmGated || mode == kGemmI8) && g.M <= 32;
}

cudaError_t launch_gemm_few(int mode, int dtype, const GemmArgs& g, cudaStream_t s) {
  return dtype == AR_BF16 ? launch_type<Bf16>(mode, g, s) : launch_type<F16>(mode, g, s);
}

}  // namespace ar
