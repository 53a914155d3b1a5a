// Products with 4-bit weights and group scales for a few tokens, and the
// weights' layout (formulas in include/ar.h).
//
// The layout is the one in which a warp's lanes hold the A operand of
// mma.sync m16n8k16, whose 16 rows stand for 16 output channels and whose 8
// columns for tokens: tiles of 16 channels by 64 k, 512 bytes each, one after the other
// along k, in which lane 4 (n % 8) + t has its 16 bytes together.  Word 2p + h of them
// holds channels n and n + 8 at k = 32p + 8t + 4h + 0..3: which k an instruction's k slots
// stand for is free as long as both operands agree, and so a lane's eight values of x
// for two instructions are 16 contiguous bytes.  An instruction's k lie
// within one group of 32 or more, so the group's scale multiplies the fp32 sums and never
// a weight: q - zero is exact in 16 bits.
#include "ops_internal.cuh"

namespace ar {
namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;

// Scales (and zero points) of a tile lie by spans of 64 k, or of a group where that is
// longer: for each channel n < 8 the span's groups, channels n and n + 8 of each.
__host__ __device__ constexpr int span_of(int group) { return group > 64 ? group : 64; }
__host__ __device__ constexpr int groups_in(int group) { return span_of(group) / group; }
__device__ __forceinline__ int64_t scale_at(int64_t n, int64_t g, int64_t spans, int per) {
  return (((n / 16) * spans + g / per) * 8 + n % 8) * per * 2 + g % per * 2 + n % 16 / 8;
}

// A word's eight weights as the A operand: 128 + q (bf16) or 1024 + q (fp16) is the
// number whose lowest mantissa bits are q; less 128 or 1024 + zero leaves q - zero, exactly.
template <class E>
__device__ __forceinline__ uint32_t biased(uint32_t q) { return q | (IsBf16<E>::value ? 0x43004300u : 0x64006400u); }
template <class E>
__device__ __forceinline__ uint32_t less(uint32_t a, uint32_t b) {
  uint32_t d;
  if (IsBf16<E>::value)
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <class E>
__device__ __forceinline__ void unpack(uint32_t w, uint32_t zero_lo, uint32_t zero_hi, uint32_t (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = less<E>(biased<E>(w >> (4 * i) & 0x000F000Fu), i & 1 ? zero_hi : zero_lo);
}

// 16 bytes of a token's row at byte k, of which `left` are there.
template <bool VEC>
__device__ __forceinline__ uint4 row_piece(const char* row, int64_t k, int64_t left) {
  if (VEC && left >= 16) return *reinterpret_cast<const uint4*>(row + k);
  uint32_t w[4] = {};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (2 * i < left) w[i / 2] |= ld_elem<2>(row + k + 2 * i) << (16 * (i % 2));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A span's weights of one tile, and its scales and zero points.
template <int GROUP, bool ZERO>
struct Span {
  static constexpr int kPer = groups_in(GROUP), kTiles = span_of(GROUP) / 64;
  uint4 w[kTiles];
  uint32_t scale[kPer], zero[kPer];

  // The pointers are those of the lane in the tile.
  __device__ __forceinline__ void load(const uint4* data, const uint16_t* scales, const uint8_t* zeros, int64_t s) {
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      const uint4* p = data + (s * kTiles + i) * 32;
      asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
                   : "l"(p));
    }
    if (kPer == 2) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(scales + s * 8 * kPer * 2));
      scale[0] = v.x, scale[kPer - 1] = v.y;
      if (ZERO) {
        const uint32_t z = __ldg(reinterpret_cast<const uint32_t*>(zeros + s * 8 * kPer * 2));
        zero[0] = z & 0xFFFFu, zero[kPer - 1] = z >> 16;
      }
    } else {
      scale[0] = __ldg(reinterpret_cast<const uint32_t*>(scales + s * 8 * kPer * 2));
      if (ZERO) zero[0] = __ldg(reinterpret_cast<const uint16_t*>(zeros + s * 8 * kPer * 2));
    }
  }

  // acc += the span's products with x, pieces p of tile i for 8 NB tokens.
  template <class E, int NB>
  __device__ __forceinline__ void multiply(float (&acc)[NB][4], const uint4 (&x)[kTiles][2][NB]) const {
    float sum[NB][4];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      const uint32_t words[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int g = kPer == 2 ? h / 2 : 0;
        const bool first = GROUP == 32 ? h % 2 == 0 : i == 0 && h == 0, last = GROUP == 32 ? h % 2 == 1 : i == kTiles - 1 && h == 3;
        const uint32_t zl = ZERO ? zero[g] & 0xFFu : 8u, zh = ZERO ? zero[g] >> 8 : 8u;
        uint32_t f[4];
        unpack<E>(words[h], biased<E>(zl * 0x10001u), biased<E>(zh * 0x10001u), f);
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const uint4& v = x[i][h / 2][j];
          const uint32_t y[2] = {h % 2 ? v.z : v.x, h % 2 ? v.w : v.y};
          if (first) sum[j][0] = sum[j][1] = sum[j][2] = sum[j][3] = 0.0f;
          mma_16816<E>(sum[j], f, y);
        }
        if (last) {
          const float lo = E::lo(scale[g]), hi = E::hi(scale[g]);
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            acc[j][0] = __fmaf_rn(lo, sum[j][0], acc[j][0]);
            acc[j][1] = __fmaf_rn(lo, sum[j][1], acc[j][1]);
            acc[j][2] = __fmaf_rn(hi, sum[j][2], acc[j][2]);
            acc[j][3] = __fmaf_rn(hi, sum[j][3], acc[j][3]);
          }
        }
      }
    }
  }
};

// A tile of sixteen channels for up to 8 NB tokens a CTA; its warps take turns at the spans
// along k, and their sums are joined in a fixed order.
//
// With few tokens the loads in flight bound it: a warp has four pieces of 512 bytes under way and none while it
// multiplies.  Three CTAs an SM with four pieces a warp were the fastest of 2 to 8 pieces and 1 to 5 CTAs.  Unpacking, 7/8 of an
// integer instruction a weight (four logical operations and three shifts for every eight), costs at most 2 us of the 17.5, and the
// integer pipe is 54% active; CTAs that are no multiple of the 456 on the device at once cost 0.7 (2 rounds of them 15.2 us, 2.25
// 17.5, 3 21.7).  With more tokens it is x, of which every CTA reads all through L1: 32 bytes for a block of eight tokens beside 16 of
// weights.  8192 -> 16384 in groups of 128 (69 MB): one token 17.5 us (58% of the copy rate), 8 tokens 18.4, 13 25.8, 32 47.6, 64
// (weights twice) 82.6.  Weights copied ahead by a persistent CTA with x in shared memory took 21.7 us for one token.
template <class E, int GROUP, bool ZERO, int NB, bool VEC>
__global__ void __launch_bounds__(kThreads, NB > 2 ? 2 : 3) k_linear_i4(I4Args a) {
  constexpr int kSpan = span_of(GROUP), kPer = groups_in(GROUP), kTiles = kSpan / 64;
  constexpr int U = NB == 1 ? 4 / kTiles : NB == 2 ? 2 / kTiles : 1;  // spans in flight
  __shared__ float4 part[kWarps][NB][32];
  pdl_enter();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g8 = lane >> 2, t4 = lane & 3;
  const int64_t m0 = (int64_t)blockIdx.y * 32, M = min(a.M - m0, (int64_t)32), spans = a.spans, bytes = a.K * 2;
  const int64_t tile = blockIdx.x;
  const uint4* data = reinterpret_cast<const uint4*>(a.data) + tile * spans * kTiles * 32 + lane;
  const uint16_t* scales = static_cast<const uint16_t*>(a.scale) + (tile * spans * 8 + g8) * kPer * 2;
  const uint8_t* zeros = ZERO ? a.zero + (tile * spans * 8 + g8) * kPer * 2 : nullptr;
  // A token past the last is read as the last: its column of the results is dropped.
  const char* xs[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j)
    xs[j] = static_cast<const char*>(a.x) + (m0 + min((int64_t)(8 * j + g8), M - 1)) * a.ldx * 2 + 16 * t4;

  float acc[NB][4] = {};
  Span<GROUP, ZERO> span[U];
  uint4 x[U][kTiles][2][NB];
  const int64_t whole = bytes / (kSpan * 2);  // spans that x has all of
  int64_t s = (int64_t)warp * U;
  for (; s + U <= whole; s += kWarps * U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      span[u].load(data, scales, zeros, s + u);
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int j = 0; j < NB; ++j) x[u][i][p][j] = row_piece<VEC>(xs[j], (s + u) * kSpan * 2 + 128 * i + 64 * p, 16);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) span[u].template multiply<E, NB>(acc, x[u]);
  }
  for (int u = 0; u < U && s + u < spans; ++u) {
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const int64_t k = (s + u) * kSpan * 2 + 128 * i + 64 * p;
          x[0][i][p][j] = row_piece<VEC>(xs[j], k, bytes - k - 16 * t4);
        }
    span[0].load(data, scales, zeros, s + u);
    span[0].template multiply<E, NB>(acc, x[0]);
  }
#pragma unroll
  for (int j = 0; j < NB; ++j) part[warp][j][lane] = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
  __syncthreads();
  if (warp >= NB) return;
  float v[4] = {};
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    const float4 p = part[i][warp][lane];
    v[0] += p.x, v[1] += p.y, v[2] += p.z, v[3] += p.w;
  }
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t m = 8 * warp + 2 * t4 + c, n = tile * 16 + g8 + 8 * h;
      if (m < M && n < a.N) static_cast<uint16_t*>(a.y)[(m0 + m) * a.ldy + n] = (uint16_t)E::from_f32(v[2 * h + c]);
    }
}

// One lane's 16 bytes of a tile; get(n, k): the whole number at channel n and k.
template <class F>
__device__ __forceinline__ uint4 lay_out(F get, int64_t tile, int64_t kb, int lane, int64_t N, int64_t K) {
  uint32_t w[4] = {};
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t n = tile * 16 + lane / 4 + 8 * half, k = kb * 64 + i / 2 * 32 + lane % 4 * 8 + i % 2 * 4 + j;
        if (n < N && k < K) w[i] |= (get(n, k) & 15u) << (4 * (j / 2 * 2 + half) + 16 * (j % 2));
      }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Whole numbers, scales and zero points a row, laid out.
__global__ void __launch_bounds__(256) k_pack_i4(I4Pack a) {
  pdl_enter();
  const int per = groups_in(a.group), tiles = span_of(a.group) / 64;
  const int64_t nt = (a.N + 15) / 16, lanes = nt * a.spans * tiles * 32, groups = (a.K + a.group - 1) / a.group;
  const int64_t slots = nt * a.spans * 8 * per * 2;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < (lanes > slots ? lanes : slots); i += (int64_t)gridDim.x * 256) {
    if (i < lanes) {
      const int64_t at = i / 32, tile = at / (a.spans * tiles), kb = at % (a.spans * tiles);
      a.data[i] = lay_out([&](int64_t n, int64_t k) { return (uint32_t)a.q[n * a.ldq + k]; }, tile, kb, (int)(i % 32), a.N, a.K);
    }
    if (i < slots) {
      const int64_t half = i % 2, in = i / 2 % per, n8 = i / 2 / per % 8, s = i / 2 / per / 8 % a.spans, tile = i / 2 / per / 8 / a.spans;
      const int64_t n = tile * 16 + n8 + 8 * half, g = s * per + in;
      const bool there = n < a.N && g < groups;
      a.scale[i] = there ? a.row_scale[n * a.lds + g] : 0;
      if (a.zero) a.zero[i] = there ? a.row_zero[n * a.ldz + g] & 15 : 0;
    }
  }
}

// A warp a group of a row: its scale and zero point, then its whole numbers into q (a row of K bytes for each channel).
template <class E>
__global__ void __launch_bounds__(256) k_quantize_i4(I4Quantize a) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int64_t groups = (a.K + a.group - 1) / a.group, total = a.N * groups;
  for (int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < total; i += (int64_t)gridDim.x * 8) {
    const int64_t n = i / groups, k0 = i % groups * a.group, k1 = min(k0 + a.group, a.K);
    float v[4], high = 0.0f, low = 0.0f;
    bool finite = true;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t k = k0 + 32 * j + lane;
      v[j] = k < k1 ? E::to_f32(ld_elem<2>(static_cast<const char*>(a.w) + (n * a.ldw + k) * 2)) : 0.0f;
      finite = finite && fabsf(v[j]) < INFINITY;
      high = fmaxf(high, v[j]);
      low = fminf(low, v[j]);
    }
    finite = __all_sync(0xFFFFFFFFu, finite);
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      high = fmaxf(high, __shfl_xor_sync(0xFFFFFFFFu, high, o));
      low = fminf(low, __shfl_xor_sync(0xFFFFFFFFu, low, o));
    }
    const float want = a.row_zero ? high / 15.0f - low / 15.0f : fmaxf(high, -low) / 7.0f;
    const uint32_t bits = finite ? E::from_f32(want) : 0x7FFFu;  // NaN
    const float scale = E::to_f32(bits);
    const bool none = !finite || scale == 0.0f;
    const float zero = !a.row_zero ? 8.0f : none ? 0.0f : fminf(rintf(-low / scale), 15.0f);
    if (lane == 0) {
      a.row_scale[i] = (uint16_t)bits;
      if (a.row_zero) a.row_zero[i] = (uint8_t)zero;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t k = k0 + 32 * j + lane;
      if (k >= k1) continue;
      const float q = none ? zero : rintf(v[j] / scale) + zero;
      a.q[n * a.K + k] = (uint8_t)fminf(fmaxf(q, a.row_zero ? 0.0f : 1.0f), 15.0f);
    }
  }
}

// The weights that a layout stands for, rounded to 16 bits.
template <class E>
__global__ void __launch_bounds__(256) k_unpack_i4(I4Unpack a) {
  pdl_enter();
  const int per = groups_in(a.group), tiles = span_of(a.group) / 64;
  const int64_t total = a.N * a.K;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t n = i / a.K, k = i % a.K, kb = k / 64, in = k % 64;
    const int64_t lane = n % 8 * 4 + in % 32 / 8, word = in / 32 * 2 + in % 8 / 4, j = in % 4, half = n % 16 / 8;
    const uint32_t w = a.data[(((n / 16) * a.spans * tiles + kb) * 32 + lane) * 4 + word];
    const int64_t at = scale_at(n, k / a.group, a.spans, per);
    const float q = (float)(w >> (4 * (j / 2 * 2 + half) + 16 * (j % 2)) & 15u) - (a.zero ? (float)a.zero[at] : 8.0f);
    static_cast<uint16_t*>(a.w)[n * a.ldw + k] = (uint16_t)E::from_f32(q * E::to_f32(a.scale[at]));
  }
}

unsigned grid_for(int64_t items, int64_t per, int num_sms) {
  const int64_t want = (items + per - 1) / per, most = (int64_t)num_sms * 16;
  return (unsigned)(want < most ? want : most);
}

template <class E, int GROUP, bool ZERO>
cudaError_t linear(const I4Args& a, cudaStream_t s) {
  const int64_t tiles = (a.N + 15) / 16, runs = (a.M + 31) / 32;
  const bool vec = (reinterpret_cast<uintptr_t>(a.x) & 15u) == 0 && a.ldx % 8 == 0;
#define AR_I4_TOKENS(VEC) \
  (a.M <= 8 ? k_linear_i4<E, GROUP, ZERO, 1, VEC> : a.M <= 16 ? k_linear_i4<E, GROUP, ZERO, 2, VEC> : k_linear_i4<E, GROUP, ZERO, 4, VEC>)
  auto* k = vec ? AR_I4_TOKENS(true) : AR_I4_TOKENS(false);
#undef AR_I4_TOKENS
  return launch_op(k, dim3((unsigned)tiles, (unsigned)runs), kThreads, 0, 1, s, a);
}

template <class E>
cudaError_t linear_group(const I4Args& a, int group, cudaStream_t s) {
  switch (group) {
    case 32: return a.zero ? linear<E, 32, true>(a, s) : linear<E, 32, false>(a, s);
    case 64: return a.zero ? linear<E, 64, true>(a, s) : linear<E, 64, false>(a, s);
    default: return a.zero ? linear<E, 128, true>(a, s) : linear<E, 128, false>(a, s);
  }
}

}  // namespace

int i4_span(int group) { return span_of(group); }

cudaError_t launch_linear_i4(int dtype, int group, const I4Args& a, cudaStream_t s) {
  return dtype == AR_BF16 ? linear_group<Bf16>(a, group, s) : linear_group<F16>(a, group, s);
}

cudaError_t launch_pack_i4(const I4Pack& a, int num_sms, cudaStream_t s) {
  return launch_op(k_pack_i4, dim3(grid_for((a.N + 15) / 16 * a.spans * span_of(a.group) / 2, 256, num_sms)), 256, 0, 1, s, a);
}

cudaError_t launch_quantize_i4(int dtype, const I4Quantize& a, int num_sms, cudaStream_t s) {
  const unsigned grid = grid_for(a.N * ((a.K + a.group - 1) / a.group), 8, num_sms);
  return dtype == AR_BF16 ? launch_op(k_quantize_i4<Bf16>, dim3(grid), 256, 0, 1, s, a)
                          : launch_op(k_quantize_i4<F16>, dim3(grid), 256, 0, 1, s, a);
}

cudaError_t launch_unpack_i4(int dtype, const I4Unpack& a, int num_sms, cudaStream_t s) {
  const unsigned grid = grid_for(a.N * a.K, 256, num_sms);
  return dtype == AR_BF16 ? launch_op(k_unpack_i4<Bf16>, dim3(grid), 256, 0, 1, s, a)
                          : launch_op(k_unpack_i4<F16>, dim3(grid), 256, 0, 1, s, a);
}

}  // namespace ar
