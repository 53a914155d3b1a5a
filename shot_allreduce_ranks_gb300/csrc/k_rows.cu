// Element-wise and row-wise steps of the feed-forward operators: the gradients
// of the two pre-activations, the quantisation of rows to 8 bits, and the copy
// of unaligned rows to where a tensor map can read them.
#include "ops_internal.cuh"

namespace ar {
namespace {

constexpr int kPackThreads = 256, kGateThreads = 256;

struct PackJobs {
  PackJob job[3];
};

// Both 16-bit elements of a word, 0 in the place of an infinity or NaN.
template <class E>
__device__ __forceinline__ uint32_t finite_only(uint32_t w) {
  constexpr uint32_t kExponents = IsBf16<E>::value ? 0x7F807F80u : 0x7C007C00u;
  return w & ~__vcmpeq2(w & kExponents, kExponents);
}

// One matrix's rows, 16 bytes a thread.  E, the type of 16-bit elements, matters
// where rows go to both rows of their token: infinities and NaN go to the first
// alone, since what a value's rounding left may be 0, or of the other sign, and
// with an infinity would make NaN of an infinite sum.
template <int B, class E = F16>
__device__ __forceinline__ void pack_rows(const PackJob& j) {
  constexpr int G = 16 / B;
  const int64_t per_row = (j.cols + G - 1) / G, total = j.rows * per_row, sources = j.twice ? j.twice : j.rows;
  const char* begin = static_cast<const char*>(j.from);
  const char* end = begin + ((sources - 1) * j.ld_from + j.cols) * B;
  for (int64_t i = (int64_t)blockIdx.x * kPackThreads + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * kPackThreads) {
    const int64_t row = total >> 32 ? i / per_row : (int64_t)((uint32_t)i / (uint32_t)per_row);
    const int64_t col = (i - row * per_row) * G;
    const int64_t source = j.twice ? row / 32 * 16 + row % 16 : row;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (source < sources) v = load_anywhere<B>(begin + (source * j.ld_from + col) * B, (j.cols - col) * B, begin, end);
    if (B == 2 && j.twice && row % 32 >= 16)
      v = make_uint4(finite_only<E>(v.x), finite_only<E>(v.y), finite_only<E>(v.z), finite_only<E>(v.w));
    *reinterpret_cast<uint4*>(static_cast<char*>(j.to) + (row * j.ld_to + col) * B) = v;
  }
}

template <int B>
__global__ void __launch_bounds__(kPackThreads) k_pack(const __grid_constant__ PackJobs jobs) {
  pdl_enter();
  pack_rows<B>(jobs.job[blockIdx.y]);
}

// CTAs in x for the largest of the jobs, and the jobs side by side.
int64_t pack_ctas(const PackJob* jobs, int count, int elem_bytes, PackJobs* all) {
  int64_t most = 0;
  for (int i = 0; i < count; ++i) {
    all->job[i] = jobs[i];
    const int64_t g = 16 / elem_bytes, n = jobs[i].rows * ((jobs[i].cols + g - 1) / g);
    most = n > most ? n : most;
  }
  return (most + kPackThreads - 1) / kPackThreads;
}

// dgate = dout * up * act'(gate), dup = dout * act(gate): 3 reads and 2 writes
// an element, bound by memory.  A thread takes eight columns of a row at a
// time; the workspace rows are 16-byte aligned, the caller's need not be.  The
// rows of CTAs past the first copy the operands that the products want laid out:
// neither waits for the other, and a launch costs about 2 us.  512 x 3584: 6 us
// under a profiler from cold caches, of a call's 89.
template <class E, int ACT, bool VEC>
__global__ void __launch_bounds__(kGateThreads)
    k_gate_grad(const char* gate, const char* up, const char* dout, int64_t ldo, char* dgate,
                char* dup, int64_t ldw, int64_t rows, int64_t cols, int64_t groups_per_row,
                int two_parts, const __grid_constant__ PackJobs jobs) {
  pdl_enter();
  if (blockIdx.y > 0) {
    pack_rows<2, E>(jobs.job[blockIdx.y - 1]);
    return;
  }
  const int64_t total = (two_parts ? (rows + 15) / 16 * 16 : rows) * groups_per_row;
  for (int64_t i = (int64_t)blockIdx.x * kGateThreads + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * kGateThreads) {
    const int64_t row = total >> 32 ? i / groups_per_row : (int64_t)((uint32_t)i / (uint32_t)groups_per_row);
    const int64_t col = (i - row * groups_per_row) * 8;
    const int64_t from = (row * ldo + col) * 2;
    const int64_t to = ((two_parts ? two_part_row(row) : row) * ldw + col) * 2;
    const int n = row >= rows ? 0 : (int)(cols - col < 8 ? cols - col : 8);
    uint32_t gw[4] = {}, uw[4] = {}, dw[4] = {};
    if (VEC && n == 8) {
      const uint4 a = ld_v4_stream(gate + from), b = ld_v4_stream(up + from),
                  c = ld_v4_stream(dout + from);
      gw[0] = a.x, gw[1] = a.y, gw[2] = a.z, gw[3] = a.w;
      uw[0] = b.x, uw[1] = b.y, uw[2] = b.z, uw[3] = b.w;
      dw[0] = c.x, dw[1] = c.y, dw[2] = c.z, dw[3] = c.w;
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < n) {
          gw[k >> 1] |= ld_elem<2>(gate + from + 2 * k) << (16 * (k & 1));
          uw[k >> 1] |= ld_elem<2>(up + from + 2 * k) << (16 * (k & 1));
          dw[k >> 1] |= ld_elem<2>(dout + from + 2 * k) << (16 * (k & 1));
        }
    }
    uint32_t og[4], ou[4], rg[4], ru[4];  // rounded, and what that left
    const auto rest = [](float v, float rounded) { return fabsf(rounded) < INFINITY ? v - rounded : 0.0f; };
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float f0, s0, f1, s1;
      act_slope<ACT>(E::lo(gw[k]), f0, s0);
      act_slope<ACT>(E::hi(gw[k]), f1, s1);
      const float d0 = E::lo(dw[k]), d1 = E::hi(dw[k]);
      const float g0 = d0 * E::lo(uw[k]) * s0, g1 = d1 * E::hi(uw[k]) * s1, u0 = d0 * f0, u1 = d1 * f1;
      og[k] = E::pack(g0, g1);
      ou[k] = E::pack(u0, u1);
      rg[k] = E::pack(rest(g0, E::lo(og[k])), rest(g1, E::hi(og[k])));
      ru[k] = E::pack(rest(u0, E::lo(ou[k])), rest(u1, E::hi(ou[k])));
    }
    // The workspace row is longer than cols, up to a whole group at least; what
    // lies past cols is never read.
    st_v4_stream(dgate + to, make_uint4(og[0], og[1], og[2], og[3]));
    st_v4_stream(dup + to, make_uint4(ou[0], ou[1], ou[2], ou[3]));
    if (two_parts) {
      st_v4_stream(dgate + to + 32 * ldw, make_uint4(rg[0], rg[1], rg[2], rg[3]));
      st_v4_stream(dup + to + 32 * ldw, make_uint4(ru[0], ru[1], ru[2], ru[3]));
    }
  }
}

template <class E, int ACT>
cudaError_t gate_grad(const void* gate, const void* up, const void* dout, int64_t ldo, void* dgate,
                      void* dup, int64_t ldw, int64_t rows, int64_t cols, bool two_parts, const PackJob* jobs,
                      int count, int num_sms, cudaStream_t s) {
  const int64_t gpr = (cols + 7) / 8;
  PackJobs all = {};
  const int64_t pack = pack_ctas(jobs, count, 2, &all), gate_ctas = ((rows + 15) * gpr + kGateThreads - 1) / kGateThreads;
  const int64_t want = pack > gate_ctas ? pack : gate_ctas, cap = (int64_t)num_sms * 8;
  const dim3 grid((unsigned)(want < cap ? want : cap), (unsigned)(1 + count));
  const bool vec = ((reinterpret_cast<uintptr_t>(gate) | reinterpret_cast<uintptr_t>(up) |
                     reinterpret_cast<uintptr_t>(dout)) & 15u) == 0 && ldo % 8 == 0;
  auto* k = vec ? k_gate_grad<E, ACT, true> : k_gate_grad<E, ACT, false>;
  return launch_op(k, grid, kGateThreads, 0, 1, s, static_cast<const char*>(gate),
                   static_cast<const char*>(up), static_cast<const char*>(dout), ldo,
                   static_cast<char*>(dgate), static_cast<char*>(dup), ldw, rows, cols, gpr, two_parts ? 1 : 0, all);
}

// ---------------------------------------------------------------------------
constexpr int kQuantThreads = 256;

// Absolute values as unsigned integers are ordered as the floats are, with every
// NaN above infinity, so that a NaN in a row becomes its scale.
template <class E>
__device__ __forceinline__ uint32_t magnitude(uint32_t bits) {
  return __float_as_uint(E::to_f32(bits)) & 0x7FFFFFFFu;
}

// A row's divisor, 1 for a scale of 0, and its reciprocal.
struct Divisor {
  float by, inverse;
  bool finite;  // no infinity or NaN in the row, which gives zeros
  bool exact;   // below 2^-100, where the reciprocal could overflow: always divide
};

// rint(x / s), s = absmax / 127, with the division an IEEE one, rounded once.
__device__ __forceinline__ uint32_t divided(float x, const Divisor& d) {
  return (uint32_t)min(127, max(-127, __float2int_rn(__fdiv_rn(x, d.by)))) & 0xFFu;
}

// The same integers for a group of G values, mostly without dividing.  x times
// the reciprocal is within 127 x 1.5 x 2^-23 < 3e-5 of the quotient, so only next
// to a half can the two round differently, and a group with such a value is
// divided.  Adding 1.5 x 2^23 rounds to an integer, ties to even, and leaves it in
// the low bits.  Divisions alone took 27 us for 4096 x 8192, whose bytes take 15.
template <int G>
__device__ __forceinline__ void quantized(const float (&x)[G], const Divisor& d, uint32_t (&out)[2]) {
  constexpr float kRound = 12582912.0f;
  uint32_t n[G];
  bool near = d.exact;
#pragma unroll
  for (int k = 0; k < G; ++k) {
    const float t = __fmul_rn(x[k], d.inverse), r = __fadd_rn(t, kRound);
    n[k] = __float_as_uint(r) & 0xFFu;
    near = near || fabsf(__fadd_rn(t, -__fadd_rn(r, -kRound))) > 0.5f - 1e-4f;
  }
  if (near) {
#pragma unroll
    for (int k = 0; k < G; ++k) n[k] = divided(x[k], d);
  }
  out[0] = out[1] = 0;
#pragma unroll
  for (int k = 0; k < G; ++k) out[k / 4] |= d.finite ? n[k] << (8 * (k & 3)) : 0u;
}

// LANES threads a row: a warp for short rows, of which a CTA then makes eight,
// else the CTA.  Rows are read once: each thread keeps up to HELD groups of 16
// bytes in registers between the maximum and the division (2048 16-bit columns
// a warp, 8192 a CTA).  HELD = 0, for longer rows and rows that do not start on
// 16 bytes: read twice, an element at a time.  (A CTA for each row of 512
// columns took 16 us for 8192 of them, whose bytes take 2.)
template <class E, int LANES, int HELD>
__global__ void __launch_bounds__(kQuantThreads)
    k_quantize_rows(const char* x, int64_t ldx, int8_t* q, int64_t ldq, float* scale, int64_t rows, int64_t cols) {
  pdl_enter();
  __shared__ uint32_t part[kQuantThreads / 32];
  constexpr int G = E::kGroup, B = E::kBytes, kRows = kQuantThreads / LANES;
  const int lane = threadIdx.x % LANES;
  const int64_t at = (int64_t)blockIdx.x * kRows + threadIdx.x / LANES;
  if (at >= rows) return;  // whole warps: LANES is 32 there
  const char* row = x + at * ldx * B;
  int8_t* to = q + at * ldq;
  uint4 held[HELD ? HELD : 1];
  uint32_t top = 0;
  const auto bits = [](const uint4& v, int k) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    return B == 2 ? (w[k / 2] >> (16 * (k & 1))) & 0xFFFFu : w[k & 3];
  };
  const int groups = HELD ? (int)(cols / G) : 0;  // whole ones: the columns left are read below
#pragma unroll
  for (int i = 0; i < HELD; ++i) {
    const int g = lane + i * LANES;
    held[i] = g < groups ? ld_v4_stream(row + (int64_t)g * 16) : make_uint4(0, 0, 0, 0);
  }
  // 16-bit types' magnitudes are ordered as integers too: two at a time.
  uint32_t pair = 0;
#pragma unroll
  for (int i = 0; i < HELD; ++i) {
    const uint32_t w[4] = {held[i].x, held[i].y, held[i].z, held[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (B == 2)
        pair = __vmaxu2(pair, w[k] & 0x7FFF7FFFu);
      else
        top = max(top, magnitude<E>(w[k]));
    }
  }
  if (B == 2) top = magnitude<E>(max(pair & 0xFFFFu, pair >> 16));
  const int64_t rest = (int64_t)groups * G;
  for (int64_t c = rest + lane; c < cols; c += LANES) top = max(top, magnitude<E>(ld_elem<B>(row + c * B)));
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  if (LANES > 32) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kQuantThreads / 32; ++w) top = max(top, part[w]);
  }
  const float s = __fdiv_rn(__uint_as_float(top), 127.0f);
  if (lane == 0) scale[at] = s;
  Divisor by;
  by.by = s > 0.0f ? s : 1.0f;
  by.inverse = __frcp_rn(by.by);
  by.finite = top < 0x7F800000u;
  by.exact = by.by < 7.9e-31f;
#pragma unroll
  for (int i = 0; i < HELD; ++i) {
    const int g = lane + i * LANES;
    if (g >= groups) break;
    float v[G];
#pragma unroll
    for (int k = 0; k < G; ++k) v[k] = E::to_f32(bits(held[i], k));
    uint32_t w[2];
    quantized<G>(v, by, w);
    if (G == 8)
      *reinterpret_cast<uint2*>(to + (int64_t)g * G) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint32_t*>(to + (int64_t)g * G) = w[0];
  }
  for (int64_t c = rest + lane; c < cols; c += LANES) {
    const uint32_t n = divided(E::to_f32(ld_elem<B>(row + c * B)), by);
    to[c] = (int8_t)(by.finite ? n : 0u);
  }
}

template <class E>
cudaError_t quantize(const void* x, int64_t ldx, int8_t* q, int64_t ldq, float* scale, int64_t rows, int64_t cols,
                     int num_sms, cudaStream_t s) {
  constexpr int64_t G = E::kGroup;
  const bool aligned = reinterpret_cast<uintptr_t>(x) % 16 == 0 && reinterpret_cast<uintptr_t>(q) % G == 0 &&
                       (rows == 1 || (ldx % G == 0 && ldq % G == 0));
  // A warp a row where that fills the SMs (440 rows of 2048: 5.4 us by warps, 3.0
  // by CTAs; 3104: 8.6 and 9.8).
  const bool warp = aligned && cols <= 8 * 32 * G && rows > 8 * num_sms;
  const bool held = aligned && cols <= 4 * kQuantThreads * G;
  const dim3 grid((unsigned)(warp ? (rows + kQuantThreads / 32 - 1) / (kQuantThreads / 32) : rows));
  return launch_op(warp   ? k_quantize_rows<E, 32, 8>
                   : held ? k_quantize_rows<E, kQuantThreads, 4>
                          : k_quantize_rows<E, kQuantThreads, 0>,
                   grid, kQuantThreads, 0, 1, s, static_cast<const char*>(x), ldx, q, ldq, scale, rows, cols);
}

}  // namespace

cudaError_t launch_pack(const PackJob* jobs, int count, int elem_bytes, int num_sms, cudaStream_t s) {
  PackJobs all = {};
  const int64_t want = pack_ctas(jobs, count, elem_bytes, &all), cap = (int64_t)num_sms * 8;
  const dim3 grid((unsigned)(want < cap ? want : cap), (unsigned)count);
  return launch_op(elem_bytes == 2 ? k_pack<2> : k_pack<1>, grid, kPackThreads, 0, 1, s, all);
}

cudaError_t launch_gate_grad(int dtype, int act, const void* gate, const void* up, const void* dout,
                             int64_t ldo, void* dgate, void* dup, int64_t ldw, int64_t rows,
                             int64_t cols, bool two_parts, const PackJob* jobs, int count, int num_sms,
                             cudaStream_t s) {
  if (dtype == AR_BF16)
    return act == AR_ACT_SILU
               ? gate_grad<Bf16, AR_ACT_SILU>(gate, up, dout, ldo, dgate, dup, ldw, rows, cols, two_parts, jobs, count, num_sms, s)
               : gate_grad<Bf16, AR_ACT_GELU_TANH>(gate, up, dout, ldo, dgate, dup, ldw, rows, cols, two_parts, jobs, count, num_sms, s);
  return act == AR_ACT_SILU
             ? gate_grad<F16, AR_ACT_SILU>(gate, up, dout, ldo, dgate, dup, ldw, rows, cols, two_parts, jobs, count, num_sms, s)
             : gate_grad<F16, AR_ACT_GELU_TANH>(gate, up, dout, ldo, dgate, dup, ldw, rows, cols, two_parts, jobs, count, num_sms, s);
}

cudaError_t launch_quantize_rows(int dtype, const void* x, int64_t ldx, int8_t* q, int64_t ldq,
                                 float* scale, int64_t rows, int64_t cols, int num_sms, cudaStream_t s) {
  if (dtype == AR_BF16) return quantize<Bf16>(x, ldx, q, ldq, scale, rows, cols, num_sms, s);
  if (dtype == AR_FP16) return quantize<F16>(x, ldx, q, ldq, scale, rows, cols, num_sms, s);
  return quantize<F32>(x, ldx, q, ldq, scale, rows, cols, num_sms, s);
}

}  // namespace ar
