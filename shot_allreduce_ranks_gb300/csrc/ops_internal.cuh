// Declarations shared by the feed-forward operators' translation units: the
// gated feed-forward shard and its gradients, the 8-bit product, dropout.
// Their entry points and contracts are in include/ar.h.
#pragma once

#include "ar_internal.cuh"

namespace ar {

// ---------------------------------------------------------------------------
// Launch of one of these operators' kernels, each of which calls pdl_enter()
// before it touches global memory: with programmatic dependent launch its
// launch and set-up overlap the end of the kernel before (AR_PDL=0 turns it
// off, as for the collectives).
bool ops_pdl();

template <class... P, class... A>
cudaError_t launch_op(void (*kernel)(P...), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t s, A... args) {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = plain_config({0, threads, ops_pdl()}, grid, smem, s, attr);
  if (cluster > 1) {
    cudaLaunchAttribute& a = attr[cfg.numAttrs++];
    a.id = cudaLaunchAttributeClusterDimension;
    a.val.clusterDim.x = (unsigned)cluster;
    a.val.clusterDim.y = a.val.clusterDim.z = 1;
  }
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// ---------------------------------------------------------------------------
// Matrix products.  All of them are C[m, n] = sum_k A(m, k) B(n, k); what
// differs is which matrices stand for A and B, which of their two axes is
// contiguous, and what is done with the sum.
enum GemmMode : int {
  // A = x [M, K], B = both projections' weights [N, K]:
  // h = act(gate) * up, with gate and up stored where c1 is set.
  kGemmGated = 0,
  // A = {dgate, dup} [M, K], B = {Wgate, Wup} [K, N]: the sum of both products.
  kGemmDx = 1,
  // A = dgate then dup, [K, M] each, B = x [K, N]: two outputs of M rows.
  kGemmDw = 2,
  // A = int8 [M, K], B = int8 [N, K]: sm[m] * sn[n] * sum.
  kGemmI8 = 3
};

struct GemmArgs {
  const void* a0;
  const void* a1;
  const void* b0;
  const void* b1;
  void* c0;
  void* c1;
  void* c2;
  const float* sm;
  const float* sn;
  int64_t lda, ldb, ldb1, ldc;  // elements between rows (ldb1: b1's)
  int64_t M, N, K;
  int act;                // ar_activation_t (kGemmGated)
  // kGemmDx on two-part rows (see launch_gate_grad): the tokens, whose results are
  // the sums of both parts' rows; 0: rows are tokens.
  int64_t tokens;
};

// On tcgen05, for operands that a tensor map can describe; gemm_tc_error reads
// and clears the flag that a wait which gave up leaves on the device.
bool gemm_tc_takes(int mode, const GemmArgs& g);
cudaError_t launch_gated_tc(int dtype, const GemmArgs& g, int num_sms, cudaStream_t s);
cudaError_t launch_grad_tc(int dtype, const GemmArgs* dx, const GemmArgs* dw, int num_sms, cudaStream_t s);  // null: absent
cudaError_t gemm_tc_error(cudaStream_t s, uint32_t* error);

cudaError_t take_error_word(void* p, cudaStream_t s, uint32_t* error);  // reads and clears

// The gated product on tcgen05 for at most 128 tokens.
bool gemm_mid_takes(int mode, const GemmArgs& g);
cudaError_t launch_gemm_mid(int dtype, const GemmArgs& g, int num_sms, cudaStream_t s);
cudaError_t gemm_mid_error(cudaStream_t s, uint32_t* error);

// The 8-bit product on tcgen05.
bool gemm_i8_takes(int mode, const GemmArgs& g);
cudaError_t launch_gemm_i8(int dtype, const GemmArgs& g, int num_sms, cudaStream_t s);
cudaError_t gemm_i8_error(cudaStream_t s, uint32_t* error);

// For at most 32 tokens of the gated and the 8-bit product.
bool gemm_few_takes(int mode, const GemmArgs& g);
cudaError_t launch_gemm_few(int mode, int dtype, const GemmArgs& g, cudaStream_t s);

// On mma.sync, for any alignment and stride.
cudaError_t launch_gemm_any(int mode, int dtype, const GemmArgs& g, cudaStream_t s);

// One int8 row and one scale for each row of x.
cudaError_t launch_quantize_rows(int dtype, const void* x, int64_t ldx, int8_t* q, int64_t ldq,
                                 float* scale, int64_t rows, int64_t cols, int num_sms, cudaStream_t s);

// Copies up to three matrices to rows that start on 16 bytes.
struct PackJob {
  const void* from;
  void* to;
  int64_t rows, cols, ld_from, ld_to;  // elements
  int64_t twice;  // 0, or the source's rows, each copied to both rows of its token in two-part rows (see pack_rows)
};
cudaError_t launch_pack(const PackJob* jobs, int count, int elem_bytes, int num_sms, cudaStream_t s);

// dgate = dout * up * act'(gate), dup = dout * act(gate), the operands of the
// tensor cores' products, rounded to the element type; and the copies of `jobs`,
// 16-bit matrices, in the same launch.
// two_parts: each value as the sum of two numbers of the element type, the
// second what the first's rounding left, so that about 16 (bfloat16) or 22
// (float16) bits reach the products.  Token t's first parts are row 32 (t / 16) + t % 16, its
// second parts 16 rows on; rows without a token are zeros.
constexpr int64_t two_part_rows(int64_t tokens) { return (tokens + 15) / 16 * 32; }
__host__ __device__ constexpr int64_t two_part_row(int64_t t) { return (t / 16) * 32 + t % 16; }
cudaError_t launch_gate_grad(int dtype, int act, const void* gate, const void* up, const void* dout,
                             int64_t ldo, void* dgate, void* dup, int64_t ldw, int64_t rows,
                             int64_t cols, bool two_parts, const PackJob* jobs, int count, int num_sms,
                             cudaStream_t s);

struct DropoutArgs {
  const void* x;
  const void* residual;  // or null
  void* out;
  int64_t ldx, ldr, ldo;
  int64_t rows, cols;
  uint64_t seed, sequence, offset;
  uint32_t threshold;  // an element is kept where its draw >= threshold
  int drop_all;
  float scale;
};
cudaError_t launch_dropout(int dtype, const DropoutArgs& a, int num_sms, cudaStream_t s);

// ---------------------------------------------------------------------------
// Activations.  Both are v * sigmoid(s(v)): s(v) = v for SiLU, and for the
// tanh form of GELU s(v) = 2 sqrt(2/pi) (v + 0.044715 v^3), because
// (1 + tanh t) / 2 = sigmoid(2 t).  __expf and __fdividef are good to a few
// units in 2^-23 here, far below the 16-bit results' rounding.
__device__ __forceinline__ float sigmoid_fast(float s) {
  return __fdividef(1.0f, 1.0f + __expf(-s));
}

constexpr float kGeluTwoC = 1.5957691216057308f;  // 2 sqrt(2/pi)
constexpr float kGeluA = 0.044715f;

template <int ACT>
__device__ __forceinline__ float act_value(float v) {
  if (ACT == AR_ACT_SILU) return v * sigmoid_fast(v);
  return v * sigmoid_fast(kGeluTwoC * (v + kGeluA * v * v * v));
}

// act(v) and act'(v).  Past |v| = 88 the sigmoid is 0 or 1 and its slope 0 in
// fp32, so the slope is taken at the clamped value, where v^3 and v (1 - sig)
// stay finite; a NaN passes through the comparisons.
template <int ACT>
__device__ __forceinline__ void act_slope(float v, float& f, float& df) {
  float c = v > 88.0f ? 88.0f : v;
  c = c < -88.0f ? -88.0f : c;
  if (ACT == AR_ACT_SILU) {
    const float sig = sigmoid_fast(c);
    f = v * sig;
    df = sig * (1.0f + c * (1.0f - sig));
  } else {
    const float sig = sigmoid_fast(kGeluTwoC * (c + kGeluA * c * c * c));
    f = v * sig;
    df = sig + c * sig * (1.0f - sig) * kGeluTwoC * (1.0f + 3.0f * kGeluA * c * c);
  }
}

// 16 bytes that begin o bytes into the aligned 32 of u and v.
__device__ __forceinline__ uint4 shift_window(const uint4& u, const uint4& v, uint32_t o) {
  const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
  uint32_t by8[6], by4[5], r[4];
#pragma unroll
  for (int i = 0; i < 6; ++i) by8[i] = o & 8 ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) by4[i] = o & 4 ? by8[i + 1] : by8[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = __funnelshift_r(by4[i], by4[i + 1], 8 * (o & 3));
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// 16 bytes at p, which may lie anywhere: the two aligned 16-byte pieces around
// them, shifted into place.  `left` of them may be read, the rest is zero; what
// would touch memory before `begin` or from `end` on (a matrix's first and last
// elements) is read an element of B bytes at a time.
template <int B>
__device__ __forceinline__ uint4 load_anywhere(const char* p, int64_t left, const char* begin, const char* end) {
  const uint32_t o = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u);
  const uint4* base = reinterpret_cast<const uint4*>(p - o);
  if (left >= 16 && p - o >= begin && p - o + 32 <= end) return shift_window(__ldg(base), __ldg(base + 1), o);
  uint32_t w[4] = {};
#pragma unroll
  for (int i = 0; i < 16 / B; ++i)
    if (i * B < left) {
      const uint32_t v = B == 2 ? ld_elem<2>(p + 2 * i) : *reinterpret_cast<const uint8_t*>(p + i);
      w[i * B / 4] |= v << (8 * (i * B % 4));
    }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A 16-bit type's two-element word and its mma.sync.
template <class E>
struct IsBf16 {
  static constexpr bool value = false;
};
template <>
struct IsBf16<Bf16> {
  static constexpr bool value = true;
};

// D (16x8, fp32) += A (16x16) B (16x8); lane l holds rows l/4 and l/4 + 8.
template <class E>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4],
                                          const uint32_t (&b)[2]) {
  if (IsBf16<E>::value) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
  }
}

// Four int8 to four fp16: a byte b + 128 under the exponent of 1024 is the
// fp16 number 1152 + b, exactly; one subtraction leaves b.
__device__ __forceinline__ void i8_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  uint32_t a, b;
  asm("prmt.b32 %0, %1, %2, 0x4140;" : "=r"(a) : "r"(u), "r"(0x64646464u));
  asm("prmt.b32 %0, %1, %2, 0x4342;" : "=r"(b) : "r"(u), "r"(0x64646464u));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
}

}  // namespace ar
