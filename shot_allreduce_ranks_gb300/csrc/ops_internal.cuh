// Declarations shared by the feed-forward operators' translation units: the
// gated feed-forward shard and its gradients, the 8-bit product, dropout.
// Their entry points and contracts are in include/ar.h.
#pragma once

#include <atomic>

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

// The same for a kernel whose dynamic shared memory changes from call to call and may pass 48 KB.  The limit is
// state of the kernel on the device, which calls from other host threads share: it is raised to all that
// a block can have, once for each device, and never set to a call's own size.
template <auto K, class... A>
cudaError_t launch_raised(dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
  static std::atomic<bool> raised[64];  // by device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !raised[dev].load(std::memory_order_acquire)) {
    cudaFuncAttributes own;
    int most = 0;
    e = cudaFuncGetAttributes(&own, K);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, most - (int)own.sharedSizeBytes);
    if (e != cudaSuccess) return e;
    if (dev < 64) raised[dev].store(true, std::memory_order_release);
  }
  return launch_op(K, grid, threads, smem, 1, s, args...);
}

// ---------------------------------------------------------------------------
// Checks that the entry points share.
constexpr size_t kMaxElems = (size_t)1 << 40;  // of a matrix: more than the memory holds

inline bool half_type(int dtype) { return dtype == AR_BF16 || dtype == AR_FP16; }
inline bool any_type(int dtype) { return half_type(dtype) || dtype == AR_FP32; }
inline ar_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? AR_OK : AR_ERR_CUDA; }
inline bool bad_matrix(const void* p, size_t rows, size_t cols, size_t ld) {
  return !p || ld < cols || ld > kMaxElems || (ld && rows > kMaxElems / ld);
}
inline bool misaligned(const void* p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes != 0; }
constexpr int64_t kMostSms = 160;  // bounds scratch memory that is sized without a device
ar_status_t current_sms(int* sms);  // SMs of the current device, looked up once for each

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
// Norms and the residual (k_norm.cu).  Absent arrays are null.
struct NormArgs {
  const void *x, *residual, *gate, *after_weight, *after_bias, *weight, *bias;
  void *r, *y;
  int64_t ldx, ldres, ldg, ldr, ldy;
  int64_t rows, cols, gate_run;  // gate_run: rows of one gate row
  int64_t gate_extent;           // elements from the gate's first to behind its last
  float eps, alpha, offset;
  int layer;
};
cudaError_t launch_norm(int dtype, const NormArgs& a, int num_sms, cudaStream_t s);

// The sums over rows that the backward pass makes, in the order of their parts.
enum NormSum : int { kSumWeight = 0, kSumBias, kSumAfterWeight, kSumAfterBias, kSumGate, kNormSums };

struct NormGradArgs {
  const void *dy, *dr, *x, *r, *gate, *after_weight, *after_bias, *weight;
  void *dx, *dresidual;
  void* sum[kNormSums];    // outputs
  float* part[kNormSums];  // a row of cols floats for every CTA; null where sum is
  int64_t lddy, lddr, ldx, ldr, ldg, lddx, lddres, lddg;
  int64_t rows, cols, gate_rows, gate_run;  // gate_rows is 1 and gate_run is rows where there is no gate
  // How the rows are dealt out: with `split` CTAs to each gate row (1 or more),
  // or (split = 0) with several whole gate rows to each of `ctas` CTAs.
  int64_t ctas, split, chunk;  // chunk: rows of a CTA where split > 0
  int sums_at;  // bytes of shared memory before the sums that are kept there
  int direct;   // the one CTA writes the sums itself: there are no parts to join
  float eps, alpha, offset;
  int layer;
};
// CTAs of the backward pass at most, a row of the parts each, which bounds scratch memory without a device: four
// an SM up to 4,096 columns, two up to 8,192, else one, and no more than rows.  Where an SM would hold more (narrow rows
// without a branch, the kernel for any row), the launch is held to it.
int64_t norm_parts(int64_t rows, int64_t cols);
cudaError_t launch_norm_grad(int dtype, NormGradArgs& a, int num_sms, cudaStream_t s);

// ---------------------------------------------------------------------------
// 4-bit weights (k_i4.cu).  spans: runs of max(group, 64) along k.
struct I4Args {
  const void *x, *data, *scale;
  const uint8_t* zero;  // or null: 8
  void* y;
  int64_t ldx, ldy, M, N, K, spans;
};
cudaError_t launch_linear_i4(int dtype, int group, const I4Args& a, cudaStream_t s);
int i4_span(int group);

struct I4Pack {
  const uint8_t* q;
  const uint16_t* row_scale;  // 16 bits of either type
  const uint8_t* row_zero;
  uint4* data;
  uint16_t* scale;
  uint8_t* zero;
  int64_t ldq, lds, ldz, N, K, spans;
  int group;
};
cudaError_t launch_pack_i4(const I4Pack& a, int num_sms, cudaStream_t s);

struct I4Quantize {
  const void* w;
  uint8_t* q;
  uint16_t* row_scale;
  uint8_t* row_zero;  // null: symmetric
  int64_t ldw, N, K;
  int group;
};
cudaError_t launch_quantize_i4(int dtype, const I4Quantize& a, int num_sms, cudaStream_t s);

struct I4Unpack {
  const uint32_t* data;
  const uint16_t* scale;
  const uint8_t* zero;
  void* w;
  int64_t ldw, N, K, spans;
  int group;
};
cudaError_t launch_unpack_i4(int dtype, const I4Unpack& a, int num_sms, cudaStream_t s);

// ---------------------------------------------------------------------------
// Gated feed-forward experts for at most AR_FEW_TOKENS tokens (k_moe.cu).
struct MoeArgs {
  const void *x, *logits, *w_gate, *w_up, *w_down;
  void *h, *out;   // h: row t * top_k + j for choice j of token t, rows on 16 bytes
  void* h_rest;    // like h: what h's rounding left; null where h is one number of 16 bits
  uint32_t* done;  // of each 16 columns of out: the parts that are there
  float* parts;    // two for every CTA, [AR_FEW_TOKENS][16]
  int32_t* out_expert;
  float* out_weight;  // of the routing, or null
  int64_t ldx, ldl, ldw, esw, ldd, esd, ldh, ldo;  // es: elements from one expert's matrix to the next
  int64_t hidden, width;
  int tokens, experts, first, local, top_k, normalize, logits_dtype;
};
// The scratch memory's size, and (m not null) its pieces in place; two_parts: with h_rest, behind all else.
size_t moe_scratch(int64_t tokens, int64_t top_k, int64_t width, int64_t hidden, bool two_parts, MoeArgs* m, char* base);
cudaError_t launch_moe(int dtype, int act, const MoeArgs& m, int num_sms, cudaStream_t s);

// ---------------------------------------------------------------------------
// Activations.  Both are v * sigmoid(s(v)): s(v) = v for SiLU, and for the
// tanh form of GELU s(v) = 2 sqrt(2/pi) (v + 0.044715 v^3), because
// (1 + tanh t) / 2 = sigmoid(2 t).  __expf and __fdividef leave the sigmoid good to (8 + 2 |s|) units in 2^-23 of its
// value, below the 16-bit results' rounding also where s is far below 0 (at -40, where it is 4e-18, 2^-16.5).
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
      const uint32_t v = B == 1 ? *reinterpret_cast<const uint8_t*>(p + i) : ld_elem<B == 1 ? 2 : B>(p + B * i);
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
