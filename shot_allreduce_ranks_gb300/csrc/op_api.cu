// C ABI of the feed-forward operators: argument checks, workspaces and the
// choice of kernel.  Declarations and contracts are in include/ar.h.
#include <math.h>
#include <stdlib.h>
#include <string.h>

#include <new>

#include "ops_internal.cuh"

struct ar_ffn_ctx {
  size_t max_tokens = 0, hidden = 0, width = 0;
  int dtype = AR_BF16, act = AR_ACT_SILU;
  int num_sms = 0;
  size_t ldw = 0;         // workspace leading dimension: width rounded up to 128 bytes
  size_t ldx = 0;         // hidden rounded up likewise
  size_t rows = 0;        // of dgate and of dup
  char* work = nullptr;   // dgate, dup: rows x ldw each; x for two-part rows: up to 128 x ldx
};

namespace {

constexpr int kMaxDevices = 64;
constexpr size_t kMaxElems = (size_t)1 << 40;  // of a matrix: more than the memory holds
constexpr size_t kMaxSize = (size_t)1 << 30;  // the sizes a handle is made for
// Up to this many tokens the gradients of the pre-activations reach the products
// in two parts: with few values the rounding of each shows most.  In dx the second
// parts fill rows of a tile that are idle otherwise; in the weights' gradients they
// are more k, a second step from 33 tokens on, and x is copied beside both.  8192 ->
// 3584, two parts against one: 8 and 16 tokens 50.1 against 50.6 us, 17 and 32 50.5
// against 49.8, 33 to 64 51.0 against 49.5.
constexpr size_t kTwoPartTokens = 64;
// Up to this many tokens a forward product reads the weights once, where they
// are: laying them out first costs two passes more.
constexpr size_t kFewTokens = AR_FEW_TOKENS;

bool half_type(int dtype) { return dtype == AR_BF16 || dtype == AR_FP16; }
bool any_type(int dtype) { return half_type(dtype) || dtype == AR_FP32; }

ar_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? AR_OK : AR_ERR_CUDA; }

// SMs of the current device, looked up once for each.
ar_status_t current_sms(int* sms) {
  static int known[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return AR_ERR_CUDA;
  if (dev >= 0 && dev < kMaxDevices && known[dev] > 0) {
    *sms = known[dev];
    return AR_OK;
  }
  if (cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return AR_ERR_CUDA;
  if (dev >= 0 && dev < kMaxDevices) known[dev] = *sms;
  return AR_OK;
}

bool bad_matrix(const void* p, size_t rows, size_t cols, size_t ld) {
  return !p || ld < cols || ld > kMaxElems || (ld && rows > kMaxElems / ld);
}

bool misaligned(const void* p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes != 0; }

// A matrix with its row stride; packed rows take the place of ones that do not
// start on 16 bytes where the caller gave scratch memory for them.
struct Rows {
  const void* p;
  size_t rows, cols, ld;
};

bool on_16(const Rows& r, size_t elem) { return !misaligned(r.p, 16) && r.ld * elem % 16 == 0; }
// Packed rows start on 128 bytes, so that a box's rows of 128 bytes are whole
// cache lines.
size_t packed_ld(const Rows& r, size_t elem) { return (r.cols * elem + 127) / 128 * 128 / elem; }

// Bytes that packing takes: 0 where every matrix can be read as it is.
size_t pack_bytes(const Rows* m, int count, size_t elem) {
  size_t bytes = 0;
  for (int i = 0; i < count; ++i)
    if (!on_16(m[i], elem)) bytes += m[i].rows * packed_ld(m[i], elem) * elem;
  return bytes;
}

// Points such matrices at their place in scratch and lists the copies.
ar_status_t plan_pack(Rows* m, int count, size_t elem, void* scratch, size_t scratch_bytes, ar::PackJob* jobs, int* n) {
  const size_t need = pack_bytes(m, count, elem);
  *n = 0;
  if (need == 0 || !scratch) return AR_OK;
  if (misaligned(scratch, 16) || scratch_bytes < need) return AR_ERR_INVALID_ARG;
  char* to = static_cast<char*>(scratch);
  for (int i = 0; i < count; ++i) {
    if (on_16(m[i], elem)) continue;
    const size_t ld = packed_ld(m[i], elem);
    jobs[(*n)++] = {m[i].p, to, (int64_t)m[i].rows, (int64_t)m[i].cols, (int64_t)m[i].ld, (int64_t)ld, 0};
    m[i].p = to;
    m[i].ld = ld;
    to += m[i].rows * ld * elem;
  }
  return AR_OK;
}

ar_status_t pack(Rows* m, int count, size_t elem, void* scratch, size_t scratch_bytes, int num_sms, cudaStream_t s) {
  ar::PackJob jobs[3];
  int n = 0;
  if (ar_status_t st = plan_pack(m, count, elem, scratch, scratch_bytes, jobs, &n)) return st;
  return n ? cuda_status(ar::launch_pack(jobs, n, (int)elem, num_sms, s)) : AR_OK;
}

// Which kernel makes a forward product.  Up to 32 tokens the weights can be streamed
// past them by mma.sync, whose time grows with every eight tokens; the tensor
// cores' form for some tens of tokens costs about 2 us more to set up but
// stays flat: it takes over where tokens x width x hidden passes 2^26 (16 tokens
// of 2048 x 1024: 3.6 against 5.1 us, of 2048 x 2048: 5.4 against 5.2; 32 tokens
// of 2048 x 1024: 4.8 against 5.5, of 2048 x 2048: 7.1 against 5.5), but not
// for the eight tokens of one instruction (8192 x 3584: 21.3 against 22.3 us).
// The 8-bit product likewise, at 2^28 and past 16 tokens (24 tokens of 5120 x
// 2048: 8.3 against 8.4 us, of 8192 x 3584: 16.4 against 12.2; 16 tokens of that:
// 11.9 against 11.5, of 2048 x 8192: 8.1 against 11.3).
cudaError_t gemm(int mode, int dtype, const ar::GemmArgs& g, int num_sms, cudaStream_t s) {
  const bool mid = ar::gemm_mid_takes(mode, g), i8 = ar::gemm_i8_takes(mode, g);
  const double work = (double)g.M * (double)g.N * (double)g.K;
  if (ar::gemm_few_takes(mode, g) && ((!mid && !i8) || (mid ? g.M <= 8 || work <= (double)(1 << 26)
                                                           : g.M <= 16 || work <= (double)(1 << 28))))
    return ar::launch_gemm_few(mode, dtype, g, s);
  if (mid) return ar::launch_gemm_mid(dtype, g, num_sms, s);
  if (ar::gemm_tc_takes(mode, g)) return ar::launch_gated_tc(dtype, g, num_sms, s);
  if (i8) return ar::launch_gemm_i8(dtype, g, num_sms, s);
  return ar::launch_gemm_any(mode, dtype, g, s);
}

// x, w_gate, w_up of a call.
void operands(const ar_ffn_ctx* h, const void* x, size_t ldx, const void* w_gate, const void* w_up, size_t ldw,
              size_t tokens, Rows (&m)[3]) {
  m[0] = {x, tokens, h->hidden, ldx};
  m[1] = {w_gate, h->width, h->hidden, ldw};
  m[2] = {w_up, h->width, h->hidden, ldw};
}

ar_status_t dropout_call(const void* x, size_t ldx, const void* res, size_t ldr, void* out,
                         size_t ldo, size_t rows, size_t cols, int dtype, double p, uint64_t seed,
                         uint64_t sequence, uint64_t offset, void* stream) {
  if (!any_type(dtype)) return AR_ERR_UNSUPPORTED;
  if (!(p >= 0.0 && p <= 1.0)) return AR_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return AR_OK;
  if (bad_matrix(x, rows, cols, ldx) || bad_matrix(out, rows, cols, ldo) ||
      (res && bad_matrix(res, rows, cols, ldr)) || offset + (uint64_t)rows * cols < offset)
    return AR_ERR_INVALID_ARG;
  const size_t e = dtype == AR_FP32 ? 4 : 2;
  if (misaligned(x, e) || misaligned(out, e) || misaligned(res, e)) return AR_ERR_INVALID_ARG;
  int sms = 0;
  if (ar_status_t st = current_sms(&sms)) return st;
  ar::DropoutArgs a = {};
  a.x = x, a.residual = res, a.out = out;
  a.ldx = (int64_t)ldx, a.ldr = (int64_t)ldr, a.ldo = (int64_t)ldo;
  a.rows = (int64_t)rows, a.cols = (int64_t)cols;
  a.seed = seed, a.sequence = sequence, a.offset = offset;
  const double t = nearbyint(p * 4294967296.0);
  a.drop_all = t >= 4294967296.0;
  a.threshold = a.drop_all ? 0xFFFFFFFFu : (uint32_t)t;
  a.scale = a.drop_all ? 0.0f : (float)(1.0 / (1.0 - p));
  return cuda_status(ar::launch_dropout(dtype, a, sms, static_cast<cudaStream_t>(stream)));
}

}  // namespace

bool ar::ops_pdl() {
  static const bool on = [] {
    const char* v = getenv("AR_PDL");
    return !(v && strcmp(v, "0") == 0);
  }();
  return on;
}

extern "C" {

ar_status_t ar_ffn_create(size_t max_tokens, size_t hidden, size_t width, int dtype,
                          int activation, int train, ar_ffn_t* out) {
  if (!out) return AR_ERR_INVALID_ARG;
  *out = nullptr;
  if (max_tokens < 1 || max_tokens > kMaxSize || hidden < 1 || hidden > kMaxSize || width < 1 ||
      width > kMaxSize || (activation != AR_ACT_SILU && activation != AR_ACT_GELU_TANH))
    return AR_ERR_INVALID_ARG;
  if (!half_type(dtype)) return AR_ERR_UNSUPPORTED;
  int dev = 0, major = 0, minor = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
    return AR_ERR_CUDA;
  if (major != 10 || minor != 3) return AR_ERR_UNSUPPORTED;
  if (ar_status_t st = current_sms(&sms)) return st;
  ar_ffn_ctx* h = new (std::nothrow) ar_ffn_ctx;
  if (!h) return AR_ERR_OOM;
  h->max_tokens = max_tokens, h->hidden = hidden, h->width = width;
  h->dtype = dtype, h->act = activation, h->num_sms = sms;
  h->ldw = (width + 63) / 64 * 64;
  h->ldx = (hidden + 63) / 64 * 64;
  if (train) {
    const size_t two = (size_t)ar::two_part_rows((int64_t)(max_tokens < kTwoPartTokens ? max_tokens : kTwoPartTokens));
    h->rows = max_tokens > two ? max_tokens : two;
    const cudaError_t e = cudaMalloc(reinterpret_cast<void**>(&h->work), 4 * h->rows * h->ldw + 2 * two * h->ldx);
    if (e != cudaSuccess) {
      cudaGetLastError();
      delete h;
      return e == cudaErrorMemoryAllocation ? AR_ERR_OOM : AR_ERR_CUDA;
    }
  }
  *out = h;
  return AR_OK;
}

ar_status_t ar_ffn_destroy(ar_ffn_t h) {
  if (!h) return AR_OK;
  ar_status_t st = AR_OK;
  if (h->work && (cudaDeviceSynchronize() != cudaSuccess || cudaFree(h->work) != cudaSuccess))
    st = AR_ERR_CUDA;
  delete h;
  return st;
}

size_t ar_ffn_scratch_bytes(ar_ffn_t h, const void* x, size_t ldx, const void* w_gate, const void* w_up,
                            size_t ldw, size_t tokens) {
  if (!h) return 0;
  Rows m[3];
  operands(h, x, ldx, w_gate, w_up, ldw, tokens, m);
  return pack_bytes(m, 3, 2);
}

ar_status_t ar_ffn_forward(ar_ffn_t h, const void* x, size_t ldx, const void* w_gate,
                           const void* w_up, size_t ldw, void* out, void* gate, void* up,
                           size_t ldo, size_t tokens, void* scratch, size_t scratch_bytes,
                           void* stream) {
  if (!h || (gate == nullptr) != (up == nullptr)) return AR_ERR_INVALID_ARG;
  if (tokens == 0) return AR_OK;
  if (bad_matrix(x, tokens, h->hidden, ldx) || bad_matrix(w_gate, h->width, h->hidden, ldw) ||
      bad_matrix(w_up, h->width, h->hidden, ldw) || bad_matrix(out, tokens, h->width, ldo) ||
      misaligned(x, 2) || misaligned(w_gate, 2) || misaligned(w_up, 2) || misaligned(out, 2) ||
      misaligned(gate, 2) || misaligned(up, 2))
    return AR_ERR_INVALID_ARG;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  Rows m[3];
  operands(h, x, ldx, w_gate, w_up, ldw, tokens, m);
  if (tokens > kFewTokens)
    if (ar_status_t st = pack(m, 3, 2, scratch, scratch_bytes, h->num_sms, s)) return st;
  ar::GemmArgs g = {};
  g.a0 = m[0].p, g.lda = (int64_t)m[0].ld;
  g.b0 = m[1].p, g.b1 = m[2].p, g.ldb = (int64_t)m[1].ld, g.ldb1 = (int64_t)m[2].ld;
  g.c0 = out, g.c1 = gate, g.c2 = up, g.ldc = (int64_t)ldo;
  g.M = (int64_t)tokens, g.N = (int64_t)h->width, g.K = (int64_t)h->hidden;
  g.act = h->act;
  return cuda_status(gemm(ar::kGemmGated, h->dtype, g, h->num_sms, s));
}

ar_status_t ar_ffn_backward(ar_ffn_t h, const void* x, size_t ldx, const void* w_gate,
                            const void* w_up, size_t ldw, const void* gate, const void* up,
                            const void* dout, size_t ldo, void* dx, size_t lddx, void* dw_gate,
                            void* dw_up, size_t lddw, size_t tokens, void* scratch,
                            size_t scratch_bytes, void* stream) {
  if (!h || (dw_gate == nullptr) != (dw_up == nullptr) || tokens > h->max_tokens)
    return AR_ERR_INVALID_ARG;
  if (!h->work) return AR_ERR_UNSUPPORTED;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t K = h->hidden, F = h->width;
  if (dw_gate && (bad_matrix(dw_gate, F, K, lddw) || bad_matrix(dw_up, F, K, lddw) ||
                  misaligned(dw_gate, 2) || misaligned(dw_up, 2)))
    return AR_ERR_INVALID_ARG;
  if (tokens == 0) {
    if (dw_gate && (cudaMemset2DAsync(dw_gate, lddw * 2, 0, K * 2, F, s) != cudaSuccess ||
                    cudaMemset2DAsync(dw_up, lddw * 2, 0, K * 2, F, s) != cudaSuccess))
      return AR_ERR_CUDA;
    return AR_OK;
  }
  if (bad_matrix(gate, tokens, F, ldo) || bad_matrix(up, tokens, F, ldo) ||
      bad_matrix(dout, tokens, F, ldo) || misaligned(gate, 2) || misaligned(up, 2) ||
      misaligned(dout, 2) || (dx && (bad_matrix(dx, tokens, K, lddx) || misaligned(dx, 2) ||
                                     bad_matrix(w_gate, F, K, ldw) || bad_matrix(w_up, F, K, ldw) ||
                                     misaligned(w_gate, 2) || misaligned(w_up, 2))) ||
      (dw_gate && (bad_matrix(x, tokens, K, ldx) || misaligned(x, 2))))
    return AR_ERR_INVALID_ARG;
  if (!dx && !dw_gate) return AR_OK;

  char* dgate = h->work;
  char* dup = h->work + 2 * h->rows * h->ldw;
  char* x_twice = h->work + 4 * h->rows * h->ldw;
  // dx wants the weights, the weights' gradients want x.
  Rows m[3];
  operands(h, x, ldx, w_gate, w_up, ldw, tokens, m);
  ar::PackJob jobs[3];
  int copies = 0;
  Rows* const from = dw_gate ? m : m + 1;
  if (ar_status_t st = plan_pack(from, dx ? (dw_gate ? 3 : 2) : 1, 2, scratch, scratch_bytes, jobs, &copies)) return st;
  ar::GemmArgs gx = {}, gw = {};
  gx.a0 = gw.a0 = dgate, gx.a1 = gw.a1 = dup, gx.lda = gw.lda = (int64_t)h->ldw;
  gx.b0 = m[1].p, gx.b1 = m[2].p, gx.ldb = (int64_t)m[1].ld, gx.ldb1 = (int64_t)m[2].ld;
  gx.c0 = dx, gx.ldc = (int64_t)lddx;
  gx.M = (int64_t)tokens, gx.N = (int64_t)K, gx.K = (int64_t)F;
  gw.b0 = m[0].p, gw.ldb = (int64_t)m[0].ld;
  gw.c0 = dw_gate, gw.c1 = dw_up, gw.ldc = (int64_t)lddw;
  gw.M = (int64_t)F, gw.N = (int64_t)K, gw.K = (int64_t)tokens;
  const bool tc_x = dx && ar::gemm_tc_takes(ar::kGemmDx, gx), tc_w = dw_gate && ar::gemm_tc_takes(ar::kGemmDw, gw);
  const bool two_parts = tokens <= kTwoPartTokens && tc_x == (dx != nullptr) && tc_w == (dw_gate != nullptr);
  if (two_parts) {
    gx.tokens = (int64_t)tokens;
    gx.M = gw.K = ar::two_part_rows((int64_t)tokens);
    if (dw_gate) {  // x beside both parts, from where the caller has it
      int at = 0;
      while (at < copies && jobs[at].to != m[0].p) ++at;
      copies += at == copies;
      jobs[at] = {x, x_twice, gw.K, (int64_t)K, (int64_t)ldx, (int64_t)h->ldx, (int64_t)tokens};
      gw.b0 = x_twice, gw.ldb = (int64_t)h->ldx;
    }
  }
  cudaError_t e = ar::launch_gate_grad(h->dtype, h->act, gate, up, dout, (int64_t)ldo, dgate, dup, (int64_t)h->ldw,
                                       (int64_t)tokens, (int64_t)F, two_parts, jobs, copies, h->num_sms, s);
  if (e == cudaSuccess && (tc_x || tc_w))
    e = ar::launch_grad_tc(h->dtype, tc_x ? &gx : nullptr, tc_w ? &gw : nullptr, h->num_sms, s);
  if (e == cudaSuccess && dx && !tc_x) e = ar::launch_gemm_any(ar::kGemmDx, h->dtype, gx, s);
  if (e == cudaSuccess && dw_gate && !tc_w) e = ar::launch_gemm_any(ar::kGemmDw, h->dtype, gw, s);
  return cuda_status(e);
}

ar_status_t ar_dropout(const void* x, size_t ldx, const void* residual, size_t ldr, void* out,
                       size_t ldo, size_t rows, size_t cols, int dtype, double p, uint64_t seed,
                       uint64_t sequence, uint64_t offset, void* stream) {
  return dropout_call(x, ldx, residual, ldr, out, ldo, rows, cols, dtype, p, seed, sequence, offset,
                      stream);
}

ar_status_t ar_dropout_backward(const void* dy, size_t lddy, void* dx, size_t lddx, size_t rows,
                                size_t cols, int dtype, double p, uint64_t seed,
                                uint64_t sequence, uint64_t offset, void* stream) {
  return dropout_call(dy, lddy, nullptr, 0, dx, lddx, rows, cols, dtype, p, seed, sequence, offset,
                      stream);
}

ar_status_t ar_quantize_rows(const void* x, size_t ldx, int8_t* q, size_t ldq, float* scale,
                             size_t rows, size_t cols, int dtype, void* stream) {
  if (!any_type(dtype)) return AR_ERR_UNSUPPORTED;
  if (rows == 0) return AR_OK;
  if (cols == 0 || !scale || misaligned(scale, 4) || bad_matrix(x, rows, cols, ldx) ||
      rows > 0x7FFFFFFF || misaligned(x, dtype == AR_FP32 ? 4 : 2) || bad_matrix(q, rows, cols, ldq))
    return AR_ERR_INVALID_ARG;
  int sms = 0;
  if (ar_status_t st = current_sms(&sms)) return st;
  return cuda_status(ar::launch_quantize_rows(dtype, x, (int64_t)ldx, q, (int64_t)ldq, scale,
                                              (int64_t)rows, (int64_t)cols, sms,
                                              static_cast<cudaStream_t>(stream)));
}

ar_status_t ar_linear_i8(const int8_t* x, size_t ldx, const float* x_scale, const int8_t* w,
                         size_t ldw, const float* w_scale, void* y, size_t ldy, size_t tokens,
                         size_t in, size_t out, int dtype, void* scratch, size_t scratch_bytes,
                         void* stream) {
  if (!half_type(dtype)) return AR_ERR_UNSUPPORTED;
  if (in == 0 || out == 0) return AR_ERR_INVALID_ARG;
  if (tokens == 0) return AR_OK;
  if (bad_matrix(x, tokens, in, ldx) || bad_matrix(w, out, in, ldw) ||
      bad_matrix(y, tokens, out, ldy) || !x_scale || !w_scale || misaligned(x_scale, 4) ||
      misaligned(w_scale, 4) || misaligned(y, 2))
    return AR_ERR_INVALID_ARG;
  int sms = 0;
  if (ar_status_t st = current_sms(&sms)) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  Rows m[2] = {{x, tokens, in, ldx}, {w, out, in, ldw}};
  if (tokens > kFewTokens)
    if (ar_status_t st = pack(m, 2, 1, scratch, scratch_bytes, sms, s)) return st;
  ar::GemmArgs g = {};
  g.a0 = m[0].p, g.lda = (int64_t)m[0].ld;
  g.b0 = m[1].p, g.ldb = (int64_t)m[1].ld;
  g.c0 = y, g.ldc = (int64_t)ldy;
  g.sm = x_scale, g.sn = w_scale;
  g.M = (int64_t)tokens, g.N = (int64_t)out, g.K = (int64_t)in;
  return cuda_status(gemm(ar::kGemmI8, dtype, g, sms, s));
}

size_t ar_linear_i8_scratch_bytes(const int8_t* x, size_t ldx, const int8_t* w, size_t ldw, size_t tokens, size_t in,
                                  size_t out) {
  const Rows m[2] = {{x, tokens, in, ldx}, {w, out, in, ldw}};
  return tokens > kFewTokens ? pack_bytes(m, 2, 1) : 0;
}

ar_status_t ar_ops_get_device_status(void* stream) {
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint32_t tc = 0, mid = 0, i8 = 0;
  if (ar::gemm_tc_error(s, &tc) != cudaSuccess || ar::gemm_mid_error(s, &mid) != cudaSuccess ||
      ar::gemm_i8_error(s, &i8) != cudaSuccess)
    return AR_ERR_CUDA;
  return tc || mid || i8 ? AR_ERR_TIMEOUT : AR_OK;
}

}  // extern "C"
