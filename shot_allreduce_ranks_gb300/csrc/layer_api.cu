// C ABI of a layer's steps around the feed-forward block: argument checks,
// workspaces and the choice of kernel.  Declarations and contracts are in
// include/ar.h.
#include <math.h>

#include "ops_internal.cuh"

namespace {

using namespace ar;  // the entry points' shared checks

constexpr size_t kMaxCols = (size_t)1 << 30, kMaxInner = (size_t)1 << 22;

size_t elem_bytes(int dtype) { return dtype == AR_FP32 ? 4 : 2; }

// What both passes check of the description; rows = 0 is left to the caller.
ar_status_t check_norm(const ar_norm_t* n, const void* gate, size_t ldg, const void* after_weight,
                       const void* after_bias, const void* weight) {
  if (!n) return AR_ERR_INVALID_ARG;
  if (!any_type(n->dtype) || (n->kind != AR_NORM_RMS && n->kind != AR_NORM_LAYER)) return AR_ERR_UNSUPPORTED;
  if (n->cols == 0 || n->cols > kMaxCols || n->rows > kMaxElems || !(n->eps >= 0.0) || isinf(n->eps) ||
      (!weight && !after_weight) || (after_bias && !after_weight))
    return AR_ERR_INVALID_ARG;
  const size_t e = elem_bytes(n->dtype);
  if (misaligned(after_weight, e) || misaligned(after_bias, e) || misaligned(weight, e)) return AR_ERR_INVALID_ARG;
  if ((gate != nullptr) != (n->gate_rows != 0)) return AR_ERR_INVALID_ARG;
  if (gate && (n->rows % n->gate_rows || bad_matrix(gate, n->gate_rows, n->cols, ldg) || misaligned(gate, e)))
    return AR_ERR_INVALID_ARG;
  return AR_OK;
}

// Experts' matrices, es elements from one to the next (0: all the same).
bool bad_stack(const void* p, size_t count, size_t rows, size_t cols, size_t ld, size_t es) {
  return bad_matrix(p, rows, cols, ld) || misaligned(p, 2) || es > kMaxElems || (es && count > kMaxElems / es);
}

bool bad_i4(size_t out, size_t in, int group) {
  return out < 1 || out > kMaxCols || in < 1 || in > kMaxCols || (group != 32 && group != 64 && group != 128);
}
size_t i4_groups(size_t in, int group) { return (in + (size_t)group - 1) / (size_t)group; }
size_t i4_spans(size_t in, int group) { return i4_groups(in, i4_span(group)); }
// The laid-out arrays of a call.
bool bad_i4_arrays(const void* data, const void* scale, const void* zero) {
  return !data || !scale || misaligned(data, 16) || misaligned(scale, 16) || misaligned(zero, 16);
}

ar_status_t check_moe(const ar_moe_t* m) {
  if (!m) return AR_ERR_INVALID_ARG;
  if (!half_type(m->dtype) || !any_type(m->logits_dtype)) return AR_ERR_UNSUPPORTED;
  if ((m->activation != AR_ACT_SILU && m->activation != AR_ACT_GELU_TANH) || m->experts < 1 ||
      m->experts > AR_MAX_EXPERTS || m->local_experts < 1 || m->local_experts > m->experts || m->first_expert < 0 ||
      m->first_expert > m->experts - m->local_experts || m->top_k < 1 || m->top_k > AR_MAX_TOP_K ||
      m->top_k > m->experts || m->hidden < 1 || m->hidden > kMaxInner || m->width < 1 || m->width > kMaxInner)
    return AR_ERR_INVALID_ARG;
  // The kernels count a layer's pieces (16 rows of 64) in 32 bits: 2^31 of them are 4 TB of weights.
  const size_t most = (size_t)m->local_experts, pieces = ((m->width + 63) / 64) * ((m->hidden + 63) / 64) * 8;
  return most * pieces >> 31 ? AR_ERR_INVALID_ARG : AR_OK;
}

size_t moe_bytes(const ar_moe_t* m, size_t tokens, bool two_parts, MoeArgs* a = nullptr, void* base = nullptr) {
  if (check_moe(m) || tokens == 0) return 0;
  const size_t run = tokens < AR_FEW_TOKENS ? tokens : AR_FEW_TOKENS;
  return moe_scratch((int64_t)run, m->top_k, (int64_t)m->width, (int64_t)m->hidden, two_parts, a, static_cast<char*>(base));
}

}  // namespace

extern "C" {

ar_status_t ar_i4_sizes(size_t out, size_t in, int group, size_t* data_bytes, size_t* scales) {
  if (bad_i4(out, in, group) || !data_bytes || !scales) return AR_ERR_INVALID_ARG;
  const size_t tiles = (out + 15) / 16, span = (size_t)i4_span(group), spans = i4_spans(in, group);
  *data_bytes = tiles * spans * span * 8;
  *scales = tiles * spans * 16 * (span / (size_t)group);
  return AR_OK;
}

ar_status_t ar_pack_i4(const uint8_t* q, size_t ldq, const void* scale, size_t lds, const uint8_t* zero,
                       size_t ldz, size_t out, size_t in, int group, void* data, void* packed_scale,
                       void* packed_zero, void* stream) {
  if (bad_i4(out, in, group)) return AR_ERR_INVALID_ARG;
  const size_t groups = i4_groups(in, group);
  if (bad_i4_arrays(data, packed_scale, packed_zero) || (zero != nullptr) != (packed_zero != nullptr) ||
      bad_matrix(q, out, in, ldq) || bad_matrix(scale, out, groups, lds) || misaligned(scale, 2) ||
      (zero && bad_matrix(zero, out, groups, ldz)))
    return AR_ERR_INVALID_ARG;
  int sms = 0;
  if (ar_status_t st = current_sms(&sms)) return st;
  I4Pack a = {};
  a.q = q, a.row_scale = static_cast<const uint16_t*>(scale), a.row_zero = zero;
  a.data = static_cast<uint4*>(data), a.scale = static_cast<uint16_t*>(packed_scale), a.zero = static_cast<uint8_t*>(packed_zero);
  a.ldq = (int64_t)ldq, a.lds = (int64_t)lds, a.ldz = (int64_t)ldz, a.N = (int64_t)out, a.K = (int64_t)in;
  a.spans = (int64_t)i4_spans(in, group), a.group = group;
  return cuda_status(launch_pack_i4(a, sms, static_cast<cudaStream_t>(stream)));
}

size_t ar_quantize_i4_scratch_bytes(size_t out, size_t in, int group) {
  if (bad_i4(out, in, group)) return 0;
  return out * i4_groups(in, group) * 3 + out * in;
}

ar_status_t ar_quantize_i4(const void* w, size_t ldw, size_t out, size_t in, int group, int dtype,
                           void* data, void* packed_scale, void* packed_zero, void* scratch,
                           size_t scratch_bytes, void* stream) {
  if (!half_type(dtype)) return AR_ERR_UNSUPPORTED;
  if (bad_i4(out, in, group) || bad_i4_arrays(data, packed_scale, packed_zero) || bad_matrix(w, out, in, ldw) ||
      misaligned(w, 2) || !scratch || misaligned(scratch, 16) || scratch_bytes < ar_quantize_i4_scratch_bytes(out, in, group))
    return AR_ERR_INVALID_ARG;
  int sms = 0;
  if (ar_status_t st = current_sms(&sms)) return st;
  const size_t groups = i4_groups(in, group);
  I4Quantize a = {};
  a.w = w, a.row_scale = static_cast<uint16_t*>(scratch);
  uint8_t* const zero = static_cast<uint8_t*>(scratch) + out * groups * 2;
  a.row_zero = packed_zero ? zero : nullptr;
  a.q = zero + out * groups;
  a.ldw = (int64_t)ldw, a.N = (int64_t)out, a.K = (int64_t)in, a.group = group;
  const cudaError_t e = launch_quantize_i4(dtype, a, sms, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return AR_ERR_CUDA;
  return ar_pack_i4(a.q, in, a.row_scale, groups, a.row_zero, groups, out, in, group, data, packed_scale, packed_zero, stream);
}

ar_status_t ar_dequantize_i4(const void* data, const void* packed_scale, const void* packed_zero,
                             size_t out, size_t in, int group, int dtype, void* w, size_t ldw,
                             void* stream) {
  if (!half_type(dtype)) return AR_ERR_UNSUPPORTED;
  if (bad_i4(out, in, group) || bad_i4_arrays(data, packed_scale, packed_zero) || bad_matrix(w, out, in, ldw) || misaligned(w, 2))
    return AR_ERR_INVALID_ARG;
  int sms = 0;
  if (ar_status_t st = current_sms(&sms)) return st;
  I4Unpack a = {};
  a.data = static_cast<const uint32_t*>(data), a.scale = static_cast<const uint16_t*>(packed_scale);
  a.zero = static_cast<const uint8_t*>(packed_zero);
  a.w = w, a.ldw = (int64_t)ldw, a.N = (int64_t)out, a.K = (int64_t)in;
  a.spans = (int64_t)i4_spans(in, group), a.group = group;
  return cuda_status(launch_unpack_i4(dtype, a, sms, static_cast<cudaStream_t>(stream)));
}

ar_status_t ar_linear_i4(const void* x, size_t ldx, const void* data, const void* packed_scale,
                         const void* packed_zero, void* y, size_t ldy, size_t tokens, size_t in,
                         size_t out, int group, int dtype, void* stream) {
  if (!half_type(dtype)) return AR_ERR_UNSUPPORTED;
  if (bad_i4(out, in, group) || tokens > (size_t)32 * 65535) return AR_ERR_INVALID_ARG;
  if (tokens == 0) return AR_OK;
  if (bad_i4_arrays(data, packed_scale, packed_zero) || bad_matrix(x, tokens, in, ldx) || misaligned(x, 2) ||
      bad_matrix(y, tokens, out, ldy) || misaligned(y, 2))
    return AR_ERR_INVALID_ARG;
  I4Args a = {};
  a.x = x, a.data = data, a.scale = packed_scale, a.zero = static_cast<const uint8_t*>(packed_zero), a.y = y;
  a.ldx = (int64_t)ldx, a.ldy = (int64_t)ldy, a.M = (int64_t)tokens, a.N = (int64_t)out, a.K = (int64_t)in;
  a.spans = (int64_t)i4_spans(in, group);
  return cuda_status(launch_linear_i4(dtype, group, a, static_cast<cudaStream_t>(stream)));
}

size_t ar_moe_scratch_bytes(const ar_moe_t* m, size_t tokens) { return moe_bytes(m, tokens, false); }
size_t ar_moe_two_part_scratch_bytes(const ar_moe_t* m, size_t tokens) { return moe_bytes(m, tokens, true); }

ar_status_t ar_moe_ffn(const ar_moe_t* m, const void* x, size_t ldx, const void* logits, size_t ldl,
                       const void* w_gate, const void* w_up, size_t ldw, size_t esw,
                       const void* w_down, size_t ldd, size_t esd, void* out, size_t ldo,
                       int32_t* expert, float* weight, size_t tokens, void* scratch,
                       size_t scratch_bytes, void* stream) {
  if (ar_status_t st = check_moe(m)) return st;
  if (tokens == 0) return AR_OK;
  const size_t K = m->hidden, F = m->width, le = elem_bytes(m->logits_dtype), n = (size_t)m->local_experts;
  if (bad_matrix(x, tokens, K, ldx) || misaligned(x, 2) || bad_matrix(logits, tokens, (size_t)m->experts, ldl) ||
      misaligned(logits, le) || bad_stack(w_gate, n, F, K, ldw, esw) || bad_stack(w_up, n, F, K, ldw, esw) ||
      bad_stack(w_down, n, K, F, ldd, esd) || bad_matrix(out, tokens, K, ldo) || misaligned(out, 2) ||
      misaligned(expert, 4) || misaligned(weight, 4) || !scratch || misaligned(scratch, 16) ||
      scratch_bytes < ar_moe_scratch_bytes(m, tokens))
    return AR_ERR_INVALID_ARG;
  int sms = 0;
  if (ar_status_t st = current_sms(&sms)) return st;
  MoeArgs a = {};
  a.w_gate = w_gate, a.w_up = w_up, a.w_down = w_down;
  moe_bytes(m, tokens, scratch_bytes >= moe_bytes(m, tokens, true), &a, scratch);
  a.ldx = (int64_t)ldx, a.ldl = (int64_t)ldl, a.ldw = (int64_t)ldw, a.esw = (int64_t)esw;
  a.ldd = (int64_t)ldd, a.esd = (int64_t)esd, a.ldo = (int64_t)ldo;
  a.hidden = (int64_t)K, a.width = (int64_t)F;
  a.experts = m->experts, a.first = m->first_expert, a.local = m->local_experts;
  a.top_k = m->top_k, a.normalize = m->normalize != 0, a.logits_dtype = m->logits_dtype;
  for (size_t t = 0; t < tokens; t += AR_FEW_TOKENS) {
    a.tokens = (int)(tokens - t < AR_FEW_TOKENS ? tokens - t : AR_FEW_TOKENS);
    a.x = static_cast<const char*>(x) + t * ldx * 2;
    a.logits = static_cast<const char*>(logits) + t * ldl * le;
    a.out = static_cast<char*>(out) + t * ldo * 2;
    a.out_expert = expert ? expert + t * (size_t)m->top_k : nullptr;
    a.out_weight = weight ? weight + t * (size_t)m->top_k : nullptr;
    const cudaError_t e = launch_moe(m->dtype, m->activation, a, sms, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return AR_ERR_CUDA;
  }
  return AR_OK;
}

ar_status_t ar_residual_norm(const ar_norm_t* n, const void* x, size_t ldx, const void* residual,
                             size_t ldres, const void* gate, size_t ldg, const void* after_weight,
                             const void* after_bias, const void* weight, const void* bias, void* r,
                             size_t ldr, void* y, size_t ldy, void* stream) {
  if (ar_status_t st = check_norm(n, gate, ldg, after_weight, after_bias, weight)) return st;
  const size_t rows = n->rows, cols = n->cols, e = elem_bytes(n->dtype);
  if ((bias && !weight) || misaligned(bias, e)) return AR_ERR_INVALID_ARG;
  if (rows == 0) return AR_OK;
  if ((y != nullptr) != (weight != nullptr) || bad_matrix(x, rows, cols, ldx) || misaligned(x, e) ||
      (residual && (bad_matrix(residual, rows, cols, ldres) || misaligned(residual, e))) ||
      (r && (bad_matrix(r, rows, cols, ldr) || misaligned(r, e))) ||
      (y && (bad_matrix(y, rows, cols, ldy) || misaligned(y, e))) || (r && r == y))
    return AR_ERR_INVALID_ARG;
  if (!r && !y) return AR_OK;
  int sms = 0;
  if (ar_status_t st = current_sms(&sms)) return st;
  NormArgs a = {};
  a.x = x, a.residual = residual, a.gate = gate;
  a.after_weight = after_weight, a.after_bias = after_bias, a.weight = weight, a.bias = bias;
  a.r = r, a.y = y;
  a.ldx = (int64_t)ldx, a.ldres = (int64_t)ldres, a.ldg = (int64_t)ldg, a.ldr = (int64_t)ldr, a.ldy = (int64_t)ldy;
  a.rows = (int64_t)rows, a.cols = (int64_t)cols;
  a.gate_run = gate ? (int64_t)(rows / n->gate_rows) : (int64_t)rows;
  a.gate_extent = gate ? (int64_t)((n->gate_rows - 1) * ldg + cols) : 0;
  a.eps = (float)n->eps, a.alpha = (float)n->residual_scale, a.offset = (float)n->weight_offset;
  a.layer = n->kind == AR_NORM_LAYER;
  return cuda_status(launch_norm(n->dtype, a, sms, static_cast<cudaStream_t>(stream)));
}

size_t ar_residual_norm_scratch_bytes(size_t rows, size_t cols, int vectors) {
  if (vectors <= 0 || rows > kMaxElems || cols > kMaxCols) return 0;
  return (size_t)vectors * (size_t)norm_parts((int64_t)rows, (int64_t)cols) * cols * sizeof(float);
}

ar_status_t ar_residual_norm_backward(const ar_norm_t* n, const void* dy, size_t lddy, const void* dr,
                                      size_t lddr, const void* x, size_t ldx, const void* r, size_t ldr,
                                      const void* gate, size_t ldg, const void* after_weight,
                                      const void* after_bias, const void* weight, void* dx, size_t lddx,
                                      void* dresidual, size_t lddres, void* dgate, size_t lddg,
                                      void* dweight, void* dbias, void* dafter_weight,
                                      void* dafter_bias, void* scratch, size_t scratch_bytes,
                                      void* stream) {
  if (ar_status_t st = check_norm(n, gate, ldg, after_weight, after_bias, weight)) return st;
  const size_t rows = n->rows, cols = n->cols, e = elem_bytes(n->dtype);
  void* const sums[kNormSums] = {dweight, dbias, dafter_weight, dafter_bias, dgate};
  int vectors = 0;
  for (void* p : sums) {
    if (misaligned(p, e)) return AR_ERR_INVALID_ARG;
    vectors += p != nullptr;
  }
  if (((dweight || dbias) && !weight) || ((dafter_weight || dafter_bias) && !after_weight) || (dgate && !gate) ||
      (dgate && bad_matrix(dgate, n->gate_rows, cols, lddg)))
    return AR_ERR_INVALID_ARG;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    for (int k = 0; k < kNormSums; ++k) {
      const size_t m = k == kSumGate ? n->gate_rows : 1, ld = k == kSumGate ? lddg : cols;
      if (sums[k] && cudaMemset2DAsync(sums[k], ld * e, 0, cols * e, m, s) != cudaSuccess) return AR_ERR_CUDA;
    }
    return AR_OK;
  }
  if ((dy != nullptr) != (weight != nullptr) || (!dy && !dr)) return AR_ERR_INVALID_ARG;
  if ((dy && (bad_matrix(dy, rows, cols, lddy) || misaligned(dy, e) || bad_matrix(r, rows, cols, ldr) || misaligned(r, e))) ||
      (dr && (bad_matrix(dr, rows, cols, lddr) || misaligned(dr, e))) ||
      ((gate || after_weight) && (bad_matrix(x, rows, cols, ldx) || misaligned(x, e))) ||
      (dx && (bad_matrix(dx, rows, cols, lddx) || misaligned(dx, e))) ||
      (dresidual && (bad_matrix(dresidual, rows, cols, lddres) || misaligned(dresidual, e))))
    return AR_ERR_INVALID_ARG;
  if (vectors && (!scratch || misaligned(scratch, 16) || scratch_bytes < ar_residual_norm_scratch_bytes(rows, cols, vectors)))
    return AR_ERR_INVALID_ARG;
  if (!vectors && !dx && !dresidual) return AR_OK;
  int sms = 0;
  if (ar_status_t st = current_sms(&sms)) return st;
  NormGradArgs a = {};
  // What is not read has no say in how the rows are read.
  a.dy = dy, a.dr = dr, a.x = gate || after_weight ? x : nullptr, a.r = weight ? r : nullptr, a.gate = gate;
  a.after_weight = after_weight, a.after_bias = gate ? after_bias : nullptr, a.weight = weight;
  a.dx = dx, a.dresidual = dresidual;
  const size_t parts = (size_t)norm_parts((int64_t)rows, (int64_t)cols);
  float* part = static_cast<float*>(scratch);
  for (int k = 0; k < kNormSums; ++k) {
    a.sum[k] = sums[k];
    if (!sums[k]) continue;
    a.part[k] = part;
    part += parts * cols;
  }
  a.lddy = (int64_t)lddy, a.lddr = (int64_t)lddr, a.ldx = (int64_t)ldx, a.ldr = (int64_t)ldr, a.ldg = (int64_t)ldg;
  a.lddx = (int64_t)lddx, a.lddres = (int64_t)lddres, a.lddg = (int64_t)lddg;
  a.rows = (int64_t)rows, a.cols = (int64_t)cols;
  a.gate_rows = gate ? (int64_t)n->gate_rows : 1;
  a.gate_run = (int64_t)rows / a.gate_rows;
  a.eps = (float)n->eps, a.alpha = (float)n->residual_scale, a.offset = (float)n->weight_offset;
  a.layer = n->kind == AR_NORM_LAYER;
  return cuda_status(launch_norm_grad(n->dtype, a, sms, s));
}

}  // extern "C"
