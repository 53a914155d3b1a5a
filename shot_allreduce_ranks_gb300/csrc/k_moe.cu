// A layer of gated feed-forward experts for a few tokens (formulas in
// include/ar.h), in two kernels: the gated products of the experts that have
// tokens, then the down products summed over each token's experts.
//
// Each used expert's matrices are read once, and memory bounds both kernels.  A
// CTA finds the routing for itself from the logits: a few hundred
// instructions, against a kernel of its own and its launch.
#include "ops_internal.cuh"

namespace ar {
namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32, kTokens = AR_FEW_TOKENS, kTop = AR_MAX_TOP_K;

// Logits in an order of whole numbers: NaN first, then by value, -0 as 0; what
// cannot be chosen (-infinity) is kNever or less.
constexpr uint32_t kNever = 0x007FFFFFu;
__device__ __forceinline__ uint32_t order_of(float v) {
  if (v != v) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}

// The routing of up to 32 tokens, in shared memory.
struct Routes {
  float weight[kTokens][kTop];
  int expert[kTokens][kTop];  // -1: none
  int active;                 // local experts that have tokens
};
// Behind it: for each local expert the tokens that it has (a bit each) and its
// place among the active ones; for each active one its number; and which of a
// token's choices it is.
struct RouteTables {
  uint32_t* tokens;
  uint16_t* place;
  uint16_t* number;
  uint8_t* choice;  // [active][32]
};
__host__ __device__ constexpr size_t route_bytes(int64_t local, int64_t pairs) {
  return (sizeof(Routes) + 15) / 16 * 16 + (size_t)local * 8 + (size_t)(local < pairs ? local : pairs) * kTokens;
}
__device__ __forceinline__ RouteTables tables(char* smem, int local) {
  RouteTables t;
  t.tokens = reinterpret_cast<uint32_t*>(smem + (sizeof(Routes) + 15) / 16 * 16);
  t.place = reinterpret_cast<uint16_t*>(t.tokens + local);
  t.number = t.place + local;
  t.choice = reinterpret_cast<uint8_t*>(t.number + local);
  return t;
}

__device__ __forceinline__ float logit(const MoeArgs& m, int64_t t, int e) {
  const char* p = static_cast<const char*>(m.logits);
  const int64_t i = t * m.ldl + e;
  return m.logits_dtype == AR_FP32   ? __uint_as_float(ld_elem<4>(p + 4 * i))
         : m.logits_dtype == AR_BF16 ? Bf16::to_f32(ld_elem<2>(p + 2 * i))
                                     : F16::to_f32(ld_elem<2>(p + 2 * i));
}

// One token's choices by one warp: lane j gets the j-th (its order and expert).
// R > 0: up to 32 R experts, held in registers; 0: any number, read again for every choice.
template <int R>
__device__ __forceinline__ void choose(const MoeArgs& m, int64_t t, int lane, uint32_t& mine, int& expert, float& total) {
  constexpr int N = R ? R : 1;
  uint32_t o[N];
  if (R)
#pragma unroll
    for (int r = 0; r < N; ++r) o[r] = 32 * r + lane < m.experts ? order_of(logit(m, t, 32 * r + lane)) : 0;
  mine = 0, expert = -1;
  uint32_t last = 0xFFFFFFFFu;  // the choice before: nothing before it comes again
  int last_e = -1;
  for (int j = 0; j < m.top_k; ++j) {
    uint32_t best = 0;
    int e = 0x7FFFFFFF;
    if (R) {
#pragma unroll
      for (int r = 0; r < N; ++r)
        if (o[r] > best) best = o[r], e = 32 * r + lane;
    } else {
      for (int i = lane; i < m.experts; i += 32) {
        const uint32_t v = order_of(logit(m, t, i));
        if (v > best && (v < last || (v == last && i > last_e))) best = v, e = i;
      }
    }
    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
    e = (int)__reduce_min_sync(0xFFFFFFFFu, best == top ? (uint32_t)e : 0x7FFFFFFFu);
    if (R) {
#pragma unroll
      for (int r = 0; r < N; ++r)
        if (32 * r + lane == e) o[r] = 0;
    }
    if (lane == j && top > kNever) mine = top, expert = e;
    last = top, last_e = e;
  }
  total = 0.0f;
  const float first = value_of(__shfl_sync(0xFFFFFFFFu, mine, 0));
  if (!m.normalize)
    for (int i = lane; i < m.experts; i += 32) total += expf(logit(m, t, i) - first);
}

// write: this CTA also stores the routing for the caller.
__device__ __forceinline__ void route(const MoeArgs& m, char* smem, bool write) {
  Routes& s = *reinterpret_cast<Routes*>(smem);
  const RouteTables tab = tables(smem, m.local);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < m.local; e += kThreads) tab.tokens[e] = 0;
  __syncthreads();
  for (int t = warp; t < m.tokens; t += kWarps) {
    uint32_t mine;
    int expert;
    float total;
    if (m.experts <= 64)
      choose<2>(m, t, lane, mine, expert, total);
    else if (m.experts <= 256)
      choose<8>(m, t, lane, mine, expert, total);
    else
      choose<0>(m, t, lane, mine, expert, total);
    const float first = value_of(__shfl_sync(0xFFFFFFFFu, mine, 0));
    float p = expert >= 0 ? expf(value_of(mine) - first) : 0.0f;
    if (m.normalize) total = p;
#pragma unroll
    for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
    if (expert >= 0) p = p / total;
    if (lane < m.top_k) {
      s.weight[t][lane] = p;
      s.expert[t][lane] = expert;
      const int e = expert - m.first;
      if (expert >= 0 && e >= 0 && e < m.local) atomicOr(&tab.tokens[e], 1u << t);
      if (write && m.out_expert) m.out_expert[t * m.top_k + lane] = expert;
      if (write && m.out_weight) m.out_weight[t * m.top_k + lane] = p;
    }
  }
  __syncthreads();
  if (warp == 0) {
    int count = 0;
    for (int base = 0; base < m.local; base += 32) {
      const int e = base + lane;
      const uint32_t with = __ballot_sync(0xFFFFFFFFu, e < m.local && tab.tokens[e] != 0);
      const int at = count + __popc(with & ((1u << lane) - 1));
      if (with >> lane & 1) tab.place[e] = (uint16_t)at, tab.number[at] = (uint16_t)e;
      count += __popc(with);
    }
    if (lane == 0) s.active = count;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < m.tokens * m.top_k; i += kThreads) {
    const int t = i / m.top_k, j = i % m.top_k, e = s.expert[t][j] - m.first;
    if (s.expert[t][j] >= 0 && e >= 0 && e < m.local) tab.choice[tab.place[e] * kTokens + t] = (uint8_t)j;
  }
  __syncthreads();
}

template <bool VEC>
__device__ __forceinline__ uint4 weights16(const char* p, int64_t left, const char* begin, const char* end) {
  if (VEC && left >= 16) return ld_v4_stream(p);
  return load_anywhere<2>(p, left, begin, end);
}
// 16 bytes of an operand that other CTAs of the SM read too.
template <bool VEC>
__device__ __forceinline__ uint4 tokens16(const char* p, int64_t left, const char* begin, const char* end) {
  if (VEC && left >= 16) return *reinterpret_cast<const uint4*>(p);
  return load_anywhere<2>(p, left, begin, end);
}

template <class E, int NB>
__device__ __forceinline__ void multiply(float (&acc)[NB][4], const uint4& a, const uint4& b, const uint4 (&x)[NB]) {
  const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const uint32_t f[4] = {aw[2 * w], bw[2 * w], aw[2 * w + 1], bw[2 * w + 1]};
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const uint32_t xw[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
      const uint32_t y[2] = {xw[2 * w], xw[2 * w + 1]};
      mma_16816<E>(acc[j], f, y);
    }
  }
}

// Eight rows of one expert's gate and of its up projection for its tokens, 8 NB at
// most: the rows of mma.sync are the gate's and the up projection's, its
// columns the tokens; a lane loads 16 contiguous bytes of its rows and its token
// (which k an instruction's k slots stand for is free as long as they agree).
// The warps take turns along k.
template <class E, int ACT, int NB, bool VEC>
__device__ __forceinline__ void gated_rows(const MoeArgs& m, const RouteTables& tab, int place, int64_t f0,
                                           uint8_t* list, float4 (*part)[4][32]) {
  constexpr int U = NB > 2 ? 2 : 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g8 = lane >> 2, t4 = lane & 3;
  const int e = tab.number[place];
  const uint32_t tokens = tab.tokens[e];
  const int count = __popc(tokens);
  if (tokens >> lane & 1) list[__popc(tokens & ((1u << lane) - 1))] = (uint8_t)lane;
  __syncwarp();
  const int64_t f = min(f0 + g8, m.width - 1), bytes = m.hidden * 2;
  const char *bg = static_cast<const char*>(m.w_gate), *bu = static_cast<const char*>(m.w_up), *bx = static_cast<const char*>(m.x);
  const int64_t extent = ((m.local - 1) * m.esw + (m.width - 1) * m.ldw + m.hidden) * 2;
  const char *wg = bg + (e * m.esw + f * m.ldw) * 2, *wu = bu + (e * m.esw + f * m.ldw) * 2;
  const char* ex = bx + ((m.tokens - 1) * m.ldx + m.hidden) * 2;
  const char* xs[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) xs[j] = 8 * j + g8 < count ? bx + list[8 * j + g8] * m.ldx * 2 : nullptr;
  float acc[NB][4] = {};
  for (int64_t at = (int64_t)warp * 64 * U; at < bytes; at += kWarps * 64 * U) {
    uint4 a[U], b[U], x[U][NB];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t k = at + 64 * i + 16 * t4;
      a[i] = weights16<VEC>(wg + k, bytes - k, bg, bg + extent);
      b[i] = weights16<VEC>(wu + k, bytes - k, bu, bu + extent);
#pragma unroll
      for (int j = 0; j < NB; ++j) x[i][j] = xs[j] ? tokens16<VEC>(xs[j] + k, bytes - k, bx, ex) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) multiply<E, NB>(acc, a[i], b[i], x[i]);
  }
#pragma unroll
  for (int j = 0; j < NB; ++j) part[warp][j][lane] = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
  __syncthreads();
  if (warp < NB) {
    float v[4] = {};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 p = part[w][warp][lane];
      v[0] += p.x, v[1] += p.y, v[2] += p.z, v[3] += p.w;
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int i = 8 * warp + 2 * t4 + c;
      if (i >= count) continue;
      const int t = list[i];
      const int64_t row = t * m.top_k + tab.choice[place * kTokens + t];
      // The row's end, up to a whole group, is read with it: zeros.
      const float h = f0 + g8 < m.width ? act_value<ACT>(v[c]) * v[c + 2] : 0.0f;
      static_cast<uint16_t*>(m.h)[row * m.ldh + f0 + g8] = (uint16_t)E::from_f32(h);
    }
  }
  __syncthreads();
}

template <class E, int ACT, bool VEC>
__global__ void __launch_bounds__(kThreads) k_moe_gated(MoeArgs m) {
  extern __shared__ __align__(16) char smem[];
  __shared__ float4 part[kWarps][4][32];
  __shared__ uint8_t lists[kWarps][kTokens];
  pdl_enter();
  route(m, smem, blockIdx.x == 0);
  const RouteTables tab = tables(smem, m.local);
  const int64_t strips = (m.width + 7) / 8, items = reinterpret_cast<const Routes*>(smem)->active * strips;
  uint8_t* list = lists[threadIdx.x >> 5];
  for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
    const int place = (int)(i / strips), count = __popc(tab.tokens[tab.number[place]]);
    const int64_t f0 = i % strips * 8;
    if (count <= 8)
      gated_rows<E, ACT, 1, VEC>(m, tab, place, f0, list, part);
    else if (count <= 16)
      gated_rows<E, ACT, 2, VEC>(m, tab, place, f0, list, part);
    else
      gated_rows<E, ACT, 4, VEC>(m, tab, place, f0, list, part);
  }
}

// Sixteen output columns for all tokens (8 NB at most): the warps take turns at
// pieces of 128 of the experts' inner columns; each piece's sums are weighted and
// added in fp32, in a fixed order.
template <class E, int NB, bool VEC>
__global__ void __launch_bounds__(kThreads) k_moe_down(MoeArgs m) {
  extern __shared__ __align__(16) char smem[];
  __shared__ float4 part[kWarps][NB][32];
  constexpr int U = NB > 2 ? 2 : 4;
  pdl_enter();
  route(m, smem, false);
  const Routes& s = *reinterpret_cast<const Routes*>(smem);
  const RouteTables tab = tables(smem, m.local);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g8 = lane >> 2, t4 = lane & 3;
  const int64_t n0 = (int64_t)blockIdx.x * 16, bytes = m.width * 2;
  const int64_t ra = min(n0 + g8, m.hidden - 1), rb = min(n0 + g8 + 8, m.hidden - 1);
  const char *bd = static_cast<const char*>(m.w_down), *ed = bd + ((m.local - 1) * m.esd + (m.hidden - 1) * m.ldd + m.width) * 2;
  const char* h = static_cast<const char*>(m.h);
  const int pieces = (int)((bytes + 64 * U - 1) / (64 * U)), units = s.active * pieces;
  float total[NB][4] = {};
  for (int u = warp; u < units; u += kWarps) {
    const int place = u / pieces, e = tab.number[place];
    const uint32_t tokens = tab.tokens[e];
    const int64_t at = (int64_t)(u % pieces) * 64 * U;
    const char *wa = bd + (e * m.esd + ra * m.ldd) * 2, *wb = bd + (e * m.esd + rb * m.ldd) * 2;
    uint4 a[U], b[U], x[U][NB];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t k = at + 64 * i + 16 * t4;
      a[i] = weights16<VEC>(wa + k, bytes - k, bd, ed);
      b[i] = weights16<VEC>(wb + k, bytes - k, bd, ed);
    }
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int t = 8 * j + g8;
      const bool has = tokens >> t & 1;
      const char* row = h + (has ? t * m.top_k + tab.choice[place * kTokens + t] : 0) * m.ldh * 2;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int64_t k = at + 64 * i + 16 * t4;
        // rows of h start on 16 bytes and end in zeros
        x[i][j] = has && k < bytes ? *reinterpret_cast<const uint4*>(row + k) : make_uint4(0, 0, 0, 0);
      }
    }
    float acc[NB][4] = {};
#pragma unroll
    for (int i = 0; i < U; ++i) multiply<E, NB>(acc, a[i], b[i], x[i]);
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int t = 8 * j + 2 * t4 + c;
        if (!(tokens >> t & 1)) continue;  // 0 times an infinite weight would be NaN
        const float w = s.weight[t][tab.choice[place * kTokens + t]];
        total[j][c] = __fmaf_rn(w, acc[j][c], total[j][c]);
        total[j][c + 2] = __fmaf_rn(w, acc[j][c + 2], total[j][c + 2]);
      }
  }
#pragma unroll
  for (int j = 0; j < NB; ++j) part[warp][j][lane] = make_float4(total[j][0], total[j][1], total[j][2], total[j][3]);
  __syncthreads();
  if (warp >= NB) return;
  float v[4] = {};
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const float4 p = part[w][warp][lane];
    v[0] += p.x, v[1] += p.y, v[2] += p.z, v[3] += p.w;
  }
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int64_t t = 8 * warp + 2 * t4 + c, n = n0 + g8 + 8 * r;
      if (t < m.tokens && n < m.hidden) static_cast<uint16_t*>(m.out)[t * m.ldo + n] = (uint16_t)E::from_f32(v[2 * r + c]);
    }
}

template <class E, int ACT, bool VEC>
cudaError_t moe(const MoeArgs& m, int num_sms, cudaStream_t s) {
  const int64_t pairs = m.tokens * m.top_k, most = m.local < pairs ? m.local : pairs;
  const int64_t strips = (m.width + 7) / 8, tiles = (m.hidden + 15) / 16;
  if (tiles > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  const size_t smem = route_bytes(m.local, pairs);
  const int64_t items = most * strips, slots = (int64_t)num_sms * 3;
  cudaError_t e = launch_op(k_moe_gated<E, ACT, VEC>, dim3((unsigned)(items < slots ? items : slots)), kThreads, smem, 1, s, m);
  if (e != cudaSuccess) return e;
  auto* k = m.tokens <= 8 ? k_moe_down<E, 1, VEC> : m.tokens <= 16 ? k_moe_down<E, 2, VEC> : k_moe_down<E, 4, VEC>;
  return launch_op(k, dim3((unsigned)tiles), kThreads, smem, 1, s, m);
}

template <class E, int ACT>
cudaError_t moe_align(const MoeArgs& m, int num_sms, cudaStream_t s) {
  const bool vec = ((reinterpret_cast<uintptr_t>(m.x) | reinterpret_cast<uintptr_t>(m.w_gate) | reinterpret_cast<uintptr_t>(m.w_up) |
                     reinterpret_cast<uintptr_t>(m.w_down)) & 15u) == 0 &&
                   (m.ldx | m.ldw | m.esw | m.ldd | m.esd) % 8 == 0;
  return vec ? moe<E, ACT, true>(m, num_sms, s) : moe<E, ACT, false>(m, num_sms, s);
}

}  // namespace

cudaError_t launch_moe(int dtype, int act, const MoeArgs& m, int num_sms, cudaStream_t s) {
  if (dtype == AR_BF16)
    return act == AR_ACT_SILU ? moe_align<Bf16, AR_ACT_SILU>(m, num_sms, s) : moe_align<Bf16, AR_ACT_GELU_TANH>(m, num_sms, s);
  return act == AR_ACT_SILU ? moe_align<F16, AR_ACT_SILU>(m, num_sms, s) : moe_align<F16, AR_ACT_GELU_TANH>(m, num_sms, s);
}

}  // namespace ar
