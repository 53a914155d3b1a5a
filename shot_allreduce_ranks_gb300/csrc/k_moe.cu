// A layer of gated feed-forward experts for a few tokens (formulas in
// include/ar.h), in two kernels: the gated products of the experts that have
// tokens, then the down products summed over each token's experts.
//
// Each used expert's matrices are read once, and memory bounds both kernels: one
// CTA an SM walks over its part of the matrices, and each of its warps copies the
// next pieces of its own (kStages - 1 of 2 KB: 128 KB an SM in flight) into shared memory
// while it multiplies.  A lane copies just the 16 bytes that it will use, so
// a warp waits for nothing but its own copies.  A CTA finds the routing for itself from the
// logits: a few hundred instructions, against a kernel of its own and its launch.
#include <type_traits>

#include "ops_internal.cuh"

namespace ar {
namespace {

constexpr int kWarps = 16, kThreads = kWarps * 32, kTokens = AR_FEW_TOKENS, kTop = AR_MAX_TOP_K;

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

// 16 bytes of an operand that other CTAs of the SM read too.
template <bool VEC>
__device__ __forceinline__ uint4 tokens16(const char* p, int64_t left, const char* begin, const char* end) {
  if (VEC && left >= 16) return *reinterpret_cast<const uint4*>(p);
  return load_anywhere<2>(p, left, begin, end);
}

// The pieces of 64 k (two steps of 32) of sixteen rows that a warp copies ahead:
// lane 4 g + t has rows g and g + 8 at k = 8 t .. 8 t + 7 of each step.
constexpr int kStages = 5, kSteps = 2, kPieceBytes = 128, kRingBytes = kWarps * kStages * kSteps * 2 * 512;

struct Ring {
  char* mine;  // this lane's place in its warp's ring
  __device__ __forceinline__ explicit Ring(char* smem)
      : mine(smem + (threadIdx.x >> 5) * kStages * kSteps * 2 * 512 + (threadIdx.x & 31) * 16) {}
  __device__ __forceinline__ char* at(int stage, int step, int row) const { return mine + ((stage * kSteps + step) * 2 + row) * 512; }

  // Rows a and b (this lane's) at byte k of `bytes`; what lies past a row's end is zeros.
  template <bool VEC>
  __device__ __forceinline__ void fetch(int stage, const char* a, const char* b, int64_t k, int64_t bytes, const char* begin_a,
                                        const char* begin_b, int64_t extent) const {
    const int t4 = threadIdx.x & 3;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int64_t at_k = k + 64 * i + 16 * t4, left = bytes - at_k;
      if (VEC) {
        const int n = left >= 16 ? 16 : left > 0 ? (int)left : 0;
        copy(at(stage, i, 0), n ? a + at_k : a, n);
        copy(at(stage, i, 1), n ? b + at_k : b, n);
      } else {
        *reinterpret_cast<uint4*>(at(stage, i, 0)) = load_anywhere<2>(a + at_k, left, begin_a, begin_a + extent);
        *reinterpret_cast<uint4*>(at(stage, i, 1)) = load_anywhere<2>(b + at_k, left, begin_b, begin_b + extent);
      }
    }
  }
  static __device__ __forceinline__ void copy(char* to, const char* from, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from), "r"(bytes)
                 : "memory");
  }
  static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  static __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory"); }
};

// Sums of a step: the rows of mma.sync are the sixteen, its columns eight tokens; which k
// an instruction's k slots stand for is free as long as both operands agree.
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

// An item: eight rows of one expert's gate and the same of its up projection, whose
// sums of one output land in one lane.  The warps take turns at the pieces along k, and
// their sums are joined in a fixed order.
template <class E, int ACT, bool VEC>
__global__ void __launch_bounds__(kThreads, 1) k_moe_gated(MoeArgs m) {
  extern __shared__ __align__(16) char smem[];
  pdl_enter();
  char* const tables_at = smem + kRingBytes;
  const Ring ring(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g8 = lane >> 2, t4 = lane & 3;
  // The down kernel's counts of finished parts.
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < (m.hidden + 15) / 16; i += (int64_t)gridDim.x * kThreads) m.done[i] = 0;
  route(m, tables_at, blockIdx.x == 0);
  const RouteTables tab = tables(tables_at, m.local);
  float4* const part = reinterpret_cast<float4*>(tables_at + (route_bytes(m.local, (int64_t)m.tokens * m.top_k) + 15) / 16 * 16);
  __shared__ uint8_t lists[kWarps][kTokens];
  uint8_t* const list = lists[warp];

  const int strips = (int)((m.width + 7) / 8);
  const int64_t items = (int64_t)reinterpret_cast<const Routes*>(tables_at)->active * strips, bytes = m.hidden * 2;
  const int turns = (int)((bytes + kWarps * kPieceBytes - 1) / (kWarps * kPieceBytes));
  const char *bg = static_cast<const char*>(m.w_gate), *bu = static_cast<const char*>(m.w_up), *bx = static_cast<const char*>(m.x);
  const int64_t extent = ((m.local - 1) * m.esw + (m.width - 1) * m.ldw + m.hidden) * 2;
  const char* ex = bx + ((m.tokens - 1) * m.ldx + m.hidden) * 2;

  // What is copied next: turn next_turn of item next, rows at wg and wu.
  int64_t next = blockIdx.x;
  int next_turn = 0;
  const char *wg = nullptr, *wu = nullptr;
  const auto fetch = [&](int stage) {
    if (next < items) {
      if (next_turn == 0) {
        const int place = (int)(next / strips), e = tab.number[place];
        const int64_t f = min((next - (int64_t)place * strips) * 8 + g8, m.width - 1), at = (e * m.esw + f * m.ldw) * 2;
        wg = bg + at, wu = bu + at;
      }
      const int64_t k = (int64_t)(next_turn * kWarps + warp) * kPieceBytes;
      if (k < bytes) ring.fetch<VEC>(stage, wg, wu, k, bytes, bg, bu, extent);
      if (++next_turn == turns) next_turn = 0, next += gridDim.x;
    }
    Ring::commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(i);

  int stage = 0;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int place = (int)(item / strips), e = tab.number[place];
    const int64_t f0 = (item - (int64_t)place * strips) * 8;
    const uint32_t tokens = tab.tokens[e];
    const int count = __popc(tokens);
    __syncwarp();
    if (tokens >> lane & 1) list[__popc(tokens & ((1u << lane) - 1))] = (uint8_t)lane;
    __syncwarp();
    const auto run = [&](auto blocks) {
      constexpr int NB = decltype(blocks)::value;
      const char* xs[NB];
#pragma unroll
      for (int j = 0; j < NB; ++j) xs[j] = 8 * j + g8 < count ? bx + list[8 * j + g8] * m.ldx * 2 : nullptr;
      float acc[NB][4] = {};
      for (int turn = 0; turn < turns; ++turn) {
        fetch(stage == 0 ? kStages - 1 : stage - 1);
        const int64_t k0 = (int64_t)(turn * kWarps + warp) * kPieceBytes + 16 * t4;
        uint4 x[kSteps][NB];
        if (k0 - 16 * t4 < bytes) {
#pragma unroll
          for (int i = 0; i < kSteps; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j)
              x[i][j] = xs[j] ? tokens16<VEC>(xs[j] + k0 + 64 * i, bytes - k0 - 64 * i, bx, ex) : make_uint4(0, 0, 0, 0);
          Ring::wait();
#pragma unroll
          for (int i = 0; i < kSteps; ++i)
            multiply<E, NB>(acc, *reinterpret_cast<const uint4*>(ring.at(stage, i, 0)), *reinterpret_cast<const uint4*>(ring.at(stage, i, 1)), x[i]);
        }
        stage = stage == kStages - 1 ? 0 : stage + 1;
      }
#pragma unroll
      for (int j = 0; j < NB; ++j) part[(warp * NB + j) * 32 + lane] = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
      __syncthreads();
      if (warp < NB) {
        float v[4] = {};
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float4 p = part[(w * NB + warp) * 32 + lane];
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
    };
    if (count <= 8)
      run(std::integral_constant<int, 1>());
    else if (count <= 16)
      run(std::integral_constant<int, 2>());
    else
      run(std::integral_constant<int, 4>());
  }
}

// Sixteen output columns are a tile, for which there are as many units as pieces
// of 64 of the used experts' inner columns.  All tiles' units are dealt out evenly in one
// row, so that every SM reads as much; a CTA's part of a tile is shared out among its
// warps in runs.  A run's sums of one expert's tokens (eight at a time) are weighted and
// added to the warp's own sums in fp32, and those are joined in the warps' order.  A tile that
// lies on several CTAs is left in parts, which the CTA that finishes last
// adds in their order: nothing is waited for, and every call gives the same bits.
template <class E, bool VEC>
__global__ void __launch_bounds__(kThreads, 1) k_moe_down(MoeArgs m) {
  extern __shared__ __align__(16) char smem[];
  char* const tables_at = smem + kRingBytes;
  const Ring ring(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g8 = lane >> 2, t4 = lane & 3;
  // The kernel before this one, which made h, has itself waited for what came before
  // it: the logits and the weights may be read before it ends.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  route(m, tables_at, false);
  const Routes& s = *reinterpret_cast<const Routes*>(tables_at);
  const RouteTables tab = tables(tables_at, m.local);
  // sums[warp][token][16], 17 apart against bank conflicts
  float* const sums = reinterpret_cast<float*>(tables_at + (route_bytes(m.local, (int64_t)m.tokens * m.top_k) + 15) / 16 * 16);
  __shared__ uint8_t lists[kWarps][kTokens];
  __shared__ int finished;
  uint8_t* const list = lists[warp];
  const int entries = m.tokens * 17;
  float* const own = sums + warp * entries;

  const int64_t tiles = (m.hidden + 15) / 16, bytes = m.width * 2;
  const int pieces = (int)((bytes + kPieceBytes - 1) / kPieceBytes), units = s.active * pieces;
  const int64_t total = tiles * units;
  const int G = (int)min((int64_t)gridDim.x, total);  // CTAs that have a part, none of it empty
  const char* bd = static_cast<const char*>(m.w_down);
  const int64_t extent = ((m.local - 1) * m.esd + (m.hidden - 1) * m.ldd + m.width) * 2;
  const char* h = static_cast<const char*>(m.h);

  if (units == 0) {  // no token has an expert here
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < m.tokens * m.hidden; i += (int64_t)gridDim.x * kThreads)
      static_cast<uint16_t*>(m.out)[i / m.hidden * m.ldo + i % m.hidden] = 0;
    return;
  }
  // This CTA's part of the row of units, and this warp's run of a tile's.
  const int64_t cta = min((int)blockIdx.x, G), begin = cta * total / G, end = min(cta + 1, (int64_t)G) * total / G;
  struct Run {
    int64_t tile, pos;  // pos: where the CTA's part of the tile begins
    int u0, u1;         // that part
    int at, stop;       // this warp's run
  };
  const auto run_at = [&](int64_t pos) {
    Run r;
    r.pos = pos, r.tile = pos / units, r.u0 = (int)(pos - r.tile * units);
    r.u1 = (int)min((int64_t)units, r.u0 + (end - pos));
    const int n = r.u1 - r.u0, each = (n + kWarps - 1) / kWarps;
    r.at = r.u0 + min(warp * each, n), r.stop = r.u0 + min((warp + 1) * each, n);
    return r;
  };
  Run next = begin < end ? run_at(begin) : Run{0, end, 0, 0, 0, 0};
  const auto fetch = [&](int stage) {
    while (next.at >= next.stop && next.pos < end) {
      const int64_t pos = next.pos + (next.u1 - next.u0);
      if (pos >= end) {
        next.pos = end;
        break;
      }
      next = run_at(pos);
    }
    if (next.pos < end) {
      const int place = next.at / pieces, e = tab.number[place];
      const int64_t n0 = next.tile * 16, ra = min(n0 + g8, m.hidden - 1), rb = min(n0 + g8 + 8, m.hidden - 1);
      const char* we = bd + e * m.esd * 2;
      ring.fetch<VEC>(stage, we + ra * m.ldd * 2, we + rb * m.ldd * 2, (int64_t)(next.at - place * pieces) * kPieceBytes, bytes, bd, bd, extent);
      ++next.at;
    }
    Ring::commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(i);
  asm volatile("griddepcontrol.wait;" ::: "memory");

  int stage = 0;
  for (int64_t pos = begin; pos < end;) {
    const Run r = run_at(pos);
    for (int i = lane; i < entries; i += 32) own[i] = 0.0f;
    int u = r.at;
    while (u < r.stop) {
      const int place = u / pieces, until = min(r.stop, (place + 1) * pieces);
      const uint32_t tokens = tab.tokens[tab.number[place]];
      const int count = __popc(tokens);
      __syncwarp();
      if (tokens >> lane & 1) list[__popc(tokens & ((1u << lane) - 1))] = (uint8_t)lane;
      __syncwarp();
      const auto run = [&](auto blocks) {
        constexpr int NB = decltype(blocks)::value;
        const char* xs[NB];
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const int t = 8 * j + g8 < count ? list[8 * j + g8] : -1;
          xs[j] = t < 0 ? nullptr : h + (int64_t)(t * m.top_k + tab.choice[place * kTokens + t]) * m.ldh * 2;
        }
        float acc[NB][4] = {};
        for (; u < until; ++u) {
          fetch(stage == 0 ? kStages - 1 : stage - 1);
          const int64_t k0 = (int64_t)(u - place * pieces) * kPieceBytes + 16 * t4;
          uint4 x[kSteps][NB];
#pragma unroll
          for (int i = 0; i < kSteps; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j)  // rows of h start on 16 bytes and end in zeros
              x[i][j] = xs[j] && k0 + 64 * i < bytes ? *reinterpret_cast<const uint4*>(xs[j] + k0 + 64 * i) : make_uint4(0, 0, 0, 0);
          Ring::wait();
#pragma unroll
          for (int i = 0; i < kSteps; ++i)
            multiply<E, NB>(acc, *reinterpret_cast<const uint4*>(ring.at(stage, i, 0)), *reinterpret_cast<const uint4*>(ring.at(stage, i, 1)), x[i]);
          stage = stage == kStages - 1 ? 0 : stage + 1;
        }
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int i = 8 * j + 2 * t4 + c;
            if (i >= count) continue;
            const int t = list[i];
            const float w = s.weight[t][tab.choice[place * kTokens + t]];
            own[t * 17 + g8] = __fmaf_rn(w, acc[j][c], own[t * 17 + g8]);
            own[t * 17 + g8 + 8] = __fmaf_rn(w, acc[j][c + 2], own[t * 17 + g8 + 8]);
          }
      };
      if (count <= 8)
        run(std::integral_constant<int, 1>());
      else if (count <= 16)
        run(std::integral_constant<int, 2>());
      else
        run(std::integral_constant<int, 4>());
    }
    __syncthreads();
    const bool whole = r.u0 == 0 && r.u1 == units;
    float* const mine = m.parts + ((int64_t)blockIdx.x * 2 + (r.u0 == 0)) * kTokens * 16;
    for (int i = threadIdx.x; i < m.tokens * 16; i += kThreads) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += sums[w * entries + i / 16 * 17 + i % 16];
      const int64_t n = r.tile * 16 + i % 16;
      if (!whole)
        mine[i] = v;
      else if (n < m.hidden)
        static_cast<uint16_t*>(m.out)[i / 16 * m.ldo + n] = (uint16_t)E::from_f32(v);
    }
    if (!whole) {
      // CTA c has unit p of the row where c is the last whose part begins at or before p.
      const int64_t p0 = r.tile * units, p1 = p0 + units - 1;
      const int c0 = (int)(((p0 + 1) * G - 1) / total), c1 = (int)(((p1 + 1) * G - 1) / total);
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) finished = atomicAdd(&m.done[r.tile], 1u) == (uint32_t)(c1 - c0);
      __syncthreads();
      if (finished) {
        __threadfence();
        for (int i = threadIdx.x; i < m.tokens * 16; i += kThreads) {
          float v = 0.0f;
          for (int c = c0; c <= c1; ++c) v += __ldcg(m.parts + ((int64_t)c * 2 + (c == c0)) * kTokens * 16 + i);
          const int64_t n = r.tile * 16 + i % 16;
          if (n < m.hidden) static_cast<uint16_t*>(m.out)[i / 16 * m.ldo + n] = (uint16_t)E::from_f32(v);
        }
      }
    }
    __syncthreads();
    pos += r.u1 - r.u0;
  }
}

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <class E, int ACT>
cudaError_t moe(const MoeArgs& m, int num_sms, cudaStream_t s) {
  const int64_t pairs = (int64_t)m.tokens * m.top_k, most = m.local < pairs ? m.local : pairs, strips = (m.width + 7) / 8;
  const size_t tables = (route_bytes(m.local, pairs) + 15) / 16 * 16;
  const size_t blocks = m.tokens <= 8 ? 1 : m.tokens <= 16 ? 2 : 4;
  const size_t gated = kRingBytes + tables + kWarps * blocks * 512, down = kRingBytes + tables + (size_t)kWarps * m.tokens * 17 * 4;
  const bool vec = on16(m.x) && on16(m.w_gate) && on16(m.w_up) && (m.ldx | m.ldw | m.esw) % 8 == 0;
  auto* k = vec ? k_moe_gated<E, ACT, true> : k_moe_gated<E, ACT, false>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)gated);
  if (e != cudaSuccess) return e;
  const int64_t slots = num_sms < kMostSms ? num_sms : kMostSms, items = most * strips;
  e = launch_op(k, dim3((unsigned)(items < slots ? items : slots)), kThreads, gated, 1, s, m);
  if (e != cudaSuccess) return e;
  auto* d = on16(m.w_down) && (m.ldd | m.esd) % 8 == 0 ? k_moe_down<E, true> : k_moe_down<E, false>;
  e = cudaFuncSetAttribute(d, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)down);
  if (e != cudaSuccess) return e;
  return launch_op(d, dim3((unsigned)slots), kThreads, down, 1, s, m);
}

}  // namespace

size_t moe_scratch(int64_t tokens, int64_t top_k, int64_t width, int64_t hidden, MoeArgs* m, char* base) {
  const size_t ldh = (size_t)(width + 7) / 8 * 8, t = tokens < kTokens ? tokens : kTokens;
  const size_t h = (t * top_k * ldh * 2 + 15) / 16 * 16, done = ((size_t)(hidden + 15) / 16 * 4 + 15) / 16 * 16;
  if (m) {
    m->h = base, m->ldh = (int64_t)ldh;
    m->done = reinterpret_cast<uint32_t*>(base + h);
    m->parts = reinterpret_cast<float*>(base + h + done);
  }
  return h + done + (size_t)kMostSms * 2 * kTokens * 16 * 4;
}

cudaError_t launch_moe(int dtype, int act, const MoeArgs& m, int num_sms, cudaStream_t s) {
  if (dtype == AR_BF16) return act == AR_ACT_SILU ? moe<Bf16, AR_ACT_SILU>(m, num_sms, s) : moe<Bf16, AR_ACT_GELU_TANH>(m, num_sms, s);
  return act == AR_ACT_SILU ? moe<F16, AR_ACT_SILU>(m, num_sms, s) : moe<F16, AR_ACT_GELU_TANH>(m, num_sms, s);
}

}  // namespace ar
