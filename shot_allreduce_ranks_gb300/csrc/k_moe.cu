// A layer of gated feed-forward experts for a few tokens (formulas in
// include/ar.h), in two kernels: the gated products of the experts that have
// tokens, then the down products summed over each token's experts.
//
// Each used expert's matrices are read once, and memory bounds both kernels: one
// CTA an SM walks over its part of the matrices, and each of its warps copies the
// next pieces of its own (kStages - 1 of 2 KB: 64 KB an SM in flight) into shared memory
// while it multiplies.  A lane copies just the 16 bytes that it will use, so
// a warp waits for nothing but its own copies.  A CTA finds the routing for itself from the
// logits: a few hundred instructions, against a kernel of its own and its launch.
//
// Measured on one GB300: 32 tokens through 8 of 64 experts 2048 -> 1024 160-167 us (794 MB: 70-73% of the copy
// rate), 1 token through 4 of 32 experts 5120 -> 1736 49.8 (213 MB: 63%), 9 tokens on half of 16 experts 2048 -> 1032 28 (71
// MB). While it runs each loop reads at the copy rate (77 us for 520 MB, 20 for 142); what is left is the
// routing (2.3 us at one token, 4.2 at 32), the first pieces' way (1.7), the joining of sums (2
// to 5) and the start of the second kernel, whose registers leave no room beside the first's. Eight warps with
// longer rings were slower (62 us at one token), and so was a barrier for every item (240 at 32).
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

// A logit's bits as they are stored, and its value.
__device__ __forceinline__ uint32_t logit_bits(const MoeArgs& m, int t, int e) {
  const char* p = static_cast<const char*>(m.logits);
  const int64_t i = t * m.ldl + e;
  return m.logits_dtype == AR_FP32 ? ld_elem<4>(p + 4 * i) : ld_elem<2>(p + 2 * i);
}
__device__ __forceinline__ float logit_value(const MoeArgs& m, uint32_t bits) {
  return m.logits_dtype == AR_FP32 ? __uint_as_float(bits) : m.logits_dtype == AR_BF16 ? Bf16::to_f32(bits) : F16::to_f32(bits);
}

// A token's choices by one warp: lane j gets the j-th (its order and expert); lanes' parts of the sum of all experts'
// exponentials in `total` where that is wanted.
// R > 0: up to 32 R experts, whose bits are in `raw`; 0: any number, read again for every choice.
template <int R>
__device__ __forceinline__ void choose(const MoeArgs& m, int t, int lane, const uint32_t (&raw)[R ? R : 1], uint32_t& mine, int& expert,
                                       float& total) {
  constexpr int N = R ? R : 1;
  uint32_t o[N];
  if (R)
#pragma unroll
    for (int r = 0; r < N; ++r) o[r] = 32 * r + lane < m.experts ? order_of(logit_value(m, raw[r])) : 0;
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
        const uint32_t v = order_of(logit_value(m, logit_bits(m, t, i)));
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
  if (!m.normalize) {
    const float first = value_of(__shfl_sync(0xFFFFFFFFu, mine, 0));
    if (R) {
#pragma unroll
      for (int r = 0; r < N; ++r)
        if (32 * r + lane < m.experts) total += expf(logit_value(m, raw[r]) - first);
    } else {
      for (int i = lane; i < m.experts; i += 32) total += expf(logit_value(m, logit_bits(m, t, i)) - first);
    }
  }
}

// The choices of a warp's tokens; all of a token's logits are loaded at once, the next token's before this one's choices.
template <int R>
__device__ __forceinline__ void choose_all(const MoeArgs& m, Routes& s, const RouteTables& tab, bool write) {
  constexpr int N = R ? R : 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t raw[N], next[N];
  const auto load = [&](int t, uint32_t(&v)[N]) {
    if (R)
#pragma unroll
      for (int r = 0; r < N; ++r) v[r] = t < m.tokens && 32 * r + lane < m.experts ? logit_bits(m, t, 32 * r + lane) : 0;
  };
  load(warp, raw);
  for (int e = threadIdx.x; e < m.local; e += kThreads) tab.tokens[e] = 0;
  __syncthreads();
  for (int t = warp; t < m.tokens; t += kWarps) {
    load(t + kWarps, next);
    uint32_t mine;
    int expert;
    float total;
    choose<R>(m, t, lane, raw, mine, expert, total);
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
#pragma unroll
    for (int r = 0; r < N; ++r) raw[r] = next[r];
  }
}

// The routing by a whole CTA; write: it also stores it for the caller.
__device__ __forceinline__ void route(const MoeArgs& m, char* smem, bool write) {
  Routes& s = *reinterpret_cast<Routes*>(smem);
  const RouteTables tab = tables(smem, m.local);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (m.experts <= 64)
    choose_all<2>(m, s, tab, write);
  else if (m.experts <= 256)
    choose_all<8>(m, s, tab, write);
  else
    choose_all<0>(m, s, tab, write);
  __syncthreads();
  // Every warp counts the active experts for itself, and stores its share of them.
  int count = 0;
  for (int base = 0; base < m.local; base += 32) {
    const int e = base + lane;
    const uint32_t with = __ballot_sync(0xFFFFFFFFu, e < m.local && tab.tokens[e] != 0);
    if (base / 32 % kWarps == warp && with >> lane & 1) {
      const int at = count + __popc(with & ((1u << lane) - 1));
      tab.place[e] = (uint16_t)at, tab.number[at] = (uint16_t)e;
    }
    count += __popc(with);
  }
  if (threadIdx.x == 0) s.active = count;
  __syncthreads();
  for (int i = threadIdx.x; i < kTokens * m.top_k; i += kThreads) {
    const int t = i % kTokens, j = i / kTokens;
    if (t >= m.tokens) continue;
    const int e = s.expert[t][j] - m.first;
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
constexpr int kStages = 3, kSteps = 2, kPieceBytes = 128, kStageBytes = kSteps * 2 * 512, kRingBytes = kWarps * kStages * kStageBytes;

__device__ __forceinline__ void copy16(uint32_t to, const char* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_some(uint32_t to, const char* from, int bytes) {  // the rest of the 16 is zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}

// What a warp copies next: `more` pieces of this lane's rows, now at a and b (its 16 bytes of the
// first step), of which `left` bytes remain from the piece's begin on.
struct Feed {
  const char *a, *b;
  int left, more;
};

struct Ring {
  uint32_t mine;  // this lane's place in its warp's ring
  int stage;      // the one that is used next
  __device__ __forceinline__ explicit Ring(char* smem)
      : mine((uint32_t)__cvta_generic_to_shared(smem) + (threadIdx.x >> 5) * kStages * kStageBytes + (threadIdx.x & 31) * 16), stage(0) {}
  __device__ __forceinline__ uint4 row(int step, int r) const {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(mine + stage * kStageBytes + (step * 2 + r) * 512)
                 : "memory");
    return v;
  }
  static __device__ __forceinline__ void put(uint32_t to, const uint4& v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(to), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
  }
  __device__ __forceinline__ void advance() { stage = stage == kStages - 1 ? 0 : stage + 1; }

  // The next piece to the stage that is `ahead` of the one used next; the matrices' ends bound what is read where
  // rows begin anywhere.  What lies past a row's end is zeros.
  template <bool VEC>
  __device__ __forceinline__ void fetch(int ahead, Feed& f, const char* begin_a, const char* begin_b, int64_t extent) const {
    if (f.more > 0) {
      const int to_stage = stage + ahead < kStages ? stage + ahead : stage + ahead - kStages;
      const uint32_t at = mine + to_stage * kStageBytes;
      if (VEC) {
        if (f.left >= kPieceBytes) {
#pragma unroll
          for (int i = 0; i < kSteps; ++i) {
            copy16(at + i * 1024, f.a + 64 * i);
            copy16(at + i * 1024 + 512, f.b + 64 * i);
          }
        } else {
#pragma unroll
          for (int i = 0; i < kSteps; ++i) {
            const int left = f.left - 64 * i - 16 * (int)(threadIdx.x & 3), n = left >= 16 ? 16 : left > 0 ? left : 0;
            copy_some(at + i * 1024, n ? f.a + 64 * i : begin_a, n);
            copy_some(at + i * 1024 + 512, n ? f.b + 64 * i : begin_b, n);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const int left = f.left - 64 * i - 16 * (int)(threadIdx.x & 3);
          put(at + i * 1024, load_anywhere<2>(f.a + 64 * i, left, begin_a, begin_a + extent));
          put(at + i * 1024 + 512, load_anywhere<2>(f.b + 64 * i, left, begin_b, begin_b + extent));
        }
      }
      f.a += kPieceBytes, f.b += kPieceBytes, f.left -= kPieceBytes, --f.more;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
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

// The first of `total` that share r has of n even ones: total / n each, and one more for the first total % n.
__device__ __forceinline__ int share(int r, int total, int n) { return r * (total / n) + min(r, total % n); }
__device__ __forceinline__ int warp_share(int w, int total) { return share(w, total, kWarps); }
// Which share has number p.
__device__ __forceinline__ int share_of(int p, int total, int n) {
  const int each = total / n, longer = total % n;
  return p < longer * (each + 1) ? p / (each + 1) : longer + (p - longer * (each + 1)) / max(each, 1);
}

// An item: eight rows of one expert's gate and the same of its up projection, whose
// sums of one output land in one lane.  A CTA has as many items as the others; their pieces along k, one
// item's behind the other's, are dealt out evenly to its warps.  A warp finishes the
// items that are its own; those that lie on several warps are joined once, at the end,
// in the warps' order.
template <class E, int ACT, bool VEC>
__global__ void __launch_bounds__(kThreads, 1) k_moe_gated(MoeArgs m) {
  extern __shared__ __align__(16) char smem[];
  pdl_enter();
  char* const tables_at = smem + kRingBytes;
  Ring ring(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g8 = lane >> 2, t4 = lane & 3;
  // The down kernel's counts of finished parts.
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < (m.hidden + 15) / 16; i += (int64_t)gridDim.x * kThreads) m.done[i] = 0;
  route(m, tables_at, blockIdx.x == 0);
  const RouteTables tab = tables(tables_at, m.local);
  // Sums of the items that a warp has a part of: that which begins before it, and that which ends behind it.
  const int blocks = m.tokens <= 8 ? 1 : m.tokens <= 16 ? 2 : 4;
  float4* const part = reinterpret_cast<float4*>(tables_at + (route_bytes(m.local, (int64_t)m.tokens * m.top_k) + 15) / 16 * 16);
  const auto part_at = [&](int w, int which) { return part + (w * 2 + which) * blocks * 32 + lane; };
  __shared__ uint8_t lists[kWarps][kTokens];
  uint8_t* const list = lists[warp];

  const int strips = (int)((m.width + 7) / 8), bytes = (int)m.hidden * 2, pieces = (bytes + kPieceBytes - 1) / kPieceBytes;
  const int items = reinterpret_cast<const Routes*>(tables_at)->active * strips;
  const int item0 = share(blockIdx.x, items, (int)gridDim.x), total = (share(blockIdx.x + 1, items, (int)gridDim.x) - item0) * pieces;
  if (total == 0) return;
  const int first = warp_share(warp, total), last = warp_share(warp + 1, total);
  const char *bg = static_cast<const char*>(m.w_gate), *bu = static_cast<const char*>(m.w_up), *bx = static_cast<const char*>(m.x);
  const int64_t extent = ((m.local - 1) * m.esw + (m.width - 1) * m.ldw + m.hidden) * 2;
  const char* ex = bx + ((m.tokens - 1) * m.ldx + m.hidden) * 2;

  Feed feed = {nullptr, nullptr, 0, 0};
  int fed = first;  // pieces before this one have been given to `feed`
  const auto fetch = [&](int ahead) {
    if (feed.more == 0 && fed < last) {
      const int q = fed / pieces, p = fed - q * pieces, place = (item0 + q) / strips;
      const int64_t f = min((int64_t)(item0 + q - place * strips) * 8 + g8, m.width - 1);
      const int64_t at = (tab.number[place] * m.esw + f * m.ldw) * 2 + p * kPieceBytes + 16 * t4;
      feed = {bg + at, bu + at, bytes - p * kPieceBytes, min(pieces - p, last - fed)};
      fed += feed.more;
    }
    ring.fetch<VEC>(ahead, feed, bg, bu, extent);
  };
#pragma unroll 1
  for (int i = 0; i < kStages - 1; ++i) fetch(i);

  // An item's expert, its tokens in `list`, their number.
  const auto open = [&](int item, int& place) {
    place = item / strips;
    const uint32_t tokens = tab.tokens[tab.number[place]];
    __syncwarp();
    if (tokens >> lane & 1) list[__popc(tokens & ((1u << lane) - 1))] = (uint8_t)lane;
    __syncwarp();
    return __popc(tokens);
  };
  const auto finish = [&](int item, int place, int count, int j, const float4& v) {
    const int f = (item - place * strips) * 8 + g8;
    const float sums[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int i = 8 * j + 2 * t4 + c;
      if (i >= count) continue;
      const int t = list[i];
      const int64_t row = t * m.top_k + tab.choice[place * kTokens + t];
      // The row's end, up to a whole group, is read with it: zeros.
      const float h = f < m.width ? act_value<ACT>(sums[c]) * sums[c + 2] : 0.0f;
      const uint32_t rounded = E::from_f32(h);
      static_cast<uint16_t*>(m.h)[row * m.ldh + f] = (uint16_t)rounded;
      // What the rounding left goes to the second product beside it, so that 16 (bfloat16) or 22 (float16) bits of h
      // reach the result; an infinity has nothing left, for a NaN beside it would spoil an infinite sum.
      if (m.h_rest) {
        const float there = E::to_f32(rounded);
        static_cast<uint16_t*>(m.h_rest)[row * m.ldh + f] = fabsf(there) < INFINITY ? (uint16_t)E::from_f32(h - there) : (uint16_t)0;
      }
    }
  };

  for (int pos = first; pos < last;) {
    const int q = pos / pieces, p0 = pos - q * pieces, p1 = min(pieces, p0 + (last - pos));
    int place;
    const int count = open(item0 + q, place);
    const auto run = [&](auto number) {
      constexpr int NB = decltype(number)::value;
      // A token past the last is read as the last: its column of the sums is dropped.
      const char* xs[NB];
#pragma unroll
      for (int j = 0; j < NB; ++j) xs[j] = bx + list[min(8 * j + g8, count - 1)] * m.ldx * 2 + p0 * kPieceBytes + 16 * t4;
      float acc[NB][4] = {};
      const auto step = [&](auto whole, int left) {
        uint4 x[kSteps][NB];
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
#pragma unroll
          for (int j = 0; j < NB; ++j)
            x[i][j] = tokens16<VEC>(xs[j] + 64 * i, decltype(whole)::value && VEC ? 16 : left - 64 * i - 16 * t4, bx, ex);
        fetch(kStages - 1);
        Ring::wait();
#pragma unroll
        for (int i = 0; i < kSteps; ++i) multiply<E, NB>(acc, ring.row(i, 0), ring.row(i, 1), x[i]);
        ring.advance();
#pragma unroll
        for (int j = 0; j < NB; ++j) xs[j] += kPieceBytes;
      };
      const int whole = min(p1, bytes / kPieceBytes);
      int p = p0;
      for (; p < whole; ++p) {
        step(std::true_type(), bytes - p * kPieceBytes);
      }
      for (; p < p1; ++p) {
        step(std::false_type(), bytes - p * kPieceBytes);
      }
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const float4 v = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
        if (p1 - p0 == pieces)
          finish(item0 + q, place, count, j, v);
        else
          part_at(warp, p0 == 0)[j * 32] = v;
      }
    };
    if (count <= 8)
      run(std::integral_constant<int, 1>());
    else if (count <= 16)
      run(std::integral_constant<int, 2>());
    else
      run(std::integral_constant<int, 4>());
    pos += p1 - p0;
  }
  __syncthreads();
  // An item that this warp begins and does not end.
  const int q = max(last - 1, 0) / pieces, end = q * pieces + pieces;
  if (first < last && last < end && q * pieces >= first) {
    // the last warp that has a part of it
    const int until = __popc(__ballot_sync(0xFFFFFFFFu, lane < kWarps && warp_share(lane, total) < end)) - 1;
    int place;
    const int count = open(item0 + q, place);
    for (int j = 0; 8 * j < count; ++j) {
      float4 v = part_at(warp, 1)[j * 32];
      for (int w = warp + 1; w <= until; ++w) {
        const float4 t = part_at(w, 0)[j * 32];
        v.x += t.x, v.y += t.y, v.z += t.z, v.w += t.w;
      }
      finish(item0 + q, place, count, j, v);
    }
  }
}

// Sixteen output columns are a tile, for which there are as many units as pieces
// of 64 of the used experts' inner columns.  All tiles' units are dealt out evenly in one
// row, first to the CTAs, then to a CTA's warps, so that every SM reads as much.  A
// warp's sums of one expert's tokens (eight at a time) are weighted and added to its
// sums of the tile in fp32, and those are joined at the end, in the warps' order.  A
// tile that lies on several CTAs is left in parts, which the CTA that finishes last
// adds in their order: nothing is waited for, and every call gives the same bits.
//
// TWO: h is the sum of two numbers, each of which meets the weights in registers; one call of 1 token 49.8 us (with h
// rounded to one 49.0), of 32 tokens 167 (161), of 32 through 8 experts 56 (50).
template <class E, bool VEC, bool TWO>
__global__ void __launch_bounds__(kThreads, 1) k_moe_down(MoeArgs m) {
  extern __shared__ __align__(16) char smem[];
  char* const tables_at = smem + kRingBytes;
  Ring ring(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g8 = lane >> 2, t4 = lane & 3;
  // The kernel before this one, which made h, has itself waited for what came before
  // it: the logits and the weights may be read before it ends.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  route(m, tables_at, false);
  const Routes& s = *reinterpret_cast<const Routes*>(tables_at);
  const RouteTables tab = tables(tables_at, m.local);
  __shared__ uint8_t lists[kWarps][kTokens];
  __shared__ int finished[2];
  uint8_t* const list = lists[warp];
  // A warp's sums of the tile that begins before its run, and of that which ends behind it (or, whole, of
  // any between): [token][16], 17 apart against bank conflicts.
  float* const sums = reinterpret_cast<float*>(tables_at + (route_bytes(m.local, (int64_t)m.tokens * m.top_k) + 15) / 16 * 16);
  const int entries = m.tokens * 17;
  const auto sums_of = [&](int w, int which) { return sums + (w * 2 + which) * entries; };

  const int tiles = (int)((m.hidden + 15) / 16), bytes = (int)m.width * 2, pieces = (bytes + kPieceBytes - 1) / kPieceBytes, active = s.active;
  const int units = active * pieces, total = tiles * units;
  const char* bd = static_cast<const char*>(m.w_down);
  const int64_t extent = ((m.local - 1) * m.esd + (m.hidden - 1) * m.ldd + m.width) * 2;
  const char* h = static_cast<const char*>(m.h);
  const int64_t to_rest = TWO ? static_cast<const char*>(m.h_rest) - h : 0;
  uint16_t* const out = static_cast<uint16_t*>(m.out);

  if (units == 0) {  // no token has an expert here
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < m.tokens * m.hidden; i += (int64_t)gridDim.x * kThreads)
      out[i / m.hidden * m.ldo + i % m.hidden] = 0;
    return;
  }
  const int begin = share(blockIdx.x, total, (int)gridDim.x), mine = share(blockIdx.x + 1, total, (int)gridDim.x) - begin, end = begin + mine;
  if (mine == 0) return;
  const auto begin_of = [&](int w) { return begin + warp_share(w, mine); };
  const int first = begin_of(warp), last = begin_of(warp + 1);

  Feed feed = {nullptr, nullptr, 0, 0};
  int fed = first;  // units before this one have been given to `feed`
  const auto fetch = [&](int ahead) {
    if (feed.more == 0 && fed < last) {
      const int q = fed / pieces, p = fed - q * pieces, tile = q / active, place = q - tile * active;
      const int64_t n0 = (int64_t)tile * 16, ra = min(n0 + g8, m.hidden - 1), rb = min(n0 + g8 + 8, m.hidden - 1);
      const char* from = bd + tab.number[place] * m.esd * 2 + (int64_t)p * kPieceBytes + 16 * t4;
      feed = {from + ra * m.ldd * 2, from + rb * m.ldd * 2, bytes - p * kPieceBytes, min(pieces - p, last - fed)};
      fed += feed.more;
    }
    ring.fetch<VEC>(ahead, feed, bd, bd, extent);
  };
#pragma unroll 1
  for (int i = 0; i < kStages - 1; ++i) fetch(i);
  for (int i = lane; i < 2 * entries; i += 32) sums_of(warp, 0)[i] = 0.0f;
  asm volatile("griddepcontrol.wait;" ::: "memory");

  for (int pos = first; pos < last;) {
    // One expert's units of a tile.
    const int q = pos / pieces, p0 = pos - q * pieces, tile = q / active, place = q - tile * active, p1 = min(pieces, p0 + (last - pos));
    float* const own = sums_of(warp, tile * units >= first);
    const uint32_t tokens = tab.tokens[tab.number[place]];
    const int count = __popc(tokens);
    __syncwarp();
    if (tokens >> lane & 1) list[__popc(tokens & ((1u << lane) - 1))] = (uint8_t)lane;
    __syncwarp();
    const auto run = [&](auto blocks) {
      constexpr int NB = decltype(blocks)::value;
      constexpr bool EARLY = TWO && NB <= 2;  // four blocks leave no registers to load both parts ahead
      // A token past the last is read as the last: its column of the sums is dropped.
      const char* xs[NB];
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const int t = list[min(8 * j + g8, count - 1)];
        xs[j] = h + (int64_t)(t * m.top_k + tab.choice[place * kTokens + t]) * m.ldh * 2 + p0 * kPieceBytes + 16 * t4;
      }
      float acc[NB][4] = {};
      for (int p = p0; p < p1; ++p) {
        uint4 x[kSteps][NB], rest[EARLY ? kSteps : 1][NB];
        const int left = bytes - p * kPieceBytes - 16 * t4;
        const auto load = [&](uint4(&v)[NB], int i, int64_t from) {  // rows of h start on 16 bytes and end in zeros
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            v[j] = make_uint4(0, 0, 0, 0);
            if (left > 64 * i) v[j] = *reinterpret_cast<const uint4*>(xs[j] + from + 64 * i);
          }
        };
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          load(x[i], i, 0);
          if (EARLY) load(rest[EARLY ? i : 0], i, to_rest);
        }
        fetch(kStages - 1);
        Ring::wait();
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          if (TWO && !EARLY) load(rest[0], i, to_rest);
          const uint4 a = ring.row(i, 0), b = ring.row(i, 1);
          multiply<E, NB>(acc, a, b, x[i]);
          if (TWO) multiply<E, NB>(acc, a, b, rest[EARLY ? i : 0]);
        }
        ring.advance();
#pragma unroll
        for (int j = 0; j < NB; ++j) xs[j] += kPieceBytes;
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
    pos += p1 - p0;
    if (tile * units >= first && pos == (tile + 1) * units) {  // the whole tile was this warp's
      __syncwarp();
      for (int i = lane; i < m.tokens * 16; i += 32) {
        const int64_t n = (int64_t)tile * 16 + i % 16;
        if (n < m.hidden) out[i / 16 * m.ldo + n] = (uint16_t)E::from_f32(own[i / 16 * 17 + i % 16]);
        own[i / 16 * 17 + i % 16] = 0.0f;
      }
    }
  }
  // The tiles that lie on several warps are named by the first warp that has a part: the CTA's first, where another
  // CTA began it, and the one that a warp begins and does not end.
  __shared__ int split[kWarps + 1][2];  // tile (-1: none), its last warp
  const int tile0 = begin / units, tile1 = (end - 1) / units;
  const auto name = [&](int at, int tile, bool there) {
    const int until = __popc(__ballot_sync(0xFFFFFFFFu, lane < kWarps && begin_of(lane) < min((tile + 1) * units, end))) - 1;
    if (lane == 0) split[at][0] = there ? tile : -1, split[at][1] = until;
  };
  if (warp == 0) name(kWarps, tile0, tile0 * units < begin);
  const int my_last = max(last - 1, 0) / units;
  name(warp, my_last, first < last && my_last * units >= first && last < (my_last + 1) * units);
  __syncthreads();
  const auto part_of = [&](int cta, bool begun) { return m.parts + ((int64_t)cta * 2 + begun) * kTokens * 16; };
  const auto store = [&](int tile, int i, float v) {
    const int64_t n = (int64_t)tile * 16 + i % 16;
    if (n < m.hidden) out[i / 16 * m.ldo + n] = (uint16_t)E::from_f32(v);
  };
#pragma unroll 1
  for (int k = 0; k <= kWarps; ++k) {
    const int tile = split[k][0], until = split[k][1], w0 = k % kWarps;
    if (tile < 0) continue;
    const bool whole = k < kWarps && (tile + 1) * units <= end;
    for (int i = threadIdx.x; i < m.tokens * 16; i += kThreads) {
      const int at = i / 16 * 17 + i % 16;
      float v = sums_of(w0, k < kWarps)[at];
      for (int w = w0 + 1; w <= until; ++w) v += sums_of(w, 0)[at];
      if (whole)
        store(tile, i, v);
      else
        part_of(blockIdx.x, k < kWarps)[i] = v;
    }
  }
  if (tile0 * units == begin && (tile1 + 1) * units == end) return;
  __threadfence();
  __syncthreads();
  if (threadIdx.x < 2) {
    const int tile = threadIdx.x ? tile1 : tile0;
    finished[threadIdx.x] = -1;
    if ((tile * units < begin || (tile + 1) * units > end) && (threadIdx.x == 0 || tile1 != tile0)) {
      const int c0 = share_of(tile * units, total, (int)gridDim.x), c1 = share_of((tile + 1) * units - 1, total, (int)gridDim.x);
      if (atomicAdd(&m.done[tile], 1u) == (uint32_t)(c1 - c0)) finished[threadIdx.x] = c0 << 16 | c1;
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    if (finished[k] < 0) continue;
    __threadfence();
    const int tile = k ? tile1 : tile0, c0 = finished[k] >> 16, c1 = finished[k] & 0xFFFF;
    for (int i = threadIdx.x; i < m.tokens * 16; i += kThreads) {
      float v = __ldcg(part_of(c0, true) + i);
      for (int c = c0 + 1; c <= c1; ++c) v += __ldcg(part_of(c, false) + i);
      store(tile, i, v);
    }
  }
}

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <class E, int ACT>
cudaError_t moe(const MoeArgs& m, int num_sms, cudaStream_t s) {
  const int64_t pairs = (int64_t)m.tokens * m.top_k, most = m.local < pairs ? m.local : pairs, strips = (m.width + 7) / 8;
  const size_t tables = (route_bytes(m.local, pairs) + 15) / 16 * 16;
  const size_t blocks = m.tokens <= 8 ? 1 : m.tokens <= 16 ? 2 : 4;
  const size_t gated = kRingBytes + tables + kWarps * 2 * blocks * 512, down = kRingBytes + tables + (size_t)kWarps * 2 * m.tokens * 17 * 4;
  const bool vec = on16(m.x) && on16(m.w_gate) && on16(m.w_up) && (m.ldx | m.ldw | m.esw) % 8 == 0;
  // The kernels count items and units in 32 bits; the entry point refuses sizes beyond that.
  const int64_t slots = num_sms < kMostSms ? num_sms : kMostSms, items = most * strips;
  const dim3 grid((unsigned)(items < slots ? items : slots)), all((unsigned)slots);
  const cudaError_t e = vec ? launch_raised<k_moe_gated<E, ACT, true>>(grid, kThreads, gated, s, m)
                            : launch_raised<k_moe_gated<E, ACT, false>>(grid, kThreads, gated, s, m);
  if (e != cudaSuccess) return e;
  const bool vec_down = on16(m.w_down) && (m.ldd | m.esd) % 8 == 0;
  if (m.h_rest)
    return vec_down ? launch_raised<k_moe_down<E, true, true>>(all, kThreads, down, s, m)
                    : launch_raised<k_moe_down<E, false, true>>(all, kThreads, down, s, m);
  return vec_down ? launch_raised<k_moe_down<E, true, false>>(all, kThreads, down, s, m)
                  : launch_raised<k_moe_down<E, false, false>>(all, kThreads, down, s, m);
}

}  // namespace

size_t moe_scratch(int64_t tokens, int64_t top_k, int64_t width, int64_t hidden, bool two_parts, MoeArgs* m, char* base) {
  const size_t ldh = (size_t)(width + 7) / 8 * 8, t = tokens < kTokens ? tokens : kTokens;
  const size_t h = (t * top_k * ldh * 2 + 15) / 16 * 16, done = ((size_t)(hidden + 15) / 16 * 4 + 15) / 16 * 16;
  const size_t all = h + done + (size_t)kMostSms * 2 * kTokens * 16 * 4;
  if (m) {
    m->h = base, m->ldh = (int64_t)ldh;
    m->done = reinterpret_cast<uint32_t*>(base + h);
    m->parts = reinterpret_cast<float*>(base + h + done);
    m->h_rest = two_parts ? base + all : nullptr;
  }
  return two_parts ? all + h : all;
}

cudaError_t launch_moe(int dtype, int act, const MoeArgs& m, int num_sms, cudaStream_t s) {
  if (dtype == AR_BF16) return act == AR_ACT_SILU ? moe<Bf16, AR_ACT_SILU>(m, num_sms, s) : moe<Bf16, AR_ACT_GELU_TANH>(m, num_sms, s);
  return act == AR_ACT_SILU ? moe<F16, AR_ACT_SILU>(m, num_sms, s) : moe<F16, AR_ACT_GELU_TANH>(m, num_sms, s);
}

}  // namespace ar
