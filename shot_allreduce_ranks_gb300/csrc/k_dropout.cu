// Dropout whose mask is drawn from a counter-based generator and never stored.
//
// Element i of the whole tensor (i = offset + row * cols + column) is kept
// where draw(i) >= round(p 2^32); draw(i) is word i mod 4 of Philox4x32-10
// ("Parallel random numbers: as easy as 1, 2, 3", Salmon, Moraes, Dror, Shaw,
// 2011) of the 128-bit counter {i / 4, sequence} under the 64-bit key `seed`.
// The mask is a function of the element's place alone: every rank that holds
// a copy draws the same one without an exchange, a rank that holds a block
// draws its part by `offset`, and the backward pass draws it again.
//
// Bound by memory with a residual in 16 bits, 6 bytes an element; without one,
// nearest to the generator's multiplications (18 wide ones for 4 elements): their
// pipe is active 68% of the time, more than any other, and memory 53%; neither is
// full, nor was that pipe at 77% with 20 of them.  Measured on one
// GB300 (replayed graph): with residual 16384 x 8192 bf16 121.6 us (6.62 TB/s, 98%
// of a copy's rate); without 113 us (4.8 TB/s); fp32 without, 680 x 5120 at an odd
// place 8.8 us; one row of 5120 1.9 us, the launch.  A persistent grid of 5 CTAs
// an SM: 153 us; one run of groups a warp at a time instead of two: 143.
#include "ops_internal.cuh"

namespace ar {
namespace {

constexpr int kDropThreads = 256;
constexpr int kRuns = 2;  // of 32 groups that a warp takes at a time

constexpr uint32_t kMul0 = 0xD2511F53u, kMul1 = 0xCD9E8D57u;

// What a call's blocks share, computed on the host: the ten rounds' keys, and,
// where all block numbers have one upper word, the values of the first two
// rounds that do not depend on the lower one (two multiplications less of 20).
struct RoundKeys {
  uint32_t k0[10], k1[10];
  uint32_t c2_1;              // c3 ^ k1[0]
  uint32_t c0_2, c2_2, c3_2;  // c1' ^ k0[1];  high(c0' kMul0) ^ k1[1];  low(c0' kMul0)
};

template <bool ONE_UPPER>
__device__ __forceinline__ void philox(uint32_t (&d)[4], uint64_t block, uint64_t sequence, const RoundKeys& key) {
  uint32_t c0, c1, c2, c3;
  if (ONE_UPPER) {
    const uint64_t a = (uint64_t)(uint32_t)block * kMul0;
    const uint64_t b = (uint64_t)((uint32_t)(a >> 32) ^ key.c2_1) * kMul1;
    c0 = (uint32_t)(b >> 32) ^ key.c0_2;
    c1 = (uint32_t)b;
    c2 = (uint32_t)a ^ key.c2_2;
    c3 = key.c3_2;
  } else {
    c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32);
    c2 = (uint32_t)sequence, c3 = (uint32_t)(sequence >> 32);
  }
#pragma unroll
  for (int r = ONE_UPPER ? 2 : 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)c0 * kMul0, b = (uint64_t)c2 * kMul1;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ key.k0[r];
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ key.k1[r];
    c3 = (uint32_t)a;
  }
  d[0] = c0, d[1] = c1, d[2] = c2, d[3] = c3;
}

RoundKeys round_keys(uint64_t seed, uint64_t sequence, uint32_t upper) {
  RoundKeys key;
  for (int r = 0; r < 10; ++r) {
    key.k0[r] = (uint32_t)seed + (uint32_t)r * 0x9E3779B9u;
    key.k1[r] = (uint32_t)(seed >> 32) + (uint32_t)r * 0xBB67AE85u;
  }
  const uint64_t b = (sequence & 0xFFFFFFFFu) * kMul1;           // of the first round
  const uint32_t c0 = (uint32_t)(b >> 32) ^ upper ^ key.k0[0];  // after it
  const uint64_t a = (uint64_t)c0 * kMul0;                      // of the second
  key.c2_1 = (uint32_t)(sequence >> 32) ^ key.k1[0];
  key.c0_2 = (uint32_t)b ^ key.k0[1];
  key.c2_2 = (uint32_t)(a >> 32) ^ key.k1[1];
  key.c3_2 = (uint32_t)a;
  return key;
}

// Element k of a group of 16 bytes.  The lower bfloat16 of a word is moved up by
// a byte permutation: a shift compiles to a multiplication on the pipe that the
// generator's multiplications keep busy.
template <class E>
__device__ __forceinline__ float element(const uint32_t (&v)[4], int k) {
  if constexpr (IsBf16<E>::value) {
    if (k & 1) return E::hi(v[k / 2]);
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, 0x1044;" : "=r"(d) : "r"(v[k / 2]), "r"(0));
    return __uint_as_float(d);
  } else if constexpr (E::kBytes == 2) {
    return k & 1 ? E::hi(v[k / 2]) : E::lo(v[k / 2]);
  } else {
    return __uint_as_float(v[k]);
  }
}

template <class E, int G>
__device__ __forceinline__ void pack_group(uint32_t (&o)[4], const float (&y)[G]) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if constexpr (E::kBytes == 2)
      o[w] = E::pack(y[2 * w], y[2 * w + 1]);
    else
      o[w] = __float_as_uint(y[w]);
  }
}

// How a group's draws lie to the generator's blocks of four.  The first two
// also say that all blocks of the call have one upper word.
enum Phase {
  kWhole = 0,   // every group begins a block
  kShifted = 1, // groups follow one another in the element order, each beginning inside a block
  kAny = 2      // rows begin anywhere
};

// A warp takes U runs of 32 groups of 16 bytes, a lane one group of each.  A
// group's draws come from G/4 blocks; one that begins inside a block also
// wants words of the next block, which (kShifted) the next lane has drawn as
// its first, and the last lane finds in the next run's first lane, so that a
// warp draws one block more for its U runs instead of one for each group.
template <class E, bool RES, bool VEC, int PHASE>
__global__ void __launch_bounds__(kDropThreads)
    k_dropout(const __grid_constant__ DropoutArgs a, const __grid_constant__ RoundKeys key, int64_t groups_per_row) {
  pdl_enter();
  constexpr int G = E::kGroup, B = E::kBytes, W = 4, U = kRuns;
  const int64_t total = a.rows * groups_per_row;
  const int lane = (int)(threadIdx.x & 31);
  const int64_t warps = (int64_t)gridDim.x * (kDropThreads / 32);
  for (int64_t run = ((int64_t)blockIdx.x * (kDropThreads / 32) + (threadIdx.x >> 5)) * (32 * U); run < total;
       run += warps * (32 * U)) {
    uint32_t xw[U][W], rw[U][W], d[U][G + 4];
    int n[U];        // elements of the group
    char* po[U];
    uint64_t first[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = run + 32 * u + lane;
      int64_t col = i * G, ax = col, ar = col, ao = col;
      first[u] = a.offset + (uint64_t)col;
      if (a.rows > 1) {
        const int64_t row = total >> 32 ? i / groups_per_row
                                        : (int64_t)((uint32_t)i / (uint32_t)groups_per_row);
        col = (i - row * groups_per_row) * G;
        ax = row * a.ldx + col, ar = row * a.ldr + col, ao = row * a.ldo + col;
        first[u] = a.offset + (uint64_t)row * (uint64_t)a.cols + (uint64_t)col;
      }
      n[u] = i >= total ? 0 : (int)(a.cols - col < G ? a.cols - col : G);
      po[u] = static_cast<char*>(a.out) + ao * B;
      const char* px = static_cast<const char*>(a.x) + ax * B;
      const char* pr = RES ? static_cast<const char*>(a.residual) + ar * B : nullptr;
#pragma unroll
      for (int w = 0; w < W; ++w) xw[u][w] = rw[u][w] = 0;
      if (VEC && n[u] == G) {
        const uint4 v = ld_v4_stream(px);
        xw[u][0] = v.x, xw[u][1] = v.y, xw[u][2] = v.z, xw[u][3] = v.w;
        if (RES) {
          const uint4 r = ld_v4_stream(pr);
          rw[u][0] = r.x, rw[u][1] = r.y, rw[u][2] = r.z, rw[u][3] = r.w;
        }
      } else {
#pragma unroll
        for (int k = 0; k < G; ++k)
          if (k < n[u]) {
            xw[u][k * B / 4] |= ld_elem<B>(px + k * B) << (8 * (k * B % 4));
            if (RES) rw[u][k * B / 4] |= ld_elem<B>(pr + k * B) << (8 * (k * B % 4));
          }
      }
    }

    if (!a.drop_all) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int b = 0; b < G / 4 + (PHASE == kAny ? 1 : 0); ++b) {
          uint32_t w[4];
          philox<PHASE != kAny>(w, (first[u] >> 2) + b, a.sequence, key);
#pragma unroll
          for (int k = 0; k < 4; ++k) d[u][4 * b + k] = w[k];
        }
      if (PHASE == kShifted) {
        uint32_t next[4];  // the first block after this warp's runs (lane 0's is used)
        philox<true>(next, (first[U - 1] >> 2) + 32 * (G / 4), a.sequence, key);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t after = u + 1 < U ? d[u + 1 < U ? u + 1 : u][k] : next[k];
            d[u][G + k] = __shfl_sync(0xFFFFFFFFu, lane == 0 ? after : d[u][k], (lane + 1) & 31);
          }
      }
      if (PHASE != kWhole) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int phase = (int)(first[u] & 3);
#pragma unroll
          for (int k = 0; k < G; ++k) {
            const uint32_t far = phase & 2 ? d[u][k + 2] : d[u][k], near = phase & 2 ? d[u][k + 3] : d[u][k + 1];
            d[u][k] = phase & 1 ? near : far;
          }
        }
      }
    }

#pragma unroll
    for (int u = 0; u < U; ++u) {
      float y[G];
#pragma unroll
      for (int k = 0; k < G; ++k) {
        // A dropped element counts as 0 whatever it held, a NaN too.
        const float r = RES ? element<E>(rw[u], k) : 0.0f, x = element<E>(xw[u], k);
        y[k] = r;
        if (!a.drop_all && d[u][k] >= a.threshold) y[k] = RES ? __fmaf_rn(x, a.scale, r) : x * a.scale;
      }
      uint32_t o[W];
      pack_group<E>(o, y);
      if (VEC && n[u] == G) {
        st_v4_stream(po[u], make_uint4(o[0], o[1], o[2], o[3]));
      } else {
#pragma unroll
        for (int k = 0; k < G; ++k)
          if (k < n[u]) {
            if (B == 2)
              reinterpret_cast<uint16_t*>(po[u])[k] = (uint16_t)(o[k / 2] >> (16 * (k & 1)));
            else
              reinterpret_cast<uint32_t*>(po[u])[k] = o[k & 3];
          }
      }
    }
  }
}

template <class E>
cudaError_t dropout(DropoutArgs a, int num_sms, cudaStream_t s) {
  // Rows that follow one another without a gap are one row.
  if (a.ldx == a.cols && a.ldo == a.cols && (!a.residual || a.ldr == a.cols)) {
    a.cols *= a.rows;
    a.rows = 1;
    a.ldx = a.ldo = a.ldr = a.cols;
  }
  const int64_t gpr = (a.cols + E::kGroup - 1) / E::kGroup;
  uintptr_t ptrs = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.out) |
                   reinterpret_cast<uintptr_t>(a.residual);
  bool vec = (ptrs & 15u) == 0;
  if (a.rows > 1)
    vec = vec && a.ldx % E::kGroup == 0 && a.ldo % E::kGroup == 0 &&
          (!a.residual || a.ldr % E::kGroup == 0);
  const bool in_order = a.rows == 1 || a.cols % E::kGroup == 0;
  const uint64_t first = a.offset >> 2, last = (a.offset + (uint64_t)a.rows * (uint64_t)a.cols - 1) >> 2;
  const int phase = first >> 32 != last >> 32                              ? kAny
                    : a.offset % 4 == 0 && (in_order || a.cols % 4 == 0) ? kWhole
                    : in_order                                            ? kShifted
                                                                          : kAny;
  const int64_t per_cta = kDropThreads * kRuns, want = (a.rows * gpr + per_cta - 1) / per_cta;
  const unsigned grid = (unsigned)(want < (int64_t)num_sms * 32 ? want : (int64_t)num_sms * 32);
  const RoundKeys key = round_keys(a.seed, a.sequence, (uint32_t)(first >> 32));
  using Kernel = void (*)(DropoutArgs, RoundKeys, int64_t);
#define AR_DROPOUT_PHASES(RES, VEC) \
  { k_dropout<E, RES, VEC, kWhole>, k_dropout<E, RES, VEC, kShifted>, k_dropout<E, RES, VEC, kAny> }
  static const Kernel kernels[2][2][3] = {{AR_DROPOUT_PHASES(false, false), AR_DROPOUT_PHASES(false, true)},
                                          {AR_DROPOUT_PHASES(true, false), AR_DROPOUT_PHASES(true, true)}};
#undef AR_DROPOUT_PHASES
  return launch_op(kernels[a.residual ? 1 : 0][vec ? 1 : 0][phase], dim3(grid), kDropThreads, 0, 1, s, a, key, gpr);
}

}  // namespace

cudaError_t launch_dropout(int dtype, const DropoutArgs& a, int num_sms, cudaStream_t s) {
  switch (dtype) {
    case AR_BF16: return dropout<Bf16>(a, num_sms, s);
    case AR_FP16: return dropout<F16>(a, num_sms, s);
    default: return dropout<F32>(a, num_sms, s);
  }
}

}  // namespace ar
