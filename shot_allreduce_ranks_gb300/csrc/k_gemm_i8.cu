// The 8-bit product on the fifth-generation tensor cores:
// y[m, n] = sm[m] sn[n] sum_k x[m, k] w[n, k].
//
// This GPU's tensor cores have no fast path for 8-bit integers, but fp16 holds
// every int8 exactly, a product of two is exact in fp32, and so is their sum
// while it stays within 2^24 (K <= 1024 whatever the values, far longer for
// values that vary).  So the operands stay 8-bit in memory, in L2 and on the
// way into an SM, and converter warps turn each tile into fp16 (a byte
// permutation and a subtraction for every two values): x into tensor memory,
// which the matrix instruction can take its A operand from, w into shared memory in
// the swizzled layout that it reads B in.  Shared memory's bandwidth is what
// bounds this (copy in, read, write, and read by the instruction), and x takes
// only the first two of those four there.
//
// Roles, persistent over tiles of 128 CG x bn: one thread copies int8 tiles of
// 128 k into a staging ring by tensor maps, groups of warps convert them, one
// thread issues the matrix instructions, eight warps scale and store.  Four
// groups of converters take steps of 64 k in turn, so that their latencies
// overlap, and eight operand stages cover the way from a conversion through the
// pair's barriers and the instruction back to a free stage.  A pair of CTAs (CG = 2) shares one instruction over
// 256 rows, each converting its own 128 rows of x and half of the rows of w.
//
// Up to 128 tokens (SWAP, CG = 1) would leave rows of x empty: there w's rows
// are the instruction's A and the tokens its columns, one tile of 128 channels to
// a cluster whose KS CTAs split k, and the sums are sent to the CTAs' shared
// memory, quarter of the channels by quarter, and added in the order of the parts.
//
// Measured on one GB300 (replayed graph): 4096 x 8192 x 8192 282-286 us, 1,920-1,950
// TFLOP/s counted as products (a 16-bit library product of 8192^3 reached 1,924);
// 321 us in a loop under the power limit.  Steps on the way, none of which yet
// waited for a staged row's loads before giving it back, so that rows could be
// overwritten (waiting costs 3-5%): 395 us with x in shared memory, 387 with x in
// tensor memory, 365 with eight operand stages instead of four, 285 with the pair's
// arrivals ordered for shared memory alone (358 now with the cluster's full fence,
// by two warps that only pass arrivals on), 273 with eight instead of four warps
// storing.  440 x 2048 -> 5120: 14.2-15.8 us, of which about 7 are launch, set-up
// and the last tile.  64 tokens 3584 -> 8192: 13.9-15.8 us (16.9 by padded tiles
// of tokens).
#include "tc_device.cuh"

namespace ar {
namespace {

using namespace tc;

constexpr int kRowsMax = 256;                        // rows of x and w in a CTA's stage
constexpr uint32_t kStaged = kRowsMax * 128;         // bytes of a staging stage, 128 k
constexpr uint32_t kOperand = (kRowsMax - 128) * 128;  // of an operand stage of w, 64 k
constexpr int kSS = 3, kOS = 8;                      // stages of the two rings
constexpr int kGroups = 4, kGroupWarps = 4;          // converters: a warp for each quarter of tensor memory's lanes
constexpr int kGroupThreads = 32 * kGroupWarps;
constexpr int kStoreWarps = 8;                       // two for each quarter, taking turns by 32 columns
constexpr int kFirstConverter = 2 + kStoreWarps;     // warp
constexpr int kI8Threads = 32 * kFirstConverter + kGroups * kGroupThreads;
constexpr int kPieces = (kRowsMax - 128) / (8 * kGroupWarps);  // 16-byte pieces of w that a converter takes of a step
constexpr uint32_t kI8Smem = kSS * kStaged + kOS * kOperand + 1024;
// Tensor memory: accumulators from column 0, two of up to 128 columns or one of
// 256, and eight stages of x, 32 columns each.
constexpr uint32_t kI8TmemCols = 512, kAccStride = 128, kXCols = 256;

__device__ uint32_t g_i8_error;  // set by a wait that gave up

struct I8Args {
  GemmArgs g;
  TileWalk walk;
  int units;      // of 128 k
  int bn;         // columns of a tile, a multiple of 32
  int out_align;
};

// The end of a tile of 128 channels and up to 128 tokens, by all of the CTA's
// threads: sums go to [part][quarter here][token][channel] in the CTA that
// finishes that quarter of the channels, in the rings' memory, which is idle by
// then, and from there, scaled, to y.
template <class E, int KS>
__device__ __forceinline__ void join_parts(const I8Args& a, uint32_t room, uint32_t tmem, uint32_t done, uint32_t tile,
                                           uint32_t part, volatile uint32_t* dead) {
  constexpr int kHere = 4 / KS;  // quarters that a CTA finishes
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quarter = warp & 3, M = (int)a.g.M;
  if (!bar_wait(done, 0, dead) && lane == 0) atomicExch(&g_i8_error, 1u);
  fence_after_sync();
  __syncthreads();
  if (KS > 1) cluster_sync();  // every CTA's rings are idle
  const uint32_t own = room + (uint32_t)((int)part * kHere + quarter % kHere) * (128 * 128);
  const uint32_t to = KS > 1 ? map_to_cta(own, (uint32_t)(quarter / kHere)) : own;
  // Columns of 32 by turns: warps 4 i + quarter.
  for (int c = (warp >> 2) * 32; c < M; c += (kI8Threads / 128) * 32) {
    if (warp >= kI8Threads / 128 * 4) break;  // the last, incomplete set of four warps
    uint32_t r[32];
    __syncwarp();
    tmem_load32(r, tmem + ((uint32_t)quarter << 21) + c);
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (c + i < M) {
        const uint32_t at = to + (uint32_t)((c + i) * 32 + lane) * 4;
        const float v = __uint_as_float(r[i]);
        if (KS > 1)
          asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
        else
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
      }
  }
  fence_before_sync();
  if (KS > 1)
    cluster_sync();
  else
    __syncthreads();
  for (int e = warp; e < kHere * M; e += kI8Threads / 32) {
    const int q = e / M, m = e % M;
    const int64_t n = (int64_t)tile * 128 + ((int)part * kHere + q) * 32 + lane;
    float sum = 0.0f;
#pragma unroll
    for (int p = 0; p < KS; ++p) {
      float v;
      asm volatile("ld.shared.f32 %0, [%1];"
                   : "=f"(v) : "r"(room + (uint32_t)(p * kHere + q) * (128 * 128) + (uint32_t)(m * 32 + lane) * 4));
      sum = p ? sum + v : v;
    }
    if (n < a.g.N)
      static_cast<uint16_t*>(a.g.c0)[(int64_t)m * a.g.ldc + n] = (uint16_t)E::from_f32(sum * a.g.sm[m] * a.g.sn[n]);
  }
}

// map_x and map_w: the matrices whose rows are the instruction's rows and its
// columns (SWAP: w and x).
template <class E, int CG, bool SWAP, int KS>
__global__ void __launch_bounds__(kI8Threads, 1)
    k_gemm_i8(const __grid_constant__ I8Args a, const __grid_constant__ CUtensorMap map_x,
              const __grid_constant__ CUtensorMap map_w) {
  static_assert(SWAP == (CG == 1) && (SWAP || KS == 1), "");
  extern __shared__ uint8_t raw[];
  __shared__ __align__(8) uint64_t bars[2 * kSS + 2 * kOS + 5];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile uint32_t dead;

  const uint32_t operands = (smem_u32(raw) + 1023u) & ~1023u, staging = operands + kOS * kOperand;
  const uint32_t landed = smem_u32(bars), taken = landed + 8 * kSS;      // staging: copied in, converted
  const uint32_t ready = taken + 8 * kSS, used = ready + 8 * kOS;        // operands: converted, multiplied
  const uint32_t done = used + 8 * kOS, freed = done + 16, drained = freed + 16;
  const int warp = threadIdx.x >> 5;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0;
  const int rows = 128 + a.bn / CG;  // of a stage: x, then w
  const uint32_t accs = a.bn <= (int)kAccStride ? 2 : 1;  // accumulators
  const uint32_t part = KS > 1 ? cluster_rank() : 0;       // of k
  const int u0 = (int)((int64_t)a.units * part / KS), u1 = (int)((int64_t)a.units * (part + 1) / KS);
  const int steps = 2 * (u1 - u0);  // of 64 k, of a tile

  if (threadIdx.x == 0) {
    for (int i = 0; i < kSS; ++i) {
      bar_init(landed + 8 * i, 1);
      bar_init(taken + 8 * i, 2 * kGroupWarps);
    }
    for (int i = 0; i < kOS; ++i) {
      bar_init(ready + 8 * i, kGroupWarps * CG);
      bar_init(used + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(done + 8 * i, 1);
      bar_init(freed + 8 * i, kStoreWarps * CG);
    }
    bar_init(drained, 1);
    dead = 0;
    bar_init_done();
    prefetch_map(&map_x);
    prefetch_map(&map_w);
  }
  __syncwarp();
  if (warp == 1) {
    tmem_alloc<CG>(smem_u32(&tmem_slot), kI8TmemCols);
    tmem_no_more_allocs<CG>();
    fence_before_sync();
  }
  __syncthreads();
  if (CG == 2) cluster_sync();
  fence_after_sync();
  const uint32_t tmem = tmem_slot;
  pdl_enter();  // nothing before this has touched global memory
  // SWAP: a cluster makes one tile.
  const uint32_t first = blockIdx.x / (CG * KS), stride = SWAP ? 1u << 30 : gridDim.x / CG;
  const int64_t total = (int64_t)(first < a.walk.tiles ? (a.walk.tiles - 1 - first) / stride + 1 : 0) * steps;

  if (warp == 0) {
    if (elect_one()) {
      uint32_t it = 0;
      bool ok = true;
      for (uint32_t t = first; t < a.walk.tiles && ok; t += stride) {
        const Tile tile = tile_at(a.walk, t);
        const int m0 = (tile.m * CG + (int)rank) * 128, n0 = tile.n * a.bn + (int)rank * (a.bn / CG);
        for (int s = u0; s < u1; ++s, ++it) {
          const uint32_t st = it % kSS;
          if (!(ok = bar_wait(taken + 8 * st, ((it / kSS) & 1) ^ 1, &dead))) break;
          const uint32_t dst = staging + st * kStaged, bar = landed + 8 * st;
          bar_expect_tx(bar, (uint32_t)rows * 128);
          load_box<1>(dst, &map_x, s * 128, m0, bar);
          load_box<1>(dst + 128 * 128, &map_w, s * 128, n0, bar);
        }
      }
      if (!ok) atomicExch(&g_i8_error, 1u);
      for (uint32_t k = it > kSS ? it - kSS : 0; k < it; ++k) bar_wait_copies(landed + 8 * (k % kSS), (k / kSS) & 1);
    }
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      const uint32_t idesc = instr_desc(false, false, false, 128 * CG, a.bn);
      uint32_t it = 0, at = 0;
      bool ok = true;
      for (uint32_t t = first; t < a.walk.tiles && ok; t += stride, ++at) {
        const uint32_t buf = at % accs;
        if (!(ok = bar_wait(freed + 8 * buf, (at / accs & 1) ^ 1, &dead))) break;
        fence_after_sync();
        for (int s = 0; s < steps; ++s, ++it) {
          const uint32_t st = it % kOS;
          if (!(ok = bar_wait<CG == 2>(ready + 8 * st, (it / kOS) & 1, &dead))) break;
          fence_after_sync();
          const uint32_t x = tmem + kXCols + st * 32;
          const uint64_t w = operand_desc(operands + st * kOperand, 16, 1024);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_f16_ts<CG>(tmem + buf * kAccStride, x + 8 * k, w + 2 * k, idesc, s > 0 || k > 0);
          mma_commit<CG>(used + 8 * st);
        }
        if (ok) mma_commit<CG>(done + 8 * buf);
      }
      if (!ok) {
        atomicExch(&g_i8_error, 1u);
        mma_commit<CG>(drained);  // what was issued ends before tensor memory is freed
        bar_wait_copies(drained, 0);
      }
    }
  } else if (warp < kFirstConverter && !SWAP) {
    const uint32_t lane0 = (uint32_t)(warp & 3) * 32;
    uint32_t at = 0;
    for (uint32_t t = first; t < a.walk.tiles; t += stride, ++at) {
      const Tile tile = tile_at(a.walk, t);
      const uint32_t buf = at % accs;
      const int64_t m0 = ((int64_t)tile.m * CG + rank) * 128 + lane0, m = m0 + (threadIdx.x & 31);
      const int n0 = tile.n * a.bn;
      // The scales are on their way while the tile is multiplied: a lane holds
      // its row's, and one column's for every 32 columns that the warp stores.
      const float sm = m < a.g.M ? a.g.sm[m] : 0.0f;
      const int c0 = warp < 6 ? 0 : 32;
      float sn[kRowsMax / 64];
#pragma unroll
      for (int j = 0; j < kRowsMax / 64; ++j) {
        const int n = n0 + c0 + 64 * j + (int)(threadIdx.x & 31);
        sn[j] = c0 + 64 * j < a.bn && n < a.g.N ? a.g.sn[n] : 0.0f;
      }
      if (!bar_wait(done + 8 * buf, at / accs & 1, &dead)) {
        atomicExch(&g_i8_error, 1u);
        break;
      }
      fence_after_sync();
#pragma unroll
      for (int j = 0; j < kRowsMax / 64; ++j) {
        const int c = c0 + 64 * j;
        if (c >= a.bn || n0 + c >= a.g.N) break;
        uint32_t r[32];
        __syncwarp();
        tmem_load32(r, tmem + (lane0 << 16) + buf * kAccStride + c);
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]) * sm * __shfl_sync(0xFFFFFFFFu, sn[j], i);
        store_chunk<E>(a.g.c0, a.g.ldc, m0, n0 + c, a.g.M, a.g.N, v, a.out_align);
      }
      fence_before_sync();
      __syncwarp();
      if (elect_one()) bar_arrive_cluster(map_to_cta(freed + 8 * buf, 0));
    }
  } else if (warp >= kFirstConverter) {
    // Staged rows are 128 bytes whose 16-byte piece p lies at p ^ (row % 8), and
    // so are w's operand rows.  A step converts half of a staged row, pieces 4h ..
    // 4h + 3.  A thread takes a whole such row of x (eight lanes read eight
    // different banks) into its lane of tensor memory.  Of w, eight lanes take four
    // pieces of rows r and r + 4 (eight banks again) into all eight of an
    // operand row, and the lanes of the second row store their two results in
    // the other order, which again makes eight.
    const int group = (warp - kFirstConverter) / kGroupWarps;
    const int thread = (int)(threadIdx.x - kFirstConverter * 32) % kGroupThreads;
    const int lane = thread & 31, j = lane & 3, second = (lane >> 2) & 1;
    const int row0 = (thread >> 5) * 8 + (lane >> 3) + 4 * second;  // of w, + 8 kGroupWarps each time
    const int x_row = (warp & 3) * 32 + lane;
    bool ok = true;
    int64_t it = group;
    for (; it < total && ok; it += kGroups) {
      const uint32_t unit = (uint32_t)(it >> 1), ss = unit % kSS, half = (uint32_t)it & 1;
      const uint32_t os = (uint32_t)(it % kOS), round = (uint32_t)(it / kOS);
      if (!(ok = bar_wait(landed + 8 * ss, (unit / kSS) & 1, &dead))) break;
      const uint32_t from = staging + ss * kStaged, to = operands + os * kOperand;
      uint4 q[kPieces], xq[4];
      const auto load = [&](uint4& v, int row, int piece) {
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "r"(from + (uint32_t)row * 128 + 16u * ((half * 4 + piece) ^ (row & 7))));
      };
#pragma unroll
      for (int p = 0; p < 4; ++p) load(xq[p], x_row, p);
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        if (row0 + i * 8 * kGroupWarps < rows - 128) load(q[i], 128 + row0 + i * 8 * kGroupWarps, j);
      // Once the staged rows are in registers the next copy may come: it need not wait
      // for the operand stage.  A load that was issued has read nothing yet, and an
      // arrival can overtake it, so the arrival's address is made of what all lanes
      // have loaded (blockIdx.y is 0, which the compiler does not know).
      uint32_t seen = 0;
#pragma unroll
      for (int p = 0; p < 4; ++p) seen ^= xq[p].x ^ xq[p].y ^ xq[p].z ^ xq[p].w;
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        if (row0 + i * 8 * kGroupWarps < rows - 128) seen ^= q[i].x ^ q[i].y ^ q[i].z ^ q[i].w;
      seen = __reduce_or_sync(0xFFFFFFFFu, seen & blockIdx.y);
      if (elect_one()) bar_arrive(taken + 8 * ss + seen);
      if (!(ok = bar_wait(used + 8 * os, (round & 1) ^ 1, &dead))) break;
      fence_after_sync();
      {
        uint32_t h[32];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          i8_to_f16(xq[p].x, h[8 * p], h[8 * p + 1]);
          i8_to_f16(xq[p].y, h[8 * p + 2], h[8 * p + 3]);
          i8_to_f16(xq[p].z, h[8 * p + 4], h[8 * p + 5]);
          i8_to_f16(xq[p].w, h[8 * p + 6], h[8 * p + 7]);
        }
        __syncwarp();
        tmem_store32(tmem + ((uint32_t)(warp & 3) << 21) + kXCols + os * 32, h);
      }
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int row = row0 + i * 8 * kGroupWarps;
        if (row < rows - 128) {
          const uint32_t line = to + (uint32_t)row * 128;
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            const int c = o ^ second;
            uint32_t h[4];
            i8_to_f16(c ? q[i].z : q[i].x, h[0], h[1]);
            i8_to_f16(c ? q[i].w : q[i].y, h[2], h[3]);
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(line + 16u * ((2 * j + c) ^ (row & 7))),
                         "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]) : "memory");
          }
        }
      }
      fence_before_sync();
      fence_async_smem();  // the matrix unit reads through the asynchronous proxy
      __syncwarp();
      if (elect_one()) {
        if (CG == 2) {
          fence_cluster_smem();  // the pair's first CTA issues, and reads both CTAs' shared memory
          bar_arrive_cluster(map_to_cta(ready + 8 * os, 0));
        } else {
          bar_arrive(ready + 8 * os);
        }
      }
    }
    if (!ok) atomicExch(&g_i8_error, 1u);
    // What the group made last is multiplied before the CTA ends, and so is all
    // that it made before.
    if (ok && it >= kGroups && it - kGroups < total) {
      const uint32_t last = (uint32_t)(it - kGroups);
      bar_wait(used + 8 * (last % kOS), last / kOS & 1, &dead);
    }
  }
  __syncwarp();
  if (SWAP) {
    join_parts<E, KS>(a, operands, tmem, done, first, part, &dead);
  } else {
    fence_before_sync();
    __syncthreads();
    cluster_sync();
  }
  fence_after_sync();
  if (warp == 1) tmem_free<CG>(tmem, kI8TmemCols);
}

template <class E, int CG, bool SWAP, int KS>
cudaError_t launch(const I8Args& a, const CUtensorMap& mx, const CUtensorMap& mw, unsigned ctas, cudaStream_t s) {
  auto* kernel = k_gemm_i8<E, CG, SWAP, KS>;
  static bool raised[64];  // by device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && !raised[dev & 63])
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kI8Smem);
  if (e != cudaSuccess) return e;
  raised[dev & 63] = dev < 64;
  return launch_op(kernel, dim3(ctas), kI8Threads, kI8Smem, CG * KS, s, a, mx, mw);
}

// Pairs.  Columns of a tile: the number of rounds of tiles over the pairs times a
// round's time, which is a step's traffic in shared memory at 128 bytes a clock
// (a row of x 128 bytes, one of w 384) or its matrix instruction (2 clocks a column).
template <class E>
cudaError_t launch_pairs(const GemmArgs& g, int num_sms, cudaStream_t s) {
  const int64_t tiles_m = (g.M + 255) / 256, pairs = num_sms / 2;
  I8Args a = {};
  a.g = g;
  a.units = (int)((g.K + 127) / 128);
  double least = 1e300;
  for (int bn = 256; bn >= 32; bn -= 32) {
    const int64_t rounds = (tiles_m * ((g.N + bn - 1) / bn) + pairs - 1) / pairs;
    const double smem = 128.0 + 1.5 * bn, step = smem > 2 * bn ? smem : 2 * bn, stores = 15.0 * bn;
    // One accumulator: each tile's stores are waited for; two: the last tile's.
    const bool one = bn > (int)kAccStride;
    const double cost = (double)rounds * (2 * a.units * step + (one ? stores : 0)) + (one ? 0 : stores);
    if (cost < least) least = cost, a.bn = bn;
  }
  if (!make_walk(&a.walk, tiles_m, (g.N + a.bn - 1) / a.bn, 1, 8)) return cudaErrorInvalidConfiguration;
  const uintptr_t out = reinterpret_cast<uintptr_t>(g.c0) | (uintptr_t)g.ldc * 2;
  a.out_align = out % 32 == 0 ? 32 : out % 16 == 0 ? 16 : out % 4 == 0 ? 4 : 2;
  CUtensorMap mx, mw;
  if (!tc_make_map(&mx, kMapU8, g.a0, g.M, g.K, g.lda, 128, 128) ||
      !tc_make_map(&mw, kMapU8, g.b0, g.N, g.K, g.ldb, a.bn / 2, 128))
    return cudaErrorInvalidValue;
  const unsigned slots = a.walk.tiles < (uint32_t)pairs ? a.walk.tiles : (unsigned)pairs;
  return launch<E, 2, false, 1>(a, mx, mw, slots * 2, s);
}

// Up to 128 tokens: as many parts of k as fill the SMs, none of them empty.
template <class E>
cudaError_t launch_swapped(const GemmArgs& g, int num_sms, cudaStream_t s) {
  const int64_t tiles = (g.N + 127) / 128;
  I8Args a = {};
  a.g = g;
  a.units = (int)((g.K + 127) / 128);
  a.bn = (int)((g.M + 31) / 32 * 32);
  CUtensorMap mw, mx;
  if (!make_walk(&a.walk, tiles, 1, 1, 1)) return cudaErrorInvalidConfiguration;
  if (!tc_make_map(&mw, kMapU8, g.b0, g.N, g.K, g.ldb, 128, 128) ||
      !tc_make_map(&mx, kMapU8, g.a0, g.M, g.K, g.lda, a.bn, 128))
    return cudaErrorInvalidValue;
  if (tiles * 4 <= num_sms && a.units >= 4) return launch<E, 1, true, 4>(a, mw, mx, (unsigned)tiles * 4, s);
  if (tiles * 2 <= num_sms && a.units >= 2) return launch<E, 1, true, 2>(a, mw, mx, (unsigned)tiles * 2, s);
  return launch<E, 1, true, 1>(a, mw, mx, (unsigned)tiles, s);
}

template <class E>
cudaError_t launch_type(const GemmArgs& g, int num_sms, cudaStream_t s) {
  return g.M > 128 ? launch_pairs<E>(g, num_sms, s) : launch_swapped<E>(g, num_sms, s);
}

}  // namespace

// A tensor map wants rows that start on 16 bytes, and strides below 2^40.
bool gemm_i8_takes(int mode, const GemmArgs& g) {
  const int64_t most = (int64_t)1 << 30;
  return mode == kGemmI8 && tc_available() && g.M <= most && g.N <= most && g.K <= most && g.lda % 16 == 0 &&
         g.ldb % 16 == 0 && g.lda < most << 9 && g.ldb < most << 9 && ((reinterpret_cast<uintptr_t>(g.a0) | reinterpret_cast<uintptr_t>(g.b0)) & 15u) == 0;
}

cudaError_t launch_gemm_i8(int dtype, const GemmArgs& g, int num_sms, cudaStream_t s) {
  return dtype == AR_BF16 ? launch_type<Bf16>(g, num_sms, s) : launch_type<F16>(g, num_sms, s);
}

cudaError_t gemm_i8_error(cudaStream_t s, uint32_t* error) {
  void* p = nullptr;
  const cudaError_t e = cudaGetSymbolAddress(&p, g_i8_error);
  return e == cudaSuccess ? take_error_word(p, s, error) : e;
}

}  // namespace ar
