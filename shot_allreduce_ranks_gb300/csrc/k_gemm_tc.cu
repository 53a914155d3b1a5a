// The feed-forward operators' matrix products on the fifth-generation tensor
// cores, for operands whose rows start on 16 bytes.
//
// C[m, n] = sum_k A(m, k) B(n, k) with fp32 accumulators in tensor memory.  A
// persistent CTA (or a pair of them, CG = 2, that share one instruction over
// 256 rows) makes tiles of 128 CG x BN.  One thread copies operand tiles of 64
// k into a ring of shared-memory stages by tensor maps with 128-byte swizzle
// (out-of-range elements arrive as zeros, so ragged sizes need no other code),
// one thread issues the matrix instructions, and eight warps (two for each
// quarter of the rows, taking turns by 32 columns) read a finished accumulator
// while the next tile is multiplied into the other half of tensor memory.
//
// In the gated product the BN rows of B are BN/2 rows of the gate's weights and
// the same BN/2 of the up projection's, so both pre-activations of an element
// lie in one lane, BN/2 columns apart, and act(gate) * up leaves the kernel
// without a trip through memory.  Of the backward products, dx contracts over
// both projections in one accumulation, with B read along its other axis
// (MN-major), and the two weight gradients read both operands so: nothing is
// transposed in memory.  All three are one launch: one kind's last round of tiles
// would leave SMs idle, which the other's tiles fill.
//
// What bounds it.  A 256x256 tile's step of 64 k keeps a pair's tensor pipes busy
// for 512 clocks, and each SM's shared memory for as long: 32 KB copied in and 32
// KB read by the instruction, at 128 bytes a clock.  (A CTA by itself, 128x256,
// copies in 48 KB a step and measured 613 us where the pairs take 501.)  Stores
// come on top, 64 KB written and read again a tile, which shows where the
// contraction is short.  Measured on one GB300 (bf16, replayed graph):
//   forward with saved pre-activations, 8192 tokens x 8192 -> 3584: 490-510 us,
//   1,900-1,960 TFLOP/s, tensor pipe active 94% of the time (a library product
//   of 8192^3 reached 1,924); in a loop the power limit takes the clock from
//   2,070 to about 1,470 MHz and the time to 560 us;
//   forward 440 x 5120 -> 1736: 18.3 us (21.0 with six stages for narrow tiles too,
//   instead of eight), on 56 of 76 pairs: 80 steps of 128 columns at about 350
//   clocks, nearer to the copies' 384 than to the instruction's 256, and 4 us of
//   launch, set-up and last stores (1280, 2560, 10240 instead of 5120: 7.8, 11.3,
//   31.1 us);
//   gradients 4096 x 8192 -> 3584: 545 us (1,770 TFLOP/s); 512 x 8192 -> 3584: 89-90
//   us (tensor pipe active 60%: the weights' tiles have eight steps each).
// Measured and left out: clusters of four that share A by multicast (the same
// time: an SM's own intake binds, and only 36 of 38 such clusters fit).
#include <math.h>

#include "tc_device.cuh"

namespace ar {
namespace tc {

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

bool tc_available() { return encode_fn() != nullptr; }

bool tc_make_map(CUtensorMap* map, MapType type, const void* p, int64_t rows, int64_t cols, int64_t ld, int box_rows,
                 int box_cols) {
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * (type == kMapU8 ? 1 : 2)};
  const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows}, step[2] = {1, 1};
  const CUtensorMapDataType t = type == kMapBf16  ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                : type == kMapF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                  : CU_TENSOR_MAP_DATA_TYPE_UINT8;
  return encode_fn()(map, t, 2, const_cast<void*>(p), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     box_cols * (type == kMapU8 ? 1 : 2) == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace tc

namespace {

using namespace tc;

constexpr int kBK = 64;                // k of one stage: 128 bytes
constexpr int kTcThreads = 320;        // copy, matrix, eight epilogue warps
constexpr uint32_t kTmemCols = 512;

__device__ uint32_t g_tc_error;  // set by a wait that gave up

enum { kTcGated = 0, kTcGrad = 1 };

// One product's tiles and outputs.
struct Part {
  TileWalk walk;
  int64_t M, N, ldc;
  int steps;      // k steps of one segment
  int out_align;  // bytes that every output row start is a multiple of
  int fold;       // rows come in blocks of 16 first and 16 second parts: added, M counts the sums
};

struct TcArgs {
  Part part[2];      // kTcGrad: dx, then the two weight gradients; kTcGated: part[1] alone
  void* c[3];        // h, gate, up; or dx, dWgate, dWup
  int bn;            // columns of the matrix instruction, a multiple of 32
  // See job_at: dx's whole rounds and the tiles left over, the slots that those
  // leave free, and the tiles of the weights' gradients that a free slot takes first.
  uint32_t rounds, left, free, ahead;
};

// kTcGated: a[0] = x, b = the two weights.  kTcGrad: a[0], a[1] = dgate, dup along
// their columns and b[0], b[1] = the weights, for dx; a[2], a[3] = dgate, dup
// along their rows and b[2] = x, for the weights' gradients.
struct TcMaps {
  CUtensorMap a[4], b[3], c[3];
};

// The j-th tile of slot p (a CTA or a pair) of P: its part and number.  dx's tiles
// come first, round by round; where its last round leaves slots free, those
// take `ahead` tiles of the weight gradients each (about as many as fit beside one
// of dx), and the rest goes round all slots.  With fewer tiles than the machine has
// slots `ahead` is 0: the slots with a tile of dx then take the first tiles of the
// weights' gradients too, and as many of the last slots get none.  Every tile has
// one slot, fixed by its number.
template <int WHAT>
__device__ __forceinline__ bool job_at(const TcArgs& a, uint32_t p, uint32_t P, uint32_t j, int& part, uint32_t& t) {
  t = p + j * P;
  part = 1;
  if (WHAT == kTcGrad) {
    const uint32_t mine = a.rounds + (p < a.left ? 1 : 0);
    if (j < mine) {
      part = 0;
    } else {
      const uint32_t k = j - mine;
      if (p < a.left || a.left == 0)
        t = a.ahead * a.free + k * P + p;
      else
        t = k < a.ahead ? k * a.free + (p - a.left) : a.ahead * a.free + (k - a.ahead) * P + p;
    }
  }
  return t < a.part[part].walk.tiles;
}

// The ring has as many stages as fit: 128 rows of A and what a tile's columns
// need of B each.  More stages matter where tiles are narrow: copies take about
// 1,800 clocks to arrive, 3,000 under load, and a step of 128 columns 256.
constexpr uint32_t kRing = 196608;
constexpr int kMostStages = 10;
constexpr uint32_t kABytes = 128 * kBK * 2;
constexpr uint32_t kStores = 8 * 2 * 2048;  // two 32 x 32 boxes an epilogue warp
constexpr uint32_t kTcSmem = kRing + kStores + 1024;  // 1 KiB aligns the ring

template <int WHAT, class E, int ACT, int CG>
__global__ void __launch_bounds__(kTcThreads, 1)
    k_gemm_tc(const __grid_constant__ TcArgs a, const __grid_constant__ TcMaps maps) {
  static_assert(WHAT == kTcGrad || CG == 2, "the gated product is made by pairs");
  constexpr bool kBmn = WHAT == kTcGrad;
  const int cols = WHAT == kTcGated ? a.bn / 2 : a.bn;  // output columns of a tile
  extern __shared__ uint8_t raw[];
  __shared__ __align__(8) uint64_t bars[2 * kMostStages + 5];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile uint32_t dead;

  const uint32_t ring = (smem_u32(raw) + 1023u) & ~1023u;
  const uint32_t full = smem_u32(bars), empty = full + 8 * kMostStages, done = empty + 8 * kMostStages,
                 freed = done + 16, drained = freed + 16;
  const int chunks = (a.bn / CG + 63) / 64;  // of an MN-major B
  const uint32_t stage_bytes = kABytes + (WHAT == kTcGated ? a.bn / CG * 128 : chunks * 8192);
  const uint32_t stages = min((uint32_t)kMostStages, kRing / stage_bytes);
  const int warp = threadIdx.x >> 5;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kMostStages; ++i) {
      bar_init(full + 8 * i, 1);
      bar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(done + 8 * i, 1);
      bar_init(freed + 8 * i, 8 * CG);
    }
    bar_init(drained, 1);
    dead = 0;
    bar_init_done();
    prefetch_map(&maps.a[0]);
    prefetch_map(&maps.b[0]);
  }
  __syncwarp();
  if (warp == 1) {
    tmem_alloc<CG>(smem_u32(&tmem_slot), kTmemCols);
    tmem_no_more_allocs<CG>();
    fence_before_sync();
  }
  __syncthreads();
  if (CG == 2) cluster_sync();
  fence_after_sync();
  const uint32_t tmem = tmem_slot;
  pdl_enter();  // nothing before this has touched global memory

  const uint32_t slot = blockIdx.x / CG, slots = gridDim.x / CG;
  int which;       // part and number of the tile at hand
  uint32_t number;

  if (warp == 0) {
    if (elect_one()) {
      Stage stage;
      uint32_t filled = 0;  // stages in use, up to all
      bool ok = true;
      for (uint32_t j = 0; ok && job_at<WHAT>(a, slot, slots, j, which, number); ++j) {
        const Tile tile = tile_at(a.part[which].walk, number);
        const int m0 = (tile.m * CG + (int)rank) * 128, n0 = tile.n * cols;
        const bool dx = WHAT == kTcGrad && which == 0, dw = WHAT == kTcGrad && which == 1;
        const int steps = a.part[which].steps, total = dx ? 2 * steps : steps;
        for (int s = 0; s < total; ++s, stage.next(stages)) {
          if (!(ok = bar_wait(empty + 8 * stage.at, stage.parity ^ 1, &dead))) break;
          const uint32_t sa = ring + stage.at * stage_bytes, sb = sa + kABytes;
          uint32_t bar = full + 8 * stage.at;
          filled += filled < stages;
          if (rank == 0) bar_expect_tx(bar, CG * stage_bytes);
          if (CG == 2) bar = map_to_cta(bar, 0);
          const int up = dx ? s >= steps : tile.z;  // which projection
          const int k0 = (dx && up ? s - steps : s) * kBK;
          if (dw) {
            load_box<CG>(sa, &maps.a[2 + up], m0, k0, bar);
            load_box<CG>(sa + 8192, &maps.a[2 + up], m0 + 64, k0, bar);
          } else {
            load_box<CG>(sa, &maps.a[up], k0, m0, bar);
          }
          if (WHAT == kTcGated) {
            // The pair's first CTA holds the gate's rows, its second the up projection's.
            load_box<CG>(sb, &maps.b[rank], k0, n0, bar);
          } else {
            const CUtensorMap* mb = &maps.b[dw ? 2 : up];
            for (int c = 0; c < chunks; ++c)
              load_box<CG>(sb + 8192 * c, mb, n0 + (int)rank * (a.bn / CG) + 64 * c, k0, bar);
          }
        }
      }
      // Nothing of the ring is left behind: every stage in use is consumed, or, after
      // a wait that gave up, at least its copies are done.  The stages before the
      // next one have been filled last; from there on, a round earlier.
      const auto parity_of = [&](uint32_t i) { return i < stage.at ? stage.parity : stage.parity ^ 1; };
      for (uint32_t i = 0; i < filled && ok; ++i) ok = bar_wait(empty + 8 * i, parity_of(i), &dead);
      if (!ok) {
        atomicExch(&g_tc_error, 1u);
        if (rank == 0)
          for (uint32_t i = 0; i < filled; ++i) bar_wait_copies(full + 8 * i, parity_of(i));
      }
    }
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      Stage stage;
      uint32_t at = 0;
      bool ok = true;
      for (; ok && job_at<WHAT>(a, slot, slots, at, which, number); ++at) {
        const bool a_mn = WHAT == kTcGrad && which == 1;
        const uint32_t idesc = instr_desc(IsBf16<E>::value, a_mn, kBmn, 128 * CG, a.bn);
        const int total = a.part[which].steps * (WHAT == kTcGrad && which == 0 ? 2 : 1);
        const uint32_t buf = at & 1;
        if (!(ok = bar_wait(freed + 8 * buf, ((at >> 1) & 1) ^ 1, &dead))) break;
        fence_after_sync();
        const uint32_t acc = tmem + buf * 256;
        for (int s = 0; s < total; ++s, stage.next(stages)) {
          if (!(ok = bar_wait(full + 8 * stage.at, stage.parity, &dead))) break;
          fence_after_sync();
          const uint32_t sa = ring + stage.at * stage_bytes, sb = sa + kABytes;
          const uint64_t da = operand_desc(sa, a_mn ? 8192 : 16, 1024);
          const uint64_t db = kBmn ? operand_desc(sb, 8192, 1024) : operand_desc(sb, 16, 1024);
#pragma unroll
          for (int k = 0; k < 4; ++k)  // 16 k: 32 bytes of a K-major row, 16 rows of an MN-major tile
            mma_f16<CG>(acc, da + (a_mn ? 128 : 2) * k, db + (kBmn ? 128 : 2) * k, idesc, s > 0 || k > 0);
          mma_commit<CG>(empty + 8 * stage.at);
        }
        if (ok) mma_commit<CG>(done + 8 * buf);
      }
      if (!ok) {
        atomicExch(&g_tc_error, 1u);
        mma_commit<CG>(drained);  // what was issued ends before tensor memory is freed
        bar_wait_copies(drained, 0);
      }
    }
  } else {
    const uint32_t lane0 = (uint32_t)(warp & 3) * 32;  // this warp's lanes of tensor memory
    const int lane = (int)(threadIdx.x & 31);
    const uint32_t boxes = ring + kRing + (uint32_t)(warp - 2) * 4096;
    uint32_t stored = 0, at = 0;
    for (; job_at<WHAT>(a, slot, slots, at, which, number); ++at) {
      const Part& part = a.part[which];
      const Tile tile = tile_at(part.walk, number);
      const uint32_t buf = at & 1;
      if (!bar_wait(done + 8 * buf, (at >> 1) & 1, &dead)) {
        atomicExch(&g_tc_error, 1u);
        break;
      }
      fence_after_sync();
      const int fold = WHAT == kTcGrad ? part.fold : 0;
      const int64_t m0 = (((int64_t)tile.m * CG + rank) * 128 + lane0) >> fold;
      const int n0 = tile.n * cols;
      const uint32_t acc = tmem + (lane0 << 16) + buf * 256;
      // A warp whose rows lie past the last has nothing to store.  It must not go
      // through the boxes either: their turns below count on a copy for every write.
#pragma unroll 1
      for (int c = warp < 6 ? 0 : 32; c < cols && m0 < part.M; c += 64) {
        if (n0 + c >= part.N) break;
        uint32_t r[32], u[32];
        __syncwarp();
        if (WHAT == kTcGated)
          tmem_load32(r, u, acc + c, acc + cols + c);
        else
          tmem_load32(r, acc + c);
        // Rows that start on 16 bytes leave through shared memory as boxes of 64-byte
        // rows; a lane storing its own row would touch 32 lines at a time.  Two boxes
        // take turns, and every write to one is followed by its copy, so the copy that
        // may still be reading when all but one have is the other box's.  The copy
        // engine writes pieces of 16 bytes, zeros past the last column: a box that
        // reaches past a row whose end lies inside a piece is stored by lanes.
        const auto store = [&](int to, const float(&v)[32]) {
          if (part.out_align < 16 || (part.N % 8 != 0 && n0 + c + 32 > part.N)) {
            store_chunk<E>(a.c[to], part.ldc, m0, n0 + c, fold ? min(part.M, m0 + 16) : part.M, min(part.N, (int64_t)(n0 + cols)), v, part.out_align);
            return;
          }
          const uint32_t box = boxes + (stored & 1) * 2048, row = box + (uint32_t)lane * 64;
          if (lane == 0) store_box_wait_read<1>();  // this box's last copy has been read
          __syncwarp();
#pragma unroll
          for (int p = 0; p < 4; ++p)
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(row + 16u * (uint32_t)(p ^ ((lane >> 1) & 3))),
                         "r"(E::pack(v[8 * p], v[8 * p + 1])), "r"(E::pack(v[8 * p + 2], v[8 * p + 3])),
                         "r"(E::pack(v[8 * p + 4], v[8 * p + 5])), "r"(E::pack(v[8 * p + 6], v[8 * p + 7])) : "memory");
          fence_async_smem();
          __syncwarp();
          if (lane == 0) store_box(&maps.c[to], n0 + c, (int)m0, box);
          ++stored;
        };
        float v[32];
        if (WHAT == kTcGated) {
          if (a.c[1]) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
            store(1, v);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(u[i]);
            store(2, v);
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = act_value<ACT>(__uint_as_float(r[i])) * __uint_as_float(u[i]);
          store(0, v);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
          if (fold) {
            // An infinite sum stays as the first parts make it: with an infinite weight
            // the second's is NaN where nothing was left, or of the other sign.
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float second = __shfl_down_sync(0xFFFFFFFFu, v[i], 16);
              v[i] = fabsf(v[i]) < INFINITY ? v[i] + second : v[i];
            }
          }
          store(which == 0 ? 0 : 1 + tile.z, v);
        }
      }
      fence_before_sync();
      __syncwarp();
      if (elect_one()) {
        if (CG == 2)
          bar_arrive_cluster(map_to_cta(freed + 8 * buf, 0));
        else
          bar_arrive(freed + 8 * buf);
      }
    }
    if (lane == 0) store_box_wait_all();
  }
  __syncwarp();
  fence_before_sync();
  __syncthreads();
  if (CG == 2) cluster_sync();
  fence_after_sync();
  if (warp == 1) tmem_free<CG>(tmem, kTmemCols);
}

bool make_map(CUtensorMap* map, int dtype, const void* p, int64_t rows, int64_t cols, int64_t ld, int box_rows,
              int box_cols = 64) {
  return tc_make_map(map, dtype == AR_BF16 ? kMapBf16 : kMapF16, p, rows, cols, ld, box_rows, box_cols);
}

bool rows_on_16(const void* p, int64_t ld) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0 && ld < (int64_t)1 << 38;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// One product's tiles; false if there are too many or an output map could not be made.
bool make_part(TcArgs& a, TcMaps& maps, int which, int dtype, const GemmArgs& g, int cols, int planes, int cg,
               void* const* c, int outs) {
  Part& p = a.part[which];
  p.fold = g.tokens > 0;
  p.M = p.fold ? g.tokens : g.M, p.N = g.N, p.ldc = g.ldc;
  if (!make_walk(&p.walk, ceil_div(g.M, 128 * cg), ceil_div(g.N, cols), planes, 16 / cg)) return false;
  p.steps = (int)ceil_div(g.K, kBK);
  uintptr_t bits = (uintptr_t)g.ldc * 2;
  for (int i = 0; i < outs; ++i) bits |= reinterpret_cast<uintptr_t>(c[i]);
  p.out_align = bits % 16 == 0 && rows_on_16(c[0], g.ldc) ? 16 : bits % 4 == 0 ? 4 : 2;
  for (int i = 0; i < outs && p.out_align == 16; ++i)
    if (c[i] && !make_map(&maps.c[c - a.c + i], dtype, c[i], p.M, g.N, g.ldc, p.fold ? 16 : 32, 32)) return false;
  return true;
}

template <int WHAT, class E, int ACT, int CG>
cudaError_t launch(const TcArgs& a, const TcMaps& maps, int num_sms, cudaStream_t s) {
  auto* kernel = k_gemm_tc<WHAT, E, ACT, CG>;
  static bool raised[64];  // by device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && !raised[dev & 63])
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kTcSmem);
  if (e != cudaSuccess) return e;
  raised[dev & 63] = dev < 64;
  const int64_t slots = num_sms / CG, tiles = (int64_t)a.part[0].walk.tiles + a.part[1].walk.tiles;
  const dim3 grid((unsigned)((tiles < slots ? tiles : slots) * CG));
  return launch_op(kernel, grid, kTcThreads, kTcSmem, CG, s, a, maps);
}

// What a tile takes, in clocks: a step of 64 k the longer of its instruction (2
// a column) and its copies (an SM takes in 64 bytes a clock); its stores about
// ten a column, or forty where rows do not start on 16 bytes, which the next
// tile hides.
struct TileCost {
  double steps, stores;
  double whole() const { return fmax(steps, stores); }
};
TileCost tile_cost(int64_t steps, int bn, int64_t b_rows, bool aligned) {
  return {(double)steps * fmax(2.0 * bn, 2.0 * (double)(128 + b_rows)), (aligned ? 10.0 : 40.0) * bn};
}

template <class E, int ACT>
cudaError_t launch_gated(int dtype, const GemmArgs& g, int num_sms, cudaStream_t s) {
  constexpr int CG = 2;
  const int64_t slots = num_sms / CG;
  int bn = 256;
  double least = 1e300;
  for (int b = 256; b >= 64; b -= 64) {
    const TileCost c = tile_cost(ceil_div(g.K, kBK), b, b / CG, rows_on_16(g.c0, g.ldc));
    const int64_t rounds = ceil_div(ceil_div(g.M, 128 * CG) * ceil_div(g.N, b / 2), slots);
    const double cost = (double)rounds * c.whole() + fmin(c.steps, c.stores);
    if (cost < 0.98 * least) least = cost, bn = b;
  }
  TcArgs a = {};
  TcMaps maps = {};
  a.c[0] = g.c0, a.c[1] = g.c1, a.c[2] = g.c2;
  a.bn = bn;
  if (!make_part(a, maps, 1, dtype, g, bn / 2, 1, CG, a.c, 3) ||
      !make_map(&maps.a[0], dtype, g.a0, g.M, g.K, g.lda, 128) ||
      !make_map(&maps.b[0], dtype, g.b0, g.N, g.K, g.ldb, bn / 2) ||
      !make_map(&maps.b[1], dtype, g.b1, g.N, g.K, g.ldb1, bn / 2))
    return cudaErrorInvalidValue;
  return launch<kTcGated, E, ACT, CG>(a, maps, num_sms, s);
}

// dx and the weights' gradients, either of which may be absent.
template <class E, int CG>
cudaError_t launch_grad(int dtype, const GemmArgs* dx, const GemmArgs* dw, int num_sms, cudaStream_t s) {
  const int64_t N = (dx ? dx : dw)->N, P = num_sms / CG;
  int bn = 256;
  int64_t ahead = 0;
  double least = 1e300;
  for (int b = 256; b >= 64; b -= 32) {
    const int64_t tiles_n = ceil_div(N, b), b_rows = ceil_div(b / CG, 64) * 64;
    const TileCost cx = tile_cost(dx ? 2 * ceil_div(dx->K, kBK) : 0, b, b_rows, !dx || rows_on_16(dx->c0, dx->ldc));
    const TileCost cw = tile_cost(dw ? ceil_div(dw->K, kBK) : 0, b, b_rows, !dw || rows_on_16(dw->c0, dw->ldc));
    const int64_t D = dx ? ceil_div(dx->M, 128 * CG) * tiles_n : 0, left = D % P;
    int64_t W = dw ? 2 * ceil_div(dw->M, 128 * CG) * tiles_n : 0, first = 0;
    double cost = (double)(D / P) * cx.whole();
    if (left) {
      first = W ? (int64_t)(cx.whole() / cw.whole()) : 0;
      if (first > ceil_div(W, P - left)) first = ceil_div(W, P - left);
      W -= first * (P - left);
      cost += fmax(cx.whole(), (double)first * cw.whole());
    }
    if (W > 0) cost += (double)ceil_div(W, P) * cw.whole();
    cost += dw ? fmin(cw.steps, cw.stores) : fmin(cx.steps, cx.stores);
    if (cost < 0.98 * least) least = cost, bn = b, ahead = first;
  }
  TcArgs a = {};
  TcMaps maps = {};
  a.bn = bn;
  bool ok = true;
  if (dx) {
    a.c[0] = dx->c0;
    ok = make_part(a, maps, 0, dtype, *dx, bn, 1, CG, a.c, 1) &&
         make_map(&maps.a[0], dtype, dx->a0, dx->M, dx->K, dx->lda, 128) &&
         make_map(&maps.a[1], dtype, dx->a1, dx->M, dx->K, dx->lda, 128) &&
         make_map(&maps.b[0], dtype, dx->b0, dx->K, dx->N, dx->ldb, 64) &&
         make_map(&maps.b[1], dtype, dx->b1, dx->K, dx->N, dx->ldb1, 64);
  }
  if (dw && ok) {
    a.c[1] = dw->c0, a.c[2] = dw->c1;
    ok = make_part(a, maps, 1, dtype, *dw, bn, 2, CG, a.c + 1, 2) &&
         make_map(&maps.a[2], dtype, dw->a0, dw->K, dw->M, dw->lda, 64) &&
         make_map(&maps.a[3], dtype, dw->a1, dw->K, dw->M, dw->lda, 64) &&
         make_map(&maps.b[2], dtype, dw->b0, dw->K, dw->N, dw->ldb, 64);
  }
  if (!ok) return cudaErrorInvalidValue;
  // The grid is smaller than P where there are fewer tiles.
  const int64_t D = a.part[0].walk.tiles, all = D + a.part[1].walk.tiles, slots = all < P ? all : P;
  a.rounds = (uint32_t)(D / slots), a.left = (uint32_t)(D % slots), a.free = (uint32_t)(slots - D % slots);
  a.ahead = a.left && all >= P ? (uint32_t)ahead : 0;
  return launch<kTcGrad, E, 0, CG>(a, maps, num_sms, s);
}

template <class E>
cudaError_t gated_type(int dtype, const GemmArgs& g, int num_sms, cudaStream_t s) {
  return g.act == AR_ACT_SILU ? launch_gated<E, AR_ACT_SILU>(dtype, g, num_sms, s)
                              : launch_gated<E, AR_ACT_GELU_TANH>(dtype, g, num_sms, s);
}

// Pairs, unless every matrix has no more rows than one CTA's tile.
template <class E>
cudaError_t grad_type(int dtype, const GemmArgs* dx, const GemmArgs* dw, int num_sms, cudaStream_t s) {
  if ((!dx || dx->M <= 128) && (!dw || dw->M <= 128)) return launch_grad<E, 1>(dtype, dx, dw, num_sms, s);
  return launch_grad<E, 2>(dtype, dx, dw, num_sms, s);
}

}  // namespace

// A tensor map wants rows that start on 16 bytes, strides below 2^40 bytes and
// extents within 32 bits; coordinates are 32-bit.
bool gemm_tc_takes(int mode, const GemmArgs& g) {
  const int64_t most = (int64_t)1 << 30;
  return mode != kGemmI8 && tc_available() && g.M <= most && g.N <= most && g.K <= most && rows_on_16(g.a0, g.lda) &&
         rows_on_16(g.a1, g.lda) && rows_on_16(g.b0, g.ldb) && rows_on_16(g.b1, g.ldb1);
}

cudaError_t launch_gated_tc(int dtype, const GemmArgs& g, int num_sms, cudaStream_t s) {
  return dtype == AR_BF16 ? gated_type<Bf16>(dtype, g, num_sms, s) : gated_type<F16>(dtype, g, num_sms, s);
}

cudaError_t launch_grad_tc(int dtype, const GemmArgs* dx, const GemmArgs* dw, int num_sms, cudaStream_t s) {
  return dtype == AR_BF16 ? grad_type<Bf16>(dtype, dx, dw, num_sms, s) : grad_type<F16>(dtype, dx, dw, num_sms, s);
}

cudaError_t take_error_word(void* p, cudaStream_t s, uint32_t* error) {
  const uint32_t zero = 0;
  cudaError_t e = cudaMemcpyAsync(error, p, sizeof *error, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && *error) e = cudaMemcpyAsync(p, &zero, sizeof zero, cudaMemcpyHostToDevice, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  return e;
}

cudaError_t gemm_tc_error(cudaStream_t s, uint32_t* error) {
  void* p = nullptr;
  const cudaError_t e = cudaGetSymbolAddress(&p, g_tc_error);
  return e == cudaSuccess ? take_error_word(p, s, error) : e;
}

}  // namespace ar
