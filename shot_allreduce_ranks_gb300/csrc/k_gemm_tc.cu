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
// transposed in memory.
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

struct TcArgs {
  GemmArgs g;
  TileWalk walk;
  int steps;                    // k steps of one segment
  int bn;                       // columns of the matrix instruction, a multiple of 32
  int out_align;                // bytes that every output row start is a multiple of
};

// A stage holds 128 rows of A and up to 256 / CG of B.  1 KiB aligns the ring.
template <int CG>
struct Shape {
  static constexpr uint32_t kA = 128 * kBK * 2, kB = 256 / CG * kBK * 2, kStage = kA + kB;
  static constexpr int kStages = 196608 / kStage;
  static constexpr uint32_t kStores = 8 * 2 * 2048;  // two 32 x 32 boxes an epilogue warp
  static constexpr uint32_t kSmem = kStages * kStage + kStores + 1024;
};

struct OutMaps {
  CUtensorMap c[3];
};

template <int MODE, class E, int ACT, int CG>
__global__ void __launch_bounds__(kTcThreads, 1)
    k_gemm_tc(const __grid_constant__ TcArgs a, const __grid_constant__ CUtensorMap map_a0,
              const __grid_constant__ CUtensorMap map_a1, const __grid_constant__ CUtensorMap map_b0,
              const __grid_constant__ CUtensorMap map_b1, const __grid_constant__ OutMaps out) {
  using S = Shape<CG>;
  constexpr bool kAmn = MODE == kGemmDw, kBmn = MODE != kGemmGated;
  const int cols = MODE == kGemmGated ? a.bn / 2 : a.bn;  // output columns of a tile
  constexpr int kST = S::kStages;
  extern __shared__ uint8_t raw[];
  __shared__ __align__(8) uint64_t bars[2 * kST + 5];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile uint32_t dead;

  const uint32_t ring = (smem_u32(raw) + 1023u) & ~1023u;
  const uint32_t full = smem_u32(bars), empty = full + 8 * kST, done = empty + 8 * kST, freed = done + 16,
                 drained = freed + 16;
  const int warp = threadIdx.x >> 5;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kST; ++i) {
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
    prefetch_map(&map_a0);
    prefetch_map(&map_b0);
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

  const int total = MODE == kGemmDx ? 2 * a.steps : a.steps;
  const int64_t first = blockIdx.x / CG, stride = gridDim.x / CG;

  if (warp == 0) {
    if (elect_one()) {
      const int chunks = (a.bn / CG + 63) / 64;  // of an MN-major B
      const uint32_t stage_bytes = S::kA + (MODE == kGemmGated ? a.bn / CG * 128 : chunks * 8192);
      uint32_t it = 0;
      bool ok = true;
      for (int64_t t = first; t < a.walk.tiles && ok; t += stride) {
        const Tile tile = tile_at(a.walk, t);
        const int m0 = (tile.m * CG + (int)rank) * 128, n0 = tile.n * cols;
        for (int s = 0; s < total; ++s, ++it) {
          const uint32_t st = it % kST, round = it / kST;
          if (!(ok = bar_wait(empty + 8 * st, (round & 1) ^ 1, &dead))) break;
          const uint32_t sa = ring + st * S::kStage, sb = sa + S::kA;
          uint32_t bar = full + 8 * st;
          if (rank == 0) bar_expect_tx(bar, CG * stage_bytes);
          if (CG == 2) bar = map_to_cta(bar, 0);
          const bool up = MODE == kGemmDx ? s >= a.steps : MODE == kGemmDw && tile.z != 0;
          const int k0 = (MODE == kGemmDx && up ? s - a.steps : s) * kBK;
          const CUtensorMap* ma = up ? &map_a1 : &map_a0;
          if (kAmn) {
            load_box<CG>(sa, ma, m0, k0, bar);
            load_box<CG>(sa + 8192, ma, m0 + 64, k0, bar);
          } else {
            load_box<CG>(sa, ma, k0, m0, bar);
          }
          if (MODE == kGemmGated) {
            // The pair's first CTA holds the gate's rows, its second the up projection's.
            if (CG == 2) {
              load_box<CG>(sb, rank ? &map_b1 : &map_b0, k0, n0, bar);
            } else {
              load_box<CG>(sb, &map_b0, k0, n0, bar);
              load_box<CG>(sb + (uint32_t)a.bn * 64, &map_b1, k0, n0, bar);
            }
          } else {
            const CUtensorMap* mb = MODE == kGemmDx && up ? &map_b1 : &map_b0;
            for (int c = 0; c < chunks; ++c)
              load_box<CG>(sb + 8192 * c, mb, n0 + (int)rank * (a.bn / CG) + 64 * c, k0, bar);
          }
        }
      }
      // Nothing of the ring is left behind: the last stages are consumed, or, after
      // a wait that gave up, at least their copies are done.
      const uint32_t oldest = it > kST ? it - kST : 0;
      for (uint32_t k = oldest; k < it && ok; ++k) ok = bar_wait(empty + 8 * (k % kST), (k / kST) & 1, &dead);
      if (!ok) {
        atomicExch(&g_tc_error, 1u);
        if (rank == 0)
          for (uint32_t k = oldest; k < it; ++k) bar_wait_copies(full + 8 * (k % kST), (k / kST) & 1);
      }
    }
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      const uint32_t idesc = instr_desc(IsBf16<E>::value, kAmn, kBmn, 128 * CG, a.bn);
      uint32_t it = 0, at = 0;
      bool ok = true;
      for (int64_t t = first; t < a.walk.tiles && ok; t += stride, ++at) {
        const uint32_t buf = at & 1;
        if (!(ok = bar_wait(freed + 8 * buf, ((at >> 1) & 1) ^ 1, &dead))) break;
        fence_after_sync();
        const uint32_t acc = tmem + buf * 256;
        for (int s = 0; s < total; ++s, ++it) {
          const uint32_t st = it % kST, round = it / kST;
          if (!(ok = bar_wait(full + 8 * st, round & 1, &dead))) break;
          fence_after_sync();
          const uint32_t sa = ring + st * S::kStage, sb = sa + S::kA;
          const uint64_t da = kAmn ? operand_desc(sa, 8192, 1024) : operand_desc(sa, 16, 1024);
          const uint64_t db = kBmn ? operand_desc(sb, 8192, 1024) : operand_desc(sb, 16, 1024);
#pragma unroll
          for (int k = 0; k < 4; ++k)  // 16 k: 32 bytes of a K-major row, 16 rows of an MN-major tile
            mma_f16<CG>(acc, da + (kAmn ? 128 : 2) * k, db + (kBmn ? 128 : 2) * k, idesc, s > 0 || k > 0);
          mma_commit<CG>(empty + 8 * st);
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
    const uint32_t boxes = ring + kST * S::kStage + (uint32_t)(warp - 2) * 4096;
    uint32_t stored = 0, at = 0;
    for (int64_t t = first; t < a.walk.tiles; t += stride, ++at) {
      const Tile tile = tile_at(a.walk, t);
      const uint32_t buf = at & 1;
      if (!bar_wait(done + 8 * buf, (at >> 1) & 1, &dead)) {
        atomicExch(&g_tc_error, 1u);
        break;
      }
      fence_after_sync();
      const int64_t m0 = ((int64_t)tile.m * CG + rank) * 128 + lane0;
      const int n0 = tile.n * cols;
      const uint32_t acc = tmem + (lane0 << 16) + buf * 256;
#pragma unroll 1
      for (int c = warp < 6 ? 0 : 32; c < cols; c += 64) {
        if (n0 + c >= a.g.N) break;
        uint32_t r[32], u[32];
        __syncwarp();
        tmem_load32(r, acc + c);
        if (MODE == kGemmGated) tmem_load32(u, acc + cols + c);
        tmem_wait_load32(r);
        if (MODE == kGemmGated) tmem_wait_load32(u);
        // Rows that start on 16 bytes leave through shared memory as boxes of 64-byte
        // rows; a lane storing its own row would touch 32 lines at a time.
        const auto store = [&](int which, void* c_out, const float(&v)[32]) {
          if (a.out_align < 16) {
            store_chunk<E>(c_out, a.g.ldc, m0, n0 + c, a.g.M, min(a.g.N, (int64_t)(n0 + cols)), v, a.out_align);
            return;
          }
          const uint32_t box = boxes + (stored & 1) * 2048, row = box + (uint32_t)lane * 64;
          if (lane == 0) store_box_wait_read<1>();  // the box's last copy but one has been read
          __syncwarp();
#pragma unroll
          for (int p = 0; p < 4; ++p)
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(row + 16u * (uint32_t)(p ^ ((lane >> 1) & 3))),
                         "r"(E::pack(v[8 * p], v[8 * p + 1])), "r"(E::pack(v[8 * p + 2], v[8 * p + 3])),
                         "r"(E::pack(v[8 * p + 4], v[8 * p + 5])), "r"(E::pack(v[8 * p + 6], v[8 * p + 7])) : "memory");
          fence_async_smem();
          __syncwarp();
          if (lane == 0 && m0 < a.g.M) store_box(&out.c[which], n0 + c, (int)m0, box);
          ++stored;
        };
        float v[32];
        if (MODE == kGemmGated) {
          if (a.g.c1) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
            store(1, a.g.c1, v);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(u[i]);
            store(2, a.g.c2, v);
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = act_value<ACT>(__uint_as_float(r[i])) * __uint_as_float(u[i]);
          store(0, a.g.c0, v);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
          store(MODE == kGemmDw ? tile.z : 0, MODE == kGemmDw && tile.z ? a.g.c1 : a.g.c0, v);
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

bool make_map(CUtensorMap* map, int dtype, const void* p, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
  return tc_make_map(map, dtype == AR_BF16 ? kMapBf16 : kMapF16, p, rows, cols, ld, box_rows, 64);
}

template <int MODE, class E, int ACT, int CG>
cudaError_t launch(int dtype, const GemmArgs& g, int bn, int num_sms, cudaStream_t s) {
  using S = Shape<CG>;
  const int cols = MODE == kGemmGated ? bn / 2 : bn;
  CUtensorMap ma0, ma1, mb0, mb1;
  bool ok;
  if (MODE == kGemmDw) {
    ok = make_map(&ma0, dtype, g.a0, g.K, g.M, g.lda, 64) && make_map(&ma1, dtype, g.a1, g.K, g.M, g.lda, 64);
  } else {
    ok = make_map(&ma0, dtype, g.a0, g.M, g.K, g.lda, 128);
    ma1 = ma0;
    if (MODE == kGemmDx) ok = ok && make_map(&ma1, dtype, g.a1, g.M, g.K, g.lda, 128);
  }
  if (MODE == kGemmGated) {
    ok = ok && make_map(&mb0, dtype, g.b0, g.N, g.K, g.ldb, bn / 2) && make_map(&mb1, dtype, g.b1, g.N, g.K, g.ldb1, bn / 2);
  } else {
    ok = ok && make_map(&mb0, dtype, g.b0, g.K, g.N, g.ldb, 64);
    mb1 = mb0;
    if (MODE == kGemmDx) ok = ok && make_map(&mb1, dtype, g.b1, g.K, g.N, g.ldb1, 64);
  }
  if (!ok) return cudaErrorInvalidValue;

  TcArgs a = {};
  a.g = g;
  a.walk.tiles_m = (int)((g.M + 128 * CG - 1) / (128 * CG));
  a.walk.tiles_n = (int)((g.N + cols - 1) / cols);
  a.walk.tiles = (int64_t)a.walk.tiles_m * a.walk.tiles_n * (MODE == kGemmDw ? 2 : 1);
  a.walk.group = 16 / CG;
  a.bn = bn;
  a.steps = (int)((g.K + kBK - 1) / kBK);
  const uintptr_t out = reinterpret_cast<uintptr_t>(g.c0) | reinterpret_cast<uintptr_t>(g.c1) |
                        reinterpret_cast<uintptr_t>(g.c2) | (uintptr_t)g.ldc * 2;
  a.out_align = out % 32 == 0 ? 32 : out % 16 == 0 ? 16 : out % 4 == 0 ? 4 : 2;

  OutMaps out_maps;
  if (a.out_align >= 16) {
    void* const c[3] = {g.c0, g.c1 ? g.c1 : g.c0, g.c2 ? g.c2 : g.c0};
    for (int i = 0; i < 3; ++i)
      if (!tc_make_map(&out_maps.c[i], dtype == AR_BF16 ? kMapBf16 : kMapF16, c[i], g.M, g.N, g.ldc, 32, 32))
        return cudaErrorInvalidValue;
  }
  auto* kernel = k_gemm_tc<MODE, E, ACT, CG>;
  static bool raised[64];  // by device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && !raised[dev & 63])
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kSmem);
  if (e != cudaSuccess) return e;
  raised[dev & 63] = dev < 64;
  const int64_t pairs = num_sms / CG;
  const dim3 grid((unsigned)((a.walk.tiles < pairs ? a.walk.tiles : pairs) * CG));
  return launch_op(kernel, grid, kTcThreads, S::kSmem, CG, s, a, ma0, ma1, mb0, mb1, out_maps);
}

// Columns of the matrix instruction.  A step of 64 k takes the longer of its
// instruction (bn clocks x 2) and its copies (an SM takes in 64 bytes a clock);
// a tile ends with its stores, about ten clocks a column, which the next tile
// hides; the tiles go round the SMs in whole rounds.
int columns(int mode, const GemmArgs& g, int cg, int num_sms) {
  const int64_t slots = num_sms / cg, steps = (g.K + kBK - 1) / kBK * (mode == kGemmDx ? 2 : 1);
  int best = 256;
  double least = 1e300;
  for (int bn = 256; bn >= 64; bn -= mode == kGemmGated ? 64 : 32) {
    const int64_t cols = mode == kGemmGated ? bn / 2 : bn, planes = mode == kGemmDw ? 2 : 1;
    const int64_t tiles = (g.M + 128 * cg - 1) / (128 * cg) * ((g.N + cols - 1) / cols) * planes;
    const int64_t b_rows = mode == kGemmGated ? bn / cg : (bn / cg + 63) / 64 * 64;
    const double step = fmax(2.0 * bn, 2.0 * (128 + b_rows)), stores = 10.0 * bn;
    const double rounds = (double)((tiles + slots - 1) / slots);
    const double cost = rounds * fmax(steps * step, stores) + fmin(steps * step, stores);
    if (cost < 0.98 * least) least = cost, best = bn;
  }
  return best;
}

template <int MODE, class E, int ACT>
cudaError_t launch_shape(int dtype, const GemmArgs& g, int num_sms, cudaStream_t s) {
  if (g.M > 128) return launch<MODE, E, ACT, 2>(dtype, g, columns(MODE, g, 2, num_sms), num_sms, s);
  return launch<MODE, E, ACT, 1>(dtype, g, columns(MODE, g, 1, num_sms), num_sms, s);
}

template <class E>
cudaError_t launch_type(int mode, int dtype, const GemmArgs& g, int num_sms, cudaStream_t s) {
  switch (mode) {
    case kGemmGated:
      return g.act == AR_ACT_SILU ? launch_shape<kGemmGated, E, AR_ACT_SILU>(dtype, g, num_sms, s)
                                  : launch_shape<kGemmGated, E, AR_ACT_GELU_TANH>(dtype, g, num_sms, s);
    case kGemmDx: return launch_shape<kGemmDx, E, 0>(dtype, g, num_sms, s);
    default: return launch_shape<kGemmDw, E, 0>(dtype, g, num_sms, s);
  }
}

bool rows_on_16(const void* p, int64_t ld) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0;
}

}  // namespace

// A tensor map wants rows that start on 16 bytes and extents within 32 bits;
// coordinates are 32-bit.
bool gemm_tc_takes(int mode, const GemmArgs& g) {
  const int64_t most = (int64_t)1 << 30;
  return mode != kGemmI8 && tc_available() && g.M <= most && g.N <= most && g.K <= most && rows_on_16(g.a0, g.lda) &&
         rows_on_16(g.a1, g.lda) && rows_on_16(g.b0, g.ldb) && rows_on_16(g.b1, g.ldb1);
}

cudaError_t launch_gemm_tc(int mode, int dtype, const GemmArgs& g, int num_sms, cudaStream_t s) {
  return dtype == AR_BF16 ? launch_type<Bf16>(mode, dtype, g, num_sms, s) : launch_type<F16>(mode, dtype, g, num_sms, s);
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
