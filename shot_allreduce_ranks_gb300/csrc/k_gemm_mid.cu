// The gated product for a serving batch of some tens of tokens: too many for
// mma.sync to stream the weights past, too few to fill 128 rows of tokens.
//
// Here the weights stand for the matrix instruction's 128 rows and the tokens
// for its columns, so that nothing is padded but the last 16 tokens.  A
// tile's rows are 64 of the gate's weights and the same 64 of the up projection's, in
// alternating blocks of 16, so that 32 lanes of tensor memory hold both
// pre-activations of 16 outputs.  That makes width / 64 tiles, too few for the
// SMs, so a cluster of KS CTAs splits a tile's k: each takes every KS-th part,
// and at the end sends its sums to the CTAs' shared memory, quarter of the rows
// by quarter, where they are added in the order of the parts.
//
// Bound by the weights' way into the SMs (about 64 bytes a clock each), and below
// that by launch, set-up and two trips through the cluster, about 7 us.  Measured
// on one GB300 (bf16, replayed graph): 13 tokens 5120 -> 2048 10.2 us (42 MB of
// weights, 4.1 TB/s), 64 tokens 11.4 us (25 us by tiles of 128 padded tokens), 64
// tokens 8192 -> 3584 22.8 us (117 MB, 5.1 TB/s; was 40), 128 tokens 25.4 us.
#include "tc_device.cuh"

namespace ar {
namespace {

using namespace tc;

constexpr int kMidBK = 64, kMidMost = 128;  // k of a stage; tokens
constexpr int kMidThreads = 256;
// The ring: 128 rows of weights and the tokens' a stage, as many as fit (11 for
// 16 tokens, six for 128): what is on its way hides the copies' latency.
constexpr uint32_t kMidA = 128 * 128, kMidRing = 208896;
constexpr int kMidStages = 11;
constexpr uint32_t kMidSmem = kMidRing + 1024;
constexpr int kMidBlock = 16;               // rows of a block of either projection

__device__ uint32_t g_mid_error;  // set by a wait that gave up

struct MidArgs {
  GemmArgs g;
  int steps;   // k steps in all
  int tokens;  // columns of the instruction: M rounded up to 16
};

__device__ __forceinline__ void store_remote(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ float load_shared(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}

template <class E, int ACT, int KS>
__global__ void __launch_bounds__(kMidThreads, 1)
    k_gemm_mid(const __grid_constant__ MidArgs a, const __grid_constant__ CUtensorMap map_x,
               const __grid_constant__ CUtensorMap map_g, const __grid_constant__ CUtensorMap map_u) {
  extern __shared__ uint8_t raw[];
  __shared__ __align__(8) uint64_t bars[2 * kMidStages + 1];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile uint32_t dead;

  const uint32_t ring = (smem_u32(raw) + 1023u) & ~1023u;
  const uint32_t full = smem_u32(bars), empty = full + 8 * kMidStages, done = empty + 8 * kMidStages;
  const uint32_t stage_bytes = kMidA + (uint32_t)a.tokens * 128;
  const uint32_t stages = min((uint32_t)kMidStages, kMidRing / stage_bytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t part = KS > 1 ? cluster_rank() : 0;
  const int f0 = (int)(blockIdx.x / KS) * 64;  // outputs of this tile
  const int s0 = (int)((int64_t)a.steps * part / KS), s1 = (int)((int64_t)a.steps * (part + 1) / KS);

  if (threadIdx.x == 0) {
    for (int i = 0; i < kMidStages; ++i) {
      bar_init(full + 8 * i, 1);
      bar_init(empty + 8 * i, 1);
    }
    bar_init(done, 1);
    dead = 0;
    bar_init_done();
    prefetch_map(&map_x);
    prefetch_map(&map_g);
    prefetch_map(&map_u);
  }
  __syncwarp();
  if (warp == 1) {
    tmem_alloc<1>(smem_u32(&tmem_slot), kMidMost);
    tmem_no_more_allocs<1>();
    fence_before_sync();
  }
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = tmem_slot;
  pdl_enter();  // nothing before this has touched global memory

  if (warp == 0) {
    if (elect_one()) {
      bool ok = true;
      Stage stage;
      uint32_t filled = 0;  // stages in use, up to all
      for (int s = s0; s < s1; ++s, stage.next(stages)) {
        if (!(ok = bar_wait(empty + 8 * stage.at, stage.parity ^ 1, &dead))) break;
        filled += filled < stages;
        const uint32_t sa = ring + stage.at * stage_bytes, bar = full + 8 * stage.at;
        bar_expect_tx(bar, stage_bytes);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          load_box<1>(sa + (2 * b) * kMidBlock * 128, &map_g, s * kMidBK, f0 + b * kMidBlock, bar);
          load_box<1>(sa + (2 * b + 1) * kMidBlock * 128, &map_u, s * kMidBK, f0 + b * kMidBlock, bar);
        }
        load_box<1>(sa + kMidA, &map_x, s * kMidBK, 0, bar);
      }
      // The ring is used again below: every copy has landed by then, consumed or not.
      for (uint32_t i = 0; i < filled; ++i)
        bar_wait_copies(full + 8 * i, i < stage.at ? stage.parity : stage.parity ^ 1);
      if (!ok) atomicExch(&g_mid_error, 1u);
    }
  } else if (warp == 1) {
    if (elect_one()) {
      const uint32_t idesc = instr_desc(IsBf16<E>::value, false, false, 128, a.tokens);
      bool ok = true;
      Stage stage;
      for (int s = s0; s < s1; ++s, stage.next(stages)) {
        if (!(ok = bar_wait(full + 8 * stage.at, stage.parity, &dead))) break;
        fence_after_sync();
        const uint64_t dw = operand_desc(ring + stage.at * stage_bytes, 16, 1024);
        const uint64_t dx = operand_desc(ring + stage.at * stage_bytes + kMidA, 16, 1024);
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_f16<1>(tmem, dw + 2 * k, dx + 2 * k, idesc, s > s0 || k > 0);
        mma_commit<1>(empty + 8 * stage.at);
      }
      mma_commit<1>(done);  // of whatever was issued
      if (!ok) atomicExch(&g_mid_error, 1u);
    }
  }
  __syncwarp();
  if (!bar_wait(done, 0, &dead) && lane == 0) atomicExch(&g_mid_error, 1u);
  fence_after_sync();
  __syncthreads();
  if (KS > 1) cluster_sync();  // every CTA's ring is idle

  // Sums go to [part][quarter here][token][row] in the CTA that finishes that
  // quarter of the rows.
  constexpr int kHere = 4 / KS;  // quarters a CTA finishes
  const int quarter = warp & 3;
  const uint32_t own = ring + (uint32_t)((int)part * kHere + quarter % kHere) * (kMidMost * 128);
  const uint32_t to = KS > 1 ? map_to_cta(own, (uint32_t)(quarter / kHere)) : own;
  for (int c = warp < 4 ? 0 : 32; c < a.tokens; c += 64) {
    uint32_t r[32];
    __syncwarp();
    tmem_load32(r, tmem + ((uint32_t)quarter << 21) + c);
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (c + i < a.g.M) {
        const uint32_t at = to + (uint32_t)((c + i) * 32 + lane) * 4;
        const float v = __uint_as_float(r[i]);
        if (KS > 1)
          store_remote(at, v);
        else
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
      }
  }
  fence_before_sync();
  if (KS > 1)
    cluster_sync();
  else
    __syncthreads();
  fence_after_sync();
  if (warp == 1) tmem_free<1>(tmem, kMidMost);

  const int f = (int)threadIdx.x % kMidBlock;
  for (int e = (int)threadIdx.x / kMidBlock; e < kHere * (int)a.g.M; e += kMidThreads / kMidBlock) {
    const int q = e / (int)a.g.M, m = e % (int)a.g.M;
    const int64_t n = f0 + ((int)part * kHere + q) * kMidBlock + f;
    float gate = 0.0f, up = 0.0f;
#pragma unroll
    for (int p = 0; p < KS; ++p) {
      const uint32_t from = ring + (uint32_t)(p * kHere + q) * (kMidMost * 128) + (uint32_t)(m * 32 + f) * 4;
      const float gp = load_shared(from), up_p = load_shared(from + kMidBlock * 4);
      gate = p ? gate + gp : gp;
      up = p ? up + up_p : up_p;
    }
    if (n >= a.g.N) continue;
    const int64_t at = (int64_t)m * a.g.ldc + n;
    static_cast<uint16_t*>(a.g.c0)[at] = (uint16_t)E::from_f32(act_value<ACT>(gate) * up);
    if (a.g.c1) {
      static_cast<uint16_t*>(a.g.c1)[at] = (uint16_t)E::from_f32(gate);
      static_cast<uint16_t*>(a.g.c2)[at] = (uint16_t)E::from_f32(up);
    }
  }
}

template <class E, int ACT, int KS>
cudaError_t launch(int dtype, const GemmArgs& g, cudaStream_t s) {
  const MapType type = dtype == AR_BF16 ? kMapBf16 : kMapF16;
  MidArgs a = {};
  a.g = g;
  a.steps = (int)((g.K + kMidBK - 1) / kMidBK);
  a.tokens = (int)((g.M + 15) / 16 * 16);
  CUtensorMap mx, mg, mu;
  if (!tc_make_map(&mx, type, g.a0, g.M, g.K, g.lda, a.tokens, kMidBK) ||
      !tc_make_map(&mg, type, g.b0, g.N, g.K, g.ldb, kMidBlock, kMidBK) ||
      !tc_make_map(&mu, type, g.b1, g.N, g.K, g.ldb1, kMidBlock, kMidBK))
    return cudaErrorInvalidValue;
  auto* kernel = k_gemm_mid<E, ACT, KS>;
  static bool raised[64];  // by device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && !raised[dev & 63])
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMidSmem);
  if (e != cudaSuccess) return e;
  raised[dev & 63] = dev < 64;
  const int64_t tiles = (g.N + 63) / 64;
  return launch_op(kernel, dim3((unsigned)(tiles * KS)), kMidThreads, kMidSmem, KS, s, a, mx, mg, mu);
}

// As many parts of k as fill the SMs, none of them empty.
template <class E, int ACT>
cudaError_t launch_split(int dtype, const GemmArgs& g, int num_sms, cudaStream_t s) {
  const int64_t tiles = (g.N + 63) / 64, steps = (g.K + kMidBK - 1) / kMidBK;
  if (tiles * 4 <= num_sms && steps >= 8) return launch<E, ACT, 4>(dtype, g, s);
  if (tiles * 2 <= num_sms && steps >= 4) return launch<E, ACT, 2>(dtype, g, s);
  return launch<E, ACT, 1>(dtype, g, s);
}

template <class E>
cudaError_t launch_type(int dtype, const GemmArgs& g, int num_sms, cudaStream_t s) {
  return g.act == AR_ACT_SILU ? launch_split<E, AR_ACT_SILU>(dtype, g, num_sms, s)
                              : launch_split<E, AR_ACT_GELU_TANH>(dtype, g, num_sms, s);
}

}  // namespace

bool gemm_mid_takes(int mode, const GemmArgs& g) { return mode == kGemmGated && g.M <= kMidMost && gemm_tc_takes(mode, g); }

cudaError_t launch_gemm_mid(int dtype, const GemmArgs& g, int num_sms, cudaStream_t s) {
  return dtype == AR_BF16 ? launch_type<Bf16>(dtype, g, num_sms, s) : launch_type<F16>(dtype, g, num_sms, s);
}

cudaError_t gemm_mid_error(cudaStream_t s, uint32_t* error) {
  void* p = nullptr;
  const cudaError_t e = cudaGetSymbolAddress(&p, g_mid_error);
  return e == cudaSuccess ? take_error_word(p, s, error) : e;
}

}  // namespace ar
