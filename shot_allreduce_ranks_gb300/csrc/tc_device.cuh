// Device helpers of the tcgen05 kernels: mbarriers, tensor-map copies, tensor
// memory and the matrix instruction, as inline PTX.
#pragma once

#include <cuda.h>

#include "ops_internal.cuh"

namespace ar {
namespace tc {

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The address of the same shared variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_to_cta(uint32_t addr, uint32_t rank) {
  uint32_t d;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(addr), "r"(rank));
  return d;
}

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_init_done() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
__device__ __forceinline__ void bar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Arrival on a barrier of any CTA of the cluster that orders no memory between
// CTAs: enough where it announces that tensor memory has been read (the read was
// waited for), or behind fence_cluster_smem() for what was written to shared memory.
__device__ __forceinline__ void bar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Orders what this thread did in its CTA's shared memory, and what it has learned
// of others there, before its next arrivals for every CTA of the cluster.  (All of
// memory at that scope, as a release does, took 1,300 clocks.)
__device__ __forceinline__ void fence_cluster_smem() {
  asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
}

// CLUSTER: what the arrivals announce was written by other CTAs.
template <bool CLUSTER = false>
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  if (CLUSTER)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}
__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

// Every wait is bounded: after kWaitNs it gives up, and so do the CTA's other
// waits once one of them has raised *dead.
constexpr uint64_t kWaitNs = 2000ull * 1000ull * 1000ull;

template <bool CLUSTER>
static __device__ __noinline__ bool bar_wait_slow(uint32_t bar, uint32_t parity, volatile uint32_t* dead) {
  const uint64_t t0 = now_ns();
  for (uint32_t k = 0; k < (1u << 30); ++k) {
    if (bar_try<CLUSTER>(bar, parity)) return true;
    if ((k & 31u) == 31u && (*dead != 0 || now_ns() - t0 > kWaitNs)) break;
  }
  *dead = 1;
  return false;
}

template <bool CLUSTER = false>
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile uint32_t* dead) {
#pragma unroll 1
  for (int k = 0; k < 16; ++k)
    if (bar_try<CLUSTER>(bar, parity)) return true;
  return bar_wait_slow<CLUSTER>(bar, parity, dead);
}

// The same for what is still under way after a wait gave up.
static __device__ __noinline__ void bar_wait_copies(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = now_ns();
  for (uint32_t k = 0; k < (1u << 30) && !bar_try(bar, parity); ++k)
    if ((k & 31u) == 31u && now_ns() - t0 > kWaitNs) break;
}

// A stage of a ring and the parity of its use, step by step.
struct Stage {
  uint32_t at = 0, parity = 0;
  __device__ __forceinline__ void next(uint32_t stages) {
    if (++at == stages) at = 0, parity ^= 1;
  }
};

// A box of a 2-D tensor map into shared memory; CG = 2: the barrier may be the
// pair's other CTA's.
template <int CG>
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y,
                                         uint32_t bar) {
  if (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}

// The other way, for what the thread's earlier fence has made visible; done
// (shared memory free again, all written) by the thread's waits below.
__device__ __forceinline__ void store_box(const CUtensorMap* map, int32_t x, int32_t y, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];\n\t"
               "cp.async.bulk.commit_group;" ::"l"(map), "r"(src), "r"(x), "r"(y) : "memory");
}
template <int N>
__device__ __forceinline__ void store_box_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void store_box_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// ---- tensor memory -----------------------------------------------------------

template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t cols) {
  if (CG == 2)
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
  else
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
}
template <int CG>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  if (CG == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
  else
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}
template <int CG>
__device__ __forceinline__ void tmem_no_more_allocs() {
  if (CG == 2)
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  else
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}

// 32 columns of the warp's 32 lanes: lane l gets its row's values.  Load and wait
// are one statement: the registers are not to be touched before the wait, not even
// by a copy that the compiler puts between two statements.
__device__ __forceinline__ void tmem_load32(uint32_t (&r)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr) : "memory");
}
// Two such loads behind one wait.
__device__ __forceinline__ void tmem_load32(uint32_t (&r)[32], uint32_t (&u)[32], uint32_t addr_r, uint32_t addr_u) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%64];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%65];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3]), "=&r"(r[4]), "=&r"(r[5]), "=&r"(r[6]), "=&r"(r[7]),
        "=&r"(r[8]), "=&r"(r[9]), "=&r"(r[10]), "=&r"(r[11]), "=&r"(r[12]), "=&r"(r[13]), "=&r"(r[14]), "=&r"(r[15]),
        "=&r"(r[16]), "=&r"(r[17]), "=&r"(r[18]), "=&r"(r[19]), "=&r"(r[20]), "=&r"(r[21]), "=&r"(r[22]), "=&r"(r[23]),
        "=&r"(r[24]), "=&r"(r[25]), "=&r"(r[26]), "=&r"(r[27]), "=&r"(r[28]), "=&r"(r[29]), "=&r"(r[30]), "=&r"(r[31]),
        "=&r"(u[0]), "=&r"(u[1]), "=&r"(u[2]), "=&r"(u[3]), "=&r"(u[4]), "=&r"(u[5]), "=&r"(u[6]), "=&r"(u[7]),
        "=&r"(u[8]), "=&r"(u[9]), "=&r"(u[10]), "=&r"(u[11]), "=&r"(u[12]), "=&r"(u[13]), "=&r"(u[14]), "=&r"(u[15]),
        "=&r"(u[16]), "=&r"(u[17]), "=&r"(u[18]), "=&r"(u[19]), "=&r"(u[20]), "=&r"(u[21]), "=&r"(u[22]), "=&r"(u[23]),
        "=&r"(u[24]), "=&r"(u[25]), "=&r"(u[26]), "=&r"(u[27]), "=&r"(u[28]), "=&r"(u[29]), "=&r"(u[30]), "=&r"(u[31])
      : "r"(addr_r), "r"(addr_u) : "memory");
}
// Writes 32 columns of the warp's 32 lanes, and waits until that is done.
__device__ __forceinline__ void tmem_store32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
      "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(addr)
      : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void fence_before_sync() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after_sync() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// ---- the matrix instruction ----------------------------------------------------

// Shared-memory operand in the 128-byte swizzled layout: rows of 128 bytes, eight
// of them (1024 bytes) a swizzle atom.  An operand whose contracted axis is
// contiguous (K-major) has its 8-row groups `sbo` bytes apart; in one whose
// other axis is contiguous (MN-major) each row is 64 elements of that axis at
// one k, `sbo` separates groups of eight k and `lbo` the next 64 elements.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)(lbo >> 4) << 16 | (uint64_t)(sbo >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// kind::f16, fp32 accumulators; a_mn / b_mn: that operand is MN-major.
__host__ __device__ constexpr uint32_t instr_desc(bool bf16, bool a_mn, bool b_mn, int m, int n) {
  return 1u << 4 | (bf16 ? 1u << 7 | 1u << 10 : 0u) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
         (uint32_t)(n >> 3) << 17 | (uint32_t)(m >> 4) << 24;
}

template <int CG>
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  if (CG == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}

// The same with A in tensor memory: row r in lane r, two k of a row a column.
template <int CG>
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  if (CG == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}

// Arrives on `bar` (CG = 2: on both CTAs' barrier at that offset) when the
// thread's earlier matrix instructions are done.
template <int CG>
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  if (CG == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3) : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// Tiles of the output: `group` rows of tiles are walked column by column, so
// that the tiles in flight at one time form a block whose operands stay in L2.
// (Eight rows of 256, 8192 tokens x 8192 -> 3584 in loops on one machine:
// 614 and 619 us in two runs; four: 634, twelve 625, sixteen 632.  Other sizes
// differ less than their runs do.)
// 32-bit numbers: a thread that copies or stores finds its next tile by four
// divisions, which 64-bit ones would make a good part of a short tile's time.
struct TileWalk {
  uint32_t tiles_m, tiles_n, group;
  uint32_t tiles;  // all planes
};

struct Tile {
  int m, n, z;
};

__device__ __forceinline__ Tile tile_at(const TileWalk& w, uint32_t t) {
  const uint32_t plane = w.tiles_m * w.tiles_n;
  Tile r;
  r.z = (int)(t / plane);
  t -= (uint32_t)r.z * plane;
  const uint32_t band = w.group * w.tiles_n, b = t / band;
  const uint32_t first = b * w.group, rows = min(w.group, w.tiles_m - first);
  t -= b * band;
  r.n = (int)(t / rows);
  r.m = (int)(first + t - (uint32_t)r.n * rows);
  return r;
}

// Host: false where there are more tiles than the numbers hold.
inline bool make_walk(TileWalk* w, int64_t tiles_m, int64_t tiles_n, int64_t planes, int group) {
  if (tiles_m > (1 << 30) || tiles_n > (1 << 30) || tiles_m * tiles_n > (1 << 30)) return false;
  *w = {(uint32_t)tiles_m, (uint32_t)tiles_n, (uint32_t)group, (uint32_t)(tiles_m * tiles_n * planes)};
  return true;
}

// A warp's 32 x 32 results, lane l holding row m0 + l, to columns n0 .. of an
// M x N matrix.  Rows that start on 16 bytes: each lane stores its row's 64
// bytes.  Others: the lanes exchange their words (four butterfly steps swap the
// low four bits of lane and word), so that 16 lanes store 64 contiguous bytes
// of a row; a lane on its own would touch a sector for every element.  All
// lanes of the warp call this.
template <class E>
__device__ __forceinline__ void store_chunk(void* out, int64_t ldc, int64_t m0, int64_t n0, int64_t M, int64_t N,
                                            const float (&v)[32], int align) {
  const int lane = (int)(threadIdx.x & 31);
  const int left = (int)min((int64_t)32, N - n0);
  uint32_t w[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) w[i] = E::pack(v[2 * i], v[2 * i + 1]);
  if (left == 32 && align >= 16) {
    if (m0 + lane >= M) return;
    char* p = static_cast<char*>(out) + ((m0 + lane) * ldc + n0) * 2;
    if (align >= 32) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        st_wide(p + 32 * i, make_uint4(w[8 * i], w[8 * i + 1], w[8 * i + 2], w[8 * i + 3]),
                make_uint4(w[8 * i + 4], w[8 * i + 5], w[8 * i + 6], w[8 * i + 7]));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        st_v4_stream(p + 16 * i, make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]));
    }
    return;
  }
#pragma unroll
  for (int bit = 1; bit < 16; bit <<= 1) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (!(i & bit)) {
        const bool up = (lane & bit) != 0;
        const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, up ? w[i] : w[i | bit], bit);
        w[i] = up ? got : w[i];
        w[i | bit] = up ? w[i | bit] : got;
      }
  }
  const int c = 2 * (lane & 15);
  const int64_t first = m0 + (lane & 16);
  const int rows = first < M ? (int)min((int64_t)16, M - first) : 0;
  char* p = static_cast<char*>(out) + (first * ldc + n0 + c) * 2;
  const bool two = c + 1 < left;
  if (c >= left) return;
#pragma unroll
  for (int j = 0; j < 16; ++j, p += ldc * 2) {
    if (j >= rows) break;
    if (align >= 4 && two) {
      *reinterpret_cast<uint32_t*>(p) = w[j];
    } else {
      *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[j];
      if (two) *reinterpret_cast<uint16_t*>(p + 2) = (uint16_t)(w[j] >> 16);
    }
  }
}

// ---- host: a [rows, cols] matrix copied in boxes of box_rows x box_cols --------------

enum MapType { kMapBf16, kMapF16, kMapU8 };
bool tc_available();
// Boxes of 128-byte rows in the 128-byte swizzle (the 16-byte piece p of row r at
// p ^ (r % 8)), of 64-byte rows in the 64-byte one (p ^ (r / 2 % 4)).
bool tc_make_map(CUtensorMap* map, MapType type, const void* p, int64_t rows, int64_t cols, int64_t ld, int box_rows,
                 int box_cols);

}  // namespace tc
}  // namespace ar
