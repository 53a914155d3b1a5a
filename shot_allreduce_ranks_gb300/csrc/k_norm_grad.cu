// Gradients of the norms before and after a block, its gate and the residual
// (formulas in include/ar.h): every matrix is read and written once.  With hat = N(r) and
// d = dy (offset + weight), the gradient of the norm is factor (d - mean d - hat mean(d hat)), the first
// mean 0 for the mean square, whose two sums, of r^2 and of d r, are therefore one joint sum.
//
// Measured on one GB300: 8192 x 8192 bf16 105 us (537 MB: 75% of the copy rate; the instructions for a row bind),
// 8192 x 4096 60, 4096 x 8192 fp32 87 (91%), 440 x 5120 11.7, one row 5.0. With a norm after the block 8192 x 4096
// 103, and 8192 x 8192 317: a thread of 1,024 has too few registers and reads vectors and rows again. 680 x
// 5120 fp32 with every part 50 (floor 12), likewise: 640 threads of 96 registers spill, and shared memory holds one
// row ahead. 8192 x 1031 bf16 with a mean and biases 71.
#include "norm_device.cuh"

namespace ar {
namespace {

// The rows of a CTA, all of one gate row where split > 0.
__device__ __forceinline__ void rows_of(const NormGradArgs& a, int64_t cta, int64_t& first, int64_t& last) {
  if (a.split) {
    const int64_t g = cta / a.split, j = cta % a.split;
    first = g * a.gate_run + min(j * a.chunk, a.gate_run);
    last = g * a.gate_run + min((j + 1) * a.chunk, a.gate_run);
  } else {
    first = cta * a.gate_rows / a.ctas * a.gate_run;
    last = (cta + 1) * a.gate_rows / a.ctas * a.gate_run;
  }
}

// Any row: a CTA takes its rows one after the other, reads each again for every
// statistic and adds to its own row of the parts, a thread to its own columns.
template <class E>
__global__ void __launch_bounds__(kAnyThreads) k_norm_grad_any(NormGradArgs a) {
  __shared__ float room[8][32];
  pdl_enter();
  const int64_t cta = blockIdx.x;
  int64_t first, last;
  rows_of(a, cta, first, last);
  const auto add = [&](int k, int64_t c, bool start, float v) {
    float* p = a.part[k] + cta * a.cols + c;
    *p = start ? v : *p + v;
  };
  for (int64_t row = first; row < last; ++row) {
    const int64_t gate_row = row / a.gate_run;
    Stats sr = {0.0f, 1.0f}, sx = {0.0f, 1.0f};
    float m[2] = {0.0f, 0.0f};  // means of d and d * N(r), d the gradient of N(r)
    const auto r_hat = [&](int64_t c) { return (value<E>(a.r, row * a.ldr + c) - sr.mean) * sr.factor; };
    const auto d_hat = [&](int64_t c) { return value<E>(a.dy, row * a.lddy + c) * (a.offset + value<E>(a.weight, c)); };
    if (a.weight) {
      sr = stats_any([&](int64_t c) { return value<E>(a.r, row * a.ldr + c); }, a.cols, a.layer, a.eps, room);
      for (int64_t c = threadIdx.x; c < a.cols; c += kAnyThreads) {
        const float d = d_hat(c);
        m[0] += d;
        m[1] = __fmaf_rn(d, r_hat(c), m[1]);
      }
      cta_sums<2>(m, room + 2);
      m[0] = a.layer ? m[0] / (float)a.cols : 0.0f;
      m[1] /= (float)a.cols;
    }
    const auto g = [&](int64_t c) {
      float v = a.dr ? value<E>(a.dr, row * a.lddr + c) : 0.0f;
      if (a.weight) v = __fmaf_rn(sr.factor, d_hat(c) - m[0] - r_hat(c) * m[1], v);
      return v;
    };
    const auto x_hat = [&](int64_t c) { return (value<E>(a.x, row * a.ldx + c) - sx.mean) * sx.factor; };
    const auto dz = [&](int64_t c) { return a.gate ? g(c) * value<E>(a.gate, gate_row * a.ldg + c) : g(c); };
    float n[2] = {0.0f, 0.0f};  // likewise of the norm after the block
    if (a.after_weight) {
      sx = stats_any([&](int64_t c) { return value<E>(a.x, row * a.ldx + c); }, a.cols, a.layer, a.eps, room + 4);
      for (int64_t c = threadIdx.x; c < a.cols; c += kAnyThreads) {
        const float d = dz(c) * (a.offset + value<E>(a.after_weight, c));
        n[0] += d;
        n[1] = __fmaf_rn(d, x_hat(c), n[1]);
      }
      cta_sums<2>(n, room + 6);
      n[0] = a.layer ? n[0] / (float)a.cols : 0.0f;
      n[1] /= (float)a.cols;
    }
    const bool gate_done = a.split == 0 && (row + 1) % a.gate_run == 0;
    for (int64_t c = threadIdx.x; c < a.cols; c += kAnyThreads) {
      const float gv = g(c), dzv = dz(c), hat = a.after_weight ? x_hat(c) : 0.0f;
      if (a.sum[kSumWeight]) add(kSumWeight, c, row == first, value<E>(a.dy, row * a.lddy + c) * r_hat(c));
      if (a.sum[kSumBias]) add(kSumBias, c, row == first, value<E>(a.dy, row * a.lddy + c));
      if (a.sum[kSumAfterWeight]) add(kSumAfterWeight, c, row == first, dzv * hat);
      if (a.sum[kSumAfterBias]) add(kSumAfterBias, c, row == first, dzv);
      if (a.sum[kSumGate]) {
        float z = a.after_weight ? hat * (a.offset + value<E>(a.after_weight, c)) : value<E>(a.x, row * a.ldx + c);
        if (a.after_bias) z += value<E>(a.after_bias, c);
        add(kSumGate, c, row % a.gate_run == 0 || row == first, gv * z);
        if (gate_done) put<E>(a.sum[kSumGate], gate_row * a.lddg + c, a.part[kSumGate][cta * a.cols + c]);
      }
      if (a.dresidual) put<E>(a.dresidual, row * a.lddres + c, a.alpha * gv);
      if (a.dx)
        put<E>(a.dx, row * a.lddx + c,
               a.after_weight ? sx.factor * (dzv * (a.offset + value<E>(a.after_weight, c)) - n[0] - hat * n[1]) : dzv);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Gradients of rows that T threads hold in registers and shared memory.
//
// (A kernel for any row, which read it again for every statistic, took 1,238 us at 8192 x 8192.)
//
// The columns' sums over rows stay in a thread's registers while its CTA walks
// its rows; a CTA of short rows has several groups of T threads, each with rows of
// its own.  A row's statistics and the two means that the gradient wants come out of one
// joint sum (mean square) or two (differences from the mean), and one more for the norm
// after the block.  The next rows are copied to shared memory meanwhile, as many as fit beside a row's own: one to three, or none
// (8,192 columns of fp32 with a gate or biases).
constexpr int kGroupThreads = 256;  // of a CTA of short rows

__host__ __device__ constexpr int row_threads(int64_t cols, int n) { return (int)((cols + 32 * n - 1) / (32 * n) * 32); }
__host__ __device__ constexpr int row_groups(int threads) { return threads < kGroupThreads ? kGroupThreads / threads : 1; }

// Sums of up to four values over a warp: at the first steps a lane gives away the
// values that its half (or quarter) does not finish, so that N values cost about
// as many shuffles as one (the SM does one of them a clock).  Lane 32 / P * k
// and the ones after it end with value k, P = N rounded up to a power of two.
template <int N>
__device__ __forceinline__ float spread_sums(const float (&v)[N], int lane) {
  constexpr int P = N == 1 ? 1 : N == 2 ? 2 : 4;
  float a = v[0];
  if (P == 2) {
    const bool high = lane & 16;
    a = (high ? v[N > 1 ? 1 : 0] : v[0]) + __shfl_xor_sync(0xFFFFFFFFu, high ? v[0] : v[N > 1 ? 1 : 0], 16);
  }
  if (P == 4) {
    const bool high = lane & 16, odd = lane & 8;
    const float v1 = v[N > 1 ? 1 : 0], v2 = v[N > 2 ? 2 : 0], v3 = N > 3 ? v[N - 1] : 0.0f;
    const float b0 = (high ? v2 : v[0]) + __shfl_xor_sync(0xFFFFFFFFu, high ? v[0] : v2, 16);
    const float b1 = (high ? v3 : v1) + __shfl_xor_sync(0xFFFFFFFFu, high ? v1 : v3, 16);
    a = (odd ? b1 : b0) + __shfl_xor_sync(0xFFFFFFFFu, odd ? b0 : b1, 8);
  }
#pragma unroll
  for (int o = 16 / P; o; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
  return a;
}

// Sums over the T threads of a group, which has its own barrier; room: a row of 32 for each value.
template <int N>
__device__ __forceinline__ void group_sums(float (&v)[N], float (*room)[32], int group, int T) {
  constexpr int P = N == 1 ? 1 : N == 2 ? 2 : 4, kSpan = 32 / P;
  const int lane = threadIdx.x & 31, k = lane / kSpan, in = lane % kSpan;
  float a = spread_sums<N>(v, lane);
  if (T > 32) {
    const int warp = (threadIdx.x >> 5) - group * (T >> 5), warps = T >> 5;
    if (in == 0 && k < N) room[k][warp] = a;
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(T) : "memory");
    a = 0.0f;
    if (k < N) {
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (in + kSpan * i < warps) a += room[k][in + kSpan * i];
    }
#pragma unroll
    for (int o = kSpan / 2; o; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = P == 1 ? a : __shfl_sync(0xFFFFFFFFu, a, kSpan * i);
}

enum { kDy = 0, kDr, kR, kX };  // the matrices that are read

// What stands between x and r.  kNothing; kAfter: the norm after the block alone, without biases; kAll: any
// of it.
enum { kNothing = 0, kAfter, kAll };

// BIAS: dbias is wanted (kAll always has it).  In kAll the sums of the norm after the block and of the
// gate are kept in shared memory, each thread's its own, since five sums would not fit a thread's registers.
template <class E, int N, int MAXT, int MINB, bool VEC, bool LAYER, int BRANCH, bool BIAS>
__global__ void __launch_bounds__(MAXT, MINB) k_norm_grad_rows(NormGradArgs a, int T, int stages) {
  constexpr int G = E::kGroup, kPieces = N / G, kMats = BRANCH ? 4 : 3;
  constexpr bool FULL = BRANCH != kNothing, ALL = BRANCH == kAll;
  extern __shared__ __align__(16) char smem[];
  __shared__ float rooms[MAXT > kGroupThreads ? 1 : 4][2][8][32];  // groups of one warp use none
  pdl_enter();
  const int groups = (int)blockDim.x / T, group = (int)threadIdx.x / T;
  const Columns<E, N, VEC ? kAligned : kShifted> c = {(int)threadIdx.x - group * T, T, (int)a.cols};
  const float inv = 1.0f / (float)a.cols;
  int64_t first, last, step;
  if (a.split) {
    rows_of(a, blockIdx.x, first, last);
    first += group, step = groups;
  } else {
    const int64_t unit = (int64_t)blockIdx.x * groups + group, units = a.ctas * groups;
    first = unit * a.gate_rows / units * a.gate_run, last = (unit + 1) * a.gate_rows / units * a.gate_run, step = 1;
  }
  const bool has_weight = !FULL || a.weight;  // one of the two norms is there
  const void* const mats[4] = {a.dy, a.dr, has_weight ? a.r : nullptr, FULL ? a.x : nullptr};
  const int64_t lds[4] = {a.lddy, a.lddr, a.ldr, a.ldx};
  const Staged<E, N, VEC> rows = {c};
  const int mat_bytes = rows.bytes(T), stage_bytes = kMats * mat_bytes;
  const uint32_t mine = (uint32_t)__cvta_generic_to_shared(smem) + group * stages * stage_bytes;
  const auto row_of = [&](int m, int64_t row) { return static_cast<const char*>(mats[m]) + row * (lds[m] * E::kBytes); };
  const auto fetch = [&](int64_t row, int stage) {
    if (row < last) {
#pragma unroll
      for (int m = 0; m < kMats; ++m)
        if (mats[m])
          rows.fetch(mine + stage * stage_bytes + m * mat_bytes, row_of(m, row), row_of(m, 0),
                     VEC ? nullptr : row_of(m, a.rows - 1) + a.cols * E::kBytes);
    }
    copies_commit();
  };
  // The row's part of matrix m in v.
  const auto get = [&](int m, int64_t row, int stage, float(&v)[N]) {
    rows.read(mine + stage * stage_bytes + m * mat_bytes, VEC ? 0 : (int)(reinterpret_cast<uintptr_t>(row_of(m, row)) & 15u), v);
  };

  // The weight stays in registers where no other vector takes turns with it.
  float w[N];
  if constexpr (!FULL) {
    c.load_shared(a.weight, 0, a.cols, w);
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] += a.offset;  // past the last column dy is 0
  }
  float dw[N] = {}, db[BIAS ? N : 1] = {}, daw[BRANCH == kAfter ? N : 1] = {};
  // kAll's sums: piece q of sum k, four columns; and what is added to them.
  float4* const sums = reinterpret_cast<float4*>(smem + a.sums_at) + threadIdx.x;
  constexpr int kQuads = N / 4;
  const auto sum_at = [&](int k, int q) -> float4& { return sums[((k - kSumAfterWeight) * kQuads + q) * (int)blockDim.x]; };
  const auto add = [&](int k, const float(&v)[N]) {
#pragma unroll
    for (int q = 0; q < kQuads; ++q) {
      float4 t = sum_at(k, q);
      t.x += v[4 * q], t.y += v[4 * q + 1], t.z += v[4 * q + 2], t.w += v[4 * q + 3];
      sum_at(k, q) = t;
    }
  };
  const auto clear = [&](int k) {
#pragma unroll
    for (int q = 0; q < kQuads; ++q) sum_at(k, q) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  };
  const auto total = [&](int k, float(&v)[N]) {
#pragma unroll
    for (int q = 0; q < kQuads; ++q) {
      const float4 t = sum_at(k, q);
      v[4 * q] = t.x, v[4 * q + 1] = t.y, v[4 * q + 2] = t.z, v[4 * q + 3] = t.w;
    }
  };
  if constexpr (ALL) clear(kSumAfterWeight), clear(kSumAfterBias), clear(kSumGate);
  const auto meet = [&] {
    if (T == 32)
      __syncwarp();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(T) : "memory");
  };
  const auto wait_but = [](int later) {  // for all copies but the latest `later` groups
    if (later == 3)
      copies_wait<3>();
    else if (later == 2)
      copies_wait<2>();
    else if (later == 1)
      copies_wait<1>();
    else
      copies_wait<0>();
  };
  for (int i = 0; i < stages - 1; ++i) fetch(first + i * step, i);
  // The gate's row that a row is of, and where that one's rows end: all of a CTA's rows are of one gate row, or they follow one another.
  int64_t gate_row = 0, gate_end = 0;
  if (ALL && a.gate) gate_row = first / a.gate_run, gate_end = (gate_row + 1) * a.gate_run;
  int stage = 0, parity = 0;
  for (int64_t row = first; row < last; row += step) {
    const int64_t ahead = row + (stages - 1) * step;
    const int refilled = stage == 0 ? stages - 1 : stage - 1;
    if (VEC) {
      fetch(ahead, refilled);
      wait_but(stages - 1);
    } else {
      // Neighbours read each other's copies: a stage is refilled once all have left its row.
      if (stages == 1) {
        meet();
        fetch(ahead, refilled);
        wait_but(0);
        meet();
      } else {
        wait_but(stages - 2);
        meet();
        fetch(ahead, refilled);
      }
    }
    float(*room)[32] = rooms[group][parity];
    float r[N], d[N];
    float rmean = 0.0f, rfactor = 1.0f, xmean = 0.0f, xfactor = 1.0f, m0 = 0.0f, m1 = 0.0f;
    if (has_weight) {
      get(kR, row, stage, r);
      get(kDy, row, stage, d);
      if constexpr (FULL) {
        c.load_shared(a.weight, 0, a.cols, w);
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] += a.offset;
      }
    }
    float x[FULL ? N : 1];
    if constexpr (FULL) get(kX, row, stage, x);
    // Two sums of the norm before the next block, and one of that after this one.
    constexpr int kSums = FULL ? 3 : 2;
    const auto centred = [&](float v, float mean, int i) { return LAYER ? (c.has(i) ? v - mean : 0.0f) : v; };
    if (LAYER) {
      float s[kSums] = {};
      if (has_weight) {
#pragma unroll
        for (int i = 0; i < N; ++i) s[0] += r[i], s[1] = __fmaf_rn(d[i], w[i], s[1]);
      }
      if constexpr (FULL) {
#pragma unroll
        for (int i = 0; i < N; ++i) s[2] += x[i];
        group_sums<kSums>(s, room, group, T);
        xmean = s[2] * inv;
      } else {
        group_sums<kSums>(s, room, group, T);
      }
      rmean = s[0] * inv, m0 = s[1] * inv;
    }
    {
      float s[kSums] = {};
      if (has_weight) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float v = centred(r[i], rmean, i);
          s[0] = __fmaf_rn(v, v, s[0]);
          s[1] = __fmaf_rn(d[i] * w[i], v, s[1]);
        }
      }
      if constexpr (FULL) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float v = centred(x[i], xmean, i);
          s[2] = __fmaf_rn(v, v, s[2]);
        }
      }
      group_sums<kSums>(s, room + 3, group, T);
      if (has_weight) {
        rfactor = rsqrtf(__fmaf_rn(s[0], inv, a.eps));
        m1 = s[1] * inv * rfactor;
      }
      if constexpr (FULL) {
        if (a.after_weight) xfactor = rsqrtf(__fmaf_rn(s[2], inv, a.eps));
      }
    }
    // What a thread of a large CTA has no registers for it reads again: with 80 of them where a gate or biases take
    // more (4096 x 6144 bf16 197 us, kept 206; after the block alone 92, kept 89), with 64 always.
    constexpr bool kAgain = FULL && MAXT > (ALL ? 640 : 768);
    if constexpr (kAgain) {
      if (has_weight) {
        get(kR, row, stage, r);
        get(kDy, row, stage, d);
        c.load_shared(a.weight, 0, a.cols, w);
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] += a.offset;
      }
    }
    float g[N];
    if (a.dr) {
      get(kDr, row, stage, g);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) g[i] = 0.0f;
    }
    if (has_weight) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float hat = (LAYER ? r[i] - rmean : r[i]) * rfactor, t = LAYER ? __fmaf_rn(d[i], w[i], -m0) : d[i] * w[i];
        g[i] = __fmaf_rn(rfactor, __fmaf_rn(-hat, m1, t), g[i]);
        dw[i] = __fmaf_rn(d[i], hat, dw[i]);
        if constexpr (BIAS) db[i] += d[i];
      }
    }
    if (a.dresidual) {
#pragma unroll
      for (int i = 0; i < N; ++i) r[i] = a.alpha * g[i];
      c.store(a.dresidual, row * a.lddres, r);
    }
    if constexpr (kAgain) get(kX, row, stage, x);
    if constexpr (ALL) {
      if (a.gate) {
        float v[N];
        if (a.after_weight) {
          c.load_shared(a.after_weight, 0, a.cols, w);
          if (a.after_bias)
            c.load_shared(a.after_bias, 0, a.cols, d);
          else
#pragma unroll
            for (int i = 0; i < N; ++i) d[i] = 0.0f;
#pragma unroll
          for (int i = 0; i < N; ++i) v[i] = g[i] * __fmaf_rn((LAYER ? x[i] - xmean : x[i]) * xfactor, a.offset + w[i], d[i]);
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i) v[i] = g[i] * x[i];
        }
        add(kSumGate, v);
        if (!a.split && row + 1 == gate_end) {
          total(kSumGate, v);
          if (a.sum[kSumGate]) c.store(a.sum[kSumGate], gate_row * a.lddg, v);
          clear(kSumGate);
        }
        c.load_shared(a.gate, gate_row * a.ldg, (a.gate_rows - 1) * a.ldg + a.cols, w);
#pragma unroll
        for (int i = 0; i < N; ++i) g[i] *= w[i];
        if (!a.split && row + 1 == gate_end) ++gate_row, gate_end += a.gate_run;
      }
    }
    if constexpr (FULL) {
      if (a.after_weight) {
        c.load_shared(a.after_weight, 0, a.cols, w);
        float s[2] = {}, v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
          w[i] += a.offset;
          const float hat = centred(x[i], xmean, i) * xfactor;
          v[i] = g[i] * hat;
          if (LAYER) s[0] += c.has(i) ? g[i] * w[i] : 0.0f;
          s[1] = __fmaf_rn(v[i], w[i], s[1]);
          if constexpr (!ALL) daw[i] += v[i];
        }
        if constexpr (ALL) {
          add(kSumAfterWeight, v);
          if (a.sum[kSumAfterBias]) add(kSumAfterBias, g);
        }
        if constexpr (LAYER) {
          group_sums<2>(s, room + 6, group, T);
        } else {
          float one[1] = {s[1]};
          group_sums<1>(one, room + 6, group, T);
          s[1] = one[0];
        }
        const float n0 = LAYER ? s[0] * inv : 0.0f, n1 = s[1] * inv;
#pragma unroll
        for (int i = 0; i < N; ++i)
          g[i] = xfactor * __fmaf_rn(LAYER ? xmean - x[i] : -x[i], xfactor * n1, LAYER ? __fmaf_rn(g[i], w[i], -n0) : g[i] * w[i]);
      }
    }
    if (a.dx) c.store(a.dx, row * a.lddx, g);
    parity ^= 1;
    stage = stage == stages - 1 ? 0 : stage + 1;
  }

  // The groups' sums are joined in their order, through shared memory, and stored as the CTA's part.
  copies_wait<0>();
  float* sum = reinterpret_cast<float*>(smem);
  const auto finish = [&](int k, const float(&v)[N]) {
    if (!a.sum[k] || (k == kSumGate && !a.split)) return;
    for (int q = 0; q < groups; ++q) {
      if (groups > 1) __syncthreads();
      if (q != group) continue;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (!c.has(i)) continue;
        const float t = q ? sum[c.at(i)] + v[i] : v[i];
        if (q < groups - 1)
          sum[c.at(i)] = t;
        else if (a.direct)
          put<E>(a.sum[k], c.at(i), t);
        else
          a.part[k][(int64_t)blockIdx.x * a.cols + c.at(i)] = t;
      }
    }
  };
  finish(kSumWeight, dw);
  if constexpr (BIAS) finish(kSumBias, db);
  if constexpr (BRANCH == kAfter) finish(kSumAfterWeight, daw);
  if constexpr (ALL) {
#pragma unroll
    for (int k = kSumAfterWeight; k <= kSumGate; ++k) {
      total(k, dw);
      finish(k, dw);
    }
  }
}

// The CTAs' parts joined: output row blockIdx.z of sum blockIdx.y.  32 columns a
// CTA; its warps take turns at the parts and are joined in their order.
struct JoinArgs {
  const float* part[kNormSums];
  void* sum[kNormSums];
  int64_t count[kNormSums], rows[kNormSums], ld[kNormSums];  // parts of an output row; output rows
  int64_t cols;
};
constexpr int kJoinWarps = 16;

template <class E>
__global__ void __launch_bounds__(32 * kJoinWarps) k_norm_join(JoinArgs a) {
  __shared__ float room[kJoinWarps][32];
  pdl_enter();
  const int k = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = blockIdx.z, c = (int64_t)blockIdx.x * 32 + lane;
  if (row >= a.rows[k]) return;
  const float* p = a.part[k] + row * a.count[k] * a.cols;
  float v = 0.0f;
  if (c < a.cols) {
#pragma unroll 8
    for (int64_t i = warp; i < a.count[k]; i += kJoinWarps) v += p[i * a.cols + c];
  }
  room[warp][lane] = v;
  __syncthreads();
  if (warp || c >= a.cols) return;
  v = 0.0f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) v += room[w][lane];
  put<E>(a.sum[k], row * a.ld[k] + c, v);
}

// The rows dealt out to at most `want` CTAs: where there are fewer gate rows each is
// split among as many CTAs; where there are more, a CTA takes several whole ones.
void deal(NormGradArgs& a, int64_t want) {
  if (a.gate_rows <= want) {
    const int64_t parts = want / a.gate_rows;
    a.chunk = (a.gate_run + parts - 1) / parts;
    a.split = (a.gate_run + a.chunk - 1) / a.chunk;
    a.ctas = a.gate_rows * a.split;
  } else {
    a.split = a.chunk = 0;
    a.ctas = want;
  }
}

template <class E, int N, bool VEC, bool LAYER, int BRANCH, bool BIAS>
cudaError_t norm_grad_rows_kind(NormGradArgs& a, int num_sms, cudaStream_t s) {
  constexpr int kMats = BRANCH ? 4 : 3;
  constexpr bool ALL = BRANCH == kAll;
  const int T = row_threads(a.cols, N), cta = T < kGroupThreads ? T * row_groups(T) : T;
  // 64 registers a thread, or 128 with a branch up to 512 threads; as many stages as fit beside one another.
  const int per_sm = cta > 512 || (BRANCH && cta > 256) ? 1 : BRANCH ? 512 / cta : 1024 / cta;
  const int64_t stage = (int64_t)kMats * Staged<E, N, VEC>::bytes(T) * (cta / T), sums = ALL ? (int64_t)3 * N * 4 * cta : 0;
  const int64_t room = (228 * 1024) / per_sm - 1024 - (cta > kGroupThreads ? 2048 : 8192) - sums;
  const int stages = room >= 4 * stage ? 4 : room >= 3 * stage ? 3 : room >= 2 * stage ? 2 : 1;
  int64_t smem = stages * stage;
  // The groups' sums are joined at the front, where no thread's sums may lie yet.
  if (smem < a.cols * 4 && cta > T) smem = a.cols * 4;
  a.sums_at = (int)((smem + 15) / 16 * 16);
  smem = a.sums_at + sums;
  int64_t want = (int64_t)per_sm * num_sms;
  const int64_t most = norm_parts(a.rows, a.cols);
  if (want > most) want = most;
  // A CTA that takes two rows a group costs less than joining two CTAs' parts (a launch, 3 us).
  if (a.gate_rows == 1 && a.rows <= 2 * (cta / T)) want = 1;
  deal(a, want);
  a.direct = a.ctas == 1;
  const dim3 grid((unsigned)a.ctas);
#define AR_GRAD_ROWS(MAXT, MINB) launch_raised<k_norm_grad_rows<E, N, MAXT, MINB, VEC, LAYER, BRANCH, BIAS>>(grid, cta, (size_t)smem, s, a, T, stages)
  if constexpr (N == 8) {
    if (cta <= 256) return AR_GRAD_ROWS(256, (BRANCH ? 2 : 4));
    if (cta <= 512) return AR_GRAD_ROWS(512, (BRANCH ? 1 : 2));
    // A scheduler's registers are shared by its warps: five of them (up to 640 threads) have 96 each, six (768) 80, eight 64.
    // With a branch, 680 x 5120 fp32 with every part takes 51 us of 96 registers and 58 of 80, 680 x 6144 66 of 80 and
    // 73 of 64; with a norm after the block alone 27 and 30, 33 and 43, and 4096 x 6144 bf16 89 and 140. (Seven warps
    // with 72: 680 x 7168 79 and 84, 4096 x 7168 bf16 139 and 160; not built.)
    if constexpr (BRANCH != kNothing) {
      if (cta <= 640) return AR_GRAD_ROWS(640, 1);
      if (cta <= 768) return AR_GRAD_ROWS(768, 1);
    }
  }
  return AR_GRAD_ROWS(1024, 1);
#undef AR_GRAD_ROWS
}

template <class E, int N, bool VEC, int BRANCH, bool BIAS>
cudaError_t norm_grad_rows(NormGradArgs& a, int num_sms, cudaStream_t s) {
  return a.layer ? norm_grad_rows_kind<E, N, VEC, true, BRANCH, BIAS>(a, num_sms, s)
                 : norm_grad_rows_kind<E, N, VEC, false, BRANCH, BIAS>(a, num_sms, s);
}

template <class E>
cudaError_t norm_grad(NormGradArgs& a, int num_sms, cudaStream_t s) {
  const bool branch = a.gate || a.after_weight, after = a.after_weight && !a.gate && !a.sum[kSumAfterBias] && !a.sum[kSumBias];
  const bool vec = on16<E>(a.dy, a.lddy, a.rows) && on16<E>(a.dr, a.lddr, a.rows) && on16<E>(a.r, a.ldr, a.rows) &&
                   on16<E>(a.x, a.ldx, a.rows) && on16<E>(a.dx, a.lddx, a.rows) && on16<E>(a.dresidual, a.lddres, a.rows) &&
                   on16<E>(a.gate, a.ldg, a.gate_rows) && on16<E>(a.sum[kSumGate], a.lddg, a.gate_rows) && on16(a.after_weight) &&
                   on16(a.after_bias) && on16(a.weight);
  cudaError_t e;
  if (a.cols <= 8192) {
    if (vec)
      e = after               ? norm_grad_rows<E, 8, true, kAfter, false>(a, num_sms, s)
          : branch            ? norm_grad_rows<E, 8, true, kAll, true>(a, num_sms, s)
          : a.sum[kSumBias] ? norm_grad_rows<E, 8, true, kNothing, true>(a, num_sms, s)
                            : norm_grad_rows<E, 8, true, kNothing, false>(a, num_sms, s);
    else
      e = branch              ? norm_grad_rows<E, 8, false, kAll, true>(a, num_sms, s)
          : a.sum[kSumBias] ? norm_grad_rows<E, 8, false, kNothing, true>(a, num_sms, s)
                            : norm_grad_rows<E, 8, false, kNothing, false>(a, num_sms, s);
  } else if (a.cols <= 16384 && vec && !branch && E::kBytes == 2) {
    e = norm_grad_rows<E, 16, true, kNothing, true>(a, num_sms, s);
  } else {
    const int64_t want = 2 * (int64_t)num_sms, most = norm_parts(a.rows, a.cols);
    deal(a, want < most ? want : most);
    e = launch_op(k_norm_grad_any<E>, dim3((unsigned)a.ctas), kAnyThreads, 0, 1, s, a);
  }
  if (e != cudaSuccess) return e;
  JoinArgs j = {};
  j.cols = a.cols;
  int n = 0;
  int64_t deepest = 1;
  for (int k = 0; k < kNormSums; ++k) {
    if (!a.sum[k] || (k == kSumGate && !a.split)) continue;  // those gates are whole already
    if (a.direct) continue;
    const bool gate = k == kSumGate;
    j.part[n] = a.part[k], j.sum[n] = a.sum[k];
    j.count[n] = gate ? a.split : a.ctas, j.rows[n] = gate ? a.gate_rows : 1, j.ld[n] = gate ? a.lddg : 0;
    deepest = j.rows[n] > deepest ? j.rows[n] : deepest;
    ++n;
  }
  if (!n) return cudaSuccess;
  return launch_op(k_norm_join<E>, dim3((unsigned)((a.cols + 31) / 32), (unsigned)n, (unsigned)deepest), 32 * kJoinWarps, 0, 1, s, j);
}

}  // namespace

int64_t norm_parts(int64_t rows, int64_t cols) {
  const int64_t most = cols <= 4096 ? 4 * kMostSms : cols <= 8192 ? 2 * kMostSms : kMostSms;
  return rows < most ? rows : most;
}

cudaError_t launch_norm_grad(int dtype, NormGradArgs& a, int num_sms, cudaStream_t s) {
  switch (dtype) {
    case AR_BF16: return norm_grad<Bf16>(a, num_sms, s);
    case AR_FP16: return norm_grad<F16>(a, num_sms, s);
    default: return norm_grad<F32>(a, num_sms, s);
  }
}

}  // namespace ar
