// Dropout whose mask is drawn from a counter-based generator and never stored.
//
// Element i of the whole tensor (i = offset + row * cols + column) is kept
// where draw(i) >= round(p 2^32); draw(i) is word i mod 4 of Philox4x32-10
// ("Parallel random numbers: as easy as 1, 2, 3", Salmon, Moraes, Dror, Shaw,
// 2011) of the 128-bit counter {i / 4, sequence} under the 64-bit key `seed`.
// The mask is a function of the element's place alone: every rank that holds
// a copy draws the same one without an exchange, a rank that holds a block
// draws its part by `offset`, and the backward pass draws it again.
#include "ops_internal.cuh"

namespace ar {
namespace {

constexpr int kDropThreads = 256;

// The ten rounds' keys: one set for a call, computed on the host.
struct RoundKeys {
  uint32_t k0[10], k1[10];
};

__device__ __forceinline__ void philox(uint32_t (&d)[4], uint32_t lo, uint32_t hi, uint64_t sequence,
                                       const RoundKeys& key) {
  uint32_t c0 = lo, c1 = hi, c2 = (uint32_t)sequence, c3 = (uint32_t)(sequence >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ key.k0[r];
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ key.k1[r];
    c3 = (uint32_t)a;
  }
  d[0] = c0, d[1] = c1, d[2] = c2, d[3] = c3;
}

__device__ __forceinline__ uint64_t f32x2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Elements 2w and 2w + 1 of a group whose 16 bytes are `v` (B = 2: word w; B = 4: words 2w and 2w + 1).
template <class E>
__device__ __forceinline__ uint64_t pair_of(const uint32_t (&v)[4], int w) {
  return Acc2<E>::widen(v[w]);
}
template <>
__device__ __forceinline__ uint64_t pair_of<F32>(const uint32_t (&v)[4], int w) {
  return f32x2_make(v[(2 * w) & 3], v[(2 * w + 1) & 3]);
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

// A thread takes one group (16 bytes) of a row at a time.  The draws of a
// group come from G/4 blocks; WHOLE: every group begins where a block does,
// else one block more is drawn and the words shifted into place.
template <class E, bool RES, bool VEC, bool WHOLE>
__global__ void __launch_bounds__(kDropThreads)
    k_dropout(const __grid_constant__ DropoutArgs a, const __grid_constant__ RoundKeys key, int64_t groups_per_row) {
  pdl_enter();
  constexpr int G = E::kGroup, B = E::kBytes, W = 4;
  const int64_t total = a.rows * groups_per_row;
  const uint64_t scale = f32x2_make(__float_as_uint(a.scale), __float_as_uint(a.scale));
  for (int64_t i = (int64_t)blockIdx.x * kDropThreads + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * kDropThreads) {
    const int64_t row = groups_per_row == total ? 0
                        : total >> 32           ? i / groups_per_row
                                                : (int64_t)((uint32_t)i / (uint32_t)groups_per_row);
    const int64_t col = (i - row * groups_per_row) * G;
    const int n = (int)(a.cols - col < G ? a.cols - col : G);
    const char* px = static_cast<const char*>(a.x) + (row * a.ldx + col) * B;
    const char* pr = RES ? static_cast<const char*>(a.residual) + (row * a.ldr + col) * B : nullptr;
    char* po = static_cast<char*>(a.out) + (row * a.ldo + col) * B;

    uint32_t xw[W] = {}, rw[W] = {};
    if (VEC && n == G) {
      const uint4 v = ld_v4_stream(px);
      xw[0] = v.x, xw[1] = v.y, xw[2] = v.z, xw[3] = v.w;
      if (RES) {
        const uint4 r = ld_v4_stream(pr);
        rw[0] = r.x, rw[1] = r.y, rw[2] = r.z, rw[3] = r.w;
      }
    } else {
#pragma unroll
      for (int k = 0; k < G; ++k)
        if (k < n) {
          xw[k * B / 4] |= ld_elem<B>(px + k * B) << (8 * (k * B % 4));
          if (RES) rw[k * B / 4] |= ld_elem<B>(pr + k * B) << (8 * (k * B % 4));
        }
    }

    const uint64_t first = a.offset + (uint64_t)row * (uint64_t)a.cols + (uint64_t)col;
    const uint64_t block = first >> 2;
    uint32_t d[G + 4];
#pragma unroll
    for (int b = 0; b < G / 4 + (WHOLE ? 0 : 1); ++b) {
      uint32_t w[4];
      philox(w, (uint32_t)(block + b), (uint32_t)((block + b) >> 32), a.sequence, key);
#pragma unroll
      for (int k = 0; k < 4; ++k) d[4 * b + k] = w[k];
    }
    if (!WHOLE) {
      const int phase = (int)(first & 3);
#pragma unroll
      for (int k = 0; k < G; ++k) {
        const uint32_t far = phase & 2 ? d[k + 2] : d[k], near = phase & 2 ? d[k + 3] : d[k + 1];
        d[k] = phase & 1 ? near : far;
      }
    }

    float y[G];
#pragma unroll
    for (int w = 0; w < G / 2; ++w) {
      float lo, hi;
      f32x2_split(f32x2_mul(pair_of<E>(xw, w), scale), lo, hi);
      // A dropped element is 0 whatever it held, a NaN too: selected, not multiplied.
      lo = d[2 * w] >= a.threshold ? lo : 0.0f;
      hi = d[2 * w + 1] >= a.threshold ? hi : 0.0f;
      if (a.drop_all) lo = hi = 0.0f;
      if (RES)
        f32x2_split(f32x2_add(f32x2_make(__float_as_uint(lo), __float_as_uint(hi)), pair_of<E>(rw, w)), lo, hi);
      y[2 * w] = lo, y[2 * w + 1] = hi;
    }
    uint32_t o[W];
    pack_group<E>(o, y);
    if (VEC && n == G) {
      st_v4_stream(po, make_uint4(o[0], o[1], o[2], o[3]));
    } else {
#pragma unroll
      for (int k = 0; k < G; ++k)
        if (k < n) {
          if (B == 2)
            reinterpret_cast<uint16_t*>(po)[k] = (uint16_t)(o[k / 2] >> (16 * (k & 1)));
          else
            reinterpret_cast<uint32_t*>(po)[k] = o[k & 3];
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
  const int64_t want = (a.rows * gpr + kDropThreads - 1) / kDropThreads;
  const unsigned grid = (unsigned)(want < (int64_t)num_sms * 32 ? want : (int64_t)num_sms * 32);
  uintptr_t ptrs = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.out) |
                   reinterpret_cast<uintptr_t>(a.residual);
  bool vec = (ptrs & 15u) == 0;
  if (a.rows > 1)
    vec = vec && a.ldx % E::kGroup == 0 && a.ldo % E::kGroup == 0 &&
          (!a.residual || a.ldr % E::kGroup == 0);
  const bool whole = a.offset % 4 == 0 && (a.rows == 1 || a.cols % 4 == 0);
  RoundKeys key;
  for (int r = 0; r < 10; ++r) {
    key.k0[r] = (uint32_t)a.seed + (uint32_t)r * 0x9E3779B9u;
    key.k1[r] = (uint32_t)(a.seed >> 32) + (uint32_t)r * 0xBB67AE85u;
  }
  using Kernel = void (*)(DropoutArgs, RoundKeys, int64_t);
  static const Kernel kernels[8] = {
      k_dropout<E, false, false, false>, k_dropout<E, false, false, true>, k_dropout<E, false, true, false>,
      k_dropout<E, false, true, true>,   k_dropout<E, true, false, false>, k_dropout<E, true, false, true>,
      k_dropout<E, true, true, false>,   k_dropout<E, true, true, true>};
  const Kernel k = kernels[(a.residual ? 4 : 0) + (vec ? 2 : 0) + (whole ? 1 : 0)];
  return launch_op(k, dim3(grid), kDropThreads, 0, 1, s, a, key, gpr);
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
