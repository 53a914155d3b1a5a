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

struct Draws4 {
  uint32_t w[4];
};

__device__ __forceinline__ Draws4 philox(uint64_t at, uint64_t sequence, uint64_t seed) {
  uint32_t c0 = (uint32_t)at, c1 = (uint32_t)(at >> 32);
  uint32_t c2 = (uint32_t)sequence, c3 = (uint32_t)(sequence >> 32);
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return {{c0, c1, c2, c3}};
}

// A thread takes one group (16 bytes) of a row at a time.  The draws of a
// group come from G/4 blocks, one more where the group begins inside a block.
template <class E, bool RES, bool VEC>
__global__ void __launch_bounds__(kDropThreads) k_dropout(DropoutArgs a, int64_t groups_per_row) {
  constexpr int G = E::kGroup, B = E::kBytes, W = 4;
  const int64_t total = a.rows * groups_per_row;
  for (int64_t i = (int64_t)blockIdx.x * kDropThreads + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * kDropThreads) {
    const int64_t row = groups_per_row == total ? 0 : i / groups_per_row;
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
    const int phase = (int)(first & 3);
    uint32_t d[G + 4];
#pragma unroll
    for (int b = 0; b < G / 4; ++b) {
      const Draws4 w = philox(first / 4 + b, a.sequence, a.seed);
#pragma unroll
      for (int k = 0; k < 4; ++k) d[4 * b + k] = w.w[k];
    }
    if (phase) {
      const Draws4 w = philox(first / 4 + G / 4, a.sequence, a.seed);
#pragma unroll
      for (int k = 0; k < 4; ++k) d[G + k] = w.w[k];
#pragma unroll
      for (int k = 0; k < G; ++k) {
        const uint32_t far = phase & 2 ? d[k + 2] : d[k], near = phase & 2 ? d[k + 3] : d[k + 1];
        d[k] = phase & 1 ? near : far;
      }
    }

    float y[G];
#pragma unroll
    for (int k = 0; k < G; ++k) {
      const uint32_t bits = B == 2 ? (xw[k / 2] >> (16 * (k & 1))) & 0xFFFFu : xw[k & 3];
      const uint32_t rbits = B == 2 ? (rw[k / 2] >> (16 * (k & 1))) & 0xFFFFu : rw[k & 3];
      // A dropped element is 0 whatever it held, a NaN too: selected, not multiplied.
      y[k] = d[k] >= a.threshold && !a.drop_all ? E::to_f32(bits) * a.scale : 0.0f;
      if (RES) y[k] = y[k] + E::to_f32(rbits);
    }
    if (VEC && n == G) {
      uint32_t o[W];
#pragma unroll
      for (int w = 0; w < W; ++w)
        o[w] = B == 2 ? E::from_f32(y[(2 * w) % G]) | E::from_f32(y[(2 * w + 1) % G]) << 16
                      : __float_as_uint(y[w % G]);
      st_v4_stream(po, make_uint4(o[0], o[1], o[2], o[3]));
    } else {
#pragma unroll
      for (int k = 0; k < G; ++k)
        if (k < n) {
          if (B == 2)
            reinterpret_cast<uint16_t*>(po)[k] = (uint16_t)E::from_f32(y[k]);
          else
            reinterpret_cast<float*>(po)[k] = y[k];
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
  auto* k = a.residual ? (vec ? k_dropout<E, true, true> : k_dropout<E, true, false>)
                       : (vec ? k_dropout<E, false, true> : k_dropout<E, false, false>);
  k<<<grid, kDropThreads, 0, s>>>(a, gpr);
  return cudaGetLastError();
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
