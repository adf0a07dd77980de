// Warp-level tf32 products of 64-row tiles held in shared memory as fp32, shared by
// the softmax-attention kernels that do not run on tcgen05.
#pragma once

#include "attn.cuh"
#include "tc_util.cuh"

namespace falcon {

constexpr int kMmaRows = 64;  // of a staged tile

// rows [first, first + 64) of x (zeros from `end` on), by THREADS threads, as fp32 into dst, pitch D + 4
template <typename T, int D, int THREADS>
__device__ __forceinline__ void stage_rows(float* dst, const T* x, int64_t stride, bool vec, int first, int end) {
  constexpr int kPieces = D / 8;
  for (int i = threadIdx.x; i < kMmaRows * kPieces; i += THREADS) {
    const int r = i / kPieces, c = i % kPieces * 8;
    float v[8];
    if (first + r < end) {
      const T* row = x + (first + r) * stride;
      if (vec) unpack8(load8<true, false>(row, Pieces{c, c + 4}), v);
      else unpack8(load8<false, false>(row, Pieces{c, c + 4}), v);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = 0.f;
    }
    float4* o = reinterpret_cast<float4*>(dst + r * (D + 4) + c);
    o[0] = make_float4(v[0], v[1], v[2], v[3]);
    o[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// NP = 2: x = hi + lo; NP = 1: x alone (exact in tf32, or rounded to it)
template <int NP>
__device__ __forceinline__ void split(float x, uint32_t (&out)[NP]) {
  if (NP == 1) {
    out[0] = __float_as_uint(x);
  } else {
    out[0] = (__float_as_uint(x) + 0x1000u) & 0xFFFFE000u;  // to nearest; cvt to tf32 has a quarter of the rate
    out[NP - 1] = __float_as_uint(x - __uint_as_float(out[0]));  // its lowest bits are ignored
  }
}
template <int NP>
__device__ __forceinline__ void product(float (&d)[4], const uint32_t (&a)[NP][4], const uint32_t (&b)[NP][2]) {
  tc::mma_tf32_16x8x8(d, a[0], b[0]);
  if (NP == 2) {
    tc::mma_tf32_16x8x8(d, a[0], b[NP - 1]);
    tc::mma_tf32_16x8x8(d, a[NP - 1], b[0]);
  }
}

}  // namespace falcon
