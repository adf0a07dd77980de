// One row of causal attention by one warp, straight from the definition: only
// the keys that the row sees are touched.
#pragma once

#include "attn.cuh"

namespace falcon {

// o (lane t's dims t, t + 32, ...) and the log of the sum of exponentials of
// the first n keys; o = 0 and -inf where nothing weighs.
template <typename T>
__device__ __noinline__ void attention_row(const T* q, const T* k, int64_t k_stride, const T* v,
                                              int64_t v_stride, int n, int d, float scale, float (&o)[4], float* lse) {
  const int lane = threadIdx.x & 31;
  float qv[4], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    qv[j] = lane + 32 * j < d ? to_f32(q[lane + 32 * j]) * scale : 0.f;
    o[j] = 0.f;
  }
  for (int t = 0; t < n; ++t) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (lane + 32 * j < d) s = fmaf(qv[j], to_f32(k[t * k_stride + lane + 32 * j]), s);
#pragma unroll
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    const float mn = fmaxf(m, s), ref = mn == -INFINITY ? 0.f : mn;
    const float old = expf(m - ref), p = expf(s - ref);
    l = l * old + p;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (lane + 32 * j < d) o[j] = o[j] * old + p * to_f32(v[t * v_stride + lane + 32 * j]);
    m = mn;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = l == 0.f ? 0.f : o[j] / l;
  *lse = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace falcon
