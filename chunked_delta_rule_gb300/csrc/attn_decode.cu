// Attention of one token per sequence over the paged 8-bit cache.
//
//   s_j = scale q . (2^ek Kc_j),  o = sum_j exp(s_j) 2^ev Vc_j / sum_j exp(s_j)
//
// One warp per (sequence, query head); lane t holds dims t, t + 32, ...; the
// running maximum and sum of the softmax in fp32.

#include "attn.cuh"

namespace falcon {
namespace {

__device__ __forceinline__ float code_value(uint8_t c) {
  const uint32_t h = e4m3x2_to_half2(c);
  return __half2float(*reinterpret_cast<const __half*>(&h));
}

template <typename T>
__global__ void __launch_bounds__(128) attn_decode_kernel(DecodeArgs a, int64_t items) {
  const int lane = threadIdx.x & 31;
  const int64_t it = blockIdx.x * static_cast<int64_t>(blockDim.x >> 5) + (threadIdx.x >> 5);
  if (it >= items) return;
  const int h = static_cast<int>(it % a.Hq), hk = h / (a.Hq / a.Hkv);
  const int64_t b = it / a.Hq;
  const int64_t cap = min(static_cast<int64_t>(a.max_k), static_cast<int64_t>(a.max_pages) * a.page);
  const int len = static_cast<int>(min(static_cast<int64_t>(a.lens[b]), cap));
  const T* q = static_cast<const T*>(a.q.p) + b * a.q.stride + h * a.d;
  float qv[4], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) qv[i] = lane + 32 * i < a.d ? to_f32(q[lane + 32 * i]) * a.scale : 0.f;
  for (int t = 0; t < len; ++t) {
    const int pg = a.blocks[b * a.max_pages + t / a.page];
    if (pg < 0 || pg >= a.num_pages) continue;
    const int64_t ph = static_cast<int64_t>(pg) * a.Hkv + hk;
    const int64_t at = (ph * a.page + t % a.page) * a.d;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (lane + 32 * i < a.d) s = fmaf(qv[i], code_value(a.cache.k[at + lane + 32 * i]), s);
#pragma unroll
    for (int k = 16; k; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    s *= e8m0(a.cache.k_scale[ph]);
    const float mn = fmaxf(m, s), ref = mn == -INFINITY ? 0.f : mn;
    const float old = expf(m - ref), p = expf(s - ref);
    l = l * old + p;
    const float pv = p * e8m0(a.cache.v_scale[ph]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (lane + 32 * i < a.d) o[i] = o[i] * old + pv * code_value(a.cache.v[at + lane + 32 * i]);
    m = mn;
  }
  T* out = static_cast<T*>(a.o.p) + b * a.o.stride + h * a.d;
  const bool none = l == 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (lane + 32 * i < a.d) out[lane + 32 * i] = from_f32<T>(none ? 0.f : o[i] / l);
  if (a.lse && lane == 0) a.lse[b * a.Hq + h] = none ? -INFINITY : m + logf(l);
}

}  // namespace

size_t attn_decode_ws_bytes(int, int, int, int, int, int) { return 256; }

int launch_attn_decode(const DecodeArgs& a, int dtype, cudaStream_t s) {
  const int64_t items = static_cast<int64_t>(a.B) * a.Hq, blocks = (items + 3) / 4;
  if (blocks > INT32_MAX) return FALCON_ERR_UNSUPPORTED;
  if (dtype == FALCON_BF16)
    attn_decode_kernel<__nv_bfloat16><<<static_cast<unsigned>(blocks), 128, 0, s>>>(a, items);
  else
    attn_decode_kernel<float><<<static_cast<unsigned>(blocks), 128, 0, s>>>(a, items);
  return cudaGetLastError() == cudaSuccess ? FALCON_OK : FALCON_ERR_CUDA;
}

}  // namespace falcon
