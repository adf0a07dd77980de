// Causal attention over packed prompts, portable form.
//
//   s_ij = scale q_i . k_j for j <= i + lk - lq,  o_i = softmax(s_i) V
//
// One warp per (query, head); lane t holds dims t, t + 32, ...; the running
// maximum and sum of the softmax in fp32.

#include "attn_row.cuh"

namespace falcon {
namespace {

template <typename T>
__global__ void __launch_bounds__(128) attn_prompt_kernel(PromptArgs a, int64_t items) {
  const int lane = threadIdx.x & 31;
  int64_t it = blockIdx.x * static_cast<int64_t>(blockDim.x >> 5) + (threadIdx.x >> 5);
  if (it >= items) return;
  const int h = static_cast<int>(it % a.Hq), hk = h / (a.Hq / a.Hkv);
  it /= a.Hq;
  const int i = static_cast<int>(it % a.max_q), b = static_cast<int>(it / a.max_q);
  const int64_t q0 = a.cu_q[b], k0 = a.cu_k[b];
  const int lq = static_cast<int>(a.cu_q[b + 1] - q0);
  const int lk = static_cast<int>(a.cu_k[b + 1] - k0);
  if (i >= lq || q0 < 0 || k0 < 0 || q0 + lq > a.tokens || k0 + lk > a.k_tokens) return;
  const int n = i + lk - lq + 1;  // keys that the query sees
  const T* q = static_cast<const T*>(a.q.p) + (q0 + i) * a.q.stride + h * a.d;
  const T* k = static_cast<const T*>(a.k.p) + k0 * a.k.stride + hk * a.d;
  const T* v = static_cast<const T*>(a.v.p) + k0 * a.v.stride + hk * a.d;
  float o[4], lse;
  attention_row(q, k, a.k.stride, v, a.v.stride, n, a.d, a.scale, o, &lse);
  T* out = static_cast<T*>(a.o.p) + (q0 + i) * a.o.stride + h * a.d;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (lane + 32 * j < a.d) out[lane + 32 * j] = from_f32<T>(o[j]);
  if (a.lse && lane == 0) a.lse[(q0 + i) * a.Hq + h] = lse;
}

}  // namespace

int launch_attn_prompt(const PromptArgs& a, int dtype, cudaStream_t s) {
  if (a.max_q == 0 || a.tokens == 0) return FALCON_OK;
  if (attn_prompt_tc_supported(a, dtype)) return launch_attn_prompt_tc(a, s);
  const int64_t items = static_cast<int64_t>(a.B) * a.max_q * a.Hq, blocks = (items + 3) / 4;
  if (blocks > INT32_MAX) return FALCON_ERR_UNSUPPORTED;
  if (dtype == FALCON_BF16)
    attn_prompt_kernel<__nv_bfloat16><<<static_cast<unsigned>(blocks), 128, 0, s>>>(a, items);
  else
    attn_prompt_kernel<float><<<static_cast<unsigned>(blocks), 128, 0, s>>>(a, items);
  return cudaGetLastError() == cudaSuccess ? FALCON_OK : FALCON_ERR_CUDA;
}

}  // namespace falcon
