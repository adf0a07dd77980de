// What the kernels of prompt attention share: the grid, and one row by one warp,
// straight from the definition, touching only the keys that the row sees.
#pragma once

#include "attn.cuh"

namespace falcon {

// The grid of a prompt call, blocks of `rows` queries for every query head.  Each sequence gets the blocks of max_q rows,
// the longest first over the batch; or, where that bound leaves more than half of them without rows, sequence b gets the
// blocks from cu_q[b] / rows + b on, whose number the tokens bound (256 x 128 tokens, 12 heads of 64, bf16, a bound of
// 32768 rows: 1747 us the first way, 57 the second, 43 with the exact bound; 16 x 1024: 96, 50 and 45).
struct PromptGrid {
  int64_t blocks;  // of a head
  bool packed;
};
inline PromptGrid prompt_grid(const PromptArgs& a, int rows) {
  const int64_t each = (static_cast<int64_t>(a.max_q) + rows - 1) / rows * a.B, packed = a.tokens / rows + a.B;
  return each > 2 * packed ? PromptGrid{packed, true} : PromptGrid{each, false};
}
// Block j of a packed grid: its sequence (the last one that begins no later) and its first row there, its sequence's
// last rows first; below 0 or past the sequence where the block has none.
__device__ __forceinline__ int2 packed_block(const int32_t* cu, int B, int rows, int j) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (static_cast<int64_t>(__ldg(cu + mid)) / rows + mid <= j) lo = mid;
    else hi = mid;
  }
  const int64_t first = static_cast<int64_t>(__ldg(cu + lo)) / rows + lo;
  const int64_t next = static_cast<int64_t>(__ldg(cu + lo + 1)) / rows + lo + 1;
  const int64_t row = (next - 1 - j) * rows;
  return make_int2(lo, j < first || row > INT32_MAX ? -1 : static_cast<int>(row));
}

// out (lane t's dims t, t + 32, ...) and the log of the sum of exponentials of
// the first n keys; out = 0 and -inf where nothing weighs.  A few keys at a time:
// all their loads are in flight before the first is used, and their sums over
// the lanes run side by side (0.15 us a key, 0.5 one by one).  Ends where the sum is
// NaN: it and every dim stay so.
template <typename T, int D>
__device__ __noinline__ void attention_row(const T* q, const T* k, int64_t k_stride, const T* v, int64_t v_stride,
                                           int n, int d, float scale, float (&out)[4], float* lse) {
  constexpr int J = (D + 31) / 32, kBatch = J == 4 ? 4 : 8;
  const int lane = threadIdx.x & 31;
  float qv[J], o[J], m = -INFINITY, l = 0.f;
  int at[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    at[j] = min(lane + 32 * j, d - 1);
    qv[j] = lane + 32 * j < d ? to_f32(q[at[j]]) * scale : 0.f;
    o[j] = 0.f;
  }
  for (int t = 0; t < n && l == l; t += kBatch) {
    T kt[kBatch][J], vt[kBatch][J];
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
#pragma unroll
      for (int j = 0; j < J; ++j) kt[u][j] = k[min(t + u, n - 1) * k_stride + at[j]];
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
#pragma unroll
      for (int j = 0; j < J; ++j) vt[u][j] = v[min(t + u, n - 1) * v_stride + at[j]];
    float s[kBatch], top = m;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      s[u] = 0.f;
#pragma unroll
      for (int j = 0; j < J; ++j) s[u] = fmaf(qv[j], lane + 32 * j < d ? to_f32(kt[u][j]) : 0.f, s[u]);
    }
#pragma unroll
    for (int x = 16; x; x >>= 1)
#pragma unroll
      for (int u = 0; u < kBatch; ++u) s[u] += __shfl_xor_sync(0xffffffffu, s[u], x);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) top = fmaxf(top, s[u]);  // (the last key's score again past the end)
    const float ref = top == -INFINITY ? 0.f : top, old = expf(m - ref);
    l *= old;
#pragma unroll
    for (int j = 0; j < J; ++j) o[j] *= old;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const bool in = t + u < n;
      const float p = in ? expf(s[u] - ref) : 0.f;
      l += p;
#pragma unroll
      for (int j = 0; j < J; ++j) o[j] = fmaf(p, in ? to_f32(vt[u][j]) : 0.f, o[j]);
    }
    m = top;
  }
#pragma unroll
  for (int j = 0; j < J; ++j) out[j] = l == 0.f ? 0.f : o[j] / l;
  *lse = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace falcon
