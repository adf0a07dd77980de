// Causal attention over packed prompts where the tcgen05 kernel does not go:
// fp32, rows off the 16-byte boundaries, a few short prompts.
//
//   S = Q K^T,  P = exp(scale S - m),  O += P V
//
// Warp-level tf32 MMAs (m16n8k8) with fp32 sums.  An fp32 operand is split into
// two tf32 parts, hi rounded and lo the rest, and a product taken as hi hi +
// hi lo + lo hi: about 2^-21 of it is lost at most.  The tensor cores cut their
// sums off instead of rounding them, which adds up over many steps: for fp32 the
// small products of S have sums of their own, and so has P V of every tile (at
// 2000 keys, d = 64 an error of 5.5e-7; 4.2e-6 without).  bf16 inputs are exact in
// tf32; their weights are rounded to 11 bits.  A CTA takes 64 queries of one
// head, 16 rows a warp; K and V tiles of 64 keys lie in shared memory as fp32,
// rows padded by 4 words so that no fragment load has a bank conflict.  The
// weights go from one product's result to the next one's operand in registers:
// key 2c of a group of 8 takes the place of column c, key 2c + 1 that of c + 4.
//
// Bound by the chain of a row block: products of three parts, the splits, the
// softmax, tile after tile.  Measured: 7 prompts of <= 333, 12 / 4 heads of 64,
// fp32: 37 us with the call; 8 x 1024 x 12 x 64, fp32: 261 us (the sums apart cost some
// 40 of them).
//
// Keys that no row of the tile sees are not touched, tile rows past the last key
// are zeros.  A row whose result is not finite (a masked key of its own
// sequence may hold an infinity) is computed again from the definition.

#include "attn_mma.cuh"
#include "attn_row.cuh"

namespace falcon {
namespace {

constexpr int kRows = kMmaRows, kKeys = kMmaRows;

template <typename T, int D>
__global__ void __launch_bounds__(128) attn_prompt_kernel(PromptArgs a, int qblocks, bool packed) {
  constexpr int NP = sizeof(T) == 4 ? 2 : 1, LD = D + 4, NT = kKeys / 8;
  extern __shared__ float smem[];
  float *sq = smem, *sk = sq + kRows * LD, *sv = sk + kKeys * LD;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, tig = lane & 3;
  if (blockIdx.x == 0 && threadIdx.x == 0) *static_cast<uint32_t*>(a.ws) = 0;  // the status: no wait here can run out
  int b, h, row0;
  if (packed) {
    const int2 x = packed_block(a.cu_q, a.B, kRows, static_cast<int>(blockIdx.x / a.Hq));
    b = x.x, row0 = x.y, h = static_cast<int>(blockIdx.x % a.Hq);
  } else {
    const uint32_t bh = static_cast<uint32_t>(a.B) * a.Hq, at = blockIdx.x % bh;
    b = static_cast<int>(at) / a.Hq, h = static_cast<int>(at) % a.Hq;
    row0 = (qblocks - 1 - static_cast<int>(blockIdx.x / bh)) * kRows;  // the longest rows first
  }
  const int hk = h / (a.Hq / a.Hkv);
  const int64_t q0 = a.cu_q[b], k0 = a.cu_k[b];
  const int lq_all = static_cast<int>(a.cu_q[b + 1] - q0), lk = static_cast<int>(a.cu_k[b + 1] - k0);
  const int lq = min(lq_all, a.max_q), off = lk - lq_all;
  if (row0 < 0 || row0 >= lq || q0 < 0 || k0 < 0 || q0 + lq_all > a.tokens || k0 + lk > a.k_tokens) return;
  const T* q = static_cast<const T*>(a.q.p) + q0 * a.q.stride + static_cast<int64_t>(h) * D;
  const T* k = static_cast<const T*>(a.k.p) + k0 * a.k.stride + static_cast<int64_t>(hk) * D;
  const T* v = static_cast<const T*>(a.v.p) + k0 * a.v.stride + static_cast<int64_t>(hk) * D;
  stage_rows<T, D, 128>(sq, q, a.q.stride, a.q.vec, row0, lq);

  float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
  const float sl2 = a.scale * kLog2e;
  const int r0 = warp * 16 + gid;  // this thread's rows: r0 and r0 + 8 of the block
  const int keys = min(min(row0 + kRows, lq) + off, lk);  // that some row of the block sees
  for (int j0 = 0; j0 < keys; j0 += kKeys) {
    __syncthreads();
    stage_rows<T, D, 128>(sk, k, a.k.stride, a.k.vec, j0, lk);
    stage_rows<T, D, 128>(sv, v, a.v.stride, a.v.vec, j0, lk);
    __syncthreads();
    float s[NT][4], low[NT][4];  // fp32: the small products apart
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[t][e] = low[t][e] = 0.f;
#pragma unroll 2
    for (int ks = 0; ks < D / 8; ++ks) {
      uint32_t af[NP][4];
      const float* qa = sq + r0 * LD + ks * 8 + tig;
      const float av[4] = {qa[0], qa[8 * LD], qa[4], qa[8 * LD + 4]};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t w[NP];
        split<NP>(av[e], w);
#pragma unroll
        for (int p = 0; p < NP; ++p) af[p][e] = w[p];
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float* kb = sk + (t * 8 + gid) * LD + ks * 8 + tig;
        uint32_t bf[NP][2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t w[NP];
          split<NP>(kb[4 * e], w);
#pragma unroll
          for (int p = 0; p < NP; ++p) bf[p][e] = w[p];
        }
        tc::mma_tf32_16x8x8(s[t], af[0], bf[0]);
        if (NP == 2) {
          tc::mma_tf32_16x8x8(low[t], af[0], bf[NP - 1]);
          tc::mma_tf32_16x8x8(low[t], af[NP - 1], bf[0]);
        }
      }
    }
    if (NP == 2) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[t][e] += low[t][e];
    }
    // columns 2 tig and 2 tig + 1 of each group of 8 keys
    const int lim0 = min(row0 + r0 + off + 1, lk) - j0, lim1 = min(row0 + r0 + 8 + off + 1, lk) - j0;
    if (j0 + kKeys > min(row0 + off + 1, lk)) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int c = t * 8 + 2 * tig + e;
          if (c >= lim0) s[t][e] = -INFINITY;
          if (c >= lim1) s[t][2 + e] = -INFINITY;
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float top = -INFINITY;
#pragma unroll
      for (int t = 0; t < NT; ++t) top = fmaxf(top, fmaxf(s[t][2 * i], s[t][2 * i + 1]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      top = fmaxf(top, m[i]);
      const float f = top == -INFINITY ? 1.f : ex2((m[i] - top) * sl2), ref = top == -INFINITY ? 0.f : top;
      m[i] = top;
      float sum = 0.f;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // the difference first: it is exact near the maximum, which fp32 results need
          const float p = ex2((s[t][2 * i + e] - ref) * sl2);
          s[t][2 * i + e] = p;
          sum += p;
        }
      l[i] = l[i] * f + sum;
#pragma unroll
      for (int t = 0; t < D / 8; ++t) o[t][2 * i] *= f, o[t][2 * i + 1] *= f;
    }
    // fp32: a tile's products in sums of their own
    float part[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) part[i][e] = 0.f;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      uint32_t pf[NP][4];
      const float pv[4] = {s[t][0], s[t][2], s[t][1], s[t][3]};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t w[NP];
        split<NP>(NP == 1 ? __uint_as_float(tc::to_tf32(pv[e])) : pv[e], w);
#pragma unroll
        for (int p = 0; p < NP; ++p) pf[p][e] = w[p];
      }
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const float* vb = sv + (t * 8 + 2 * tig) * LD + i * 8 + gid;
        uint32_t bf[NP][2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t w[NP];
          split<NP>(vb[e * LD], w);
#pragma unroll
          for (int p = 0; p < NP; ++p) bf[p][e] = w[p];
        }
        product<NP>(NP == 2 ? part[i] : o[i], pf, bf);
      }
    }
    if (NP == 2) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] += part[i][e];
    }
  }

  bool bad[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float sum = l[i];
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    const int row = row0 + r0 + 8 * i;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    bad[i] = !(sum <= 3.402823466e38f);
    T* out = static_cast<T*>(a.o.p) + (q0 + row) * a.o.stride + static_cast<int64_t>(h) * D + 2 * tig;
#pragma unroll
    for (int t = 0; t < D / 8; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float x = o[t][2 * i + e];
        bad[i] |= !(fabsf(x) <= 3.402823466e38f);
        if (row < lq) out[t * 8 + e] = from_f32<T>(sum == 0.f ? 0.f : x * inv);
      }
    if (a.lse && row < lq && tig == 0)
      a.lse[(q0 + row) * a.Hq + h] = sum == 0.f ? -INFINITY : m[i] * a.scale + logf(sum);
    bad[i] = bad[i] && row < lq;
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 2; ++i)
    for (uint32_t again = __ballot_sync(0xffffffffu, bad[i]); again;) {
      const int g = (__ffs(again) - 1) >> 2, row = row0 + warp * 16 + g + 8 * i;
      again &= ~(0xFu << (4 * g));
      float y[4], z;
      attention_row<T, D>(q + row * a.q.stride, k, a.k.stride, v, a.v.stride, min(row + off + 1, lk), D, a.scale, y, &z);
      T* out = static_cast<T*>(a.o.p) + (q0 + row) * a.o.stride + static_cast<int64_t>(h) * D;
#pragma unroll
      for (int e = 0; e < (D + 31) / 32; ++e)
        if (lane + 32 * e < D) out[lane + 32 * e] = from_f32<T>(y[e]);
      if (a.lse && lane == 0) a.lse[(q0 + row) * a.Hq + h] = z;
    }
}

template <typename T, int D>
int launch(const PromptArgs& a, cudaStream_t s) {
  const PromptGrid g = prompt_grid(a, kRows);
  if (g.blocks < 1 || g.blocks > INT32_MAX / a.Hq) return FALCON_ERR_UNSUPPORTED;
  const int64_t n = g.blocks * a.Hq;
  constexpr size_t smem = static_cast<size_t>(kRows + 2 * kKeys) * (D + 4) * 4;
  const auto kern = attn_prompt_kernel<T, D>;
  if (!set_smem_limit(reinterpret_cast<const void*>(kern), smem)) return FALCON_ERR_CUDA;
  kern<<<static_cast<unsigned>(n), 128, smem, s>>>(a, static_cast<int>(g.blocks / a.B), g.packed);
  return cudaGetLastError() == cudaSuccess ? FALCON_OK : FALCON_ERR_CUDA;
}
template <typename T>
int launch_d(const PromptArgs& a, cudaStream_t s) {
  switch (a.d) {
    case 16: return launch<T, 16>(a, s);
    case 32: return launch<T, 32>(a, s);
    case 64: return launch<T, 64>(a, s);
    default: return launch<T, 128>(a, s);
  }
}

}  // namespace

int launch_attn_prompt(const PromptArgs& a, int dtype, cudaStream_t s) {
  if (a.max_q == 0 || a.tokens == 0) return FALCON_OK;
  if (attn_prompt_tc_supported(a, dtype)) return launch_attn_prompt_tc(a, s);
  return dtype == FALCON_BF16 ? launch_d<__nv_bfloat16>(a, s) : launch_d<float>(a, s);
}

}  // namespace falcon
