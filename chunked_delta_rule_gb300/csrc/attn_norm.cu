// Per-head norm of queries and keys with the rotary positions in the same
// pass, and the rotary table.
//
//   y = x / sqrt(mean(x^2) + eps) * w,  (a, b) -> (a c - b s, b c + a s)
//
// Memory bound: each row is read and written once (2 d elements), the table
// row of a token once per warp.  d / 8 neighbouring lanes hold a head row (8
// elements a lane, so a bf16 row is one 16-byte access a lane), the sum of
// squares is a shuffle over them, and with the half layout the partner
// elements come from another lane by shuffle.  A warp keeps one token's
// angles and weights in registers and takes several of its heads, all loads
// first.

#include "attn.cuh"

namespace falcon {
namespace {

__global__ void rope_table_kernel(const double* __restrict__ f, int half, int64_t n, float m, float2* out) {
  const int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
  if (i >= n) return;
  double s, c;
  sincos(static_cast<double>(i / half) * f[i % half], &s, &c);
  out[i] = make_float2(static_cast<float>(c * static_cast<double>(m)), static_cast<float>(s * static_cast<double>(m)));
}

// rows of one token that a warp takes: kBatch passes of 256 / d rows
constexpr int kBatch = 4;

template <typename T, bool VEC>
__global__ void __launch_bounds__(256) qk_norm_rope_kernel(HeadArgs h, int64_t tokens, int Hq, int Hkv, int wq_warps,
                                                           int wk_warps, RowsIn q, RowsIn k,
                                                           const float* __restrict__ w_q,
                                                           const float* __restrict__ w_k,
                                                           const int64_t* __restrict__ pos, RowsOut qo, RowsOut ko) {
  const int lane = threadIdx.x & 31;
  const int64_t warp = blockIdx.x * static_cast<int64_t>(blockDim.x >> 5) + (threadIdx.x >> 5);
  const int per = wq_warps + wk_warps;
  const int64_t tok = warp / per;
  if (tok >= tokens) return;
  const int part = static_cast<int>(warp - tok * per);
  const bool is_q = part < wq_warps;
  const int H = is_q ? Hq : Hkv;
  const RowsIn in = is_q ? q : k;
  const RowsOut out = is_q ? qo : ko;
  const float* w = is_q ? w_q : w_k;
  const int L = h.d >> 3, rows = 32 / L;  // lanes of a row, rows of a pass
  const int c0 = (lane % L) * 8;
  const int first = (is_q ? part : part - wq_warps) * (kBatch * rows) + lane / L;
  const T* src = static_cast<const T*>(in.p) + tok * in.stride + c0;
  T* dst = static_cast<T*>(out.p) + tok * out.stride + c0;

  Raw8<T> raw[kBatch];
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    const int hh = first + u * rows;
    if (hh < H) raw[u] = load8<VEC>(src + hh * h.d);
  }
  HeadPiece hp;
  load_weights(hp, h, w, c0);
  load_angles(hp, h, h.rot ? pos[tok] : 0, c0);
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    const int hh = first + u * rows;
    const bool live = hh < H;
    float x[8];
    if (live) {
      unpack8(raw[u], x);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = 0.f;
    }
    norm_rotate8<T>(x, hp, h, w, src - c0 + hh * h.d, live, c0, lane);
    if (live) store8<VEC>(dst + hh * h.d, x);
  }
}

}  // namespace

int launch_rope_table(const double* inv_freq, int rot, int rows, float mscale, float* table, cudaStream_t s) {
  const int64_t n = static_cast<int64_t>(rows) * (rot / 2);
  if (n == 0) return FALCON_OK;
  if ((n + 255) / 256 > INT32_MAX) return FALCON_ERR_UNSUPPORTED;
  rope_table_kernel<<<static_cast<unsigned>((n + 255) / 256), 256, 0, s>>>(inv_freq, rot / 2, n, mscale,
                                                                            reinterpret_cast<float2*>(table));
  return cudaGetLastError() == cudaSuccess ? FALCON_OK : FALCON_ERR_CUDA;
}

template <typename T>
static int launch_norm(const HeadArgs& h, int64_t tokens, int Hq, int Hkv, RowsIn q, RowsIn k, const float* w_q,
                       const float* w_k, const int64_t* pos, RowsOut qo, RowsOut ko, cudaStream_t s) {
  const int per = kBatch * (256 / h.d);
  const int wq = q.p ? (Hq + per - 1) / per : 0, wk = k.p ? (Hkv + per - 1) / per : 0;
  if (tokens == 0 || wq + wk == 0) return FALCON_OK;
  const bool vec = (!q.p || (q.vec && qo.vec)) && (!k.p || (k.vec && ko.vec));
  const int64_t blocks = (tokens * (wq + wk) + 7) / 8;
  if (blocks > INT32_MAX) return FALCON_ERR_UNSUPPORTED;
  const unsigned g = static_cast<unsigned>(blocks);
  if (vec)
    qk_norm_rope_kernel<T, true><<<g, 256, 0, s>>>(h, tokens, Hq, Hkv, wq, wk, q, k, w_q, w_k, pos, qo, ko);
  else
    qk_norm_rope_kernel<T, false><<<g, 256, 0, s>>>(h, tokens, Hq, Hkv, wq, wk, q, k, w_q, w_k, pos, qo, ko);
  return cudaGetLastError() == cudaSuccess ? FALCON_OK : FALCON_ERR_CUDA;
}

int launch_qk_norm_rope(const HeadArgs& h, int dtype, int64_t tokens, int Hq, int Hkv, RowsIn q, RowsIn k,
                        const float* w_q, const float* w_k, const int64_t* pos, RowsOut qo, RowsOut ko,
                        cudaStream_t s) {
  return dtype == FALCON_BF16 ? launch_norm<__nv_bfloat16>(h, tokens, Hq, Hkv, q, k, w_q, w_k, pos, qo, ko, s)
                              : launch_norm<float>(h, tokens, Hq, Hkv, q, k, w_q, w_k, pos, qo, ko, s);
}

}  // namespace falcon
