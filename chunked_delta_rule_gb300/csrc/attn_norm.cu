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

// A warp takes up to kBatch passes of 256 / d rows of one token, its query
// rows first and then its key rows.
constexpr int kBatch = 4;

template <typename T, bool VEC, int MODE>
__global__ void __launch_bounds__(256) qk_norm_rope_kernel(HeadArgs h, int64_t tokens, int Hq, int Hkv, int passes,
                                                           RowsIn q, RowsIn k, const float* __restrict__ w_q,
                                                           const float* __restrict__ w_k,
                                                           const int64_t* __restrict__ pos, RowsOut qo, RowsOut ko) {
  const int lane = threadIdx.x & 31;
  const int64_t tok = blockIdx.x * static_cast<int64_t>(8) + (threadIdx.x >> 5);
  if (tok >= tokens) return;
  const int ls = 28 - __clz(h.d), rows = 32 >> ls;  // log2 of the lanes of a row, rows of a pass
  const int c0 = (lane & ((1 << ls) - 1)) * 8;
  const int first = static_cast<int>(blockIdx.y) * passes * rows + (lane >> ls), end = min(static_cast<int>(blockIdx.y + 1) * passes * rows, Hq + Hkv);
  const T* src_q = static_cast<const T*>(q.p) + tok * q.stride;
  const T* src_k = static_cast<const T*>(k.p) + tok * k.stride;
  auto source = [&](int r) { return r < Hq ? src_q + r * h.d : src_k + (r - Hq) * h.d; };

  Raw8<T> raw[kBatch];
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    const int r = first + u * rows;
    if (r < end) raw[u] = load8<VEC>(source(r) + c0);
  }
  HeadPiece hp;
  load_angles<MODE>(hp, h, MODE != kRotNone && h.rot ? pos[tok] : 0, c0);
  load_weights(hp, h, first < Hq ? w_q : w_k, c0);
  bool of_q = first < Hq;  // whose weights hp holds
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    const int r = first + u * rows;
    const bool live = r < end;
    if (live && of_q && r >= Hq) {
      of_q = false;
      load_weights(hp, h, w_k, c0);
    }
    float x[8];
    if (live) {
      unpack8(raw[u], x);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = 0.f;
    }
    norm_rotate8<MODE, T>(x, hp, h, of_q ? w_q : w_k, live ? source(r) : nullptr, live, c0, lane);
    if (live) {
      T* dst = r < Hq ? static_cast<T*>(qo.p) + tok * qo.stride + r * h.d
                      : static_cast<T*>(ko.p) + tok * ko.stride + (r - Hq) * h.d;
      store8<VEC>(dst + c0, x);
    }
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
  if (!q.p) Hq = 0;
  if (!k.p) Hkv = 0;
  if (tokens == 0 || Hq + Hkv == 0) return FALCON_OK;
  const bool vec = (!q.p || (q.vec && qo.vec)) && (!k.p || (k.vec && ko.vec));
  const int all = (Hq + Hkv + 256 / h.d - 1) / (256 / h.d), parts = (all + kBatch - 1) / kBatch;
  const int64_t blocks = (tokens + 7) / 8;
  if (blocks > INT32_MAX || parts > 65535) return FALCON_ERR_UNSUPPORTED;
  const dim3 g(static_cast<unsigned>(blocks), static_cast<unsigned>(parts));
  const int passes = (all + parts - 1) / parts;
  const RotMode mode = vec ? rot_mode(h) : kRotAny;
  const auto kern = mode == kRotNone ? qk_norm_rope_kernel<T, true, kRotNone>
                    : mode == kRotHalf ? qk_norm_rope_kernel<T, true, kRotHalf>
                    : mode == kRotInterleaved ? qk_norm_rope_kernel<T, true, kRotInterleaved>
                                              : qk_norm_rope_kernel<T, false, kRotAny>;
  kern<<<g, 256, 0, s>>>(h, tokens, Hq, Hkv, passes, q, k, w_q, w_k, pos, qo, ko);
  return cudaGetLastError() == cudaSuccess ? FALCON_OK : FALCON_ERR_CUDA;
}

int launch_qk_norm_rope(const HeadArgs& h, int dtype, int64_t tokens, int Hq, int Hkv, RowsIn q, RowsIn k,
                        const float* w_q, const float* w_k, const int64_t* pos, RowsOut qo, RowsOut ko,
                        cudaStream_t s) {
  return dtype == FALCON_BF16 ? launch_norm<__nv_bfloat16>(h, tokens, Hq, Hkv, q, k, w_q, w_k, pos, qo, ko, s)
                              : launch_norm<float>(h, tokens, Hq, Hkv, q, k, w_q, w_k, pos, qo, ko, s);
}

}  // namespace falcon
