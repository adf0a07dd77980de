// Per-head norm of queries and keys with the rotary positions in the same
// pass, and the rotary table.
//
//   y = x / sqrt(mean(x^2) + eps) * w,  (a, b) -> (a c - b s, b c + a s)
//
// Memory bound: each row is read and written once (2 d elements), the table
// row of a token once per warp.  d / 8 neighbouring lanes hold a head row, 8
// elements a lane: one 16-byte access, or with the half layout two of 8, so
// that a lane holds both members of its pairs.  The sum of squares is a
// shuffle over the row's lanes.  A warp keeps one token's angles and weights in
// registers and takes its heads, two passes' loads at a time (with four, 80
// registers leave too few warps: 84 us for the case below).
// 32768 tokens x (16 + 4) heads of 128, bf16: 344 MB in 74 us, 4.7 TB/s;
// 9984 x (12 + 4) of 64, fp32: 82 MB in 18.5 us with the launch.

#include "attn.cuh"
#include "tc_util.cuh"

namespace falcon {
namespace {

__global__ void rope_table_kernel(const double* __restrict__ f, int half, int64_t n, float m, float2* out) {
  const int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
  if (i >= n) return;
  double s, c;
  sincos(static_cast<double>(i / half) * f[i % half], &s, &c);
  out[i] = make_float2(static_cast<float>(c * static_cast<double>(m)), static_cast<float>(s * static_cast<double>(m)));
}

// A warp takes passes of 256 / d rows of one token, its query rows first and
// then its key rows, kBatch passes at a time.
constexpr int kBatch = 2;

template <typename T, bool VEC, int MODE>
__global__ void __launch_bounds__(256, 4) qk_norm_rope_kernel(HeadArgs h, int64_t tokens, int Hq, int Hkv, int passes,
                                                           RowsIn q, RowsIn k, const float* __restrict__ w_q,
                                                           const float* __restrict__ w_k,
                                                           const int64_t* __restrict__ pos, RowsOut qo, RowsOut ko) {
  const int lane = threadIdx.x & 31;
  const int64_t tok = blockIdx.x * static_cast<int64_t>(8) + (threadIdx.x >> 5);
  if (tok >= tokens) return;
  const int ls = 28 - __clz(h.d), rows = 32 >> ls;  // log2 of the lanes of a row, rows of a pass
  const Pieces at = pieces_of<MODE>(h, lane & ((1 << ls) - 1));
  constexpr bool kSplit = MODE == kRotHalf;
  const int first = static_cast<int>(blockIdx.y) * passes * rows + (lane >> ls), end = min(static_cast<int>(blockIdx.y + 1) * passes * rows, Hq + Hkv);
  const T* src_q = static_cast<const T*>(q.p) + tok * q.stride;
  const T* src_k = static_cast<const T*>(k.p) + tok * k.stride;
  auto source = [&](int r) { return r < Hq ? src_q + r * h.d : src_k + (r - Hq) * h.d; };

  HeadPiece hp;
  bool of_q = first < Hq;  // whose weights hp holds
  const float2* row = nullptr;
  for (int p = 0; p < passes; p += kBatch) {
    Raw8<T> raw[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int r = first + (p + u) * rows;
      if (r < end) raw[u] = load8<VEC, kSplit>(source(r), at);
    }
    if (p == 0) {
      if (MODE != kRotNone && h.rot) row = table_row(h, pos[tok]);
      load_angles<MODE>(hp, h, row, at);
      load_weights(hp, h, of_q ? w_q : w_k, at);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int r = first + (p + u) * rows;
      const bool live = r < end;
      if (live && of_q && r >= Hq) {
        of_q = false;
        load_weights(hp, h, w_k, at);
      }
      float x[8];
      if (live) {
        unpack8(raw[u], x);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 0.f;
      }
      norm_rotate8<MODE, T>(x, hp, h, of_q ? w_q : w_k, row, live ? source(r) : nullptr, live, at);
      if (live) {
        T* dst = r < Hq ? static_cast<T*>(qo.p) + tok * qo.stride + r * h.d
                        : static_cast<T*>(ko.p) + tok * ko.stride + (r - Hq) * h.d;
        store8<VEC, kSplit>(dst, at, x);
      }
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
  // a warp a token where that gives every SM 32 of them (32768 tokens x 20 heads of 128: 74 us, with three warps a token
  // 88), else a warp for every kBatch passes
  const int all = (Hq + Hkv + 256 / h.d - 1) / (256 / h.d);
  const int parts = tokens >= int64_t(32) * tcu::sm_count() ? 1 : (all + kBatch - 1) / kBatch;
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
