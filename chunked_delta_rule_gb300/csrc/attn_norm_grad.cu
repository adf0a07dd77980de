// Gradient of the per-head norm and the rotary positions.
//
//   n = dy rotated back, r = 1 / sqrt(mean(x^2) + eps), u = n w
//   dx = r (u - x r mean(u x r)),  dw = sum over tokens and heads of n x r
//
// Memory bound: x and dy are read once, dx is written once.  Lanes, pieces and
// angles as in the forward: d / 8 neighbouring lanes hold a head row, 8 elements a lane;
// both sums of a row (x^2 and u x) go through one set of shuffles.  A warp walks
// tokens with the stride of the grid and adds its dw up in registers; the CTAs' sums
// go through the workspace to a second kernel, which adds them in one order.

#include <algorithm>

#include "attn.cuh"
#include "tc_util.cuh"

namespace falcon {
namespace {

constexpr int kWarps = 8;
constexpr int kMostCtas = 1024;  // whose sums the workspace holds

template <int MODE>
__device__ __forceinline__ void rotate_back8(float (&y)[8], const HeadPiece& hp, const HeadArgs& h, Pieces at) {
  if ((MODE != kRotHalf && MODE != kRotInterleaved) || at.a >= h.rot) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    constexpr bool kHalf = MODE == kRotHalf;
    float &p = y[kHalf ? i : 2 * i], &q = y[kHalf ? 4 + i : 2 * i + 1];
    const float a = p, b = q;
    p = a * hp.co[i] + b * hp.si[i];
    q = b * hp.co[i] - a * hp.si[i];
  }
}

// An item is a token's rows [part * passes * rows, ...): its query rows first, then its key rows.
template <typename T, bool VEC, int MODE, bool NORM>
__global__ void __launch_bounds__(32 * kWarps) qk_norm_rope_grad_kernel(NormGradArgs a, int passes, int parts) {
  const HeadArgs& h = a.h;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ls = 28 - __clz(h.d), rows = 32 >> ls;  // log2 of the lanes of a row, rows of a pass
  const Pieces at = pieces_of<MODE>(h, lane & ((1 << ls) - 1));
  constexpr bool kSplit = MODE == kRotHalf;
  const int Hq = a.H[0], all = a.H[0] + a.H[1];
  HeadPiece hp;
  float wq[8], wk[8], dwq[8], dwk[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) dwq[i] = dwk[i] = 0.f;
  if (NORM) {
    load_weights(hp, h, a.w[0], at);
#pragma unroll
    for (int i = 0; i < 8; ++i) wq[i] = hp.w[i];
    load_weights(hp, h, a.w[1], at);
#pragma unroll
    for (int i = 0; i < 8; ++i) wk[i] = hp.w[i];
  }
  const int64_t items = a.tokens * parts, step = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + warp; item < items; item += step) {
    const int64_t tok = item / parts;
    const int first = static_cast<int>(item % parts) * passes * rows, end = min(first + passes * rows, all);
    const float2* row = nullptr;
    if (MODE != kRotNone && h.rot) row = table_row(h, a.pos[tok]);
    load_angles<MODE>(hp, h, row, at);
    for (int p = 0; p < passes; ++p) {
      const int r = first + p * rows + (lane >> ls);
      const bool live = r < end, of_q = r < Hq;
      const int s = of_q ? 0 : 1, head = of_q ? r : r - Hq;
      const T* src = static_cast<const T*>(a.dy[s].p) + tok * a.dy[s].stride + head * h.d;
      float x[8], y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = y[i] = 0.f;
      if (live) {
        unpack8(load8<VEC, kSplit>(src, at), y);
        if (NORM) unpack8(load8<VEC, kSplit>(static_cast<const T*>(a.x[s].p) + tok * a.x[s].stride + head * h.d, at), x);
      }
      if constexpr (MODE == kRotAny) {
        const int half = h.rot >> 1;
        const bool hl = h.layout == FALCON_ROPE_HALF;
        float z[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = (i < 4 ? at.a : at.b - 4) + i, j = hl ? (c < half ? c : c - half) : c >> 1;  // element, its pair
          const bool low = hl ? c < half : !(c & 1);
          z[i] = y[i];
          if (live && c < h.rot) {
            const float other = to_f32(src[hl ? (low ? c + half : c - half) : c ^ 1]);
            const float2 t = row ? __ldg(row + j) : make_float2(__int_as_float(0x7fffffff), 0.f);
            z[i] = y[i] * t.x + (low ? t.y : -t.y) * other;
          }
        }
        __syncwarp();  // read before any lane writes the row in place
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = z[i];
      } else {
        rotate_back8<MODE>(y, hp, h, at);
      }
      if (NORM) {
        float s0 = 0.f, s1 = 0.f, u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          u[i] = y[i] * (of_q ? wq[i] : wk[i]);
          s0 = fmaf(x[i], x[i], s0);
          s1 = fmaf(u[i], x[i], s1);
        }
        // over the d / 8 lanes: 2, 4, 8 or 16
#pragma unroll
        for (int m = 1; m < 16; m <<= 1) {
          const float v0 = __shfl_xor_sync(0xffffffffu, s0, m), v1 = __shfl_xor_sync(0xffffffffu, s1, m);
          if (m < 1 << ls) s0 += v0, s1 += v1;
        }
        const float rs = rsqrtf(fmaf(s0, h.inv_d, h.eps));
        const float c = rs == 0.f ? 0.f : s1 * rs * h.inv_d;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float xr = x[i] * rs, n = y[i] * xr;
          if (live && of_q) dwq[i] += n;
          if (live && !of_q) dwk[i] += n;
          y[i] = rs * (u[i] - xr * c);
        }
      }
      if (live)
        store8<VEC, kSplit>(static_cast<T*>(a.dx[s].p) + tok * a.dx[s].stride + head * h.d, at, y);
    }
  }
  if (!NORM || !a.partial) return;
  // the warp's rows, then the CTA's warps
  __shared__ float sum[kWarps][2][128];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    for (int m = 16; m >= 1 << ls; m >>= 1) {
      dwq[i] += __shfl_xor_sync(0xffffffffu, dwq[i], m);
      dwk[i] += __shfl_xor_sync(0xffffffffu, dwk[i], m);
    }
    const int c = (i < 4 ? at.a : at.b - 4) + i;
    if (lane < 1 << ls) sum[warp][0][c] = dwq[i], sum[warp][1][c] = dwk[i];
  }
  __syncthreads();
  for (int t = threadIdx.x; t < 2 * h.d; t += 32 * kWarps) {
    const int s = t / h.d, c = t % h.d;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += sum[w][s][c];
    if (gridDim.x > 1) a.partial[blockIdx.x * (2 * h.d) + t] = v;
    else if (a.dw[s]) a.dw[s][c] = v;
  }
}

// dw from the sums of n CTAs (none: 0): a CTA for the queries' and one for the keys'
__global__ void __launch_bounds__(1024) norm_weight_sums_kernel(const float* partial, int n, int d, float* dw_q, float* dw_k) {
  float* dw = blockIdx.x ? dw_k : dw_q;
  if (!dw) return;
  __shared__ float sum[1024];
  const int c = threadIdx.x % d, slices = 1024 / d;
  float v = 0.f;
  for (int i = threadIdx.x / d; i < n; i += slices) v += partial[(i * 2 + blockIdx.x) * d + c];
  sum[threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.x < d) {
    v = 0.f;
    for (int i = 0; i < slices; ++i) v += sum[i * d + c];
    dw[c] = v;
  }
}

template <typename T, bool NORM>
int launch(NormGradArgs a, cudaStream_t s) {
  if (!NORM || (!a.dw[0] && !a.dw[1])) a.partial = nullptr;
  const int all = a.H[0] + a.H[1];
  int ctas = 0;
  if (a.tokens > 0) {
    bool vec = true;
    for (int i = 0; i < 2; ++i)
      if (a.H[i]) vec = vec && a.dy[i].vec && a.dx[i].vec && (!NORM || a.x[i].vec);
    const int64_t all_passes = (static_cast<int64_t>(all) * a.h.d + 255) / 256;
    const int parts = static_cast<int>(a.tokens >= int64_t(32) * tcu::sm_count() ? 1 : (all_passes + 1) / 2);
    const int passes = static_cast<int>((all_passes + parts - 1) / parts);
    const int64_t want = (a.tokens * parts + kWarps - 1) / kWarps;
    ctas = static_cast<int>(std::min<int64_t>(want, std::min(4 * tcu::sm_count(), kMostCtas)));
    const RotMode mode = vec ? rot_mode(a.h) : kRotAny;
    const auto kern = mode == kRotNone ? qk_norm_rope_grad_kernel<T, true, kRotNone, NORM>
                      : mode == kRotHalf ? qk_norm_rope_grad_kernel<T, true, kRotHalf, NORM>
                      : mode == kRotInterleaved ? qk_norm_rope_grad_kernel<T, true, kRotInterleaved, NORM>
                                                : qk_norm_rope_grad_kernel<T, false, kRotAny, NORM>;
    kern<<<ctas, 32 * kWarps, 0, s>>>(a, passes, parts);
    if (cudaGetLastError() != cudaSuccess) return FALCON_ERR_CUDA;
  }
  if (ctas != 1 && (a.dw[0] || a.dw[1])) {
    norm_weight_sums_kernel<<<2, 1024, 0, s>>>(a.partial, ctas, a.h.d, a.dw[0], a.dw[1]);
    if (cudaGetLastError() != cudaSuccess) return FALCON_ERR_CUDA;
  }
  return FALCON_OK;
}

}  // namespace

size_t norm_grad_ws_bytes(int d) { return static_cast<size_t>(kMostCtas) * 2 * d * sizeof(float); }

int launch_qk_norm_rope_backward(const NormGradArgs& a, int dtype, cudaStream_t s) {
  if (dtype == FALCON_BF16) return a.h.norm ? launch<__nv_bfloat16, true>(a, s) : launch<__nv_bfloat16, false>(a, s);
  return a.h.norm ? launch<float, true>(a, s) : launch<float, false>(a, s);
}

}  // namespace falcon
