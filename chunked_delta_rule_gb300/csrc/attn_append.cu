// Append of new keys and values to the paged 8-bit cache, the norm and the
// rotation of the keys on the way.
//
// Per page, head and K or V: e_new from the largest finite magnitude of the
// page's new rows, e = e_new or max(e_old, e_new), old codes rounded again
// where the scale grew, new code = e4m3(x 2^-e).  Scales are powers of two:
// e4m3 keeps its relative precision at any of them, and a growing scale
// re-rounds only what falls below the normal range.
// Memory bound: 2 n Hkv d elements read, as many bytes written.

#include "attn.cuh"

namespace falcon {
namespace {

// One warp per (sequence, page, head, K or V); rows are read twice.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) kv_append_kernel(HeadArgs h, AppendArgs a, int cols, int64_t items) {
  const int lane = threadIdx.x & 31;
  int64_t it = blockIdx.x * static_cast<int64_t>(blockDim.x >> 5) + (threadIdx.x >> 5);
  if (it >= items) return;
  const bool is_v = it & 1;
  it >>= 1;
  const int head = static_cast<int>(it % a.Hkv);
  it /= a.Hkv;
  const int col = static_cast<int>(it % cols), b = static_cast<int>(it / cols);
  const int64_t first = a.cu[b];
  const int n_new = min(static_cast<int>(a.cu[b + 1] - first), a.max_q);
  const int64_t ctx = a.ctx[b];
  const int64_t pcol = ctx / a.page + col;             // column of the block table
  const int64_t t0 = max(pcol * a.page, ctx);          // first and last new token of the page
  const int64_t t1 = min((pcol + 1) * a.page, ctx + n_new);
  if (first < 0 || ctx < 0 || t0 >= t1 || pcol >= a.max_pages) return;
  const int pg = a.blocks[static_cast<int64_t>(b) * a.max_pages + pcol];
  if (pg < 0 || pg >= a.num_pages) return;
  const int n = static_cast<int>(t1 - t0), slot0 = static_cast<int>(t0 - pcol * a.page);
  const int64_t row0 = first + (t0 - ctx);
  if (row0 + n > a.tokens) return;

  const int L = h.d >> 3, rows = 32 / L, c0 = (lane % L) * 8, r0 = lane / L;
  const RowsIn in = is_v ? a.v : a.k;
  const T* src = static_cast<const T*>(in.p) + row0 * in.stride + static_cast<int64_t>(head) * h.d + c0;
  HeadArgs hv = h;
  if (is_v) hv.norm = hv.rot = 0;
  HeadPiece hp;
  load_weights(hp, hv, a.w_k, c0);
  auto row = [&](int r, float(&x)[8]) {
    const bool live = r < n;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.f;
    if (live) unpack8(load8<VEC>(src + r * in.stride), x);
    load_angles(hp, hv, t0 + r, c0);
    norm_rotate8<T>(x, hp, hv, a.w_k, src - c0 + r * in.stride, live, c0, lane);
  };

  float top = 0.f, x[8];
  for (int r = r0; r - r0 < n; r += rows) {
    row(r, x);
    if (r < n) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float m = fabsf(x[i]);
        if (m <= 3.402823466e38f) top = fmaxf(top, m);
      }
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  int e = scale_exponent(top);
  const int64_t ph = static_cast<int64_t>(pg) * a.Hkv + head;
  uint8_t* scale = (is_v ? a.cache.v_scale : a.cache.k_scale) + ph;
  uint8_t* codes = (is_v ? a.cache.v : a.cache.k) + ph * a.page * h.d;
  if (slot0 > 0) {
    const int old = static_cast<int>(*scale) - 127;
    __syncwarp();
    if (old >= e) {
      e = min(old, 127);
    } else {  // the scale grows: what the page holds is rounded again
      const float f = exp2i(max(old - e, -149));
      for (int i = lane * 8; i < slot0 * h.d; i += 256) {
        uint2 c = *reinterpret_cast<const uint2*>(codes + i);
        uint32_t w[2] = {c.x, c.y};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t lo = e4m3x2_to_half2(w[j] & 0xFFFFu), hi = e4m3x2_to_half2(w[j] >> 16);
          const float2 fl = __half22float2(*reinterpret_cast<const __half2*>(&lo));
          const float2 fh = __half22float2(*reinterpret_cast<const __half2*>(&hi));
          w[j] = to_e4m3x2(fl.x * f, fl.y * f) | (to_e4m3x2(fh.x * f, fh.y * f) << 16);
        }
        *reinterpret_cast<uint2*>(codes + i) = make_uint2(w[0], w[1]);
      }
    }
  }
  if (lane == 0) *scale = static_cast<uint8_t>(e + 127);
  const float f = exp2i(-e);
  codes += slot0 * h.d + c0;
  for (int r = r0; r - r0 < n; r += rows) {
    row(r, x);
    if (r < n) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = to_e4m3x2(x[2 * i] * f, x[2 * i + 1] * f);
      *reinterpret_cast<uint2*>(codes + r * h.d) = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
    }
  }
}

}  // namespace

int launch_kv_append(const HeadArgs& h, int dtype, const AppendArgs& a, cudaStream_t s) {
  if (a.max_q == 0 || a.tokens == 0) return FALCON_OK;
  const int cols = (a.page - 1 + a.max_q + a.page - 1) / a.page;  // pages that max_q tokens can touch
  const int64_t items = static_cast<int64_t>(a.B) * cols * a.Hkv * 2;
  const int64_t blocks = (items + 7) / 8;
  if (blocks > INT32_MAX) return FALCON_ERR_UNSUPPORTED;
  const bool vec = a.k.vec && a.v.vec;
  const unsigned g = static_cast<unsigned>(blocks);
  if (dtype == FALCON_BF16) {
    if (vec) kv_append_kernel<__nv_bfloat16, true><<<g, 256, 0, s>>>(h, a, cols, items);
    else kv_append_kernel<__nv_bfloat16, false><<<g, 256, 0, s>>>(h, a, cols, items);
  } else {
    if (vec) kv_append_kernel<float, true><<<g, 256, 0, s>>>(h, a, cols, items);
    else kv_append_kernel<float, false><<<g, 256, 0, s>>>(h, a, cols, items);
  }
  return cudaGetLastError() == cudaSuccess ? FALCON_OK : FALCON_ERR_CUDA;
}

}  // namespace falcon
