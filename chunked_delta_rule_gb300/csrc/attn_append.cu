// Append of new keys and values to the paged 8-bit cache, the norm and the
// rotation of the keys on the way.
//
// Per page, head and K or V: e_new from the largest finite magnitude of the
// page's new rows, e = e_new or max(e_old, e_new), old codes rounded again
// where the scale grew, new code = e4m3(x 2^-e).  Scales are powers of two:
// e4m3 keeps its relative precision at any of them, and a growing scale
// re-rounds only what falls below the normal range.
// Memory bound: 2 n Hkv d elements read, as many bytes written.  The new rows of
// one page, head and K or V are read once and stay in registers, normed and
// rotated, while their largest magnitude is found: by a warp where a sequence
// brings few tokens (a decode step: 256 x 12 heads of 64 in one launch of
// small warps), else by a CTA.  d / 8 neighbouring lanes hold a row.
// Measured: 2 x 16384 tokens, 16 heads of 128, bf16: 403 MB in 76 us, 5.3 TB/s;
// 256 x 1 x 12 heads of 64: 6.2 us with the call, most of it the launch.

#include "attn.cuh"

namespace falcon {
namespace {

// THREADS (32 or 256) work on one (sequence, page, head, K or V); a thread
// holds 8 elements of NP rows.
template <typename T, bool VEC, int MODE, int THREADS, int NP>
__global__ void __launch_bounds__(256) kv_append_kernel(HeadArgs h, AppendArgs a, uint32_t cols) {
  constexpr int kItems = 256 / THREADS;  // of a CTA: neighbouring heads
  const int lane = threadIdx.x & 31, tid = threadIdx.x % THREADS;
  const int hv = blockIdx.y * kItems + threadIdx.x / THREADS, head = hv >> 1;
  if (head >= a.Hkv) return;
  const bool is_v = hv & 1;
  const int b = static_cast<int>(blockIdx.x / cols), col = static_cast<int>(blockIdx.x % cols);
  const int64_t first = a.cu[b];
  const int n_new = min(static_cast<int>(a.cu[b + 1] - first), a.max_q);
  const int64_t ctx = a.ctx[b];
  const int shift = 31 - __clz(a.page);
  const int64_t pcol = (ctx >> shift) + col;              // column of the block table
  const int64_t t0 = max(pcol << shift, ctx);             // first and past the last new token of the page
  const int64_t t1 = min((pcol + 1) << shift, ctx + n_new);
  if (first < 0 || ctx < 0 || t0 >= t1 || pcol >= a.max_pages) return;
  const int n = static_cast<int>(t1 - t0), slot0 = static_cast<int>(t0 & (a.page - 1));
  const int64_t row0 = first + (t0 - ctx);
  if (row0 + n > a.tokens) return;
  const int pg = a.blocks[static_cast<int64_t>(b) * a.max_pages + pcol];

  const int ls = 28 - __clz(h.d), rows = THREADS >> ls, r0 = tid >> ls;
  const Pieces at = pieces_of<MODE>(h, tid & ((1 << ls) - 1));
  constexpr bool kSplit = MODE == kRotHalf;
  const RowsIn in = is_v ? a.v : a.k;
  const T* src = static_cast<const T*>(in.p) + row0 * in.stride + static_cast<int64_t>(head) * h.d;
  Raw8<T> raw[NP];
#pragma unroll
  for (int u = 0; u < NP; ++u)
    if (r0 + u * rows < n) raw[u] = load8<VEC, kSplit>(src + (r0 + u * rows) * in.stride, at);
  if (pg < 0 || pg >= a.num_pages) return;
  const int64_t ph = static_cast<int64_t>(pg) * a.Hkv + head;
  uint8_t* scale = (is_v ? a.cache.v_scale : a.cache.k_scale) + ph;
  uint8_t* codes = ((is_v ? a.cache.v : a.cache.k) + ((ph * h.d) << shift));
  const int old = slot0 > 0 ? static_cast<int>(*scale) - 127 : 0;

  float x[NP][8], top = 0.f;
#pragma unroll
  for (int u = 0; u < NP; ++u) {
    if (r0 + u * rows < n) {
      unpack8(raw[u], x[u]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[u][i] = 0.f;
    }
  }
  if (!is_v && (MODE != kRotNone || h.norm)) {
    HeadPiece hp;
    load_weights(hp, h, a.w_k, at);
#pragma unroll
    for (int u = 0; u < NP; ++u) {
      const int r = r0 + u * rows;
      const float2* row = MODE != kRotNone && h.rot ? table_row(h, t0 + r) : nullptr;
      load_angles<MODE>(hp, h, row, at);
      norm_rotate8<MODE, T>(x[u], hp, h, a.w_k, row, src + r * in.stride, r < n, at);
    }
  }
#pragma unroll
  for (int u = 0; u < NP; ++u)
    if (r0 + u * rows < n) {
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[u][i]));
    }
  if (top == INFINITY) {  // the largest finite one then
    top = 0.f;
#pragma unroll
    for (int u = 0; u < NP; ++u)
      if (r0 + u * rows < n) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float m = fabsf(x[u][i]);
          if (m < INFINITY) top = fmaxf(top, m);
        }
      }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (THREADS == 256) {
    __shared__ float tops[8];
    if (lane == 0) tops[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, tops[i]);
  } else {
    __syncwarp();
  }
  int e = scale_exponent(top);
  if (slot0 > 0) {
    if (old >= e) {
      e = min(old, 127);
    } else {  // the scale grows: what the page holds is rounded again
      const float f = exp2i(max(old - e, -149));
      for (int i = tid * 8; i < slot0 * h.d; i += THREADS * 8) {
        const uint2 c = *reinterpret_cast<const uint2*>(codes + i);
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
  if (tid == 0) *scale = static_cast<uint8_t>(e + 127);
  const float f = exp2i(-e);
  codes += slot0 * h.d;
#pragma unroll
  for (int u = 0; u < NP; ++u) {
    const int r = r0 + u * rows;
    if (r < n) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = to_e4m3x2(x[u][2 * i] * f, x[u][2 * i + 1] * f);
      const uint2 c = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
      if (kSplit) {
        *reinterpret_cast<uint32_t*>(codes + r * h.d + at.a) = c.x;
        *reinterpret_cast<uint32_t*>(codes + r * h.d + at.b) = c.y;
      } else {
        *reinterpret_cast<uint2*>(codes + r * h.d + at.a) = c;
      }
    }
  }
}

template <typename T, bool VEC, int MODE, int THREADS, int NP>
int launch(const HeadArgs& h, const AppendArgs& a, cudaStream_t s) {
  const int64_t cols = (static_cast<int64_t>(a.page) - 1 + a.max_q + a.page - 1) / a.page;  // pages that max_q tokens touch
  constexpr int items = 256 / THREADS;
  const int64_t x = cols * a.B, y = (2 * static_cast<int64_t>(a.Hkv) + items - 1) / items;
  if (x > INT32_MAX || y > 65535) return FALCON_ERR_UNSUPPORTED;
  kv_append_kernel<T, VEC, MODE, THREADS, NP><<<dim3(static_cast<unsigned>(x), static_cast<unsigned>(y)), 256, 0, s>>>(
      h, a, static_cast<uint32_t>(cols));
  return cudaGetLastError() == cudaSuccess ? FALCON_OK : FALCON_ERR_CUDA;
}
template <typename T, bool VEC, int MODE>
int launch_size(const HeadArgs& h, const AppendArgs& a, cudaStream_t s) {
  // up to 8 or 16 elements a lane: a warp an item; else a CTA, the page's rows over its threads
  const int most = a.max_q < a.page ? a.max_q : a.page;
  if (most * h.d <= 256) return launch<T, VEC, MODE, 32, 1>(h, a, s);
  if (most * h.d <= 512) return launch<T, VEC, MODE, 32, 2>(h, a, s);
  if (most * h.d <= 4096) return launch<T, VEC, MODE, 256, 2>(h, a, s);
  if (most * h.d <= 8192) return launch<T, VEC, MODE, 256, 4>(h, a, s);
  return launch<T, VEC, MODE, 256, 8>(h, a, s);
}
template <typename T>
int launch_mode(const HeadArgs& h, const AppendArgs& a, cudaStream_t s) {
  switch (a.k.vec && a.v.vec ? rot_mode(h) : kRotAny) {
    case kRotNone: return launch_size<T, true, kRotNone>(h, a, s);
    case kRotHalf: return launch_size<T, true, kRotHalf>(h, a, s);
    case kRotInterleaved: return launch_size<T, true, kRotInterleaved>(h, a, s);
    default: return launch_size<T, false, kRotAny>(h, a, s);
  }
}

}  // namespace

int launch_kv_append(const HeadArgs& h, int dtype, const AppendArgs& a, cudaStream_t s) {
  if (a.max_q == 0 || a.tokens == 0) return FALCON_OK;
  return dtype == FALCON_BF16 ? launch_mode<__nv_bfloat16>(h, a, s) : launch_mode<float>(h, a, s);
}

}  // namespace falcon
