// Gradient of the per-head norm and the rotary positions.
//
//   n = dy rotated back, r = 1 / sqrt(mean(x^2) + eps), u = n w
//   dx = r (u - x r mean(u x r)),  dw = sum over tokens and heads of n x r
//
// Bound by memory on paper, where x and dy are read once and dx is written once, and
// as close by the instructions (250 for 256 elements by a warp; issue slots 2 / 3 full).  Lanes,
// pieces and angles as in the forward: d / 8 neighbouring lanes hold a head row, 8
// elements a lane; arithmetic on pairs; both sums of a row (x^2 and u x) go through
// one set of shuffles.  A warp walks tokens with the stride of the grid and adds its
// dw up in registers; the CTAs' sums go through the workspace to a second kernel, launched
// under the first, which adds them in one order.
// 32768 tokens of 20 heads of 128, bf16: 103 us, 5.0 TB/s (176 us with loads just
// ahead of their use, 126 with four passes' loads at once in registers, 110 with a pass at a time
// from the ring).

#include <algorithm>

#include "attn.cuh"
#include "attn_tc.cuh"

namespace falcon {
namespace {

constexpr int kWarps = 8;
constexpr int kMostCtas = 1024;  // whose sums the workspace holds
// CTAs of an SM: with three of the norm's the registers spill (the call above: 154 us); of the others' three take 20.5
// us for 16384 x 24 x 64 bf16, two 21.6
template <bool NORM>
constexpr int kResident = NORM ? 2 : 3;
constexpr int kPasses = 2;  // of a stage
template <typename T, bool NORM>
constexpr int kStages = NORM ? (sizeof(T) == 2 ? 4 : 3) : (sizeof(T) == 2 ? 8 : 4);  // 8 or 12 KB a warp

using tcu::fma2, tcu::mul2, tcu::pack2, tcu::unpack2;

template <typename T>
__device__ __forceinline__ void unpack8(const Raw8<T>& r, uint64_t (&x)[4]) {
  float f[8];
  falcon::unpack8(r, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = pack2(f[2 * i], f[2 * i + 1]);
}

// 8 elements to shared memory, 16 bytes at a time; bytes = 0: zeros
template <typename T>
__device__ __forceinline__ void copy8(uint32_t dst, const char* src, int bytes) {
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + 16 * i), "l"(src + 16 * i), "r"(bytes)
                 : "memory");
}
// y rotated back by the angles (co, si) of its pairs; ns = -si
template <int MODE>
__device__ __forceinline__ void rotate_back8(uint64_t (&y)[4], const uint64_t (&co)[4], const uint64_t (&si)[4],
                                             const uint64_t (&ns)[2]) {
  if constexpr (MODE == kRotHalf) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint64_t p = y[i], q = y[2 + i];
      y[i] = fma2(p, co[i], mul2(q, si[i]));
      y[2 + i] = fma2(q, co[i], mul2(p, ns[i]));
    }
  } else if constexpr (MODE == kRotInterleaved) {  // co = (cos, cos), si = (sin, -sin)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float p, q;
      unpack2(y[i], p, q);
      y[i] = fma2(y[i], co[i], mul2(pack2(q, p), si[i]));
    }
  }
}

// An item is a token's rows [part * passes * rows, ...): its query rows first, then its key rows.  A warp walks the
// passes of its items, whose rows come through a ring of its own in shared memory, kStages times kPasses passes.
template <typename T, bool VEC, int MODE, bool NORM>
__global__ void __launch_bounds__(32 * kWarps, MODE == kRotAny ? 1 : kResident<NORM>)
    qk_norm_rope_grad_kernel(NormGradArgs a, int passes, int parts) {
  const HeadArgs& h = a.h;
  if (NORM && a.partial) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ls = 28 - __clz(h.d), rows = 32 >> ls;  // log2 of the lanes of a row, rows of a pass
  const int li = lane & ((1 << ls) - 1);
  const Pieces at = pieces_of<MODE>(h, li);
  constexpr bool kSplit = MODE == kRotHalf, kRot = MODE == kRotHalf || MODE == kRotInterleaved;
  constexpr int S = kStages<T, NORM>, K = MODE == kRotAny ? 1 : kPasses;
  constexpr int kPass = NORM ? 512 : 256;  // elements of a pass: 256 of dy, 256 of x
  const int Hq = a.H[0], all = a.H[0] + a.H[1];
  extern __shared__ float4 ring_smem[];
  T* ring = reinterpret_cast<T*>(ring_smem) + warp * (S * K * kPass);
  __shared__ float4 weights[2][32][2];  // a lane's 8 of the queries' and of the keys' (the same in every warp)
  uint64_t dwq[4], dwk[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) dwq[i] = dwk[i] = 0;
  HeadPiece hp;
  if (NORM && warp < 2) {
    load_weights(hp, h, a.w[warp], at);
    weights[warp][lane][0] = make_float4(hp.w[0], hp.w[1], hp.w[2], hp.w[3]);
    weights[warp][lane][1] = make_float4(hp.w[4], hp.w[5], hp.w[6], hp.w[7]);
  }
  if (NORM) __syncthreads();
  uint64_t co[4], si[4], ns[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) co[i] = pack2(1.f, 1.f), si[i] = 0;  // dims that are not rotated
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps, start = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int64_t tok_step = step / parts;
  const int part_step = static_cast<int>(step % parts);
  auto advance = [&](int64_t& tok, int& part) {
    tok += tok_step;
    if ((part += part_step) >= parts) part -= parts, ++tok;
  };
  auto position = [&](int64_t t) { return MODE != kRotNone && h.rot && t < a.tokens ? a.pos[t] : 0; };
  // where row 0 of a token's queries lies (s = 0), and where it would lie for the keys' rows to follow at Hq
  auto row0 = [&](const auto& x, int64_t tok, int s) {
    return static_cast<const char*>(x.p) + (tok * x.stride - s * Hq * h.d) * static_cast<int64_t>(sizeof(T));
  };
  const uint32_t row_bytes = h.d * sizeof(T);

  // the item whose rows are copied next, the row of this lane there, the stage
  int64_t ahead = start / parts;
  int ahead_part = static_cast<int>(start % parts), ahead_p = 0, ahead_st = 0, ahead_r = 0, ahead_end = 0;
  const char *yq = nullptr, *yk = nullptr, *xq = nullptr, *xk = nullptr;
  const uint32_t to0 = tc::smem_u32(ring) + lane * 8 * sizeof(T), own = li * 8 * sizeof(T);
  auto copy = [&] {
    if (ahead < a.tokens) {
      if (ahead_p == 0) {
        yq = row0(a.dy[0], ahead, 0), yk = row0(a.dy[1], ahead, 1);
        if (NORM) xq = row0(a.x[0], ahead, 0), xk = row0(a.x[1], ahead, 1);
        ahead_r = ahead_part * passes * rows + (lane >> ls);
        ahead_end = min((ahead_part + 1) * passes * rows, all);
      }
#pragma unroll
      for (int k = 0; k < K; ++k) {
        // a lane past the rows: zeros
        const bool live = ahead_r < ahead_end, of_q = live ? ahead_r < Hq : Hq > 0;
        const uint32_t to = to0 + (ahead_st * K + k) * (kPass * sizeof(T));
        const int64_t off = (live ? ahead_r : of_q ? 0 : Hq) * row_bytes + own;
        copy8<T>(to, (of_q ? yq : yk) + off, live ? 16 : 0);
        if (NORM) copy8<T>(to + 256 * sizeof(T), (of_q ? xq : xk) + off, live ? 16 : 0);
        ahead_r += rows;
      }
      if ((ahead_p += K) >= passes) ahead_p = 0, advance(ahead, ahead_part);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (++ahead_st == S) ahead_st = 0;
  };
  int64_t tok = ahead;
  int part = ahead_part, st = 0;
  // angles and position of an item's token are under way an item before: the angles of the next one, the position of
  // the one after it
  int64_t tok1 = tok;
  int part1 = part;
  advance(tok1, part1);
  auto row_of = [&](int64_t pos) { return MODE != kRotNone && h.rot ? table_row(h, pos) : nullptr; };
  const float2* row = row_of(position(tok));
  load_angles<MODE>(hp, h, row, at);
  int64_t pos1 = position(tok1);
  if (MODE != kRotAny)
    for (int i = 0; i < S - 1; ++i) copy();
  while (tok < a.tokens) {
    const int first = part * passes * rows, end = min(first + passes * rows, all);
    if (kRot && at.a < h.rot) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        co[i] = pack2(hp.co[2 * i], hp.co[2 * i + 1]), si[i] = pack2(hp.si[2 * i], hp.si[2 * i + 1]);
        ns[i] = pack2(-hp.si[2 * i], -hp.si[2 * i + 1]);
      }
      if (MODE == kRotInterleaved)
#pragma unroll
        for (int i = 0; i < 4; ++i) co[i] = pack2(hp.co[i], hp.co[i]), si[i] = pack2(hp.si[i], -hp.si[i]);
    }
    const float2* row1 = row_of(pos1);
    load_angles<MODE>(hp, h, row1, at);
    char *oq = const_cast<char*>(row0(a.dx[0], tok, 0)), *ok = const_cast<char*>(row0(a.dx[1], tok, 1));
    const int64_t tok0 = tok;
    tok = tok1, part = part1;
    advance(tok1, part1);
    pos1 = position(tok1);
    for (int p = 0; p < passes; p += K) {
      const T* from = nullptr;
      if constexpr (MODE != kRotAny) {
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
        __syncwarp();  // the others' copies are there, and they have read the stage that is copied into next
        from = ring + st * (K * kPass) + (lane >> ls) * h.d;
        if (++st == S) st = 0;
        copy();
      }
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int r = first + (p + k) * rows + (lane >> ls);
        const bool live = r < end, of_q = r < Hq;
        uint64_t x[4] = {0, 0, 0, 0}, y[4] = {0, 0, 0, 0};
        if constexpr (MODE == kRotAny) {
          const int s = of_q ? 0 : 1;
          if (live) {
            unpack8(load8<VEC, kSplit>(reinterpret_cast<const T*>(row0(a.dy[s], tok0, s)) + r * h.d, at), y);
            if (NORM) unpack8(load8<VEC, kSplit>(reinterpret_cast<const T*>(row0(a.x[s], tok0, s)) + r * h.d, at), x);
          }
        } else {
          unpack8(load8<true, kSplit>(from + k * kPass, at), y);
          if (NORM) unpack8(load8<true, kSplit>(from + k * kPass + 256, at), x);
        }
        if constexpr (MODE == kRotAny) {
          const T* src = reinterpret_cast<const T*>(row0(a.dy[of_q ? 0 : 1], tok0, of_q ? 0 : 1)) + r * h.d;
          const int half = h.rot >> 1;
          const bool hl = h.layout == FALCON_ROPE_HALF;
          float z[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int c = (i < 4 ? at.a : at.b - 4) + i, j = hl ? (c < half ? c : c - half) : c >> 1;  // element, its pair
            const bool low = hl ? c < half : !(c & 1);
            float mine[2];
            unpack2(y[i >> 1], mine[0], mine[1]);
            z[i] = mine[i & 1];
            if (live && c < h.rot) {
              const float other = to_f32(src[hl ? (low ? c + half : c - half) : c ^ 1]);
              const float2 t = row ? __ldg(row + j) : make_float2(__int_as_float(0x7fffffff), 0.f);
              z[i] = z[i] * t.x + (low ? t.y : -t.y) * other;
            }
          }
          __syncwarp();  // read before any lane writes the row in place
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = pack2(z[2 * i], z[2 * i + 1]);
        } else if (kRot && at.a < h.rot) {
          rotate_back8<MODE>(y, co, si, ns);
        }
        if (NORM) {
          const float4 w0 = weights[of_q ? 0 : 1][lane][0], w1 = weights[of_q ? 0 : 1][lane][1];
          const uint64_t w[4] = {pack2(w0.x, w0.y), pack2(w0.z, w0.w), pack2(w1.x, w1.y), pack2(w1.z, w1.w)};
          uint64_t v[4], xx = mul2(x[0], x[0]), vx;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[i] = mul2(y[i], w[i]);
            vx = i ? fma2(v[i], x[i], vx) : mul2(v[i], x[i]);
            if (i) xx = fma2(x[i], x[i], xx);
          }
          float s0, s1, t0, t1;
          unpack2(xx, s0, t0);
          unpack2(vx, s1, t1);
          s0 += t0, s1 += t1;
          // over the d / 8 lanes: 2, 4, 8 or 16
#pragma unroll
          for (int m = 1; m < 16; m <<= 1) {
            if (m >= 1 << ls) break;
            s0 += __shfl_xor_sync(0xffffffffu, s0, m);
            s1 += __shfl_xor_sync(0xffffffffu, s1, m);
          }
          const float rs = live ? rsqrtf(fmaf(s0, h.inv_d, h.eps)) : 0.f;
          const float c = rs == 0.f ? 0.f : s1 * rs * h.inv_d;
          const uint64_t rs2 = pack2(rs, rs), nc = pack2(-c, -c);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint64_t xr = mul2(x[i], rs2);
            if (of_q) dwq[i] = fma2(y[i], xr, dwq[i]);
            else dwk[i] = fma2(y[i], xr, dwk[i]);
            y[i] = mul2(rs2, fma2(xr, nc, v[i]));
          }
        }
        if (live) {
          float z[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) unpack2(y[i], z[2 * i], z[2 * i + 1]);
          store8<VEC, kSplit>(reinterpret_cast<T*>((of_q ? oq : ok) + static_cast<int64_t>(r) * row_bytes), at, z);
        }
      }
    }
    row = row1;
  }
  if (!NORM || !a.partial) return;
  // the warp's rows, then the CTA's warps
  __syncthreads();  // every copy has been waited for and read
  float(*sum)[2][128] = reinterpret_cast<float(*)[2][128]>(ring_smem);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float q[2], k[2];
    unpack2(dwq[i >> 1], q[0], q[1]);
    unpack2(dwk[i >> 1], k[0], k[1]);
    for (int m = 16; m >= 1 << ls; m >>= 1) {
      q[i & 1] += __shfl_xor_sync(0xffffffffu, q[i & 1], m);
      k[i & 1] += __shfl_xor_sync(0xffffffffu, k[i & 1], m);
    }
    const int c = (i < 4 ? at.a : at.b - 4) + i;
    if (lane < 1 << ls) sum[warp][0][c] = q[i & 1], sum[warp][1][c] = k[i & 1];
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

// dw from the sums of n CTAs (none: 0): a CTA for 16 dims of the queries' or of the keys', 64 threads a dim
constexpr int kSumDims = 16, kSlices = 64;
__global__ void __launch_bounds__(kSumDims * kSlices)
    norm_weight_sums_kernel(const float* partial, int n, int d, float* dw_q, float* dw_k) {
  float* dw = blockIdx.y ? dw_k : dw_q;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!dw) return;
  __shared__ float sum[kSlices][kSumDims];
  const int c = threadIdx.x % kSumDims, slice = threadIdx.x / kSumDims, at = blockIdx.x * kSumDims + c;
  float v = 0.f;
#pragma unroll 4
  for (int i = slice; i < n; i += kSlices) v += partial[(i * 2 + blockIdx.y) * d + at];
  sum[slice][c] = v;
  __syncthreads();
  if (threadIdx.x < 32) {  // half of the slices a lane
    v = 0.f;
#pragma unroll
    for (int i = 0; i < kSlices / 2; ++i) v += sum[2 * i + (threadIdx.x >> 4)][c];
    v += __shfl_xor_sync(0xffffffffu, v, 16);
    if (threadIdx.x < kSumDims) dw[at] = v;
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
    ctas = static_cast<int>(std::min<int64_t>(want, std::min(kResident<NORM> * tcu::sm_count(), kMostCtas)));
    const RotMode mode = vec ? rot_mode(a.h) : kRotAny;
    const auto kern = mode == kRotNone ? qk_norm_rope_grad_kernel<T, true, kRotNone, NORM>
                      : mode == kRotHalf ? qk_norm_rope_grad_kernel<T, true, kRotHalf, NORM>
                      : mode == kRotInterleaved ? qk_norm_rope_grad_kernel<T, true, kRotInterleaved, NORM>
                                                : qk_norm_rope_grad_kernel<T, false, kRotAny, NORM>;
    const size_t smem = static_cast<size_t>(kWarps) * kStages<T, NORM> * kPasses * (NORM ? 512 : 256) * sizeof(T);
    if (!set_smem_limit(reinterpret_cast<const void*>(kern), smem)) return FALCON_ERR_CUDA;
    kern<<<ctas, 32 * kWarps, smem, s>>>(a, passes, parts);
    if (cudaGetLastError() != cudaSuccess) return FALCON_ERR_CUDA;
  }
  if (ctas != 1 && (a.dw[0] || a.dw[1])) {
    // launched while the rows' kernel runs, which it waits for
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.h.d / kSumDims, 2);
    cfg.blockDim = dim3(kSumDims * kSlices);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas ? 1 : 0;
    const float* partial = a.partial;
    if (cudaLaunchKernelEx(&cfg, norm_weight_sums_kernel, partial, ctas, a.h.d, a.dw[0], a.dw[1]) != cudaSuccess)
      return FALCON_ERR_CUDA;
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
