// Gradient of causal attention over packed prompts: the rows' sums that the bf16
// kernels read, and the products where the tcgen05 kernels do not go (bf16 rows off
// the 16-byte boundaries, scales below 2^-100, calls without query rows).
//
//   P = exp(scale Q K^T - log sum),  dS = P (dO V^T - D),  D = sum_c dO_c o_c - dlse
//   dV = P^T dO,  dK = scale dS^T Q,  dQ = scale dS K
//
// The weights are formed again from the log sums that the forward left.  Two kernels,
// so that every sum has one owner and one order: a CTA of the first takes 64 queries
// of one head and walks their keys (dQ), one of the second 64 keys of a key head and
// walks the queries of all its heads (dK by four of its warps, dV by the other four).
// Rows of the tile that a CTA owns lie in shared memory throughout, the others come 64 at a
// time.  Products are warp-level tf32 MMAs as in the forward; P and dS are rounded to 11
// bits.  Bound by the instructions around the MMAs: 8 x 2048 tokens, 12 heads of 64, 2.3 ms.
//
// A masked weight is 0, but 0 times an infinite or NaN value of a row that the
// owner does not see would spoil it.  A row of a result that is not finite is
// therefore computed again from the definition, touching only what it sees.

#include "attn_grad.cuh"
#include "attn_mma.cuh"

namespace falcon {
namespace {

using T = __nv_bfloat16;

// ---------------------------------------------------------------- sums of the rows
// x as three bf16 numbers (24 bits), packed in pairs
__device__ __forceinline__ uint2 three_parts(float x) {
  const float hi = __bfloat162float(__float2bfloat16_rn(x)), mid = __bfloat162float(__float2bfloat16_rn(x - hi));
  return make_uint2(tcu::pack_bf16(x, x - hi), tcu::pack_bf16(x - hi - mid, 0.f));
}
// A CTA takes 128 rows of one head: d / 8 lanes a row, two rows' loads of each under way at once; then a thread a row.
// Bound by memory: 13906 x 16 x 128 bf16, 24 us, 4.7 TB/s.
__global__ void __launch_bounds__(256, 6) attn_grad_sums_kernel(GradArgs g) {
  const PromptArgs& a = g.a;
  launch_dependents();
  // the call's status, and the blocks of dQ that have begun
  if (blockIdx.x == 0 && threadIdx.x == 0) *static_cast<uint2*>(a.ws) = make_uint2(0u, 0u);
  const int h = static_cast<int>(blockIdx.x % a.Hq);
  const int64_t j = blockIdx.x / a.Hq;
  const int2 x = find_block(a.cu_q, a.B, kSumRows, static_cast<int>(j));
  const int64_t q0 = a.cu_q[x.x], q1 = a.cu_q[x.x + 1];
  if (x.y < 0 || q0 < 0 || q1 > a.tokens || x.y >= q1 - q0) return;
  const int lq = static_cast<int>(min(q1 - q0, static_cast<int64_t>(a.max_q)));
  const int rows = min(lq - x.y, kSumRows);  // live ones
  __shared__ float dots[kSumRows];
  float l = -INFINITY, dl = 0.f;  // of the thread's row
  if (static_cast<int>(threadIdx.x) < rows) {
    const int64_t i = (q0 + x.y + threadIdx.x) * a.Hq + h;
    l = g.lse[i];
    if (g.dlse) dl = g.dlse[i];
  }
  const int ls = 28 - __clz(a.d), li = threadIdx.x & ((1 << ls) - 1), step = 256 >> ls;
  const Pieces p{li * 8, li * 8 + 4};
  const T* o = static_cast<const T*>(g.o.p) + (q0 + x.y) * g.o.stride + h * a.d;
  const T* d_o = static_cast<const T*>(g.d_o.p) + (q0 + x.y) * g.d_o.stride + h * a.d;
  for (int r0 = threadIdx.x >> ls; r0 < kSumRows; r0 += 2 * step) {
    Raw8<T> u[2], v[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int r = r0 + k * step;
      if (r >= rows) continue;
      u[k] = g.o.vec ? load8<true, false>(o + r * g.o.stride, p) : load8<false, false>(o + r * g.o.stride, p);
      v[k] = g.d_o.vec ? load8<true, false>(d_o + r * g.d_o.stride, p) : load8<false, false>(d_o + r * g.d_o.stride, p);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int r = r0 + k * step;
      float s = 0.f;
      if (r < rows) {
        float y[8], z[8];
        unpack8(u[k], y);
        unpack8(v[k], z);
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(y[e], z[e], s);
      }
      for (int m = 1; m < 1 << ls; m <<= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
      if (li == 0 && r < kSumRows) dots[r] = s;
    }
  }
  __syncthreads();
  const int r = threadIdx.x;
  if (r >= kSumRows) return;
  // find_block deals a sequence's blocks out from the last; here block n of a sequence holds its rows 128 n ..
  const int64_t at = h * g.blocks + first_block(q0, x.x) + x.y / kSumRows;
  const float lse = l == -INFINITY ? INFINITY : l == INFINITY ? __int_as_float(0x7fffffff) : l;
  const float delta = l == -INFINITY ? 0.f : dots[r] - dl;
  g.sums[row_sums(1, 0, at) + r] = lse;
  g.sums[row_sums(1, 0, at) + kSumRows + r] = delta;
  if (!g.images) return;
  // no weight: bf16's lowest number (an infinity would spoil the columns' zeros) in all three parts, so that whatever
  // finite score they are added to, the sum is -inf or fp32's lowest number: see attn_grad_tc_supported for the scale
  const uint2 y = lse == INFINITY ? make_uint2(0xFF7FFF7Fu, 0xFF7Fu) : three_parts(-lse / a.scale), z = three_parts(-delta);
  uint4* to = reinterpret_cast<uint4*>(g.images + at * kImageBytes + (r >> 3) * 256 + (r & 7) * 16);
  to[0] = make_uint4(y.x, y.y, z.x, z.y);
  to[8] = make_uint4(0u, 0u, 0u, 0u);
}

// ---------------------------------------------------------------- warp-level kernels
constexpr int kRows = kMmaRows, NT = kRows / 8;

// x (16 rows of a warp x 64) = A B^T, A and B rows of D in shared memory
template <int D>
__device__ __forceinline__ void rows_product(float (&x)[NT][4], const float* A, const float* Bm, int gid, int tig) {
  constexpr int LD = D + 4;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) x[t][e] = 0.f;
#pragma unroll 2
  for (int ks = 0; ks < D / 8; ++ks) {
    const float* qa = A + gid * LD + ks * 8 + tig;
    const uint32_t af[4] = {__float_as_uint(qa[0]), __float_as_uint(qa[8 * LD]), __float_as_uint(qa[4]),
                            __float_as_uint(qa[8 * LD + 4])};
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float* kb = Bm + (t * 8 + gid) * LD + ks * 8 + tig;
      const uint32_t bf[2] = {__float_as_uint(kb[0]), __float_as_uint(kb[4])};
      tc::mma_tf32_16x8x8(x[t], af, bf);
    }
  }
}

// acc (16 rows x D) += W B: W the warp's 16 x 64 weights as rows_product leaves them, B 64 rows of D.  Column 2c of a
// group of 8 takes the place of column c, 2c + 1 that of c + 4, in both operands.
template <int D>
__device__ __forceinline__ void add_product(float (&acc)[D / 8][4], const float (&w)[NT][4], const float* Bm, int gid,
                                            int tig) {
  constexpr int LD = D + 4;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const uint32_t pf[4] = {tc::to_tf32(w[t][0]), tc::to_tf32(w[t][2]), tc::to_tf32(w[t][1]), tc::to_tf32(w[t][3])};
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      const float* vb = Bm + (t * 8 + 2 * tig) * LD + i * 8 + gid;
      const uint32_t bf[2] = {__float_as_uint(vb[0]), __float_as_uint(vb[LD])};
      tc::mma_tf32_16x8x8(acc[i], pf, bf);
    }
  }
}

// Rows of a warp's sums to their places (out: row 0 of the block's), and which of this thread's two rows are not finite.
template <int D>
__device__ __forceinline__ void store_sums(const float (&acc)[D / 8][4], float f, T* out, int64_t stride, int rows, int r0,
                                           int tig, bool (&bad)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = r0 + 8 * i;
    bad[i] = false;
#pragma unroll
    for (int t = 0; t < D / 8; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float x = acc[t][2 * i + e] * f;
        bad[i] |= !(fabsf(x) <= 3.402823466e38f);
        if (r < rows) out[r * stride + t * 8 + 2 * tig + e] = from_f32<T>(x);
      }
    bad[i] = bad[i] && r < rows;
  }
}

// dQ: a CTA takes 64 queries of one head
template <int D>
__global__ void __launch_bounds__(128) attn_grad_queries_kernel(GradArgs g, int qblocks, bool packed) {
  constexpr int LD = D + 4;
  const PromptArgs& a = g.a;
  extern __shared__ float smem[];
  float *sq = smem, *sg = sq + kRows * LD, *sk = sg + kRows * LD, *sv = sk + kRows * LD;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, tig = lane & 3;
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
  const T* d_o = static_cast<const T*>(g.d_o.p) + q0 * g.d_o.stride + static_cast<int64_t>(h) * D;
  const T* k = static_cast<const T*>(a.k.p) + k0 * a.k.stride + static_cast<int64_t>(hk) * D;
  const T* v = static_cast<const T*>(a.v.p) + k0 * a.v.stride + static_cast<int64_t>(hk) * D;
  stage_rows<T, D, 128>(sq, q, a.q.stride, a.q.vec, row0, lq);
  stage_rows<T, D, 128>(sg, d_o, g.d_o.stride, g.d_o.vec, row0, lq);
  const float* sums = g.sums + row_sums(g.blocks, h, first_block(q0, b) + row0 / kSumRows) + row0 % kSumRows;
  const int r0 = warp * 16 + gid;  // this thread's rows: r0 and r0 + 8 of the block
  const float lse[2] = {sums[r0], sums[r0 + 8]}, delta[2] = {sums[kSumRows + r0], sums[kSumRows + r0 + 8]};

  float acc[D / 8][4];
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
  const int keys = min(min(row0 + kRows, lq) + off, lk);  // that some row of the block sees
  for (int j0 = 0; j0 < keys; j0 += kRows) {
    __syncthreads();
    stage_rows<T, D, 128>(sk, k, a.k.stride, a.k.vec, j0, lk);
    stage_rows<T, D, 128>(sv, v, a.v.stride, a.v.vec, j0, lk);
    __syncthreads();
    float p[NT][4], y[NT][4];
    rows_product<D>(p, sq + warp * 16 * LD, sk, gid, tig);
    rows_product<D>(y, sg + warp * 16 * LD, sv, gid, tig);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = j0 + t * 8 + 2 * tig + (e & 1), i = e >> 1;
        // the difference first: it is small where the weight is not
        const float w = ex2(fmaf(p[t][e], a.scale, -lse[i]) * kLog2e);
        y[t][e] = c < min(row0 + r0 + 8 * i + off + 1, lk) ? w * (y[t][e] - delta[i]) : 0.f;
      }
    add_product<D>(acc, y, sk, gid, tig);
  }
  bool bad[2];
  T* out = static_cast<T*>(g.dq.p) + (q0 + row0) * g.dq.stride + static_cast<int64_t>(h) * D;
  store_sums<D>(acc, a.scale, out, g.dq.stride, lq - row0, r0, tig, bad);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 2; ++i)
    for (uint32_t again = __ballot_sync(0xffffffffu, bad[i]); again;) {
      const int r = warp * 16 + ((__ffs(again) - 1) >> 2) + 8 * i, row = row0 + r;
      again &= ~(0xFu << (4 * ((__ffs(again) - 1) >> 2)));
      float x[4];
      grad_query_row<T, D>(q + row * a.q.stride, d_o + row * g.d_o.stride, sums[r], sums[kSumRows + r], k, a.k.stride, v,
                           a.v.stride, min(row + off + 1, lk), D, a.scale, x);
      store_row<T, D>(out + r * g.dq.stride, x, D);
    }
}

// dK and dV: a CTA takes 64 keys of a key head; warps 0 to 3 form dV, 4 to 7 dK
template <int D>
__global__ void __launch_bounds__(256) attn_grad_keys_kernel(GradArgs g) {
  constexpr int LD = D + 4;
  const PromptArgs& a = g.a;
  // the call's status: a call without queries has no rows' sums, whose kernel clears it otherwise
  if (blockIdx.x == 0 && threadIdx.x == 0) *static_cast<uint32_t*>(a.ws) = 0;
  extern __shared__ float smem[];
  float *sk = smem, *sv = sk + kRows * LD, *sq = sv + kRows * LD, *sg = sq + kRows * LD, *ss = sg + kRows * LD;
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3, gid = lane >> 2, tig = lane & 3;
  const bool of_k = threadIdx.x >= 128;
  const int hk = static_cast<int>(blockIdx.x % a.Hkv), G = a.Hq / a.Hkv;
  const int2 x = packed_block(a.cu_k, a.B, kRows, static_cast<int>(blockIdx.x / a.Hkv));
  const int b = x.x;
  const int64_t q0 = a.cu_q[b], k0 = a.cu_k[b];
  const int lq_all = static_cast<int>(a.cu_q[b + 1] - q0), lk = static_cast<int>(a.cu_k[b + 1] - k0);
  const int lq = min(lq_all, a.max_q), off = lk - lq_all;
  if (x.y < 0 || x.y >= lk || q0 < 0 || k0 < 0 || q0 + lq_all > a.tokens || k0 + lk > a.k_tokens) return;
  // a sequence's blocks come from its last here: the first keys, which the most queries see, first
  const int row0 = (lk - 1) / kRows * kRows - x.y;
  if (row0 < 0) return;
  const T* k = static_cast<const T*>(a.k.p) + k0 * a.k.stride + static_cast<int64_t>(hk) * D;
  const T* v = static_cast<const T*>(a.v.p) + k0 * a.v.stride + static_cast<int64_t>(hk) * D;
  const T* q = static_cast<const T*>(a.q.p) + q0 * a.q.stride + static_cast<int64_t>(hk) * G * D;
  const T* d_o = static_cast<const T*>(g.d_o.p) + q0 * g.d_o.stride + static_cast<int64_t>(hk) * G * D;
  const float* sums = g.sums + row_sums(g.blocks, hk * G, first_block(q0, b));
  stage_rows<T, D, 256>(sk, k, a.k.stride, a.k.vec, row0, lk);
  stage_rows<T, D, 256>(sv, v, a.v.stride, a.v.vec, row0, lk);

  float acc[D / 8][4];
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
  const int r0 = warp * 16 + gid;
  const int first = max(row0 - off, 0) / kRows * kRows;  // queries before it see none of these keys
  for (int h = 0; h < G; ++h)
    for (int i0 = first; i0 < lq; i0 += kRows) {
      __syncthreads();
      stage_rows<T, D, 256>(sq, q + h * D, a.q.stride, a.q.vec, i0, lq);
      stage_rows<T, D, 256>(sg, d_o + h * D, g.d_o.stride, g.d_o.vec, i0, lq);
      if (threadIdx.x < 2 * kRows) {
        const float* from = sums + row_sums(g.blocks, h, i0 / kSumRows) + i0 % kSumRows;
        ss[threadIdx.x] = threadIdx.x < kRows ? from[threadIdx.x] : from[kSumRows + threadIdx.x - kRows];
      }
      __syncthreads();
      float p[NT][4];
      rows_product<D>(p, sk + warp * 16 * LD, sq, gid, tig);
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = t * 8 + 2 * tig + (e & 1);
          const float w = ex2(fmaf(p[t][e], a.scale, -ss[c]) * kLog2e);
          p[t][e] = row0 + r0 + 8 * (e >> 1) <= i0 + c + off && i0 + c < lq ? w : 0.f;
        }
      if (of_k) {
        float y[NT][4];
        rows_product<D>(y, sv + warp * 16 * LD, sg, gid, tig);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int c = t * 8 + 2 * tig + (e & 1);
            p[t][e] = row0 + r0 + 8 * (e >> 1) <= i0 + c + off && i0 + c < lq ? p[t][e] * (y[t][e] - ss[kRows + c]) : 0.f;
          }
      }
      add_product<D>(acc, p, of_k ? sq : sg, gid, tig);
    }
  bool bad[2];
  const RowsOut& to = of_k ? g.dk : g.dv;
  T* out = static_cast<T*>(to.p) + (k0 + row0) * to.stride + static_cast<int64_t>(hk) * D;
  store_sums<D>(acc, of_k ? a.scale : 1.f, out, to.stride, lk - row0, r0, tig, bad);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 2; ++i)
    for (uint32_t again = __ballot_sync(0xffffffffu, bad[i]); again;) {
      const int r = warp * 16 + ((__ffs(again) - 1) >> 2) + 8 * i, row = row0 + r;
      again &= ~(0xFu << (4 * ((__ffs(again) - 1) >> 2)));
      float xk[4], xv[4];
      grad_key_row<T, D>(k + row * a.k.stride, v + row * a.v.stride, q, a.q.stride, d_o, g.d_o.stride, sums, g.blocks, G,
                         max(row - off, 0), lq, D, a.scale, xk, xv);
      store_row<T, D>(out + r * to.stride, of_k ? xk : xv, D);
    }
}

template <int D>
int launch(const GradArgs& g, cudaStream_t s) {
  const PromptArgs& a = g.a;
  constexpr int LD = D + 4;
  if (g.dq.p && a.tokens > 0 && a.max_q > 0) {
    const PromptGrid pg = prompt_grid(a, kRows);
    if (pg.blocks < 1 || pg.blocks > INT32_MAX / a.Hq) return FALCON_ERR_UNSUPPORTED;
    constexpr size_t smem = static_cast<size_t>(4 * kRows * LD) * 4;
    const auto kern = attn_grad_queries_kernel<D>;
    if (!set_smem_limit(reinterpret_cast<const void*>(kern), smem)) return FALCON_ERR_CUDA;
    kern<<<static_cast<unsigned>(pg.blocks * a.Hq), 128, smem, s>>>(g, static_cast<int>(pg.blocks / a.B), pg.packed);
    if (cudaGetLastError() != cudaSuccess) return FALCON_ERR_CUDA;
  }
  if (g.dk.p && a.k_tokens > 0) {
    const int64_t blocks = a.k_tokens / kRows + a.B;
    if (blocks > INT32_MAX / a.Hkv) return FALCON_ERR_UNSUPPORTED;
    constexpr size_t smem = static_cast<size_t>(4 * kRows * LD + 2 * kRows) * 4;
    const auto kern = attn_grad_keys_kernel<D>;
    if (!set_smem_limit(reinterpret_cast<const void*>(kern), smem)) return FALCON_ERR_CUDA;
    kern<<<static_cast<unsigned>(blocks * a.Hkv), 256, smem, s>>>(g);
    if (cudaGetLastError() != cudaSuccess) return FALCON_ERR_CUDA;
  }
  return FALCON_OK;
}

int launch_bf16(const GradArgs& g, cudaStream_t s) {
  const PromptArgs& a = g.a;
  if (a.tokens > 0 && a.max_q > 0) {
    if (g.blocks > INT32_MAX / a.Hq) return FALCON_ERR_UNSUPPORTED;
    attn_grad_sums_kernel<<<static_cast<unsigned>(g.blocks * a.Hq), 256, 0, s>>>(g);
    if (cudaGetLastError() != cudaSuccess) return FALCON_ERR_CUDA;
  }
  if (g.images) return launch_attn_grad_tc(g, s);
  switch (a.d) {
    case 16: return launch<16>(g, s);
    case 32: return launch<32>(g, s);
    case 64: return launch<64>(g, s);
    default: return launch<128>(g, s);
  }
}

}  // namespace

size_t attn_grad_ws_bytes(int64_t tokens, int64_t k_tokens, int B, int Hq, int Hkv, int d, int dtype) {
  const size_t blocks = static_cast<size_t>(tokens / kSumRows + B) * Hq, sums = blocks * (2 * kSumRows * sizeof(float));
  return 256 + sums + (dtype == FALCON_BF16 ? blocks * kImageBytes : attn_grad_tc32_ws_bytes(tokens, k_tokens, B, Hq, Hkv, d));
}

int launch_attn_grad(const GradArgs& args, int dtype, cudaStream_t s) {
  if (dtype == FALCON_F32) return launch_attn_grad_tc32(args, s);
  GradArgs g = args;
  g.images = attn_grad_tc_supported(g, dtype) ? reinterpret_cast<uint8_t*>(g.sums + row_sums(g.blocks, g.a.Hq, 0)) : nullptr;
  return launch_bf16(g, s);
}

}  // namespace falcon
