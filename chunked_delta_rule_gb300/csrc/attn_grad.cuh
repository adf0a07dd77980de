// Internals of the softmax-attention backward: resolved arguments, the rows' sums
// that the first kernel leaves in the workspace, and one row of a gradient by one
// warp, straight from the definition.
#pragma once

#include <algorithm>
#include <cmath>

#include "attn_row.cuh"
#include "tc_util.cuh"

namespace falcon {

// What a call needs.  `a` holds the forward's operands; a.o and a.lse are not set.
struct GradArgs {
  PromptArgs a;
  RowsIn o, d_o;
  const float* lse;
  const float* dlse;    // may be NULL
  RowsOut dq, dk, dv;   // dq.p, or dk.p and dv.p, may be NULL
  float* sums;          // in the workspace, see row_sums
  uint8_t* images;      // the same as bf16 operand tiles, see kImageBytes; NULL: not wanted
  int64_t blocks;       // of 128 rows of queries, of a head, counted over the packed sequences
};
size_t attn_grad_ws_bytes(int64_t tokens, int64_t k_tokens, int B, int Hq, int Hkv, int d, int dtype);
int launch_attn_grad(const GradArgs& g, int dtype, cudaStream_t s);
bool attn_grad_tc_supported(const GradArgs& g, int dtype);
int launch_attn_grad_tc(const GradArgs& g, cudaStream_t s);
int launch_attn_grad_dq_tc(const GradArgs& g, bool second, cudaStream_t s);
size_t attn_grad_tc32_ws_bytes(int64_t tokens, int64_t k_tokens, int B, int Hq, int Hkv, int d);
int launch_attn_grad_tc32(const GradArgs& g, cudaStream_t s);

// The rows of query block j (of 128, counted from cu_q[b] / 128 + b on for sequence b) and head h: 128 times the
// log sum of the scores (natural), then 128 times
// D = sum_c dO_c o_c - dlse.  Rows past the sequence and rows that see no key
// have log sum +inf: exp(score - log sum) = 0, no weight anywhere.
constexpr int kSumRows = 128;
__host__ __device__ __forceinline__ int64_t row_sums(int64_t blocks, int h, int64_t j) {
  return (static_cast<int64_t>(h) * blocks + j) * (2 * kSumRows);
}
// The same 128 rows as the B operand (16 columns, no swizzle: 8 rows x 16 bytes at (2 (row / 8) + half) 128) of one
// more step of the products Q K^T and dO V^T: columns 0 to 2 hold -log sum / scale in three bf16 parts, 4 to 6 hold -D.
// Against ones in those columns the products come out less them.
constexpr int kImageBytes = kSumRows * 32;
// first block of a sequence whose rows begin at q0
__device__ __forceinline__ int64_t first_block(int64_t q0, int b) { return q0 / kSumRows + b; }

// The kernels of a call overlap: the products' first kernel is launched while the rows' sums are formed, which it waits for
// before it reads them; the second one (the two do not depend on one another) once the last CTAs of the first have
// begun, so that its CTAs take the SMs as these fall free.  It ends no sooner than the first: a thread of its last CTA
// waits for that.
// The second one reads what the sums' kernel wrote too.  To wait for it as the first one does would be to wait for the first
// one's end, so it goes by this: it begins when every CTA of the first has waited, that is after the sums' kernel has ended and
// its writes are in memory; and it reads them past the L1 cache (load_past_l1, bulk copies), which might hold older lines.
// The programming model promises the sums to a grid that waits alone: this is what the hardware does, not what a document says.
// (Fences in both kernels, which leave the same gap: 1 us a call, 13.9 us for 12.3 at 77 tokens of 12 heads of 64.)
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ float load_past_l1(const float* p) { return __ldcg(p); }
inline cudaLaunchAttribute overlap_attribute() {
  cudaLaunchAttribute a;
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  return a;
}
inline cudaLaunchAttribute cluster_attribute(int ctas) {
  cudaLaunchAttribute a;
  a.id = cudaLaunchAttributeClusterDimension;
  a.val.clusterDim.x = static_cast<unsigned>(ctas);
  a.val.clusterDim.y = a.val.clusterDim.z = 1;
  return a;
}
// packed_block by a whole warp: 32 sequences a look
__device__ __forceinline__ int2 find_block(const int32_t* cu, int B, int rows, int j) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B;
  while (n > 1) {
    const int step = (n + 31) / 32, i = lo + lane * step;
    const bool begun = lane * step < n && static_cast<int64_t>(__ldg(cu + min(i, B))) / rows + i <= j;
    const int c = max(__popc(__ballot_sync(0xffffffffu, begun)) - 1, 0);
    lo += c * step;
    n = min(step, n - c * step);
  }
  const int64_t first = static_cast<int64_t>(__ldg(cu + lo)) / rows + lo;
  const int64_t next = static_cast<int64_t>(__ldg(cu + lo + 1)) / rows + lo + 1;
  const int64_t row = (next - 1 - j) * rows;
  return make_int2(lo, j < first || row > INT32_MAX ? -1 : static_cast<int>(row));
}

// Sums over the lanes, a few at a time.
template <int N>
__device__ __forceinline__ void lane_sums(float (&x)[N]) {
#pragma unroll
  for (int s = 16; s; s >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], s);
}

// dq (lane t's dims t, t + 32, ...) of one query over the first n keys.  Ends where every dim is NaN: they stay so.
template <typename T, int D>
__device__ __noinline__ void grad_query_row(const T* q, const T* d_o, float lse, float delta, const T* k,
                                            int64_t k_stride, const T* v, int64_t v_stride, int n, int d, float scale,
                                            float (&out)[4]) {
  constexpr int J = (D + 31) / 32, kBatch = 4;
  const int lane = threadIdx.x & 31;
  float qv[J], gv[J];
  int at[J];
#pragma unroll
  for (int j = 0; j < 4; ++j) out[j] = 0.f;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const bool in = lane + 32 * j < d;
    at[j] = min(lane + 32 * j, d - 1);
    qv[j] = in ? to_f32(q[at[j]]) : 0.f;
    gv[j] = in ? to_f32(d_o[at[j]]) : 0.f;
  }
  if (lse == INFINITY) return;
  for (int t = 0; t < n; t += kBatch) {
    float kt[kBatch][J], s[2 * kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      s[u] = s[kBatch + u] = 0.f;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const bool in = lane + 32 * j < d;
        kt[u][j] = in ? to_f32(k[min(t + u, n - 1) * k_stride + at[j]]) : 0.f;
        s[u] = fmaf(qv[j], kt[u][j], s[u]);
        s[kBatch + u] = fmaf(gv[j], in ? to_f32(v[min(t + u, n - 1) * v_stride + at[j]]) : 0.f, s[kBatch + u]);
      }
    }
    lane_sums(s);
    bool nan = true;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (t + u >= n) break;
      const float ds = expf(fmaf(s[u], scale, -lse)) * (s[kBatch + u] - delta) * scale;
#pragma unroll
      for (int j = 0; j < J; ++j) out[j] = fmaf(ds, kt[u][j], out[j]);
    }
#pragma unroll
    for (int j = 0; j < J; ++j) nan = nan && (lane + 32 * j >= d || out[j] != out[j]);
    if (__all_sync(0xffffffffu, nan)) break;
  }
}

// dk and dv of one key, over the `heads` query heads of its group and the queries [i0, i1) of its sequence, whose rows
// begin at q and d_o (of the group's first head); sums: of that head's first block, `blocks` blocks a head.
template <typename T, int D>
__device__ __noinline__ void grad_key_row(const T* k, const T* v, const T* q, int64_t q_stride, const T* d_o,
                                          int64_t o_stride, const float* sums, int64_t blocks, int heads, int i0, int i1,
                                          int d, float scale, float (&dk)[4], float (&dv)[4]) {
  constexpr int J = (D + 31) / 32, kBatch = 4;
  const int lane = threadIdx.x & 31;
  float kv[J], vv[J];
  int at[J];
#pragma unroll
  for (int j = 0; j < 4; ++j) dk[j] = dv[j] = 0.f;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const bool in = lane + 32 * j < d;
    at[j] = min(lane + 32 * j, d - 1);
    kv[j] = in ? to_f32(k[at[j]]) : 0.f;
    vv[j] = in ? to_f32(v[at[j]]) : 0.f;
  }
  for (int h = 0; h < heads; ++h, q += d, d_o += d, sums += blocks * (2 * kSumRows)) {
    for (int t = i0; t < i1; t += kBatch) {
      float qt[kBatch][J], gt[kBatch][J], s[2 * kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        s[u] = s[kBatch + u] = 0.f;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const bool in = lane + 32 * j < d;
          qt[u][j] = in ? to_f32(q[min(t + u, i1 - 1) * q_stride + at[j]]) : 0.f;
          gt[u][j] = in ? to_f32(d_o[min(t + u, i1 - 1) * o_stride + at[j]]) : 0.f;
          s[u] = fmaf(kv[j], qt[u][j], s[u]);
          s[kBatch + u] = fmaf(vv[j], gt[u][j], s[kBatch + u]);
        }
      }
      lane_sums(s);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int i = t + u;
        if (i >= i1) break;
        const float* row = sums + static_cast<int64_t>(i / kSumRows) * (2 * kSumRows) + i % kSumRows;
        const float lse = row[0];
        if (lse == INFINITY) continue;
        const float p = expf(fmaf(s[u], scale, -lse)), ds = p * (s[kBatch + u] - row[kSumRows]) * scale;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          dv[j] = fmaf(p, gt[u][j], dv[j]);
          dk[j] = fmaf(ds, qt[u][j], dk[j]);
        }
      }
      bool nan = true;
#pragma unroll
      for (int j = 0; j < J; ++j) nan = nan && (lane + 32 * j >= d || (dk[j] != dk[j] && dv[j] != dv[j]));
      if (__all_sync(0xffffffffu, nan)) return;
    }
  }
}

// 32-lane rows of d dims to global memory
template <typename T, int D>
__device__ __forceinline__ void store_row(T* out, const float (&x)[4], int d) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < (D + 31) / 32; ++j)
    if (lane + 32 * j < d) out[lane + 32 * j] = from_f32<T>(x[j]);
}

// ---------------------------------------------------------------- a block's dK and dV by a cluster of CTAs
// The grid of fp32's dQ, blocks of 128 rows, as prompt_grid: but a block without rows costs a CTA that has an SM to itself its
// start, so that the packed grid is taken from an eighth more blocks on.
inline PromptGrid query_grid(const PromptArgs& a) {
  const int64_t each = (static_cast<int64_t>(a.max_q) + kSumRows - 1) / kSumRows * a.B, packed = a.tokens / kSumRows + a.B;
  return each > packed + packed / 8 ? PromptGrid{packed, true} : PromptGrid{each, false};
}
// How many CTAs take a block of 128 keys together.  In units of a tile of N queries: the call takes as long as its longest
// CTA (the keys that every query of all heads sees; sequences taken as half as long again as their mean) or as all
// tiles of both kernels dealt out over `slots` CTAs, a tile of dQ at 0.7 of one of dK and dV.  A CTA costs `begin` tiles to begin
// and end, one of a cluster `join`.
// (us, unsplit and 2, 4, 8 CTAs: 2048 tokens, 12 heads of 64: 41, 52; 2048 tokens, 16 over 4 heads of 128: 93, 60, 71;
// 4 x 300 after 500 keys, 8 over 1 heads of 32: 41, 31, 25, 21; 8 x 300: 49, 37, 34, 35.)
inline int keys_split(const PromptArgs& a, int N, int slots, double begin, double join) {
  const double lq = static_cast<double>(a.tokens) / a.B, lk = static_cast<double>(a.k_tokens) / a.B;
  const double G = a.Hq / a.Hkv, longest = std::ceil((a.B > 1 ? 1.5 : 1.0) * lq / N) * G;
  const double seen = lk >= lq ? 1.0 - 0.5 * lq / lk : 0.5 * lk / lq;  // of all pairs
  const double blocks = std::ceil(lk / kSumRows) * a.B * a.Hkv;
  const double tiles = 1.7 * blocks * std::ceil(lq / N) * G * seen + begin * std::ceil(lq / kSumRows) * a.B * a.Hq;
  int split = 1;
  double best = std::max(longest + begin, (tiles + blocks * begin) / slots);
  for (int s = 2; s <= 8; s *= 2) {
    const double cost = std::max(longest / s + join, (tiles + blocks * s * join) / slots);
    if (cost < best) best = cost, split = s;
  }
  return split;
}
// every thread of the cluster's CTAs
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_smem(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 load_peer4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t load_peer(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
// This CTA's share of the rows of a block's dV and dK, added up over the SPLIT CTAs in their order; eight loads of a thread
// are under way at once (the CTAs' shared memory is far: one after another they took some 5 us).
template <typename T, int D, int THREADS, int SPLIT>
__device__ __forceinline__ void add_cluster(const GradArgs& g, uint32_t smem, uint32_t (&bad)[2][4], int rank, int row0,
                                            int rows, int64_t k0, int head, int d) {
  constexpr int kShare = kSumRows / SPLIT, kPieces = D / 4, kItems = 2 * kShare * kPieces / THREADS, U = 8 / SPLIT;
  static_assert(kItems * THREADS == 2 * kShare * kPieces && (kItems % U == 0 || kItems < U), "whole rounds");
  const int rs = rank * kShare;
  uint32_t peer[SPLIT];
#pragma unroll
  for (int s = 0; s < SPLIT; ++s) peer[s] = peer_smem(smem, s);
#pragma unroll 1
  for (int i0 = 0; i0 < kItems; i0 += U) {
    float4 y[U][SPLIT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u >= kItems) break;
      const int x = (i0 + u) * THREADS + threadIdx.x, c = x % kPieces, rr = rs + x / kPieces % kShare, out = x / kPieces / kShare;
      const uint32_t at = out * (kSumRows * D * 4) + rr * (D * 4) + ((c ^ (rr & 7)) << 4);
#pragma unroll
      for (int s = 0; s < SPLIT; ++s) y[u][s] = load_peer4(peer[s] + at);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u >= kItems) break;
      const int x = (i0 + u) * THREADS + threadIdx.x, c = x % kPieces, rr = rs + x / kPieces % kShare, out = x / kPieces / kShare;
      if (row0 + rr >= rows || 4 * c >= d) continue;  // out: dV, dK
      float4 sum = y[u][0];
#pragma unroll
      for (int s = 1; s < SPLIT; ++s) sum.x += y[u][s].x, sum.y += y[u][s].y, sum.z += y[u][s].z, sum.w += y[u][s].w;
      const float f = out ? g.a.scale : 1.f;
      sum.x *= f, sum.y *= f, sum.z *= f, sum.w *= f;
      const float rest = fmaf(sum.x, 0.f, fmaf(sum.y, 0.f, fmaf(sum.z, 0.f, sum.w * 0.f)));
      if (!(rest == 0.f)) atomicOr(&bad[out][rr >> 5], 1u << (rr & 31));
      const RowsOut& to = out ? g.dk : g.dv;
      T* dst = static_cast<T*>(to.p) + (k0 + row0 + rr) * to.stride + static_cast<int64_t>(head) * d + 4 * c;
      if constexpr (sizeof(T) == 2)
        *reinterpret_cast<uint2*>(dst) = make_uint2(tcu::pack_bf16(sum.x, sum.y), tcu::pack_bf16(sum.z, sum.w));
      else if (to.vec)
        *reinterpret_cast<float4*>(dst) = sum;
      else
        dst[0] = sum.x, dst[1] = sum.y, dst[2] = sum.z, dst[3] = sum.w;
    }
  }
}
// The sums of a block of 128 keys from the cluster's CTAs, which each left theirs in fp32 at `smem`: rows of dV, then of dK,
// D numbers each, 16-byte pieces swizzled by row.  By `THREADS` threads, all others of the CTA pass two cluster barriers
// meanwhile.  again(i, dk, dv): row i from the definition.
template <typename T, int D, int THREADS, typename F>
__device__ __forceinline__ void cluster_sums(const GradArgs& g, const uint8_t* smem, const uint32_t* failed,
                                             uint32_t (&bad)[2][4], int split, int rank, int row0, int rows, int64_t k0,
                                             int head, int d, F again) {
  const int tid = threadIdx.x;
  cluster_barrier();
  bool fine = true;
  for (int s = 0; s < split; ++s) fine = fine && load_peer(peer_smem(tc::smem_u32(failed), s)) == 0;
  if (fine) {
    const int share = kSumRows / split, rs = rank * share;
    const uint32_t at = tc::smem_u32(smem);
    if (split == 2) add_cluster<T, D, THREADS, 2>(g, at, bad, rank, row0, rows, k0, head, d);
    else if (split == 4) add_cluster<T, D, THREADS, 4>(g, at, bad, rank, row0, rows, k0, head, d);
    else add_cluster<T, D, THREADS, 8>(g, at, bad, rank, row0, rows, k0, head, d);
    tcu::named_bar(1, THREADS);
    for (int x = tid >> 5; x < 2 * share; x += THREADS / 32) {
      const int rr = rs + x % share, out = x / share;
      if (!(bad[out][rr >> 5] >> (rr & 31) & 1)) continue;
      float x1[4], x2[4];
      again(row0 + rr, x1, x2);
      const RowsOut& to = out ? g.dk : g.dv;
      store_row<T, D>(static_cast<T*>(to.p) + (k0 + row0 + rr) * to.stride + static_cast<int64_t>(head) * d, out ? x1 : x2, d);
    }
  }
  cluster_barrier();  // the others have read what lies here
}

}  // namespace falcon
