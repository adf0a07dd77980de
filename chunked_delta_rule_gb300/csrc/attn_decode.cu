// Attention of one token per sequence over the paged 8-bit cache.
//
//   s_j = scale q . (2^ek Kc_j),  o = sum_j exp(s_j) 2^ev Vc_j / sum_j exp(s_j)
//
// Memory bound: the codes are read once, 2 d bytes a key and key head, so
// everything between the load and the sums has to keep up with HBM.  The
// products run on warp-level MMAs (m16n8k16, half inputs, fp32 sums): e4m3
// codes are exact in half, and the up to 8 query heads of a key head are the
// narrow side, S^T = K Q^T (16 keys x 8 heads) and O^T = V^T P^T (16 dims x 8
// heads), so heads that a group lacks cost little.  A tcgen05 tile has 64 or
// 128 rows on its wide side and would need the codes widened in shared
// memory first, for a product that is far from being the bound.
//
// A warp takes 16-key tiles of one page; each lane fetches exactly the bytes
// that its fragments need (cp.async into a ring of its own in shared memory,
// read back without bank conflicts and without any barrier):
//   K: keys r and r + 8 (r = lane / 4), the lane's quarter of the head dim;
//      the order of the dims within the sum is free, so that is contiguous
//   V: keys 2c, 2c+1, 2c+8, 2c+9 (c = lane % 4), the lane group's eighth of
//      the head dim; pairs of keys are interleaved with byte permutes
// Queries are scaled by a power of two for each head to at most 2 in
// magnitude before they become halves: bf16 queries are then exact, up to
// elements 2^-22 below the largest.  fp32 queries and weights are split in two
// halves each.  Weights p = 2^(s - m) carry the page's V scale relative to
// the largest one seen, 2^(ev - E); the running reference m moves only when a
// score passes it by more than 8, so most tiles need no exchange between lanes.
//
// Long sequences are cut in chunks of keys, one CTA each (four warps take
// their tiles in turn and join in shared memory); a second kernel joins the
// chunks of a sequence.

#include "attn.cuh"
#include "tc_util.cuh"

namespace falcon {
namespace {

constexpr int kWarps = 4;
constexpr float kSlack = 8.f;       // scores may pass the reference by 2^8 ...
constexpr int kHeadroom = 6;        // ... and weights are kept 2^6 up: 2^14 < 65504

template <int D>
struct Tile {
  static constexpr int kKeys = D == 128 ? 16 : 32;            // keys of a stage
  static constexpr int kSub = kKeys / 16;
  static constexpr int kKSize = D >= 64 ? 16 : D / 4;         // bytes of one K load
  static constexpr int kKLoads = D == 128 ? 2 : 1;            // per key
  static constexpr int kVSize = D == 16 ? 4 : D / 8;          // bytes of one V load
  static constexpr int kStage = kSub * (2 * kKLoads * kKSize + 4 * kVSize) * 32;  // bytes a warp
  static constexpr int kStages = 4;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <int N>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool live) {
  const int n = live ? N : 0;  // bytes past n are filled with zeros
  if (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(n) : "memory");
}
template <int N>
__device__ __forceinline__ void lds(uint32_t src, uint32_t (&w)[N / 4]) {
  if constexpr (N == 16)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(src));
  else if constexpr (N == 8)
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(src));
  else
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(src));
}
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// NP: halves that an fp32 factor is split into (1 for bf16 inputs).
template <int NP>
__device__ __forceinline__ void split2(float lo, float hi, uint32_t (&out)[NP]) {
  out[0] = half2_bits(lo, hi);
  if (NP == 2) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&out[0]));
    out[NP - 1] = half2_bits(lo - f.x, hi - f.y);
  }
}

struct DecodePlan {
  int groups;   // groups of query heads for each key head
  int per;      // query heads of a group (the last one may hold fewer)
  int chunk;    // keys of a CTA
  int chunks;   // CTAs of a sequence and group
};

// T: dtype of q and o; NG: groups of 8 query heads that a warp takes at once
template <typename T, int D, int NG>
__global__ void __launch_bounds__(kWarps * 32) attn_decode_kernel(DecodeArgs a, DecodePlan pl, float* part_o,
                                                                 float2* part_ml) {
  using L = Tile<D>;
  constexpr int NP = sizeof(T) == 4 ? 2 : 1;
  constexpr int KS = D / 16;             // 16-wide steps of the head dim
  constexpr int KW = L::kKSize / 4, VW = L::kVSize / 4;
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, tig = lane & 3;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  int64_t it = blockIdx.x;
  const int c = static_cast<int>(it % pl.chunks);
  it /= pl.chunks;
  const int grp = static_cast<int>(it % pl.groups);
  it /= pl.groups;
  const int hk = static_cast<int>(it % a.Hkv);
  const int64_t b = it / a.Hkv;
  const int G = a.Hq / a.Hkv, g0 = grp * pl.per, heads = min(pl.per, G - g0);
  const int h0 = hk * G + g0;
  const int64_t cap = min(static_cast<int64_t>(a.max_k), static_cast<int64_t>(a.max_pages) * a.page);
  const int len = static_cast<int>(max(min(static_cast<int64_t>(a.lens[b]), cap), static_cast<int64_t>(0)));
  const int first = c * pl.chunk, end = min(len, first + pl.chunk);  // this CTA's keys
  if (first >= end && c > 0) return;

  // queries: a power of two brings the largest magnitude of a head into [1, 2)
  uint32_t qf[NG][NP][KS][2];
  float hs[NG][2];  // scale of the scores of heads 2 tig, 2 tig + 1 (log2 units)
#pragma unroll
  for (int n = 0; n < NG; ++n) {
    const int h = n * 8 + gid;
    const T* q = static_cast<const T*>(a.q.p) + b * a.q.stride + static_cast<int64_t>(h0 + (h < heads ? h : 0)) * D;
    float x[KS][4], top = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d = (ks / 4) * 64 + (D < 64 ? D / 4 : 16) * tig + 4 * (ks % 4) + i;
        x[ks][i] = h < heads ? to_f32(q[d]) : 0.f;
        const float m = fabsf(x[ks][i]);
        if (m <= 3.402823466e38f) top = fmaxf(top, m);
      }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int e = max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -126);  // 2^e <= top < 2^(e+1)
    const float up0 = exp2i(-e / 2), up1 = exp2i(-e - (-e / 2));
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t f[NP];
        split2<NP>(x[ks][2 * i] * up0 * up1, x[ks][2 * i + 1] * up0 * up1, f);
#pragma unroll
        for (int p = 0; p < NP; ++p) qf[n][p][ks][i] = f[p];
      }
    const float down = exp2i(e) * a.scale * kLog2e;
#pragma unroll
    for (int i = 0; i < 2; ++i) hs[n][i] = __shfl_sync(0xffffffffu, down, (2 * tig + i) * 4);
  }

  // running reference and sum of the heads 2 tig, 2 tig + 1, and O^T
  float m[NG][2], l[NG][2], o[NG][KS][4];
#pragma unroll
  for (int n = 0; n < NG; ++n) {
#pragma unroll
    for (int i = 0; i < 2; ++i) m[n][i] = -INFINITY, l[n][i] = 0.f;
#pragma unroll
    for (int j = 0; j < KS; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[n][j][i] = 0.f;
  }
  int E = -1000;  // largest V exponent so far

  // pages of this chunk: lane i holds page (base + i)'s number and scales
  const int page_shift = 31 - __clz(a.page);
  const int32_t* table = a.blocks + b * a.max_pages;
  int base = -64, pg = -1;
  auto load_pages = [&](int at) {
    base = at;
    const int64_t col = static_cast<int64_t>(at) + lane;
    pg = col < a.max_pages && (col << page_shift) < end ? table[col] : -1;
    if (pg < 0 || pg >= a.num_pages) pg = -1;
  };
  // scales are kept apart from the page numbers: the ring runs ahead of the products
  int sbase = -64;
  uint32_t sbytes = 0;  // K scale | V scale << 8, 0x10000: no such page
  auto load_scales = [&](int at) {
    sbase = at;
    const int64_t col = static_cast<int64_t>(at) + lane;
    int p = col < a.max_pages && (col << page_shift) < end ? table[col] : -1;
    if (p < 0 || p >= a.num_pages) {
      sbytes = 0x10000u;
    } else {
      const int64_t ph = static_cast<int64_t>(p) * a.Hkv + hk;
      sbytes = a.cache.k_scale[ph] | (static_cast<uint32_t>(a.cache.v_scale[ph]) << 8);
    }
  };

  const uint32_t ring = tc::smem_u32(smem) + warp * (L::kStages * L::kStage);
  const int tiles = (end - first + L::kKeys - 1) / L::kKeys;
  auto fetch = [&](int tile, int stage) {
    const uint32_t dst0 = ring + stage * L::kStage;
#pragma unroll
    for (int s = 0; s < L::kSub; ++s) {
      const int t = first + tile * L::kKeys + s * 16, col = t >> page_shift;
      if (tile < tiles && col - base >= 32) load_pages(col);
      const int p = __shfl_sync(0xffffffffu, pg, (col - base) & 31);
      const bool some = tile < tiles && p >= 0;
      const int64_t row = ((static_cast<int64_t>(some ? p : 0) * a.Hkv + hk) << page_shift) + (t & (a.page - 1));
      uint32_t dst = dst0 + s * (L::kStage / L::kSub);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int key = gid + 8 * r;
        const uint8_t* src = a.cache.k + (row + key) * D + tig * L::kKSize;
#pragma unroll
        for (int i = 0; i < L::kKLoads; ++i) {
          cp_async<L::kKSize>(dst + lane * L::kKSize, src + i * 64, some && t + key < end);
          dst += 32 * L::kKSize;
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int key = 2 * tig + (r & 1) + 8 * (r >> 1);
        const uint8_t* src = a.cache.v + (row + key) * D + (D == 16 ? (gid >> 1) * 4 : gid * L::kVSize);
        cp_async<L::kVSize>(dst + lane * L::kVSize, src, some && t + key < end);
        dst += 32 * L::kVSize;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  // this warp's tiles: warp, warp + kWarps, ...
#pragma unroll
  for (int i = 0; i < L::kStages - 1; ++i) fetch(warp + i * kWarps, i);
  load_scales(first >> page_shift);
  int stage = 0;
  for (int tile = warp; tile < tiles; tile += kWarps) {
    asm volatile("cp.async.wait_group %0;" ::"n"(L::kStages - 2) : "memory");
    const uint32_t src0 = ring + stage * L::kStage;
    // scores of the stage's 16-key tiles, two sums each for short chains
    float sc[L::kSub][NG][4];
    uint32_t bytes[L::kSub];
    bool past = false;
    int evmax = E;
#pragma unroll
    for (int sub = 0; sub < L::kSub; ++sub) {
      const int t = first + tile * L::kKeys + sub * 16, col = t >> page_shift;
      if (t < end && col - sbase >= 32) load_scales(col);
      bytes[sub] = __shfl_sync(0xffffffffu, sbytes, (col - sbase) & 31);
      const bool some = t < end && !(bytes[sub] & 0x10000u);
      if (!some) bytes[sub] = 0;  // zeros in the ring, weights 0, the smallest V scale
      const uint32_t src = src0 + sub * (L::kStage / L::kSub);
      float s[NG][2][4];
#pragma unroll
      for (int n = 0; n < NG; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[n][0][i] = s[n][1][i] = 0.f;
#pragma unroll
      for (int ld = 0; ld < L::kKLoads; ++ld) {
        uint32_t k0[KW], k1[KW];
        lds<L::kKSize>(src + (ld * 32 + lane) * L::kKSize, k0);
        lds<L::kKSize>(src + ((L::kKLoads + ld) * 32 + lane) * L::kKSize, k1);
#pragma unroll
        for (int j = 0; j < KW; ++j) {
          const uint32_t a0 = e4m3x2_to_half2(k0[j] & 0xFFFFu), a2 = e4m3x2_to_half2(k0[j] >> 16);
          const uint32_t a1 = e4m3x2_to_half2(k1[j] & 0xFFFFu), a3 = e4m3x2_to_half2(k1[j] >> 16);
#pragma unroll
          for (int n = 0; n < NG; ++n)
#pragma unroll
            for (int p = 0; p < NP; ++p)
              mma_f16(s[n][j & 1], a0, a1, a2, a3, qf[n][p][ld * KW + j][0], qf[n][p][ld * KW + j][1]);
        }
      }
      const float ks = e8m0(bytes[sub] & 0xFFu);
      const bool in0 = some && t + gid < end, in1 = some && t + gid + 8 < end;
#pragma unroll
      for (int n = 0; n < NG; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float f = hs[n][i] * ks;
          sc[sub][n][i] = in0 ? (s[n][0][i] + s[n][1][i]) * f : -INFINITY;
          sc[sub][n][2 + i] = in1 ? (s[n][0][2 + i] + s[n][1][2 + i]) * f : -INFINITY;
          past |= fmaxf(sc[sub][n][i], sc[sub][n][2 + i]) > m[n][i] + kSlack;
        }
      evmax = max(evmax, static_cast<int>(bytes[sub] >> 8) - 127);
    }
    if (__any_sync(0xffffffffu, past)) {  // move the reference to the maximum
#pragma unroll
      for (int n = 0; n < NG; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float x = m[n][i];
#pragma unroll
          for (int sub = 0; sub < L::kSub; ++sub) x = fmaxf(x, fmaxf(sc[sub][n][i], sc[sub][n][2 + i]));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          const float f = x == -INFINITY ? 1.f : ex2(m[n][i] - x);
          m[n][i] = x;
          l[n][i] *= f;
#pragma unroll
          for (int j = 0; j < KS; ++j) o[n][j][i] *= f, o[n][j][2 + i] *= f;
        }
    }
    if (evmax > E) {  // sums so far in units of the new, larger V scale
      const float f = exp2i(max(E - evmax, -149));
      E = evmax;
#pragma unroll
      for (int n = 0; n < NG; ++n)
#pragma unroll
        for (int j = 0; j < KS; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[n][j][i] *= f;
    }
#pragma unroll
    for (int sub = 0; sub < L::kSub; ++sub) {
      const float vs = exp2i(max(static_cast<int>(bytes[sub] >> 8) - 127 - E + kHeadroom, -126));
      uint32_t pb[NG][NP][2];
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        float p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float ref = m[n][i & 1];
          p[i] = ex2(sc[sub][n][i] - (ref == -INFINITY ? 0.f : ref));
        }
        l[n][0] += p[0] + p[2];
        l[n][1] += p[1] + p[3];
        uint32_t f0[NP], f1[NP];
        split2<NP>(p[0] * vs, p[1] * vs, f0);
        split2<NP>(p[2] * vs, p[3] * vs, f1);
#pragma unroll
        for (int x = 0; x < NP; ++x) {
          pb[n][x][0] = transpose8x8(f0[x]);
          pb[n][x][1] = transpose8x8(f1[x]);
        }
      }
      const uint32_t vsrc = src0 + sub * (L::kStage / L::kSub) + 2 * L::kKLoads * 32 * L::kKSize;
      uint32_t v[4][VW];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        lds<L::kVSize>(vsrc + (r * 32 + lane) * L::kVSize, v[r]);
        if (D == 16) v[r][0] >>= (gid & 1) * 16;
      }
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        const uint32_t sel = (j & 1) ? 0x7362u : 0x5140u;
        const uint32_t lo = __byte_perm(v[0][j / 2], v[1][j / 2], sel), hi = __byte_perm(v[2][j / 2], v[3][j / 2], sel);
        const uint32_t a0 = e4m3x2_to_half2(lo & 0xFFFFu), a1 = e4m3x2_to_half2(lo >> 16);
        const uint32_t a2 = e4m3x2_to_half2(hi & 0xFFFFu), a3 = e4m3x2_to_half2(hi >> 16);
#pragma unroll
        for (int n = 0; n < NG; ++n)
#pragma unroll
          for (int x = 0; x < NP; ++x) mma_f16(o[n][j], a0, a1, a2, a3, pb[n][x][0], pb[n][x][1]);
      }
    }
    fetch(tile + (L::kStages - 1) * kWarps, (stage + L::kStages - 1) % L::kStages);
    stage = (stage + 1) % L::kStages;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");

  // join the warps: o, m, l of each in shared memory, then a dim a thread
  constexpr int H8 = NG * 8, LD = D + 4;
  __syncthreads();
  float* so = reinterpret_cast<float*>(smem);
  float2* sml = reinterpret_cast<float2*>(so + kWarps * H8 * LD);
  const float unit = exp2i(max(min(E - kHeadroom, 127), -149));
#pragma unroll
  for (int n = 0; n < NG; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float x = l[n][i];
      x += __shfl_xor_sync(0xffffffffu, x, 4);
      x += __shfl_xor_sync(0xffffffffu, x, 8);
      x += __shfl_xor_sync(0xffffffffu, x, 16);
      const int h = n * 8 + 2 * tig + i;
      if (gid == 0) sml[warp * H8 + h] = make_float2(m[n][i], x);
      float* row = so + (warp * H8 + h) * LD;
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        row[gid * (D / 8) + 2 * j] = o[n][j][i] * unit;
        row[gid * (D / 8) + 2 * j + 1] = o[n][j][2 + i] * unit;
      }
    }
  __syncthreads();
  const bool whole = len <= pl.chunk;  // this CTA holds the sequence's every key
  for (int i = threadIdx.x; i < heads * D; i += kWarps * 32) {
    const int h = i / D, d = i % D;
    float top = -INFINITY, sum = 0.f, acc = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sml[w * H8 + h].x);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 x = sml[w * H8 + h];
      const float f = x.x == -INFINITY ? (x.y == 0.f ? 0.f : 1.f) : ex2(x.x - top);
      sum += x.y * f;
      acc += so[(w * H8 + h) * LD + d] * f;
    }
    const int64_t bh = b * a.Hq + h0 + h;
    if (whole) {
      T* out = static_cast<T*>(a.o.p) + b * a.o.stride + static_cast<int64_t>(h0 + h) * D;
      out[d] = from_f32<T>(sum == 0.f ? 0.f : acc / sum);
      if (a.lse && d == 0) a.lse[bh] = sum == 0.f ? -INFINITY : ((top == -INFINITY ? 0.f : top) + log2f(sum)) * kLn2;
    } else {
      part_o[(bh * pl.chunks + c) * D + d] = acc;
      if (d == 0) part_ml[bh * pl.chunks + c] = make_float2(top, sum);
    }
  }
}

// Joins the chunks of a sequence: one CTA per query head; D / 4 lanes take the
// head's dims, the groups of lanes the chunks in turn.
template <typename T, int D>
__global__ void __launch_bounds__(256) attn_decode_join_kernel(DecodeArgs a, DecodePlan pl, const float* part_o,
                                                               const float2* part_ml) {
  constexpr int W = D / 4, NGR = 256 / W;
  __shared__ float4 so[NGR][W];
  __shared__ float2 sml[NGR];
  const int w = threadIdx.x % W, g = threadIdx.x / W;
  const int64_t bh = blockIdx.x, b = bh / a.Hq;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int h = static_cast<int>(bh % a.Hq);
  const int64_t cap = min(static_cast<int64_t>(a.max_k), static_cast<int64_t>(a.max_pages) * a.page);
  const int len = static_cast<int>(min(static_cast<int64_t>(a.lens[b]), cap));
  if (len <= pl.chunk) return;  // written by its only CTA
  const int n = (len + pl.chunk - 1) / pl.chunk;
  const float2* ml = part_ml + bh * pl.chunks;
  const float4* po = reinterpret_cast<const float4*>(part_o + bh * pl.chunks * D);
  float top = -INFINITY, sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = g; i < n; i += NGR) top = fmaxf(top, ml[i].x);
#pragma unroll 4
  for (int i = g; i < n; i += NGR) {
    const float2 x = ml[i];
    const float4 v = po[static_cast<int64_t>(i) * W + w];
    const float f = x.x == -INFINITY ? (x.y == 0.f ? 0.f : 1.f) : ex2(x.x - top);
    sum += x.y * f;
    acc.x += v.x * f, acc.y += v.y * f, acc.z += v.z * f, acc.w += v.w * f;
  }
  so[g][w] = acc;
  if (w == 0) sml[g] = make_float2(top, sum);
  __syncthreads();
  if (threadIdx.x >= D) return;
  const int d = threadIdx.x;
  top = -INFINITY, sum = 0.f;
  float y = 0.f;
#pragma unroll
  for (int i = 0; i < NGR; ++i) top = fmaxf(top, sml[i].x);
#pragma unroll
  for (int i = 0; i < NGR; ++i) {
    const float2 x = sml[i];
    const float f = x.x == -INFINITY ? (x.y == 0.f ? 0.f : 1.f) : ex2(x.x - top);
    sum += x.y * f;
    y += reinterpret_cast<const float*>(so[i])[d] * f;
  }
  T* out = static_cast<T*>(a.o.p) + b * a.o.stride + static_cast<int64_t>(h) * D;
  out[d] = from_f32<T>(sum == 0.f ? 0.f : y / sum);
  if (a.lse && d == 0) a.lse[bh] = sum == 0.f ? -INFINITY : ((top == -INFINITY ? 0.f : top) + log2f(sum)) * kLn2;
}

// Keys of a CTA: as many CTAs as the card holds at a time (two 131072-key
// sequences: 48 us, with twice as many 61), at least 256 keys (the partial
// results of a chunk are then at most a sixteenth of what it reads), whole
// 128-key pages.
DecodePlan decode_plan(int B, int Hq, int Hkv, int max_k) {
  DecodePlan p;
  const int G = Hq / Hkv;
  p.per = G <= 8 ? 8 : 16;
  p.groups = (G + p.per - 1) / p.per;
  const int64_t rows = static_cast<int64_t>(B) * Hkv * p.groups, want = 152 * 4;
  int64_t chunks = (want + rows - 1) / rows;
  int64_t chunk = (max_k + chunks - 1) / chunks;
  chunk = (chunk + 127) / 128 * 128;
  p.chunk = static_cast<int>(chunk < 256 ? 256 : chunk);
  p.chunks = max_k <= 0 ? 1 : static_cast<int>((static_cast<int64_t>(max_k) + p.chunk - 1) / p.chunk);
  return p;
}

template <typename T, int D, int NG>
int launch_decode(const DecodeArgs& a, const DecodePlan& p, cudaStream_t s) {
  using L = Tile<D>;
  constexpr size_t ring = static_cast<size_t>(kWarps) * L::kStages * L::kStage;
  constexpr size_t join = static_cast<size_t>(kWarps) * NG * 8 * ((D + 4) * 4 + 8);
  constexpr size_t smem = ring > join ? ring : join;
  const int64_t n = static_cast<int64_t>(a.B) * a.Hkv * p.groups * p.chunks;
  if (n > INT32_MAX) return FALCON_ERR_UNSUPPORTED;
  const auto kern = attn_decode_kernel<T, D, NG>;
  if (!set_smem_limit(reinterpret_cast<const void*>(kern), smem)) return FALCON_ERR_CUDA;
  float2* ml = static_cast<float2*>(a.ws);
  float* po = reinterpret_cast<float*>(ml + align_up(static_cast<size_t>(a.B) * a.Hq * p.chunks, 32));
  kern<<<static_cast<unsigned>(n), kWarps * 32, smem, s>>>(a, p, po, ml);
  if (cudaGetLastError() != cudaSuccess) return FALCON_ERR_CUDA;
  if (p.chunks == 1) return FALCON_OK;
  FwdArgs fa = {};
  fa.stream = s;
  const int64_t rows = static_cast<int64_t>(a.B) * a.Hq;
  if (rows > INT32_MAX) return FALCON_ERR_UNSUPPORTED;
  return tcu::launch_overlapped(fa, attn_decode_join_kernel<T, D>, dim3(static_cast<unsigned>(rows)), dim3(256), 0, a, p, static_cast<const float*>(po), static_cast<const float2*>(ml));
}
template <typename T, int D>
int launch_decode_g(const DecodeArgs& a, const DecodePlan& p, cudaStream_t s) {
  return p.per == 8 ? launch_decode<T, D, 1>(a, p, s) : launch_decode<T, D, 2>(a, p, s);
}
template <typename T>
int launch_decode_d(const DecodeArgs& a, const DecodePlan& p, cudaStream_t s) {
  switch (a.d) {
    case 16: return launch_decode_g<T, 16>(a, p, s);
    case 32: return launch_decode_g<T, 32>(a, p, s);
    case 64: return launch_decode_g<T, 64>(a, p, s);
    default: return launch_decode_g<T, 128>(a, p, s);
  }
}

}  // namespace

size_t attn_decode_ws_bytes(int B, int Hq, int Hkv, int d, int, int max_k) {
  const DecodePlan p = decode_plan(B, Hq, Hkv, max_k);
  if (p.chunks == 1) return 256;
  const size_t n = static_cast<size_t>(B) * Hq * p.chunks;
  return align_up(n, 32) * sizeof(float2) + n * d * sizeof(float);
}

int launch_attn_decode(const DecodeArgs& a, int dtype, cudaStream_t s) {
  const DecodePlan p = decode_plan(a.B, a.Hq, a.Hkv, a.max_k);
  return dtype == FALCON_BF16 ? launch_decode_d<__nv_bfloat16>(a, p, s) : launch_decode_d<float>(a, p, s);
}

}  // namespace falcon
