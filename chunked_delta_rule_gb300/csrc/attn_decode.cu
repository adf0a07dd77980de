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
// A producer warp brings 16-key tiles of K and V into a ring in shared memory
// (TMA, 128-byte swizzle where a row of keys is that wide) and runs ahead of
// the four consumer warps across rows of work; a tile goes to one warp:
//   K: a lane holds keys r and r + 8 (r = lane / 4, in an order that keeps the
//      reads free of bank conflicts) and its quarter of the head dim; the order of
//      the dims within a sum is free, so that is 16 neighbouring bytes
//   V: the keys of two columns of the weights (lane % 4), the lane group's eighth
//      of the head dim; pairs of keys are interleaved with byte permutes
// Queries are scaled by a power of two for each head to at most 2 in
// magnitude before they become halves: bf16 elements are then exact down to
// 2^-17 of the head's largest, below that off by 2^-25 of it at most.  fp32
// queries and weights are split in two halves each: 2^-22.
// Weights p = 2^(s - m) become halves (11 bits) relative to the largest one of
// their tile and head, a power of two found with three shuffles, and the tile's
// products are added to the fp32 sums times that power and the page's V scale: no
// weight and no V scale is lost to another tile's.  (Halves relative to what the warp
// had met before lose the bits of weights under 2^-20 of the largest, or values
// beside a page of a larger scale; they took 66 and 39 us where these take 70 and 40.)  Sums
// of their own for every tile are also what keeps fp32 results: the tensor cores
// cut their sums off, which adds up over the keys.  The running reference m moves
// only when a score passes it by more than 8.
//
// Every CTA gets the same number of keys (the lengths are known on the device
// only); a second kernel joins the rows that several CTAs share.
// Measured: 256 sequences of 410 .. 2048 keys, 16 / 4 heads of 128: 325 MB of
// codes in 70 us, 4.7 TB/s (about 4 us a row and CTA around the stream; fp32: 84 us);
// 2 of <= 131072 keys, 16 / 2 heads of 128: 40 us (fp32: 43); 1 x 777 keys: 10.2 us,
// the call.
// Waits are bounded and reported through the workspace's status word.

#include "attn.cuh"
#include "tc_util.cuh"

namespace falcon {
namespace {

constexpr int kWarps = 4;           // consumers
constexpr float kSlack = 8.f;       // scores (log2) may pass the reference by this
constexpr int kTop = 14;            // a tile's largest weight for a head lies in [2^14, 2^15) as a half (< 65504)

template <int D>
struct Tile {
  static constexpr int kSub = D == 128 ? 1 : 2;                // 16-key tiles of a warp and stage
  static constexpr int kKeys = 16 * kSub * kWarps;             // keys of a stage: the unit of work
  static constexpr int kBytes = 16 * D;                        // of a tile of K or V
  static constexpr int kKSize = D >= 64 ? 16 : D / 4;          // bytes of one K load
  static constexpr int kKLoads = D == 128 ? 2 : 1;             // per key
  static constexpr int kVSize = D == 16 ? 4 : D / 8;           // bytes of one V load
  static constexpr int kStage = kSub * kWarps * 2 * kBytes;    // bytes
  static constexpr int kStages = 3;
};

// CTAs that the registers of an SM hold
constexpr int ctas_of_sm(int elem, int d) { return d == 128 && elem == 4 ? 2 : 3; }

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
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
// Address of byte `off` of a tile: rows of 128 bytes, their 16-byte pieces
// swizzled by the row, where a tile has 8 of them; else as they come.
template <int D>
__device__ __forceinline__ uint32_t in_tile(uint32_t off) {
  return D >= 64 ? off ^ ((off >> 3) & 0x70) : off;
}
// Key of row r of a score tile.  With 128-byte keys the two keys that
// neighbouring lanes of a quarter-warp read have to differ in bit 2.
template <int D>
__device__ __forceinline__ int key_of(int r) {
  return D == 128 ? ((r & 1) << 2) | ((r >> 1) & 3) | (r & 8) : r;
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

// weight of a part (reference, sum) where the joint reference is `top`, and the
// log of the sum of exponentials
__device__ __forceinline__ float weight_of(float2 x, float top) {
  return x.x == -INFINITY ? (x.y == 0.f ? 0.f : 1.f) : ex2(x.x - top);
}
__device__ __forceinline__ float log_sum(float2 x) {
  return x.y == 0.f ? -INFINITY : ((x.x == -INFINITY ? 0.f : x.x) + log2f(x.y)) * kLn2;
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

// Work is counted in units of Tile<D>::kKeys keys, laid out by sequence, then
// key head and group.  direct: a CTA for each (sequence, key head, group).
// Otherwise CTA c of n (ctas, or as many as there are units) takes units
// [total c / n, total (c + 1) / n): it may end one row of units, take some whole
// and begin another.  Parts of rows go to slot 0 (its first row) or 1 (its
// last) of the CTA.
struct DecodePlan {
  int groups;   // groups of 8 query heads (the last one may hold fewer) for each key head
  int direct;
  int ctas;
};

__device__ __forceinline__ int cached_keys(const DecodeArgs& a, int64_t b) {
  const int64_t cap = min(static_cast<int64_t>(a.max_k), static_cast<int64_t>(a.max_pages) * a.page);
  return static_cast<int>(max(min(static_cast<int64_t>(a.lens[b]), cap), static_cast<int64_t>(0)));
}

// T: dtype of q and o
template <typename T, int D>
__global__ void __launch_bounds__((kWarps + 1) * 32, ctas_of_sm(sizeof(T), D))
    attn_decode_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const DecodeArgs a,
                       const DecodePlan pl, float* part_o, float2* part_ml, int* begun_in, int* ended_in, uint32_t* status,
                       uint64_t limit, int stall) {
  using L = Tile<D>;
  constexpr int NP = sizeof(T) == 4 ? 2 : 1;
  constexpr int KS = D / 16;             // 16-wide steps of the head dim
  constexpr int KW = L::kKSize / 4, VW = L::kVSize / 4;
  constexpr int H8 = 8, kFrag = KS * 4;  // heads of a group; sums of O^T that a lane holds
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = tcu::align1024(smem_raw);
  float* joint = reinterpret_cast<float*>(smem + L::kStages * L::kStage);      // [kWarps / 2][kFrag][32]
  float2* ml = reinterpret_cast<float2*>(joint + kWarps / 2 * kFrag * 32);     // [kWarps][H8]
  // scales of each tile of a stage: K | V << 8, or 0x10000: no such tile
  uint32_t* scales = reinterpret_cast<uint32_t*>(ml + kWarps * H8);            // [kStages][kSub * kWarps]
  __shared__ uint64_t full[L::kStages], empty[L::kStages], never;
  __shared__ int s_sum[kWarps], s_b, s_base;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, tig = lane & 3;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int R = a.Hkv * pl.groups;  // rows of units of a sequence
  const int G = a.Hq / a.Hkv;
  if (blockIdx.x == 0 && threadIdx.x == 0) atomicExch(status, 0u);  // before any wait of this call can run out
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kStages; ++i) {
      tc::mbar_init(&full[i], 1);
      tc::mbar_init(&empty[i], kWarps);
    }
    tc::mbar_init(&never, 1);
    tc::fence_mbar_init();
  }
  auto wait = [&](uint64_t* m, uint32_t parity) {
    if (tc::mbar_wait(m, parity, limit)) return true;
    atomicExch(status, tcu::kStatusTimeout);
    return false;
  };

  // where this CTA's units begin: sequence b, row r, unit `off` of it, `left` units to go
  int b, r, off = 0, keys;
  int64_t left;
  if (pl.direct) {
    b = static_cast<int>(blockIdx.x / R);
    r = static_cast<int>(blockIdx.x % R);
    keys = cached_keys(a, b);
    left = (keys + L::kKeys - 1) / L::kKeys;
    __syncthreads();
  } else {
    // units before each thread's share of the sequences
    const int share = (a.B + kWarps * 32 - 1) / (kWarps * 32), b0 = min(static_cast<int>(threadIdx.x) * share, a.B);
    const int b1 = warp < kWarps ? min(b0 + share, a.B) : b0;
    int sum = 0;
    for (int i = b0; i < b1; ++i) sum += (cached_keys(a, i) + L::kKeys - 1) / L::kKeys;
    int before = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += x;
    }
    if (lane == 31 && warp < kWarps) s_sum[warp] = before;
    if (threadIdx.x == 0) s_b = a.B;
    __syncthreads();
    before -= sum;
    int all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += s_sum[w];
      all += s_sum[w];
    }
    const int64_t total = static_cast<int64_t>(all) * R;
    const int64_t n_ctas = min(static_cast<int64_t>(pl.ctas), total), me = min(static_cast<int64_t>(blockIdx.x), n_ctas);
    const int64_t u0 = n_ctas ? total * me / n_ctas : 0, u1 = me < n_ctas ? total * (me + 1) / n_ctas : u0;
    left = u1 - u0;
    for (int i = b0; i < b1; ++i) {
      const int n = (cached_keys(a, i) + L::kKeys - 1) / L::kKeys;
      if (u0 >= static_cast<int64_t>(before) * R && u0 < static_cast<int64_t>(before + n) * R) s_b = i, s_base = before;
      before += n;
    }
    if (threadIdx.x == 0) begun_in[blockIdx.x] = -1;
    // sequences without keys
    for (int i = blockIdx.x; i < a.B; i += pl.ctas) {
      if (cached_keys(a, i) > 0) continue;
      for (int x = threadIdx.x; x < a.Hq * D; x += (kWarps + 1) * 32)
        static_cast<T*>(a.o.p)[i * a.o.stride + x] = from_f32<T>(0.f);
      if (a.lse)
        for (int x = threadIdx.x; x < a.Hq; x += (kWarps + 1) * 32) a.lse[static_cast<int64_t>(i) * a.Hq + x] = -INFINITY;
    }
    __syncthreads();
    if (left <= 0) return;
    b = s_b;
    keys = cached_keys(a, b);
    const int n = (keys + L::kKeys - 1) / L::kKeys;
    const int64_t in = u0 - static_cast<int64_t>(s_base) * R;
    r = static_cast<int>(in / n);
    off = static_cast<int>(in - static_cast<int64_t>(r) * n);
  }

  const int page_shift = 31 - __clz(a.page);
  int units = (keys + L::kKeys - 1) / L::kKeys;  // of the row
  int count = static_cast<int>(min(static_cast<int64_t>(units - off), left));  // of them this CTA's
  auto next_row = [&]() {
    off = 0;
    if (++r == R) {
      r = 0;
      do {
        keys = cached_keys(a, ++b);
      } while (keys == 0);
      units = (keys + L::kKeys - 1) / L::kKeys;
    }
    count = static_cast<int>(min(static_cast<int64_t>(units), left));
  };
  int stage = 0, phase = 0;
  auto next_stage = [&]() {
    if (++stage == L::kStages) stage = 0, phase ^= 1;
  };

  if (warp == kWarps) {
    // the producer: lane i brings tile i of each stage
    constexpr int kTiles = L::kSub * kWarps;
    bool ok = !stall || wait(&never, 0);
    int64_t n = 0;  // stages filled
    while (left > 0 && ok) {
      const int hk = r / pl.groups;
      const int32_t* table = a.blocks + static_cast<int64_t>(b) * a.max_pages;
      const int end = min(keys, (off + count) * L::kKeys);
      // lane i: number (-1: none) and scales of page (base + i), and of page (base + 32 + i), fetched long before use
      struct Page {
        int pg;
        uint32_t sc;
      };
      auto page_at = [&](int col) {
        Page x = {-1, 0x10000u};
        if (col < a.max_pages && (static_cast<int64_t>(col) << page_shift) < end) x.pg = table[col];
        if (x.pg < 0 || x.pg >= a.num_pages) {
          x.pg = -1;
        } else {
          const int64_t ph = static_cast<int64_t>(x.pg) * a.Hkv + hk;
          x.sc = a.cache.k_scale[ph] | (static_cast<uint32_t>(a.cache.v_scale[ph]) << 8);
        }
        return x;
      };
      int base = (off * L::kKeys) >> page_shift;
      Page now = page_at(base + lane), then = page_at(base + 32 + lane);
      for (int u = off; u < off + count && ok; ++u, ++n) {
        if (((u * L::kKeys) >> page_shift) - base >= 32) {
          base += 32;
          now = then;
          then = page_at(base + 32 + lane);
        }
        const int t = u * L::kKeys + lane * 16, i = (t >> page_shift) - base;
        const int pn = __shfl_sync(0xffffffffu, now.pg, i & 31), pt = __shfl_sync(0xffffffffu, then.pg, i & 31);
        const uint32_t sn = __shfl_sync(0xffffffffu, now.sc, i & 31), st = __shfl_sync(0xffffffffu, then.sc, i & 31);
        const bool tile = lane < kTiles && t < end;
        const int pg = tile ? (i < 32 ? pn : pt) : -1;
        const uint32_t sc = tile ? (i < 32 ? sn : st) : 0x10000u;
        const int64_t ph = static_cast<int64_t>(pg) * a.Hkv + hk;
        if (n >= L::kStages) ok = __all_sync(0xffffffffu, wait(&empty[stage], phase ^ 1)) != 0;
        if (!ok) break;
        if (lane < kTiles) scales[stage * kTiles + lane] = sc;
        const int live = __popc(__ballot_sync(0xffffffffu, pg >= 0));
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_expect_tx(&full[stage], live * 2 * L::kBytes);  // releases the scales too
        __syncwarp();
        if (pg >= 0) {
          // in rows of 128 bytes, as the maps see the cache
          const int at = static_cast<int>(((ph << page_shift) + (t & (a.page - 1))) * D / 128);
          const uint32_t dst = tc::smem_u32(smem) + stage * L::kStage + lane * 2 * L::kBytes, bar = tc::smem_u32(&full[stage]);
          tma_load_2d(dst, &mk, bar, 0, at);
          tma_load_2d(dst + L::kBytes, &mv, bar, 0, at);
        }
        next_stage();
      }
      left -= count;
      if (left > 0) next_row();
    }
    // every copy has landed before the CTA may end
    if (lane == 0)
      for (int64_t i = max(static_cast<int64_t>(0), n - L::kStages); i < n; ++i)
        wait(&full[i % L::kStages], static_cast<uint32_t>(i / L::kStages) & 1);
    return;
  }

  bool ok = true;
  int begun = 0;  // 1 after the CTA's first row
  for (;;) {
    const int hk = r / pl.groups, h0 = hk * G + (r % pl.groups) * 8, heads = min(8, G - (r % pl.groups) * 8);
    // queries: a power of two brings the largest magnitude of a head into [1, 2)
    uint32_t qf[NP][KS][2];
    float hs[2];  // scale of the scores of heads 2 tig, 2 tig + 1 (log2 units)
    const T* q = static_cast<const T*>(a.q.p) + b * a.q.stride + static_cast<int64_t>(h0 + (gid < heads ? gid : 0)) * D;
    float x[KS][4], largest = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const T* at = q + (ks / 4) * 64 + (D < 64 ? D / 4 : 16) * tig + 4 * (ks % 4);
      if (sizeof(T) == 2 && a.q.vec) {  // 4 bf16 at a time
        const uint2 w = *reinterpret_cast<const uint2*>(at);
        x[ks][0] = __uint_as_float(w.x << 16), x[ks][1] = __uint_as_float(w.x & 0xFFFF0000u);
        x[ks][2] = __uint_as_float(w.y << 16), x[ks][3] = __uint_as_float(w.y & 0xFFFF0000u);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[ks][i] = to_f32(at[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (gid >= heads) x[ks][i] = 0.f;
        const float m = fabsf(x[ks][i]);
        if (m < INFINITY) largest = fmaxf(largest, m);
      }
    }
    largest = fmaxf(largest, __shfl_xor_sync(0xffffffffu, largest, 1));
    largest = fmaxf(largest, __shfl_xor_sync(0xffffffffu, largest, 2));
    const int e = max(static_cast<int>(__float_as_uint(largest) >> 23) - 127, -126);  // 2^e <= largest < 2^(e+1)
    const float up0 = exp2i(-e / 2), up1 = exp2i(-e - (-e / 2));
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t f[NP];
        split2<NP>(x[ks][2 * i] * up0 * up1, x[ks][2 * i + 1] * up0 * up1, f);
#pragma unroll
        for (int p = 0; p < NP; ++p) qf[p][ks][i] = f[p];
      }
    const float down = exp2i(e) * a.scale * kLog2e;
#pragma unroll
    for (int i = 0; i < 2; ++i) hs[i] = __shfl_sync(0xffffffffu, down, (2 * tig + i) * 4);

    // running reference and sum of the heads 2 tig, 2 tig + 1, and O^T
    float m[2], l[2], o[KS][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
    for (int j = 0; j < KS; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[j][i] = 0.f;

    for (int u = off; u < off + count; ++u) {
      ok = ok && __all_sync(0xffffffffu, wait(&full[stage], phase)) != 0;
      const uint32_t src0 = tc::smem_u32(smem) + stage * L::kStage + warp * L::kSub * 2 * L::kBytes;
      // scores of the warp's 16-key tiles, two sums each for short chains
      float sc[L::kSub][4];
      uint32_t bytes[L::kSub];
      int have[L::kSub];
      bool past = false;
#pragma unroll
      for (int sub = 0; sub < L::kSub; ++sub) {
        const int t = u * L::kKeys + (warp * L::kSub + sub) * 16;
        bytes[sub] = scales[stage * L::kSub * kWarps + warp * L::kSub + sub];
        have[sub] = ok && !(bytes[sub] & 0x10000u) ? keys - t : 0;  // keys of the tile that exist
        if (have[sub] <= 0) bytes[sub] = 0;                         // weights 0, the smallest scales
        const uint32_t src = src0 + sub * 2 * L::kBytes;
        float s[2][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) s[0][i] = s[1][i] = 0.f;
#pragma unroll
        for (int ld = 0; ld < L::kKLoads; ++ld) {
          uint32_t k0[KW], k1[KW];
          lds<L::kKSize>(src + in_tile<D>(key_of<D>(gid) * D + tig * L::kKSize + ld * 64), k0);
          lds<L::kKSize>(src + in_tile<D>(key_of<D>(gid + 8) * D + tig * L::kKSize + ld * 64), k1);
#pragma unroll
          for (int j = 0; j < KW; ++j) {
            const uint32_t a0 = e4m3x2_to_half2(k0[j] & 0xFFFFu), a2 = e4m3x2_to_half2(k0[j] >> 16);
            const uint32_t a1 = e4m3x2_to_half2(k1[j] & 0xFFFFu), a3 = e4m3x2_to_half2(k1[j] >> 16);
#pragma unroll
            for (int p = 0; p < NP; ++p)
              mma_f16(s[j & 1], a0, a1, a2, a3, qf[p][ld * KW + j][0], qf[p][ld * KW + j][1]);
          }
        }
        const float ks = e8m0(bytes[sub] & 0xFFu);
        const bool in0 = key_of<D>(gid) < have[sub], in1 = key_of<D>(gid + 8) < have[sub];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float f = hs[i] * ks;
          sc[sub][i] = in0 ? (s[0][i] + s[1][i]) * f : -INFINITY;
          sc[sub][2 + i] = in1 ? (s[0][2 + i] + s[1][2 + i]) * f : -INFINITY;
          past |= fmaxf(sc[sub][i], sc[sub][2 + i]) > m[i] + kSlack;
        }
      }
      if (__any_sync(0xffffffffu, past)) {  // move the reference to the maximum
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float x = m[i];
#pragma unroll
          for (int sub = 0; sub < L::kSub; ++sub) x = fmaxf(x, fmaxf(sc[sub][i], sc[sub][2 + i]));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          const float f = x == -INFINITY ? 1.f : ex2(m[i] - x);
          m[i] = x;
          l[i] *= f;
#pragma unroll
          for (int j = 0; j < KS; ++j) o[j][i] *= f, o[j][2 + i] *= f;
        }
      }
#pragma unroll
      for (int sub = 0; sub < L::kSub; ++sub) {
        uint32_t pb[NP][2];
        float p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float ref = m[i & 1];
          p[i] = ex2(sc[sub][i] - (ref == -INFINITY ? 0.f : ref));
        }
        l[0] += p[0] + p[2];
        l[1] += p[1] + p[3];
        // the exponent of each head's largest weight of the tile: upper halves of two floats side by side
        uint32_t big = __byte_perm(__float_as_uint(fmaxf(p[0], p[2])), __float_as_uint(fmaxf(p[1], p[3])), 0x7632);
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) big = __vmaxu2(big, __shfl_xor_sync(0xffffffffu, big, x));
        // weights times up[] become halves, the tile's products times back[] are values again
        float up[2], back[2];
        const int ev = static_cast<int>(bytes[sub] >> 8) - 127;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int e = max(static_cast<int>(big >> (7 + 16 * i)) & 0xFF, kTop);
          up[i] = __uint_as_float(static_cast<uint32_t>(2 * 127 + kTop - e) << 23);
          const int x = e - 127 - kTop + ev;
          back[i] = x < -149 ? 0.f : exp2i(x);
        }
        uint32_t f0[NP], f1[NP];
        split2<NP>(p[0] * up[0], p[1] * up[1], f0);
        split2<NP>(p[2] * up[0], p[3] * up[1], f1);
#pragma unroll
        for (int x = 0; x < NP; ++x) {
          pb[x][0] = transpose8x8(f0[x]);
          pb[x][1] = transpose8x8(f1[x]);
        }
        const uint32_t vsrc = src0 + sub * 2 * L::kBytes + L::kBytes;
        uint32_t v[4][VW];
        const int gv = D == 128 ? ((gid & 1) << 2) | (gid >> 1) : gid;  // this lane group's eighth of the dims
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          // the two keys of a pair trade places in odd lanes where that keeps their reads apart (d = 64)
          const int y = D == 64 ? x ^ (tig & 1) : x, key = key_of<D>(2 * tig + (y & 1) + 8 * (y >> 1));
          lds<L::kVSize>(vsrc + in_tile<D>(key * D + (D == 16 ? (gid >> 1) * 4 : gv * L::kVSize)), v[x]);
          if (D == 16) v[x][0] >>= (gid & 1) * 16;
          if (have[sub] < 16 && key >= have[sub]) {  // whatever lies there, it must not meet a weight of 0
#pragma unroll
            for (int w = 0; w < VW; ++w) v[x][w] = 0;
          }
        }
        const uint32_t low = D == 64 && (tig & 1) ? 0x1504u : 0x5140u, high = D == 64 && (tig & 1) ? 0x3726u : 0x7362u;
#pragma unroll
        for (int j = 0; j < KS; ++j) {
          const uint32_t sel = (j & 1) ? high : low;
          const uint32_t lo = __byte_perm(v[0][j / 2], v[1][j / 2], sel), hi = __byte_perm(v[2][j / 2], v[3][j / 2], sel);
          const uint32_t a0 = e4m3x2_to_half2(lo & 0xFFFFu), a1 = e4m3x2_to_half2(lo >> 16);
          const uint32_t a2 = e4m3x2_to_half2(hi & 0xFFFFu), a3 = e4m3x2_to_half2(hi >> 16);
          float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int x = 0; x < NP; ++x) mma_f16(part, a0, a1, a2, a3, pb[x][0], pb[x][1]);
#pragma unroll
          for (int e = 0; e < 4; ++e) o[j][e] = fmaf(part[e], back[e & 1], o[j][e]);
        }
      }
      __syncwarp();
      if (lane == 0) tcu::mbar_arrive(&empty[stage]);
      next_stage();
    }

    const bool whole = count == units;  // this CTA holds the row's every key
    const int64_t done_b = b;
    const int slot = begun;
    if (!whole && threadIdx.x == 0) {   // what the kernel that joins the parts goes by
      if (off == 0) begun_in[blockIdx.x] = (b * R + r) * 2 + slot;
      if (off + count == units) ended_in[b * R + r] = blockIdx.x;
    }
    left -= count;
    begun = 1;
    if (left > 0) next_row();

    // join the warps: weights of each head, then the sums by halves
    float top[2], sum[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float x = l[i];
      x += __shfl_xor_sync(0xffffffffu, x, 4);
      x += __shfl_xor_sync(0xffffffffu, x, 8);
      x += __shfl_xor_sync(0xffffffffu, x, 16);
      if (gid == 0) ml[warp * H8 + 2 * tig + i] = make_float2(m[i], x);
    }
    const bool fine = !tcu::named_bar_any(1, kWarps * 32, !ok);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2* x = ml + 2 * tig + i;
      top[i] = -INFINITY, sum[i] = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top[i] = fmaxf(top[i], x[w * H8].x);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum[i] += x[w * H8].y * weight_of(x[w * H8], top[i]);
      const float f = weight_of(x[warp * H8], top[i]);
#pragma unroll
      for (int j = 0; j < KS; ++j) o[j][i] *= f, o[j][2 + i] *= f;
    }
    auto give = [&](float* to) {
#pragma unroll
      for (int j = 0; j < KS; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) to[(j * 4 + i) * 32 + lane] = o[j][i];
    };
    auto take = [&](const float* from) {
#pragma unroll
      for (int j = 0; j < KS; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[j][i] += from[(j * 4 + i) * 32 + lane];
    };
#pragma unroll
    for (int half = kWarps / 2; half >= 1; half >>= 1) {
      if (warp >= half && warp < 2 * half) give(joint + (warp - half) * kFrag * 32);
      tcu::named_bar(1, kWarps * 32);
      if (warp < half) take(joint + warp * kFrag * 32);
      if (half > 1) tcu::named_bar(1, kWarps * 32);
    }
    if (warp == 0 && fine) {
      // this lane: an eighth of the dims of heads 2 tig and 2 tig + 1
      const int dim0 = (D == 128 ? ((gid & 1) << 2) | (gid >> 1) : gid) * (D / 8);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int h = 2 * tig + i;
        if (h >= heads) continue;
        const float x = sum[i];
        if (whole) {
          T* out = static_cast<T*>(a.o.p) + done_b * a.o.stride + static_cast<int64_t>(h0 + h) * D + dim0;
          const float inv = x == 0.f ? 0.f : 1.f / x;
#pragma unroll
          for (int j = 0; j < KS; ++j) {
            out[2 * j] = from_f32<T>(x == 0.f ? 0.f : o[j][i] * inv);
            out[2 * j + 1] = from_f32<T>(x == 0.f ? 0.f : o[j][2 + i] * inv);
          }
          if (a.lse && gid == 0) a.lse[done_b * a.Hq + h0 + h] = log_sum(make_float2(top[i], x));
        } else {
          const int64_t at = (static_cast<int64_t>(blockIdx.x) * 2 + slot) * H8 + h;
          float* out = part_o + at * D + dim0;
#pragma unroll
          for (int j = 0; j < KS; ++j) out[2 * j] = o[j][i], out[2 * j + 1] = o[j][2 + i];
          if (gid == 0) part_ml[at] = make_float2(top[i], x);
        }
      }
    }
    if (left <= 0) break;
  }
}

// Joins the parts of the row that CTA blockIdx.x of the first kernel has begun
// and not ended, for head blockIdx.y of its group: the part that it left, then
// the first parts of the CTAs up to the one that ended the row.  D / 4 lanes
// take the dims, the groups of lanes the parts in turn.
template <typename T, int D>
__global__ void __launch_bounds__(256) attn_decode_join_kernel(const DecodeArgs a, const DecodePlan pl, const float* part_o,
                                                               const float2* part_ml, const int* begun_in,
                                                               const int* ended_in) {
  constexpr int W = D / 4, NGR = 256 / W;
  __shared__ float4 so[NGR][W];
  __shared__ float2 sml[NGR];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int begun = begun_in[blockIdx.x];
  if (begun < 0) return;
  const int w = threadIdx.x % W, g = threadIdx.x / W, G = a.Hq / a.Hkv, R = a.Hkv * pl.groups;
  const int row = begun >> 1, r = row % R, hh = r % pl.groups * 8 + static_cast<int>(blockIdx.y);
  if (hh >= G) return;
  const int64_t b = row / R;
  const int h = r / pl.groups * G + hh, c0 = blockIdx.x, n = ended_in[row] - c0 + 1;
  auto part = [&](int i) {
    return (static_cast<int64_t>(c0 + i) * 2 + (i == 0 ? begun & 1 : 0)) * 8 + static_cast<int>(blockIdx.y);
  };
  float top = -INFINITY, sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = g; i < n; i += NGR) top = fmaxf(top, part_ml[part(i)].x);
#pragma unroll 4
  for (int i = g; i < n; i += NGR) {
    const float2 x = part_ml[part(i)];
    const float4 v = reinterpret_cast<const float4*>(part_o + part(i) * D)[w];
    const float f = weight_of(x, top);
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
    const float f = weight_of(sml[i], top);
    sum += sml[i].y * f;
    y += reinterpret_cast<const float*>(so[i])[d] * f;
  }
  T* out = static_cast<T*>(a.o.p) + b * a.o.stride + static_cast<int64_t>(h) * D;
  out[d] = from_f32<T>(sum == 0.f ? 0.f : y / sum);
  if (a.lse && d == 0) a.lse[b * a.Hq + h] = log_sum(make_float2(top, sum));
}



// Few keys a row: a CTA for each row, one launch (measured when the batch below
// took 68 us: 256 rows of 500 keys, 4 key heads of 128 31 us, in equal shares
// 37).  Otherwise as many CTAs as the card holds at a time, each with the same
// number of units, so that none waits for a longer one (256 rows of 410 .. 2048
// keys: 68 us, with chunks of 1024 keys 75).
DecodePlan decode_plan(int B, int Hq, int Hkv, int d, int elem, int max_k) {
  DecodePlan p;
  const int G = Hq / Hkv;
  p.groups = (G + 7) / 8;
  const int64_t rows = static_cast<int64_t>(B) * Hkv * p.groups, sms = tcu::sm_count();
  p.direct = max_k <= 512 || (max_k <= 1024 && d < 128 && rows >= 3 * sms);
  const int unit = d == 128 ? Tile<128>::kKeys : Tile<64>::kKeys;
  const int64_t want = rows * ((static_cast<int64_t>(max_k) + unit - 1) / unit);
  const int64_t held = sms * ctas_of_sm(elem, d);
  p.ctas = static_cast<int>(p.direct ? (rows > INT32_MAX ? INT32_MAX : rows) : want < held ? want : held);
  return p;
}

// The codes as rows of 128 bytes, boxes of 16 keys.
bool make_cache_map(CUtensorMap* m, const uint8_t* codes, const DecodeArgs& a, int d) {
  tcu::EncodeFn enc = tcu::get_encode();
  if (!enc) return false;
  const uint64_t rows = static_cast<uint64_t>(a.num_pages) * a.Hkv * a.page * d / 128;
  cuuint64_t dims[2] = {128, rows};
  cuuint64_t strides[1] = {128};
  cuuint32_t box[2] = {128, static_cast<cuuint32_t>(16 * d / 128)};
  cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(codes), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, d >= 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct DecodeWs {
  size_t ml, o, begun, ended, total;
};
DecodeWs decode_ws(const DecodePlan& p, int B, int Hkv, int d) {
  DecodeWs w = {256, 256, 256, 256, 256};  // the status word first
  if (p.direct) return w;
  const size_t n = static_cast<size_t>(p.ctas) * 2 * 8;
  w.o = w.ml + align_up(n * sizeof(float2), 256);
  w.begun = w.o + align_up(n * d * sizeof(float), 256);
  w.ended = w.begun + align_up(static_cast<size_t>(p.ctas) * sizeof(int), 256);
  w.total = w.ended + align_up(static_cast<size_t>(B) * Hkv * p.groups * sizeof(int), 256);
  return w;
}

template <typename T, int D>
int launch_decode(const DecodeArgs& a, const DecodePlan& p, cudaStream_t s) {
  using L = Tile<D>;
  constexpr size_t smem = 1024 + static_cast<size_t>(L::kStages) * L::kStage +
                          static_cast<size_t>(kWarps / 2) * (D / 16) * 4 * 32 * 4 + static_cast<size_t>(kWarps) * 8 * 8 +
                          static_cast<size_t>(L::kStages) * L::kSub * kWarps * 4;
  CUtensorMap mk, mv;
  if (!make_cache_map(&mk, a.cache.k, a, D) || !make_cache_map(&mv, a.cache.v, a, D)) return FALCON_ERR_CUDA;
  const int64_t rows = static_cast<int64_t>(a.B) * a.Hq;
  // rows of 128 bytes of the cache are 32-bit coordinates of the maps
  if (rows > INT32_MAX / 2 || static_cast<int64_t>(a.num_pages) * a.Hkv > INT32_MAX / (a.page * D / 128))
    return FALCON_ERR_UNSUPPORTED;
  const auto kern = attn_decode_kernel<T, D>;
  if (!set_smem_limit(reinterpret_cast<const void*>(kern), smem)) return FALCON_ERR_CUDA;
  const DecodeWs w = decode_ws(p, a.B, a.Hkv, D);
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  float2* ml = reinterpret_cast<float2*>(ws + w.ml);
  float* po = reinterpret_cast<float*>(ws + w.o);
  int *begun = reinterpret_cast<int*>(ws + w.begun), *ended = reinterpret_cast<int*>(ws + w.ended);
  kern<<<static_cast<unsigned>(p.ctas), (kWarps + 1) * 32, smem, s>>>(mk, mv, a, p, po, ml, begun, ended,
                                                                       reinterpret_cast<uint32_t*>(ws), wait_limit_ns(),
                                                                       take_test_stall() ? 1 : 0);
  if (cudaGetLastError() != cudaSuccess) return FALCON_ERR_CUDA;
  if (p.direct) return FALCON_OK;
  FwdArgs fa = {};
  fa.stream = s;
  return tcu::launch_overlapped(fa, attn_decode_join_kernel<T, D>, dim3(static_cast<unsigned>(p.ctas), 8), dim3(256), 0, a,
                                p, static_cast<const float*>(po), static_cast<const float2*>(ml),
                                static_cast<const int*>(begun), static_cast<const int*>(ended));
}
template <typename T>
int launch_decode_d(const DecodeArgs& a, const DecodePlan& p, cudaStream_t s) {
  switch (a.d) {
    case 16: return launch_decode<T, 16>(a, p, s);
    case 32: return launch_decode<T, 32>(a, p, s);
    case 64: return launch_decode<T, 64>(a, p, s);
    default: return launch_decode<T, 128>(a, p, s);
  }
}

}  // namespace

size_t attn_decode_ws_bytes(int B, int Hq, int Hkv, int d, int elem, int max_k) {
  return decode_ws(decode_plan(B, Hq, Hkv, d, elem, max_k), B, Hkv, d).total;
}

int launch_attn_decode(const DecodeArgs& a, int dtype, cudaStream_t s) {
  const DecodePlan p = decode_plan(a.B, a.Hq, a.Hkv, a.d, dtype == FALCON_BF16 ? 2 : 4, a.max_k);
  return dtype == FALCON_BF16 ? launch_decode_d<__nv_bfloat16>(a, p, s) : launch_decode_d<float>(a, p, s);
}

}  // namespace falcon
