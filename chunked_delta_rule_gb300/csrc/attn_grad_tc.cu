// Gradient of causal attention over packed prompts on the tensor cores (bf16).
//
//   P = exp(scale Q K^T - log sum),  dS = P (dO V^T - D)
//   dV = P^T dO,  dK = scale dS^T Q,  dQ = scale dS K
//
// Two kernels from one template, so that every sum has one owner and one order (7
// products of a tile where one kernel with dQ added up in memory would have 5; that
// adds 64 KB in fp32 for every tile of 128 x 128, and in another order each
// time).  A CTA owns 128 rows: of K and V (dK and dV; X = K Q^T, Y = V dO^T, the
// queries of all heads of the group come past) or of Q and dO (dQ; X = Q K^T, Y = dO
// V^T, the keys come past).  Per tile of rows that come past (128; 64 at d = 64, with two
// CTAs on an SM):
//   load warp    TMA: the two tiles, through a ring of pairs
//   MMA warp     X, Y and the sums' products in the order that keeps the tensor
//                cores ahead of the softmax warps, see the loops
//   softmax      64 columns of a row a thread (32: 290 us for 281 in the packed case): P
//   warps        from X, dS from P and Y.  They go back to TMEM in bf16 over the scores
//                that they came from, as the A operand of the sums' products.
// dK and dV: a thread holds one key and 64 queries, so that log sums and D would be
// loads for every element; they come out of the products instead, one more step of 16
// columns: [K | 1] [Q | -log sum / scale]^T and [V | 1] [dO | -D]^T, in three bf16
// parts (24 bits).
// dQ: Q and dO are copied to TMEM, as the A operands there of X and Y: both operands in
// shared memory would ask it for 8 KB a step of 128 x 128 x 16, all that it gives in
// the 64 cycles of the step, before the TMA writes.  (For dK and dV the four
// accumulators of d = 128 fill TMEM.)
// Where the keys' blocks alone do not fill the GPU, 2, 4 or 8 CTAs of a cluster take a
// block together, a share of the queries' tiles each; their sums are added over
// distributed shared memory, in the CTAs' order.
//
// P and dS are rounded to bf16 as V and K are held in it: at most 2^-8 of each.
// Everything else is fp32.
//
// Masked scores are set to -inf after the product.  A masked weight is 0, but 0
// times an infinite or NaN value of a row that the owner does not see would spoil
// it: a row of a result that is not finite is computed again from the definition,
// after the pipeline has ended.

#include <algorithm>

#include "attn_grad.cuh"
#include "attn_tc.cuh"

namespace falcon {
namespace {

using namespace tcu;

template <int D, bool KEYS>
struct Cfg {
  static constexpr int kCtas = D == 64 ? 2 : 1;           // CTAs of an SM
  static constexpr int kN = D == 64 ? 64 : 128;           // rows of a tile that comes past
  static constexpr int kW = 2;                            // times 32 columns of a row: a softmax thread's
  static constexpr int kSplit = kN / (32 * kW);           // softmax threads of a row
  static constexpr int kOut = (KEYS ? 2 : 1) * D / kSplit;  // columns of the sums that each of them writes
  static constexpr int kWarps = 4 * kSplit;
  static constexpr int kLoadWarp = kWarps, kMmaWarp = kWarps + 1;
  static constexpr int kThreads = 32 * kWarps + 128;
  static constexpr int kOwnBytes = kTile * D * 2, kTileBytes = kN * D * 2;
  // dQ: the owned rows' place joins the ring (its last pairs) once they are in TMEM
  static constexpr int kOwnPairs = KEYS ? 0 : kOwnBytes / kTileBytes;
  static constexpr int kPairs = D == 64 ? (KEYS ? 3 : 5) : (KEYS ? 2 : 3);
  static constexpr int kRing = 2 * kPairs * kTileBytes;
  static constexpr int kOwnAt = KEYS ? kRing : kRing - 2 * kOwnBytes;
  static constexpr int kImage = kN * 32;                  // log sums and D of a tile of queries
  static constexpr int kExtra = KEYS ? 2 * kOwnBytes + kPairs * kImage + 2 * kImageBytes : 0;
  // TMEM: X, Y, the sums, and for dQ the owned rows
  static constexpr uint32_t kColX = 0, kColY = kN, kColV = 2 * kN, kColS = KEYS ? 2 * kN + D : 2 * kN;
  static constexpr uint32_t kColA1 = 2 * kN + D, kColA2 = kColA1 + D / 2;
  static constexpr uint32_t kCols = D == 64 ? 256 : 512;
};
constexpr int kMostPairs = 5;
struct Bars {
  uint64_t own, ready, full[2 * kMostPairs], empty[2 * kMostPairs], x, y;
  uint64_t p;  // dK and dV: P is there; dQ: X has been read
  uint64_t ds, drain, stall;
  uint32_t tmem, failed;
  uint32_t bad[2][4];  // rows that are not finite, a bit each
};
template <int D, bool KEYS>
constexpr int smem_bytes() {
  return Cfg<D, KEYS>::kRing + Cfg<D, KEYS>::kExtra + 1024 + static_cast<int>(sizeof(Bars));
}
static_assert(smem_bytes<128, true>() <= 227 * 1024 && smem_bytes<128, false>() <= 227 * 1024, "shared memory");
static_assert(smem_bytes<64, true>() <= 113 * 1024 && smem_bytes<64, false>() <= 113 * 1024, "shared memory");

struct TcGradArgs {
  GradArgs g;
  int qblocks;  // of a sequence
  bool packed;
  bool second;  // of the call's two kernels
  int split;    // CTAs of a cluster
  uint32_t* status;
  uint64_t limit;
  int stall;
};

// no swizzle: 8 rows x 16 bytes, halves of a row 128 bytes apart, groups of 8 rows 256
__device__ __forceinline__ uint64_t sdesc_plain16(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(128 >> 4) << 16;
  d |= static_cast<uint64_t>(256 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  return d;
}
template <int D, bool KEYS>
__global__ void __launch_bounds__(Cfg<D, KEYS>::kThreads, Cfg<D, KEYS>::kCtas)
    attn_grad_tc_kernel(const __grid_constant__ CUtensorMap own1, const __grid_constant__ CUtensorMap own2,
                        const __grid_constant__ CUtensorMap past1, const __grid_constant__ CUtensorMap past2,
                        const TcGradArgs t) {
  using C = Cfg<D, KEYS>;
  constexpr int N = C::kN, P = C::kPairs;
  const GradArgs& g = t.g;
  const PromptArgs& a = g.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint8_t *ring = smem, *s1 = smem + C::kOwnAt, *s2 = s1 + C::kOwnBytes;  // ring: pairs of a first and a second tile
  uint8_t* images = smem + C::kRing + 2 * C::kOwnBytes;
  uint8_t* ones = images + P * C::kImage;
  Bars* bar = reinterpret_cast<Bars*>(smem + C::kRing + C::kExtra);
  if (warp == C::kMmaWarp) {
    tmem_alloc(&bar->tmem, C::kCols);
    tmem_relinquish();
  }
  if (warp == C::kLoadWarp && lane == 0) {
    for (const CUtensorMap* m : {&own1, &own2, &past1, &past2})
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
    mbar_init(&bar->own, 1);
    mbar_init(&bar->ready, C::kWarps);
    for (int i = 0; i < 2 * P; ++i) {
      mbar_init(&bar->full[i], 1);
      mbar_init(&bar->empty[i], 1);
    }
    mbar_init(&bar->x, 1);
    mbar_init(&bar->y, 1);
    mbar_init(&bar->p, C::kWarps + 1);
    mbar_init(&bar->ds, C::kWarps + 1);
    mbar_init(&bar->drain, 1);
    mbar_init(&bar->stall, 1);
    bar->failed = 0;
    for (int i = 0; i < 8; ++i) bar->bad[i >> 2][i & 3] = 0;
    fence_mbar_init();
  }
  if (KEYS) {  // ones against the log sums (columns 0 to 2), ones against D (4 to 6)
    for (int i = tid; i < 4 * kTile; i += C::kThreads) {
      const int r = i & (kTile - 1), half = (i >> 7) & 1, which = i >> 8;
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (half == 0 && which == 0) v.x = 0x3F803F80u, v.y = 0x3F80u;
      if (half == 0 && which == 1) v.z = 0x3F803F80u, v.w = 0x3F80u;
      *reinterpret_cast<uint4*>(ones + which * kImageBytes + (r >> 3) * 256 + half * 128 + (r & 7) * 16) = v;
    }
    fence_proxy_async();
  }

  // whose rows
  const int G = a.Hq / a.Hkv;
  const uint32_t block = KEYS ? blockIdx.x / t.split : blockIdx.x;
  const int rank = KEYS ? static_cast<int>(blockIdx.x % t.split) : 0;
  int b, head, row0;
  if (KEYS) {
    const int2 x = find_block(a.cu_k, a.B, kTile, static_cast<int>(block / a.Hkv));
    b = x.x, row0 = x.y, head = static_cast<int>(block % a.Hkv);
  } else if (t.packed) {
    const int2 x = find_block(a.cu_q, a.B, kTile, static_cast<int>(block / a.Hq));
    b = x.x, row0 = x.y, head = static_cast<int>(block % a.Hq);
  } else {
    const uint32_t bh = static_cast<uint32_t>(a.B) * a.Hq, at = block % bh;
    b = static_cast<int>(at) / a.Hq, head = static_cast<int>(at) % a.Hq;
    row0 = (t.qblocks - 1 - static_cast<int>(block / bh)) * kTile;  // the longest rows first
  }
  const int64_t q0 = a.cu_q[b], k0 = a.cu_k[b];
  const int lq_all = static_cast<int>(a.cu_q[b + 1] - q0), lk = static_cast<int>(a.cu_k[b + 1] - k0);
  const int lq = min(lq_all, a.max_q), off = lk - lq_all, rows = KEYS ? lk : lq;
  const bool valid = row0 >= 0 && row0 < rows && q0 >= 0 && k0 >= 0 && q0 + lq_all <= a.tokens && k0 + lk <= a.k_tokens;
  // a sequence's blocks are dealt out from its last; the first keys, which the most queries see, come first
  if (KEYS) row0 = (lk - 1) / kTile * kTile - row0;
  // the tiles that come past, [first, first + each N) of every head, and this CTA's of them
  const int first = KEYS ? max(row0 - off, 0) / N * N : 0;
  const int end = KEYS ? lq : min(min(row0 + kTile, lq) + off, lk);
  const int each = end > first ? (end - first + N - 1) / N : 0;
  int i0 = 0, n = each;
  if (KEYS) {
    const int64_t all = static_cast<int64_t>(each) * G;
    i0 = static_cast<int>(all * rank / t.split);
    n = static_cast<int>(all * (rank + 1) / t.split) - i0;
  }
  __syncthreads();
  const uint32_t tmem = bar->tmem;
  if (!t.second) {  // what the sums' kernel wrote is there
    wait_for_previous();
    launch_dependents();
  }
  const bool last = t.second && blockIdx.x == gridDim.x - 1 && tid == C::kThreads - 1;  // ends no sooner than the first kernel
  if (!valid) {  // (the whole cluster)
    if (warp == C::kMmaWarp) tmem_dealloc(tmem, C::kCols);
    if (last) wait_for_previous();
    return;
  }
  auto wait = [&](uint64_t* m, uint32_t parity) {
    if (mbar_wait_sleep(m, parity, t.limit)) return true;
    atomicExch(t.status, kStatusTimeout);
    *static_cast<volatile uint32_t*>(&bar->failed) = 1;
    return false;
  };
  // Tile i's places in the ring, and how often they were used before.  dK and dV: the first tile (Q) is read until the
  // tile's last product, the second (dO) until its last but two; they change places from use to use, so that each
  // copy has a whole tile's products of time.
  auto place = [&](int i, int second) { return 2 * (i % P) + (KEYS ? (i / P + second) & 1 : second); };

  // registers: the softmax threads take what the last warpgroup gives up
  // (128 x 200 + 128 x 56 = 256 x 128; 256 x 208 + 128 x 88 = 384 x 168)
  if (warp >= C::kLoadWarp) {
    if (D == 64) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (last) wait_for_previous();
    __syncwarp();
  }
  if (warp == C::kLoadWarp) {
    if (lane == 0 && n > 0) {
      bool ok = !t.stall || wait(&bar->stall, 0);
      int loads = 0;  // tiles begun: the first and the second of pair 0, of pair 1 ...
      bool own = false, ready = false;
      if (ok) {
        own = true;
        const int at = static_cast<int>((KEYS ? k0 : q0) + row0);
        mbar_arrive_expect_tx(&bar->own, 2 * C::kOwnBytes);
        for (int c = 0; c < D / 64; ++c) {
          tma_load_3d(s1 + c * kTile * 128, &own1, &bar->own, c * 64, head, at);
          tma_load_3d(s2 + c * kTile * 128, &own2, &bar->own, c * 64, head, at);
        }
      }
      for (; loads < 2 * n && ok; ++loads) {
        const int i = loads >> 1, second = loads & 1, st = i % P, use = i / P, slot = place(i, second);
        if (!KEYS && !ready && st >= P - C::kOwnPairs) {
          if (!(ok = wait(&bar->ready, 0))) break;
          ready = true;
        }
        if (use > 0 && !(ok = wait(&bar->empty[slot], (use - 1) & 1))) break;
        const int h = KEYS ? head * G + (i0 + i) / each : head / G, at = first + (KEYS ? (i0 + i) % each : i) * N;
        const int row = static_cast<int>((KEYS ? q0 : k0) + at);
        const bool image = KEYS && !second;  // its place was last read by the product before the one that freed this
        mbar_arrive_expect_tx(&bar->full[slot], C::kTileBytes + (image ? C::kImage : 0));
        for (int c = 0; c < D / 64; ++c)
          tma_load_3d(ring + slot * C::kTileBytes + c * N * 128, second ? &past2 : &past1, &bar->full[slot], c * 64, h, row);
        if (image)
          bulk_load(images + st * C::kImage,
                    g.images + (static_cast<int64_t>(h) * g.blocks + first_block(q0, b) + at / kSumRows) * kImageBytes +
                        at % kSumRows * 32,
                    C::kImage, &bar->full[slot]);
      }
      // every copy has landed before the CTA may end
      if (own) wait(&bar->own, 0);
      for (int l = max(0, loads - 2 * P); l < loads; ++l) wait(&bar->full[place(l >> 1, l & 1)], ((l >> 1) / P) & 1);
    }
    __syncwarp();
  } else if (warp == C::kMmaWarp) {
    // One lane walks the loop: it issues a product in 16 cycles (the whole warp with an elected lane in 46) and a wait that
    // has come true costs it 66; the tensor cores' queue hides some 250 cycles between two batches.
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    if (elect_one()) {
      constexpr uint32_t id_x = idesc_bf16(kTile, N), id_s = idesc_bf16(kTile, D, false, true);
      const uint64_t a1 = sdesc_k128(smem_u32(s1)), a2 = sdesc_k128(smem_u32(s2)), bk = sdesc_k128(smem_u32(ring));
      const uint64_t bm = D == 64 ? sdesc_mn128(smem_u32(ring)) : sdesc_mn128_wide(smem_u32(ring), N * 128);
      const uint64_t one = sdesc_plain16(smem_u32(ones)), img = sdesc_plain16(smem_u32(images));
      auto arrived = [&](uint64_t* m, uint32_t parity) {
        const bool ok = wait(m, parity);
        tc_fence_after();
        return ok;
      };
      // X (second = 0) or Y of tile i, with what its completion tells
      auto scores = [&](int i, int second, uint64_t* then, bool frees) {
        const int slot = place(i, second);
        const uint64_t bs = bk + slot * (C::kTileBytes >> 4);
        const uint32_t to = tm + (second ? C::kColY : C::kColX);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint64_t bd = bs + (((ks >> 2) * N * 128 + (ks & 3) * 32) >> 4);
          if (KEYS) umma_bf16(to, (second ? a2 : a1) + (((ks >> 2) * kTile * 128 + (ks & 3) * 32) >> 4), bd, id_x, ks > 0);
          else umma_ts(to, tm + (second ? C::kColA2 : C::kColA1) + ks * 8, bd, id_x, ks > 0);
        }
        if (KEYS) umma_bf16(to, one + second * (kImageBytes >> 4), img + i % P * (C::kImage >> 4), id_x, 1);
        umma_commit(then);
        if (frees) umma_commit(&bar->empty[slot]);
      };
      // sum += W (bf16, in TMEM) times the first or second tile of pair i
      auto add = [&](uint32_t sum, uint32_t w, int i, int second) {
        const int slot = place(i, second);
        const uint64_t bs = bm + slot * (C::kTileBytes >> 4);
#pragma unroll
        for (int ks = 0; ks < N / 16; ++ks)
          umma_ts(tm + sum, tm + w + (ks >> 1) * 32 + (ks & 1) * 8, bs + ks * 128, id_s, i > 0 || ks > 0);
        umma_commit(&bar->empty[slot]);
      };
      bool ok = n > 0 && arrived(KEYS ? &bar->own : &bar->ready, 0) && arrived(&bar->full[place(0, 0)], 0);
      if (ok) {
        scores(0, 0, &bar->x, false);
        if ((ok = arrived(&bar->full[place(0, 1)], 0))) scores(0, 1, &bar->y, !KEYS);
      }
      // dK and dV: ... X(i) dK(i - 1) Y(i) dV(i) X(i + 1) ...: P(i) is formed under dK(i - 1) and Y(i), dS(i) under dV(i)
      // and X(i + 1).  dQ: ... Y(i) X(i + 1) dQ(i) Y(i + 1) ...: P(i + 1) is formed under dQ(i) and Y(i + 1), dS(i) under
      // X(i + 1).  What these wait for holds the next tile's copies too.
      for (int i = 0; i < n && ok; ++i) {
        if (!(ok = arrived(&bar->p, i & 1))) break;
        if (KEYS) add(C::kColV, C::kColX, i, 1);
        if (i + 1 < n) scores(i + 1, 0, &bar->x, false);
        if (!(ok = arrived(&bar->ds, i & 1))) break;
        add(C::kColS, C::kColY, i, 0);
        if (i + 1 < n) scores(i + 1, 1, &bar->y, !KEYS);
      }
      umma_commit(&bar->drain);  // products in flight end before the memory is freed
      wait(&bar->drain, 0);
    }
    __syncwarp();
  } else if (warp == C::kMmaWarp + 1) {
    // waits for the next tile's copies in the MMA warp's place, and joins the softmax warps' arrivals
    if (lane == 0) {
      bool ok = true;
      for (int i = 0; i < n && ok; ++i)
        for (int second = 0; second < 2 && ok; ++second) {
          uint64_t* m = second ? &bar->ds : &bar->p;
          if (i + 1 < n) ok = wait(&bar->full[place(i + 1, second)], ((i + 1) / P) & 1);
          if (!ok) break;
          mbar_arrive(m);
          ok = wait(m, i & 1);  // so that the next arrival counts for the next tile
        }
    }
    __syncwarp();
  } else if (warp < C::kLoadWarp) {
    if (D == 64) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int part = warp >> 2, quad = warp & 3, r = quad * 32 + lane;
    const uint32_t mine = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const int row = row0 + r;
    const float sl2 = a.scale * kLog2e;
    const uint64_t scale2 = pack2(sl2, sl2);
    const float* sums = g.sums + row_sums(g.blocks, KEYS ? head * G : head, first_block(q0, b));
    auto arrive = [&](uint64_t* m) {  // once for the warp: arrivals of 32 lanes on one word take their turns
      __syncwarp();
      if (lane == 0) mbar_arrive(m);
    };
    auto waited = [&](uint64_t* m, uint32_t parity) { return __all_sync(0xffffffffu, wait(m, parity)) != 0; };
    bool ok = true;
    uint64_t lse2 = 0, delta2 = 0;  // of this thread's query, negative
    if (!KEYS && n > 0) {
      const float* at = sums + static_cast<int64_t>(row0 / kSumRows) * (2 * kSumRows) + r;
      lse2 = pack2(-at[0] * kLog2e, -at[0] * kLog2e);
      delta2 = pack2(-at[kSumRows], -at[kSumRows]);
      // the owned rows to TMEM, a share of the columns each; rows past the sequence are some others', or zeros
      if ((ok = waited(&bar->own, 0))) {
        constexpr int kSlabs = 2 * D / 64 / C::kSplit;  // of 64 of the 2 D elements of a row of Q and dO
        static_assert(kSlabs * C::kSplit * 64 == 2 * D, "whole slabs a thread");
#pragma unroll
        for (int sl = 0; sl < kSlabs; ++sl) {
          const uint8_t* from = s1 + (part * kSlabs + sl) * kTile * 128;
          uint32_t w[32];
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const uint4 x = *reinterpret_cast<const uint4*>(from + sw128(r, c * 8));
            w[4 * c] = x.x, w[4 * c + 1] = x.y, w[4 * c + 2] = x.z, w[4 * c + 3] = x.w;
          }
          tmem_st32(mine + C::kColA1 + (part * kSlabs + sl) * 32, w);
        }
        tmem_wait_st();
        tc_fence_before();
        arrive(&bar->ready);
      }
    }
    int past = KEYS && n > 0 ? i0 % each : 0;  // the tile's place among a head's
    for (int i = 0; i < n && ok; ++i) {
      constexpr int W = C::kW;
      const int at = first + past * N + part * (32 * W);  // of the first column
      if (++past == each) past = 0;
      const uint32_t tx = mine + C::kColX + part * (32 * W), ty = mine + C::kColY + part * (32 * W);
      if (!(ok = waited(&bar->x, i & 1))) break;
      tc_fence_after();
      uint64_t x[W][16];  // X, then P
      {
        uint32_t v[W][32];
#pragma unroll
        for (int c = 0; c < W; ++c) tmem_ld32(tx + 32 * c, v[c]);
        tmem_wait_ld();
        if (!KEYS) {
          tc_fence_before();
          arrive(&bar->p);
        }
#pragma unroll
        for (int c = 0; c < W; ++c)
#pragma unroll
          for (int e = 0; e < 16; ++e) x[c][e] = pack2(__uint_as_float(v[c][2 * e]), __uint_as_float(v[c][2 * e + 1]));
      }
      // keys behind a query of these, or past the last
      if (KEYS ? at + off < row0 + kTile - 1 : at + 32 * W > min(row0 + off + 1, lk)) {
        const int lim = KEYS ? row - off - at : min(row + off + 1, lk) - at;
#pragma unroll
        for (int c = 0; c < W; ++c)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int first_of = 32 * c + 2 * e;
            float z0, z1;
            unpack2(x[c][e], z0, z1);
            if (KEYS ? first_of < lim : first_of >= lim) z0 = -INFINITY;
            if (KEYS ? first_of + 1 < lim : first_of + 1 >= lim) z1 = -INFINITY;
            x[c][e] = pack2(z0, z1);
          }
      }
#pragma unroll
      for (int c = 0; c < W; ++c) {
        uint32_t u[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float z0, z1;
          unpack2(KEYS ? mul2(x[c][e], scale2) : fma2(x[c][e], scale2, lse2), z0, z1);
          z0 = ex2(z0), z1 = ex2(z1);
          x[c][e] = pack2(z0, z1);
          if (KEYS) u[e] = pack_bf16(z0, z1);
        }
        if (KEYS) tmem_st16(tx + 32 * c, u);
      }
      if (KEYS) {
        tmem_wait_st();
        tc_fence_before();
        arrive(&bar->p);
      }
      if (!(ok = waited(&bar->y, i & 1))) break;
      tc_fence_after();
      {
        uint32_t v[W][32];
#pragma unroll
        for (int c = 0; c < W; ++c) tmem_ld32(ty + 32 * c, v[c]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < W; ++c) {
          uint32_t u[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            uint64_t z = pack2(__uint_as_float(v[c][2 * e]), __uint_as_float(v[c][2 * e + 1]));
            if (!KEYS) z = add2(z, delta2);
            float z0, z1;
            unpack2(mul2(x[c][e], z), z0, z1);
            u[e] = pack_bf16(z0, z1);
          }
          tmem_st16(ty + 32 * c, u);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      arrive(&bar->ds);
    }
    // the last product is the one that frees the last pair's first tile
    if (ok && n > 0) ok = waited(&bar->empty[place(n - 1, 0)], ((n - 1) / P) & 1);
    tc_fence_after();
    const int d = D == 64 ? a.d : D;  // of the rows
    // a row of a result (x1: dK or dQ, x2: dV) from the definition
    auto compute_again = [&](int i, float (&x1)[4], float (&x2)[4]) {
      const __nv_bfloat16 *q = static_cast<const __nv_bfloat16*>(a.q.p), *d_o = static_cast<const __nv_bfloat16*>(g.d_o.p);
      const __nv_bfloat16 *k = static_cast<const __nv_bfloat16*>(a.k.p), *v = static_cast<const __nv_bfloat16*>(a.v.p);
      if constexpr (KEYS) {
        const int64_t h0 = static_cast<int64_t>(head) * G * d, hk = static_cast<int64_t>(head) * d;
        grad_key_row<__nv_bfloat16, D>(k + (k0 + i) * a.k.stride + hk, v + (k0 + i) * a.v.stride + hk,
                                       q + q0 * a.q.stride + h0, a.q.stride, d_o + q0 * g.d_o.stride + h0, g.d_o.stride,
                                       sums, g.blocks, G, max(i - off, 0), lq, d, a.scale, x1, x2);
      } else {
        const int64_t h0 = static_cast<int64_t>(head) * d, hk = static_cast<int64_t>(head / G) * d;
        const float* s = sums + static_cast<int64_t>(i / kSumRows) * (2 * kSumRows) + i % kSumRows;
        grad_query_row<__nv_bfloat16, D>(q + (q0 + i) * a.q.stride + h0, d_o + (q0 + i) * g.d_o.stride + h0, s[0],
                                         s[kSumRows], k + k0 * a.k.stride + hk, a.k.stride, v + k0 * a.v.stride + hk,
                                         a.v.stride, min(i + off + 1, lk), d, a.scale, x1);
      }
    };
    if (!KEYS || t.split == 1) {
      if (__all_sync(0xffffffffu, ok)) {
        // this thread's columns of a row, of dV and then dK, or of dQ, up to 64 at a time
        constexpr int PW = C::kOut < 64 ? C::kOut : 64;
#pragma unroll 1
        for (int start = part * C::kOut; start < (part + 1) * C::kOut; start += PW) {
          const bool of_v = KEYS && start < D;
          const int c0 = start % D;
          const RowsOut& to = KEYS ? (of_v ? g.dv : g.dk) : g.dq;
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(to.p) + ((KEYS ? k0 : q0) + row0) * to.stride +
                               static_cast<int64_t>(head) * d + c0;
          const float f = of_v ? 1.f : a.scale;
          const uint64_t f2 = pack2(f, f);
          const uint32_t from = mine + (of_v ? C::kColV : C::kColS) + c0;
          uint64_t rest = 0;  // z * 0 added up: NaN where some z is not finite
          // a warp's 32 rows through shared memory (the ring's place: every product is done), so that a store covers
          // whole lines
          uint8_t* stage = ring + (start >> 6) * kTile * 128;
          const int sc = start & 63;
#pragma unroll
          for (int c = 0; c < PW; c += 32) {
            uint32_t v[32];
            if (n > 0) {
              tmem_ld32(from + c, v);
              tmem_wait_ld();
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = 0;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint64_t z = mul2(pack2(__uint_as_float(v[8 * e + 2 * k]), __uint_as_float(v[8 * e + 2 * k + 1])), f2);
                float z0, z1;
                rest = fma2(z, 0, rest);
                unpack2(z, z0, z1);
                w[k] = pack_bf16(z0, z1);
              }
              *reinterpret_cast<uint4*>(stage + sw128(r, sc + c + e * 8)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          __syncwarp();
          constexpr int kPieces = PW / 8;  // 16 bytes each
#pragma unroll
          for (int e = 0; e < kPieces; ++e) {
            const int x = e * 32 + lane, rr = quad * 32 + x / kPieces, c = x % kPieces * 8;
            if (row0 + rr >= rows || (D == 64 && c0 + c >= d)) continue;
            *reinterpret_cast<uint4*>(dst + rr * to.stride + c) = *reinterpret_cast<const uint4*>(stage + sw128(rr, sc + c));
          }
          float ra, rb;
          unpack2(rest, ra, rb);
          __syncwarp();
          for (uint32_t again = __ballot_sync(0xffffffffu, row < rows && !(ra + rb == 0.f)); again; again &= again - 1) {
            const int i = row0 + quad * 32 + __ffs(again) - 1;
            float x1[4], x2[4];
            compute_again(i, x1, x2);
            // this warp's part of the row
#pragma unroll
            for (int m = 0; m < D / 32; ++m) {
              const int c = m * 32 + lane;
              if (m * 32 >= c0 && m * 32 < c0 + PW && c < d)
                dst[(i - row0) * to.stride + c - c0] = __float2bfloat16_rn(of_v ? x2[m] : x1[m]);
            }
          }
        }
      }
    } else {
      // The sums in fp32 to shared memory (the ring's place and on: every product is done), 128 rows of dV, then of dK,
      // 16-byte pieces swizzled by row; then each CTA adds up its share of the rows.
#pragma unroll 1
      for (int start = part * C::kOut; start < (part + 1) * C::kOut; start += 32) {
        const int c0 = start % D;
        uint8_t* dst = smem + start / D * (kTile * D * 4) + r * D * 4;
        uint32_t v[32];
        if (n > 0 && ok) {
          tmem_ld32(mine + C::kColV + start, v);  // the sums of dK lie behind those of dV
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = 0;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
          *reinterpret_cast<uint4*>(dst + (((c0 >> 2) + e) ^ (r & 7)) * 16) =
              make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
      }
      cluster_sums<__nv_bfloat16, D, 32 * C::kWarps>(g, smem, &bar->failed, bar->bad, t.split, rank, row0, rows, k0, head, d, compute_again);
    }
    tc_fence_before();
  }
  if (KEYS && t.split > 1 && warp >= C::kLoadWarp) {
    __syncwarp();
    cluster_barrier();
    cluster_barrier();
  }
  __syncthreads();
  if (warp == C::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
}

template <int D, bool KEYS>
int launch_kernel(TcGradArgs& t, int64_t grid, const CUtensorMap (&m)[4], cudaStream_t s) {
  if (grid < 1 || grid > INT32_MAX / t.split) return FALCON_ERR_UNSUPPORTED;
  t.stall = take_test_stall() ? 1 : 0;
  const auto kern = attn_grad_tc_kernel<D, KEYS>;
  if (!set_smem_limit(reinterpret_cast<const void*>(kern), smem_bytes<D, KEYS>())) return FALCON_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid * t.split));
  cfg.blockDim = dim3(Cfg<D, KEYS>::kThreads);
  cfg.dynamicSmemBytes = smem_bytes<D, KEYS>();
  cfg.stream = s;
  cudaLaunchAttribute attr[2] = {overlap_attribute(), cluster_attribute(t.split)};
  cfg.attrs = attr;
  cfg.numAttrs = t.split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, m[0], m[1], m[2], m[3], t) == cudaSuccess ? FALCON_OK : FALCON_ERR_CUDA;
}

template <int D>
int launch_d(const GradArgs& g, cudaStream_t s) {
  const PromptArgs& a = g.a;
  TcGradArgs t;
  t.g = g;
  t.qblocks = 0, t.packed = false, t.split = 1;
  t.status = static_cast<uint32_t*>(a.ws);
  t.limit = wait_limit_ns();
  CUtensorMap m[4];
  auto maps = [&](const RowsIn& x, int64_t n, int H, int rows, CUtensorMap* to) { return make_rows_map(to, x, n, H, a.d, rows); };
  t.second = false;
  if (g.dk.p) {  // first: its CTAs run longest
    constexpr int N = Cfg<D, true>::kN;
    const int64_t blocks = a.k_tokens / kTile + a.B;
    if (blocks > INT32_MAX / a.Hkv) return FALCON_ERR_UNSUPPORTED;
    if (!maps(a.k, a.k_tokens, a.Hkv, kTile, m) || !maps(a.v, a.k_tokens, a.Hkv, kTile, m + 1) ||
        !maps(a.q, a.tokens, a.Hq, N, m + 2) || !maps(g.d_o, a.tokens, a.Hq, N, m + 3))
      return FALCON_ERR_CUDA;
    const int64_t ctas = blocks * a.Hkv;
    t.split = keys_split(a, N, sm_count() * Cfg<D, true>::kCtas, D == 64 ? 4 : 2, D == 64 ? 14 : 9);
    const int st = launch_kernel<D, true>(t, ctas, m, s);
    if (st != FALCON_OK) return st;
    t.split = 1;
    t.second = true;
  }
  if (g.dq.p) return launch_attn_grad_dq_tc(g, t.second, s);
  return FALCON_OK;
}

}  // namespace

// The tensor-core kernels take bf16 rows on 16-byte boundaries (their TMA copies and stores), with token strides below
// the maps' 2^40 bytes.
bool attn_grad_tc_supported(const GradArgs& g, int dtype) {
  const PromptArgs& a = g.a;
  if (dtype != FALCON_BF16 || a.k_tokens == 0 || a.tokens == 0 || a.max_q == 0) return false;
  if (!a.q.vec || !a.k.vec || !a.v.vec || !g.d_o.vec) return false;
  for (const RowsOut& x : {g.dq, g.dk, g.dv})
    if (x.p && !x.vec) return false;
  for (int64_t st : {a.q.stride, a.k.stride, a.v.stride, g.d_o.stride})
    if (st * 2 >= (int64_t(1) << 40)) return false;
  return true;
}

int launch_attn_grad_tc(const GradArgs& g, cudaStream_t s) {
  return g.a.d <= 64 ? launch_d<64>(g, s) : launch_d<128>(g, s);
}

}  // namespace falcon
