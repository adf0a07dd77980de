// dQ of causal attention over packed prompts on the tensor cores (bf16).
//
//   X = Q K^T,  Y = dO V^T,  P = exp(scale X - log sum),  dS = P (Y - D),  dQ = scale dS K
//
// A CTA takes blocks of 128 queries of one head as it gets ready for them, the longest first; per block the keys come past,
// 128 at a time (d = 64: 64, with two CTAs on an SM).
//   load warp    TMA: Q and dO of the next block, K and V through a ring of pairs
//   clear warp   zeros in the rows of a tile that lie past the sequence
//   MMA warp     ... Y(i) X(i + 1) dQ(i) Y(i + 1) ...: P(i + 1) is formed under dQ(i) and Y(i + 1), dS(i) under X(i + 1)
//   softmax      64 columns of a row a thread: P from X, dS from P and Y; dS goes back to TMEM in bf16
//   warps        over Y, as the A operand of dQ
// Q and dO are copied to TMEM, as the A operands there of X and Y: both operands in shared memory would ask it for 8
// KB a step of 128 x 128 x 16, all that it gives in the 64 cycles of the step, before the TMA writes.  The copy
// of the next block comes before the rows of the last one are written, so that its first products run meanwhile: of
// 20 us that a CTA a block took at 1130 tokens, d = 128, 5 were its beginning and its end (12 documents, 16 heads: 137 us,
// now 113; blocks dealt out beforehand: 130).
// d = 128: 2020 cycles a tile (16384 tokens), 1536 of them products: Y, dS, dQ and the next Y follow one another.
//
// dS is rounded to bf16 as K is held in it: at most 2^-8.  Everything else is fp32.
//
// Masked scores are set to -inf after the product.  A masked weight is 0, but 0 times an infinite or NaN value of a
// row that the owner does not see would spoil it: a row of a result that is not finite is computed again from the
// definition.

#include <algorithm>

#include "attn_grad.cuh"
#include "attn_tc.cuh"

namespace falcon {
namespace {

using namespace tcu;

template <int D>
struct CfgQ {
  static constexpr int kCtas = D == 64 ? 2 : 1;  // of an SM
  static constexpr int kN = D == 64 ? 64 : 128;  // keys of a tile
  static constexpr int kSplit = kN / 64;         // softmax threads of a row; each also writes 64 of the row's dims
  static_assert(D / kSplit == 64, "64 dims a thread");
  static constexpr int kWarps = 4 * kSplit, kLoadWarp = kWarps, kMmaWarp = kWarps + 1;
  static constexpr int kThreads = 32 * kWarps + 128;
  static constexpr int kOwnBytes = kTile * D * 2, kTileBytes = kN * D * 2;
  static constexpr int kPairs = D == 64 ? 4 : 3, kOwnPairs = D == 64 ? 2 : 1;  // of tiles; of them a block's Q and dO
  static constexpr int kRing = 2 * kPairs * kTileBytes;
  // TMEM: X, Y (then dS), dQ, the block's Q and dO
  static constexpr uint32_t kColX = 0, kColY = kN, kColS = 2 * kN, kColA1 = kColS + D, kColA2 = kColA1 + D / 2;
  static constexpr uint32_t kCols = D == 64 ? 256 : 512;
};
struct Block {
  int b, head, row0, lq, lk, off, n;  // n: tiles of keys; below 0: no block
  int64_t q0, k0;
};
struct BarsQ {
  uint64_t ready, full[10], empty[10], raw[10], x, x_read, y, ds, drain, stall, told[2], heard[2];
  Block next[2];  // what the loading warp tells the others
  uint64_t held;  // until when rows that are computed again may hold up the CTA's next block
  uint32_t tmem;
};
constexpr int kRaw = 20;  // from full to raw
static_assert(offsetof(BarsQ, raw) == offsetof(BarsQ, full) + kRaw * sizeof(uint64_t), "places");
template <int D>
constexpr int smem_bytes() {  // the ring, the rows of dQ on their way out
  return CfgQ<D>::kRing + CfgQ<D>::kOwnBytes + 1024 + static_cast<int>(sizeof(BarsQ));
}
static_assert(smem_bytes<128>() <= 227 * 1024 && smem_bytes<64>() <= 113 * 1024, "shared memory");

struct TcQArgs {
  GradArgs g;
  uint32_t blocks;
  int qblocks;  // of a sequence
  bool packed;
  bool second;  // of the call's two kernels
  uint32_t *status, *counter;
  uint64_t limit;
  int stall;
};
template <int D>
__global__ void __launch_bounds__(CfgQ<D>::kThreads, CfgQ<D>::kCtas)
    attn_grad_dq_tc_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap o_map,
                           const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                           const TcQArgs t) {
  using C = CfgQ<D>;
  constexpr int N = C::kN, P = C::kPairs;
  const GradArgs& g = t.g;
  const PromptArgs& a = g.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, G = a.Hq / a.Hkv;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint8_t *ring = smem, *rows_out = ring + C::kRing;
  BarsQ* bar = reinterpret_cast<BarsQ*>(rows_out + C::kOwnBytes);
  if (warp == C::kMmaWarp) {
    tmem_alloc(&bar->tmem, C::kCols);
    tmem_relinquish();
  }
  if (warp == C::kLoadWarp && lane == 0) {
    for (const CUtensorMap* m : {&q_map, &o_map, &k_map, &v_map})
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
    mbar_init(&bar->ready, C::kWarps);
    for (int i = 0; i < 2 * P; ++i) {
      mbar_init(&bar->full[i], 1);
      mbar_init(&bar->empty[i], 1);
      mbar_init(&bar->raw[i], 1);
    }
    mbar_init(&bar->x, 1);
    mbar_init(&bar->x_read, C::kWarps + 1);
    mbar_init(&bar->y, 1);
    mbar_init(&bar->ds, C::kWarps + 1);
    mbar_init(&bar->drain, 1);
    mbar_init(&bar->stall, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar->told[i], 1);
      mbar_init(&bar->heard[i], C::kWarps + 3);
    }
    bar->held = 0;
    fence_mbar_init();
  }
  __syncthreads();
  const uint32_t tmem = bar->tmem;
  if (!t.second) {  // what the sums' kernel wrote is there
    wait_for_previous();
    launch_dependents();
  }
  const bool last = t.second && blockIdx.x == gridDim.x - 1 && tid == C::kThreads - 1;  // ends no sooner than the first kernel
  auto wait = [&](uint64_t* m, uint32_t parity) {
    if (mbar_wait_sleep(m, parity, t.limit, &bar->held)) return true;
    atomicExch(t.status, kStatusTimeout);
    return false;
  };
  // Places of the ring, two of pair j: a block's Q and dO come first (d = 128: a place each, d = 64: a pair each), then its
  // tiles of K and V.
  auto place = [&](int j, int second) { return 2 * (j % P) + second; };
  // The next block that has rows, by the loading warp: the CTA's own number, then the next one that no CTA has asked for,
  // so that CTAs that begin late (the first kernel of the call holds their SM) take fewer.
  bool asked = false;
  auto take = [&] {
    for (;;) {
      uint32_t at = blockIdx.x;
      if (asked) {
        if (lane == 0) at = gridDim.x + atomicAdd(t.counter, 1);
        at = __shfl_sync(0xffffffffu, at, 0);
      }
      asked = true;
      if (at >= t.blocks) break;
      Block x;
      if (t.packed) {
        const int2 y = find_block(a.cu_q, a.B, kTile, static_cast<int>(at / a.Hq));
        x.b = y.x, x.row0 = y.y, x.head = static_cast<int>(at % a.Hq);
      } else {
        const uint32_t bh = static_cast<uint32_t>(a.B) * a.Hq, y = at % bh;
        x.b = static_cast<int>(y) / a.Hq, x.head = static_cast<int>(y) % a.Hq;
        x.row0 = (t.qblocks - 1 - static_cast<int>(at / bh)) * kTile;  // the longest rows first
      }
      x.q0 = a.cu_q[x.b], x.k0 = a.cu_k[x.b];
      const int64_t lq = a.cu_q[x.b + 1] - x.q0, lk = a.cu_k[x.b + 1] - x.k0;
      x.lq = static_cast<int>(min(lq, static_cast<int64_t>(a.max_q)));
      if (x.row0 < 0 || x.row0 >= x.lq || x.q0 < 0 || x.k0 < 0 || lk < 0 || x.q0 + lq > a.tokens || x.k0 + lk > a.k_tokens)
        continue;
      x.lk = static_cast<int>(lk), x.off = static_cast<int>(lk - lq);
      x.n = (max(min(min(x.row0 + kTile, x.lq) + x.off, x.lk), 0) + N - 1) / N;
      return x;
    }
    Block none = {};
    none.n = -1;
    return none;
  };

  // the next block, for the other warps; told = blocks before
  int told = 0;
  auto hear = [&] {
    Block x;
    x.n = -1;
    if (__all_sync(0xffffffffu, wait(&bar->told[told & 1], (told >> 1) & 1))) {
      x = bar->next[told & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar->heard[told & 1]);
    }
    ++told;
    return x;
  };

  // registers: the softmax threads take what the last warpgroup gives up
  // (128 x 200 + 128 x 56 = 256 x 128; 256 x 208 + 128 x 88 = 384 x 168)
  if (warp >= C::kLoadWarp) {
    if (D == 64) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  }
  // In every role: tiles, pairs = those of the blocks before, begun = blocks with tiles before.
  int tiles = 0, pairs = 0, begun = 0;
  constexpr int O = C::kOwnPairs;
  bool ok = true;
  if (warp == C::kLoadWarp) {
    int loads = 0;  // places filled
    if (lane == 0) ok = !t.stall || wait(&bar->stall, 0);
    ok = __all_sync(0xffffffffu, ok);
    for (int told = 0; ok; ++told) {
      const Block x = take();
      if (lane == 0 && (ok = told < 2 || wait(&bar->heard[told & 1], ((told >> 1) - 1) & 1))) {
        bar->next[told & 1] = x;
        mbar_arrive(&bar->told[told & 1]);
      }
      if (x.n < 0) break;
      const int cut = x.n * N > x.lk ? x.n - 1 : x.n;  // the tile that reaches past the sequence
      if (lane == 0 && x.n > 0)
        for (int l = 0; l < 2 * (O + x.n) && ok; ++l, ++loads) {
          const int j = pairs + (l >> 1), second = l & 1, slot = place(j, second), i = (l >> 1) - O;
          uint64_t* full = bar->full + slot + (i == cut ? kRaw : 0);  // of K and V
          if (j >= P && !(ok = wait(&bar->empty[slot], (j / P - 1) & 1))) break;
          uint8_t* to = ring + slot * C::kTileBytes;
          if (i >= 0) {
            mbar_arrive_expect_tx(full, C::kTileBytes);
            for (int c = 0; c < D / 64; ++c)
              tma_load_3d(to + c * N * 128, second ? &v_map : &k_map, full, c * 64, x.head / G,
                          static_cast<int>(x.k0 + i * N));
          } else if (D == 128 || second) {
            // d = 64: both places of the pair are free
            const bool of_o = D == 128 ? second : l >> 1;
            if (D == 64) to -= C::kTileBytes;
            mbar_arrive_expect_tx(&bar->full[slot], C::kOwnBytes);
            for (int c = 0; c < D / 64; ++c)
              tma_load_3d(to + c * kTile * 128, of_o ? &o_map : &q_map, &bar->full[slot], c * 64, x.head,
                          static_cast<int>(x.q0 + x.row0));
          } else {
            mbar_arrive(&bar->full[slot]);
          }
        }
      ok = __all_sync(0xffffffffu, ok);
      if (x.n > 0) pairs += O + x.n;
    }
    // every copy has landed before the CTA may end
    if (lane == 0)
      for (int l = max(0, loads - 2 * P); l < loads; ++l) wait(&bar->full[place(l >> 1, l & 1)], ((l >> 1) / P) & 1);
    __syncwarp();
  } else if (warp == C::kMmaWarp) {
    // One lane issues, see the kernel of dK and dV.
    constexpr uint32_t id_x = idesc_bf16(kTile, N), id_s = idesc_bf16(kTile, D, false, true);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t bk = sdesc_k128(smem_u32(ring));
    const uint64_t bm = D == 64 ? sdesc_mn128(smem_u32(ring)) : sdesc_mn128_wide(smem_u32(ring), N * 128);
    auto arrived = [&](uint64_t* m, uint32_t parity) {
      const bool r = wait(m, parity);
      tc_fence_after();
      return r;
    };
    auto full = [&](int j, int second) { return arrived(&bar->full[place(j, second)], (j / P) & 1); };
    // X (second = 0) or Y of pair j
    auto scores = [&](int j, int second) {
      const int slot = place(j, second);
      const uint64_t bs = bk + slot * (C::kTileBytes >> 4);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
        umma_ts(tm + (second ? C::kColY : C::kColX), tm + (second ? C::kColA2 : C::kColA1) + ks * 8,
                bs + (((ks >> 2) * N * 128 + (ks & 3) * 32) >> 4), id_x, ks > 0);
      umma_commit(second ? &bar->y : &bar->x);
      if (second) umma_commit(&bar->empty[slot]);
    };
    for (Block x = hear(); x.n >= 0 && ok; x = hear()) {
      if (x.n == 0) continue;
      if (elect_one()) {
        const int j0 = pairs + O;
        if ((ok = arrived(&bar->ready, begun & 1))) {
          for (int l = 0; l < 2 * O; ++l) mbar_arrive(&bar->empty[place(pairs + (l >> 1), l & 1)]);  // Q and dO are in TMEM
          if ((ok = full(j0, 0))) scores(j0, 0);
          if (ok && (ok = full(j0, 1))) scores(j0, 1);
        }
        for (int l = 0; l < x.n && ok; ++l) {  // what these wait for holds the next tile's copies too
          const int i = tiles + l, j = j0 + l;
          if (!(ok = arrived(&bar->x_read, i & 1))) break;
          if (l + 1 < x.n) scores(j + 1, 0);
          if (!(ok = arrived(&bar->ds, i & 1))) break;
          const uint64_t bs = bm + place(j, 0) * (C::kTileBytes >> 4);
#pragma unroll
          for (int ks = 0; ks < N / 16; ++ks)
            umma_ts(tm + C::kColS, tm + C::kColY + (ks >> 1) * 32 + (ks & 1) * 8, bs + ks * 128, id_s, l > 0 || ks > 0);
          umma_commit(&bar->empty[place(j, 0)]);
          if (l + 1 < x.n) scores(j + 1, 1);
        }
      }
      ok = __all_sync(0xffffffffu, ok);
      tiles += x.n, pairs += O + x.n, ++begun;
    }
    if (elect_one()) {
      umma_commit(&bar->drain);  // products in flight end before the memory is freed
      wait(&bar->drain, 0);
    }
    __syncwarp();
  } else if (warp == C::kMmaWarp + 1) {
    // waits for the next tile's copies in the MMA warp's place, and joins the softmax warps' arrivals
    for (Block x = hear(); x.n >= 0 && ok; x = hear()) {
      if (x.n == 0) continue;
      if (lane == 0)
        for (int l = 0; l < 2 * x.n && ok; ++l) {
          const int i = tiles + (l >> 1), j = pairs + O + (l >> 1) + 1, second = l & 1;
          uint64_t* m = second ? &bar->ds : &bar->x_read;
          if ((l >> 1) + 1 < x.n) ok = wait(&bar->full[place(j, second)], (j / P) & 1);
          if (!ok) break;
          mbar_arrive(m);
          ok = wait(m, i & 1);  // so that the next arrival counts for the next tile
        }
      ok = __all_sync(0xffffffffu, ok);
      tiles += x.n, pairs += O + x.n;
    }
  } else if (warp == C::kMmaWarp + 2) {
    // The last keys' tile may reach past the sequence: zeros there before it counts as copied, see the kernel of dK and dV.
    // (NaN in all rows behind the last of 8 x 2000 tokens of 12 heads of 64: a call of 11.4 ms without it for 0.21.)
    uint32_t parity = 0;  // a bit each place
    for (Block x = hear(); x.n >= 0 && ok; x = hear()) {
      if (x.n == 0) continue;
      pairs += O + x.n;
      if (x.n * N <= x.lk) continue;
      for (int second = 0; second < 2 && ok; ++second) {
        const int slot = place(pairs - 1, second);
        if (!(ok = __all_sync(0xffffffffu, wait(&bar->raw[slot], (parity >> slot) & 1)))) break;
        parity ^= 1u << slot;
        zero_rows<N, D / 64>(ring + slot * C::kTileBytes, x.lk - (x.n - 1) * N);
        if (lane == 0) mbar_arrive(&bar->full[slot]);
      }
    }
  } else if (warp < C::kLoadWarp) {
    if (D == 64) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int part = warp >> 2, quad = warp & 3, r = quad * 32 + lane;
    const uint32_t mine = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t tx = mine + C::kColX + part * 64, ty = mine + C::kColY + part * 64;
    const float sl2 = a.scale * kLog2e;
    const uint64_t scale2 = pack2(sl2, sl2);
    const int d = D == 64 ? a.d : D;  // of the rows
    auto arrive = [&](uint64_t* m) {  // once for the warp: arrivals of 32 lanes on one word take their turns
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(m);
    };
    auto waited = [&](uint64_t* m, uint32_t parity) {
      const bool w = __all_sync(0xffffffffu, wait(m, parity)) != 0;
      tc_fence_after();
      return w;
    };
    auto sums_of = [&](const Block& x) { return g.sums + row_sums(g.blocks, x.head, first_block(x.q0, x.b)); };
    // a block's Q and dO to TMEM, a slab of 64 columns of each a thread; rows past the sequence are some others', or zeros
    auto bring = [&] {
      const int last = pairs + O - 1;  // d = 64: Q's pair is the one before
      if (!waited(&bar->full[place(pairs, D == 64)], (pairs / P) & 1) || !waited(&bar->full[place(last, 1)], (last / P) & 1))
        return false;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint8_t* from = ring + place(D == 64 && s ? last : pairs, D == 128 && s) * C::kTileBytes + part * kTile * 128;
        uint32_t w[32];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint4 x = *reinterpret_cast<const uint4*>(from + sw128(r, c * 8));
          w[4 * c] = x.x, w[4 * c + 1] = x.y, w[4 * c + 2] = x.z, w[4 * c + 3] = x.w;
        }
        tmem_st32(mine + (s ? C::kColA2 : C::kColA1) + part * 32, w);
      }
      tmem_wait_st();
      arrive(&bar->ready);
      return true;
    };
    Block x = hear();
    float lse = 0.f, delta = 0.f;  // of this thread's query
    if (x.n > 0) {
      const float* s = sums_of(x) + static_cast<int64_t>(x.row0 / kSumRows) * (2 * kSumRows) + r;
      lse = load_past_l1(s), delta = load_past_l1(s + kSumRows);
      ok = bring();
    }
    while (x.n >= 0 && ok) {
      const int row = x.row0 + r;
      const uint64_t lse2 = pack2(-lse * kLog2e, -lse * kLog2e), delta2 = pack2(-delta, -delta);
      for (int l = 0; l < x.n; ++l) {
        const int i = tiles + l, c0 = l * N + part * 64;  // of the first column
        if (!(ok = waited(&bar->x, i & 1))) break;
        uint64_t p[2][16];  // X, then P
        {
          uint32_t v[2][32];
          tmem_ld32(tx, v[0]);
          tmem_ld32(tx + 32, v[1]);
          tmem_wait_ld();
          arrive(&bar->x_read);
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int e = 0; e < 16; ++e) p[c][e] = pack2(__uint_as_float(v[c][2 * e]), __uint_as_float(v[c][2 * e + 1]));
        }
        if (c0 + 64 > min(x.row0 + x.off + 1, x.lk)) {  // keys behind a query of these, or past the last
          const int lim = min(row + x.off + 1, x.lk) - c0;
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float z0, z1;
              unpack2(p[c][e], z0, z1);
              if (32 * c + 2 * e >= lim) z0 = -INFINITY;
              if (32 * c + 2 * e + 1 >= lim) z1 = -INFINITY;
              p[c][e] = pack2(z0, z1);
            }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float z0, z1;
            unpack2(fma2(p[c][e], scale2, lse2), z0, z1);
            p[c][e] = pack2(ex2(z0), ex2(z1));
          }
        if (!(ok = waited(&bar->y, i & 1))) break;
        uint32_t v[2][32];
        tmem_ld32(ty, v[0]);
        tmem_ld32(ty + 32, v[1]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t u[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float z0, z1;
            const uint64_t z = add2(pack2(__uint_as_float(v[c][2 * e]), __uint_as_float(v[c][2 * e + 1])), delta2);
            unpack2(mul2(p[c][e], z), z0, z1);
            u[e] = pack_bf16(z0, z1);
          }
          tmem_st16(ty + 32 * c, u);
        }
        tmem_wait_st();
        arrive(&bar->ds);
      }
      // the block's last product
      if (ok && x.n > 0) {
        const int j = pairs + O + x.n - 1;
        ok = waited(&bar->empty[place(j, 0)], (j / P) & 1);
        tiles += x.n, pairs += O + x.n;
      }
      if (!ok) break;
      // the next block's rows first: its first products run while this one's results are written
      const Block next = hear();
      if (next.n > 0) {
        const float* s = sums_of(next) + static_cast<int64_t>(next.row0 / kSumRows) * (2 * kSumRows) + r;
        lse = load_past_l1(s), delta = load_past_l1(s + kSumRows);
        if (!(ok = bring())) break;
      }
      // this thread's 64 dims of a row; a warp's 32 rows through shared memory, so that a store covers whole lines
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(g.dq.p) + (x.q0 + x.row0) * g.dq.stride +
                           static_cast<int64_t>(x.head) * d + part * 64;
      uint8_t* stage = rows_out + part * kTile * 128;
      const uint64_t f2 = pack2(a.scale, a.scale);
      uint64_t rest = 0;  // z * 0 added up: NaN where some z is not finite
      __syncwarp();  // the last block's rows have been read
#pragma unroll
      for (int c = 0; c < 64; c += 32) {
        uint32_t v[32];
        if (x.n > 0) {
          tmem_ld32(mine + C::kColS + part * 64 + c, v);
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
          *reinterpret_cast<uint4*>(stage + sw128(r, c + e * 8)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      __syncwarp();
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int y = e * 32 + lane, rr = quad * 32 + y / 8, c = y % 8 * 8;
        if (x.row0 + rr >= x.lq || (D == 64 && c >= d)) continue;
        *reinterpret_cast<uint4*>(dst + rr * g.dq.stride + c) = *reinterpret_cast<const uint4*>(stage + sw128(rr, c));
      }
      float ra, rb;
      unpack2(rest, ra, rb);
      __syncwarp();
      uint32_t again = __ballot_sync(0xffffffffu, row < x.lq && !(ra + rb == 0.f));
      // They hold up the CTA's next block: no wait runs out meanwhile.  2 us a key and row, several times what it takes.
      // (Counts of the warps that begin and end, looked at where a wait runs out: 212 us for 205 at 8 x 2048.)
      if (again && lane == 0)
        atomicMax(reinterpret_cast<unsigned long long*>(&bar->held),
                  globaltimer() + static_cast<uint64_t>(__popc(again)) * x.lk * 2000);
      for (; again; again &= again - 1) {
        const int i = x.row0 + quad * 32 + __ffs(again) - 1;
        float z[4];
        const __nv_bfloat16 *q = static_cast<const __nv_bfloat16*>(a.q.p), *d_o = static_cast<const __nv_bfloat16*>(g.d_o.p);
        const __nv_bfloat16 *k = static_cast<const __nv_bfloat16*>(a.k.p), *v = static_cast<const __nv_bfloat16*>(a.v.p);
        const int64_t h0 = static_cast<int64_t>(x.head) * d, hk = static_cast<int64_t>(x.head / G) * d;
        const float* s = sums_of(x) + static_cast<int64_t>(i / kSumRows) * (2 * kSumRows) + i % kSumRows;
        grad_query_row<__nv_bfloat16, D>(q + (x.q0 + i) * a.q.stride + h0, d_o + (x.q0 + i) * g.d_o.stride + h0,
                                         load_past_l1(s), load_past_l1(s + kSumRows), k + x.k0 * a.k.stride + hk,
                                         a.k.stride, v + x.k0 * a.v.stride + hk, a.v.stride, min(i + x.off + 1, x.lk), d,
                                         a.scale, z);
#pragma unroll
        for (int m = 0; m < D / 32; ++m) {
          const int c = m * 32 + lane;
          if (m / 2 == part && c < d) dst[(i - x.row0) * g.dq.stride + c - part * 64] = __float2bfloat16_rn(z[m]);
        }
      }
      x = next;
    }
    tc_fence_before();
  }
  if (last) wait_for_previous();
  __syncthreads();
  if (warp == C::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
}

template <int D>
int launch_d(const GradArgs& g, bool second, cudaStream_t s) {
  using C = CfgQ<D>;
  const PromptArgs& a = g.a;
  const PromptGrid pg = prompt_grid(a, kTile);
  if (pg.blocks < 1 || pg.blocks > INT32_MAX / a.Hq) return FALCON_ERR_UNSUPPORTED;
  CUtensorMap m[4];
  if (!make_rows_map(m, a.q, a.tokens, a.Hq, a.d) || !make_rows_map(m + 1, g.d_o, a.tokens, a.Hq, a.d) ||
      !make_rows_map(m + 2, a.k, a.k_tokens, a.Hkv, a.d, C::kN) || !make_rows_map(m + 3, a.v, a.k_tokens, a.Hkv, a.d, C::kN))
    return FALCON_ERR_CUDA;
  TcQArgs t;
  t.g = g;
  t.blocks = static_cast<uint32_t>(pg.blocks * a.Hq);
  t.qblocks = static_cast<int>(pg.blocks / a.B);
  t.packed = pg.packed;
  t.second = second;
  t.status = static_cast<uint32_t*>(a.ws);
  t.counter = t.status + 1;
  t.limit = wait_limit_ns();
  t.stall = take_test_stall() ? 1 : 0;
  const auto kern = attn_grad_dq_tc_kernel<D>;
  if (!set_smem_limit(reinterpret_cast<const void*>(kern), smem_bytes<D>())) return FALCON_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  // up to two rounds of blocks a CTA each: blocks asked for ahead would leave SMs without work
  const uint32_t slots = sm_count() * C::kCtas;
  cfg.gridDim = dim3(t.blocks <= 2 * slots ? t.blocks : slots);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = smem_bytes<D>();
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {overlap_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, m[0], m[1], m[2], m[3], t) == cudaSuccess ? FALCON_OK : FALCON_ERR_CUDA;
}

}  // namespace

int launch_attn_grad_dq_tc(const GradArgs& g, bool second, cudaStream_t s) {
  return g.a.d <= 64 ? launch_d<64>(g, second, s) : launch_d<128>(g, second, s);
}

}  // namespace falcon
