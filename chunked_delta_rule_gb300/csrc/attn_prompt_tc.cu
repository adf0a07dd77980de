// Causal attention over packed prompts on the tensor cores (bf16).
//
//   S = Q K^T (128 queries x 128 keys),  P = exp(scale S - m),  O += P V
//
// The floor is the tensor cores': 4 d flops a visible (query, key) pair and head.
// A CTA takes 256 queries of one head as two 128-row tiles (d = 128), or two
// CTAs of an SM one tile each (d = 64): while one tile's P V and next Q K^T run,
// the other's softmax does, so that neither waits for the other:
//   softmax warps    d = 128: 8 a tile, two threads a row, 64 of a tile's keys
//                    each; d = 64: 4, a thread a row (two threads of 96
//                    registers measured 78 us where one takes 70).  The scores
//                    are read from TMEM once; P (bf16) goes back there as the
//                    next product's A operand
//   load warp        TMA: queries, K and V tiles through a ring
//   a warp a tile    the products (idle warps fill the last warpgroup)
// TMEM: S0 | S1 (128 columns each, P in their first 64) | O0 | O1 (d each), or
// S | P | O at d = 64.  Rows of 16 and 32 dims run as 64, the rest zeros from the
// TMA copies: 8 x 2048 x 12 heads of 32 take 64 us, 248 with warp-level tf32 MMAs.
// The grid has a block for every 256 (128) queries and head, the longest rows
// first where max_q is near the lengths.  At d = 64, where a block is over in 2 to 20 us, a CTA that nears its
// end asks for one of those that have not begun and goes on with it: the next
// queries come while the last rows are written.  8 x 2048 x 12 heads: 77 us with
// a CTA a block, 66 so, 70 with the blocks dealt out beforehand; 8 ragged prompts
// of <= 2048: 47, 39 and 63 us.
// Measured: 8 x 2048 x 12 heads, d = 64: 67 us, 775 TFLOP/s, bound by the softmax
// warps' latencies (half the issue slots, a third of the tensor cores' time);
// 16384 x 16/4 heads, d = 128: 714 us, 1540 TFLOP/s, bound by the products in the
// main loop.  (Both with the flops of the visible pairs alone.)
//
// The reference m of a row is the maximum of its first tile.  Weights, sums and
// O keep their relative precision at any scale (bf16 has fp32's range), so m
// moves, and O is rescaled, only after a tile whose sum passed 2^40: the other
// tiles need no maximum.  A tile that passes m by 2^64 at once is weighed again
// against its own maximum before anything uses it (d <= 64: 0.3 us of 66).  At d = 128
// the two threads of a row would have to agree on that at every tile: with a barrier
// 920 us where 709 are, with the maximum taken first 738.  There a tile that overflows
// (2^127) sends its row through the definition as below.  Sums are of the unrounded
// weights, fp32.
// P is rounded to bf16 as V is held in it: at most 2^-8 of a weight.
//
// Masked scores are set to -inf after the product, so what the masked keys
// hold does not matter; a masked weight is 0, but 0 times an infinite or NaN
// value of a key that only other rows see would still spoil the row.  A row
// whose result is not finite is therefore computed again from the definition,
// by its warp, touching only the keys that it sees, after the CTA's last block: a
// CTA that has found such rows asks for no further one.

#include "attn_row.cuh"
#include "tc_util.cuh"

namespace falcon {
namespace {

using namespace tcu;

constexpr int kTile = 128;        // queries and keys of a tile
constexpr float kMost = 1099511627776.f;  // 2^40: a larger sum of a tile's weights moves the reference at the next,
constexpr float kFar = 1.8446744e19f;     // 2^64: at once (d = 64)

// One block of queries of one head: where its rows and keys are, and the tiles of
// keys that each of its query tiles sees.
template <int TILES>
struct Item {
  uint32_t id;  // of the grid
  int h, hk, lq, lk, off, row0, nmax, n[TILES];
  int64_t q0, k0;
  bool valid;
};
struct Bars {
  uint64_t q[2], q_free[2], full[5], empty[5], s[2], p[2], read, o, drain[2], stall;
  uint64_t answer;  // its barrier
  uint4 next;       // answer to the request for one more block
  Item<1> item[2];  // whose queries the buffers hold (d = 64)
  uint32_t tmem;
  uint32_t stop;    // some row has to be computed again: no more blocks are asked for
  uint2 again[4][4];  // (block, rows) of them: 4 entries a warp (d = 64)
  float row[2][kTile];  // of each tile: what the two threads of a row tell each other
};

template <int D>
struct Cfg {
  static constexpr int kTiles = D == 64 ? 1 : 2;          // query tiles of a CTA
  static constexpr int kCtas = D == 64 ? 2 : 1;           // CTAs of an SM
  static constexpr int kSplit = D == 64 ? 1 : 2;          // softmax threads of a row
  static constexpr int kWarps = 4 * kSplit;               // softmax warps of a tile
  static constexpr int kLoadWarp = kWarps * kTiles, kMmaWarp = kLoadWarp + 1;
  static constexpr int kThreads = 32 * kLoadWarp + 128;
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kStages = D == 64 ? 4 : 5;
  static constexpr bool kLoop = D == 64;                  // a CTA takes one block of queries after another, or one
  static constexpr int kQBufs = kLoop ? 2 : 1;            // query buffers
  static constexpr int kSmem = (kQBufs * kTiles + kStages) * kTileBytes + 1024 + static_cast<int>(sizeof(Bars));
  static_assert(kSmem <= 227 * 1024, "more shared memory than a CTA can have");
  // d = 64 leaves room for P beside S, so that S of the next keys is formed
  // while the softmax of these runs; at d = 128 P lies over S
  static constexpr bool kAhead = D == 64;
  static constexpr uint32_t kColS = 0, kColP = kAhead ? 128 : 0, kColO = kAhead ? 192 : kTiles * kTile;
  static constexpr uint32_t kCols = D == 64 ? 256 : 512;
};

struct TcArgs {
  PromptArgs a;
  int qblocks;  // of a sequence
  bool packed;
  uint32_t* status;
  uint64_t limit;
  int stall;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// pairs of floats in one instruction
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t x, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

// Asks for a block of the grid that has not begun; the 16-byte answer is counted on `bar`.
__device__ __forceinline__ void request_block(uint4* answer, uint64_t* bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   smem_u32(answer)),
               "r"(smem_u32(bar))
               : "memory");
}
// Its index, if one was given to this CTA.  After a refusal nothing may be asked for again.
__device__ __forceinline__ bool block_given(const uint4* answer, uint32_t& x) {
  uint32_t ok, id;
  asm volatile(
      "{\n\t.reg .b64 lo, hi;\n\t.reg .b128 r;\n\t.reg .pred p;\n\t"
      "ld.shared.v2.b64 {lo, hi}, [%2];\n\t"
      "mov.b128 r, {lo, hi};\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
      : "=r"(ok), "=r"(id)
      : "r"(smem_u32(answer))
      : "memory");
  if (ok) x = id;
  return ok != 0;
}
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// tiles of 128 keys that rows up to (and with) `last` of a sequence see
__device__ __forceinline__ int key_tiles(int last, int off, int lk) {
  const int n = min(last + off + 1, lk);
  return n <= 0 ? 0 : (n + kTile - 1) / kTile;
}

template <int TILES>
__device__ __forceinline__ Item<TILES> item_at(const TcArgs& t, uint32_t id) {
  const PromptArgs& a = t.a;
  Item<TILES> w;
  w.id = id;
  int b;
  if (t.packed) {
    const int2 x = packed_block(a.cu_q, a.B, TILES * kTile, static_cast<int>(id / a.Hq));
    b = x.x, w.row0 = x.y, w.h = static_cast<int>(id % a.Hq);
  } else {
    // the longest rows first: blocks of queries descend, sequences and heads within
    const uint32_t bh = static_cast<uint32_t>(a.B) * a.Hq, at = id % bh;
    b = static_cast<int>(at) / a.Hq, w.h = static_cast<int>(at) % a.Hq;
    w.row0 = (t.qblocks - 1 - static_cast<int>(id / bh)) * TILES * kTile;
  }
  w.hk = w.h / (a.Hq / a.Hkv);
  w.q0 = a.cu_q[b], w.k0 = a.cu_k[b];
  const int lq_all = static_cast<int>(a.cu_q[b + 1] - w.q0);
  w.lk = static_cast<int>(a.cu_k[b + 1] - w.k0);
  w.lq = min(lq_all, a.max_q);
  w.off = w.lk - lq_all;
  w.valid = w.row0 >= 0 && w.row0 < w.lq && w.q0 >= 0 && w.k0 >= 0 && w.q0 + lq_all <= a.tokens && w.k0 + w.lk <= a.k_tokens;
  w.nmax = 0;
#pragma unroll
  for (int x = 0; x < TILES; ++x) {
    const int r = w.row0 + x * kTile;
    w.n[x] = w.valid && r < w.lq ? key_tiles(min(r + kTile, w.lq) - 1, w.off, w.lk) : 0;
    w.nmax = max(w.nmax, w.n[x]);
  }
  return w;
}

template <int D>
__global__ void __launch_bounds__(Cfg<D>::kThreads, Cfg<D>::kCtas)
    attn_prompt_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                          const __grid_constant__ CUtensorMap mv, const TcArgs t) {
  using C = Cfg<D>;
  const PromptArgs& a = t.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (blockIdx.x == 0 && tid == 0) atomicExch(t.status, 0u);  // before any wait of this call can run out

  using W = Item<C::kTiles>;
  W first;
  if constexpr (!C::kLoop) first = item_at<C::kTiles>(t, blockIdx.x);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint8_t* sQ = smem;
  uint8_t* ring = smem + C::kQBufs * C::kTiles * C::kTileBytes;
  Bars* bar = reinterpret_cast<Bars*>(ring + C::kStages * C::kTileBytes);
  if (warp == C::kMmaWarp) {
    tmem_alloc(&bar->tmem, C::kCols);
    tmem_relinquish();
  }
  if (warp == C::kLoadWarp && lane == 0) {
    for (int x = 0; x < C::kTiles; ++x) {
      mbar_init(&bar->s[x], 1);
      mbar_init(&bar->drain[x], 1);
      mbar_init(&bar->p[x], C::kWarps);
    }
    for (int i = 0; i < C::kQBufs; ++i) {
      mbar_init(&bar->q[i], 1);
      mbar_init(&bar->q_free[i], C::kLoadWarp + C::kTiles);
    }
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&bar->full[i], 1);
      mbar_init(&bar->empty[i], C::kTiles);
    }
    mbar_init(&bar->read, C::kWarps);
    mbar_init(&bar->o, 1);
    mbar_init(&bar->stall, 1);
    mbar_init(&bar->answer, 1);
    bar->stop = 0;
    if constexpr (C::kLoop)
      for (int i = 0; i < 16; ++i) bar->again[i >> 2][i & 3].y = 0;
    fence_mbar_init();
  }
  __syncthreads();
  const uint32_t tmem = bar->tmem;
  auto wait = [&](uint64_t* m, uint32_t parity) {
    if (mbar_wait_sleep(m, parity, t.limit)) return true;
    atomicExch(t.status, kStatusTimeout);
    return false;
  };

  // the CTA's next item, if there is one: with more than one to a CTA the load warp leaves it beside the queries
  auto take = [&](int used, W& w) {
    if constexpr (C::kLoop) {
      if (!wait(&bar->q[used % C::kQBufs], (used / C::kQBufs) & 1)) return false;
      w = bar->item[used % C::kQBufs];
      return w.valid;
    } else {
      w = first;
      return used == 0 && w.valid;
    }
  };

  // registers: the softmax threads take what the last warpgroup gives up
  // (512 x 104 + 128 x 64 = 640 x 96; 128 x 200 + 128 x 56 = 256 x 128)
  if (warp >= C::kLoadWarp) {
    if (D == 64) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
  }
  if (warp == C::kLoadWarp) {
    // K and V through the ring (K0 V0 K1 V1 ...), the queries of an item ahead of its first keys; what it waits
    // for never waits for it, and after a wait that ran out it begins no more
    if (lane == 0) {
      bool ok = !t.stall || wait(&bar->stall, 0);
      int loads = 0, used = 0;  // of the ring, of the query buffers
      uint32_t id = blockIdx.x;
      bool end = false;
      for (int round = 0; ok && (C::kLoop || round == 0); ++round) {
        W w;
        if (end) w.valid = false, w.nmax = 0;  // one without queries: the end
        else if constexpr (C::kLoop) w = item_at<C::kTiles>(t, id);
        else w = first;
        if (w.valid || end) {
          const int buf = used % C::kQBufs;
          if (used >= C::kQBufs && !(ok = wait(&bar->q_free[buf], (used / C::kQBufs - 1) & 1))) break;
          if constexpr (C::kLoop) bar->item[buf] = w;
          if (w.nmax > 0) {
            mbar_arrive_expect_tx(&bar->q[buf], C::kTiles * C::kTileBytes);
            for (int x = 0; x < C::kTiles; ++x)
              for (int c = 0; c < D / 64; ++c)
                tma_load_3d(sQ + (buf * C::kTiles + x) * C::kTileBytes + c * kTile * 128, &mq, &bar->q[buf], c * 64,
                            w.h, static_cast<int>(w.q0 + w.row0 + x * kTile));
          } else {
            mbar_arrive(&bar->q[buf]);
          }
          ++used;
        }
        if (end) break;
        bool asked = false;
        for (int i = 0; i <= 2 * w.nmax; ++i) {
          // one more block, asked for shortly before it is needed
          if (C::kLoop && i == max(2 * w.nmax - 4, 0) && !*static_cast<volatile uint32_t*>(&bar->stop)) {
            asked = true;
            mbar_arrive_expect_tx(&bar->answer, 16);
            request_block(&bar->next, &bar->answer);
          }
          if (i == 2 * w.nmax || !ok) continue;
          const int st = loads % C::kStages;
          if (loads >= C::kStages && !(ok = wait(&bar->empty[st], (loads / C::kStages - 1) & 1))) continue;
          mbar_arrive_expect_tx(&bar->full[st], C::kTileBytes);
          for (int c = 0; c < D / 64; ++c)
            tma_load_3d(ring + st * C::kTileBytes + c * kTile * 128, (i & 1) ? &mv : &mk, &bar->full[st], c * 64, w.hk,
                        static_cast<int>(w.k0 + (i >> 1) * kTile));
          ++loads;
        }
        if (!C::kLoop) break;
        if (!asked) {
          end = true;
          continue;
        }
        ok = wait(&bar->answer, round & 1) && ok;
        if (ok) end = !block_given(&bar->next, id);
        fence_proxy_async();  // the answer has been read before the next is written
      }
      // every copy has landed before the CTA may end
      for (int i = max(0, used - C::kQBufs); i < used; ++i) wait(&bar->q[i % C::kQBufs], (i / C::kQBufs) & 1);
      for (int i = max(0, loads - C::kStages); i < loads; ++i)
        wait(&bar->full[i % C::kStages], (i / C::kStages) & 1);
    }
  } else if (warp >= C::kMmaWarp && warp < C::kMmaWarp + C::kTiles) {
    // A warp a tile.  With two tiles they take turns (named barriers 9 and 10): a warp has waited for all
    // that its products need before its turn, so that the tensor cores go from one tile to the other without
    // a pause, and the tiles stay half a step apart.  Both walk every step, also after a wait that ran out.
    // The whole warp walks the loop, so that descriptors stay uniform; one lane issues.
    constexpr uint32_t id_s = idesc_bf16(kTile, kTile), id_o = idesc_bf16(kTile, D, false, true);
    const int x = __shfl_sync(0xffffffffu, warp - C::kMmaWarp, 0);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0), tm_s = tm + C::kColS + x * kTile;
    const uint32_t tm_p = tm + C::kColP + x * kTile, tm_o = tm + C::kColO + x * D;
    const uint64_t qd0 = sdesc_k128(smem_u32(sQ + x * C::kTileBytes)), kd = sdesc_k128(smem_u32(ring));
    const uint64_t vd = D == 64 ? sdesc_mn128(smem_u32(ring)) : sdesc_mn128_wide(smem_u32(ring), kTile * 128);
    auto arrived = [&](uint64_t* m, uint32_t parity) {  // one answer for the warp
      return __all_sync(0xffffffffu, wait(m, parity)) != 0;
    };
    auto turn = [&]() {
      if (C::kTiles == 2) named_bar(9 + x, 64);
    };
    auto pass = [&](bool again) {  // the other tile's turn; the first tile has none after its last step
      if (C::kTiles == 2 && (x == 0 || again)) asm volatile("bar.arrive %0, %1;" ::"r"(10 - x), "r"(64) : "memory");
    };
    // each is followed by what its completion tells: S or O is ready, a stage is free
    auto scores = [&](uint64_t qd, int st) {
      const uint64_t ks0 = kd + st * (C::kTileBytes >> 4);
      if (elect_one()) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t at = ((ks >> 2) * kTile * 128 + (ks & 3) * 32) >> 4;
          umma_bf16(tm_s, qd + at, ks0 + at, id_s, ks > 0);
        }
        umma_commit(&bar->s[x]);
        umma_commit(&bar->empty[st]);
      }
      __syncwarp();
    };
    auto values = [&](int st, bool acc, uint64_t* then) {
      const uint64_t vs = vd + st * (C::kTileBytes >> 4);
      if (elect_one()) {
#pragma unroll
        for (int ks = 0; ks < kTile / 16; ++ks) umma_ts(tm_o, tm_p + ks * 8, vs + ks * 128, id_o, acc || ks > 0);
        if (then) umma_commit(then);
        umma_commit(&bar->empty[st]);
      }
      __syncwarp();
    };
    auto leave = [&](int st) {  // a stage that this tile has no use for
      if (elect_one()) mbar_arrive(&bar->empty[st]);
      __syncwarp();
    };
    bool ok = true;
    int tiles = 0;       // this tile's key tiles so far
    int sk = 0, pk = 0;  // stage and phase of the next K; V follows it
    W w;
    for (int used = 0; (C::kLoop || used == 0) && __all_sync(0xffffffffu, take(used, w)); ++used) {
      const int nx = x == 0 ? w.n[0] : w.n[C::kTiles - 1], buf = used % C::kQBufs;
      const uint64_t qd = qd0 + buf * (C::kTiles * C::kTileBytes >> 4);
      if (w.nmax > 0) {
        if (x == 1) pass(true);
        ok = ok && arrived(&bar->full[sk], pk) && arrived(&bar->q[buf], (used / C::kQBufs) & 1);
        if (C::kAhead && nx > 0 && tiles > 0) ok = ok && arrived(&bar->read, (tiles - 1) & 1);  // S is free
        turn();
        if (ok) {
          tc_fence_after();
          if (nx > 0) scores(qd, sk);
          else leave(sk);
        }
        pass(true);
        for (int j = 0; j < w.nmax; ++j) {
          const bool more = j + 1 < w.nmax, mine = j < nx, next = j + 1 < nx;
          int sv = sk + 1, pv = pk;  // stages of V_j and K_{j+1}
          if (sv == C::kStages) sv = 0, pv ^= 1;
          sk = sv + 1, pk = pv;
          if (sk == C::kStages) sk = 0, pk ^= 1;
          if (C::kAhead && next) {
            ok = ok && arrived(&bar->full[sk], pk) && arrived(&bar->read, tiles & 1);
            if (ok) {
              tc_fence_after();
              scores(qd, sk);
            }
          }
          ok = ok && arrived(&bar->full[sv], pv);
          if (!C::kAhead && more) ok = ok && arrived(&bar->full[sk], pk);
          if (mine) ok = ok && arrived(&bar->p[x], tiles & 1);
          turn();
          if (ok) {
            if (mine) {
              tc_fence_after();
              values(sv, j > 0, C::kAhead ? &bar->o : next ? nullptr : &bar->s[x]);
              if (!C::kAhead && next) scores(qd, sk);
            } else {
              leave(sv);
            }
            if (more && !next) leave(sk);
          }
          pass(more);
          tiles += mine;
        }
      }
      if (C::kLoop) {
        __syncwarp();
        if (elect_one()) mbar_arrive(&bar->q_free[buf]);
      }
    }
    if (elect_one()) umma_commit(&bar->drain[x]);  // products in flight end before the memory is freed
    __syncwarp();
    wait(&bar->drain[x], 0);
    __syncwarp();
  } else if (warp < C::kLoadWarp) {
    if (D == 64) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    constexpr int kHalf = kTile / C::kSplit, kOut = D / C::kSplit;  // scores and output dims of a thread
    // with two threads a row, warps w and w + 4 of a tile take the same rows, the first and the second 64 keys
    const int x = warp / C::kWarps, half = C::kSplit == 2 ? (warp >> 2) & 1 : 0, quad = warp & 3, r = quad * 32 + lane;
    const int pair = 1 + x * 4 + quad;  // named barrier of the two warps
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t ts = tmem + C::kColS + x * kTile + half * kHalf + lanes;      // scores
    const uint32_t tp = tmem + C::kColP + x * kTile + half * kHalf / 2 + lanes;  // weights
    const uint32_t to = tmem + C::kColO + x * D + half * kOut + lanes;           // this thread's part of O
    const float sl2 = a.scale * kLog2e;
    float* told = &bar->row[x][r];
    auto any = [&](bool p) {  // over the warps that share the rows
      return C::kSplit == 2 ? named_bar_any(pair, 64, p) : __any_sync(0xffffffffu, p) != 0;
    };
    auto arrive = [&](uint64_t* b) {  // once for the warp: arrivals of 32 lanes on one word take their turns
      __syncwarp();
      if (lane == 0) mbar_arrive(b);
    };
    // rows of the warp (a bit each) of a block from the definition
    auto compute_again = [&](const W& w, uint32_t rows) {
      const int d = D == 64 ? a.d : D;
      for (; rows; rows &= rows - 1) {
        const int i = w.row0 + x * kTile + quad * 32 + __ffs(rows) - 1;
        const int64_t gi = w.q0 + i;
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q.p) + gi * a.q.stride + w.h * d;
        const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(a.k.p) + w.k0 * a.k.stride + w.hk * d;
        const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v.p) + w.k0 * a.v.stride + w.hk * d;
        float y[4], z;
        attention_row<__nv_bfloat16, D>(q, k, a.k.stride, v, a.v.stride, min(i + w.off + 1, w.lk), d, a.scale, y, &z);
        __nv_bfloat16* oi = static_cast<__nv_bfloat16*>(a.o.p) + gi * a.o.stride + w.h * d;
#pragma unroll
        for (int e = 0; e < D / 32; ++e)
          if (lane + 32 * e < d) oi[lane + 32 * e] = __float2bfloat16_rn(y[e]);
        if (a.lse && lane == 0) a.lse[gi * a.Hq + w.h] = z;
      }
    };
    bool ok = true;
    int tiles = 0, ss = 0;  // key tiles and phases of bar->s so far
    W w;
    for (int used = 0; C::kLoop || used == 0; ++used) {
      const bool got = ok && take(used, w);
      if (C::kLoop ? __any_sync(0xffffffffu, !got) : !got) break;
      const int nx = x == 0 ? w.n[0] : w.n[C::kTiles - 1], row = w.row0 + x * kTile + r, buf = used % C::kQBufs;
      const int seen = min(row + w.off + 1, w.lk) - half * kHalf;              // keys that this row sees
      const int all = min(w.row0 + x * kTile + w.off + 1, w.lk) - half * kHalf;  // that every row of the tile sees
      float m = -INFINITY, l = 0.f;  // reference (raw scores), sum over this thread's keys
      float s[kHalf];
      uint32_t u[32];  // packed weights
      // scores of tile j into s, those that the row does not see as -inf
      auto read_scores = [&](int j) {
#pragma unroll
        for (int c = 0; c < kHalf / 32; ++c) {
          uint32_t v[32];
          tmem_ld32(ts + c * 32, v);
#pragma unroll
          for (int i = 0; i < 32; ++i) s[c * 32 + i] = __uint_as_float(v[i]);
        }
        tmem_wait_ld();
        if (j * kTile + kHalf > all) {
          const int lim = seen - j * kTile;
#pragma unroll
          for (int i = 0; i < kHalf; ++i)
            if (i >= lim) s[i] = -INFINITY;
        }
      };
      // weights of s against the reference m, their sum; where P has a place of its own they go there at once
      auto weigh = [&]() {
        const float ref = m == -INFINITY ? 0.f : m * sl2;
        const uint64_t scale2 = pack2(sl2, sl2), ref2 = pack2(-ref, -ref);
        uint64_t l2[2] = {0, 0};  // pairs of +0
#pragma unroll
        for (int c = 0; c < kHalf / 64; ++c) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float p0, p1;
            unpack2(fma2(pack2(s[c * 64 + 2 * i], s[c * 64 + 2 * i + 1]), scale2, ref2), p0, p1);
            p0 = ex2(p0), p1 = ex2(p1);
            l2[i & 1] = add2(l2[i & 1], pack2(p0, p1));
            u[i] = pack_bf16(p0, p1);
          }
          if (C::kAhead) tmem_st32(tp + c * 32, u);
        }
        float la, lb;
        unpack2(add2(l2[0], l2[1]), la, lb);
        return la + lb;
      };
      float lt = 0.f;  // sum of the last tile's weights
      for (int j = 0; j < nx; ++j) {
        ok = wait(&bar->s[x], ss & 1);
        ++ss;
        tc_fence_after();
        read_scores(j);
        if (C::kAhead) {
          tc_fence_before();
          arrive(&bar->read);
          if (tiles > 0) {  // the last product has left P and O
            ok = wait(&bar->o, (tiles - 1) & 1) && ok;
            tc_fence_after();
          }
          ++tiles;
        }
        // also, with two threads a row: both have read their scores, the weights may go over them
        bool move = any(!ok || m == -INFINITY || !(lt <= kMost));
        if (move && any(!ok)) {  // all leave together
          ok = false;
          break;
        }
        for (;;) {
          if (move) {         // the reference moves to the maximum so far
            float t4[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) t4[i] = s[i];
#pragma unroll
            for (int i = 4; i < kHalf - 4; i += 8)
#pragma unroll
              for (int e = 0; e < 4; ++e) t4[e] = max3(t4[e], s[i + e], s[i + 4 + e]);
#pragma unroll
            for (int e = 0; e < 4; ++e) t4[e] = fmaxf(t4[e], s[kHalf - 4 + e]);
            float mn = fmaxf(m, max3(t4[0], t4[1], fmaxf(t4[2], t4[3])));
            if (C::kSplit == 2) {
              if (half == 1) *told = mn;
              named_bar(pair, 64);
              if (half == 0) *told = fmaxf(mn, *told);
              named_bar(pair, 64);
              mn = *told;
            }
            const float f = mn == -INFINITY ? 1.f : ex2((m - mn) * sl2);
            m = mn;
            l *= f;
            if (j > 0) {
#pragma unroll
              for (int c = 0; c < kOut / 16; ++c) {
                uint32_t v[16];
                tmem_ld16(to + c * 16, v);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
                tmem_st16(to + c * 16, v);
              }
            }
          }
          lt = weigh();
          if (move || C::kSplit == 2 || !any(lt > kFar)) break;
          move = true;  // finite scores stay finite
          if (C::kAhead) tmem_wait_st();  // the weights are stored once more
        }
        l += lt;
        if (!C::kAhead) tmem_st32(tp, u);
        tmem_wait_st();
        tc_fence_before();
        arrive(&bar->p[x]);
      }
      if constexpr (C::kLoop) w = bar->item[buf];  // (not held through the loop)
      const int row0 = w.row0, lq = w.lq, h = w.h;
      const int64_t q0 = w.q0;
      if (row0 + x * kTile < lq) {  // some row of this tile is the call's
        if (ok && nx > 0) ok = C::kAhead ? wait(&bar->o, (tiles - 1) & 1) : wait(&bar->s[x], ss & 1);
        if (!C::kAhead && nx > 0) ++ss;
        // without a product to wait for, the queries have to be there before their place is taken
        if (C::kTiles > 1 && ok && nx == 0 && w.nmax > 0) ok = wait(&bar->q[buf], (used / C::kQBufs) & 1);
        if (C::kSplit == 2) {
          named_bar(pair, 64);  // the last maximum has been read
          if (half == 1) *told = l;
        }
        if (!any(!ok)) {
          tc_fence_after();
          if (C::kSplit == 2) {
            if (half == 0) *told += l;
            named_bar(pair, 64);
            l = *told;
          }
          const int d = D == 64 ? a.d : D;  // of the rows
          const bool live = row < lq;
          const int64_t g = q0 + row;
          const float inv = l == 0.f ? 0.f : 1.f / l;
          bool bad = !(l <= 3.402823466e38f);
          const uint64_t inv2 = pack2(inv, inv);
          uint64_t rest = 0;  // z * 0 added up: NaN where some z is not finite
          // a warp's 32 rows x 64 dims through shared memory (the queries' place: every product is done; 16-byte
          // pieces swizzled by row), so that a store covers whole lines
          uint8_t* stage = sQ + (buf * C::kTiles + x) * C::kTileBytes + half * kTile * 128;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t u[32];
            if (nx > 0) {
              tmem_ld32(to + c * 32, u);
              tmem_wait_ld();
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) u[i] = 0;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint64_t z = pack2(__uint_as_float(u[8 * i + 2 * e]), __uint_as_float(u[8 * i + 2 * e + 1]));
                float z0, z1;
                rest = fma2(z, 0, rest);
                unpack2(fma2(z, inv2, 0), z0, z1);
                w[e] = l == 0.f ? 0u : pack_bf16(z0, z1);
              }
              *reinterpret_cast<uint4*>(stage + sw128(r, c * 32 + i * 8)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int rr = quad * 32 + i * 4 + (lane >> 3), c = (lane & 7) * 8, grow = row0 + x * kTile + rr;
            if (grow >= lq || (D == 64 && c >= a.d)) continue;
            const uint4 w = *reinterpret_cast<const uint4*>(stage + sw128(rr, c));
            __nv_bfloat16* out =
                static_cast<__nv_bfloat16*>(a.o.p) + (q0 + grow) * a.o.stride + h * d + half * kOut + c;
            if (a.o.vec) {
              *reinterpret_cast<uint4*>(out) = w;
            } else {
              unsigned short* o16 = reinterpret_cast<unsigned short*>(out);
              const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                o16[2 * e] = static_cast<unsigned short>(ws[e]);
                o16[2 * e + 1] = static_cast<unsigned short>(ws[e] >> 16);
              }
            }
          }
          float ra, rb;
          unpack2(rest, ra, rb);
          bad |= !(ra + rb == 0.f);
          if (live && half == 0 && a.lse) a.lse[g * a.Hq + h] = l == 0.f ? -INFINITY : m * a.scale + logf(l);
          // rows that are not finite, once more from the definition; with two threads a row by the second's warp,
          // after the first's has written its part
          bad = bad && live;
          __syncwarp();
          if (C::kSplit == 2) {
            named_bar(pair, 64);
            if (half == 0) *told = bad ? 1.f : 0.f;
            named_bar(pair, 64);
            bad = half == 1 && (bad || *told > 0.f);
          }
          const uint32_t again = __ballot_sync(0xffffffffu, bad);
          if constexpr (!C::kLoop) {
            compute_again(w, again);
          } else if (again != 0 && lane == 0) {
            // when the pipeline has ended: rows of many keys take longer than a wait in it may
            bar->again[warp][used & 3] = make_uint2(w.id, again);
            *static_cast<volatile uint32_t*>(&bar->stop) = 1;
          }
        } else {
          ok = false;  // all leave together
        }
      }
      if (C::kLoop) {
        fence_proxy_async();  // the next queries' copy comes after what was written here
        arrive(&bar->q_free[buf]);
      }
    }
    // At most two further blocks come to a warp after its first one with such rows: one is on its way, and one may
    // have been asked for; before the next question their queries' place must be free, which comes after `stop`.
    if constexpr (C::kLoop) {
      __syncwarp();
      for (int e = 0; e < 4; ++e) {
        const uint2 g = bar->again[warp][e];
        if (g.y != 0) compute_again(item_at<C::kTiles>(t, g.x), g.y);
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == C::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
}

// [tokens, H, d] bf16 rows, boxes of 64 columns x 128 tokens: zeros past a row's end
bool make_rows_map(CUtensorMap* m, const RowsIn& r, int64_t tokens, int H, int d) {
  EncodeFn enc = get_encode();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)tokens};
  cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)r.stride * 2};
  cuuint32_t box[3] = {64, 1, kTile};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(r.p), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
int launch_tc(const PromptArgs& a, cudaStream_t s) {
  TcArgs t;
  t.a = a;
  const PromptGrid g = prompt_grid(a, Cfg<D>::kTiles * kTile);
  if (g.blocks < 1 || g.blocks > INT32_MAX / a.Hq) return FALCON_ERR_UNSUPPORTED;
  t.qblocks = static_cast<int>(g.blocks / a.B);
  t.packed = g.packed;
  t.status = static_cast<uint32_t*>(a.ws);
  t.limit = wait_limit_ns();
  t.stall = take_test_stall() ? 1 : 0;
  CUtensorMap mq, mk, mv;
  if (!make_rows_map(&mq, a.q, a.tokens, a.Hq, a.d) || !make_rows_map(&mk, a.k, a.k_tokens, a.Hkv, a.d) ||
      !make_rows_map(&mv, a.v, a.k_tokens, a.Hkv, a.d))
    return FALCON_ERR_CUDA;
  const auto kern = attn_prompt_tc_kernel<D>;
  if (!set_smem_limit(reinterpret_cast<const void*>(kern), Cfg<D>::kSmem)) return FALCON_ERR_CUDA;
  kern<<<static_cast<unsigned>(g.blocks * a.Hq), Cfg<D>::kThreads, Cfg<D>::kSmem, s>>>(mq, mk, mv, t);
  return cudaGetLastError() == cudaSuccess ? FALCON_OK : FALCON_ERR_CUDA;
}

}  // namespace

// The tensor-core kernel takes bf16 rows on 16-byte boundaries (its TMA copies),
// with token strides below the maps' 2^40 bytes.  A call of a few short prompts
// is over before its pipeline has filled: 16 tokens x 12 heads of 64 take 8.2 us
// here and 6.2 on warp MMAs, 64 tokens of 32 dims 8.2 and 7.2, but 64 of 64 dims
// 8.2 and 8.9, 128 of 32 dims 8.2 and 9.2.
bool attn_prompt_tc_supported(const PromptArgs& a, int dtype) {
  if (dtype != FALCON_BF16 || a.k_tokens == 0 || (a.d <= 64 && a.k_tokens * a.d <= 2048)) return false;
  if (!a.q.vec || !a.k.vec || !a.v.vec || a.tokens > INT32_MAX || a.k_tokens > INT32_MAX) return false;
  for (int64_t st : {a.q.stride, a.k.stride, a.v.stride})
    if (st * 2 >= (int64_t(1) << 40)) return false;
  return true;
}
int launch_attn_prompt_tc(const PromptArgs& a, cudaStream_t s) {
  return a.d <= 64 ? launch_tc<64>(a, s) : launch_tc<128>(a, s);
}

}  // namespace falcon
