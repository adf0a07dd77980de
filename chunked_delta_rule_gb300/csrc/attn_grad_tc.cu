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
// V^T, the keys come past).  Per tile of rows that come past:
//   load warp    TMA: the two tiles, through a ring of pairs
//   MMA warp     X, Y and the sums' products in the order that keeps the tensor
//                cores ahead of the softmax warps, see the loops
//   softmax      4 warps (d = 64, a thread a row) or 8 (d = 128, two threads a row),
//   warps        64 columns each: P from X, dS from P and Y.  P and dS go back to
//                TMEM in bf16 over the scores that they came from, as the A operand
//                of the sums' products.
// dK and dV: a thread holds one key and 64 queries, so that log sums and D would be
// loads for every element; they come out of the products instead, one more step of 16
// columns: [K | 1] [Q | -log sum / scale]^T and [V | 1] [dO | -D]^T, in three bf16
// parts (24 bits).
//
// P and dS are rounded to bf16 as V and K are held in it: at most 2^-8 of each.
// Everything else is fp32.
//
// Masked scores are set to -inf after the product.  A masked weight is 0, but 0
// times an infinite or NaN value of a row that the owner does not see would spoil
// it: a row of a result that is not finite is computed again from the definition,
// after the pipeline has ended.

#include "attn_grad.cuh"
#include "attn_tc.cuh"

namespace falcon {
namespace {

using namespace tcu;

template <int D, bool KEYS>
struct Cfg {
  static constexpr int kCtas = D == 64 ? 2 : 1;           // CTAs of an SM
  static constexpr int kN = D == 64 ? 64 : 128;           // rows of a tile that comes past
  static constexpr int kSplit = D == 64 ? 1 : 2;          // softmax threads of a row, 64 columns each
  static constexpr int kWarps = 4 * kSplit;
  static constexpr int kLoadWarp = kWarps, kMmaWarp = kWarps + 1;
  static constexpr int kThreads = 32 * kWarps + 128;
  static constexpr int kOwnBytes = kTile * D * 2, kTileBytes = kN * D * 2;
  static constexpr int kPairs = D == 64 ? 3 : 2;
  static constexpr int kImage = kN * 32;                  // log sums and D of a tile of queries
  static constexpr int kExtra = KEYS ? kPairs * kImage + 2 * kImageBytes : 0;
  // X (two of them for dQ: the next one is formed while this one's dS lies over it), Y, sums
  static constexpr uint32_t kColX = 0, kColY = KEYS ? kN : 2 * kN, kColV = 2 * kN, kColS = KEYS ? 2 * kN + D : 3 * kN;
  static constexpr uint32_t kCols = D == 64 ? 256 : 512;
};
struct Bars {
  uint64_t own, full1[3], full2[3], empty1[3], empty2[3], x[2], y, p, ds, drain, stall;
  uint32_t tmem;
};
template <int D, bool KEYS>
constexpr int smem_bytes() {
  using C = Cfg<D, KEYS>;
  return 2 * C::kOwnBytes + 2 * C::kPairs * C::kTileBytes + C::kExtra + 1024 + static_cast<int>(sizeof(Bars));
}
static_assert(smem_bytes<128, true>() <= 227 * 1024 && 2 * (smem_bytes<64, true>() + 1024) <= 228 * 1024, "shared memory");

struct TcGradArgs {
  GradArgs g;
  int qblocks;  // of a sequence
  bool packed;
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
  constexpr int N = C::kN;
  const GradArgs& g = t.g;
  const PromptArgs& a = g.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // whose rows
  const int G = a.Hq / a.Hkv;
  int b, head, row0;
  if constexpr (KEYS) {
    const int2 x = packed_block(a.cu_k, a.B, kTile, static_cast<int>(blockIdx.x / a.Hkv));
    b = x.x, row0 = x.y, head = static_cast<int>(blockIdx.x % a.Hkv);
  } else if (t.packed) {
    const int2 x = packed_block(a.cu_q, a.B, kTile, static_cast<int>(blockIdx.x / a.Hq));
    b = x.x, row0 = x.y, head = static_cast<int>(blockIdx.x % a.Hq);
  } else {
    const uint32_t bh = static_cast<uint32_t>(a.B) * a.Hq, at = blockIdx.x % bh;
    b = static_cast<int>(at) / a.Hq, head = static_cast<int>(at) % a.Hq;
    row0 = (t.qblocks - 1 - static_cast<int>(blockIdx.x / bh)) * kTile;  // the longest rows first
  }
  const int64_t q0 = a.cu_q[b], k0 = a.cu_k[b];
  const int lq_all = static_cast<int>(a.cu_q[b + 1] - q0), lk = static_cast<int>(a.cu_k[b + 1] - k0);
  const int lq = min(lq_all, a.max_q), off = lk - lq_all, rows = KEYS ? lk : lq;
  if (row0 < 0 || row0 >= rows || q0 < 0 || k0 < 0 || q0 + lq_all > a.tokens || k0 + lk > a.k_tokens) return;
  // a sequence's blocks are dealt out from its last; the first keys, which the most queries see, come first
  if (KEYS) row0 = (lk - 1) / kTile * kTile - row0;
  // the tiles that come past: [first, first + each N) of every head
  const int first = KEYS ? max(row0 - off, 0) / N * N : 0;
  const int end = KEYS ? lq : min(min(row0 + kTile, lq) + off, lk);
  const int each = end > first ? (end - first + N - 1) / N : 0, n = KEYS ? each * G : each;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint8_t *s1 = smem, *s2 = s1 + C::kOwnBytes, *ring = s2 + C::kOwnBytes;  // pairs: first tile, second tile
  uint8_t* images = ring + 2 * C::kPairs * C::kTileBytes;
  uint8_t* ones = images + C::kPairs * C::kImage;
  Bars* bar = reinterpret_cast<Bars*>(ring + 2 * C::kPairs * C::kTileBytes + C::kExtra);
  if (warp == C::kMmaWarp) {
    tmem_alloc(&bar->tmem, C::kCols);
    tmem_relinquish();
  }
  if (warp == C::kLoadWarp && lane == 0) {
    mbar_init(&bar->own, 1);
    for (int i = 0; i < C::kPairs; ++i) {
      mbar_init(&bar->full1[i], 1);
      mbar_init(&bar->full2[i], 1);
      mbar_init(&bar->empty1[i], 1);
      mbar_init(&bar->empty2[i], 1);
    }
    mbar_init(&bar->x[0], 1);
    mbar_init(&bar->x[1], 1);
    mbar_init(&bar->y, 1);
    mbar_init(&bar->p, C::kWarps);
    mbar_init(&bar->ds, C::kWarps);
    mbar_init(&bar->drain, 1);
    mbar_init(&bar->stall, 1);
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
  __syncthreads();
  const uint32_t tmem = bar->tmem;
  auto wait = [&](uint64_t* m, uint32_t parity) {
    if (mbar_wait_sleep(m, parity, t.limit)) return true;
    atomicExch(t.status, kStatusTimeout);
    return false;
  };

  // registers: the softmax threads take what the last warpgroup gives up
  // (256 x 208 + 128 x 88 = 384 x 168; 128 x 200 + 128 x 56 = 256 x 128)
  if (warp >= C::kLoadWarp) {
    if (D == 64) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  }
  if (warp == C::kLoadWarp) {
    if (lane == 0 && n > 0) {
      bool ok = !t.stall || wait(&bar->stall, 0);
      int loads = 0, seconds = 0;
      bool own = false;
      if (ok) {
        own = true;
        const int64_t at = (KEYS ? k0 : q0) + row0;
        mbar_arrive_expect_tx(&bar->own, 2 * C::kOwnBytes);
        for (int c = 0; c < D / 64; ++c) {
          tma_load_3d(s1 + c * kTile * 128, &own1, &bar->own, c * 64, head, static_cast<int>(at));
          tma_load_3d(s2 + c * kTile * 128, &own2, &bar->own, c * 64, head, static_cast<int>(at));
        }
      }
      for (int i = 0; i < n && ok; ++i) {
        const int st = i % C::kPairs, use = i / C::kPairs;
        const int h = KEYS ? head * G + i / each : head / G, at = first + (KEYS ? i % each : i) * N;
        const int row = static_cast<int>((KEYS ? q0 : k0) + at);
        if (use > 0 && !(ok = wait(&bar->empty1[st], (use - 1) & 1))) break;
        mbar_arrive_expect_tx(&bar->full1[st], C::kTileBytes + (KEYS ? C::kImage : 0));
        for (int c = 0; c < D / 64; ++c)
          tma_load_3d(ring + 2 * st * C::kTileBytes + c * N * 128, &past1, &bar->full1[st], c * 64, h, row);
        if (KEYS)
          bulk_load(images + st * C::kImage,
                    g.images + (static_cast<int64_t>(h) * g.blocks + first_block(q0, b) + at / kSumRows) * kImageBytes +
                        at % kSumRows * 32,
                    C::kImage, &bar->full1[st]);
        ++loads;
        if (use > 0 && !(ok = wait(&bar->empty2[st], (use - 1) & 1))) break;
        mbar_arrive_expect_tx(&bar->full2[st], C::kTileBytes);
        for (int c = 0; c < D / 64; ++c)
          tma_load_3d(ring + (2 * st + 1) * C::kTileBytes + c * N * 128, &past2, &bar->full2[st], c * 64, h, row);
        ++seconds;
      }
      // every copy has landed before the CTA may end
      if (own) wait(&bar->own, 0);
      for (int i = max(0, loads - C::kPairs); i < loads; ++i) wait(&bar->full1[i % C::kPairs], (i / C::kPairs) & 1);
      for (int i = max(0, seconds - C::kPairs); i < seconds; ++i) wait(&bar->full2[i % C::kPairs], (i / C::kPairs) & 1);
    }
  } else if (warp == C::kMmaWarp) {
    // The whole warp walks the loop, so that descriptors stay uniform; one lane issues.
    constexpr uint32_t id_x = idesc_bf16(kTile, N), id_s = idesc_bf16(kTile, D, false, true);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t a1 = sdesc_k128(smem_u32(s1)), a2 = sdesc_k128(smem_u32(s2)), bk = sdesc_k128(smem_u32(ring));
    const uint64_t bm = D == 64 ? sdesc_mn128(smem_u32(ring)) : sdesc_mn128_wide(smem_u32(ring), N * 128);
    const uint64_t one = sdesc_plain16(smem_u32(ones)), img = sdesc_plain16(smem_u32(images));
    auto arrived = [&](uint64_t* m, uint32_t parity) {  // one answer for the warp
      return __all_sync(0xffffffffu, wait(m, parity)) != 0;
    };
    // X (second = 0) or Y of tile i, each with what its completion tells
    auto scores = [&](int i, int second, uint32_t to, uint64_t* then, uint64_t* then2) {
      const int st = i % C::kPairs;
      const uint64_t as = second ? a2 : a1, bs = bk + (2 * st + second) * (C::kTileBytes >> 4);
      if (elect_one()) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          umma_bf16(to, as + (((ks >> 2) * kTile * 128 + (ks & 3) * 32) >> 4), bs + (((ks >> 2) * N * 128 + (ks & 3) * 32) >> 4),
                    id_x, ks > 0);
        if (KEYS) umma_bf16(to, one + second * (kImageBytes >> 4), img + st * (C::kImage >> 4), id_x, 1);
        umma_commit(then);
        if (then2) umma_commit(then2);
      }
      __syncwarp();
    };
    // sum += W (bf16, in TMEM) times the first or second tile of pair i
    auto add = [&](uint32_t sum, uint32_t w, int i, int second, bool acc, uint64_t* then) {
      const uint64_t bs = bm + (2 * (i % C::kPairs) + second) * (C::kTileBytes >> 4);
      if (elect_one()) {
#pragma unroll
        for (int ks = 0; ks < N / 16; ++ks) umma_ts(sum, w + (ks >> 2) * 64 + (ks & 3) * 8, bs + ks * 128, id_s, acc || ks > 0);
        umma_commit(then);
      }
      __syncwarp();
    };
    bool ok = n > 0 && arrived(&bar->own, 0);
    auto full1 = [&](int i) { return arrived(&bar->full1[i % C::kPairs], (i / C::kPairs) & 1); };
    auto full2 = [&](int i) { return arrived(&bar->full2[i % C::kPairs], (i / C::kPairs) & 1); };
    if constexpr (KEYS) {
      // ... X(i) dK(i - 1) Y(i) dV(i) X(i + 1) ...: P(i) is formed under dK(i - 1) and Y(i), dS(i) under dV(i) and X(i + 1)
      if (ok && (ok = full1(0))) {
        tc_fence_after();
        scores(0, 0, tm + C::kColX, &bar->x[0], nullptr);
      }
      for (int i = 0; i < n && ok; ++i) {
        const int st = i % C::kPairs;
        if (!(ok = full2(i))) break;
        tc_fence_after();
        scores(i, 1, tm + C::kColY, &bar->y, nullptr);
        if (!(ok = arrived(&bar->p, i & 1))) break;
        tc_fence_after();
        add(tm + C::kColV, tm + C::kColX, i, 1, i > 0, &bar->empty2[st]);
        if (i + 1 < n) {
          if (!(ok = full1(i + 1))) break;
          tc_fence_after();
          scores(i + 1, 0, tm + C::kColX, &bar->x[0], nullptr);
        }
        if (!(ok = arrived(&bar->ds, i & 1))) break;
        tc_fence_after();
        add(tm + C::kColS, tm + C::kColY, i, 0, i > 0, &bar->empty1[st]);
      }
    } else {
      // ... Y(i + 1) dQ(i) X(i + 2) ...: Y(i + 1) as soon as Y(i) has been read, X a tile ahead
      for (int i = -1; i < n && ok; ++i) {
        if (i >= 0) {
          if (!(ok = arrived(&bar->ds, i & 1))) break;
          tc_fence_after();
        } else {
          if (!(ok = full1(0))) break;
          tc_fence_after();
          scores(0, 0, tm + C::kColX, &bar->x[0], nullptr);
        }
        if (i + 1 < n) {
          if (!(ok = full2(i + 1))) break;
          tc_fence_after();
          scores(i + 1, 1, tm + C::kColY, &bar->y, &bar->empty2[(i + 1) % C::kPairs]);
        }
        if (i >= 0) add(tm + C::kColS, tm + C::kColX + (i & 1) * N, i, 0, i > 0, &bar->empty1[i % C::kPairs]);
        if (i + 2 < n) {
          if (!(ok = full1(i + 2))) break;
          tc_fence_after();
          scores(i + 2, 0, tm + C::kColX + (i & 1) * N, &bar->x[i & 1], nullptr);
        }
      }
    }
    if (elect_one()) umma_commit(&bar->drain);  // products in flight end before the memory is freed
    __syncwarp();
    wait(&bar->drain, 0);
    __syncwarp();
  } else if (warp < C::kLoadWarp) {
    if (D == 64) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int half = C::kSplit == 2 ? warp >> 2 : 0, quad = warp & 3, r = quad * 32 + lane;
    const uint32_t mine = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const int row = row0 + r;
    const float sl2 = a.scale * kLog2e;
    const uint64_t scale2 = pack2(sl2, sl2);
    const float* sums = g.sums + row_sums(g.blocks, KEYS ? head * G : head, first_block(q0, b));
    uint64_t lse2 = 0, delta2 = 0;  // of this thread's query, negative
    if (!KEYS) {
      const float* at = sums + static_cast<int64_t>(row0 / kSumRows) * (2 * kSumRows) + r;
      lse2 = pack2(-at[0] * kLog2e, -at[0] * kLog2e);
      delta2 = pack2(-at[kSumRows], -at[kSumRows]);
    }
    auto arrive = [&](uint64_t* m) {  // once for the warp: arrivals of 32 lanes on one word take their turns
      __syncwarp();
      if (lane == 0) mbar_arrive(m);
    };
    auto waited = [&](uint64_t* m, uint32_t parity) { return __all_sync(0xffffffffu, wait(m, parity)) != 0; };
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      const int at = first + (KEYS ? i % each : i) * N + half * 64;  // of the first column
      const uint32_t tx = mine + C::kColX + (KEYS ? 0 : (i & 1) * N) + half * 64, ty = mine + C::kColY + half * 64;
      if (!(ok = waited(KEYS ? &bar->x[0] : &bar->x[i & 1], (KEYS ? i : i >> 1) & 1))) break;
      tc_fence_after();
      float p[64];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t v[32];
        tmem_ld32(tx + c * 32, v);
#pragma unroll
        for (int e = 0; e < 32; ++e) p[c * 32 + e] = __uint_as_float(v[e]);
      }
      tmem_wait_ld();
      if constexpr (KEYS) {
        if (at + off < row0 + kTile - 1) {  // queries of this half that some key is behind
          const int lim = row - off - at;
#pragma unroll
          for (int e = 0; e < 64; ++e)
            if (e < lim) p[e] = -INFINITY;
        }
      } else {
        if (at + 64 > min(row0 + off + 1, lk)) {
          const int lim = min(row + off + 1, lk) - at;
#pragma unroll
          for (int e = 0; e < 64; ++e)
            if (e >= lim) p[e] = -INFINITY;
        }
      }
      uint32_t u[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const uint64_t s = pack2(p[2 * e], p[2 * e + 1]);
        unpack2(KEYS ? mul2(s, scale2) : fma2(s, scale2, lse2), p[2 * e], p[2 * e + 1]);
        p[2 * e] = ex2(p[2 * e]), p[2 * e + 1] = ex2(p[2 * e + 1]);
        if (KEYS) u[e] = pack_bf16(p[2 * e], p[2 * e + 1]);
      }
      if (KEYS) {
        tmem_st32(tx, u);
        tmem_wait_st();
        tc_fence_before();
        arrive(&bar->p);
      }
      if (!(ok = waited(&bar->y, i & 1))) break;
      tc_fence_after();
      uint32_t y[2][32];
      tmem_ld32(ty, y[0]);
      tmem_ld32(ty + 32, y[1]);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        uint64_t z = pack2(__uint_as_float(y[e >> 4][(2 * e) & 31]), __uint_as_float(y[e >> 4][(2 * e + 1) & 31]));
        if (!KEYS) z = add2(z, delta2);
        float z0, z1;
        unpack2(mul2(pack2(p[2 * e], p[2 * e + 1]), z), z0, z1);
        u[e] = pack_bf16(z0, z1);
      }
      tmem_st32(KEYS ? ty : tx, u);
      tmem_wait_st();
      tc_fence_before();
      arrive(&bar->ds);
    }
    // the last product is the one that frees the last pair's first tile
    if (ok && n > 0) ok = waited(&bar->empty1[(n - 1) % C::kPairs], ((n - 1) / C::kPairs) & 1);
    ok = __all_sync(0xffffffffu, ok);
    if (ok) {
      tc_fence_after();
      const int d = D == 64 ? a.d : D;  // of the rows
#pragma unroll
      for (int out = KEYS ? 0 : 1; out < 2; ++out) {  // dV, then dK; or dQ
        const RowsOut& to = KEYS ? (out ? g.dk : g.dv) : g.dq;
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(to.p) + ((KEYS ? k0 : q0) + row0) * to.stride +
                             static_cast<int64_t>(head) * d;
        const float f = out ? a.scale : 1.f;
        const uint64_t f2 = pack2(f, f);
        const uint32_t from = mine + (out ? C::kColS : C::kColV) + half * 64;
        uint64_t rest = 0;  // z * 0 added up: NaN where some z is not finite
        // a warp's 32 rows x 64 dims through shared memory (the owned tiles' place: every product is done), so that a
        // store covers whole lines
        uint8_t* stage = (out ? s2 : s1) + half * kTile * 128;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t v[32];
          if (n > 0) {
            tmem_ld32(from + c * 32, v);
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
            *reinterpret_cast<uint4*>(stage + sw128(r, c * 32 + e * 8)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int rr = quad * 32 + e * 4 + (lane >> 3), c = (lane & 7) * 8;
          if (row0 + rr >= rows || (D == 64 && c >= d)) continue;
          *reinterpret_cast<uint4*>(dst + rr * to.stride + half * 64 + c) = *reinterpret_cast<const uint4*>(stage + sw128(rr, c));
        }
        float ra, rb;
        unpack2(rest, ra, rb);
        __syncwarp();
        for (uint32_t again = __ballot_sync(0xffffffffu, row < rows && !(ra + rb == 0.f)); again; again &= again - 1) {
          const int i = row0 + quad * 32 + __ffs(again) - 1;
          const __nv_bfloat16 *q = static_cast<const __nv_bfloat16*>(a.q.p), *d_o = static_cast<const __nv_bfloat16*>(g.d_o.p);
          const __nv_bfloat16 *k = static_cast<const __nv_bfloat16*>(a.k.p), *v = static_cast<const __nv_bfloat16*>(a.v.p);
          float x1[4], x2[4];
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
          // this warp's part of the row
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int c = half * 64 + e * 32 + lane, j = C::kSplit == 2 ? 2 * half + e : e;
            float z = 0.f;
#pragma unroll
            for (int m = 0; m < 4; ++m)
              if (m == j) z = KEYS && out == 0 ? x2[m] : x1[m];
            if (c < d) dst[(i - row0) * to.stride + c] = __float2bfloat16_rn(z);
          }
        }
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

template <int D, bool KEYS>
int launch_kernel(TcGradArgs& t, int64_t grid, const CUtensorMap (&m)[4], cudaStream_t s) {
  if (grid < 1 || grid > INT32_MAX) return FALCON_ERR_UNSUPPORTED;
  t.stall = take_test_stall() ? 1 : 0;
  const auto kern = attn_grad_tc_kernel<D, KEYS>;
  if (!set_smem_limit(reinterpret_cast<const void*>(kern), smem_bytes<D, KEYS>())) return FALCON_ERR_CUDA;
  kern<<<static_cast<unsigned>(grid), Cfg<D, KEYS>::kThreads, smem_bytes<D, KEYS>(), s>>>(m[0], m[1], m[2], m[3], t);
  return cudaGetLastError() == cudaSuccess ? FALCON_OK : FALCON_ERR_CUDA;
}

template <int D>
int launch_d(const GradArgs& g, cudaStream_t s) {
  const PromptArgs& a = g.a;
  TcGradArgs t;
  t.g = g;
  t.qblocks = 0, t.packed = false;
  t.status = static_cast<uint32_t*>(a.ws);
  t.limit = wait_limit_ns();
  CUtensorMap m[4];
  auto maps = [&](const RowsIn& x, int64_t n, int H, int rows, CUtensorMap* to) { return make_rows_map(to, x, n, H, a.d, rows); };
  if (g.dq.p) {
    const PromptGrid pg = prompt_grid(a, kTile);
    t.qblocks = static_cast<int>(pg.blocks / a.B);
    t.packed = pg.packed;
    constexpr int N = Cfg<D, false>::kN;
    if (!maps(a.q, a.tokens, a.Hq, kTile, m) || !maps(g.d_o, a.tokens, a.Hq, kTile, m + 1) ||
        !maps(a.k, a.k_tokens, a.Hkv, N, m + 2) || !maps(a.v, a.k_tokens, a.Hkv, N, m + 3))
      return FALCON_ERR_CUDA;
    const int st = pg.blocks > INT32_MAX / a.Hq ? FALCON_ERR_UNSUPPORTED : launch_kernel<D, false>(t, pg.blocks * a.Hq, m, s);
    if (st != FALCON_OK) return st;
  }
  if (g.dk.p) {
    const int64_t blocks = a.k_tokens / kTile + a.B;
    constexpr int N = Cfg<D, true>::kN;
    if (!maps(a.k, a.k_tokens, a.Hkv, kTile, m) || !maps(a.v, a.k_tokens, a.Hkv, kTile, m + 1) ||
        !maps(a.q, a.tokens, a.Hq, N, m + 2) || !maps(g.d_o, a.tokens, a.Hq, N, m + 3))
      return FALCON_ERR_CUDA;
    return blocks > INT32_MAX / a.Hkv ? FALCON_ERR_UNSUPPORTED : launch_kernel<D, true>(t, blocks * a.Hkv, m, s);
  }
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
