// dK and dV of causal attention over packed prompts on the tensor cores (bf16).
//
//   X = K Q^T,  Y = V dO^T,  P = exp(scale X - log sum),  dS = P (Y - D)
//   dV = P dO,  dK = scale dS Q    (P and dS with the keys as rows)
//
// dQ has a kernel of its own, so that every sum has one owner and one order (7
// products of a tile where one kernel with dQ added up in memory would have 5; that
// adds 64 KB in fp32 for every tile of 128 x 128, and in another order each
// time).  A CTA owns 128 rows of K and V; the queries of all heads of the group come
// past, 128 at a time (64 at d = 64, with two CTAs on an SM):
//   load warp    TMA: Q and dO of a tile, through a ring of pairs
//   clear warp   zeros in the rows of a tile that lie past the sequence
//   MMA warp     X, Y and the sums' products in the order that keeps the tensor
//                cores ahead of the softmax warps, see the loop
//   softmax      64 columns of a row a thread (32: 290 us for 281 for 12 ragged documents of
//   warps        16 heads of 128): P from X, dS from P and Y.  They go back to TMEM in
//                bf16 over the scores that they came from, as the A operand of the
//                sums' products.
// A thread holds one key and 64 queries, so that log sums and D would be loads for
// every element; they come out of the products instead, one more step of 16
// columns: [K | 1] [Q | -log sum / scale]^T and [V | 1] [dO | -D]^T, in three bf16
// parts (24 bits).
// d = 128: 2440 cycles a tile (16384 tokens, a launch's cycles over the tiles of an SM), 2176 of them products; shared
// memory, which gives X and Y both operands (the four accumulators fill TMEM), is busy as long as these.
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

template <int D>
struct Cfg {
  static constexpr int kCtas = D == 64 ? 2 : 1;  // CTAs of an SM
  static constexpr int kN = D == 64 ? 64 : 128;  // queries of a tile
  static constexpr int kSplit = kN / 64;         // softmax threads of an owned row
  static constexpr int kOut = 2 * D / kSplit;    // columns of the sums that each of them writes
  static constexpr int kWarps = 4 * kSplit;
  static constexpr int kLoadWarp = kWarps, kMmaWarp = kWarps + 1;
  static constexpr int kThreads = 32 * kWarps + 128;
  static constexpr int kOwnBytes = kTile * D * 2, kTileBytes = kN * D * 2;
  static constexpr int kPairs = D == 64 ? 3 : 2;
  static constexpr int kRing = 2 * kPairs * kTileBytes;
  static constexpr int kImage = kN * 32;         // log sums and D of a tile
  static constexpr int kExtra = 2 * kOwnBytes + kPairs * kImage + 2 * kImageBytes;
  // TMEM: X, Y, the sums
  static constexpr uint32_t kColX = 0, kColY = kN, kColV = 2 * kN, kColS = 2 * kN + D;
  static constexpr uint32_t kCols = D == 64 ? 256 : 512;
};
struct Bars {
  uint64_t own, full[6], empty[6], raw[6], x, y, p, ds, drain, stall;
  uint32_t tmem, failed;
  uint32_t bad[2][4];  // rows that are not finite, a bit each
};
constexpr int kRaw = 12;  // from full to raw
static_assert(offsetof(Bars, raw) == offsetof(Bars, full) + kRaw * sizeof(uint64_t), "places");
template <int D>
constexpr int smem_bytes() {
  return Cfg<D>::kRing + Cfg<D>::kExtra + 1024 + static_cast<int>(sizeof(Bars));
}
static_assert(smem_bytes<128>() <= 227 * 1024 && smem_bytes<64>() <= 113 * 1024, "shared memory");

struct TcGradArgs {
  GradArgs g;
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
// Tile i's places in the ring.  The first tile (Q) is read until the tile's last product, the second (dO) until its last
// but two; they change places from use to use, so that each copy has a whole tile's products of time.
template <int P>
__device__ __forceinline__ int place_of(int i, int second) {
  return 2 * (i % P) + ((i / P + second) & 1);
}
// A head's last tile may reach past the sequence, into the next one's rows or what lies behind the last one.  Their weights
// are 0, but 0 times one that is not finite would have every key of the sequence computed again (8 x 2000 tokens of 12
// heads of 64, NaN behind the last: 41.8 ms for 0.2; 4000 of 16 over 4 heads of 128: 102 ms).  So these rows become zeros
// before the tile counts as copied: by one warp, tiles i, i + each, ... below n, of which `live` rows stay.  (Stores one
// after another with the wait by one lane: 12 ragged documents of 16 over 4 heads of 128 269 us, so 262.)
template <int D>
__device__ __noinline__ void clear_rows(Bars* bar, uint8_t* ring, int i, int n, int each, int live, uint32_t* status,
                                        uint64_t limit) {
  using C = Cfg<D>;
  constexpr int N = C::kN;
  const int lane = threadIdx.x & 31;
  uint32_t parity = 0;  // a bit each place
  for (; i < n; i += each)
    for (int second = 0; second < 2; ++second) {
      const int slot = place_of<C::kPairs>(i, second);
      if (!__all_sync(0xffffffffu, mbar_wait_sleep(&bar->raw[slot], (parity >> slot) & 1, limit))) {
        if (lane == 0) {
          atomicExch(status, kStatusTimeout);
          *static_cast<volatile uint32_t*>(&bar->failed) = 1;
        }
        return;
      }
      parity ^= 1u << slot;
      zero_rows<N, D / 64>(ring + slot * C::kTileBytes, live);
      if (lane == 0) mbar_arrive(&bar->full[slot]);
    }
}

template <int D>
__global__ void __launch_bounds__(Cfg<D>::kThreads, Cfg<D>::kCtas)
    attn_grad_tc_kernel(const __grid_constant__ CUtensorMap own1, const __grid_constant__ CUtensorMap own2,
                        const __grid_constant__ CUtensorMap past1, const __grid_constant__ CUtensorMap past2,
                        const TcGradArgs t) {
  using C = Cfg<D>;
  constexpr int N = C::kN, P = C::kPairs;
  const GradArgs& g = t.g;
  const PromptArgs& a = g.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint8_t *ring = smem, *s1 = smem + C::kRing, *s2 = s1 + C::kOwnBytes;  // ring: pairs of a first and a second tile
  uint8_t* images = s2 + C::kOwnBytes;
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
    for (int i = 0; i < 2 * P; ++i) {
      mbar_init(&bar->full[i], 1);
      mbar_init(&bar->empty[i], 1);
      mbar_init(&bar->raw[i], 1);
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
  {  // ones against the log sums (columns 0 to 2), ones against D (4 to 6)
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
  const uint32_t block = blockIdx.x / t.split;
  const int rank = static_cast<int>(blockIdx.x % t.split), head = static_cast<int>(block % a.Hkv);
  const int2 found = find_block(a.cu_k, a.B, kTile, static_cast<int>(block / a.Hkv));
  const int b = found.x;
  const int64_t q0 = a.cu_q[b], k0 = a.cu_k[b];
  const int lq_all = static_cast<int>(a.cu_q[b + 1] - q0), lk = static_cast<int>(a.cu_k[b + 1] - k0);
  const int lq = min(lq_all, a.max_q), off = lk - lq_all;
  const bool valid = found.y >= 0 && found.y < lk && q0 >= 0 && k0 >= 0 && q0 + lq_all <= a.tokens && k0 + lk <= a.k_tokens;
  // a sequence's blocks are dealt out from its last; the first keys, which the most queries see, come first
  const int row0 = (lk - 1) / kTile * kTile - found.y;
  // the tiles that come past, [first, first + each N) of every head, and this CTA's of them
  const int first = max(row0 - off, 0) / N * N, each = lq > first ? (lq - first + N - 1) / N : 0;
  const int64_t all = static_cast<int64_t>(each) * G;
  const int i0 = static_cast<int>(all * rank / t.split), n = static_cast<int>(all * (rank + 1) / t.split) - i0;
  const int live = lq - first - (each - 1) * N;  // rows of a head's last tile
  __syncthreads();
  const uint32_t tmem = bar->tmem;
  wait_for_previous();  // what the sums' kernel wrote is there
  launch_dependents();
  if (!valid) {  // (the whole cluster)
    if (warp == C::kMmaWarp) tmem_dealloc(tmem, C::kCols);
    return;
  }
  auto wait = [&](uint64_t* m, uint32_t parity) {
    if (mbar_wait_sleep(m, parity, t.limit)) return true;
    atomicExch(t.status, kStatusTimeout);
    *static_cast<volatile uint32_t*>(&bar->failed) = 1;
    return false;
  };
  auto place = [&](int i, int second) { return place_of<P>(i, second); };

  // registers: the softmax threads take what the last warpgroup gives up
  // (128 x 200 + 128 x 56 = 256 x 128; 256 x 208 + 128 x 88 = 384 x 168)
  if (warp >= C::kLoadWarp) {
    if (D == 64) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  }
  if (warp == C::kLoadWarp) {
    if (lane == 0 && n > 0) {
      bool ok = !t.stall || wait(&bar->stall, 0);
      int loads = 0;  // tiles begun: the first and the second of pair 0, of pair 1 ...
      bool own = false;
      if (ok) {
        own = true;
        const int at = static_cast<int>(k0 + row0);
        mbar_arrive_expect_tx(&bar->own, 2 * C::kOwnBytes);
        for (int c = 0; c < D / 64; ++c) {
          tma_load_3d(s1 + c * kTile * 128, &own1, &bar->own, c * 64, head, at);
          tma_load_3d(s2 + c * kTile * 128, &own2, &bar->own, c * 64, head, at);
        }
      }
      for (; loads < 2 * n && ok; ++loads) {
        const int i = loads >> 1, second = loads & 1, st = i % P, use = i / P, slot = place(i, second);
        // (what the copy needs comes before the wait for its place)
        const int h = head * G + (i0 + i) / each, at = first + (i0 + i) % each * N;
        const int row = static_cast<int>(q0 + at);
        const bool image = !second;  // its place was last read by the product before the one that freed this
        uint64_t* full = bar->full + slot + (at + N > lq ? kRaw : 0);
        const uint8_t* from = g.images + (static_cast<int64_t>(h) * g.blocks + first_block(q0, b) + at / kSumRows) * kImageBytes +
                              at % kSumRows * 32;
        if (use > 0 && !(ok = wait(&bar->empty[slot], (use - 1) & 1))) break;
        mbar_arrive_expect_tx(full, C::kTileBytes + (image ? C::kImage : 0));
        for (int c = 0; c < D / 64; ++c)
          tma_load_3d(ring + slot * C::kTileBytes + c * N * 128, second ? &past2 : &past1, full, c * 64, h, row);
        if (image)
          bulk_load(images + st * C::kImage, from, C::kImage, full);
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
      // X (second = 0) or Y of tile i
      auto scores = [&](int i, int second) {
        const uint64_t bs = bk + place(i, second) * (C::kTileBytes >> 4);
        const uint32_t to = tm + (second ? C::kColY : C::kColX);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          umma_bf16(to, (second ? a2 : a1) + (((ks >> 2) * kTile * 128 + (ks & 3) * 32) >> 4),
                    bs + (((ks >> 2) * N * 128 + (ks & 3) * 32) >> 4), id_x, ks > 0);
        umma_bf16(to, one + second * (kImageBytes >> 4), img + i % P * (C::kImage >> 4), id_x, 1);
        umma_commit(second ? &bar->y : &bar->x);
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
      bool ok = n > 0 && arrived(&bar->own, 0) && arrived(&bar->full[place(0, 0)], 0);
      if (ok) {
        scores(0, 0);
        if ((ok = arrived(&bar->full[place(0, 1)], 0))) scores(0, 1);
      }
      // ... X(i) dK(i - 1) Y(i) dV(i) X(i + 1) ...: P(i) is formed under dK(i - 1) and Y(i), dS(i) under dV(i) and X(i + 1).
      // What these wait for holds the next tile's copies too.
      for (int i = 0; i < n && ok; ++i) {
        if (!(ok = arrived(&bar->p, i & 1))) break;
        add(C::kColV, C::kColX, i, 1);
        if (i + 1 < n) scores(i + 1, 0);
        if (!(ok = arrived(&bar->ds, i & 1))) break;
        add(C::kColS, C::kColY, i, 0);
        if (i + 1 < n) scores(i + 1, 1);
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
  } else if (warp == C::kMmaWarp + 2) {
    if (n > 0 && live < N) clear_rows<D>(bar, ring, each - 1 - i0 % each, n, each, live, t.status, t.limit);
    __syncwarp();
  } else if (warp < C::kLoadWarp) {
    if (D == 64) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int part = warp >> 2, quad = warp & 3, r = quad * 32 + lane;
    const uint32_t mine = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const int row = row0 + r;
    const float sl2 = a.scale * kLog2e;
    const uint64_t scale2 = pack2(sl2, sl2);
    const float* sums = g.sums + row_sums(g.blocks, head * G, first_block(q0, b));
    auto arrive = [&](uint64_t* m) {  // once for the warp: arrivals of 32 lanes on one word take their turns
      __syncwarp();
      if (lane == 0) mbar_arrive(m);
    };
    auto waited = [&](uint64_t* m, uint32_t parity) { return __all_sync(0xffffffffu, wait(m, parity)) != 0; };
    bool ok = true;
    int past = n > 0 ? i0 % each : 0;  // the tile's place among a head's
    for (int i = 0; i < n && ok; ++i) {
      const int at = first + past * N + part * 64;  // of the first column
      if (++past == each) past = 0;
      const uint32_t tx = mine + C::kColX + part * 64, ty = mine + C::kColY + part * 64;
      if (!(ok = waited(&bar->x, i & 1))) break;
      tc_fence_after();
      uint64_t x[2][16];  // X, then P
      {
        uint32_t v[2][32];
#pragma unroll
        for (int c = 0; c < 2; ++c) tmem_ld32(tx + 32 * c, v[c]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int e = 0; e < 16; ++e) x[c][e] = pack2(__uint_as_float(v[c][2 * e]), __uint_as_float(v[c][2 * e + 1]));
      }
      if (at + off < row0 + kTile - 1) {  // some key is behind a query of these
        const int lim = row - off - at;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float z0, z1;
            unpack2(x[c][e], z0, z1);
            if (32 * c + 2 * e < lim) z0 = -INFINITY;
            if (32 * c + 2 * e + 1 < lim) z1 = -INFINITY;
            x[c][e] = pack2(z0, z1);
          }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t u[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float z0, z1;
          unpack2(mul2(x[c][e], scale2), z0, z1);
          z0 = ex2(z0), z1 = ex2(z1);
          x[c][e] = pack2(z0, z1);
          u[e] = pack_bf16(z0, z1);
        }
        tmem_st16(tx + 32 * c, u);
      }
      tmem_wait_st();
      tc_fence_before();
      arrive(&bar->p);
      if (!(ok = waited(&bar->y, i & 1))) break;
      tc_fence_after();
      {
        uint32_t v[2][32];
#pragma unroll
        for (int c = 0; c < 2; ++c) tmem_ld32(ty + 32 * c, v[c]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t u[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const uint64_t z = pack2(__uint_as_float(v[c][2 * e]), __uint_as_float(v[c][2 * e + 1]));
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
    // a row of dK (x1) and of dV (x2) from the definition
    auto compute_again = [&](int i, float (&x1)[4], float (&x2)[4]) {
      const __nv_bfloat16 *q = static_cast<const __nv_bfloat16*>(a.q.p), *d_o = static_cast<const __nv_bfloat16*>(g.d_o.p);
      const __nv_bfloat16 *k = static_cast<const __nv_bfloat16*>(a.k.p), *v = static_cast<const __nv_bfloat16*>(a.v.p);
      const int64_t h0 = static_cast<int64_t>(head) * G * d, hk = static_cast<int64_t>(head) * d;
      grad_key_row<__nv_bfloat16, D>(k + (k0 + i) * a.k.stride + hk, v + (k0 + i) * a.v.stride + hk, q + q0 * a.q.stride + h0,
                                     a.q.stride, d_o + q0 * g.d_o.stride + h0, g.d_o.stride, sums, g.blocks, G,
                                     max(i - off, 0), lq, d, a.scale, x1, x2);
    };
    if (t.split == 1) {
      if (__all_sync(0xffffffffu, ok)) {
        // this thread's columns of a row, of dV and then of dK, 64 at a time
#pragma unroll 1
        for (int start = part * C::kOut; start < (part + 1) * C::kOut; start += 64) {
          const bool of_v = start < D;
          const int c0 = start % D;
          const RowsOut& to = of_v ? g.dv : g.dk;
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(to.p) + (k0 + row0) * to.stride +
                               static_cast<int64_t>(head) * d + c0;
          const float f = of_v ? 1.f : a.scale;
          const uint64_t f2 = pack2(f, f);
          const uint32_t from = mine + (of_v ? C::kColV : C::kColS) + c0;
          uint64_t rest = 0;  // z * 0 added up: NaN where some z is not finite
          // a warp's 32 rows through shared memory (the ring's place: every product is done), so that a store covers
          // whole lines
          uint8_t* stage = ring + (start >> 6) * kTile * 128;
#pragma unroll
          for (int c = 0; c < 64; c += 32) {
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
              *reinterpret_cast<uint4*>(stage + sw128(r, c + e * 8)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          __syncwarp();
          constexpr int kPieces = 8;  // 16 bytes each
#pragma unroll
          for (int e = 0; e < kPieces; ++e) {
            const int x = e * 32 + lane, rr = quad * 32 + x / kPieces, c = x % kPieces * 8;
            if (row0 + rr >= lk || (D == 64 && c0 + c >= d)) continue;
            *reinterpret_cast<uint4*>(dst + rr * to.stride + c) = *reinterpret_cast<const uint4*>(stage + sw128(rr, c));
          }
          float ra, rb;
          unpack2(rest, ra, rb);
          __syncwarp();
          for (uint32_t again = __ballot_sync(0xffffffffu, row < lk && !(ra + rb == 0.f)); again; again &= again - 1) {
            const int i = row0 + quad * 32 + __ffs(again) - 1;
            float x1[4], x2[4];
            compute_again(i, x1, x2);
            // this warp's part of the row
#pragma unroll
            for (int m = 0; m < D / 32; ++m) {
              const int c = m * 32 + lane;
              if (m * 32 >= c0 && m * 32 < c0 + 64 && c < d)
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
      cluster_sums<__nv_bfloat16, D, 32 * C::kWarps>(g, smem, &bar->failed, bar->bad, t.split, rank, row0, lk, k0, head, d, compute_again);
    }
    tc_fence_before();
  }
  if (t.split > 1 && warp >= C::kLoadWarp) {
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

template <int D>
int launch_kernel(TcGradArgs& t, int64_t grid, const CUtensorMap (&m)[4], cudaStream_t s) {
  if (grid < 1 || grid > INT32_MAX / t.split) return FALCON_ERR_UNSUPPORTED;
  t.stall = take_test_stall() ? 1 : 0;
  const auto kern = attn_grad_tc_kernel<D>;
  if (!set_smem_limit(reinterpret_cast<const void*>(kern), smem_bytes<D>())) return FALCON_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid * t.split));
  cfg.blockDim = dim3(Cfg<D>::kThreads);
  cfg.dynamicSmemBytes = smem_bytes<D>();
  cfg.stream = s;
  cudaLaunchAttribute attr[2] = {overlap_attribute(), cluster_attribute(t.split)};
  cfg.attrs = attr;
  cfg.numAttrs = t.split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, m[0], m[1], m[2], m[3], t) == cudaSuccess ? FALCON_OK : FALCON_ERR_CUDA;
}

template <int D>
int launch_d(const GradArgs& g, cudaStream_t s) {
  const PromptArgs& a = g.a;
  constexpr int N = Cfg<D>::kN;
  const int64_t blocks = a.k_tokens / kTile + a.B;
  if (blocks > INT32_MAX / a.Hkv) return FALCON_ERR_UNSUPPORTED;
  TcGradArgs t;
  t.g = g;
  t.split = keys_split(a, N, sm_count() * Cfg<D>::kCtas, D == 64 ? 4 : 2, D == 64 ? 14 : 9);
  t.status = static_cast<uint32_t*>(a.ws);
  t.limit = wait_limit_ns();
  CUtensorMap m[4];
  if (!make_rows_map(m, a.k, a.k_tokens, a.Hkv, a.d) || !make_rows_map(m + 1, a.v, a.k_tokens, a.Hkv, a.d) ||
      !make_rows_map(m + 2, a.q, a.tokens, a.Hq, a.d, N) || !make_rows_map(m + 3, g.d_o, a.tokens, a.Hq, a.d, N))
    return FALCON_ERR_CUDA;
  return launch_kernel<D>(t, blocks * a.Hkv, m, s);
}

}  // namespace

// The tensor-core kernels take bf16 rows on 16-byte boundaries (their TMA copies and stores), with token strides below
// the maps' 2^40 bytes, and scales from 2^-100 on: the scale comes after the log sums, and a row without weight has -3.4e38
// there at least, which 2^-100 leaves at -2.7e8 (weight 0), while 2^-126 would make a weight of 0.02 of it.
bool attn_grad_tc_supported(const GradArgs& g, int dtype) {
  const PromptArgs& a = g.a;
  if (dtype != FALCON_BF16 || a.k_tokens == 0 || a.tokens == 0 || a.max_q == 0) return false;
  if (!(a.scale >= 0x1p-100f)) return false;
  if (!a.q.vec || !a.k.vec || !a.v.vec || !g.d_o.vec) return false;
  for (const RowsOut& x : {g.dq, g.dk, g.dv})
    if (x.p && !x.vec) return false;
  for (int64_t st : {a.q.stride, a.k.stride, a.v.stride, g.d_o.stride})
    if (st * 2 >= (int64_t(1) << 40)) return false;
  return true;
}

int launch_attn_grad_tc(const GradArgs& g, cudaStream_t s) {
  if (g.dk.p) {  // first: its CTAs run longest
    const int st = g.a.d <= 64 ? launch_d<64>(g, s) : launch_d<128>(g, s);
    if (st != FALCON_OK) return st;
  }
  return g.dq.p ? launch_attn_grad_dq_tc(g, g.dk.p != nullptr, s) : FALCON_OK;
}

}  // namespace falcon
