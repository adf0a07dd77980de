// Gradient of causal attention over packed prompts on the tensor cores (fp32).
//
//   P = exp(scale Q K^T - log sum),  dS = P (dO V^T - D)
//   dV = P^T dO,  dK = scale dS^T Q,  dQ = scale dS K
//
// An operand is held as two halves, x = s (hi + lo), each rounded to 11 bits, with a power of two s for
// every row that brings the row's largest element to [2^14, 2^15): 22 bits, down to 2^-40
// of the row's largest.  A product is hi hi + hi lo + lo hi, the small ones first; its sums stay
// in the tensor cores, which cut them off, for one tile only (64 rows) and are added up in
// fp32 registers.
//
// The first kernel splits q, k, v and dO into the workspace, 64 rows of a head at a time, laid out as
// the operand tiles in shared memory, and forms D.  Two kernels from one template do the products, so
// that every sum has one owner and one order.  A CTA owns 128 rows: of K and V (dK and dV; X = K Q^T,
// Y = V dO^T, the queries of all heads of the group come past, 64 at a time) or of Q and dO (dQ;
// X = Q K^T, Y = dO V^T, the keys come past).  Two lanes of a warp hold a row of a tile, 32
// columns each.  P and dS are split like the operands, a power of two for every row of a
// tile, after the factors of the rows that the sum runs over have been multiplied in: no range
// of P or dS is out of reach.
//   dK and dV: ... X(i) dK(i - 1) Y(i) dV(i) X(i + 1) ...
//   dQ:        ... X(i + 1) Y(i + 1) dQ(i) X(i + 2) ...
// (X's owned operand lies in shared memory, Y's in TMEM, which gives the ring its room.)
//
// Masked scores are set to -inf after the product.  A masked weight is 0, but 0
// times an infinite or NaN value of a row that the owner does not see would spoil
// it: a row of a result that is not finite is computed again from the definition.

#include <cuda_fp16.h>

#include "attn_grad.cuh"
#include "attn_tc.cuh"

namespace falcon {
namespace {

using namespace tcu;

constexpr int kPast = 64;  // rows of a tile that comes past, and of a block of the workspace

// 2^k and 2^-k that bring the largest finite magnitude to [2^14, 2^15) and back
__device__ __forceinline__ void row_factors(float amax, float& up, float& down) {
  const int e = min(max(static_cast<int>(__float_as_uint(amax) >> 23), 16), 254);
  up = __uint_as_float(static_cast<uint32_t>(268 - e) << 23);
  down = __uint_as_float(static_cast<uint32_t>(e - 14) << 23);
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// a pair of scaled values: 11 bits to nearest, and the rest
__device__ __forceinline__ void split2(uint64_t x, uint32_t& hi, uint32_t& lo) {
  float a, b;
  unpack2(x, a, b);
  const float ha = __uint_as_float((__float_as_uint(a) + 0x1000u) & 0xFFFFE000u);
  const float hb = __uint_as_float((__float_as_uint(b) + 0x1000u) & 0xFFFFE000u);
  hi = pack_half(ha, hb);
  lo = pack_half(a - ha, b - hb);
}

// ---------------------------------------------------------------- operands
// 64 rows of one head's x (row `first` on, `rows` of them live) into an image: slabs of 64 columns, hi's and then lo's,
// and the rows' factors.  dot: (sum of x o of each row) of the rows, by the row's first lane.
template <int D, bool DOT, typename F>
__device__ __forceinline__ void split_rows(const RowsIn& x, const RowsIn& o, int64_t row, int head, int rows, int d,
                                           uint8_t* image, __nv_bfloat16* factor, F dot) {
  constexpr int L = D / 8, kStep = 256 / L;
  const int c = threadIdx.x % L;
  for (int r = threadIdx.x / L; r < kPast; r += kStep) {
    float v[8], w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = w[e] = 0.f;
    if (r < rows && c * 8 < d) {
      const float* p = static_cast<const float*>(x.p) + (row + r) * x.stride + static_cast<int64_t>(head) * d;
      const Pieces at{c * 8, c * 8 + 4};
      unpack8(x.vec ? load8<true, false>(p, at) : load8<false, false>(p, at), v);
      if (DOT) {
        p = static_cast<const float*>(o.p) + (row + r) * o.stride + static_cast<int64_t>(head) * d;
        unpack8(o.vec ? load8<true, false>(p, at) : load8<false, false>(p, at), w);
      }
    }
    float m = 0.f, s = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float a = fabsf(v[e]);
      m = fmaxf(m, a <= 3.402823466e38f ? a : 0.f);
      if (DOT) s = fmaf(v[e], w[e], s);
    }
#pragma unroll
    for (int i = 1; i < L; i <<= 1) {
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, i));
      if (DOT) s += __shfl_xor_sync(0xffffffffu, s, i);
    }
    float up, down;
    row_factors(m, up, down);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) split2(mul2(pack2(v[2 * e], v[2 * e + 1]), pack2(up, up)), hi[e], lo[e]);
    uint8_t* to = image + (c >> 3) * (kPast * 128) + tc::sw128(r, (c & 7) * 8);
    *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(to + kPast * D * 2) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    if (c == 0) {
      factor[r] = __float2bfloat16_rn(down);  // exact
      if (DOT) dot(r, s);
    }
  }
}

// Where the operands lie: 64-row blocks, a sequence's from cu[b] / 64 + b on.
struct Operands {
  uint8_t *q, *d_o, *k, *v;    // images of kPast * D * 4 bytes, a head's blocks behind one another
  // What the softmax threads need of a block's rows.  Queries: -log sum, -D (fp32), the factors of q and of dO; keys: the
  // factors of k and of v (bf16: powers of two).
  uint8_t *q_info, *k_info;
  int64_t q_blocks, k_blocks;     // of a head
};
constexpr int kQInfo = kPast * 12, kKInfo = kPast * 4;
__device__ __forceinline__ float factor_at(const uint8_t* factors, int i) {
  return __bfloat162float(__ldcg(reinterpret_cast<const __nv_bfloat16*>(factors) + i));
}
__host__ __device__ __forceinline__ int64_t count_blocks(int64_t rows, int B) { return rows / kPast + B + 1; }
__device__ __forceinline__ int64_t first64(int64_t q0, int b) { return q0 / kPast + b; }

template <int D>
__global__ void __launch_bounds__(256) attn_grad_split_kernel(GradArgs g, Operands w, unsigned q_ctas) {
  const PromptArgs& a = g.a;
  launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) *static_cast<uint32_t*>(a.ws) = 0;  // the call's status
  const bool of_q = blockIdx.x < q_ctas;
  const int H = of_q ? a.Hq : a.Hkv;
  const unsigned at = of_q ? blockIdx.x : blockIdx.x - q_ctas;
  const int h = static_cast<int>(at % H);
  const int32_t* cu = of_q ? a.cu_q : a.cu_k;
  const int2 x = find_block(cu, a.B, kPast, static_cast<int>(at / H));
  const int64_t r0 = cu[x.x], r1 = cu[x.x + 1];
  if (x.y < 0 || r0 < 0 || r1 > (of_q ? a.tokens : a.k_tokens) || x.y >= r1 - r0) return;
  const int rows = static_cast<int>((of_q ? min(r1 - r0, static_cast<int64_t>(a.max_q)) : r1 - r0) - x.y);
  const int64_t n = x.y / kPast, j = first64(r0, x.x) + n, row = r0 + x.y;
  const auto none = [](int, float) {};
  if (!of_q) {
    const int64_t to = h * w.k_blocks + j;
    __nv_bfloat16* factors = reinterpret_cast<__nv_bfloat16*>(w.k_info + to * kKInfo);
    split_rows<D, false>(a.k, a.k, row, h, rows, a.d, w.k + to * (kPast * D * 4), factors, none);
    split_rows<D, false>(a.v, a.v, row, h, rows, a.d, w.v + to * (kPast * D * 4), factors + kPast, none);
    return;
  }
  const int64_t to = h * w.q_blocks + j;
  float* info = reinterpret_cast<float*>(w.q_info + to * kQInfo);
  __nv_bfloat16* factors = reinterpret_cast<__nv_bfloat16*>(info + 2 * kPast);
  split_rows<D, false>(a.q, a.q, row, h, rows, a.d, w.q + to * (kPast * D * 4), factors, none);
  // the log sums and D, for the tiles and for rows that are computed again; rows without a key have no weights
  float* sums = g.sums + row_sums(g.blocks, h, first_block(r0, x.x) + n / 2) + n % 2 * kPast;
  split_rows<D, true>(g.d_o, g.o, row, h, rows, a.d, w.d_o + to * (kPast * D * 4), factors + kPast, [&](int r, float s) {
    float lse = INFINITY;
    if (r < rows) {
      const float l = g.lse[(row + r) * a.Hq + h];
      if (g.dlse) s -= g.dlse[(row + r) * a.Hq + h];
      lse = l == -INFINITY ? INFINITY : l == INFINITY ? __int_as_float(0x7fffffff) : l;
      if (l == -INFINITY) s = 0.f;
    }
    sums[r] = lse, sums[kSumRows + r] = s;
    info[r] = -lse, info[kPast + r] = -s;
  });
}

// ---------------------------------------------------------------- products
template <int D, bool KEYS>
struct Cfg32 {
  static constexpr int kWarps = 8;  // of softmax threads
  // one more warp copies the tiles and issues the products; its warpgroup gives its registers to the others
  static constexpr int kMmaWarp = kWarps, kThreads = 32 * kWarps + 128;
  static constexpr int kOwnBytes = kTile * D * 4, kTileBytes = kPast * D * 4;
  // places of the first tiles (Q; K), which are read until the tile's last product, and of the second ones (dO; V); the
  // second owned tile (V; dO) lies in the first tiles' places 1 and 2 until it is in TMEM
  static constexpr int kP1 = D == 64 ? 4 : 3, kP2 = D == 64 ? 4 : 2;
  static constexpr int kRing = (kP1 + kP2) * kTileBytes;
  static constexpr int kInfo = KEYS ? kQInfo : kKInfo;
  // TMEM: dK and dV: X (then P over it), Y (then dS), the tile's sums of dV and of dK; dQ: two of X (then dS), two of Y,
  // the tile's sums.  Then the second owned tile.
  static constexpr uint32_t kColX = 0, kColY = KEYS ? kPast : 2 * kPast, kColV = 2 * kColY, kColA = kColV + (KEYS ? 2 : 1) * D;
  static constexpr int kSmem = kOwnBytes + kRing + 2 * kInfo + 1024 + 256;
};
struct Bars32 {
  uint64_t own, ready, full1[4], empty1[4], full2[4], empty2[4], info[2], x[2], y, p, ds, drain, stall;
  uint32_t tmem, failed;
  uint32_t bad[2][4];  // rows that are not finite, a bit each
};
static_assert(sizeof(Bars32) <= 256 && Cfg32<128, true>::kSmem <= 227 * 1024 && Cfg32<128, false>::kSmem <= 227 * 1024 &&
                  Cfg32<64, true>::kSmem <= 227 * 1024 && Cfg32<128, true>::kColA + 128 <= 512 &&
                  Cfg32<128, false>::kColA + 128 <= 512, "shared memory and TMEM");

struct Tc32Args {
  GradArgs g;
  Operands w;
  int qblocks;  // of a sequence
  bool packed;
  bool second;  // of the call's two kernels
  int split;    // CTAs of a cluster
  uint32_t* status;
  uint64_t limit;
  int stall;
};

__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn = false) {
  return idesc_bf16(M, N, false, b_mn) & ~((1u << 7) | (1u << 10));
}
// A warp's 16 rows, two lanes a row: lane t < 16 holds columns c to c + 31 (or 15) of row t, lane t + 16 those OFF later.
template <int OFF>
__device__ __forceinline__ void tmem_ld_rows16(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x32bx2.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32], %33;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]),
        "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr), "n"(OFF)
      : "memory");
}
__device__ __forceinline__ void tmem_st_rows16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x32bx2.x16.b32 [%0], 16, {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// two pairs of a row of numbers, the same for every thread; four pairs of a row of factors
__device__ __forceinline__ void load_pairs(const float* p, uint64_t& a, uint64_t& b) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  a = pack2(v.x, v.y), b = pack2(v.z, v.w);
}
__device__ __forceinline__ void load_factors(const uint8_t* p, uint64_t (&f)[4]) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
// Rows of a tile of P or dS to TMEM: each with its own power of two, hi's in 32 columns, lo's in the next 32.  Returns the
// factor that undoes the power.
__device__ __forceinline__ float store_weights(uint32_t to, const uint64_t (&x)[16]) {
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    float a, b;
    unpack2(x[e], a, b);
    m = max3(m, fabsf(a), fabsf(b));
  }
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
  float up, down;
  row_factors(m, up, down);
  const uint64_t up2 = pack2(up, up);
  uint32_t hi[16], lo[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) split2(mul2(x[e], up2), hi[e], lo[e]);
  tmem_st_rows16(to, hi);
  tmem_st_rows16(to + 32, lo);
  return down;
}
// acc += f times this lane's half of a row of a tile's sums
template <int D>
__device__ __forceinline__ void add_sums(uint64_t (&acc)[D / 4], uint32_t from, float f) {
  const uint64_t f2 = pack2(f, f);
  uint32_t v[D / 64][32];
#pragma unroll
  for (int c = 0; c < D / 64; ++c) tmem_ld_rows16<D / 2>(from + 32 * c, v[c]);
  tmem_wait_ld();
#pragma unroll
  for (int e = 0; e < D / 4; ++e)
    acc[e] = fma2(pack2(__uint_as_float(v[e >> 4][(2 * e) & 31]), __uint_as_float(v[e >> 4][(2 * e + 1) & 31])), f2, acc[e]);
}

template <int D, bool KEYS>
__global__ void __launch_bounds__(Cfg32<D, KEYS>::kThreads, 1) attn_grad_tc32_kernel(const Tc32Args t) {
  using C = Cfg32<D, KEYS>;
  constexpr int N = kPast, P1 = C::kP1, P2 = C::kP2, kHalf = C::kTileBytes / 2;
  const GradArgs& g = t.g;
  const PromptArgs& a = g.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint8_t *s1 = smem, *ring1 = s1 + C::kOwnBytes, *ring2 = ring1 + P1 * C::kTileBytes, *s2 = ring1 + C::kTileBytes;
  uint8_t* infos = ring1 + C::kRing;
  Bars32* bar = reinterpret_cast<Bars32*>(infos + 2 * C::kInfo);
  if (warp == C::kMmaWarp) {
    tmem_alloc(&bar->tmem, 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    mbar_init(&bar->own, 1);
    mbar_init(&bar->ready, C::kWarps);
    mbar_init(&bar->info[0], 1);
    mbar_init(&bar->info[1], 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bar->full1[i], 1);
      mbar_init(&bar->empty1[i], 1);
      mbar_init(&bar->full2[i], 1);
      mbar_init(&bar->empty2[i], 1);
    }
    mbar_init(&bar->x[0], 1);
    mbar_init(&bar->x[1], 1);
    mbar_init(&bar->y, 1);
    mbar_init(&bar->p, C::kWarps);
    mbar_init(&bar->ds, C::kWarps);
    mbar_init(&bar->drain, 1);
    mbar_init(&bar->stall, 1);
    bar->failed = 0;
    for (int i = 0; i < 8; ++i) bar->bad[i >> 2][i & 3] = 0;
    fence_mbar_init();
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
  const bool valid = row0 >= 0 && row0 < rows && q0 >= 0 && k0 >= 0 && lq_all >= 0 && lk >= 0 && q0 + lq_all <= a.tokens &&
                     k0 + lk <= a.k_tokens;
  // a sequence's blocks are dealt out from its last; the first keys, which the most queries see, come first
  if (KEYS) row0 = (lk - 1) / kTile * kTile - row0;
  // the tiles that come past, [first, first + each N) of every head
  const int first = KEYS ? max(row0 - off, 0) / N * N : 0;
  const int end = KEYS ? lq : min(min(row0 + kTile, lq) + off, lk);
  const int each = end > first ? (end - first + N - 1) / N : 0;
  int i0 = 0, n = each;  // this CTA's
  if (KEYS) {
    const int64_t all = static_cast<int64_t>(each) * G;
    i0 = static_cast<int>(all * rank / t.split);
    n = static_cast<int>(all * (rank + 1) / t.split) - i0;
  }
  __syncthreads();
  const uint32_t tmem = bar->tmem;
  if (!t.second) {  // the operands are there
    wait_for_previous();
    launch_dependents();
  }
  const bool last = t.second && blockIdx.x == gridDim.x - 1 && tid == C::kThreads - 1;  // ends no sooner than the first kernel
  if (!valid) {  // (the whole cluster)
    if (warp == C::kMmaWarp) tmem_dealloc(tmem, 512);
    if (last) wait_for_previous();
    return;
  }
  auto wait = [&](uint64_t* m, uint32_t parity) {
    if (mbar_wait_sleep(m, parity, t.limit)) return true;
    atomicExch(t.status, kStatusTimeout);
    *static_cast<volatile uint32_t*>(&bar->failed) = 1;
    return false;
  };
  // blocks of the workspace: the owned rows' first one; tile i's
  const int64_t own_block = (KEYS ? head * t.w.k_blocks + first64(k0, b) : head * t.w.q_blocks + first64(q0, b)) + row0 / kPast;
  auto past_block = [&](int i) {
    return (KEYS ? (head * G + (i0 + i) / each) * t.w.q_blocks + first64(q0, b) : head / G * t.w.k_blocks + first64(k0, b)) +
           first / kPast + (KEYS ? (i0 + i) % each : i);
  };

  // 256 x 224 + 128 x 56 = 384 x 168
  if (warp >= C::kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (last) wait_for_previous();
    __syncwarp();
  }
  if (warp == C::kMmaWarp) {
    // One lane walks the loop, see the bf16 kernels.
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    if (elect_one()) {
      constexpr uint32_t id_x = idesc_f16(kTile, N), id_s = idesc_f16(kTile, D, true);
      const uint64_t a1 = sdesc_k128(smem_u32(s1));
      const uint64_t bk1 = sdesc_k128(smem_u32(ring1)), bk2 = sdesc_k128(smem_u32(ring2));
      const uint64_t bm1 = D == 64 ? sdesc_mn128(smem_u32(ring1)) : sdesc_mn128_wide(smem_u32(ring1), N * 128);
      const uint64_t bm2 = D == 64 ? sdesc_mn128(smem_u32(ring2)) : sdesc_mn128_wide(smem_u32(ring2), N * 128);
      auto arrived = [&](uint64_t* m, uint32_t parity) {
        const bool ok = wait(m, parity);
        tc_fence_after();
        return ok;
      };
      auto full1 = [&](int i) { return arrived(&bar->full1[i % P1], (i / P1) & 1); };
      auto full2 = [&](int i) { return arrived(&bar->full2[i % P2], (i / P2) & 1); };
      // to = the owned rows times tile i's; lo hi, hi lo, hi hi
      auto scores = [&](uint32_t to, int i, int second, uint64_t* then, uint64_t* frees) {
        const uint64_t bs = second ? bk2 + i % P2 * (C::kTileBytes >> 4) : bk1 + i % P1 * (C::kTileBytes >> 4);
#pragma unroll
        for (int part = 0; part < 3; ++part)
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint64_t bd = bs + (part == 1 ? kHalf >> 4 : 0) + (((ks >> 2) * N * 128 + (ks & 3) * 32) >> 4);
            if (second)
              umma_ts(tm + to, tm + C::kColA + (part == 0 ? D / 2 : 0) + ks * 8, bd, id_x, part > 0 || ks > 0);
            else
              umma_bf16(tm + to, a1 + (part == 0 ? C::kOwnBytes / 2 >> 4 : 0) + (((ks >> 2) * kTile * 128 + (ks & 3) * 32) >> 4),
                        bd, id_x, part > 0 || ks > 0);
          }
        if (then) umma_commit(then);
        if (frees) umma_commit(frees);
      };
      // sum = W (halves in TMEM) times tile i
      auto weighted = [&](uint32_t sum, uint32_t w, int i, int second, uint64_t* frees) {
        const uint64_t bs = second ? bm2 + i % P2 * (C::kTileBytes >> 4) : bm1 + i % P1 * (C::kTileBytes >> 4);
#pragma unroll
        for (int part = 0; part < 3; ++part)
#pragma unroll
          for (int ks = 0; ks < N / 16; ++ks)
            umma_ts(tm + sum, tm + w + (part == 0 ? 32 : 0) + ks * 8, bs + (part == 1 ? kHalf >> 4 : 0) + ks * 128, id_s,
                    part > 0 || ks > 0);
        umma_commit(frees);
      };
      // copies of the next tile's first and second part, and of its rows' numbers
      int loads1 = 0, loads2 = 0, infos_in = 0;
      auto load = [&](uint8_t* to, const uint8_t* from, int bytes, uint64_t* full) {
        mbar_arrive_expect_tx(full, bytes);
        bulk_load(to, from, bytes, full);
      };
      auto load1 = [&] {
        const int i = loads1++, at = i % P1;
        load(ring1 + at * C::kTileBytes, (KEYS ? t.w.q : t.w.k) + past_block(i) * C::kTileBytes, C::kTileBytes, &bar->full1[at]);
      };
      auto load2 = [&] {
        const int i = loads2++, at = i % P2;
        load(ring2 + at * C::kTileBytes, (KEYS ? t.w.d_o : t.w.v) + past_block(i) * C::kTileBytes, C::kTileBytes, &bar->full2[at]);
      };
      auto load_info = [&] {
        const int i = infos_in++;
        load(infos + (i & 1) * C::kInfo, (KEYS ? t.w.q_info : t.w.k_info) + past_block(i) * C::kInfo, C::kInfo, &bar->info[i & 1]);
      };
      // The place of tile i - P's is free.  Its last product is that of dK or dQ, which also ends the use of the tile's numbers.
      auto more1 = [&](int i) {
        const int done = i - P1;
        if (done + 2 >= n && i >= n) return true;
        if (!arrived(&bar->empty1[i % P1], (i / P1 - 1) & 1)) return false;
        if (done + 2 < n) load_info();
        if (i < n) load1();
        return true;
      };
      auto more2 = [&](int i) { return i >= n || (arrived(&bar->empty2[i % P2], (i / P2 - 1) & 1) && (load2(), true)); };
      bool ok = n > 0 && (!t.stall || arrived(&bar->stall, 0));
      const bool own = ok;
      if (ok) {
        // slabs of 128 rows from two blocks' of 64; the second block may not be there, no row of it counts then
        const int halves = row0 + kPast < rows ? 2 : 1;
        mbar_arrive_expect_tx(&bar->own, halves * 2 * C::kTileBytes);
        for (int s = 0; s < 2 * halves; ++s) {
          const uint8_t* from = ((s & 1) ? (KEYS ? t.w.v : t.w.d_o) : (KEYS ? t.w.k : t.w.q)) + (own_block + (s >> 1)) * C::kTileBytes;
          uint8_t* to = ((s & 1) ? s2 : s1) + (s >> 1) * (kPast * 128);
          for (int c = 0; c < D / 32; ++c) bulk_load(to + c * (kTile * 128), from + c * (kPast * 128), kPast * 128, &bar->own);
        }
        load1();
        for (int i = 0; i < min(n, P2); ++i) load2();
        for (int i = 0; i < min(n, 2); ++i) load_info();
        ok = arrived(&bar->own, 0) && full1(0);
      }
      if (ok) {
        scores(C::kColX, 0, 0, KEYS ? &bar->x[0] : nullptr, nullptr);
        ok = arrived(&bar->ready, 0);
        for (int i = 1; i < min(n, P1) && ok; ++i) load1();
      }
      // A place's next copy waits for the place's last product while another one runs.
      if constexpr (KEYS) {
        for (int i = 0; i < n && ok; ++i) {
          if (!(ok = full2(i))) break;
          scores(C::kColY, i, 1, &bar->y, nullptr);
          if (i > 0 && !(ok = more1(i - 1 + P1))) break;
          if (!(ok = arrived(&bar->p, i & 1))) break;
          weighted(C::kColV, C::kColX, i, 1, &bar->empty2[i % P2]);
          if (i + 1 < n) {
            if (!(ok = full1(i + 1))) break;
            scores(C::kColX, i + 1, 0, &bar->x[0], nullptr);
          }
          if (!(ok = more2(i + P2))) break;
          if (!(ok = arrived(&bar->ds, i & 1))) break;
          weighted(C::kColV + D, C::kColY, i, 0, &bar->empty1[i % P1]);
        }
      } else {
        // dS of tiles i and i - 1 lie over X of them; Y of tile i + 1 over that of tile i - 1
        if (ok && (ok = full2(0))) scores(C::kColY, 0, 1, &bar->x[0], &bar->empty2[0]);
        if (ok) ok = more2(P2);
        for (int i = 0; i < n && ok; ++i) {
          const uint32_t next = (i + 1) & 1;
          if (i + 1 < n) {
            if (!(ok = full1(i + 1))) break;
            scores(C::kColX + next * N, i + 1, 0, nullptr, nullptr);
            if (i > 0 && !(ok = more1(i - 1 + P1))) break;
            if (!(ok = full2(i + 1))) break;
            scores(C::kColY + next * N, i + 1, 1, &bar->x[next], &bar->empty2[(i + 1) % P2]);
          }
          if (!(ok = arrived(&bar->ds, i & 1))) break;
          weighted(C::kColV, C::kColX + (i & 1) * N, i, 0, &bar->empty1[i % P1]);
          if (i + 1 < n && !(ok = more2(i + 1 + P2))) break;
        }
      }
      umma_commit(&bar->drain);  // products in flight end before the memory is freed
      wait(&bar->drain, 0);
      // every copy has landed before the CTA may end
      if (own) wait(&bar->own, 0);
      for (int i = max(0, loads1 - P1); i < loads1; ++i) wait(&bar->full1[i % P1], (i / P1) & 1);
      for (int i = max(0, loads2 - P2); i < loads2; ++i) wait(&bar->full2[i % P2], (i / P2) & 1);
      for (int i = max(0, infos_in - 2); i < infos_in; ++i) wait(&bar->info[i & 1], (i >> 1) & 1);
    }
    __syncwarp();
  } else if (warp < C::kMmaWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    // A warp takes 16 rows, two lanes a row: 32 of a tile's columns each, half of the dims of the row's sums each.
    const int group = warp >> 2, quad = warp & 3, r = quad * 32 + group * 16 + (lane & 15), half = lane >> 4;
    const uint32_t mine = tmem + (static_cast<uint32_t>(quad * 32 + group * 16) << 16);
    const int row = row0 + r;
    auto arrive = [&](uint64_t* m) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(m);
    };
    auto waited = [&](uint64_t* m, uint32_t parity) {
      const bool ok = __all_sync(0xffffffffu, wait(m, parity)) != 0;
      tc_fence_after();
      return ok;
    };
    bool ok = true;
    uint64_t acc[D / 4], acc_v[KEYS ? D / 4 : 1];  // dK or dQ; dV
#pragma unroll
    for (int e = 0; e < D / 4; ++e) acc[e] = acc_v[KEYS ? e : 0] = 0;
    // this row's factors; of rows past the sequence anything
    const int64_t blk = own_block + (r >> 6);
    const bool live = row < rows;
    float f1 = 0.f, f2 = 0.f, lse = -INFINITY, delta = 0.f;  // lse, delta: negative
    if (live && n > 0) {
      const int at = r & 63;
      if (KEYS) {
        const uint8_t* info = t.w.k_info + blk * kKInfo;
        f1 = a.scale * factor_at(info, at), f2 = factor_at(info, kPast + at);
      } else {
        const uint8_t* info = t.w.q_info + blk * kQInfo;
        f1 = a.scale * factor_at(info + 8 * kPast, at), f2 = factor_at(info + 8 * kPast, kPast + at);
        const float* sums = reinterpret_cast<const float*>(info) + at;
        lse = load_past_l1(sums), delta = load_past_l1(sums + kPast);
      }
    }
    // the second owned tile to TMEM, a row a thread: the hi's by one warpgroup, the lo's by the other
    if (n > 0 && (ok = waited(&bar->own, 0))) {
#pragma unroll
      for (int s = 0; s < D / 64; ++s) {
        const uint8_t* from = s2 + group * (C::kOwnBytes / 2) + s * (kTile * 128);
        uint32_t w[32];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint4 x = *reinterpret_cast<const uint4*>(from + sw128(quad * 32 + lane, c * 8));
          w[4 * c] = x.x, w[4 * c + 1] = x.y, w[4 * c + 2] = x.z, w[4 * c + 3] = x.w;
        }
        tmem_st32(tmem + (static_cast<uint32_t>(quad * 32) << 16) + C::kColA + group * (D / 2) + s * 32, w);
      }
      tmem_wait_st();
      arrive(&bar->ready);
    }
    const uint64_t f1p = pack2(f1, f1), f2p = pack2(f2, f2), l2e = pack2(kLog2e, kLog2e);
    const uint64_t lse2 = pack2(lse, lse), delta2 = pack2(delta, delta);
    // P from X: ls the log sums (dQ: lse2), s the columns' factors
    auto weights = [&](uint32_t from, const uint8_t* s, const float* ls, int lim, bool cut, uint64_t (&x)[16]) {
      uint32_t v[32];
      tmem_ld_rows16<32>(from, v);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint64_t s4[4], l4[4] = {lse2, lse2, lse2, lse2};
        load_factors(s + half * 64 + 16 * e, s4);
        if (KEYS) {
          load_pairs(ls + half * 32 + 8 * e, l4[0], l4[1]);
          load_pairs(ls + half * 32 + 8 * e + 4, l4[2], l4[3]);
        }
        // The difference first: it is small where the weight is not.  The two factors first: X times one of them may pass
        // fp32's range where the score does not (an infinite score of the wrong size would be a weight of 0, unnoticed).
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint64_t y = pack2(__uint_as_float(v[8 * e + 2 * k]), __uint_as_float(v[8 * e + 2 * k + 1]));
          x[4 * e + k] = mul2(fma2(y, mul2(f1p, s4[k]), l4[k]), l2e);
        }
      }
      if (cut) {
        lim -= half * 32;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float z0, z1;
          unpack2(x[e], z0, z1);
          if (KEYS ? 2 * e < lim : 2 * e >= lim) z0 = -INFINITY;
          if (KEYS ? 2 * e + 1 < lim : 2 * e + 1 >= lim) z1 = -INFINITY;
          x[e] = pack2(z0, z1);
        }
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float z0, z1;
        unpack2(x[e], z0, z1);
        x[e] = pack2(ex2(z0), ex2(z1));
      }
    };
    // dS from P and Y, times the factors w of the rows that the sum runs over: s the columns' factors, ds their D (dQ: delta2)
    auto differences = [&](uint32_t from, const uint8_t* s, const float* ds, const uint8_t* w, uint64_t (&x)[16]) {
      uint32_t v[32];
      tmem_ld_rows16<32>(from, v);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint64_t s4[4], d4[4] = {delta2, delta2, delta2, delta2}, w4[4];
        load_factors(s + half * 64 + 16 * e, s4);
        load_factors(w + half * 64 + 16 * e, w4);
        if (KEYS) {
          load_pairs(ds + half * 32 + 8 * e, d4[0], d4[1]);
          load_pairs(ds + half * 32 + 8 * e + 4, d4[2], d4[3]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint64_t y = mul2(pack2(__uint_as_float(v[8 * e + 2 * k]), __uint_as_float(v[8 * e + 2 * k + 1])), f2p);
          x[4 * e + k] = mul2(mul2(x[4 * e + k], fma2(y, s4[k], d4[k])), w4[k]);
        }
      }
    };
    float down = 0.f, down_v = 0.f;  // of the tile whose sums come next
    for (int i = 0, past = KEYS && n > 0 ? i0 % each : 0; i < n; ++i) {
      const int at = first + past * N;
      if (KEYS && ++past == each) past = 0;
      if (!KEYS) past = i + 1;
      const uint8_t* info = infos + (i & 1) * C::kInfo;
      uint64_t x[16];
      if constexpr (KEYS) {
        const float* numbers = reinterpret_cast<const float*>(info);  // log sums, D
        const uint8_t* factors = info + 8 * kPast;                   // of Q, of dO
        // the sums of the tile before, while X and Y of this one are formed
        if (i > 0) {
          if (!(ok = waited(&bar->empty2[(i - 1) % P2], ((i - 1) / P2) & 1))) break;
          add_sums<D>(acc_v, mine + C::kColV, down_v);
        }
        if (!(ok = waited(&bar->info[i & 1], (i >> 1) & 1) && waited(&bar->x[0], i & 1))) break;
        // cut: some key is behind a query of these
        weights(mine + C::kColX, factors, numbers, row - off - at, at + off < row0 + kTile - 1, x);
        uint64_t z[16];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint64_t s4[4];
          load_factors(factors + 2 * kPast + half * 64 + 16 * e, s4);
#pragma unroll
          for (int k = 0; k < 4; ++k) z[4 * e + k] = mul2(x[4 * e + k], s4[k]);
        }
        down_v = store_weights(mine + C::kColX, z);
        tmem_wait_st();
        arrive(&bar->p);
        if (i > 0) {
          if (!(ok = waited(&bar->empty1[(i - 1) % P1], ((i - 1) / P1) & 1))) break;
          add_sums<D>(acc, mine + C::kColV + D, down);
        }
        if (!(ok = waited(&bar->y, i & 1))) break;
        differences(mine + C::kColY, factors + 2 * kPast, numbers + kPast, factors, x);
        down = store_weights(mine + C::kColY, x);
      } else {
        const uint32_t tx = mine + C::kColX + (i & 1) * N;
        if (!(ok = waited(&bar->info[i & 1], (i >> 1) & 1) && waited(&bar->x[i & 1], (i >> 1) & 1))) break;
        weights(tx, info, nullptr, min(row + off + 1, lk) - at, at + N > min(row0 + off + 1, lk), x);  // info: factors of K, of V
        differences(mine + C::kColY + (i & 1) * N, info + 2 * kPast, nullptr, info, x);
        const float was = down;
        down = store_weights(tx, x);
        if (i > 0) {  // the sums of the tile before
          if (!(ok = waited(&bar->empty1[(i - 1) % P1], ((i - 1) / P1) & 1))) break;
          add_sums<D>(acc, mine + C::kColV, was);
        }
      }
      tmem_wait_st();
      arrive(&bar->ds);
    }
    // the last tile's sums
    if (ok && n > 0 && (ok = waited(&bar->drain, 0))) {
      if constexpr (KEYS) add_sums<D>(acc_v, mine + C::kColV, down_v);
      add_sums<D>(acc, mine + C::kColV + (KEYS ? D : 0), down);
    }
    const int d = D == 64 ? a.d : D;  // of the rows
    // a row of a result (x1: dK or dQ, x2: dV) from the definition
    auto compute_again = [&](int i, float (&x1)[4], float (&x2)[4]) {
      const float *q = static_cast<const float*>(a.q.p), *d_o = static_cast<const float*>(g.d_o.p);
      const float *k = static_cast<const float*>(a.k.p), *v = static_cast<const float*>(a.v.p);
      const float* sums = g.sums + row_sums(g.blocks, KEYS ? head * G : head, first_block(q0, b));
      if constexpr (KEYS) {
        const int64_t h0 = static_cast<int64_t>(head) * G * d, hk = static_cast<int64_t>(head) * d;
        grad_key_row<float, D>(k + (k0 + i) * a.k.stride + hk, v + (k0 + i) * a.v.stride + hk, q + q0 * a.q.stride + h0,
                               a.q.stride, d_o + q0 * g.d_o.stride + h0, g.d_o.stride, sums, g.blocks, G, max(i - off, 0), lq,
                               d, a.scale, x1, x2);
      } else {
        const int64_t h0 = static_cast<int64_t>(head) * d, hk = static_cast<int64_t>(head / G) * d;
        const float* s = sums + static_cast<int64_t>(i / kSumRows) * (2 * kSumRows) + i % kSumRows;
        grad_query_row<float, D>(q + (q0 + i) * a.q.stride + h0, d_o + (q0 + i) * g.d_o.stride + h0, load_past_l1(s),
                                 load_past_l1(s + kSumRows), k + k0 * a.k.stride + hk, a.k.stride,
                                 v + k0 * a.v.stride + hk, a.v.stride, min(i + off + 1, lk), d, a.scale, x1);
      }
    };
    // this lane's half of its row of a result; which: dV (0), dK or dQ (1)
    auto finish = [&](const uint64_t (&z)[D / 4], int which) {
      const RowsOut& to = KEYS ? (which ? g.dk : g.dv) : g.dq;
      float* out = static_cast<float*>(to.p) + ((KEYS ? k0 : q0) + row0) * to.stride + static_cast<int64_t>(head) * d;
      const float f = which ? a.scale : 1.f;
      const uint64_t fp = pack2(f, f);
      uint64_t rest = 0;  // z * 0 added up: NaN where some z is not finite
#pragma unroll
      for (int e = 0; e < D / 8; ++e) {
        const uint64_t z0 = mul2(z[2 * e], fp), z1 = mul2(z[2 * e + 1], fp);
        rest = fma2(z0, 0, fma2(z1, 0, rest));
        const int c = half * (D / 2) + 4 * e;
        if (!live || c >= d) continue;
        float4 v;
        unpack2(z0, v.x, v.y);
        unpack2(z1, v.z, v.w);
        float* dst = out + r * to.stride + c;
        if (to.vec) *reinterpret_cast<float4*>(dst) = v;
        else dst[0] = v.x, dst[1] = v.y, dst[2] = v.z, dst[3] = v.w;
      }
      float ra, rb;
      unpack2(rest, ra, rb);
      __syncwarp();
      for (uint32_t again = __ballot_sync(0xffffffffu, live && !(ra + rb == 0.f)); again; again &= again - 1) {
        const int from = __ffs(again) - 1, i = row0 + quad * 32 + group * 16 + (from & 15);
        float x1[4], x2[4];
        compute_again(i, x1, x2);
#pragma unroll
        for (int m = 0; m < D / 32; ++m) {
          const int c = m * 32 + lane;
          if (m / (D / 64) == from >> 4 && c < d) out[(i - row0) * to.stride + c] = KEYS && !which ? x2[m] : x1[m];
        }
      }
    };
    if (!KEYS || t.split == 1) {
      if (ok) {  // the same in all lanes
        if constexpr (KEYS) finish(acc_v, 0);
        finish(acc, 1);
      }
    } else if constexpr (KEYS) {
      // the owned tile's and the ring's place: every product is done
      uint8_t* dst = smem + r * (D * 4);
#pragma unroll
      for (int e = 0; e < D / 8; ++e) {
        const int c = ((half * (D / 8) + e) ^ (r & 7)) << 4;
        *reinterpret_cast<ulonglong2*>(dst + c) = make_ulonglong2(acc_v[2 * e], acc_v[2 * e + 1]);
        *reinterpret_cast<ulonglong2*>(dst + kTile * D * 4 + c) = make_ulonglong2(acc[2 * e], acc[2 * e + 1]);
      }
      cluster_sums<float, D, 32 * C::kWarps>(g, smem, &bar->failed, bar->bad, t.split, rank, row0, rows, k0, head, d, compute_again);
    }
    tc_fence_before();
  }
  if (KEYS && t.split > 1 && warp >= C::kMmaWarp) {
    __syncwarp();
    cluster_barrier();
    cluster_barrier();
  }
  __syncthreads();
  if (warp == C::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool KEYS>
int launch_kernel(Tc32Args& t, int64_t grid, cudaStream_t s) {
  if (grid < 1 || grid > INT32_MAX / t.split) return FALCON_ERR_UNSUPPORTED;
  t.stall = take_test_stall() ? 1 : 0;
  const auto kern = attn_grad_tc32_kernel<D, KEYS>;
  if (!set_smem_limit(reinterpret_cast<const void*>(kern), Cfg32<D, KEYS>::kSmem)) return FALCON_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid * t.split));
  cfg.blockDim = dim3(Cfg32<D, KEYS>::kThreads);
  cfg.dynamicSmemBytes = Cfg32<D, KEYS>::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2] = {overlap_attribute(), cluster_attribute(t.split)};
  cfg.attrs = attr;
  cfg.numAttrs = t.split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, t) == cudaSuccess ? FALCON_OK : FALCON_ERR_CUDA;
}

// The parts of the workspace from `base` on; bytes: all of them.
Operands operands(uint8_t* base, const PromptArgs& a, int D, size_t* bytes) {
  Operands w;
  w.q_blocks = count_blocks(a.tokens, a.B);
  w.k_blocks = count_blocks(a.k_tokens, a.B);
  size_t at = 0;
  auto part = [&](int64_t blocks, size_t size) {
    uint8_t* p = base + at;
    at += static_cast<size_t>(blocks) * size;
    return p;
  };
  const int64_t nq = w.q_blocks * a.Hq, nk = w.k_blocks * a.Hkv;
  const size_t image = static_cast<size_t>(kPast) * D * 4;
  w.q = part(nq, image), w.d_o = part(nq, image), w.k = part(nk, image), w.v = part(nk, image);
  w.q_info = part(nq, kQInfo), w.k_info = part(nk, kKInfo);
  *bytes = at;
  return w;
}

template <int D>
int launch_d(const GradArgs& g, cudaStream_t s) {
  const PromptArgs& a = g.a;
  Tc32Args t;
  t.g = g;
  size_t bytes;
  t.w = operands(reinterpret_cast<uint8_t*>(g.sums + row_sums(g.blocks, a.Hq, 0)), a, D, &bytes);
  t.qblocks = 0, t.packed = false;
  t.status = static_cast<uint32_t*>(a.ws);
  t.limit = wait_limit_ns();
  const int64_t q_ctas = a.tokens > 0 && a.max_q > 0 ? (a.tokens / kPast + a.B) * a.Hq : 0;
  const int64_t k_ctas = a.k_tokens > 0 ? (a.k_tokens / kPast + a.B) * a.Hkv : 0;
  if (q_ctas + k_ctas > INT32_MAX) return FALCON_ERR_UNSUPPORTED;
  attn_grad_split_kernel<D><<<static_cast<unsigned>(q_ctas + k_ctas), 256, 0, s>>>(g, t.w, static_cast<unsigned>(q_ctas));
  if (cudaGetLastError() != cudaSuccess) return FALCON_ERR_CUDA;
  t.second = false;
  t.split = 1;
  if (g.dk.p && k_ctas) {  // first: its CTAs run longest
    const int64_t blocks = a.k_tokens / kTile + a.B;
    t.split = keys_split(a, kPast, sm_count(), 3, 8);
    const int st = blocks > INT32_MAX / a.Hkv ? FALCON_ERR_UNSUPPORTED : launch_kernel<D, true>(t, blocks * a.Hkv, s);
    if (st != FALCON_OK) return st;
    t.split = 1;
    t.second = true;
  }
  if (g.dq.p && q_ctas) {
    const PromptGrid pg = query_grid(a);
    t.qblocks = static_cast<int>(pg.blocks / a.B);
    t.packed = pg.packed;
    return pg.blocks > INT32_MAX / a.Hq ? FALCON_ERR_UNSUPPORTED : launch_kernel<D, false>(t, pg.blocks * a.Hq, s);
  }
  return FALCON_OK;
}

}  // namespace

size_t attn_grad_tc32_ws_bytes(int64_t tokens, int64_t k_tokens, int B, int Hq, int Hkv, int d) {
  PromptArgs a = {};
  a.B = B, a.Hq = Hq, a.Hkv = Hkv, a.tokens = tokens, a.k_tokens = k_tokens;
  size_t bytes;
  operands(nullptr, a, d <= 64 ? 64 : 128, &bytes);
  return bytes;
}

int launch_attn_grad_tc32(const GradArgs& g, cudaStream_t s) {
  return g.a.d <= 64 ? launch_d<64>(g, s) : launch_d<128>(g, s);
}

}  // namespace falcon
