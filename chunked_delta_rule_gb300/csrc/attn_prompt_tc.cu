// Causal attention over packed prompts on the tensor cores (bf16, d = 64, 128).
//
//   S = Q K^T (128 queries x 128 keys),  P = exp(scale S - m),  O += P V
//
// Bound by the tensor cores: 4 d flops a visible (query, key) pair and head.
// A CTA takes 256 queries of one head as two 128-row tiles.  One thread issues
// every tcgen05.mma; while it runs one tile's P V and next Q K^T, the other
// tile's softmax runs, so that neither waits for the other:
//   warps 0-3, 4-7   softmax of tile 0 and 1, a row a thread: the scores are
//                    read from TMEM once, P (bf16) goes back over them and
//                    is the next product's A operand from there
//   warp 8           TMA loads: Q once, K and V tiles through a ring
//   warp 9           the products (warps 10 and 11 fill the warpgroup)
// TMEM: S0 | S1 (128 columns each, P in their first 64) | O0 | O1 (d each).
// The reference m of a row moves only when a score passes it by more than
// 2^8, so O is rescaled rarely; sums are of the unrounded weights, fp32.
// P is rounded to bf16 as V is held in it: at most 2^-8 of a weight.
//
// Masked scores are set to -inf after the product, so what the masked keys
// hold does not matter; a masked weight is 0, but 0 times an infinite or NaN
// value of a key that only other rows see would still spoil the row.  A row
// whose result is not finite is therefore computed again from the definition,
// by its warp, touching only the keys that it sees.

#include "attn_row.cuh"
#include "tc_util.cuh"

namespace falcon {
namespace {

using namespace tcu;

constexpr int kTile = 128;        // queries and keys of a tile
constexpr int kThreads = 384;
// Registers: 384 x 168 at launch; 256 softmax threads take 208, the other 128 keep 88 (the same sum).
constexpr float kSlack = 8.f;     // log2

template <int D>
struct Cfg {
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kStages = D == 64 ? 8 : 5;
  static constexpr int kSmem = (2 + kStages) * kTileBytes + 1024 + 256;
  static constexpr uint32_t kColS = 0, kColO = 256;
};

struct Bars {
  uint64_t q[2], full[8], empty[8], s[2], p[2], drain, stall;
  uint32_t tmem;
};

struct TcArgs {
  PromptArgs a;
  int qblocks;
  uint32_t* status;
  uint64_t limit;
  int stall;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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

// tiles of 128 keys that rows up to (and with) `last` of a sequence see
__device__ __forceinline__ int key_tiles(int last, int off, int lk) {
  const int n = min(last + off + 1, lk);
  return n <= 0 ? 0 : (n + kTile - 1) / kTile;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_prompt_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                          const __grid_constant__ CUtensorMap mv, const TcArgs t) {
  using C = Cfg<D>;
  const PromptArgs& a = t.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (blockIdx.x == 0 && tid == 0) atomicExch(t.status, 0u);  // before any wait of this call can run out

  // the longest rows first: blocks of queries descend, sequences and heads within
  const int64_t bh = static_cast<int64_t>(a.B) * a.Hq;
  const int qb = t.qblocks - 1 - static_cast<int>(blockIdx.x / bh);
  const int b = static_cast<int>(blockIdx.x % bh) / a.Hq, h = static_cast<int>(blockIdx.x % bh) % a.Hq;
  const int64_t q0 = a.cu_q[b], k0 = a.cu_k[b];
  const int lq_all = static_cast<int>(a.cu_q[b + 1] - q0), lk = static_cast<int>(a.cu_k[b + 1] - k0);
  const int lq = min(lq_all, a.max_q), off = lk - lq_all, row0 = qb * 2 * kTile;
  if (row0 >= lq || q0 < 0 || k0 < 0 || q0 + lq_all > a.tokens || k0 + lk > a.k_tokens) return;
  const int hk = h / (a.Hq / a.Hkv);
  int n[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int r = row0 + x * kTile;
    n[x] = r < lq ? key_tiles(min(r + kTile, lq) - 1, off, lk) : 0;
  }
  const int nmax = max(n[0], n[1]);

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint8_t* sQ = smem;
  uint8_t* ring = smem + 2 * C::kTileBytes;
  Bars* bar = reinterpret_cast<Bars*>(ring + C::kStages * C::kTileBytes);
  if (warp == 9) {
    tmem_alloc(&bar->tmem, 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bar->q[x], 1);
      mbar_init(&bar->s[x], 1);
      mbar_init(&bar->p[x], kTile);
    }
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&bar->full[i], 1);
      mbar_init(&bar->empty[i], 1);
    }
    mbar_init(&bar->drain, 1);
    mbar_init(&bar->stall, 1);
    fence_mbar_init();
  }
  __syncthreads();
  const uint32_t tmem = bar->tmem;
  auto wait = [&](uint64_t* m, uint32_t parity) {
    if (mbar_wait(m, parity, t.limit)) return true;
    atomicExch(t.status, kStatusTimeout);
    return false;
  };

  if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  if (warp == 8) {
    if (lane == 0 && nmax > 0) {
      bool ok = !t.stall || wait(&bar->stall, 0);
      int issued = 0;
      if (ok) {
        for (int x = 0; x < 2; ++x) {
          if (n[x] == 0) continue;
          mbar_arrive_expect_tx(&bar->q[x], C::kTileBytes);
          for (int c = 0; c < D / 64; ++c)
            tma_load_3d(sQ + x * C::kTileBytes + c * kTile * 128, &mq, &bar->q[x], c * 64, h,
                        static_cast<int>(q0 + row0 + x * kTile));
        }
        for (int i = 0; i < 2 * nmax; ++i) {  // K0 V0 K1 V1 ...
          const int st = i % C::kStages;
          if (i >= C::kStages && !(ok = wait(&bar->empty[st], (i / C::kStages - 1) & 1))) break;
          mbar_arrive_expect_tx(&bar->full[st], C::kTileBytes);
          uint8_t* dst = ring + st * C::kTileBytes;
          const CUtensorMap* m = (i & 1) ? &mv : &mk;
          for (int c = 0; c < D / 64; ++c)
            tma_load_3d(dst + c * kTile * 128, m, &bar->full[st], c * 64, hk,
                        static_cast<int>(k0 + (i >> 1) * kTile));
          issued = i + 1;
        }
        // every copy has landed before the CTA may end
        for (int x = 0; x < 2; ++x)
          if (n[x] > 0) wait(&bar->q[x], 0);
        for (int i = max(0, issued - C::kStages); i < issued; ++i)
          wait(&bar->full[i % C::kStages], (i / C::kStages) & 1);
      }
    }
  } else if (warp == 9) {
    if (lane == 0 && nmax > 0) {
      constexpr uint32_t id_s = idesc_bf16(kTile, kTile), id_o = idesc_bf16(kTile, D, false, true);
      auto scores = [&](int x, int st) {
        const uint32_t qa = smem_u32(sQ + x * C::kTileBytes), kb = smem_u32(ring + st * C::kTileBytes);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          umma_bf16(tmem + C::kColS + x * kTile, kdesc<kTile>(qa, ks), kdesc<kTile>(kb, ks), id_s, ks > 0);
        umma_commit(&bar->s[x]);
      };
      auto values = [&](int x, int st, bool acc) {
        const uint32_t vb = smem_u32(ring + st * C::kTileBytes);
#pragma unroll
        for (int ks = 0; ks < kTile / 16; ++ks) {
          const uint64_t vd = D == 64 ? sdesc_mn128(vb + ks * 2048) : sdesc_mn128_wide(vb + ks * 2048, kTile * 128);
          umma_ts(tmem + C::kColO + x * D, tmem + C::kColS + x * kTile + ks * 8, vd, id_o, acc || ks > 0);
        }
      };
      bool ok = wait(&bar->full[0], 0);
      for (int x = 0; x < 2 && ok; ++x) {
        if (n[x] == 0) continue;
        ok = wait(&bar->q[x], 0);
        if (ok) scores(x, 0);
      }
      if (ok) umma_commit(&bar->empty[0]);
      for (int j = 0; j < nmax && ok; ++j) {
        const int iv = 2 * j + 1, ik = 2 * j + 2, sv = iv % C::kStages, sk = ik % C::kStages;
        ok = wait(&bar->full[sv], (iv / C::kStages) & 1);
        if (ok && j + 1 < nmax) ok = wait(&bar->full[sk], (ik / C::kStages) & 1);
        for (int x = 0; x < 2 && ok; ++x) {
          if (j >= n[x]) continue;
          ok = wait(&bar->p[x], j & 1);
          if (!ok) break;
          tc_fence_after();
          values(x, sv, j > 0);
          if (j + 1 < n[x]) scores(x, sk);
          else umma_commit(&bar->s[x]);  // O is complete
        }
        if (ok) {
          umma_commit(&bar->empty[sv]);
          if (j + 1 < nmax) umma_commit(&bar->empty[sk]);
        }
      }
      umma_commit(&bar->drain);  // products in flight end before the memory is freed
      wait(&bar->drain, 0);
    }
    __syncwarp();
  } else if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int x = warp >> 2, quad = warp & 3, r = quad * 32 + lane, row = row0 + x * kTile + r;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t ts = tmem + C::kColS + x * kTile + lanes, to = tmem + C::kColO + x * D + lanes;
    const float sl2 = a.scale * kLog2e;
    const int seen = row + off + 1;  // keys that this row sees (before lk)
    float m = -INFINITY, l = 0.f;    // reference (raw scores) and sum
    bool ok = true;
    for (int j = 0; j < n[x]; ++j) {
      if (!(ok = wait(&bar->s[x], j & 1))) break;
      tc_fence_after();
      float s[kTile];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t u[32];
        tmem_ld32(ts + c * 32, u);
#pragma unroll
        for (int i = 0; i < 32; ++i) s[c * 32 + i] = __uint_as_float(u[i]);
      }
      tmem_wait_ld();
      const int lim = min(seen, lk) - j * kTile;  // the row's keys in this tile
      if (j * kTile + kTile > min(row0 + x * kTile + off + 1, lk)) {  // some row of the tile sees less
#pragma unroll
        for (int i = 0; i < kTile; ++i)
          if (i >= lim) s[i] = -INFINITY;
      }
      float top = fmaxf(s[0], s[1]);
#pragma unroll
      for (int i = 2; i < kTile; i += 2) top = fmaxf(top, fmaxf(s[i], s[i + 1]));
      if (__any_sync(0xffffffffu, (top - m) * sl2 > kSlack || (m == -INFINITY && top > -INFINITY))) {
        const float mn = fmaxf(m, top);
        const float f = mn == -INFINITY ? 1.f : ex2((m - mn) * sl2);
        m = mn;
        l *= f;
        if (j > 0) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t u[32];
            tmem_ld32(to + c * 32, u);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(__uint_as_float(u[i]) * f);
            tmem_st32(to + c * 32, u);
          }
        }
      }
      const float ref = m == -INFINITY ? 0.f : m * sl2;
      float l4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t u[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float p0 = ex2(fmaf(s[c * 64 + 2 * i], sl2, -ref)), p1 = ex2(fmaf(s[c * 64 + 2 * i + 1], sl2, -ref));
          l4[(2 * i) & 3] += p0;
          l4[(2 * i + 1) & 3] += p1;
          u[i] = pack_bf16(p0, p1);
        }
        tmem_st32(ts + c * 32, u);
      }
      l += (l4[0] + l4[1]) + (l4[2] + l4[3]);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&bar->p[x]);
    }
    if (ok && row0 + x * kTile < lq) {  // some row of this tile is the call's
      if (n[x] > 0) ok = wait(&bar->s[x], n[x] & 1);
      if (ok) {
        tc_fence_after();
        const bool live = row < lq;
        const int64_t g = q0 + row;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.o.p) + g * a.o.stride + h * D;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        bool bad = false;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t u[32];
          if (n[x] > 0) {
            tmem_ld32(to + c * 32, u);
            tmem_wait_ld();
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              y[e] = l == 0.f ? 0.f : __uint_as_float(u[8 * i + e]) * inv;
              bad |= n[x] > 0 && !(fabsf(__uint_as_float(u[8 * i + e])) <= 3.402823466e38f);
            }
            if (live) {
              if (a.o.vec) store8<true>(out + c * 32 + i * 8, y);
              else store8<false>(out + c * 32 + i * 8, y);
            }
          }
        }
        bad |= !(l <= 3.402823466e38f);
        if (live && a.lse) a.lse[g * a.Hq + h] = l == 0.f ? -INFINITY : m * a.scale + logf(l);
        // rows that are not finite, once more from the definition
        for (uint32_t again = __ballot_sync(0xffffffffu, live && bad); again; again &= again - 1) {
          const int rr = __ffs(again) - 1, i = row0 + x * kTile + quad * 32 + rr;
          const int64_t gi = q0 + i;
          const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q.p) + gi * a.q.stride + h * D;
          const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(a.k.p) + k0 * a.k.stride + hk * D;
          const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v.p) + k0 * a.v.stride + hk * D;
          float y[4], z;
          attention_row(q, k, a.k.stride, v, a.v.stride, min(i + off + 1, lk), D, a.scale, y, &z);
          __nv_bfloat16* oi = static_cast<__nv_bfloat16*>(a.o.p) + gi * a.o.stride + h * D;
#pragma unroll
          for (int e = 0; e < D / 32; ++e) oi[lane + 32 * e] = __float2bfloat16_rn(y[e]);
          if (a.lse && lane == 0) a.lse[gi * a.Hq + h] = z;
        }
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// [tokens, H, D] bf16 rows, boxes of 64 columns x 128 tokens
bool make_rows_map(CUtensorMap* m, const RowsIn& r, int64_t tokens, int H, int D) {
  EncodeFn enc = get_encode();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)tokens};
  cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)r.stride * 2};
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
  t.qblocks = (a.max_q + 2 * kTile - 1) / (2 * kTile);
  t.status = static_cast<uint32_t*>(a.ws);
  t.limit = wait_limit_ns();
  t.stall = take_test_stall() ? 1 : 0;
  const int64_t n = static_cast<int64_t>(t.qblocks) * a.B * a.Hq;
  if (n > INT32_MAX) return FALCON_ERR_UNSUPPORTED;
  CUtensorMap mq, mk, mv;
  if (!make_rows_map(&mq, a.q, a.tokens, a.Hq, D) || !make_rows_map(&mk, a.k, a.k_tokens, a.Hkv, D) ||
      !make_rows_map(&mv, a.v, a.k_tokens, a.Hkv, D))
    return FALCON_ERR_CUDA;
  const auto kern = attn_prompt_tc_kernel<D>;
  if (!set_smem_limit(reinterpret_cast<const void*>(kern), Cfg<D>::kSmem)) return FALCON_ERR_CUDA;
  kern<<<static_cast<unsigned>(n), kThreads, Cfg<D>::kSmem, s>>>(mq, mk, mv, t);
  return cudaGetLastError() == cudaSuccess ? FALCON_OK : FALCON_ERR_CUDA;
}

}  // namespace

// The tensor-core kernel takes bf16 rows of 64 or 128 dims on 16-byte
// boundaries (its TMA copies), with token strides below the maps' 2^40 bytes.
bool attn_prompt_tc_supported(const PromptArgs& a, int dtype) {
  if (dtype != FALCON_BF16 || (a.d != 64 && a.d != 128) || a.k_tokens == 0) return false;
  if (!a.q.vec || !a.k.vec || !a.v.vec || a.tokens > INT32_MAX || a.k_tokens > INT32_MAX) return false;
  for (int64_t st : {a.q.stride, a.k.stride, a.v.stride})
    if (st * 2 >= (int64_t(1) << 40)) return false;
  return true;
}
int launch_attn_prompt_tc(const PromptArgs& a, cudaStream_t s) {
  return a.d == 64 ? launch_tc<64>(a, s) : launch_tc<128>(a, s);
}

}  // namespace falcon
