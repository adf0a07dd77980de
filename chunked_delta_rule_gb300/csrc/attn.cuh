// Internals shared by the softmax-attention operators: resolved arguments,
// e4m3 / e8m0 conversions and the per-head norm and rotation of a row piece.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace falcon {

// Rows of one of q, k, v, o: pointer, elements from token to token, and
// whether every row starts on a 16-byte boundary.
struct RowsIn {
  const void* p;
  int64_t stride;
  bool vec;
};
struct RowsOut {
  void* p;
  int64_t stride;
  bool vec;
};

// How the rows of a head are normed and rotated.
struct HeadArgs {
  int d, norm;
  float eps, inv_d;
  int rot, layout, rows;
  const float2* table;
  bool wide;  // table rows and weights on 16-byte boundaries
};
// How a kernel rotates: not at all, lanes that hold whole pairs of the half or
// the interleaved layout (16-byte loads of the table), or any pairs.
enum RotMode { kRotNone = 0, kRotHalf = 1, kRotInterleaved = 2, kRotAny = 3 };
inline RotMode rot_mode(const HeadArgs& h) {
  if (h.rot == 0) return kRotNone;
  if (h.layout == FALCON_ROPE_HALF) return h.wide && h.rot % 8 == 0 ? kRotHalf : kRotAny;
  return h.wide && h.rot % 8 == 0 ? kRotInterleaved : kRotAny;
}

int launch_rope_table(const double* inv_freq, int rot, int rows, float mscale, float* table, cudaStream_t s);
int launch_qk_norm_rope(const HeadArgs& h, int dtype, int64_t tokens, int Hq, int Hkv, RowsIn q, RowsIn k,
                        const float* w_q, const float* w_k, const int64_t* pos, RowsOut qo, RowsOut ko,
                        cudaStream_t s);

// The gradient of the norm and rotation; [0] the queries, [1] the keys (H = 0: none).
struct NormGradArgs {
  HeadArgs h;
  int64_t tokens;
  int H[2];
  RowsIn x[2], dy[2];  // x is read with the norm only
  RowsOut dx[2];
  const float* w[2];
  float* dw[2];        // NULL: not wanted
  const int64_t* pos;
  float* partial;      // workspace: [CTAs][2][d]
};
size_t norm_grad_ws_bytes(int d);
int launch_qk_norm_rope_backward(const NormGradArgs& a, int dtype, cudaStream_t s);

struct AppendArgs {
  int B, Hkv, page, num_pages, max_pages, max_q;
  int64_t tokens;
  RowsIn k, v;
  const float* w_k;
  const int32_t* cu;
  const int32_t* ctx;
  const int32_t* blocks;
  falcon_kv_cache_t cache;
};
int launch_kv_append(const HeadArgs& h, int dtype, const AppendArgs& a, cudaStream_t s);

struct DecodeArgs {
  int B, Hq, Hkv, d, page, num_pages, max_pages, max_k;
  float scale;
  RowsIn q;
  RowsOut o;
  float* lse;
  const int32_t* blocks;
  const int32_t* lens;
  falcon_kv_cache_t cache;
  void* ws;
};
size_t attn_decode_ws_bytes(int B, int Hq, int Hkv, int d, int elem, int max_k);
int launch_attn_decode(const DecodeArgs& a, int dtype, cudaStream_t s);

struct PromptArgs {
  int B, Hq, Hkv, d, max_q;
  float scale;
  int64_t tokens, k_tokens;
  RowsIn q, k, v;
  RowsOut o;
  float* lse;
  const int32_t* cu_q;
  const int32_t* cu_k;
  void* ws;
};
int launch_attn_prompt(const PromptArgs& a, int dtype, cudaStream_t s);
bool attn_prompt_tc_supported(const PromptArgs& a, int dtype);
int launch_attn_prompt_tc(const PromptArgs& a, cudaStream_t s);

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// 2^x
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---------------------------------------------------------------- rows
// A lane's 8 elements of a head row: two pieces of 4, at a and b.  They are
// neighbours (b = a + 4), or with the half layout (SPLIT) the two members of
// the lane's four pairs.
struct Pieces {
  int a, b;
};
template <typename T> struct Raw8;  // as loaded
template <> struct Raw8<__nv_bfloat16> { uint2 a, b; };
template <> struct Raw8<float> { float4 a, b; };

template <bool VEC, bool SPLIT>
__device__ __forceinline__ Raw8<__nv_bfloat16> load8(const __nv_bfloat16* row, Pieces at) {
  Raw8<__nv_bfloat16> r;
  if (VEC && !SPLIT) {
    const uint4 v = *reinterpret_cast<const uint4*>(row + at.a);
    r.a = make_uint2(v.x, v.y);
    r.b = make_uint2(v.z, v.w);
  } else if (VEC) {
    r.a = *reinterpret_cast<const uint2*>(row + at.a);
    r.b = *reinterpret_cast<const uint2*>(row + at.b);
  } else {
    const unsigned short* u = reinterpret_cast<const unsigned short*>(row + at.a);
    const unsigned short* v = reinterpret_cast<const unsigned short*>(row + at.b);
    r.a = make_uint2(u[0] | (static_cast<uint32_t>(u[1]) << 16), u[2] | (static_cast<uint32_t>(u[3]) << 16));
    r.b = make_uint2(v[0] | (static_cast<uint32_t>(v[1]) << 16), v[2] | (static_cast<uint32_t>(v[3]) << 16));
  }
  return r;
}
template <bool VEC, bool SPLIT>
__device__ __forceinline__ Raw8<float> load8(const float* row, Pieces at) {
  Raw8<float> r;
  if (VEC) {
    r.a = *reinterpret_cast<const float4*>(row + at.a);
    r.b = *reinterpret_cast<const float4*>(row + at.b);
  } else {
    const float *u = row + at.a, *v = row + at.b;
    r.a = make_float4(u[0], u[1], u[2], u[3]);
    r.b = make_float4(v[0], v[1], v[2], v[3]);
  }
  return r;
}
__device__ __forceinline__ void unpack8(const Raw8<__nv_bfloat16>& r, float (&x)[8]) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.b.x, r.b.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void unpack8(const Raw8<float>& r, float (&x)[8]) {
  x[0] = r.a.x; x[1] = r.a.y; x[2] = r.a.z; x[3] = r.a.w;
  x[4] = r.b.x; x[5] = r.b.y; x[6] = r.b.z; x[7] = r.b.w;
}
template <bool VEC, bool SPLIT>
__device__ __forceinline__ void store8(__nv_bfloat16* row, Pieces at, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<uint32_t*>(&v);
  }
  if (VEC && !SPLIT) {
    *reinterpret_cast<uint4*>(row + at.a) = make_uint4(w[0], w[1], w[2], w[3]);
  } else if (VEC) {
    *reinterpret_cast<uint2*>(row + at.a) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2*>(row + at.b) = make_uint2(w[2], w[3]);
  } else {
    unsigned short* u = reinterpret_cast<unsigned short*>(row + at.a);
    unsigned short* v = reinterpret_cast<unsigned short*>(row + at.b);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      u[2 * i] = static_cast<unsigned short>(w[i]);
      u[2 * i + 1] = static_cast<unsigned short>(w[i] >> 16);
      v[2 * i] = static_cast<unsigned short>(w[2 + i]);
      v[2 * i + 1] = static_cast<unsigned short>(w[2 + i] >> 16);
    }
  }
}
template <bool VEC, bool SPLIT>
__device__ __forceinline__ void store8(float* row, Pieces at, const float (&x)[8]) {
  if (VEC) {
    *reinterpret_cast<float4*>(row + at.a) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(row + at.b) = make_float4(x[4], x[5], x[6], x[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) row[at.a + i] = x[i], row[at.b + i] = x[4 + i];
  }
}

// Norm and rotation of a lane's 8 elements of a head row; the d / 8 lanes of
// the row are neighbours in the warp and every lane of the warp takes part
// (lanes without a row pass x = 0).  The pairs are (x[i], x[4 + i]) with the
// half layout and (x[2i], x[2i + 1]) with the interleaved one.
struct HeadPiece {
  float w[8];          // norm weights
  float co[4], si[4];  // angles of the lane's pairs
};
// The pieces of lane li of a row: pairs first, then the dims that are not rotated.
template <int MODE>
__device__ __forceinline__ Pieces pieces_of(const HeadArgs& h, int li) {
  const bool pairs = MODE == kRotHalf && li * 8 < h.rot;
  return pairs ? Pieces{li * 4, (h.rot >> 1) + li * 4} : Pieces{li * 8, li * 8 + 4};
}
__device__ __forceinline__ void load_weights(HeadPiece& hp, const HeadArgs& h, const float* w, Pieces at) {
  if (!h.norm) return;
  if (w && h.wide) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(w + at.a)), b = __ldg(reinterpret_cast<const float4*>(w + at.b));
    hp.w[0] = a.x; hp.w[1] = a.y; hp.w[2] = a.z; hp.w[3] = a.w;
    hp.w[4] = b.x; hp.w[5] = b.y; hp.w[6] = b.z; hp.w[7] = b.w;
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) hp.w[i] = w ? __ldg(w + at.a + i) : 1.f, hp.w[4 + i] = w ? __ldg(w + at.b + i) : 1.f;
}
// The table's row of a position, NULL outside the table.
__device__ __forceinline__ const float2* table_row(const HeadArgs& h, int64_t pos) {
  return pos >= 0 && pos < h.rows ? h.table + pos * (h.rot >> 1) : nullptr;
}
// Angles of this lane's pairs; outside the table they are NaN.
template <int MODE>
__device__ __forceinline__ void load_angles(HeadPiece& hp, const HeadArgs& h, const float2* row, Pieces at) {
  if ((MODE != kRotHalf && MODE != kRotInterleaved) || at.a >= h.rot) return;
  const float4* v = reinterpret_cast<const float4*>((row ? row : h.table) + (MODE == kRotHalf ? at.a : at.a >> 1));
  const float4 a = __ldg(v), b = __ldg(v + 1);
  hp.co[0] = a.x; hp.si[0] = a.y; hp.co[1] = a.z; hp.si[1] = a.w;
  hp.co[2] = b.x; hp.si[2] = b.y; hp.co[3] = b.z; hp.si[3] = b.w;
  if (!row) {
#pragma unroll
    for (int i = 0; i < 4; ++i) hp.co[i] = __int_as_float(0x7fffffff);
  }
}
// raw, w, row: the raw row, its weights and the table's row again (kRotAny: any pairs).
template <int MODE, typename T>
__device__ __forceinline__ void norm_rotate8(float (&x)[8], const HeadPiece& hp, const HeadArgs& h, const float* w,
                                             const float2* row, const T* raw, bool live, Pieces at) {
  float r = 1.f;
  if (h.norm) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(x[i], x[i], s);
    // over the d / 8 lanes: 2, 4, 8 or 16
    s += __shfl_xor_sync(0xffffffffu, s, 1);
    float v = __shfl_xor_sync(0xffffffffu, s, 2);
    s += h.d > 16 ? v : 0.f;
    v = __shfl_xor_sync(0xffffffffu, s, 4);
    s += h.d > 32 ? v : 0.f;
    v = __shfl_xor_sync(0xffffffffu, s, 8);
    s += h.d > 64 ? v : 0.f;
    r = rsqrtf(fmaf(s, h.inv_d, h.eps));
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * r * hp.w[i];
  }
  if constexpr (MODE == kRotHalf || MODE == kRotInterleaved) {
    if (at.a < h.rot) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        constexpr bool kHalf = MODE == kRotHalf;
        float &p = x[kHalf ? i : 2 * i], &q = x[kHalf ? 4 + i : 2 * i + 1];
        const float a = p, b = q;
        p = a * hp.co[i] - b * hp.si[i];
        q = b * hp.co[i] + a * hp.si[i];
      }
    }
  } else if constexpr (MODE == kRotAny) {
    const int half = h.rot >> 1;
    const bool hl = h.layout == FALCON_ROPE_HALF;
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = at.a + i, j = hl ? (c < half ? c : c - half) : c >> 1;  // element, its pair
      const bool low = hl ? c < half : !(c & 1);
      y[i] = x[i];
      if (live && c < h.rot) {
        const int pc = hl ? (low ? c + half : c - half) : c ^ 1;
        float other = to_f32(raw[pc]);
        if (h.norm) other = other * r * (w ? __ldg(w + pc) : 1.f);
        const float2 t = row ? __ldg(row + j) : make_float2(__int_as_float(0x7fffffff), 0.f);
        y[i] = x[i] * t.x + (low ? -t.y : t.y) * other;
      }
    }
    __syncwarp();  // read before any lane writes the row in place
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = y[i];
  }
}

// ---------------------------------------------------------------- 8-bit cache
// 2^e as a float, e in [-149, 127]
__device__ __forceinline__ float exp2i(int e) {
  return e >= -126 ? __int_as_float((e + 127) << 23) : __int_as_float(1 << (e + 149));
}
// value of a scale byte (e8m0)
__device__ __forceinline__ float e8m0(uint32_t byte) {
  return byte ? __uint_as_float(byte << 23) : __uint_as_float(0x00400000u);
}
// smallest e in [-126, 127] with amax <= 448 * 2^e (448 = 0.875 * 2^9)
__device__ __forceinline__ int scale_exponent(float amax) {
  if (!(amax > 0.f)) return -126;
  int x;
  const float m = frexpf(amax, &x);
  const int e = m <= 0.875f ? x - 9 : x - 8;
  return e < -126 ? -126 : e > 127 ? 127 : e;
}
// two floats -> two e4m3 codes (lo in the low byte), nearest even, saturating
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// two e4m3 codes -> packed halves (exact)
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
}

}  // namespace falcon
