// C ABI of the softmax-attention operators: argument checks on the host and
// dispatch to the kernels.  Nothing here allocates device memory.

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <utility>

#include "attn.cuh"

using namespace falcon;

namespace {

size_t esize(const falcon_attn_params_t* p) { return p->dtype == FALCON_BF16 ? 2 : 4; }

// Rows of a sequence: the kernels' 32-bit row and key numbers, rounded up to
// whole tiles, have to stay below 2^31.
constexpr int64_t kMostRows = INT32_MAX - 1024;

bool misaligned(const void* x, size_t n) { return (reinterpret_cast<uintptr_t>(x) & (n - 1)) != 0; }

// a row stride: 0 (dense) or at least the row's H * d elements
bool stride_ok(int64_t s, int H, int d) { return s == 0 || s >= static_cast<int64_t>(H) * d; }
int64_t stride_of(int64_t s, int H, int d) { return s ? s : static_cast<int64_t>(H) * d; }

bool vec_rows(const falcon_attn_params_t* p, const void* x, int64_t stride) {
  return !misaligned(x, 16) && (stride * esize(p)) % 16 == 0;
}
RowsIn rows_in(const falcon_attn_params_t* p, const void* x, int64_t s, int H) {
  const int64_t st = stride_of(s, H, p->d);
  return RowsIn{x, st, vec_rows(p, x, st)};
}
RowsOut rows_out(const falcon_attn_params_t* p, void* x, int64_t s, int H) {
  const int64_t st = stride_of(s, H, p->d);
  return RowsOut{x, st, vec_rows(p, x, st)};
}
// bytes from the first to past the last element of n rows
size_t span(const falcon_attn_params_t* p, int64_t n, int64_t s, int H) {
  const int64_t row = static_cast<int64_t>(H) * p->d;
  return n <= 0 ? 0 : static_cast<size_t>((n - 1) * stride_of(s, H, p->d) + row) * esize(p);
}
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const auto pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
  return pa < pb + nb && pb < pa + na;
}

// Whether rows of a and rows of b share a byte: n rows each, of ra and rb bytes, sa and sb apart.  With one stride (slices
// of a fused projection) the rows of one lie between those of the other; with two the spans are compared.
bool rows_overlap(const void* a, int64_t sa, size_t ra, const void* b, int64_t sb, size_t rb, int64_t n) {
  if (!a || !b || n <= 0) return false;
  if (!overlap(a, (n - 1) * sa + ra, b, (n - 1) * sb + rb)) return false;
  if (sa != sb || n == 1) return true;
  const auto pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
  const size_t s = static_cast<size_t>(sa), off = pb >= pa ? (pb - pa) % s : (s - (pa - pb) % s) % s;
  return off < ra || s - off < rb;  // from a row of a to the next row of b, and from there to the next of a
}
bool rows_overlap(const falcon_attn_params_t* p, const void* a, int64_t sa, int Ha, const void* b, int64_t sb, int Hb,
                  int64_t n) {
  const int64_t e = static_cast<int64_t>(esize(p));
  return rows_overlap(a, stride_of(sa, Ha, p->d) * e, Ha * p->d * e, b, stride_of(sb, Hb, p->d) * e, Hb * p->d * e, n);
}

int check_attn(const falcon_attn_params_t* p) {
  if (!p) return FALCON_ERR_INVALID_ARG;
  if (p->Hq < 1 || p->Hkv < 1 || p->Hq % p->Hkv) return FALCON_ERR_INVALID_ARG;
  if (p->dtype != FALCON_BF16 && p->dtype != FALCON_F32) return FALCON_ERR_INVALID_ARG;
  if (p->d != 16 && p->d != 32 && p->d != 64 && p->d != 128) return FALCON_ERR_UNSUPPORTED;
  // offsets within a token are 32-bit
  if ((static_cast<int64_t>(p->Hq) + p->Hkv) * p->d > INT32_MAX) return FALCON_ERR_UNSUPPORTED;
  if (p->tokens < 0 || p->k_tokens < 0 || p->max_q < 0 || p->max_k < 0) return FALCON_ERR_INVALID_ARG;
  if (!stride_ok(p->q_stride, p->Hq, p->d) || !stride_ok(p->k_stride, p->Hkv, p->d) ||
      !stride_ok(p->v_stride, p->Hkv, p->d) || !stride_ok(p->o_stride, p->Hq, p->d))
    return FALCON_ERR_INVALID_ARG;
  return FALCON_OK;
}
int check_scale(const falcon_attn_params_t* p) {
  return std::isfinite(p->scale) && p->scale >= 0.f ? FALCON_OK : FALCON_ERR_INVALID_ARG;
}
// most rows that one sequence brings: no more than the call has
int64_t most_rows(const falcon_attn_params_t* p) { return std::min<int64_t>(p->max_q, p->tokens); }
// most keys that one sequence has in the cache
int64_t most_keys(const falcon_attn_params_t* p) {
  return std::min<int64_t>(p->max_k, static_cast<int64_t>(p->max_pages) * p->page);
}
float scale_of(const falcon_attn_params_t* p) {
  return p->scale > 0.f ? p->scale : 1.f / std::sqrt(static_cast<float>(p->d));
}
// norm and rotation settings, with the table that they need
int check_head(const falcon_attn_params_t* p, const float* table, const float* w_q, const float* w_k) {
  if (p->qk_norm && !(p->norm_eps > 0.f && std::isfinite(p->norm_eps))) return FALCON_ERR_INVALID_ARG;
  if (p->rot < 0 || p->rot > p->d || (p->rot & 1)) return FALCON_ERR_INVALID_ARG;
  if (p->rope_layout != FALCON_ROPE_HALF && p->rope_layout != FALCON_ROPE_INTERLEAVED) return FALCON_ERR_INVALID_ARG;
  if (p->rot > 0 && (!table || p->rope_rows < 1 || misaligned(table, 8))) return FALCON_ERR_INVALID_ARG;
  if (p->qk_norm && (misaligned(w_q, 4) || misaligned(w_k, 4))) return FALCON_ERR_INVALID_ARG;
  return FALCON_OK;
}
HeadArgs head_args(const falcon_attn_params_t* p, const float* table, const float* w_q, const float* w_k) {
  const bool wide = !misaligned(table, 16) && !misaligned(w_q, 16) && !misaligned(w_k, 16) && p->rot % 4 == 0;
  return HeadArgs{p->d, p->qk_norm ? 1 : 0, p->norm_eps, 1.f / static_cast<float>(p->d), p->rot, p->rope_layout, p->rope_rows,
                  reinterpret_cast<const float2*>(table), wide};
}
// the cache's four buffers and their bytes
struct CacheParts {
  const void* p[4];
  size_t n[4];
};
CacheParts cache_parts(const falcon_attn_params_t* p, const falcon_kv_cache_t* c) {
  const size_t scales = static_cast<size_t>(p->num_pages) * p->Hkv, codes = scales * p->page * p->d;
  return CacheParts{{c->k, c->v, c->k_scale, c->v_scale}, {codes, codes, scales, scales}};
}
int check_cache(const falcon_attn_params_t* p, const falcon_kv_cache_t* c, const int32_t* blocks) {
  if (p->page != 16 && p->page != 32 && p->page != 64 && p->page != 128) return FALCON_ERR_UNSUPPORTED;
  if (p->B < 1 || p->num_pages < 1 || p->max_pages < 0) return FALCON_ERR_INVALID_ARG;
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale) return FALCON_ERR_INVALID_ARG;
  if (misaligned(c->k, 16) || misaligned(c->v, 16)) return FALCON_ERR_INVALID_ARG;
  if (p->max_pages > 0 && (!blocks || misaligned(blocks, 4))) return FALCON_ERR_INVALID_ARG;
  return FALCON_OK;
}

}  // namespace

extern "C" {

int falcon_rope_table(const double* inv_freq, int32_t rot, int32_t rows, float mscale, float* table, void* stream) {
  if (rot < 0 || (rot & 1) || rows < 0 || !std::isfinite(mscale)) return FALCON_ERR_INVALID_ARG;
  if (rot > 0 && rows > 0 && (!inv_freq || !table || misaligned(inv_freq, 8) || misaligned(table, 8)))
    return FALCON_ERR_INVALID_ARG;
  return launch_rope_table(inv_freq, rot, rows, mscale, table, reinterpret_cast<cudaStream_t>(stream));
}

int falcon_qk_norm_rope(const falcon_attn_params_t* p, const void* q, const void* k, const float* w_q,
                        const float* w_k, const int64_t* positions, const float* table, void* q_out, void* k_out,
                        void* stream) {
  int st = check_attn(p);
  if (st == FALCON_OK) st = check_head(p, table, w_q, w_k);
  if (st != FALCON_OK) return st;
  if (p->tokens == 0) return FALCON_OK;
  if ((!q && !k) || (q && !q_out) || (k && !k_out)) return FALCON_ERR_INVALID_ARG;
  if (p->rot > 0 && (!positions || misaligned(positions, 8))) return FALCON_ERR_INVALID_ARG;
  for (const void* x : {q, k, static_cast<const void*>(q_out), static_cast<const void*>(k_out)})
    if (misaligned(x, esize(p))) return FALCON_ERR_INVALID_ARG;
  const RowsIn qi = rows_in(p, q, p->q_stride, p->Hq), ki = rows_in(p, k, p->k_stride, p->Hkv);
  const RowsOut qo = rows_out(p, q_out, p->o_stride, p->Hq), ko = rows_out(p, k_out, 0, p->Hkv);
  const bool q_inplace = q == q_out && qi.stride == qo.stride, k_inplace = k == k_out && ki.stride == ko.stride;
  auto meet = [&](const void* x, int64_t sx, int Hx, const void* y, int64_t sy, int Hy) {
    return rows_overlap(p, x, sx, Hx, y, sy, Hy, p->tokens);
  };
  const void *xq = q ? q_out : nullptr, *xk = k ? k_out : nullptr;
  if ((!q_inplace && meet(q, p->q_stride, p->Hq, xq, p->o_stride, p->Hq)) ||
      (!k_inplace && meet(k, p->k_stride, p->Hkv, xk, 0, p->Hkv)) ||
      meet(k, p->k_stride, p->Hkv, xq, p->o_stride, p->Hq) || meet(q, p->q_stride, p->Hq, xk, 0, p->Hkv) ||
      meet(xq, p->o_stride, p->Hq, xk, 0, p->Hkv))
    return FALCON_ERR_INVALID_ARG;
  return launch_qk_norm_rope(head_args(p, table, w_q, w_k), p->dtype, p->tokens, p->Hq, p->Hkv, qi, ki, w_q, w_k, positions, qo,
                             ko, reinterpret_cast<cudaStream_t>(stream));
}

int falcon_kv_append(const falcon_attn_params_t* p, const void* k, const void* v, const float* w_k,
                     const float* table, const int32_t* cu_new, const int32_t* ctx_lens, const int32_t* block_table,
                     const falcon_kv_cache_t* cache, void* stream) {
  int st = check_attn(p);
  if (st == FALCON_OK) st = check_head(p, table, nullptr, w_k);
  if (st == FALCON_OK) st = check_cache(p, cache, block_table);
  if (st != FALCON_OK) return st;
  if (p->tokens == 0 || p->max_q == 0 || p->max_pages == 0) return FALCON_OK;
  if (most_rows(p) > kMostRows) return FALCON_ERR_UNSUPPORTED;
  if (!k || !v || !cu_new || !ctx_lens) return FALCON_ERR_INVALID_ARG;
  if (misaligned(k, esize(p)) || misaligned(v, esize(p)) || misaligned(cu_new, 4) || misaligned(ctx_lens, 4))
    return FALCON_ERR_INVALID_ARG;
  const CacheParts c = cache_parts(p, cache);
  const void* const* outs = c.p;
  const size_t* nout = c.n;
  const void* ins[2] = {k, v};
  const size_t nin[2] = {span(p, p->tokens, p->k_stride, p->Hkv), span(p, p->tokens, p->v_stride, p->Hkv)};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 2; ++j)
      if (overlap(outs[i], nout[i], ins[j], nin[j])) return FALCON_ERR_INVALID_ARG;
    for (int j = i + 1; j < 4; ++j)
      if (overlap(outs[i], nout[i], outs[j], nout[j])) return FALCON_ERR_INVALID_ARG;
  }
  const AppendArgs a{p->B, p->Hkv, p->page, p->num_pages, p->max_pages, static_cast<int>(most_rows(p)), p->tokens,
                     rows_in(p, k, p->k_stride, p->Hkv), rows_in(p, v, p->v_stride, p->Hkv), w_k, cu_new, ctx_lens,
                     block_table, *cache};
  return launch_kv_append(head_args(p, table, nullptr, w_k), p->dtype, a, reinterpret_cast<cudaStream_t>(stream));
}

size_t falcon_attn_decode_workspace_size(const falcon_attn_params_t* p) {
  if (check_attn(p) != FALCON_OK || p->B < 1) return 0;
  if (p->page != 16 && p->page != 32 && p->page != 64 && p->page != 128) return 0;
  return align_up(attn_decode_ws_bytes(p->B, p->Hq, p->Hkv, p->d, static_cast<int>(esize(p)), p->max_k), 256);
}

int falcon_attn_decode(const falcon_attn_params_t* p, const void* q, const falcon_kv_cache_t* cache,
                       const int32_t* block_table, const int32_t* lens, void* o, float* lse, void* workspace,
                       size_t workspace_bytes, void* stream) {
  int st = check_attn(p);
  if (st == FALCON_OK) st = check_scale(p);
  if (st == FALCON_OK) st = check_cache(p, cache, block_table);
  if (st != FALCON_OK) return st;
  // the kernel counts the batch's units of at least 64 keys in 32 bits too
  if (most_keys(p) > kMostRows || p->B * ((most_keys(p) + 63) / 64) > INT32_MAX) return FALCON_ERR_UNSUPPORTED;
  if (!q || !o || !lens || misaligned(q, esize(p)) || misaligned(o, esize(p)) || misaligned(lens, 4) ||
      misaligned(lse, 4))
    return FALCON_ERR_INVALID_ARG;
  const size_t no = span(p, p->B, p->o_stride, p->Hq), nl = lse ? static_cast<size_t>(p->B) * p->Hq * 4 : 0;
  if (rows_overlap(p, q, p->q_stride, p->Hq, o, p->o_stride, p->Hq, p->B) || overlap(o, no, lse, nl)) return FALCON_ERR_INVALID_ARG;
  const size_t need = falcon_attn_decode_workspace_size(p), nq = span(p, p->B, p->q_stride, p->Hq);
  const CacheParts c = cache_parts(p, cache);
  for (int i = 0; i < 4; ++i)
    if (overlap(o, no, c.p[i], c.n[i]) || overlap(lse, nl, c.p[i], c.n[i]) || overlap(workspace, need, c.p[i], c.n[i]))
      return FALCON_ERR_INVALID_ARG;
  if (overlap(q, nq, lse, nl)) return FALCON_ERR_INVALID_ARG;
  for (const auto& x : {std::make_pair(q, nq), std::make_pair(static_cast<const void*>(o), no),
                        std::make_pair(static_cast<const void*>(lse), nl)})
    if (overlap(workspace, need, x.first, x.second)) return FALCON_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < need || misaligned(workspace, 256)) return FALCON_ERR_WORKSPACE;
  const DecodeArgs a{p->B, p->Hq, p->Hkv, p->d, p->page, p->num_pages, p->max_pages, p->max_k, scale_of(p),
                     rows_in(p, q, p->q_stride, p->Hq), rows_out(p, o, p->o_stride, p->Hq), lse, block_table, lens,
                     *cache, workspace};
  return launch_attn_decode(a, p->dtype, reinterpret_cast<cudaStream_t>(stream));
}

size_t falcon_attn_prompt_workspace_size(const falcon_attn_params_t* p) {
  if (check_attn(p) != FALCON_OK || p->B < 1) return 0;
  return 256;
}

int falcon_attn_prompt(const falcon_attn_params_t* p, const void* q, const void* k, const void* v,
                       const int32_t* cu_q, const int32_t* cu_k, void* o, float* lse, void* workspace,
                       size_t workspace_bytes, void* stream) {
  int st = check_attn(p);
  if (st == FALCON_OK) st = check_scale(p);
  if (st != FALCON_OK) return st;
  if (p->B < 1) return FALCON_ERR_INVALID_ARG;
  if (p->tokens == 0 || p->max_q == 0) return FALCON_OK;
  if (most_rows(p) > kMostRows || p->k_tokens > kMostRows) return FALCON_ERR_UNSUPPORTED;
  if (!q || !o || !cu_q || !cu_k || (p->k_tokens > 0 && (!k || !v))) return FALCON_ERR_INVALID_ARG;
  for (const void* x : {q, k, v, static_cast<const void*>(o)})
    if (misaligned(x, esize(p))) return FALCON_ERR_INVALID_ARG;
  if (misaligned(cu_q, 4) || misaligned(cu_k, 4) || misaligned(lse, 4)) return FALCON_ERR_INVALID_ARG;
  const size_t no = span(p, p->tokens, p->o_stride, p->Hq), nl = lse ? static_cast<size_t>(p->tokens) * p->Hq * 4 : 0;
  const void* ins[3] = {q, k, v};
  const size_t nin[3] = {span(p, p->tokens, p->q_stride, p->Hq), span(p, p->k_tokens, p->k_stride, p->Hkv),
                         span(p, p->k_tokens, p->v_stride, p->Hkv)};
  for (int i = 0; i < 3; ++i)
    if (overlap(ins[i], nin[i], lse, nl)) return FALCON_ERR_INVALID_ARG;
  // o between the rows of a fused projection; k and v may have rows of their own number
  const bool one = p->k_tokens == p->tokens;
  if (rows_overlap(p, q, p->q_stride, p->Hq, o, p->o_stride, p->Hq, p->tokens) ||
      (one ? rows_overlap(p, k, p->k_stride, p->Hkv, o, p->o_stride, p->Hq, p->tokens) ||
                 rows_overlap(p, v, p->v_stride, p->Hkv, o, p->o_stride, p->Hq, p->tokens)
           : overlap(ins[1], nin[1], o, no) || overlap(ins[2], nin[2], o, no)))
    return FALCON_ERR_INVALID_ARG;
  if (overlap(o, no, lse, nl)) return FALCON_ERR_INVALID_ARG;
  const size_t need = falcon_attn_prompt_workspace_size(p);
  for (int i = 0; i < 3; ++i)
    if (overlap(workspace, need, ins[i], nin[i])) return FALCON_ERR_INVALID_ARG;
  if (overlap(workspace, need, o, no) || overlap(workspace, need, lse, nl)) return FALCON_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < need || misaligned(workspace, 256))
    return FALCON_ERR_WORKSPACE;
  const PromptArgs a{p->B, p->Hq, p->Hkv, p->d, static_cast<int>(most_rows(p)), scale_of(p), p->tokens, p->k_tokens,
                     rows_in(p, q, p->q_stride, p->Hq), rows_in(p, k, p->k_stride, p->Hkv),
                     rows_in(p, v, p->v_stride, p->Hkv), rows_out(p, o, p->o_stride, p->Hq), lse, cu_q, cu_k,
                     workspace};
  return launch_attn_prompt(a, p->dtype, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
