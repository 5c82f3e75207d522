// api_serving.cu -- the extern "C" entry points around the decode step
// (declared in include/lkv.h): page plan, rotary tables, norm + rotation +
// append, and attention of one or a few new tokens.  Host-side validation
// and launches; nothing here allocates device memory or synchronizes.
#include <cmath>

#include "api_common.cuh"
#include "multi.cuh"
#include "serving.cuh"

using namespace lkv;

namespace {

bool int_ptr_ok(const void* p, bool needed) { return p == nullptr ? !needed : aligned_to(p, 4); }

struct MultiCall {
  multi::MultiArgs a{};
  multi::MultiPlan p{};
};

// The shape checks of the attention and its launch plan.
int multi_shape(lkv_qspec spec, int B, int Hq, int Hkv, int T_cap, int D, int max_q, MultiCall& c) {
  if (!bits_ok(spec.k_bits) || !bits_ok(spec.v_bits)) return LKV_ERR_UNSUPPORTED;
  const int rc = check_cache_shape(B, Hkv, T_cap, D, spec.group);
  if (rc) return rc;
  if (Hq <= 0 || Hq % Hkv != 0 || max_q < 1) return LKV_ERR_INVALID_ARG;
  if (Hq / Hkv > 64 || max_q > multi::kMaxQueries || B > multi::kMaxBatch || T_cap > (1 << 30)) return LKV_ERR_UNSUPPORTED;
  multi::MultiArgs& a = c.a;
  a.B = B; a.Hq = Hq; a.Hkv = Hkv; a.T_cap = T_cap; a.G = spec.group; a.r = Hq / Hkv; a.max_q = max_q;
  a.kb = spec.k_bits; a.vb = spec.v_bits;
  multi::plan_multi(a, D, c.p);
  // tiles are numbered in 32 bits
  if ((double)B * c.p.units_max * ((double)T_cap / c.p.sh.tt + 2.0) >= 2147483647.0) return LKV_ERR_UNSUPPORTED;
  return LKV_OK;
}

int multi_impl(lkv_qspec spec, int B, int Hq, int Hkv, int T_cap, int D, int max_q, int n_rows, const int32_t* seq_lens,
               const int32_t* cu_q, const void* q, const int32_t* table, int pps, int num_pages, const void* kc,
               const float* ksz, const void* vc, const float* vsz, lkv_score_rule rule, float* out, float* lse,
               void* workspace, size_t ws_bytes, void* stream) {
  MultiCall c;
  int rc = multi_shape(spec, B, Hq, Hkv, T_cap, D, max_q, c);
  if (rc) return rc;
  if (n_rows < 0 || (cu_q == nullptr && n_rows < B)) return LKV_ERR_INVALID_ARG;
  if (!std::isfinite(rule.softmax_scale) || !std::isfinite(rule.softcap) || rule.softcap < 0.0f || rule.window < 0)
    return LKV_ERR_INVALID_ARG;
  // scores are divided by the cap: a smaller one takes them out of fp32
  if (rule.softcap > 0.0f && rule.softcap < 1e-30f) return LKV_ERR_INVALID_ARG;
  // c tanh(x / c) = x (1 - (x / c)^2 / 3 + ...) is x to fp32 for |x| < c 2^-12: above 1e30 a cap only takes x / c out of
  // the normal numbers and c log2(e) to infinity
  if (rule.softcap > 1e30f) rule.softcap = 0.0f;
  // the factor of q . khat; an infinite one would make NaN of a product that is 0
  if (!std::isfinite(rule.softcap > 0.0f ? rule.softmax_scale / rule.softcap : rule.softmax_scale * 1.442695f))
    return LKV_ERR_INVALID_ARG;
  if (!int_ptr_ok(rule.slopes, false) || !int_ptr_ok(rule.prefix_lens, false) || !int_ptr_ok(rule.doc_starts, false) ||
      !int_ptr_ok(cu_q, false) || !int_ptr_ok(lse, false) || !int_ptr_ok(seq_lens, B > 0))
    return LKV_ERR_INVALID_ARG;
  const bool ne = (long long)B * Hkv * T_cap > 0, rows = n_rows > 0;
  if (!ptr_ok(q, rows) || !ptr_ok(out, rows) || !ptr_ok(kc, ne) || !ptr_ok(ksz, ne && spec.k_bits < 16) || !ptr_ok(vc, ne) ||
      !ptr_ok(vsz, ne && spec.v_bits < 16))
    return LKV_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned_to(workspace, kAlign)) return LKV_ERR_INVALID_ARG;
  if (ws_bytes < c.p.ws_total) return LKV_ERR_WORKSPACE;
  if (B == 0 || n_rows == 0) return LKV_OK;
  multi::MultiArgs& a = c.a;
  a.n_rows = n_rows;
  a.lens = seq_lens; a.cu_q = cu_q;
  a.q = static_cast<const uint16_t*>(q);
  a.kc = static_cast<const uint8_t*>(kc); a.ksz = ksz;
  a.vc = static_cast<const uint8_t*>(vc); a.vsz = vsz;
  a.scale = rule.softmax_scale; a.softcap = rule.softcap;
  a.window = rule.window < T_cap ? rule.window : 0;  // a window over the whole capacity hides nothing
  a.slopes = rule.slopes; a.prefix = rule.prefix_lens; a.starts = rule.doc_starts;
  a.out = out; a.lse = lse;
  a.table = table; a.pps = pps; a.num_pages = num_pages;
  char* ws = static_cast<char*>(workspace);
  a.status = reinterpret_cast<int*>(ws);
  a.timeout_ns = reinterpret_cast<const unsigned long long*>(ws + 8);
  a.arrive = reinterpret_cast<int*>(ws + c.p.ws_arrive);
  a.pieces = reinterpret_cast<float*>(ws + c.p.ws_pieces);
  a.cpieces = reinterpret_cast<float*>(ws + c.p.ws_cpieces);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (a.kb) {
    case 2: return from_cuda(multi::launch_multi_k2(a, D, c.p, s));
    case 4: return from_cuda(multi::launch_multi_k4(a, D, c.p, s));
    case 6: return from_cuda(multi::launch_multi_k6(a, D, c.p, s));
    case 8: return from_cuda(multi::launch_multi_k8(a, D, c.p, s));
    default: return from_cuda(multi::launch_multi_k16(a, D, c.p, s));
  }
}

}  // namespace

extern "C" {

size_t lkv_multi_workspace_bytes(lkv_qspec spec, int B, int Hq, int Hkv, int T_cap, int D, int max_q) {
  MultiCall c;
  return multi_shape(spec, B, Hq, Hkv, T_cap, D, max_q, c) == LKV_OK ? c.p.ws_total : 0;
}

int lkv_decode_attention_multi(lkv_qspec spec, int B, int Hq, int Hkv, int T_cap, int D, int max_q, int n_rows,
                               const int32_t* seq_lens, const int32_t* cu_q, const void* q, const void* k_codes,
                               const float* k_sz, const void* v_codes, const float* v_sz, lkv_score_rule rule, float* out,
                               float* lse, void* workspace, size_t ws_bytes, void* stream) {
  return multi_impl(spec, B, Hq, Hkv, T_cap, D, max_q, n_rows, seq_lens, cu_q, q, nullptr, 0, 0, k_codes, k_sz, v_codes,
                    v_sz, rule, out, lse, workspace, ws_bytes, stream);
}

int lkv_decode_attention_multi_paged(lkv_qspec spec, int B, int Hq, int Hkv, int pages_per_seq, int num_pages, int D,
                                     int max_q, int n_rows, const int32_t* seq_lens, const int32_t* cu_q, const void* q,
                                     const int32_t* block_table, const void* k_pool, const float* k_sz_pool,
                                     const void* v_pool, const float* v_sz_pool, lkv_score_rule rule, float* out,
                                     float* lse, void* workspace, size_t ws_bytes, void* stream) {
  if (pages_per_seq <= 0 || num_pages <= 0) return LKV_ERR_INVALID_ARG;
  if ((long long)pages_per_seq * kPageTokens > (1ll << 30)) return LKV_ERR_UNSUPPORTED;
  if (!int_ptr_ok(block_table, true)) return LKV_ERR_INVALID_ARG;
  return multi_impl(spec, B, Hq, Hkv, pages_per_seq * kPageTokens, D, max_q, n_rows, seq_lens, cu_q, q, block_table,
                    pages_per_seq, num_pages, k_pool, k_sz_pool, v_pool, v_sz_pool, rule, out, lse, workspace, ws_bytes,
                    stream);
}

int lkv_page_plan(int B, int pages_per_seq, int num_pages, int n_cap, const int32_t* seq_lens, const int32_t* n_new,
                  const int32_t* free_pages, int free_cap, const int32_t* free_count, int32_t* block_table,
                  int32_t* new_lens, int32_t* cu_new, int32_t* positions, int32_t* token_seq, int64_t* slots,
                  int32_t* free_left, int32_t* status, void* stream) {
  if (B < 0 || n_cap < 0 || free_cap < 0 || pages_per_seq <= 0 || num_pages <= 0) return LKV_ERR_INVALID_ARG;
  if (B > kPlanMaxBatch || n_cap > (1 << 30) || (long long)pages_per_seq * kPageTokens > (1ll << 30)) return LKV_ERR_UNSUPPORTED;
  const bool b = B > 0, t = n_cap > 0;
  if (!int_ptr_ok(seq_lens, b) || !int_ptr_ok(n_new, b) || !int_ptr_ok(free_pages, free_cap > 0) ||
      !int_ptr_ok(free_count, true) || !int_ptr_ok(block_table, b) || !int_ptr_ok(new_lens, b) || !int_ptr_ok(cu_new, true) ||
      !int_ptr_ok(positions, t) || !int_ptr_ok(token_seq, t) || !int_ptr_ok(free_left, true) || !int_ptr_ok(status, false))
    return LKV_ERR_INVALID_ARG;
  if ((t && slots == nullptr) || !aligned_to(slots, 8)) return LKV_ERR_INVALID_ARG;
  // every block reads all the lengths, so nothing that is written may be an input, nor two outputs one
  const size_t nb = (size_t)B * 4, nt = (size_t)n_cap * 4, ntab = (size_t)B * pages_per_seq * 4;
  const struct { const void* p; size_t n; } in[] = {{seq_lens, nb}, {n_new, nb}, {free_pages, (size_t)free_cap * 4}, {free_count, 4}},
      out[] = {{block_table, ntab}, {new_lens, nb}, {cu_new, nb + 4}, {positions, nt}, {token_seq, nt},
               {slots, 2 * nt}, {free_left, 4}, {status, 4}};
  for (int i = 0; i < 8; ++i) {
    for (int j = 0; j < 4; ++j)
      if (overlap(out[i].p, out[i].n, in[j].p, in[j].n)) return LKV_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return LKV_ERR_INVALID_ARG;
  }
  PlanArgs a{};
  a.B = B; a.pps = pages_per_seq; a.num_pages = num_pages; a.n_cap = n_cap; a.free_cap = free_cap;
  a.lens = seq_lens; a.n_new = n_new; a.free_pages = free_pages; a.free_count = free_count;
  a.table = block_table; a.new_lens = new_lens; a.cu = cu_new; a.positions = positions; a.token_seq = token_seq;
  a.slots = slots; a.free_left = free_left; a.status = status;
  a.wide = aligned16(positions) && aligned16(token_seq) && aligned16(slots);
  return from_cuda(launch_page_plan(a, static_cast<cudaStream_t>(stream)));
}

int lkv_rope_table(lkv_rope_spec spec, int rows, float* table, void* stream) {
  if (rows < 0) return LKV_ERR_INVALID_ARG;
  if (spec.kind < LKV_ROPE_NONE || spec.kind > LKV_ROPE_RAMP) return LKV_ERR_UNSUPPORTED;
  if (spec.rot_dim < 16 || spec.rot_dim > 128 || spec.rot_dim % 16 != 0) return LKV_ERR_UNSUPPORTED;
  if (!std::isfinite(spec.base) || !(spec.base > 1.0) || !std::isfinite(spec.attn_factor)) return LKV_ERR_INVALID_ARG;
  if (spec.kind != LKV_ROPE_NONE && (!std::isfinite(spec.factor) || !(spec.factor > 0.0))) return LKV_ERR_INVALID_ARG;
  if (spec.kind == LKV_ROPE_SMOOTH || spec.kind == LKV_ROPE_RAMP) {
    if (!std::isfinite(spec.low) || !std::isfinite(spec.high) || !(spec.low > 0.0) || !(spec.high > spec.low))
      return LKV_ERR_INVALID_ARG;
    if (!std::isfinite(spec.orig_ctx) || !(spec.orig_ctx > 0.0)) return LKV_ERR_INVALID_ARG;
  }
  if (!ptr_ok(table, rows > 0)) return LKV_ERR_INVALID_ARG;
  RopeTableArgs a{};
  a.kind = spec.kind; a.half = spec.rot_dim / 2; a.rows = rows;
  a.base = spec.base; a.factor = spec.factor; a.low = spec.low; a.high = spec.high; a.orig = spec.orig_ctx;
  a.attn = spec.attn_factor; a.table = table;
  return from_cuda(launch_rope_table(a, static_cast<cudaStream_t>(stream)));
}

int lkv_rope_append_kv(lkv_qspec spec, int n_cap, int Hq, int Hkv, int num_pages, int page_tokens, int D,
                       const int32_t* n_tokens, const int32_t* positions, const int64_t* slots, const void* q,
                       int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                       const void* q_weight, const void* k_weight, float eps, int rot_dim, int interleaved,
                       const float* table, int table_rows, void* q_out, void* k_codes, float* k_sz, void* v_codes,
                       float* v_sz, int reciprocal, void* stream) {
  if (!bits_ok(spec.k_bits) || !bits_ok(spec.v_bits)) return LKV_ERR_UNSUPPORTED;
  const int rc = check_cache_shape(num_pages, Hkv, page_tokens, D, spec.group);
  if (rc) return rc;
  if (n_cap < 0 || Hq <= 0 || num_pages <= 0 || page_tokens <= 0 || table_rows < 0) return LKV_ERR_INVALID_ARG;
  if (rot_dim < 0 || rot_dim > D || rot_dim % 16 != 0) return LKV_ERR_UNSUPPORTED;
  if ((interleaved != 0 && interleaved != 1) || (reciprocal != 0 && reciprocal != 1)) return LKV_ERR_INVALID_ARG;
  if (!std::isfinite(eps) || eps < 0.0f) return LKV_ERR_INVALID_ARG;
  const bool ne = n_cap > 0;
  if (!int_ptr_ok(n_tokens, false) || !int_ptr_ok(positions, ne && rot_dim > 0)) return LKV_ERR_INVALID_ARG;
  if ((ne && slots == nullptr) || !aligned_to(slots, 8)) return LKV_ERR_INVALID_ARG;
  if (!ptr_ok(q, ne) || !ptr_ok(k, ne) || !ptr_ok(v, ne) || !ptr_ok(q_out, ne) || !ptr_ok(table, ne && rot_dim > 0) ||
      !ptr_ok(k_codes, ne) || !ptr_ok(v_codes, ne) || !ptr_ok(k_sz, ne && spec.k_bits < 16) ||
      !ptr_ok(v_sz, ne && spec.v_bits < 16) || !aligned16(q_weight) || !aligned16(k_weight))
    return LKV_ERR_INVALID_ARG;
  // rows are read 16 bytes at a time, and a token's heads lie side by side
  if (q_stride < (int64_t)Hq * D || k_stride < (int64_t)Hkv * D || v_stride < (int64_t)Hkv * D || q_stride % 8 != 0 ||
      k_stride % 8 != 0 || v_stride % 8 != 0)
    return LKV_ERR_INVALID_ARG;
  if (!ne) return LKV_OK;
  // a row of q_out is written while others are read: in place is refused
  const size_t qo = (size_t)n_cap * Hq * D * 2;
  const size_t last = (size_t)(n_cap - 1);
  if (overlap(q_out, qo, q, (last * q_stride + (size_t)Hq * D) * 2) || overlap(q_out, qo, k, (last * k_stride + (size_t)Hkv * D) * 2) ||
      overlap(q_out, qo, v, (last * v_stride + (size_t)Hkv * D) * 2))
    return LKV_ERR_INVALID_ARG;
  RopeAppendArgs a{};
  a.n_cap = n_cap; a.Hq = Hq; a.Hkv = Hkv; a.num_pages = num_pages; a.page_tokens = page_tokens; a.G = spec.group;
  a.kb = spec.k_bits; a.vb = spec.v_bits; a.rot = rot_dim;
  a.n_tokens = n_tokens; a.positions = positions; a.slots = slots;
  a.q = static_cast<const uint16_t*>(q); a.k = static_cast<const uint16_t*>(k); a.v = static_cast<const uint16_t*>(v);
  a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
  a.q_weight = static_cast<const uint16_t*>(q_weight); a.k_weight = static_cast<const uint16_t*>(k_weight);
  a.eps = eps; a.one = 1.0f; a.reciprocal = reciprocal != 0;
  a.table = table; a.table_rows = table_rows;
  a.q_out = static_cast<uint16_t*>(q_out);
  a.k_codes = static_cast<uint8_t*>(k_codes); a.k_sz = k_sz;
  a.v_codes = static_cast<uint8_t*>(v_codes); a.v_sz = v_sz;
  return from_cuda(launch_rope_append(a, D, interleaved != 0, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
