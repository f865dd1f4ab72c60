// hsq_heads.cu -- the C ABI of the head kernels (hsq_rope, hsq_kv_append): argument
// checks, launch planning and launches.
//
// A translation unit of its own: in one with the linears, these kernels changed what the
// compiler makes of the rank-2 activation steps, whose source stayed the same (up to 90
// registers instead of 82, and spills: 3.79 instead of 3.70 us for 8 tokens, K = 4096).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <numeric>

#include "../../include/hsq.h"
#include "hsq_device.cuh"
#include "hsq_host.cuh"
#include "hsq_rope.cuh"

namespace {

constexpr int kMaxHeadDim = 2 * hsq::kRopeMaxPairs;
constexpr int kMaxHeads = 1 << 16;
constexpr long long kMaxStride = 1ll << 40;

size_t dtype_bytes(hsq_dtype t) { return t == HSQ_F32 ? 4 : t == HSQ_BF16 ? 2 : 1; }

// Bytes of a heads view from its first element to its last.
size_t view_bytes(const hsq_heads& v, int tokens, int heads, int dim, size_t es) {
  return (static_cast<size_t>(tokens - 1) * v.token_stride + static_cast<size_t>(heads - 1) * v.head_stride + dim) * es;
}

hsq_status check_view(const hsq_heads* v, int tokens, int heads, int dim, size_t es, bool written) {
  if (!v || !v->data) return HSQ_ERR_INVALID_ARG;
  if (v->token_stride < 0 || v->head_stride < 0 || v->token_stride > kMaxStride || v->head_stride > kMaxStride)
    return HSQ_ERR_INVALID_ARG;
  if (v->token_stride > 0 && tokens - 1 > (1ll << 58) / v->token_stride) return HSQ_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(v->data) % es != 0) return HSQ_ERR_ALIGNMENT;
  if (written) {
    // the rows that are written are apart: heads inside tokens, or tokens inside heads
    const long long hs = heads > 1 ? v->head_stride : kMaxStride, ts = tokens > 1 ? v->token_stride : kMaxStride;
    if (hs < dim || ts < dim) return HSQ_ERR_INVALID_ARG;
    if (heads > 1 && tokens > 1 && ts < (heads - 1) * hs + dim && hs < (tokens - 1) * ts + dim)
      return HSQ_ERR_INVALID_ARG;
  }
  return HSQ_OK;
}

// Whether two heads views share no element: byte ranges apart, or column ranges
// of the same rows (equal token strides, the spans of a token apart), or equal
// stride patterns whose rows of `dim` fall on different residues.
bool views_apart(const hsq_heads& a, int ha, const hsq_heads& b, int hb, int tokens, int dim, size_t es) {
  if (!ranges_meet(a.data, view_bytes(a, tokens, ha, dim, es), b.data, view_bytes(b, tokens, hb, dim, es))) return true;
  const long long diff = static_cast<long long>(reinterpret_cast<uintptr_t>(b.data)) -
                         static_cast<long long>(reinterpret_cast<uintptr_t>(a.data));
  auto apart_mod = [&](long long period, long long span_a, long long span_b) {
    if (period <= 0) return false;
    const long long p = period * static_cast<long long>(es), d = ((diff % p) + p) % p;
    return span_a * static_cast<long long>(es) <= d && d + span_b * static_cast<long long>(es) <= p;
  };
  if (a.token_stride == b.token_stride &&
      apart_mod(a.token_stride, (ha - 1) * a.head_stride + dim, (hb - 1) * b.head_stride + dim))
    return true;
  return apart_mod(std::gcd(std::gcd(a.token_stride, b.token_stride),
                            std::gcd(ha > 1 ? a.head_stride : 0ll, hb > 1 ? b.head_stride : 0ll)),
                   dim, dim);
}

hsq_status check_rotation(const hsq_rotation* r, int dim) {
  if (!(std::fabs(r->scale) > 0.f) || std::isinf(r->scale)) return HSQ_ERR_INVALID_ARG;
  if (!r->freqs || r->pairs < 1 || 2 * r->pairs > dim) return HSQ_ERR_INVALID_ARG;
  if (r->n_axes < 1 || r->n_axes > HSQ_ROPE_MAX_AXES || (r->n_axes > 1 && !r->pair_axis)) return HSQ_ERR_INVALID_ARG;
  if (r->pair_axis)
    for (int i = 0; i < r->pairs; ++i)
      if (r->pair_axis[i] >= r->n_axes) return HSQ_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(r->freqs) % 4 != 0) return HSQ_ERR_ALIGNMENT;
  return HSQ_OK;
}

hsq_status check_positions(const hsq_positions* p, int n_axes, int max_rows) {
  if (!p->data || p->rows < 1 || p->rows > max_rows) return HSQ_ERR_INVALID_ARG;
  if (p->type != HSQ_POS_I32 && p->type != HSQ_POS_I64 && p->type != HSQ_POS_F32) return HSQ_ERR_INVALID_ARG;
  if (p->ld < n_axes || p->ld > kMaxStride) return HSQ_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(p->data) % (p->type == HSQ_POS_I64 ? 8 : 4) != 0) return HSQ_ERR_ALIGNMENT;
  return HSQ_OK;
}

hsq::RopeTable rope_table(const hsq_rotation* r, const hsq_positions* p) {
  hsq::RopeTable t{};
  t.pos_rows = 1;
  if (!r) return t;
  t.freqs = r->freqs;
  t.pairs = r->pairs;
  t.scale = r->scale;
  t.sign = r->transpose ? -1.f : 1.f;
  if (r->pair_axis)
    for (int i = 0; i < r->pairs; ++i) t.axis2[i / 16] |= static_cast<uint32_t>(r->pair_axis[i]) << (2 * (i % 16));
  if (p) {
    t.pos = p->data;
    t.pos_ld = p->ld;
    t.pos_rows = p->rows;
    t.pos_type = static_cast<int>(p->type);
  }
  return t;
}

// Base address and strides in bytes, or-ed: what has to be a multiple of a piece's bytes.
uintptr_t view_bits(const hsq_heads& v, int tokens, int heads, size_t es) {
  return reinterpret_cast<uintptr_t>(v.data) |
         (static_cast<uintptr_t>((tokens > 1 ? v.token_stride : 0) | (heads > 1 ? v.head_stride : 0)) * es);
}

// The widest piece (elements) that a head's layout allows: 16 bytes of input, for
// bf16 also 8 bytes, else single elements.  `bits`: view_bits of every tensor,
// scaled to the input's element size.  Measured at 4608 tokens x 48 heads x 128: 16 / 8
// bytes / an element 20 - 22 / 26 / 44 us in bf16, 37 / - / 53 in fp32.
int piece_width(hsq_dtype t, int dim, int pairs, uintptr_t bits) {
  const int es = static_cast<int>(dtype_bytes(t));
  for (int v : {16 / es, 4}) {
    if (pairs % v == 0 && (dim - 2 * pairs) % v == 0 && bits % (static_cast<uintptr_t>(v) * es) == 0) return v;
  }
  return 1;
}

// Blocks of the head kernels per SM before a block takes a second pass.  Measured at
// 3 (one resident wave) / 18 / one pass each: 4608 tokens x 48 heads x 128 in bf16 22.6 /
// 20.7 / 25.5 us, 15606 x 16 x 80 in fp32 32.5 / 28.7 / 34.2, the append of 9203 tokens (32 +
// 8 + 8 heads) 48.6 / 43.4 / 63.7.
#ifndef HSQ_ROPE_BLOCKS
#define HSQ_ROPE_BLOCKS 18
#endif
// Blocks of a call over `heads` heads of `units` pieces each, `pairs` angles a token:
// every head of a token in one block where that fits, and as many tokens as then do.
hsq::RopeGrid rope_grid(int tokens, int units, int heads, int pairs) {
  hsq::RopeGrid g{};
  g.units = units;
  g.lanes = std::min(units, hsq::kRopeThreads);
  const int slots = hsq::kRopeThreads / g.lanes;
  g.splits = std::min(slots, (heads + hsq::kRopeHeads - 1) / hsq::kRopeHeads);
  const int most = hsq::kRopeShared / static_cast<int>(pairs * sizeof(float2) + sizeof(hsq::AppendToken));
  g.tokens = std::max(1, std::min(slots / g.splits, most));
  // many tokens: several passes to a block, whose angles and page lookups are formed
  // at once in front of the first
  const int full = HSQ_ROPE_BLOCKS * device_sm_count(),
            rows = (heads + g.splits * hsq::kRopeHeads - 1) / (g.splits * hsq::kRopeHeads);
  const long long blocks = (tokens + static_cast<long long>(g.tokens) - 1) / g.tokens * rows;
  g.passes = static_cast<int>(std::max(1ll, std::min<long long>((blocks + full - 1) / full, most / g.tokens)));
  return g;
}

// Blocks along the heads, in the grid's y dimension, which holds 65535 (above that only
// with more than 131070 heads of more than 128 units: a thread row to a head).
int head_blocks(const hsq::RopeGrid& g, int heads) {
  return (heads + g.splits * hsq::kRopeHeads - 1) / (g.splits * hsq::kRopeHeads);
}

template <class Args>
cudaError_t launch_heads(void (*kernel)(Args), const Args& a, int heads, size_t smem, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>((a.tokens + static_cast<long long>(a.g.tokens) * a.g.passes - 1) / (a.g.tokens * a.g.passes)),
                  static_cast<unsigned>(head_blocks(a.g, heads)));
  const int threads = (a.g.lanes * a.g.splits * a.g.tokens + 31) / 32 * 32;
  return launch_pdl(true, kernel, grid, dim3(threads), smem, st, a);
}

template <typename T, int V>
cudaError_t launch_rope(const hsq::RopeArgs& a, bool adjacent, cudaStream_t st) {
  return launch_heads(adjacent ? hsq::rope_kernel<T, V, true> : hsq::rope_kernel<T, V, false>, a, a.heads,
                      static_cast<size_t>(a.g.tokens) * a.g.passes * a.rot.pairs * sizeof(float2), st);
}

template <typename T, typename C, int V>
cudaError_t launch_append(const hsq::AppendArgs& a, bool adjacent, cudaStream_t st) {
  return launch_heads(adjacent ? hsq::kv_append_kernel<T, C, V, true> : hsq::kv_append_kernel<T, C, V, false>, a,
                      a.q_heads + 2 * a.kv_heads,
                      static_cast<size_t>(a.g.tokens) * a.g.passes *
                          (a.rot.pairs * sizeof(float2) + sizeof(hsq::AppendToken)), st);
}

template <typename T, int V>
cudaError_t launch_append(const hsq::AppendArgs& a, hsq_dtype cache, bool adjacent, cudaStream_t st) {
  if (cache == HSQ_BF16) return launch_append<T, __nv_bfloat16, V>(a, adjacent, st);
  if (cache == HSQ_F32) return launch_append<T, float, V>(a, adjacent, st);
  return launch_append<T, uint8_t, V>(a, adjacent, st);
}

}  // namespace

cudaError_t hsq::take_heads_status(unsigned* v) { return take_status(v); }

hsq_status hsq_rope(const hsq_heads* x, const hsq_heads* y, hsq_dtype dtype, int tokens, int heads, int head_dim,
                    const hsq_rotation* rot, const hsq_positions* pos, cudaStream_t stream) {
  if (dtype != HSQ_BF16 && dtype != HSQ_F32) return HSQ_ERR_INVALID_ARG;
  if (tokens < 0 || heads < 1 || heads > kMaxHeads || head_dim < 2) return HSQ_ERR_INVALID_ARG;
  if (head_dim > kMaxHeadDim) return HSQ_ERR_UNSUPPORTED;
  if (!rot || !pos) return HSQ_ERR_INVALID_ARG;
  hsq_status st = check_rotation(rot, head_dim);
  if (st != HSQ_OK) return st;
  if (tokens == 0) return HSQ_OK;
  const size_t es = dtype_bytes(dtype);
  if ((st = check_positions(pos, rot->n_axes, tokens)) != HSQ_OK) return st;
  if ((st = check_view(x, tokens, heads, head_dim, es, false)) != HSQ_OK) return st;
  if ((st = check_view(y, tokens, heads, head_dim, es, true)) != HSQ_OK) return st;
  const bool in_place = x->data == y->data && (tokens == 1 || x->token_stride == y->token_stride) &&
                        (heads == 1 || x->head_stride == y->head_stride);
  if (!in_place && !views_apart(*x, heads, *y, heads, tokens, head_dim, es)) return HSQ_ERR_INVALID_ARG;
  hsq::RopeArgs a{};
  a.x = {x->data, x->token_stride, x->head_stride};
  a.y = {y->data, y->token_stride, y->head_stride};
  a.rot = rope_table(rot, pos);
  a.tokens = tokens; a.heads = heads;
  const uintptr_t bits = view_bits(*x, tokens, heads, es) | view_bits(*y, tokens, heads, es);
  const int v = piece_width(dtype, head_dim, rot->pairs, bits);
  a.g = rope_grid(tokens, rot->pairs / v + (in_place ? 0 : (head_dim - 2 * rot->pairs) / v), heads, rot->pairs);
  const bool adj = rot->interleaved != 0;
  cudaError_t e;
  if (dtype == HSQ_BF16)
    e = v == 8 ? launch_rope<__nv_bfloat16, 8>(a, adj, stream)
        : v == 4 ? launch_rope<__nv_bfloat16, 4>(a, adj, stream)
                 : launch_rope<__nv_bfloat16, 1>(a, adj, stream);
  else
    e = v == 4 ? launch_rope<float, 4>(a, adj, stream) : launch_rope<float, 1>(a, adj, stream);
  return (e == cudaSuccess && cudaGetLastError() == cudaSuccess) ? HSQ_OK : HSQ_ERR_CUDA;
}

hsq_status hsq_kv_append(const hsq_heads* k, const hsq_heads* v, const hsq_heads* q, const hsq_heads* q_out,
                         hsq_dtype dtype, int tokens, int q_heads, int kv_heads, int head_dim,
                         const hsq_rotation* rot, const hsq_positions* pos, const hsq_paged_cache* cache,
                         const hsq_sequences* seqs, cudaStream_t stream) {
  if (dtype != HSQ_BF16 && dtype != HSQ_F32) return HSQ_ERR_INVALID_ARG;
  if (tokens < 0 || kv_heads < 1 || kv_heads > kMaxHeads || head_dim < 1) return HSQ_ERR_INVALID_ARG;
  if (q_heads < 0 || q_heads > kMaxHeads || (q_heads > 0) != (q != nullptr) || (q != nullptr) != (q_out != nullptr))
    return HSQ_ERR_INVALID_ARG;
  if (head_dim > kMaxHeadDim) return HSQ_ERR_UNSUPPORTED;
  if (!cache || !seqs || (pos && !rot)) return HSQ_ERR_INVALID_ARG;
  hsq_status st = HSQ_OK;
  if (rot && (st = check_rotation(rot, head_dim)) != HSQ_OK) return st;
  if (cache->dtype != HSQ_BF16 && cache->dtype != HSQ_F32 && cache->dtype != HSQ_E4M3) return HSQ_ERR_INVALID_ARG;
  if (cache->dtype != HSQ_E4M3 && (cache->k_scale || cache->v_scale)) return HSQ_ERR_INVALID_ARG;
  // (one new token per sequence: none where there are no sequences)
  if (cache->pages < 1 || cache->page_size < 1 || seqs->max_pages < 1) return HSQ_ERR_INVALID_ARG;
  if (seqs->count < (!seqs->cu_seqlens && tokens == 0 ? 0 : 1)) return HSQ_ERR_INVALID_ARG;
  if (tokens == 0) return HSQ_OK;
  if (!cache->k || !cache->v || !seqs->block_table || !seqs->cache_lens) return HSQ_ERR_INVALID_ARG;
  if (seqs->table_ld < seqs->max_pages || seqs->table_ld > kMaxStride) return HSQ_ERR_INVALID_ARG;
  if (!seqs->cu_seqlens && seqs->count != tokens) return HSQ_ERR_INVALID_ARG;
  const size_t es = dtype_bytes(dtype), cs = dtype_bytes(cache->dtype);
  if ((st = check_view(k, tokens, kv_heads, head_dim, es, false)) != HSQ_OK) return st;
  if ((st = check_view(v, tokens, kv_heads, head_dim, es, false)) != HSQ_OK) return st;
  if (pos && ((st = check_positions(pos, rot->n_axes, tokens)) != HSQ_OK)) return st;
  if (pos && pos->rows != tokens) return HSQ_ERR_INVALID_ARG;
  bool in_place = false;
  if (q) {
    if ((st = check_view(q, tokens, q_heads, head_dim, es, false)) != HSQ_OK) return st;
    if ((st = check_view(q_out, tokens, q_heads, head_dim, es, true)) != HSQ_OK) return st;
    in_place = q->data == q_out->data && (tokens == 1 || q->token_stride == q_out->token_stride) &&
               (q_heads == 1 || q->head_stride == q_out->head_stride);
    if ((!in_place && !views_apart(*q, q_heads, *q_out, q_heads, tokens, head_dim, es)) ||
        !views_apart(*k, kv_heads, *q_out, q_heads, tokens, head_dim, es) ||
        !views_apart(*v, kv_heads, *q_out, q_heads, tokens, head_dim, es))
      return HSQ_ERR_INVALID_ARG;
  }
  // the caches: strides of [pages][page_size][kv_heads][head_dim] in any order of
  // the first three, rows apart, k and v apart from each other and from the inputs
  size_t c_bytes = 0;
  {
    struct Dim { long long n, s; } d[3] = {{cache->pages, cache->page_stride},
                                           {cache->page_size, cache->slot_stride},
                                           {kv_heads, cache->head_stride}};
    std::sort(d, d + 3, [](const Dim& a, const Dim& b) { return a.s < b.s; });
    long long extent = head_dim;  // elements from the first to the last so far
    for (const Dim& x : d) {
      if (x.s < 0 || x.s > kMaxStride) return HSQ_ERR_INVALID_ARG;
      if (x.n == 1) continue;
      if (x.s < extent) return HSQ_ERR_INVALID_ARG;
      if (x.n - 1 > (1ll << 60) / x.s) return HSQ_ERR_INVALID_ARG;
      extent += (x.n - 1) * x.s;
      if (extent > (1ll << 60)) return HSQ_ERR_INVALID_ARG;
    }
    c_bytes = static_cast<size_t>(extent) * cs;
  }
  if (reinterpret_cast<uintptr_t>(cache->k) % cs || reinterpret_cast<uintptr_t>(cache->v) % cs ||
      reinterpret_cast<uintptr_t>(seqs->block_table) % 4 || reinterpret_cast<uintptr_t>(seqs->cache_lens) % 4 ||
      reinterpret_cast<uintptr_t>(seqs->cu_seqlens) % 4 || reinterpret_cast<uintptr_t>(cache->k_scale) % 4 ||
      reinterpret_cast<uintptr_t>(cache->v_scale) % 4)
    return HSQ_ERR_ALIGNMENT;
  if (ranges_meet(cache->k, c_bytes, cache->v, c_bytes)) {
    // k and v as halves of one pool: each other's rows on different residues of the page or slot stride
    const long long diff = static_cast<long long>(reinterpret_cast<uintptr_t>(cache->v)) -
                           static_cast<long long>(reinterpret_cast<uintptr_t>(cache->k));
    auto apart = [&](long long period, long long span) {
      const long long p = period * static_cast<long long>(cs), m = p > 0 ? ((diff % p) + p) % p : 0;
      return span * static_cast<long long>(cs) <= m && m + span * static_cast<long long>(cs) <= p;
    };
    const long long ps = cache->pages > 1 ? cache->page_stride : 0, ss = cache->page_size > 1 ? cache->slot_stride : 0,
                    hs = kv_heads > 1 ? cache->head_stride : 0;
    const long long token = (kv_heads - 1) * hs + head_dim, page = (cache->page_size - 1) * ss + token;
    if (!apart(ps, page) && !apart(std::gcd(ps, ss), token) && !apart(std::gcd(std::gcd(ps, ss), hs), head_dim))
      return HSQ_ERR_INVALID_ARG;
  }
  const hsq_heads* in[4] = {k, v, q, q_out};
  const int in_heads[4] = {kv_heads, kv_heads, q_heads, q_heads};
  for (int i = 0; i < 4; ++i)
    if (in[i])
      for (const void* c : {cache->k, cache->v})
        if (ranges_meet(in[i]->data, view_bytes(*in[i], tokens, in_heads[i], head_dim, es), c, c_bytes))
          return HSQ_ERR_INVALID_ARG;

  hsq::AppendArgs a{};
  a.k = {k->data, k->token_stride, k->head_stride};
  a.v = {v->data, v->token_stride, v->head_stride};
  uintptr_t bits = view_bits(*k, tokens, kv_heads, es) | view_bits(*v, tokens, kv_heads, es);
  if (q) {
    a.q = {q->data, q->token_stride, q->head_stride};
    a.q_out = {q_out->data, q_out->token_stride, q_out->head_stride};
    bits |= view_bits(*q, tokens, q_heads, es) | view_bits(*q_out, tokens, q_heads, es);
  }
  // a cache piece is V elements of cs bytes, at most 16 bytes an access: its bits
  // scaled to the input's size; an fp32 cache of bf16 inputs is written in whole
  // 16-byte pieces or by elements
  const uintptr_t cbits =
      reinterpret_cast<uintptr_t>(cache->k) | reinterpret_cast<uintptr_t>(cache->v) |
      (static_cast<uintptr_t>((cache->pages > 1 ? cache->page_stride : 0) | (cache->page_size > 1 ? cache->slot_stride : 0) |
                              (kv_heads > 1 ? cache->head_stride : 0)) * cs);
  bits |= cs <= es ? cbits * (es / cs) : (cbits % 16 ? 1 : 0);
  a.kc = {cache->k, cache->page_stride, cache->slot_stride, cache->head_stride, cache->k_scale};
  a.vc = {cache->v, cache->page_stride, cache->slot_stride, cache->head_stride, cache->v_scale};
  a.rot = rope_table(rot, pos);
  a.table = seqs->block_table; a.table_ld = seqs->table_ld;
  a.lens = seqs->cache_lens; a.cu = seqs->cu_seqlens;
  a.tokens = tokens; a.seqs = seqs->count;
  a.q_heads = q_heads; a.kv_heads = kv_heads;
  a.pages = cache->pages; a.page_size = cache->page_size; a.max_pages = seqs->max_pages;
  a.q_in_place = in_place ? 1 : 0;
  const int pairs = rot ? rot->pairs : 0;
  const int w = piece_width(dtype, head_dim, pairs, bits);
  a.g = rope_grid(tokens, pairs / w + (head_dim - 2 * pairs) / w, q_heads + 2 * kv_heads, pairs);
  if (head_blocks(a.g, q_heads + 2 * kv_heads) > 65535) return HSQ_ERR_UNSUPPORTED;
  const bool adj = rot && rot->interleaved;
  cudaError_t e;
  if (dtype == HSQ_BF16)
    e = w == 8 ? launch_append<__nv_bfloat16, 8>(a, cache->dtype, adj, stream)
        : w == 4 ? launch_append<__nv_bfloat16, 4>(a, cache->dtype, adj, stream)
                 : launch_append<__nv_bfloat16, 1>(a, cache->dtype, adj, stream);
  else
    e = w == 4 ? launch_append<float, 4>(a, cache->dtype, adj, stream)
               : launch_append<float, 1>(a, cache->dtype, adj, stream);
  return (e == cudaSuccess && cudaGetLastError() == cudaSuccess) ? HSQ_OK : HSQ_ERR_CUDA;
}
