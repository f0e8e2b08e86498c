// C ABI of the attention over a paged cache: argument checks on the host and
// the choice of kernel; and the windowed mask as a slice list.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "../../include/attn_paged.h"
#include "attn_internal.h"
#include "paged_join.cuh"
#include "paged_plan.cuh"

namespace attn {

// First failure status of the paged attention and cache kernels on this device.
__device__ unsigned int g_paged_status;

unsigned int *paged_status() {
  constexpr int kDev = 64;
  static unsigned int *at[kDev] = {};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDev) return nullptr;
  std::lock_guard<std::mutex> lock(mu);
  if (!at[dev]) {
    void *x = nullptr;
    if (cudaGetSymbolAddress(&x, g_paged_status) != cudaSuccess) return nullptr;
    at[dev] = static_cast<unsigned int *>(x);
  }
  return at[dev];
}

int paged_status_take(unsigned int *status) {
  unsigned int zero = 0;
  if (cudaMemcpyFromSymbol(status, g_paged_status, sizeof(unsigned int)) != cudaSuccess) return ATTN_ERR_CUDA;
  if (*status && cudaMemcpyToSymbol(g_paged_status, &zero, sizeof(unsigned int)) != cudaSuccess)
    return ATTN_ERR_CUDA;
  return ATTN_OK;
}

namespace {
bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
}  // namespace

int paged_check_pages(const attn_pages_t *g, int *shift) {
  if (!g || !g->k || !g->v || g->n_pages < 1 || g->hk < 1) return ATTN_ERR_INVALID_ARG;
  if (g->d != 64 && g->d != 128) return ATTN_ERR_UNSUPPORTED;
  if (g->page_size < 16 || (g->page_size & (g->page_size - 1))) return ATTN_ERR_UNSUPPORTED;
  if (!al16(g->k) || !al16(g->v) || (g->page_stride | g->token_stride | g->head_stride) & 7)
    return ATTN_ERR_UNSUPPORTED;
  // strides of 0 (one page seen as many) are fine to read; negative ones are not served
  if (g->page_stride < 0 || g->token_stride < 0 || g->head_stride < 0) return ATTN_ERR_UNSUPPORTED;
  *shift = 0;
  while ((1 << *shift) < g->page_size) ++*shift;
  return ATTN_OK;
}

int paged_check_seqs(const attn_seqs_t *s, int page_size) {
  if (!s || s->n_seqs < 0 || s->n_slots < 0 || s->max_pages < 0) return ATTN_ERR_INVALID_ARG;
  if (s->n_seqs > ATTN_PAGED_MAX_SEQS) return ATTN_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(s->max_pages) * page_size > ATTN_PAGED_MAX_LEN) return ATTN_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(s->max_pages) * page_size * s->n_seqs > ATTN_PAGED_MAX_KEYS) return ATTN_ERR_UNSUPPORTED;
  if (s->n_seqs == 0) return ATTN_OK;
  if (!s->table || !s->seq_lens) return ATTN_ERR_INVALID_ARG;
  if (!s->seqs && s->n_seqs > s->n_slots) return ATTN_ERR_INVALID_ARG;
  if (s->table_stride < s->max_pages) return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

namespace {

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

int check_call(const void *q, const int32_t *q_ptr, int n_tokens, int max_q, int hq, const attn_pages_t *pages,
               const attn_pages8_t *pages8, const attn_seqs_t *seqs, float scale, const void *out, int out_dtype, const float *lse,
               int *shift) {
  if (n_tokens < 0 || hq < 1 || max_q < 1) return ATTN_ERR_INVALID_ARG;
  int rc = pages8 ? paged_check_pages8(pages8, shift) : paged_check_pages(pages, shift);
  if (rc != ATTN_OK) return rc;
  if ((rc = paged_check_seqs(seqs, pages->page_size)) != ATTN_OK) return rc;
  if (hq % pages->hk != 0) return ATTN_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  if (out_dtype != ATTN_DTYPE_BF16 && out_dtype != ATTN_DTYPE_F32) return ATTN_ERR_INVALID_ARG;
  if (!q_ptr && n_tokens != seqs->n_seqs) return ATTN_ERR_INVALID_ARG;
  if (n_tokens == 0 || seqs->n_seqs == 0) return ATTN_OK;
  if (!q || !out || !lse) return ATTN_ERR_INVALID_ARG;
  if (!al16(q) || !al16(out)) return ATTN_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(n_tokens) * hq >= (int64_t(1) << 31)) return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

// Whether q or the memory that the pages span (and, in 8 bits, their scales) meets
// out, which is written while they are read.
bool meets_out(const void *q, int n_tokens, int hq, const attn_pages_t *g, const attn_pages8_t *g8, const void *out, int out_dtype) {
  const size_t n = static_cast<size_t>(n_tokens) * hq * g->d;
  const char *ob = static_cast<const char *>(out), *oe = ob + n * (out_dtype == ATTN_DTYPE_F32 ? 4 : 2);
  auto last = [&](int64_t page, int64_t token, int64_t head) {
    return static_cast<size_t>(g->n_pages - 1) * page + static_cast<size_t>(g->page_size - 1) * token + static_cast<size_t>(g->hk - 1) * head;
  };
  const size_t span = (g8 ? 1 : 2) * (last(g->page_stride, g->token_stride, g->head_stride) + g->d);
  auto meets = [&](const void *x, size_t bytes) {
    const char *b = static_cast<const char *>(x);
    return b < oe && ob < b + bytes;
  };
  if (g8) {
    const size_t scales = 4 * (last(g8->scale_page_stride, g8->scale_token_stride, g8->scale_head_stride) + 1);
    if (meets(g8->k_scales, scales) || meets(g8->v_scales, scales)) return true;
  }
  return meets(q, 2 * n) || meets(g->k, span) || meets(g->v, span);
}

PagedParams params(const void *q, const int32_t *q_ptr, int n_tokens, int hq, const attn_pages_t *g, const attn_pages8_t *g8,
                   const attn_seqs_t *s, float scale, int shift) {
  PagedParams p;
  std::memset(&p, 0, sizeof(p));
  if (g8) {
    p.bits8 = 1;
    p.format = g8->format;
    p.k_scales = g8->k_scales;
    p.v_scales = g8->v_scales;
    p.scale_page = g8->scale_page_stride;
    p.scale_token = g8->scale_token_stride;
    p.scale_head = g8->scale_head_stride;
  }
  p.q = q;
  p.k = g->k;
  p.v = g->v;
  p.q_ptr = q_ptr;
  p.seqs = s->seqs;
  p.seq_lens = s->seq_lens;
  p.table = s->table;
  p.table_stride = s->table_stride;
  p.page_stride = g->page_stride;
  p.token_stride = g->token_stride;
  p.head_stride = g->head_stride;
  p.n_tokens = n_tokens;
  p.n_seqs = s->n_seqs;
  p.n_slots = s->n_slots;
  p.max_pages = s->max_pages;
  p.n_pages = g->n_pages;
  p.page_shift = shift;
  p.hq = hq;
  p.hk = g->hk;
  p.G = hq / g->hk;
  p.causal = 1;
  p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  p.wait_ns = wait_limit_ns();
  return p;
}

// The most slabs of 32 keys that an SM of the row kernels of codes can have.  Where they are few
// what counts is the kernels' start: a join's blocks, and the next call's, start beside a kernel
// that leaves them registers.  12 warps leave none, 8 some at head dim 64, 4 at either; and the
// kernel for few rows has tensor maps to read besides.
double slabs_of(const PagedParams &p, int64_t rows) {
  double keys = static_cast<double>(static_cast<int64_t>(p.max_pages) << p.page_shift);
  if (p.causal && p.window > 0) keys = std::min(keys, static_cast<double>(p.window) + p.sinks + 32);
  return keys * p.n_seqs * p.hk * static_cast<double>((rows + 15) / 16) / (32.0 * device_sm_count());
}

// The kernel for few rows, from 6 (head dim 64: 9) slabs for each of 8 warps.  4 query heads to
// each of 8 key/value heads of 128, it against 8 warps of the one for 16 rows.  One sequence: 512 keys 16.9,
// 14.2 us; 8192 20.7, 18.0; 16384 23.9, 22.7; 32768 29.2, 28.6.  Four: 4096 keys 24.3, 22.1;
// 6144 25.8, 26.0; 8192 29.8, 31.1; 32768 64.1, 75.5.  Of 64 columns, four sequences: 4096 keys 21.9,
// 18.6; 8192 25.5, 24.7; 12288 29.2, 30.2; 32768 50.4, 55.7.
bool few_slabs(double slabs, int d) { return slabs <= 8 * (d == 64 ? 9 : 6); }

// Warps of the kernel for 16 rows.  8 against 4, one sequence of 128 columns: 512 keys 14.0, 11.9 us; 4096
// 15.9, 14.1; 12288 20.6, 20.1; 16384 22.5, 24.5; four: 512 15.1, 12.7; 1024 15.4, 14.5; 2048 17.4,
// 18.6.  Of 64 columns, one: 512 12.6, 11.0; 8192 15.4, 14.5; 32768 22.8, 25.4; four: 2048 15.6, 14.4; 4096
// 18.5, 19.4.  12 against 8, of 64 columns, 16 rows, four sequences: 4096 28.2, 23.3; 8192 31.9, 30.7;
// 12288 35.5, 36.3; 32768 56.8, 61.7; 28 rows, which are two passes: 4096 31.8, 30.8; 6144 35.4,
// 36.3; 32768 89, 99.5.
int rows8_warps(double slabs, int d) {
  if (slabs <= 4 * (d == 64 ? 5 : 3)) return 4;
  return d == 128 || few_slabs(slabs, d) ? 8 : 12;
}

// Items of up to 16 rows (query heads of one key/value head times tokens) go to
// the warp-level kernel, larger ones to the tensor-core tiles; of codes up to 32, in
// two passes over the keys, since the tiles turn every code into an operand before they
// begin and fill 128 rows.  16 sequences of 8192 keys, 8 key/value heads of 128, e4m3, rows
// against tiles: 20 rows 120, 144 us; 32 rows 123, 145; 40 rows 169, 150.  int8: 32 rows 130,
// 138; 40 rows 181, 143.  Of 64 columns, int8: 32 rows 85, 93; 40 rows 118, 97; 32 sequences
// of 1500 keys: 40, 45; 51, 46.  What the kernel chose is left in p and, the rows of a piece,
// in `tile_rows`.
int paged_launch(PagedParams &p, int d, int tokens, cudaStream_t s, int *tile_rows) {
  const int64_t rows = static_cast<int64_t>(tokens) * p.G;
  if (rows > (p.bits8 ? 32 : 16)) {
    const int rc = paged_tiles_launch(p, d, tokens, s, tile_rows);
    if (rc != ATTN_ERR_UNSUPPORTED) return rc;
  }
  if (p.share.side == 1) p.share.side = 0;     // two passes share the SMs only where tiles are the first
  *tile_rows = 16;
  if (!p.bits8) return paged_rows_launch(p, d, s);
  const double slabs = slabs_of(p, rows);
  if (rows <= 8 && !few_slabs(slabs, d)) {
    *tile_rows = 8;
    const int rc = paged_few8_launch(p, d, s);
    if (rc != ATTN_ERR_UNSUPPORTED) return rc;
    *tile_rows = 16;
  }
  return paged_rows8_launch(p, d, rows8_warps(slabs, d), s);
}

// The prefix's tiles are bound by their products, what follows it by the cache's
// bandwidth; one after the other each leaves idle what the other wants.  So they
// run side by side: the tiles take T SMs, the others go to the rows kernel, whose
// blocks start there at once.  T balances A / T and B / (SMs - T): A from the time
// of a 128-key step of a row tile, B from the 64 (head dim 128) or 53 GB/s that
// one SM streams when the bandwidth is not what binds it, a tenth on top, and 4 us
// an SM on either side.  That T is within 3 us of the best of all at seven shapes.
// Against one pass after the other (32 query and 8 key/value heads of 128): 16
// sequences with 2048 keys before 52 each, 25.6 -> 21.6 us; 32 with 32768 before
// 109, 59 -> 46; 32 with 4096 before 1755, 77 -> 61; 256 with 32768 before 219,
// 174.7 -> 164 (155 since).  Of 16 heads of 64: 128 with 16384 before 219, 70 ->
// 63; 50 with 6817 before 150, two tokens each, 51.3 -> 50.  All of this is of bf16 pages; those of codes
// go by the same costs, which were not measured for them (a step of their tiles takes half as long again, a key half the bytes).
Share share_of(const PagedParams &p, int p_tokens, const PagedParams &r, int r_tokens, int d) {
  Share s;
  std::memset(&s, 0, sizeof(s));
  s.unit = paged_tiles_heads(device_sm_count(), p.hk);
  auto side = [](const PagedParams &x, float cost) {
    return Share::Side{x.seqs, x.seq_lens, x.n_seqs, x.n_slots, x.max_pages << x.page_shift, cost, 4000.f * device_sm_count()};
  };
  const int tpt = std::max(1, 128 / p.G), two = p_tokens > tpt, tpi = tpt << two;
  const float step = d == 128 ? (two ? 1560.f : 1000.f) : (two ? 1200.f : 820.f);
  s.of[0] = side(p, step / 128 * ((p_tokens + tpi - 1) / tpi) * p.hk);
  s.of[1] = side(r, (d == 128 ? 8.8f : 5.3f) * ((r_tokens * r.G + 15) / 16) * r.hk);
  return s;
}

size_t pieces_bytes(int d) { return up256(std::max(paged_rows_workspace(d), paged_tiles_workspace(d))); }

// attn_prefix_fwd's workspace: for each of the two passes where every row's
// pieces are, the rows finished within a span, and the pieces.
struct PairLayout {
  size_t rec[2], ml[2], o[2], pieces[2], total;
};
PairLayout pair_layout(int n_tokens, int hq, int d) {
  PairLayout L;
  const size_t rows = static_cast<size_t>(n_tokens) * hq;
  size_t at = 0;
  auto put = [&](size_t bytes) {
    const size_t x = at;
    at += up256(bytes);
    return x;
  };
  for (size_t &x : L.rec) x = put(rows * sizeof(Rec4));
  for (size_t &x : L.ml) x = put(rows * 8);
  for (size_t &x : L.o) x = put(rows * d * 4);
  for (size_t &x : L.pieces) x = put(pieces_bytes(d));
  L.total = at;
  return L;
}

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" {

int attn_paged_workspace_bytes(int n_tokens, int hq, int d, int prefix, size_t *bytes) {
  if (!bytes || n_tokens < 0 || hq < 1) return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (paged_rows_workspace(d) == 0) return ATTN_ERR_CUDA;
  *bytes = prefix ? pair_layout(n_tokens, hq, d).total : pieces_bytes(d);
  return ATTN_OK;
}

static int paged_call(const void *q, const int32_t *q_ptr, int n_tokens, int max_q, int hq, const attn_pages_t *pages,
                      const attn_pages8_t *pages8, const attn_seqs_t *seqs, float scale, int window, int sinks, void *out,
                      int out_dtype, float *lse, void *d_ws, size_t ws_bytes, attn_stream_t stream) {
  if (window < 0 || sinks < 0) return ATTN_ERR_INVALID_ARG;
  int shift = 0;
  int rc = check_call(q, q_ptr, n_tokens, max_q, hq, pages, pages8, seqs, scale, out, out_dtype, lse, &shift);
  if (rc != ATTN_OK) return rc;
  if (n_tokens == 0 || seqs->n_seqs == 0) return ATTN_OK;
  if (!d_ws) return ATTN_ERR_INVALID_ARG;
  if (!al16(d_ws)) return ATTN_ERR_UNSUPPORTED;
  if (meets_out(q, n_tokens, hq, pages, pages8, out, out_dtype)) return ATTN_ERR_INVALID_ARG;
  size_t need = 0;
  if ((rc = attn_paged_workspace_bytes(n_tokens, hq, pages->d, 0, &need)) != ATTN_OK) return rc;
  if (ws_bytes < need) return ATTN_ERR_CAPACITY;
  PagedParams p = params(q, q_ptr, n_tokens, hq, pages, pages8, seqs, scale, shift);
  // no sequence is longer than ATTN_PAGED_MAX_LEN: larger values say the same
  p.window = std::min(window, ATTN_PAGED_MAX_LEN);
  p.sinks = std::min(sinks, ATTN_PAGED_MAX_LEN);
  p.out = out;
  p.lse = lse;
  p.out_f32 = out_dtype == ATTN_DTYPE_F32;
  p.part_o = static_cast<float *>(d_ws);
  p.status = paged_status();
  if (!p.status) return ATTN_ERR_CUDA;
  int tile_rows;
  return paged_launch(p, pages->d, std::min(max_q, n_tokens), reinterpret_cast<cudaStream_t>(stream), &tile_rows);
}

static int prefix_call(const void *q, const int32_t *q_ptr, int n_tokens, int max_q, int hq, const attn_pages_t *pages,
                       const attn_pages8_t *pages8, const attn_seqs_t *prefix, const int32_t *group_ptr, const attn_seqs_t *seqs,
                       float scale, void *out, int out_dtype, float *lse, void *d_ws, size_t ws_bytes, attn_stream_t stream) {
  int shift = 0;
  int rc = check_call(q, q_ptr, n_tokens, max_q, hq, pages, pages8, seqs, scale, out, out_dtype, lse, &shift);
  if (rc != ATTN_OK) return rc;
  if ((rc = paged_check_seqs(prefix, pages->page_size)) != ATTN_OK) return rc;
  if (prefix->n_seqs > 0 && !group_ptr) return ATTN_ERR_INVALID_ARG;
  if (n_tokens == 0 || seqs->n_seqs == 0) return ATTN_OK;
  if (!d_ws) return ATTN_ERR_INVALID_ARG;
  if (!al16(d_ws)) return ATTN_ERR_UNSUPPORTED;
  if (meets_out(q, n_tokens, hq, pages, pages8, out, out_dtype)) return ATTN_ERR_INVALID_ARG;
  size_t need = 0;
  if ((rc = attn_paged_workspace_bytes(n_tokens, hq, pages->d, 1, &need)) != ATTN_OK) return rc;
  if (ws_bytes < need) return ATTN_ERR_CAPACITY;
  unsigned int *status = paged_status();
  if (!status) return ATTN_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint8_t *ws = static_cast<uint8_t *>(d_ws);
  int tile_rows;
  // what follows the prefix
  PagedParams r = params(q, q_ptr, n_tokens, hq, pages, pages8, seqs, scale, shift);
  r.out = out;
  r.lse = lse;
  r.out_f32 = out_dtype == ATTN_DTYPE_F32;
  r.status = status;
  const int tokens = std::min(max_q, n_tokens);
  if (prefix->n_seqs == 0) {
    r.part_o = reinterpret_cast<float *>(ws);
    return paged_launch(r, pages->d, tokens, s, &tile_rows);
  }
  // the prefixes: rows of a whole group against its keys, none of them masked
  PagedParams p = params(q, q_ptr, n_tokens, hq, pages, pages8, prefix, scale, shift);
  p.group_ptr = group_ptr;
  p.n_members = seqs->n_seqs;
  p.causal = 0;
  p.status = status;
  const PairLayout L = pair_layout(n_tokens, hq, pages->d);
  PagedParams *pass[2] = {&p, &r};
  for (int i = 0; i < 2; ++i) {
    pass[i]->rec = reinterpret_cast<Rec4 *>(ws + L.rec[i]);
    pass[i]->dense_ml = reinterpret_cast<float *>(ws + L.ml[i]);
    pass[i]->dense_o = reinterpret_cast<float *>(ws + L.o[i]);
    pass[i]->part_o = reinterpret_cast<float *>(ws + L.pieces[i]);
  }
  // neither pass reads what the other writes: the second starts on each SM that
  // the first leaves or does not take, and waits for its end before its own
  r.wait_end = 1;
  int pre_rows;
  const int pre_tokens = (n_tokens + prefix->n_seqs - 1) / prefix->n_seqs, G = hq / pages->hk;
  if (static_cast<int64_t>(tokens) * G <= 16) {
    p.share = share_of(p, pre_tokens, r, tokens, pages->d);
    p.share.side = 1;
  }
  if ((rc = paged_launch(p, pages->d, pre_tokens, s, &pre_rows)) != ATTN_OK) return rc;
  if (p.share.side == 1) {
    r.share = p.share;
    r.share.side = 2;
  }
  if ((rc = paged_launch(r, pages->d, tokens, s, &tile_rows)) != ATTN_OK) return rc;
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(n_tokens) * hq + 15) / 16));
  auto join = pages->d == 128 ? paged_join_pair_kernel<128> : paged_join_pair_kernel<64>;
  return launch_after(join, grid, 256, 0, s, p, r, pre_rows, tile_rows);
}

int attn_paged_fwd(const void *q, const int32_t *q_ptr, int n_tokens, int max_q, int hq,
                   const attn_pages_t *pages, const attn_seqs_t *seqs, float scale, int window, int sinks,
                   void *out, int out_dtype, float *lse, void *d_ws, size_t ws_bytes, attn_stream_t stream) {
  return paged_call(q, q_ptr, n_tokens, max_q, hq, pages, nullptr, seqs, scale, window, sinks, out, out_dtype, lse, d_ws, ws_bytes, stream);
}

int attn_paged8_fwd(const void *q, const int32_t *q_ptr, int n_tokens, int max_q, int hq,
                    const attn_pages8_t *pages, const attn_seqs_t *seqs, float scale, int window, int sinks,
                    void *out, int out_dtype, float *lse, void *d_ws, size_t ws_bytes, attn_stream_t stream) {
  if (!pages) return ATTN_ERR_INVALID_ARG;
  return paged_call(q, q_ptr, n_tokens, max_q, hq, &pages->pages, pages, seqs, scale, window, sinks, out, out_dtype, lse, d_ws, ws_bytes, stream);
}

int attn_prefix_fwd(const void *q, const int32_t *q_ptr, int n_tokens, int max_q, int hq,
                    const attn_pages_t *pages, const attn_seqs_t *prefix, const int32_t *group_ptr,
                    const attn_seqs_t *seqs, float scale, void *out, int out_dtype, float *lse, void *d_ws,
                    size_t ws_bytes, attn_stream_t stream) {
  return prefix_call(q, q_ptr, n_tokens, max_q, hq, pages, nullptr, prefix, group_ptr, seqs, scale, out, out_dtype, lse, d_ws, ws_bytes, stream);
}

int attn_prefix8_fwd(const void *q, const int32_t *q_ptr, int n_tokens, int max_q, int hq,
                     const attn_pages8_t *pages, const attn_seqs_t *prefix, const int32_t *group_ptr,
                     const attn_seqs_t *seqs, float scale, void *out, int out_dtype, float *lse, void *d_ws,
                     size_t ws_bytes, attn_stream_t stream) {
  if (!pages) return ATTN_ERR_INVALID_ARG;
  return prefix_call(q, q_ptr, n_tokens, max_q, hq, &pages->pages, pages, prefix, group_ptr, seqs, scale, out, out_dtype, lse, d_ws, ws_bytes, stream);
}

int attn_slices_from_windows(const int32_t *h_lengths, int n, int window, int sinks, attn_slice_t *h_out,
                             int capacity, int *n_out) {
  if (n < 0 || (n > 0 && !h_lengths) || window < 0 || sinks < 0 || !n_out || capacity < 0) return ATTN_ERR_INVALID_ARG;
  int64_t at = 0;
  for (int i = 0; i < n; ++i) {
    if (h_lengths[i] < 0) return ATTN_ERR_INVALID_ARG;
    at += h_lengths[i];
  }
  if (at >= (int64_t(1) << 31)) return ATTN_ERR_INVALID_ARG;
  int64_t count = 0;
  auto put = [&](int64_t q0, int64_t q1, int64_t k0, int64_t k1, int type) {
    if (q1 <= q0 || k1 <= k0) return;
    if (count < capacity && h_out)
      h_out[count] = attn_slice_t{static_cast<int32_t>(q0), static_cast<int32_t>(q1), static_cast<int32_t>(k0),
                                  static_cast<int32_t>(k1), type};
    ++count;
  };
  at = 0;
  for (int i = 0; i < n; ++i) {
    const int64_t L = h_lengths[i];
    // rows before window + sinks see every earlier key; of the others' keys
    // key `sinks` is the first that no row of theirs sees
    const int64_t m = window == 0 ? L : std::min<int64_t>(L, static_cast<int64_t>(window) + sinks);
    put(at, at + m, at, at + m, ATTN_MASK_CAUSAL);
    put(at + m, at + L, at, at + sinks, ATTN_MASK_FULL);
    // bi-causal rows a = i - m, keys b = j - (m - window + 1):
    // a <= b <= a + window - 1
    put(at + m, at + L, at + m - window + 1, at + L, ATTN_MASK_BI_CAUSAL);
    at += L;
  }
  if (count >= (int64_t(1) << 31)) return ATTN_ERR_INVALID_ARG;
  *n_out = static_cast<int>(count);
  return count > capacity ? ATTN_ERR_CAPACITY : ATTN_OK;
}

}  // extern "C"
