// How the attention over a paged cache is divided: shared by the kernels that
// compute it and the one that joins their pieces.
//
// A work item is one row tile (a few of one sequence's new tokens, packed with
// the query heads of one key/value head) against the key tiles that any of
// its rows sees.  All items' key tiles form one flat list in the order
// (sequence, group of hp key/value heads, row tile, key tile), of which every
// worker takes one contiguous span of equal length, whatever the sequences'
// lengths; hp workers side by side take the same span, one for each head of the
// group, so that rows of neighbouring heads, which lie side by side in a page,
// are read at the same time.  An
// item that ends in the span it began in is finished there; one that crosses
// spans leaves a piece (m, l, unnormalised O) per span, and join_kernel merges
// them.  The list is never written out: each CTA sums the sequences' tile
// counts into shared memory and finds its span by bisection, so one launch
// needs no plan made before it.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_device.cuh"
#include "launch.cuh"

namespace attn {

constexpr float kLn2 = 0.69314718055994531f;

// Left by each worker for the join: the item that begins in its span and goes
// on behind it (rows = 0: none).  Row x0 + r, r < rows, of the sequence whose
// tokens start at q0; np pieces, the first in the worker's slot slot0, the
// others in the first slots of every hp-th worker that follows.
struct __align__(16) Cut {
  int q0, h, x0, rows, np, slot0, pad[2];   // h: the key/value head
};

// Where a row's pieces are: np > 0 pieces, the first at row `row` of slot slot0
// of worker `worker`, the others at that row of the first slots of every hp-th
// worker worker that follows; np = 0: the dense arrays; REC_EMPTY: it sees nothing.
struct __align__(16) Rec4 {
  int worker, slot0, np, row;
};
constexpr int REC_EMPTY = -1;

// Two passes that share the GPU's SMs, each in proportion to what its sequences'
// keys cost it.
struct Share {
  int side;                   // 0: the pass has all SMs; 1, 2: the first, the second of the two
  int unit;                   // the first takes a multiple of so many SMs
  struct Side {
    const int32_t *seqs, *lens;
    int n, n_slots, max_len;
    float cost, base;         // ns of one SM's time: for a key, and whatever the keys
  } of[2];
};

struct PagedParams {
  const void *q, *k, *v;
  const int32_t *q_ptr;       // null: token b belongs to sequence b
  const int32_t *group_ptr;   // prefix pass: "sequence" b is group b of sequences; else null
  const int32_t *seqs, *seq_lens, *table;
  long long table_stride;
  long long page_stride, token_stride, head_stride;   // elements
  int n_tokens, n_seqs, n_members, n_slots, max_pages, n_pages, page_shift;
  int hq, hk, G;
  int causal, window, sinks;
  float scale_log2;
  void *out;                  // [n_tokens, hq, D]
  float *lse;                 // [hq, n_tokens]
  int out_f32;
  // one of several passes over the same rows (prefix, then what follows it):
  // rows finished within a span go to dense_o [n_tokens, hq, D] and dense_ml
  // as (m, l, unnormalised O), and rec says where every row's pieces are
  float *dense_o, *dense_ml;
  Rec4 *rec;                  // [n_tokens, hq]; null: rows are finished to out and lse
  int wait_end;               // launched beside the kernel before it, whose end it has to wait for
  float *part_o;              // pieces: [workers][2][rows][D], [workers][2][rows][2]
  float *part_ml;
  Cut *cuts;                  // [workers]
  int warp_plan;              // make_warp_plan, not make_plan
  int hp, n_spans;            // heads side by side; spans
  Share share;
  int test_stall;             // failure-path test: leave one load out
  // pages in 8 bits: strides above are bytes too, codes have scales
  const float *k_scales, *v_scales;
  long long scale_page, scale_token, scale_head;      // elements
  int bits8, format;          // bits8 = 0: bf16, no scales; format: ATTN_CODES_*
  unsigned int *status;
  unsigned long long wait_ns;
};

struct SeqInfo {
  int slot, q0, nq, len;      // slot < 0: nothing of it may be read
};

// Where the launch waits for the one before it only at its end: one block is
// enough, the others leave their SMs (2 us of a call of 52 against all waiting).
__device__ __forceinline__ void end_after_previous(const PagedParams &p) {
  if (p.wait_end && blockIdx.x == gridDim.x - 1) after_previous();
}

__device__ __forceinline__ void paged_fail(const PagedParams &p, unsigned code) {
  atomicCAS(p.status, 0u, code);
}

// Sequence (or group) b as the device arrays give it, every index checked.
// The loads that do not depend on one another are issued together.
__device__ inline SeqInfo seq_info(const PagedParams &p, int b) {
  SeqInfo s;
  s.slot = p.seqs ? p.seqs[b] : b;
  const bool in_table = s.slot >= 0 && s.slot < p.n_slots;
  s.len = p.n_slots > 0 ? p.seq_lens[in_table ? s.slot : 0] : 0;
  bool bad = !in_table;
  int t0 = b, t1 = b + 1;
  if (p.group_ptr) {
    t0 = p.group_ptr[b];
    t1 = p.group_ptr[b + 1];
    if (t0 < 0 || t1 < t0 || t1 > p.n_members) {
      bad = true;
      t0 = t1 = 0;
    }
  }
  if (p.q_ptr) {
    t0 = p.q_ptr[t0];
    t1 = p.q_ptr[t1];
  }
  if (t0 < 0 || t1 < t0 || t1 > p.n_tokens) {
    bad = true;
    t0 = t1 = 0;
  }
  s.q0 = t0;
  s.nq = t1 - t0;
  if (!in_table) {
    s.slot = -1;
    s.len = 0;
  } else if (s.len < 0 || s.len > (static_cast<long long>(p.max_pages) << p.page_shift)) {
    bad = true;
    s.len = 0;
  }
  if (bad) paged_fail(p, ATTN_ERR_INVALID_ARG);
  return s;
}

// Row tiles.  ROWS > 0: rows r = token * G + head of the group, packed ROWS to
// a tile across token boundaries.  ROWS == 0 (tensor-core tiles): whole
// tokens, `tpi` of them to a tile.
template <int ROWS>
__device__ __forceinline__ int tile_count(int nq, int G, int tpi) {
  return ROWS > 0 ? (nq * G + ROWS - 1) / (ROWS > 0 ? ROWS : 1) : (nq + tpi - 1) / tpi;
}
template <int ROWS>
__device__ __forceinline__ void tile_tokens(int rt, int nq, int G, int tpi, int &t0, int &t1) {
  if (ROWS > 0) {
    t0 = rt * ROWS / G;
    t1 = min(nq - 1, (rt * ROWS + ROWS - 1) / G);
  } else {
    t0 = rt * tpi;
    t1 = min(nq - 1, t0 + tpi - 1);
  }
}

// Key tiles (of 2^KL keys) that tokens t0..t1 of a sequence see: tiles
// [0, ns) for the first tokens, then [w0, w0 + n - ns).
struct Span {
  int ns, w0, n;
  __device__ __forceinline__ int tile(int i) const { return i < ns ? i : i - ns + w0; }
};
template <int KL>
__device__ __forceinline__ Span key_span(const PagedParams &p, const SeqInfo &s, int t0, int t1) {
  Span x;
  const int end = p.causal ? s.len - s.nq + t1 + 1 : s.len;
  x.ns = x.w0 = x.n = 0;
  if (end <= 0) return x;
  const int lo = p.causal && p.window > 0 ? max(0, s.len - s.nq + t0 - p.window + 1) : 0;
  x.w0 = lo >> KL;
  const int w1 = (end + (1 << KL) - 1) >> KL;
  if (lo > 0) x.ns = min((min(p.sinks, end) + (1 << KL) - 1) >> KL, x.w0);
  x.n = x.ns + w1 - x.w0;
  return x;
}
template <int ROWS, int KL>
__device__ __forceinline__ Span tile_span(const PagedParams &p, const SeqInfo &s, int rt, int tpi) {
  int t0, t1;
  tile_tokens<ROWS>(rt, s.nq, p.G, tpi, t0, t1);
  return key_span<KL>(p, s, t0, t1);
}
// Key tiles of all row tiles of one key/value head.
template <int ROWS, int KL>
__device__ inline long long head_tiles(const PagedParams &p, const SeqInfo &s, int tpi) {
  const int R = tile_count<ROWS>(s.nq, p.G, tpi);
  if (!p.causal) return R > 0 ? static_cast<long long>(R) * key_span<KL>(p, s, 0, 0).n : 0;
  long long n = 0;
  for (int rt = 0; rt < R; ++rt) n += tile_span<ROWS, KL>(p, s, rt, tpi).n;
  return n;
}

// Up to 32 sequences of few row tiles: each warp makes its own copy of the sums
// (in `mine`, PLAN_WARP bytes of shared memory), a lane a sequence, and the
// block need not meet.  One sequence: 12.8 -> 12.2 us a call; a prefix of 16
// sequences, 28 -> 26.7.
constexpr int PLAN_WARP = 33 * 8 + 8 + 32 * 16;
template <int ROWS, int KL>
__device__ inline void make_warp_plan(const PagedParams &p, int tpi, uint8_t *mine, long long *&first, SeqInfo *&info) {
  first = reinterpret_cast<long long *>(mine);
  info = reinterpret_cast<SeqInfo *>(mine + 33 * 8 + 8);
  const int lane = threadIdx.x & 31;
  long long x = 0;
  if (lane < p.n_seqs) {
    const SeqInfo s = seq_info(p, lane);
    info[lane] = s;
    x = head_tiles<ROWS, KL>(p, s, tpi) * (p.hk / p.hp);
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  first[lane + 1] = x;
  if (lane == 0) first[0] = 0;
  __syncwarp();
}

// The flat list's prefix sums, first[b] = key tiles before sequence b, for
// every thread of a CTA of NT threads; first has n_seqs + 1 entries in shared
// memory, info (null: sequences are read again where needed) n_seqs.  `scan`
// holds NT / 32 + 1 values.  Few sequences: a warp each, its lanes share the
// row tiles; else a thread takes one or several.
template <int ROWS, int KL, int NT>
__device__ inline void make_plan(const PagedParams &p, int tpi, long long *first, SeqInfo *info,
                                 long long *scan) {
  const int per = (p.n_seqs + NT - 1) / NT, b0 = min(p.n_seqs, static_cast<int>(threadIdx.x) * per),
            b1 = min(p.n_seqs, b0 + per), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool by_warp = p.n_seqs <= NT / 32;
  if (by_warp && warp < p.n_seqs) {
    const SeqInfo s = seq_info(p, warp);
    const int R = tile_count<ROWS>(s.nq, p.G, tpi);
    long long n = 0;
    for (int rt = lane; rt < R; rt += 32) n += tile_span<ROWS, KL>(p, s, rt, tpi).n;
#pragma unroll
    for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    if (lane == 0) {
      if (info) info[warp] = s;
      first[warp + 1] = n * (p.hk / p.hp);
    }
  }
  if (by_warp) __syncthreads();
  long long sum = 0;
  for (int b = b0; b < b1; ++b) {
    if (by_warp) {
      sum += first[b + 1];
      continue;
    }
    const SeqInfo s = seq_info(p, b);
    if (info) info[b] = s;
    const long long n = head_tiles<ROWS, KL>(p, s, tpi) * (p.hk / p.hp);
    first[b + 1] = n;
    sum += n;
  }
  long long x = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) scan[warp] = x;
  __syncthreads();
  long long base = x - sum;
  for (int w = 0; w < warp; ++w) base += scan[w];
  if (threadIdx.x == 0) first[0] = 0;
  for (int b = b0; b < b1; ++b) {
    base += first[b + 1];
    first[b + 1] = base;
  }
  __syncthreads();
}

// SMs of this pass, of `sms`: a function of the sequences' lengths alone, summed in
// whole numbers, so that both passes come to one answer whatever their NT.  All NT
// threads of the block come here; `sums` has NT / 32 places.  Out of line: in line
// it cost the calls that do not share 0.4 to 1.5 us.
template <int NT>
__device__ __noinline__ int my_sms(const PagedParams &p, int sms, longlong2 *sums) {
  long long keys[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const Share::Side &s = p.share.of[k];
    long long n = 0;
    for (int b = threadIdx.x; b < s.n; b += NT) {
      const int slot = s.seqs ? s.seqs[b] : b;
      if (slot >= 0 && slot < s.n_slots) n += min(max(s.lens[slot], 0), s.max_len);
    }
    keys[k] = n;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    keys[0] += __shfl_xor_sync(0xffffffffu, keys[0], o);
    keys[1] += __shfl_xor_sync(0xffffffffu, keys[1], o);
  }
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = make_longlong2(keys[0], keys[1]);
  __syncthreads();
  keys[0] = keys[1] = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    keys[0] += sums[w].x;
    keys[1] += sums[w].y;
  }
  const Share::Side &f = p.share.of[0], &g = p.share.of[1];
  const float a = __fmaf_rn(static_cast<float>(keys[0]), f.cost, f.base), b = __fmaf_rn(static_cast<float>(keys[1]), g.cost, g.base);
  const int u = p.share.unit, most = (sms - 1) / u;      // at least one unit, and one SM for the other
  const int first = u * min(max(static_cast<int>(sms * (a / (a + b)) / u + 0.5f), 1), most);
  return p.share.side == 1 ? first : sms - first;
}

__device__ __forceinline__ long long span_of(long long total, int n_spans) {
  const long long s = (total + n_spans - 1) / n_spans;
  return s > 1 ? s : 1;
}

// A place in the flat list: key tile i of row tile rt of head group h of sequence b.
template <int ROWS, int KL>
struct Walk {
  int b, h, rt, R, i;
  SeqInfo s;
  Span sp;
  __device__ __forceinline__ void load(const PagedParams &p, const SeqInfo *info, int tpi) {
    s = info ? info[b] : seq_info(p, b);
    R = tile_count<ROWS>(s.nq, p.G, tpi);
  }
  // flat < first[n_seqs]
  __device__ inline void seek(const PagedParams &p, const long long *first, const SeqInfo *info, int tpi,
                              long long flat) {
    int lo = 0, hi = p.n_seqs;          // first[lo] <= flat < first[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first[mid] <= flat) lo = mid;
      else hi = mid;
    }
    b = lo;
    load(p, info, tpi);
    long long rem = flat - first[b];
    const long long per = (first[b + 1] - first[b]) / (p.hk / p.hp);
    h = static_cast<int>(rem / per);
    rem -= h * per;
    rt = 0;
    if (!p.causal) {
      sp = key_span<KL>(p, s, 0, 0);
      rt = static_cast<int>(rem / sp.n);
      rem -= static_cast<long long>(rt) * sp.n;
    } else {
      for (;; ++rt) {
        sp = tile_span<ROWS, KL>(p, s, rt, tpi);
        if (rem < sp.n) break;
        rem -= sp.n;
      }
    }
    i = static_cast<int>(rem);
  }
  // To the next key tile; the caller knows that there is one.
  __device__ inline void next(const PagedParams &p, const long long *first, const SeqInfo *info, int tpi) {
    if (++i < sp.n) return;
    i = 0;
    do {
      if (++rt == R) {
        rt = 0;
        if (++h == p.hk / p.hp) {
          h = 0;
          do ++b;
          while (first[b + 1] == first[b]);
          load(p, info, tpi);
        }
      }
      sp = tile_span<ROWS, KL>(p, s, rt, tpi);
    } while (sp.n == 0);
  }
};

// What worker `worker` (of span `at`, [from, to)) leaves for head h of the item
// that w stands in, whose key tile w.i is the span's last.
template <int ROWS, int KL>
__device__ __forceinline__ void leave_cut(const PagedParams &p, const Walk<ROWS, KL> &w, int tpi, int h, long long worker,
                                          long long at, long long span, long long from, long long to) {
  Cut c = {};
  if (from < to) {
    const long long f0 = to - 1 - w.i, f1 = f0 + w.sp.n;
    if (f0 >= from && f1 > to) {
      c.q0 = w.s.q0;
      c.h = h;
      c.x0 = ROWS > 0 ? w.rt * ROWS : w.rt * tpi * p.G;
      c.rows = ROWS > 0 ? min(ROWS, w.s.nq * p.G - c.x0) : min(tpi, w.s.nq - w.rt * tpi) * p.G;
      c.np = static_cast<int>((f1 - 1) / span - at) + 1;
      c.slot0 = f0 == from ? 0 : 1;
    }
  }
  p.cuts[worker] = c;
}

// One row's summary (m in log2 units, l) made final: the factor of its
// unnormalised O, and its lse.
__device__ __forceinline__ void row_final(float m, float l, float &fo, float &lse) {
  fo = l > 0.f ? 1.f / l : 0.f;
  lse = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
  if (!(l == l)) fo = lse = l;      // what is not a number stays so
}
// A column of a finished row: fo = 0 is a row that sees nothing, whose O is not
// zero where a value that other rows see is not finite.
__device__ __forceinline__ float finished(float o, float fo) { return fo == 0.f ? 0.f : o * fo; }

// Writes columns c, c+1 of a finished row.
template <int D>
__device__ __forceinline__ void store_pair(const PagedParams &p, long long row, int c, float x, float y) {
  const long long at = row * D + c;
  if (p.out_f32)
    *reinterpret_cast<float2 *>(static_cast<float *>(p.out) + at) = make_float2(x, y);
  else
    *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.out) + at) = pack_bf16x2(x, y);
}

// Pieces of the item that starts at flat index f0 in span `at`, [from, ..): their number, and the slot of the first (np = 0: it ends there).
__device__ __forceinline__ void item_pieces(long long f0, int n, long long at, long long span, long long from,
                                            int &np, int &slot0) {
  np = static_cast<int>((f0 + n - 1) / span - at) + 1;
  slot0 = f0 == from ? 0 : 1;
  if (np == 1) np = 0;
}

// Rows of items without a key tile: their sequences see nothing (here).
template <int D, int ROWS, int KL>
__device__ inline void finish_empty(const PagedParams &p, const SeqInfo *info, int tpi, int blocks) {
  for (int b = blockIdx.x; b < p.n_seqs; b += blocks) {
    const SeqInfo s = info ? info[b] : seq_info(p, b);
    // causal rows see more keys the later they stand: the empty tiles come first
    for (int rt = 0; rt < tile_count<ROWS>(s.nq, p.G, tpi); ++rt) {
      int a, z;
      tile_tokens<ROWS>(rt, s.nq, p.G, tpi, a, z);
      if (key_span<KL>(p, s, a, z).n > 0) break;
      const int rows = ROWS > 0 ? min(ROWS, s.nq * p.G - rt * ROWS) : (z - a + 1) * p.G;
      for (long long x = threadIdx.x; x < static_cast<long long>(rows) * p.hk * (D / 2); x += blockDim.x) {
        const int c = static_cast<int>(x % (D / 2)) * 2, y = static_cast<int>(x / (D / 2)), h = y / rows,
                  r = y - h * rows + (ROWS > 0 ? rt * ROWS : a * p.G);
        const int t = r / p.G, head = h * p.G + r - t * p.G;
        const long long row = static_cast<long long>(s.q0 + t) * p.hq + head;
        if (p.rec) {
          if (c == 0) p.rec[row] = Rec4{0, 0, REC_EMPTY, 0};
          continue;
        }
        store_pair<D>(p, row, c, 0.f, 0.f);
        if (c == 0) p.lse[static_cast<long long>(head) * p.n_tokens + s.q0 + t] = -INFINITY;
      }
    }
  }
}

}  // namespace attn
