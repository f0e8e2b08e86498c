// Attention over a paged cache for few rows per key/value head: tiles of 16
// rows on warp-level matrix instructions, bound by the cache's bandwidth.
//
// One row of a decode step does 4 d flops per key read of 4 d bytes; with the
// G query heads of a group that is G flops a byte, some 70 times below what
// this GPU needs to be bound by arithmetic at G = 4.  So the kernel is a
// stream: every warp owns a contiguous span of slabs of the flat list (see
// paged_plan.cuh) and a ring of slabs in shared memory that it alone fills
// (cp.async, 16 bytes a lane, rows of keys with their 16-byte words
// xor-swizzled so that ldmatrix meets no bank conflict) and reads.  Warps never
// wait for each other.  Each 16 keys of a slab lie in one page (pages are
// powers of two of at least 16 tokens), so their address takes one table
// entry, fetched a slab ahead.
//
// The 8 warps of a CTA take neighbouring heads of the same keys, whose rows lie
// side by side in a page: a CTA reads runs of 1 to 2 KB a token instead of 128
// or 256 bytes.  At 2.9 GB of keys and values that took 33 us off the 441 of the
// kernel (a call now 412, 7.0 TB/s), at 250 MB of 64-column heads 5 off 52.  64
// sequences with a window of 4096 (763 MB): 119 us, 6.4 TB/s, 95 % of what a plain
// copy reaches.  One sequence (1028 keys) takes 12 us, all of it latency: the
// launch, then slot, length, table entry and keys one after the other, then the
// join.
// Up to 16 rows.  At 24 rows a variant of two warps to a ring took 110 us against
// the 98 of the tensor-core tiles (16 sequences of 8192 keys, 8 heads of 128), at
// 48 rows 211 against 101, which is why the rule between them stays at 16.
//
// Keys that no row of an item sees (behind the sequence's end, before the
// window) are filled with zeros instead of being read: what memory holds there
// (NaN, other sequences' tokens) must not meet the zero weights of the P V
// product.
//
// Numerics: scores, running maximum, sum and O in 32 bits; P is rounded to
// bf16 for the product with V (half a step, 2^-8 relative, of each weight; the
// row sum takes the unrounded values), as in attn_fwd.  The maximum is only
// raised when it grew by more than 8 (log2), so P stays below 2^8.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "attn_internal.h"
#include "paged_join.cuh"
#include "paged_plan.cuh"

namespace attn {

constexpr int PR_ROWS = 16;
constexpr int PR_WARPS = 8;        // warps of a CTA (12 at head dim 64: no faster)
constexpr float PR_TAU = 8.0f;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A slab is 16 keys at head dim 128 and 32 at 64: 8 KB of keys and values.
__host__ __device__ constexpr int rows_kl(int d) { return d == 128 ? 4 : 5; }

// What the fetching side of a warp tells its computing side about a slab.
struct __align__(16) Slab {
  int key0, i, n, h;          // first key; key tile i of the item's n; head
  int rt, q0, nq, len;        // row tile; the sequence's tokens and length
};

template <int D, int NST>
struct RowsSmem {
  static constexpr int W = PR_WARPS;
  static constexpr int KEYS = 1 << rows_kl(D);
  static constexpr int PART = KEYS * D * 2;                     // keys or values of one slab
  static constexpr int RING = W * NST * 2 * PART;
  static constexpr int NOTE = RING;                             // Slab [W][NST]
  static constexpr int SCAN = NOTE + W * NST * static_cast<int>(sizeof(Slab));
  static constexpr int FIRST = SCAN + (W + 2) / 2 * 16;
  static size_t bytes(const PagedParams &p) {
    return FIRST + (p.warp_plan ? static_cast<size_t>(W) * PLAN_WARP : 8ull * (p.n_seqs + 1) + sizeof(SeqInfo) * p.n_seqs);
  }
};

template <int D, int NST>
__global__ void __launch_bounds__(PR_WARPS * 32, 1) paged_rows_kernel(const PagedParams p) {
  using S = RowsSmem<D, NST>;
  constexpr int KL = rows_kl(D), KEYS = S::KEYS, NSUB = KEYS / 16, NB = KEYS / 8;
  constexpr int NOT_SEEN = INT_MIN;
  extern __shared__ __align__(256) uint8_t rows_smem[];
  long long *scan = reinterpret_cast<long long *>(rows_smem + S::SCAN);
  long long *first = reinterpret_cast<long long *>(rows_smem + S::FIRST);
  SeqInfo *info = reinterpret_cast<SeqInfo *>(first + p.n_seqs + 1);
  if (!p.wait_end) after_previous();
  admit_next();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int sms = gridDim.x;
  if (p.share.side) {
    sms = my_sms<S::W * 32>(p, sms, reinterpret_cast<longlong2 *>(rows_smem));
    if (static_cast<int>(blockIdx.x) >= sms) {
      end_after_previous(p);
      return;
    }
    __syncthreads();
  }
  if (p.warp_plan) make_warp_plan<PR_ROWS, KL>(p, 0, rows_smem + S::FIRST + warp * PLAN_WARP, first, info);
  else make_plan<PR_ROWS, KL, S::W * 32>(p, 0, first, info, scan);
  finish_empty<D, PR_ROWS, KL>(p, info, 0, sms);

  const int n_spans = p.share.side ? sms * S::W / p.hp : p.n_spans;
  const long long total = first[p.n_seqs], span = span_of(total, n_spans);
  const long long worker = static_cast<long long>(blockIdx.x) * S::W + warp, span_no = worker / p.hp;
  const int sub = static_cast<int>(worker - span_no * p.hp);    // this warp's head of a group
  const long long from = min(span_no * span, total), to = min(total, from + span);
  if (from >= to) {
    if (lane == 0 && !p.rec) p.cuts[worker] = Cut{};
    end_after_previous(p);
    return;
  }
  const int cnt = static_cast<int>(to - from);

  const uint32_t ring = smem_u32(rows_smem) + warp * (NST * 2 * S::PART);
  Slab *note = reinterpret_cast<Slab *>(rows_smem + S::NOTE) + warp * NST;
  Walk<PR_ROWS, KL> in;            // the slab to be fetched next
  in.seek(p, first, info, 0, from);
  int in_lo, in_end;               // keys that some row of its item sees (and the first ones)
  auto bounds = [&]() {
    int t0, t1;
    tile_tokens<PR_ROWS>(in.rt, in.s.nq, p.G, 0, t0, t1);
    const int pos0 = in.s.len - in.s.nq;
    in_end = p.causal ? pos0 + t1 + 1 : in.s.len;
    in_lo = p.causal && p.window > 0 ? max(0, pos0 + t0 - p.window + 1) : 0;
  };
  bounds();
  const int page_mask = (1 << p.page_shift) - 1;
  int page[NSUB];                  // of each 16 keys, read a slab ahead
  auto look_up = [&]() {
#pragma unroll
    for (int j = 0; j < NSUB; ++j) {
      const int k0 = (in.sp.tile(in.i) << KL) + 16 * j;
      if (j > 0 && p.page_shift > 4) {
        page[j] = k0 < in_end ? page[0] : NOT_SEEN;
      } else if (NSUB == 1 || (k0 < in_end && (k0 + (1 << p.page_shift) > in_lo || k0 < p.sinks))) {
        page[j] = p.table[in.s.slot * p.table_stride + (k0 >> p.page_shift)];
      } else {
        page[j] = NOT_SEEN;
      }
    }
  };
  look_up();
  constexpr int CH = D / 8, RPI = 32 / CH;                 // 16-byte words a row, rows an instruction
  const int fc = lane % CH, fr = lane / CH;
  const long long lane_off = (fr * p.token_stride + fc * 8) * 2, row_step = RPI * p.token_stride * 2;
  const char *kbase = static_cast<const char *>(p.k) + lane_off, *vbase = static_cast<const char *>(p.v) + lane_off;
  const uint32_t lane_dst = fr * (D * 2) + ((fc ^ fr) << 4);
  // fetches slab n of this worker, where `in` stands, and steps on
  auto fetch = [&](int n) {
    if (n < cnt) {
      const int key0 = in.sp.tile(in.i) << KL, slot = n % NST;
      const uint32_t dst = ring + slot * (2 * S::PART) + lane_dst;
      if (lane == 0) {
        note[slot] = Slab{key0, in.i, in.sp.n, in.h * p.hp + sub, in.rt, in.s.q0, in.s.nq, in.s.len};
      }
#pragma unroll
      for (int j = 0; j < NSUB; ++j) {
        const int k0 = key0 + 16 * j;
        const bool good = page[j] >= 0 && page[j] < p.n_pages;
        if (!good && page[j] != NOT_SEEN && lane == 0) paged_fail(p, ATTN_ERR_INVALID_ARG);
        // rows that some row of the item sees; the others are zeros, not read
        const unsigned seen = good ? bits_below(min(max(in_end - k0, 0), 16)) &
                                         (~bits_below(min(max(in_lo - k0, 0), 16)) | bits_below(min(max(p.sinks - k0, 0), 16)))
                                   : 0u;
        const unsigned mine = seen >> fr;
        const long long at = good ? (page[j] * p.page_stride + (k0 & page_mask) * p.token_stride + (in.h * p.hp + sub) * p.head_stride) * 2 : 0;
        const char *ks = kbase + at, *vs = vbase + at;
#pragma unroll
        for (int i = 0; i < 16 / RPI; ++i) {
          const int r = i * RPI;
          const uint32_t d = (dst ^ ((r & 7) << 4)) + (16 * j + r) * (D * 2);
          const bool live = mine >> r & 1u;
          cp_async16(d, live ? ks + i * row_step : p.k, live ? 16u : 0u);
          cp_async16(d + S::PART, live ? vs + i * row_step : p.v, live ? 16u : 0u);
        }
      }
      if (n + 1 < cnt) {
        in.next(p, first, info, 0);
        if (in.i == 0) bounds();
        look_up();
      }
    }
    cp_commit();
  };
#pragma unroll 1
  for (int n = 0; n < NST - 1; ++n) fetch(n);
  __syncwarp();

  uint32_t qf[D / 16][4];
  float o[D / 8][4];
  float m0 = 0.f, m1 = 0.f, l0 = 0.f, l1 = 0.f;
  int pos0 = -1, pos1 = -1, lo0 = 0, lo1 = 0;      // last key a row sees, first of its window
  int all_lo = 0, all_hi = 0;                      // keys in [all_lo, all_hi) are seen by every row
  long long row0 = -1, row1 = -1;                  // (token * hq + head), -1: no row
  int rows_here = 0, piece0 = 0;
  const float sl2 = p.scale_log2;
  const int lr = lane >> 2, lc = (lane & 3) * 2;
  // this lane's places in the keys and (transposed) the values of a slab
  const uint32_t k_place = (((lane >> 4) << 3) + (lane & 7)) * (D * 2) + ((((lane >> 3) & 1) ^ (lane & 7)) << 4);
  const uint32_t v_place = ((((lane >> 3) & 1) << 3) + (lane & 7)) * (D * 2) + (((lane >> 4) ^ (lane & 7)) << 4);

#pragma unroll 1
  for (int n = 0; n < cnt; ++n) {
    // with three slots a slab's note was left before the __syncwarp of the step before; with two, after it
    if constexpr (NST == 2) __syncwarp();
    const Slab &sl = note[n % NST];
    const int key0 = sl.key0, tile_i = sl.i, tile_n = sl.n;
    if (n == 0 || tile_i == 0) {
      // a new item: its rows of Q as matrix fragments, requested while its keys
      // are on their way; summaries empty
      const int rt = sl.rt, q0 = sl.q0, nq = sl.nq, len = sl.len, h = sl.h;
      piece0 = tile_i;
      rows_here = min(PR_ROWS, nq * p.G - rt * PR_ROWS);
      auto place = [&](int r, long long &row, int &pos, int &lo) {
        row = -1;
        pos = -1;
        lo = 0;
        if (r < rows_here) {
          const int x = rt * PR_ROWS + r, t = x / p.G;
          row = static_cast<long long>(q0 + t) * p.hq + h * p.G + x - t * p.G;
          pos = p.causal ? len - nq + t : len - 1;
          lo = p.causal && p.window > 0 ? pos - p.window + 1 : 0;
        }
      };
      place(lr, row0, pos0, lo0);
      place(lr + 8, row1, pos1, lo1);
      int t0, t1;
      tile_tokens<PR_ROWS>(rt, nq, p.G, 0, t0, t1);
      all_hi = p.causal ? len - nq + t0 + 1 : len;
      all_lo = p.causal && p.window > 0 ? len - nq + t1 - p.window + 1 : 0;
      const uint16_t *qa = static_cast<const uint16_t *>(p.q) + (row0 < 0 ? 0 : row0) * D + lc;
      const uint16_t *qb = static_cast<const uint16_t *>(p.q) + (row1 < 0 ? 0 : row1) * D + lc;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        qf[k][0] = row0 < 0 ? 0u : *reinterpret_cast<const uint32_t *>(qa + k * 16);
        qf[k][1] = row1 < 0 ? 0u : *reinterpret_cast<const uint32_t *>(qb + k * 16);
        qf[k][2] = row0 < 0 ? 0u : *reinterpret_cast<const uint32_t *>(qa + k * 16 + 8);
        qf[k][3] = row1 < 0 ? 0u : *reinterpret_cast<const uint32_t *>(qb + k * 16 + 8);
      }
      m0 = m1 = -INFINITY;
      l0 = l1 = 0.f;
#pragma unroll
      for (int j = 0; j < D / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
    }
    cp_wait<NST - 2>();
    __syncwarp();
    fetch(n + NST - 1);
    const uint32_t ks = ring + (n % NST) * (2 * S::PART), vs = ks + S::PART;
    // S = Q K^T: 16 rows x KEYS keys, in blocks of 8 keys; x[b][0..1] row lr, x[b][2..3] row lr + 8
    float x[NB][4];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[b][e] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
#pragma unroll
      for (int j = 0; j < NSUB; ++j) {
        uint32_t b[4];
        ldsm4(((ks + k_place) ^ (k << 5)) + j * 16 * (D * 2), b);
        mma16816(x[2 * j], qf[k], b[0], b[1]);
        mma16816(x[2 * j + 1], qf[k], b[2], b[3]);
      }
    }
    if (key0 + KEYS > all_hi || (key0 < all_lo && key0 + KEYS > p.sinks)) {
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int j = key0 + b * 8 + lc + e;
          if (!(j <= pos0 && (j >= lo0 || j < p.sinks))) x[b][e] = -INFINITY;
          if (!(j <= pos1 && (j >= lo1 || j < p.sinks))) x[b][2 + e] = -INFINITY;
        }
    }
    float a0 = -INFINITY, a1 = -INFINITY;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      a0 = max3f(a0, x[b][0], x[b][1]);
      a1 = max3f(a1, x[b][2], x[b][3]);
    }
    a0 = fmaxf(a0, __shfl_xor_sync(0xffffffffu, a0, 1));
    a1 = fmaxf(a1, __shfl_xor_sync(0xffffffffu, a1, 1));
    a0 = fmaxf(a0, __shfl_xor_sync(0xffffffffu, a0, 2)) * sl2;
    a1 = fmaxf(a1, __shfl_xor_sync(0xffffffffu, a1, 2)) * sl2;
    const bool g0 = a0 > m0 + PR_TAU, g1 = a1 > m1 + PR_TAU;
    if (__any_sync(0xffffffffu, g0 || g1)) {
      const float f0 = g0 ? ex2_approx(m0 - a0) : 1.f, f1 = g1 ? ex2_approx(m1 - a1) : 1.f;
      if (g0) m0 = a0;
      if (g1) m1 = a1;
      l0 *= f0;
      l1 *= f1;
#pragma unroll
      for (int j = 0; j < D / 8; ++j) {
        o[j][0] *= f0;
        o[j][1] *= f0;
        o[j][2] *= f1;
        o[j][3] *= f1;
      }
    }
    const float b0 = m0 == -INFINITY ? 0.f : -m0, b1 = m1 == -INFINITY ? 0.f : -m1;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      x[b][0] = ex2_approx(fmaf(x[b][0], sl2, b0));
      x[b][1] = ex2_approx(fmaf(x[b][1], sl2, b0));
      x[b][2] = ex2_approx(fmaf(x[b][2], sl2, b1));
      x[b][3] = ex2_approx(fmaf(x[b][3], sl2, b1));
      l0 += x[b][0] + x[b][1];
      l1 += x[b][2] + x[b][3];
    }
    // O += P V
#pragma unroll
    for (int j = 0; j < NSUB; ++j) {
      const uint32_t pf[4] = {pack_bf16x2(x[2 * j][0], x[2 * j][1]), pack_bf16x2(x[2 * j][2], x[2 * j][3]),
                              pack_bf16x2(x[2 * j + 1][0], x[2 * j + 1][1]), pack_bf16x2(x[2 * j + 1][2], x[2 * j + 1][3])};
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        uint32_t b[4];
        ldsm4t(((vs + v_place) ^ (c << 5)) + j * 16 * (D * 2), b);
        mma16816(o[2 * c], pf, b[0], b[1]);
        mma16816(o[2 * c + 1], pf, b[2], b[3]);
      }
    }
    const bool ends = tile_i == tile_n - 1;
    if (ends || n == cnt - 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
      l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
      if (p.rec && piece0 == 0 && lc == 0) {
        int np, slot0;
        item_pieces(from + n - tile_i, tile_n, span_no, span, from, np, slot0);
        if (row0 >= 0) p.rec[row0] = Rec4{static_cast<int>(worker), slot0, np, lr};
        if (row1 >= 0) p.rec[row1] = Rec4{static_cast<int>(worker), slot0, np, lr + 8};
      }
      const bool whole = ends && piece0 == 0;
      if (whole && !p.rec) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const long long row = u ? row1 : row0;
          if (row < 0) continue;
          float fo, lse;
          row_final(u ? m1 : m0, u ? l1 : l0, fo, lse);
#pragma unroll
          for (int j = 0; j < D / 8; ++j) store_pair<D>(p, row, j * 8 + lc, finished(o[j][2 * u], fo), finished(o[j][2 * u + 1], fo));
          if (lc == 0) {
            const int t = static_cast<int>(row / p.hq), head = static_cast<int>(row - static_cast<long long>(t) * p.hq);
            p.lse[static_cast<long long>(head) * p.n_tokens + t] = lse;
          }
        }
      } else {
        // to the dense arrays, or to a piece: slot 0 the one a span begins
        // with, slot 1 one that begins in it and goes on
        const long long slot = worker * 2 + (n - (tile_i - piece0) == 0 ? 0 : 1);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (lr + 8 * u >= rows_here) continue;
          const long long r = whole ? (u ? row1 : row0) : slot * PR_ROWS + lr + 8 * u;
          float *po = (whole ? p.dense_o : p.part_o) + r * D + lc;
#pragma unroll
          for (int j = 0; j < D / 8; ++j) *reinterpret_cast<float2 *>(po + j * 8) = make_float2(o[j][2 * u], o[j][2 * u + 1]);
          if (lc == 0) *reinterpret_cast<float2 *>((whole ? p.dense_ml : p.part_ml) + r * 2) = make_float2(u ? m1 : m0, u ? l1 : l0);
        }
      }
    }
  }
  if (lane == 0 && !p.rec) leave_cut<PR_ROWS, KL>(p, in, 0, in.h * p.hp + sub, worker, span_no, span, from, to);
  end_after_previous(p);
}

// ---------------------------------------------------------------------- host

template <int D, int NST>
static int launch_rows(PagedParams &p, cudaStream_t s) {
  using S = RowsSmem<D, NST>;
  constexpr int kDev = 64;
  static bool done[kDev] = {};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDev) return ATTN_ERR_CUDA;
  auto kern = paged_rows_kernel<D, NST>;
  auto join = paged_join_kernel<D, PR_ROWS, true>;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (raise_smem(kern, kSmemMax, &done[dev]) != ATTN_OK) return ATTN_ERR_CUDA;
  }
  const int sms = device_sm_count();
  if (sms <= 0) return ATTN_ERR_CUDA;
  // as many heads side by side as divide both the heads and a CTA's warps
  p.hp = 1;
  while (p.hp < S::W && p.hk % (2 * p.hp) == 0) p.hp *= 2;
  p.n_spans = sms * S::W / p.hp;
  p.warp_plan = p.n_seqs <= 32 && (!p.causal || static_cast<long long>(p.n_tokens) * p.G <= 64 * PR_ROWS);
  const int rc = launch_after(kern, dim3(sms), S::W * 32, S::bytes(p), s, p);
  if (rc != ATTN_OK || p.rec) return rc;
  // few items: each has many pieces, and its rows go to blocks of their own
  const long long items = static_cast<long long>(p.n_seqs) * p.hk;
  return launch_after(join, dim3(sms * S::W, items * 8 < sms * S::W ? 4 : 1), 256, 0, s, p);
}

// Floats of all workers' pieces of `tile_rows` rows.
size_t paged_piece_floats(int tile_rows, int d) {
  return static_cast<size_t>(device_sm_count()) * (tile_rows == PR_ROWS ? PR_WARPS : 1) * 2 * tile_rows * d;
}

size_t paged_rows_workspace(int d) {
  const int sms = device_sm_count();
  if (sms <= 0) return 0;
  return static_cast<size_t>(sms) * PR_WARPS * (2 * PR_ROWS * (d + 2) * sizeof(float) + sizeof(Cut));
}

int paged_rows_launch(PagedParams &p, int d, cudaStream_t s) {
  const int sms = device_sm_count();
  if (sms <= 0) return ATTN_ERR_CUDA;
  p.part_ml = p.part_o + paged_piece_floats(PR_ROWS, d);
  p.cuts = reinterpret_cast<Cut *>(p.part_ml + static_cast<size_t>(sms) * PR_WARPS * 2 * PR_ROWS * 2);
  // a ring of 192 KB, or 128 where thousands of sequences take the room
  const bool many = p.n_seqs > 1024;
  if (d == 128) return many ? launch_rows<128, 2>(p, s) : launch_rows<128, 3>(p, s);
  return many ? launch_rows<64, 2>(p, s) : launch_rows<64, 3>(p, s);
}

}  // namespace attn
