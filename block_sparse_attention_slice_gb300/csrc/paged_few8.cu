// Attention over a paged cache in 8 bits for up to 8 rows per key/value head, a decode
// step's: the stream of paged_rows.cu, whose plan, rings and pieces it has, over codes of
// one byte with a scale for each token and head.
//
// What bounds it.  A byte read now costs a conversion to a 16-bit operand, and
// the integer and conversion units take 2 cycles a warp's instruction on each of
// an SM's four schedulers (measured), as a product of 16 x 8 x 16 takes 8: at 22
// bytes a cycle and SM, what the cache's bandwidth comes to, a code has 5.8 lane
// operations of those units in all.  So
//   - keys and columns of values are the 16 rows of a product, the queries its 8
//     columns: S^T = K Q^T and O^T = V^T P^T.  A decode step has 4 to 8 rows of Q a
//     key/value head; with them as the 16 rows (16 x 8 keys) twice the products and
//     half of all softmax work went to rows that are not there, and twice the registers,
//     which left room for 8 warps where 12 hide more latency (64 sequences, window 4096:
//     104 us so, 84 now).  P^T comes out of the scores by transposing 8 x 8 matrices in registers;
//   - operands are f16, not bf16: e4m3 converts by one instruction a pair, int8 by
//     one logical operation and one addition (bf16 would take four);
//   - a lane reads 16 codes at once and they are its operands as they lie: the sum
//     over d and the columns of O may be taken in any order that both operands agree
//     on.  Of 64 columns of a key lane c of its four takes 16 in a row, for four
//     products; of the values it takes 16 (8) columns in a row of each of its keys, so
//     that two rows' words make operands by one byte permutation a pair;
//   - slabs are fetched by TMA, one box of a slab's keys or values for each page, whose
//     swizzle serves the reads (two lanes of eight meet a bank twice where keys are
//     read): 9 % fewer instructions than copies of 16 bytes.
//
// 16 sequences of 8191 to 131072 tokens, e4m3, 4 heads to each of 8 of 128 columns: 1.5 GB in
// 232 us with the join, 6.5 TB/s.  64 with a window of 4096, int8: 394 MB in 84 us; 46 % of the issue
// slots and 43 % of the converting unit: no path is full, a sixth of the waits are for instructions (branches
// marked unlikely changed nothing).
//
// Numerics.  Codes become f16 exactly.  A row of Q becomes f16 times a power of
// two that brings its largest value to 2^14 .. 2^15: exact but for values 2^-29
// below that one, which are off by 2^-40 of it at most.  Scores are f32 and take
// the key's scale and the row's power of two there.  The weight of a value is
// w = p vs; it is rounded to f16 (half a step, 2^-11 relative) times a power of
// two of its row, chosen so that the largest w lies between 1 and 2^15; weights
// below 2^-14 are off by 2^-25 at most.  Running maximum, sums and O are f32.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <mutex>

#include "attn_internal.h"
#include "codes.cuh"
#include "paged_join.cuh"
#include "paged_plan.cuh"
#include "warp8.cuh"

namespace attn {

constexpr int F8_ROWS = 8;
constexpr int F8_KL = 5;           // a slab is 32 keys
constexpr float F8_TAU = 8.0f;

namespace {

// A warp's wait for its own copies: false where it lasted over limit_ns.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
  bool ok = mbar_try_wait(bar, parity);
  if (!ok) {
    const uint64_t end = globaltimer_ns() + limit_ns;
    while (!(ok = mbar_try_wait(bar, parity)) && globaltimer_ns() < end) {
    }
  }
  return __all_sync(0xffffffffu, ok);
}

}  // namespace

// What the fetching side of a warp tells its computing side about a slab.
struct __align__(16) FewSlab {
  int key0, i, n, h;          // first key; key tile i of the item's n; head
  int rt, q0, nq, len;        // row tile; the sequence's tokens and length
  unsigned seen;              // bit k: some row of the item sees key key0 + k
  int pad[3];
};

template <int D, int NST, int W>
struct Few8Smem {
  static constexpr int KEYS = 1 << F8_KL;
  static constexpr int PART = KEYS * D, STAGE = 2 * PART;       // keys or values of one slab; both
  static constexpr int SCALES = W * NST * STAGE;                // [W][NST][keys', values'][KEYS]
  static constexpr int NOTE = SCALES + W * NST * 2 * KEYS * 4;  // FewSlab [W][NST]
  static_assert(W * NST * sizeof(FewSlab) >= W * 16, "my_sms puts its sums where the notes will be");
  static constexpr int BAR = NOTE + W * NST * static_cast<int>(sizeof(FewSlab));
  static constexpr int SCAN = BAR + (W * NST * 8 + 15) / 16 * 16;
  static constexpr int FIRST = SCAN + (W + 2) / 2 * 16;
  static size_t bytes(const PagedParams &p, bool infos) {
    return 1024 + FIRST + (p.warp_plan ? static_cast<size_t>(W) * PLAN_WARP : 8ull * (p.n_seqs + 1) + (infos ? sizeof(SeqInfo) * p.n_seqs : 0));
  }
};

// W: warps of a CTA.
template <int D, int NST, int W, int FMT>
__global__ void __launch_bounds__(W * 32, 1) paged_few8_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                                                               const PagedParams p, const int keep_infos) {
  using S = Few8Smem<D, NST, W>;
  using C = F16Codes<FMT>;
  constexpr int KL = F8_KL, KEYS = S::KEYS, NSUB = KEYS / 16;
  constexpr int NOT_SEEN = INT_MIN;
  extern __shared__ uint8_t few8_raw[];
  uint8_t *few8_smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(few8_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  long long *scan = reinterpret_cast<long long *>(few8_smem + S::SCAN);
  long long *first = reinterpret_cast<long long *>(few8_smem + S::FIRST);
  SeqInfo *info = keep_infos ? reinterpret_cast<SeqInfo *>(first + p.n_seqs + 1) : nullptr;
  if (!p.wait_end) after_previous();
  admit_next();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int sms = gridDim.x;
  if (p.share.side) {
    sms = my_sms<W * 32>(p, sms, reinterpret_cast<longlong2 *>(few8_smem + S::NOTE));      // not in the ring, which TMA writes
    if (static_cast<int>(blockIdx.x) >= sms) {
      end_after_previous(p);
      return;
    }
    __syncthreads();
  }
  if (p.warp_plan) make_warp_plan<F8_ROWS, KL>(p, 0, few8_smem + S::FIRST + warp * PLAN_WARP, first, info);
  else make_plan<F8_ROWS, KL, W * 32>(p, 0, first, info, scan);
  finish_empty<D, F8_ROWS, KL>(p, info, 0, sms);

  const int n_spans = p.share.side ? sms * W / p.hp : p.n_spans;
  const long long total = first[p.n_seqs], span = span_of(total, n_spans);
  const long long worker = static_cast<long long>(blockIdx.x) * W + warp, span_no = worker / p.hp;
  const int sub = static_cast<int>(worker - span_no * p.hp);    // this warp's head of a group
  const long long from = min(span_no * span, total), to = min(total, from + span);
  if (from >= to) {
    if (lane == 0 && !p.rec) p.cuts[worker] = Cut{};
    end_after_previous(p);
    return;
  }
  const int cnt = static_cast<int>(to - from);

  const uint32_t ring = smem_u32(few8_smem) + warp * (NST * S::STAGE), scale_ring = smem_u32(few8_smem) + S::SCALES + warp * (NST * 2 * KEYS * 4),
                 bars = smem_u32(few8_smem) + S::BAR + warp * (NST * 8);
  if (lane == 0) {
    for (int s = 0; s < NST; ++s) mbar_init(bars + 8 * s, 1);
    fence_mbar_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  FewSlab *note = reinterpret_cast<FewSlab *>(few8_smem + S::NOTE) + warp * NST;
  Walk<F8_ROWS, KL> in;            // the slab to be fetched next
  in.seek(p, first, info, 0, from);
  int in_lo, in_end;               // keys that some row of its item sees (and the first ones)
  auto bounds = [&]() {
    int t0, t1;
    tile_tokens<F8_ROWS>(in.rt, in.s.nq, p.G, 0, t0, t1);
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
      } else if (k0 < in_end && (k0 + (1 << p.page_shift) > in_lo || k0 < p.sinks)) {
        page[j] = p.table[in.s.slot * p.table_stride + (k0 >> p.page_shift)];
      } else {
        page[j] = NOT_SEEN;
      }
    }
  };
  look_up();
  const int box = min(1 << p.page_shift, KEYS);            // keys of a TMA box
  // fetches slab n of this worker, where `in` stands, and steps on
  auto fetch = [&](int n) {
    if (n < cnt) {
      const int key0 = in.sp.tile(in.i) << KL, slot = n % NST, head = in.h * p.hp + sub;
      const uint32_t stage = ring + slot * S::STAGE, bar = bars + 8 * slot;
      // what no row of the item sees: pages of it are read from outside the map, which
      // gives zeros, and their scales are 0
      const unsigned seen = bits_below(min(max(in_end - key0, 0), 32)) &
                            (~bits_below(min(max(in_lo - key0, 0), 32)) | bits_below(min(max(p.sinks - key0, 0), 32)));
#pragma unroll
      for (int j = 0; j < NSUB; ++j) {
        if (page[j] < 0 || page[j] >= p.n_pages) {
          if (page[j] != NOT_SEEN && lane == 0) paged_fail(p, ATTN_ERR_INVALID_ARG);
          page[j] = p.n_pages;
        }
      }
      if (lane == 0) {
        note[slot] = FewSlab{key0, in.i, in.sp.n, head, in.rt, in.s.q0, in.s.nq, in.s.len, seen, {}};
        mbar_arrive_expect_tx(bar, S::STAGE);
        const int tok = key0 & page_mask;
        // failure-path test only: the first slab's keys are left out, so that the wait for
        // them runs out
        if (!(p.test_stall && n == 0)) tma_load_4d(stage, &tm_k, bar, 0, tok, head, page[0]);
        tma_load_4d(stage + S::PART, &tm_v, bar, 0, tok, head, page[0]);
        if (box < KEYS) {
          tma_load_4d(stage + 16 * D, &tm_k, bar, 0, 0, head, page[NSUB - 1]);
          tma_load_4d(stage + S::PART + 16 * D, &tm_v, bar, 0, 0, head, page[NSUB - 1]);
        }
      }
      const int pg = lane < 16 ? page[0] : page[NSUB - 1];
      const bool live = (seen >> lane & 1u) && pg < p.n_pages;
      const long long at = live ? pg * p.scale_page + ((key0 + lane) & page_mask) * p.scale_token + head * p.scale_head : 0;
      const uint32_t sc = scale_ring + slot * (2 * KEYS * 4) + lane * 4;
      cp_async4(sc, p.k_scales + at, live ? 4u : 0u);
      cp_async4(sc + KEYS * 4, p.v_scales + at, live ? 4u : 0u);
      if (n + 1 < cnt) {
        in.next(p, first, info, 0);
        if (in.i == 0) bounds();
        look_up();
      }
    }
    cp_commit();
  };
  __syncwarp();
#pragma unroll 1
  for (int n = 0; n < NST - 1; ++n) fetch(n);
  __syncwarp();

  // This lane's rows are 2 c + e, with keys lr and lr + 8 of each 16; it shares them
  // with the lanes of equal c.  As the column of an operand it stands for row lr.
  // p = 2^(s - m), m the lazy maximum; a value's weight is p vs 2^lc (warp8.cuh).  unset, bit
  // e: no weight other than 0 has been met since m last grew, so lc may not suit what comes.
  uint32_t qf[D / 16][2];
  float o[D / 16][4];          // columns (D / 8) lr + 2 mb, of rows e = 0, 1, and the next one
  float m[2], l[2], rs[2], most[2];
  int lc[2];
  unsigned unset = 0;
  int all_lo = 0, all_hi = 0;      // keys in [all_lo, all_hi) are seen by every row
  int rows_here = 0, piece0 = 0, item_x0 = 0, item_q0 = 0, item_nq = 0, item_len = 0, item_h = 0;
  const int lr = lane >> 2, c = lane & 3;
  // token of the sequence and row of the output of the item's row r
  auto token_of = [&](int r, long long &row) -> int {
    const int x = item_x0 + r, t = x / p.G;
    row = static_cast<long long>(item_q0 + t) * p.hq + item_h * p.G + x - t * p.G;
    return t;
  };
  // This lane's words under TMA's swizzle (128 bytes: by the row; 64: by half of it).  Of a
  // block of 8 keys key lr; its halves of 64 columns are 64 bytes apart.
  auto word = [&](int row, int chunk) -> uint32_t { return row * D + ((chunk ^ (D == 128 ? row & 7 : (row >> 1) & 3)) << 4); };
  const uint32_t k_at = word(lr, c);
  // columns 16 lr .. (8 lr ..) of the values of its keys 2 c, 2 c + 1, and of those 8 on
  auto v_word = [&](int i) -> uint32_t {
    const int row = 2 * c + (i & 1) + 8 * (i >> 1);
    return D == 128 ? word(row, lr) : word(row, lr >> 1) + ((lr & 1) << 3);
  };
  const uint32_t v_at[4] = {v_word(0), v_word(1), v_word(2), v_word(3)};
  bool gave_up = false;

#pragma unroll 1
  for (int n = 0; n < cnt; ++n) {
    // with three slots a slab's note was left before the __syncwarp of the step before; with two, after it
    if constexpr (NST == 2) __syncwarp();
    const FewSlab &sl = note[n % NST];
    const int key0 = sl.key0, tile_i = sl.i, tile_n = sl.n;
    if (n == 0 || tile_i == 0) {
      // a new item: its rows of Q as f16 operands; summaries empty
      item_x0 = sl.rt * F8_ROWS, item_q0 = sl.q0, item_nq = sl.nq, item_len = sl.len, item_h = sl.h;
      piece0 = tile_i;
      rows_here = min(F8_ROWS, item_nq * p.G - item_x0);
      int t0, t1;
      tile_tokens<F8_ROWS>(sl.rt, item_nq, p.G, 0, t0, t1);
      all_hi = p.causal ? item_len - item_nq + t0 + 1 : item_len;
      all_lo = p.causal && p.window > 0 ? item_len - item_nq + t1 - p.window + 1 : 0;
      uint4 w[D / 64][2];
      long long row = 0;
      const bool on = lr < rows_here;
      if (on) token_of(lr, row);
      const uint16_t *qa = static_cast<const uint16_t *>(p.q) + row * D + 16 * c;
#pragma unroll
      for (int hh = 0; hh < D / 64; ++hh)
#pragma unroll
        for (int e = 0; e < 2; ++e) w[hh][e] = on ? *reinterpret_cast<const uint4 *>(qa + 64 * hh + 8 * e) : make_uint4(0u, 0u, 0u, 0u);
      uint32_t top = 0;
      const uint16_t *y = reinterpret_cast<const uint16_t *>(w);
#pragma unroll
      for (int k = 0; k < D / 4; ++k) top = max(top, y[k] & 0x7fffu);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^(14 - exponent of the largest), as far as an f32 power of two and its inverse go: -114 .. 100
      const int ex = min(141 - static_cast<int>(top >> 7), 100);
      const float f = pow2_of(ex);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint16_t *z = y + 4 * k;      // words 4 i .. of half k / 4: columns 64 (k / 4) + 16 c + 4 (k % 4)
        auto f16_of = [&](int a, int b) {
          return pack_f16x2(__uint_as_float(static_cast<uint32_t>(z[a]) << 16) * f, __uint_as_float(static_cast<uint32_t>(z[b]) << 16) * f);
        };
        qf[k][0] = f16_of(C::A0, C::A1);
        qf[k][1] = f16_of(C::B0, C::B1);
      }
      // the factors of this lane's own rows
#pragma unroll
      for (int e = 0; e < 2; ++e) rs[e] = p.scale_log2 * pow2_of(-__shfl_sync(0xffffffffu, ex, 4 * (2 * c + e)));
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[e] = -INFINITY;
        l[e] = 0.f;
        most[e] = 0.f;
        lc[e] = 0;
      }
#pragma unroll
      for (int mb = 0; mb < D / 16; ++mb)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mb][e] = 0.f;
      unset = 3u;
    }
    cp_wait<NST - 2>();
    if (!warp_wait(bars + 8 * (n % NST), (n / NST) & 1, p.wait_ns)) {
      gave_up = true;
      // what was issued lands before the CTA retires
      cp_wait<0>();
      for (int i = n; i < min(cnt, n + NST - 1); ++i) wait_drain(bars + 8 * (i % NST), (i / NST) & 1, 20000000ull);
      if (lane == 0) {
        paged_fail(p, ATTN_ERR_TIMEOUT);
        if (!p.rec) p.cuts[worker] = Cut{};
      }
      break;
    }
    __syncwarp();
    fetch(n + NST - 1);
    const uint32_t ks = ring + (n % NST) * S::STAGE, vs = ks + S::PART, sc = scale_ring + (n % NST) * (2 * KEYS * 4) + 4 * lr;
    if (sl.seen != 0xffffffffu) {
      // values that no row sees meet weights of 0: codes of e4m3 may be no numbers
      if (!(sl.seen >> lane & 1u)) {
#pragma unroll
        for (int x = 0; x < D; x += 16) st_shared_v4(vs + lane * D + x, make_uint4(0u, 0u, 0u, 0u));
      }
      fence_proxy_async_smem();
      __syncwarp();
    }
    auto rescale = [&](const float (&f)[2]) {
#pragma unroll
      for (int mb = 0; mb < D / 16; ++mb) {
        o[mb][0] *= f[0];
        o[mb][1] *= f[1];
        o[mb][2] *= f[0];
        o[mb][3] *= f[1];
      }
    };
    auto over_keys = [](float x) {        // the largest over the lanes that share a row
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
      return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
    };
#pragma unroll 1
    for (int j = 0; j < NSUB; ++j) {
      // S^T = K Q^T: x[e]: key 16 j + lr; x[2 + e]: key 16 j + 8 + lr
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = 0.f;
#pragma unroll
      for (int hh = 0; hh < D / 64; ++hh) {
        const uint4 u = lds16(ks + (k_at ^ (hh << 6)) + 16 * j * D), v = lds16(ks + (k_at ^ (hh << 6)) + (16 * j + 8) * D);
        const uint32_t uu[4] = {u.x, u.y, u.z, u.w}, vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t a[4];
          C::unpack(uu[i], a[0], a[2]);
          C::unpack(vv[i], a[1], a[3]);
          mma_f16(x, a, qf[4 * hh + i][0], qf[4 * hh + i][1]);
        }
      }
      // the keys' scales and the rows' factors: x becomes the score in log2 units
      const float k0 = lds4(sc + j * 64), k1 = lds4(sc + j * 64 + 32);
      const uint64_t rr = f2_make(rs[0], rs[1]);
      f2_split(f2_mul(f2_make(x[0], x[1]), f2_mul(f2_make(k0, k0), rr)), x[0], x[1]);
      f2_split(f2_mul(f2_make(x[2], x[3]), f2_mul(f2_make(k1, k1), rr)), x[2], x[3]);
      const int key = key0 + 16 * j;
      if (key + 16 > all_hi || (key < all_lo && key + 16 > p.sinks)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 2 * c + e;
          long long row;
          const int pos = r < rows_here ? (p.causal ? item_len - item_nq + token_of(r, row) : item_len - 1) : -1,
                    lo = p.causal && p.window > 0 ? pos - p.window + 1 : 0;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int k = key + 8 * u + lr;
            if (!(k <= pos && (k >= lo || k < p.sinks))) x[2 * u + e] = -INFINITY;
          }
        }
      }
      // the rows' maxima are looked at together only where one of a lane's scores calls for it
      bool high = false;
#pragma unroll
      for (int e = 0; e < 2; ++e) high |= fmaxf(x[e], x[2 + e]) > m[e] + F8_TAU;
      if (__any_sync(0xffffffffu, high)) {
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float a = over_keys(fmaxf(x[e], x[2 + e]));
          const bool g = a > m[e] + F8_TAU;
          f[e] = g ? ex2_approx(m[e] - a) : 1.f;
          if (g) m[e] = a;
          unset |= static_cast<unsigned>(g) << e;
          l[e] *= f[e];
          most[e] *= f[e];
        }
        rescale(f);
      }
      const float v0 = lds4(sc + KEYS * 4 + j * 64), v1 = lds4(sc + KEYS * 4 + j * 64 + 32);
      float w[2];            // largest weights, of this lane's keys
      bool look = unset != 0;
      const uint64_t nm = f2_make(m[0] == -INFINITY ? 0.f : -m[0], m[1] == -INFINITY ? 0.f : -m[1]);
      f2_split(f2_add(f2_make(x[0], x[1]), nm), x[0], x[1]);
      f2_split(f2_add(f2_make(x[2], x[3]), nm), x[2], x[3]);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = ex2_approx(x[e]);
      l[0] += x[0] + x[2];
      l[1] += x[1] + x[3];
      f2_split(f2_mul(f2_make(x[0], x[1]), f2_make(v0, v0)), x[0], x[1]);
      f2_split(f2_mul(f2_make(x[2], x[3]), f2_make(v1, v1)), x[2], x[3]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        w[e] = fmaxf(fabsf(x[e]), fabsf(x[2 + e]));
        look |= w[e] > most_at(lc[e]);
      }
      if (__any_sync(0xffffffffu, look)) {
        // the rows' powers of two are looked at
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          f[e] = refit(over_keys(w[e]), most[e], lc[e]);
          if (most[e] > 0.f) unset &= ~(1u << e);
        }
        if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) rescale(f);
      }
      const uint64_t cc = f2_make(pow2_of(lc[0]), pow2_of(lc[1]));
      f2_split(f2_mul(f2_make(x[0], x[1]), cc), x[0], x[1]);
      f2_split(f2_mul(f2_make(x[2], x[3]), cc), x[2], x[3]);
      // O^T += V^T W^T: row lr of block mb is column (D / 8) lr + 2 mb, row lr + 8 the next one
      const uint32_t p0 = transposed(pack_f16x2(x[0], x[1])), p1 = transposed(pack_f16x2(x[2], x[3]));
      uint32_t y[4][D / 32];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (D == 128) {
          const uint4 z = lds16(vs + v_at[i] + j * 16 * D);
          y[i][0] = z.x, y[i][1] = z.y, y[i][2] = z.z, y[i][3] = z.w;
        } else {
          const uint2 z = lds8(vs + v_at[i] + j * 16 * D);
          y[i][0] = z.x, y[i][1] = z.y;
        }
      }
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        uint32_t u[4], v[4];
        across<FMT>(y[0][q], y[1][q], u);
        across<FMT>(y[2][q], y[3][q], v);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t a[4] = {u[2 * h], u[2 * h + 1], v[2 * h], v[2 * h + 1]};
          mma_f16(o[2 * q + h], a, p0, p1);
        }
      }
    }
    const bool ends = tile_i == tile_n - 1;
    if (ends || n == cnt - 1) {
      const bool whole = ends && piece0 == 0;
      int np = 0, slot0 = 0;
      if (p.rec && piece0 == 0) item_pieces(from + n - tile_i, tile_n, span_no, span, from, np, slot0);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[e];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        const int r = 2 * c + e;
        if (r >= rows_here) continue;
        long long row;
        const int t = token_of(r, row);
        if (p.rec && piece0 == 0 && lr == 0) p.rec[row] = Rec4{static_cast<int>(worker), slot0, np, r};
        // this lane's D / 8 columns in a row; the row's power of two leaves
        float y[D / 8];
        const float f = pow2_of(-lc[e]);
#pragma unroll
        for (int mb = 0; mb < D / 16; ++mb) {
          y[2 * mb] = o[mb][e] * f;
          y[2 * mb + 1] = o[mb][2 + e] * f;
        }
        if (whole && !p.rec) {
          float fo, lse;
          row_final(m[e], sum, fo, lse);
          const long long at = row * D + lr * (D / 8);
#pragma unroll
          for (int i = 0; i < D / 8; ++i) y[i] = finished(y[i], fo);
          if (p.out_f32) {
#pragma unroll
            for (int i = 0; i < D / 8; i += 4)
              *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at + i) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
          } else {
#pragma unroll
            for (int i = 0; i < D / 8; i += 8)
              *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + at + i) =
                  make_uint4(pack_bf16x2(y[i], y[i + 1]), pack_bf16x2(y[i + 2], y[i + 3]), pack_bf16x2(y[i + 4], y[i + 5]),
                             pack_bf16x2(y[i + 6], y[i + 7]));
          }
          if (lr == 0) p.lse[(static_cast<long long>(item_h) * p.G + item_x0 + r - t * p.G) * p.n_tokens + item_q0 + t] = lse;
        } else {
          // to the dense arrays, or to a piece: slot 0 the one a span begins
          // with, slot 1 one that begins in it and goes on
          const long long slot = worker * 2 + (n - (tile_i - piece0) == 0 ? 0 : 1), to = whole ? row : slot * F8_ROWS + r;
          float *po = (whole ? p.dense_o : p.part_o) + to * D + lr * (D / 8);
#pragma unroll
          for (int i = 0; i < D / 8; i += 4) *reinterpret_cast<float4 *>(po + i) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
          if (lr == 0) *reinterpret_cast<float2 *>((whole ? p.dense_ml : p.part_ml) + to * 2) = make_float2(m[e], sum);
        }
      }
    }
  }
  if (lane == 0 && !p.rec && !gave_up) leave_cut<F8_ROWS, KL>(p, in, 0, in.h * p.hp + sub, worker, span_no, span, from, to);
  end_after_previous(p);
}

// ---------------------------------------------------------------------- host

template <int D, int NST, int W, int FMT>
static int launch_few8(PagedParams &p, const CUtensorMap &mk, const CUtensorMap &mv, cudaStream_t s) {
  using S = Few8Smem<D, NST, W>;
  constexpr int kDev = 64;
  static bool done[kDev] = {};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDev) return ATTN_ERR_CUDA;
  auto kern = paged_few8_kernel<D, NST, W, FMT>;
  auto join = paged_join_kernel<D, F8_ROWS, true>;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (raise_smem(kern, kSmemMax, &done[dev]) != ATTN_OK) return ATTN_ERR_CUDA;
  }
  const int sms = device_sm_count();
  if (sms <= 0) return ATTN_ERR_CUDA;
  // pieces of 8 rows of 12 warps, where the workspace has room for 16 of 8
  const size_t slots = static_cast<size_t>(sms) * W * 2;
  p.part_ml = p.part_o + slots * F8_ROWS * D;
  p.cuts = reinterpret_cast<Cut *>(p.part_ml + slots * F8_ROWS * 2);
  // as many heads side by side as divide the heads, up to 8
  p.hp = 1;
  while (p.hp < 8 && p.hk % (2 * p.hp) == 0) p.hp *= 2;
  p.n_spans = sms * W / p.hp;
  p.warp_plan = p.n_seqs <= 32 && (!p.causal || static_cast<long long>(p.n_tokens) * p.G <= 64 * F8_ROWS);
  if (S::bytes(p, false) > kSmemMax) return ATTN_ERR_UNSUPPORTED;
  const bool infos = S::bytes(p, true) <= kSmemMax;
  const int rc = launch_after(kern, dim3(sms), W * 32, S::bytes(p, infos), s, mk, mv, p, infos ? 1 : 0);
  if (rc != ATTN_OK || p.rec) return rc;
  // few items: each has many pieces, and its rows go to blocks of their own
  const long long items = static_cast<long long>(p.n_seqs) * p.hk;
  return launch_after(join, dim3(sms * W, items * 8 < sms * W ? 4 : 1), 256, 0, s, p);
}

// UNSUPPORTED, with nothing launched, where the tensor maps cannot say the layout (strides
// of zero) or the sums of thousands of sequences leave no room for the rings.
int paged_few8_launch(PagedParams &p, int d, cudaStream_t s) {
  // ATTN_TEST_STALL_PAGED=1 in the environment: a bounded wait runs out, which is how the
  // tests drive the abort path
  const char *stall = std::getenv("ATTN_TEST_STALL_PAGED");
  p.test_stall = stall && stall[0] == '1';
  CUtensorMap mk, mv;
  int rc;
  if ((rc = paged_map8(&mk, p.k, p, d, 1 << F8_KL)) != ATTN_OK || (rc = paged_map8(&mv, p.v, p, d, 1 << F8_KL)) != ATTN_OK) return rc;
  if (p.format == ATTN_CODES_E4M3)
    return d == 128 ? launch_few8<128, 2, 12, ATTN_CODES_E4M3>(p, mk, mv, s) : launch_few8<64, 4, 12, ATTN_CODES_E4M3>(p, mk, mv, s);
  return d == 128 ? launch_few8<128, 2, 12, ATTN_CODES_INT8>(p, mk, mv, s) : launch_few8<64, 4, 12, ATTN_CODES_INT8>(p, mk, mv, s);
}

}  // namespace attn
