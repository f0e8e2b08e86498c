// Attention over a paged cache in 8 bits for 9 to 32 rows per key/value head (and for
// fewer where paged_few8.cu does not serve), 16 at a time: the
// stream of paged_rows.cu, whose plan, rings and pieces it has, over codes of one
// byte with a scale for each token and head.
//
// What bounds it is what bounds paged_few8.cu: a byte costs a conversion, of units that have few
// operations a code to spare.  Operands are f16 for the same reason, and a lane reads 16 codes at
// once and they are its operands as they lie: the sum over d, the sum over keys and the columns
// of O may each be taken in any order that both operands agree on.  Of 64 columns of a key lane c
// of its four takes 16 in a row, for four products; of 16 keys a lane has four neighbouring ones,
// in P as in V, and of V's columns it takes 16 (8) in a row from each of these rows, so that two
// rows' words make operands by one byte permutation a pair.  ldmatrix has no part in it.
//
// 48 sequences, window 2048, 20 rows of 64 columns to each of 8 heads, e4m3: 68 MB in two passes, 35.5
// us with 10 of start and join.  Two row tiles to a pass (255 registers, 8 warps): 49 us; on 16
// sequences of 8192 keys 75, where this takes 78.
//
// Numerics as in paged_few8.cu.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "attn_internal.h"
#include "codes.cuh"
#include "paged_join.cuh"
#include "paged_plan.cuh"
#include "warp8.cuh"

namespace attn {

constexpr int R8_ROWS = 16;
constexpr int R8_KL = 5;           // a slab is 32 keys
constexpr float R8_TAU = 8.0f;

namespace {

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
}  // namespace

// What the fetching side of a warp tells its computing side about a slab.
struct __align__(16) Slab8 {
  int key0, i, n, h;          // first key; key tile i of the item's n; head
  int rt, q0, nq, len;        // row tile; the sequence's tokens and length
};

template <int D, int NST, int W>
struct Rows8Smem {
  static constexpr int KEYS = 1 << R8_KL;
  static constexpr int PART = KEYS * D;                         // keys or values of one slab
  static constexpr int SCALES = 2 * PART, STAGE = 2 * PART + 2 * KEYS * 4;
  static constexpr int NOTE = W * NST * STAGE;                  // Slab8 [W][NST]
  static constexpr int SCAN = NOTE + W * NST * static_cast<int>(sizeof(Slab8));
  static constexpr int FIRST = SCAN + (W + 2) / 2 * 16;
  static size_t bytes(const PagedParams &p, bool infos) {
    return FIRST + (p.warp_plan ? static_cast<size_t>(W) * PLAN_WARP : 8ull * (p.n_seqs + 1) + (infos ? sizeof(SeqInfo) * p.n_seqs : 0));
  }
};

// W: warps of a CTA.  At head dim 64 the 168 registers that 12 of them leave a thread are enough (8: 48
// sequences, window 2048, 20 rows 39.0 us, 12: 36.0; 16 sequences of 8192 keys 92, 80); at 128 they are not.  Short
// calls have 4 or 8 (rows8_warps).
template <int D, int NST, int FMT, int W>
__global__ void __launch_bounds__(W * 32, 1) paged_rows8_kernel(const PagedParams p, const int keep_infos) {
  using S = Rows8Smem<D, NST, W>;
  using C = F16Codes<FMT>;
  constexpr int KL = R8_KL, KEYS = S::KEYS, NSUB = KEYS / 16, NB = KEYS / 8;
  constexpr int NOT_SEEN = INT_MIN;
  extern __shared__ __align__(256) uint8_t rows8_smem[];
  long long *scan = reinterpret_cast<long long *>(rows8_smem + S::SCAN);
  long long *first = reinterpret_cast<long long *>(rows8_smem + S::FIRST);
  SeqInfo *info = keep_infos ? reinterpret_cast<SeqInfo *>(first + p.n_seqs + 1) : nullptr;
  if (!p.wait_end) after_previous();
  admit_next();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int sms = gridDim.x;
  if (p.share.side) {
    sms = my_sms<W * 32>(p, sms, reinterpret_cast<longlong2 *>(rows8_smem));
    if (static_cast<int>(blockIdx.x) >= sms) {
      end_after_previous(p);
      return;
    }
    __syncthreads();
  }
  if (p.warp_plan) make_warp_plan<R8_ROWS, KL>(p, 0, rows8_smem + S::FIRST + warp * PLAN_WARP, first, info);
  else make_plan<R8_ROWS, KL, W * 32>(p, 0, first, info, scan);
  finish_empty<D, R8_ROWS, KL>(p, info, 0, sms);

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

  const uint32_t ring = smem_u32(rows8_smem) + warp * (NST * S::STAGE);
  Slab8 *note = reinterpret_cast<Slab8 *>(rows8_smem + S::NOTE) + warp * NST;
  Walk<R8_ROWS, KL> in;            // the slab to be fetched next
  in.seek(p, first, info, 0, from);
  int in_lo, in_end;               // keys that some row of its item sees (and the first ones)
  auto bounds = [&]() {
    int t0, t1;
    tile_tokens<R8_ROWS>(in.rt, in.s.nq, p.G, 0, t0, t1);
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
  constexpr int CH = D / 16, RPI = 32 / CH;                // 16-byte words a row, rows an instruction
  const int fc = lane % CH, fr = lane / CH;
  const long long lane_off = fr * p.token_stride + fc * 16, row_step = RPI * p.token_stride;
  const char *kbase = static_cast<const char *>(p.k) + lane_off, *vbase = static_cast<const char *>(p.v) + lane_off;
  // A row's 16-byte words are xor-swizzled so that the reads below meet no bank
  // twice: by 2 (row / 4) and 4 (row odd) at head dim 128, by 2 (row / 4 odd) at 64.
  const uint32_t lane_dst = fr * D + ((D == 128 ? fc ^ ((fr & 1) << 2) : fc ^ (((fr >> 2) & 1) << 1)) << 4);
  // fetches slab n of this worker, where `in` stands, and steps on
  auto fetch = [&](int n) {
    if (n < cnt) {
      const int key0 = in.sp.tile(in.i) << KL, slot = n % NST, head = in.h * p.hp + sub;
      const uint32_t stage = ring + slot * S::STAGE, dst = stage + lane_dst;
      if (lane == 0) {
        note[slot] = Slab8{key0, in.i, in.sp.n, head, in.rt, in.s.q0, in.s.nq, in.s.len};
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
        const long long at = good ? page[j] * p.page_stride + (k0 & page_mask) * p.token_stride + head * p.head_stride : 0;
        const char *ks = kbase + at, *vs = vbase + at;
#pragma unroll
        for (int i = 0; i < 16 / RPI; ++i) {
          const int r = i * RPI;
          const uint32_t d = (D == 128 ? dst ^ (((r >> 2) & 3) << 5) : dst) + (16 * j + r) * D;
          const bool live = mine >> r & 1u;
          cp_async16(d, live ? ks + i * row_step : p.k, live ? 16u : 0u);
          cp_async16(d + S::PART, live ? vs + i * row_step : p.v, live ? 16u : 0u);
        }
        // 16 scales of keys by the first half of the warp, of values by the second
        const int r = lane & 15;
        const bool live = seen >> r & 1u;
        const float *src = lane < 16 ? p.k_scales : p.v_scales;
        const long long sat = page[j] * p.scale_page + ((k0 & page_mask) + r) * p.scale_token + head * p.scale_head;
        cp_async4(stage + S::SCALES + (lane >> 4) * (KEYS * 4) + (16 * j + r) * 4, live ? src + sat : src, live ? 4u : 0u);
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
  // p = 2^(s - m), m the lazy maximum; a value's weight is p vs 2^lc (warp8.cuh), top the
  // largest p vs that was looked at.
  float m0 = 0.f, m1 = 0.f, l0 = 0.f, l1 = 0.f, rs0 = 0.f, rs1 = 0.f, top0 = 0.f, top1 = 0.f;
  int lc0 = 0, lc1 = 0;
  int pos0 = -1, pos1 = -1, lo0 = 0, lo1 = 0;      // last key a row sees, first of its window
  int all_lo = 0, all_hi = 0;                      // keys in [all_lo, all_hi) are seen by every row
  long long row0 = -1, row1 = -1;                  // (token * hq + head), -1: no row
  int rows_here = 0, piece0 = 0;
  const int lr = lane >> 2, c = lane & 3;
  // Key i (0..3) of this lane's four of 16 is 4 c + (i ^ flip): at head dim 64 two
  // rows share a line of banks, and half of the lanes take the other one first.
  const int flip = D == 64 ? c >> 1 : 0;
  // its words in the keys: column n = lr of block b is key 4 (n / 2) + (2 b + n % 2) ^ flip
  const int kr0 = 4 * (lr >> 1) + ((lr & 1) ^ (D == 64 ? (lr >> 2) & 1 : 0)), kr1 = kr0 ^ 2;
  auto k_word = [&](int r) -> uint32_t {
    return r * D + ((D == 128 ? c ^ (((r >> 2) & 3) << 1) ^ ((r & 1) << 2) : c ^ (((r >> 2) & 1) << 1)) << 4);
  };
  const uint32_t k_at[2] = {k_word(kr0), k_word(kr1)};
  // and in the values: columns 16 lr .. (8 lr ..) of keys 4 c + (i ^ flip)
  auto v_word = [&](int i) -> uint32_t {
    const int r = 4 * c + (i ^ flip);
    return r * D + (D == 128 ? (lr ^ (c << 1) ^ ((r & 1) << 2)) << 4 : (((lr >> 1) ^ ((c & 1) << 1)) << 4) + ((lr & 1) << 3));
  };
  const uint32_t v_at[4] = {v_word(0), v_word(1), v_word(2), v_word(3)};

#pragma unroll 1
  for (int n = 0; n < cnt; ++n) {
    // with three slots a slab's note was left before the __syncwarp of the step before; with two, after it
    if constexpr (NST == 2) __syncwarp();
    const Slab8 &sl = note[n % NST];
    const int key0 = sl.key0, tile_i = sl.i, tile_n = sl.n;
    if (n == 0 || tile_i == 0) {
      // a new item: its rows of Q as f16 operands; summaries empty
      const int rt = sl.rt, q0 = sl.q0, nq = sl.nq, len = sl.len, h = sl.h;
      piece0 = tile_i;
      rows_here = min(R8_ROWS, nq * p.G - rt * R8_ROWS);
      auto place = [&](int r, long long &row, int &pos, int &lo) {
        row = -1;
        pos = -1;
        lo = 0;
        if (r < rows_here) {
          const int x = rt * R8_ROWS + r, t = x / p.G;
          row = static_cast<long long>(q0 + t) * p.hq + h * p.G + x - t * p.G;
          pos = p.causal ? len - nq + t : len - 1;
          lo = p.causal && p.window > 0 ? pos - p.window + 1 : 0;
        }
      };
      place(lr, row0, pos0, lo0);
      place(lr + 8, row1, pos1, lo1);
      int t0, t1;
      tile_tokens<R8_ROWS>(rt, nq, p.G, 0, t0, t1);
      all_hi = p.causal ? len - nq + t0 + 1 : len;
      all_lo = p.causal && p.window > 0 ? len - nq + t1 - p.window + 1 : 0;
      auto load_q = [&](long long row, int u) -> float {
        uint4 w[D / 64][2];
        const uint16_t *qa = static_cast<const uint16_t *>(p.q) + (row < 0 ? 0 : row) * D + 16 * c;
#pragma unroll
        for (int hh = 0; hh < D / 64; ++hh)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            w[hh][e] = row < 0 ? make_uint4(0u, 0u, 0u, 0u) : *reinterpret_cast<const uint4 *>(qa + 64 * hh + 8 * e);
        uint32_t top = 0;
        const uint16_t *y = reinterpret_cast<const uint16_t *>(w);
#pragma unroll
        for (int k = 0; k < D / 4; ++k) top = max(top, y[k] & 0x7fffu);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^(14 - exponent of the largest), as far as an f32 power of two and its inverse go: -114 .. 100
        const int e = min(141 - static_cast<int>(top >> 7), 100);
        const float f = pow2_of(e);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint16_t *z = y + 4 * k;      // words 4 i .. of half k / 4: columns 64 (k / 4) + 16 c + 4 (k % 4)
          auto f16_of = [&](int a, int b) {
            return pack_f16x2(__uint_as_float(static_cast<uint32_t>(z[a]) << 16) * f, __uint_as_float(static_cast<uint32_t>(z[b]) << 16) * f);
          };
          qf[k][u] = f16_of(C::A0, C::A1);
          qf[k][2 + u] = f16_of(C::B0, C::B1);
        }
        return p.scale_log2 * pow2_of(-e);
      };
      rs0 = load_q(row0, 0);
      rs1 = load_q(row1, 1);
      m0 = m1 = -INFINITY;
      l0 = l1 = 0.f;
      top0 = top1 = 0.f;
      lc0 = lc1 = 0;
#pragma unroll
      for (int j = 0; j < D / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
    }
    cp_wait<NST - 2>();
    __syncwarp();
    fetch(n + NST - 1);
    const uint32_t ks = ring + (n % NST) * S::STAGE, vs = ks + S::PART, sc = ks + S::SCALES + 16 * c;
    // S = Q K^T: 16 rows x KEYS keys; x[2 j + b][e]: row lr, key 16 j + 4 c + ((2 b + e) ^ flip); [2 + e]: row lr + 8
    float x[NB][4];
#pragma unroll
    for (int j = 0; j < NSUB; ++j) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[2 * j + b][e] = 0.f;
#pragma unroll
        for (int hh = 0; hh < D / 64; ++hh) {
          const uint4 w = lds16(ks + (k_at[b] ^ (hh << 6)) + j * 16 * D);
          uint32_t b0, b1;
          C::unpack(w.x, b0, b1);
          mma_f16(x[2 * j + b], qf[4 * hh], b0, b1);
          C::unpack(w.y, b0, b1);
          mma_f16(x[2 * j + b], qf[4 * hh + 1], b0, b1);
          C::unpack(w.z, b0, b1);
          mma_f16(x[2 * j + b], qf[4 * hh + 2], b0, b1);
          C::unpack(w.w, b0, b1);
          mma_f16(x[2 * j + b], qf[4 * hh + 3], b0, b1);
        }
      }
    }
    // the keys' scales and the rows' factors: x becomes the score in log2 units
    const uint64_t rr0 = f2_make(rs0, rs0), rr1 = f2_make(rs1, rs1);
    auto scales = [&](uint32_t a, uint64_t &lo, uint64_t &hi) {      // in the order of the lane's keys
      const uint4 w = lds16(a);
      lo = flip ? f2_make_u(w.y, w.x) : f2_make_u(w.x, w.y);
      hi = flip ? f2_make_u(w.w, w.z) : f2_make_u(w.z, w.w);
    };
    auto times = [&](float &a, float &b, uint64_t f) { f2_split(f2_mul(f2_make(a, b), f), a, b); };
#pragma unroll
    for (int j = 0; j < NSUB; ++j) {
      uint64_t k2[2];
      scales(sc + j * 64, k2[0], k2[1]);
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        times(x[2 * j + b][0], x[2 * j + b][1], f2_mul(k2[b], rr0));
        times(x[2 * j + b][2], x[2 * j + b][3], f2_mul(k2[b], rr1));
      }
    }
    if (key0 + KEYS > all_hi || (key0 < all_lo && key0 + KEYS > p.sinks)) {
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int j = key0 + (b >> 1) * 16 + 4 * c + ((2 * (b & 1) + e) ^ flip);
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
    a0 = fmaxf(a0, __shfl_xor_sync(0xffffffffu, a0, 2));
    a1 = fmaxf(a1, __shfl_xor_sync(0xffffffffu, a1, 2));
    auto rescale = [&](float f0, float f1) {
#pragma unroll
      for (int j = 0; j < D / 8; ++j) {
        o[j][0] *= f0;
        o[j][1] *= f0;
        o[j][2] *= f1;
        o[j][3] *= f1;
      }
    };
    const bool g0 = a0 > m0 + R8_TAU, g1 = a1 > m1 + R8_TAU;
    if (__any_sync(0xffffffffu, g0 || g1)) {
      const float f0 = g0 ? ex2_approx(m0 - a0) : 1.f, f1 = g1 ? ex2_approx(m1 - a1) : 1.f;
      if (g0) m0 = a0;
      if (g1) m1 = a1;
      l0 *= f0;
      l1 *= f1;
      top0 *= f0;
      top1 *= f1;
      rescale(f0, f1);
    }
    const float b0 = m0 == -INFINITY ? 0.f : -m0, b1 = m1 == -INFINITY ? 0.f : -m1;
    float w0 = 0.f, w1 = 0.f;            // largest weights, of this lane's keys
#pragma unroll
    for (int j = 0; j < NSUB; ++j) {
      uint64_t v2[2];
      scales(sc + KEYS * 4 + j * 64, v2[0], v2[1]);
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        float(&y)[4] = x[2 * j + b];
        f2_split(f2_add(f2_make(y[0], y[1]), f2_make(b0, b0)), y[0], y[1]);
        f2_split(f2_add(f2_make(y[2], y[3]), f2_make(b1, b1)), y[2], y[3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = ex2_approx(y[e]);
        l0 += y[0] + y[1];
        l1 += y[2] + y[3];
        times(y[0], y[1], v2[b]);
        times(y[2], y[3], v2[b]);
        w0 = max3f(w0, fabsf(y[0]), fabsf(y[1]));
        w1 = max3f(w1, fabsf(y[2]), fabsf(y[3]));
      }
    }
    if (__any_sync(0xffffffffu, top0 < pow2_of(-lc0) || top1 < pow2_of(-lc1) || w0 > most_at(lc0) || w1 > most_at(lc1))) {
      // the rows' powers of two are looked at
      auto fit = [](float w, float &top, int &lc) -> float {
        w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, 1));
        return refit(fmaxf(w, __shfl_xor_sync(0xffffffffu, w, 2)), top, lc);
      };
      const float f0 = fit(w0, top0, lc0), f1 = fit(w1, top1, lc1);
      if (__any_sync(0xffffffffu, f0 != 1.f || f1 != 1.f)) rescale(f0, f1);
    }
    const float c0 = pow2_of(lc0), c1 = pow2_of(lc1);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      times(x[b][0], x[b][1], f2_make(c0, c0));
      times(x[b][2], x[b][3], f2_make(c1, c1));
    }
    // O += W V: column n of block e is column (D / 8) n + e
#pragma unroll
    for (int j = 0; j < NSUB; ++j) {
      const uint32_t pf[4] = {pack_f16x2(x[2 * j][0], x[2 * j][1]), pack_f16x2(x[2 * j][2], x[2 * j][3]),
                              pack_f16x2(x[2 * j + 1][0], x[2 * j + 1][1]), pack_f16x2(x[2 * j + 1][2], x[2 * j + 1][3])};
      uint32_t w[4][D / 32];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (D == 128) {
          const uint4 y = lds16(vs + v_at[i] + j * 16 * D);
          w[i][0] = y.x, w[i][1] = y.y, w[i][2] = y.z, w[i][3] = y.w;
        } else {
          const uint2 y = lds8(vs + v_at[i] + j * 16 * D);
          w[i][0] = y.x, w[i][1] = y.y;
        }
      }
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        uint32_t u[4], v[4];
        across<FMT>(w[0][q], w[1][q], u);
        across<FMT>(w[2][q], w[3][q], v);
#pragma unroll
        for (int e = 0; e < 4; ++e) mma_f16(o[4 * q + e], pf, u[e], v[e]);
      }
    }
    const bool ends = tile_i == tile_n - 1;
    if (ends || n == cnt - 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
      l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
      if (p.rec && piece0 == 0 && c == 0) {
        int np, slot0;
        item_pieces(from + n - tile_i, tile_n, span_no, span, from, np, slot0);
        if (row0 >= 0) p.rec[row0] = Rec4{static_cast<int>(worker), slot0, np, lr};
        if (row1 >= 0) p.rec[row1] = Rec4{static_cast<int>(worker), slot0, np, lr + 8};
      }
      const bool whole = ends && piece0 == 0;
      // the rows' powers of two leave
      rescale(pow2_of(-lc0), pow2_of(-lc1));
      lc0 = lc1 = 0;
      // this lane has D / 4 columns in a row of either row, the first half of them in [..][0]
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const long long row = u ? row1 : row0;
        if (row < 0) continue;
        const float m = u ? m1 : m0, l = u ? l1 : l0;
        float y[D / 4];
#pragma unroll
        for (int e = 0; e < D / 8; ++e) {
          y[e] = o[e][2 * u];
          y[D / 8 + e] = o[e][2 * u + 1];
        }
        if (whole && !p.rec) {
          float fo, lse;
          row_final(m, l, fo, lse);
          const long long at = row * D + c * (D / 4);
#pragma unroll
          for (int e = 0; e < D / 4; ++e) y[e] = finished(y[e], fo);
          if (p.out_f32) {
#pragma unroll
            for (int e = 0; e < D / 4; e += 4)
              *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at + e) = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
          } else {
#pragma unroll
            for (int e = 0; e < D / 4; e += 8)
              *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + at + e) =
                  make_uint4(pack_bf16x2(y[e], y[e + 1]), pack_bf16x2(y[e + 2], y[e + 3]), pack_bf16x2(y[e + 4], y[e + 5]),
                             pack_bf16x2(y[e + 6], y[e + 7]));
          }
          if (c == 0) {
            const int t = static_cast<int>(row / p.hq), head = static_cast<int>(row - static_cast<long long>(t) * p.hq);
            p.lse[static_cast<long long>(head) * p.n_tokens + t] = lse;
          }
        } else {
          // to the dense arrays, or to a piece: slot 0 the one a span begins
          // with, slot 1 one that begins in it and goes on
          const long long slot = worker * 2 + (n - (tile_i - piece0) == 0 ? 0 : 1);
          const long long r = whole ? row : slot * R8_ROWS + lr + 8 * u;
          float *po = (whole ? p.dense_o : p.part_o) + r * D + c * (D / 4);
#pragma unroll
          for (int e = 0; e < D / 4; e += 4) *reinterpret_cast<float4 *>(po + e) = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
          if (c == 0) *reinterpret_cast<float2 *>((whole ? p.dense_ml : p.part_ml) + r * 2) = make_float2(m, l);
        }
      }
    }
  }
  if (lane == 0 && !p.rec) leave_cut<R8_ROWS, KL>(p, in, 0, in.h * p.hp + sub, worker, span_no, span, from, to);
  end_after_previous(p);
}

// ---------------------------------------------------------------------- host

template <int D, int NST, int FMT, int W>
static int launch_rows8(PagedParams &p, cudaStream_t s) {
  using S = Rows8Smem<D, NST, W>;
  constexpr int kDev = 64;
  static bool done[kDev] = {};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDev) return ATTN_ERR_CUDA;
  auto kern = paged_rows8_kernel<D, NST, FMT, W>;
  auto join = paged_join_kernel<D, R8_ROWS, true>;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (raise_smem(kern, kSmemMax, &done[dev]) != ATTN_OK) return ATTN_ERR_CUDA;
  }
  const int sms = device_sm_count();
  if (sms <= 0) return ATTN_ERR_CUDA;
  // as many heads side by side as divide the heads, up to 8
  p.hp = 1;
  while (p.hp < 8 && p.hk % (2 * p.hp) == 0) p.hp *= 2;
  p.n_spans = sms * W / p.hp;
  p.warp_plan = p.n_seqs <= 32 && (!p.causal || static_cast<long long>(p.n_tokens) * p.G <= 64 * R8_ROWS);
  // pieces of 16 rows: of 12 warps at head dim 64, where the workspace has room for the tiles' 512 rows an SM
  static_assert(W * 2 * R8_ROWS <= 2 * 256, "pieces");
  const size_t slots = static_cast<size_t>(sms) * W * 2 * R8_ROWS;
  p.part_ml = p.part_o + slots * D;
  p.cuts = reinterpret_cast<Cut *>(p.part_ml + slots * 2);
  const bool infos = S::bytes(p, true) <= kSmemMax;      // not above 3900 sequences
  const int rc = launch_after(kern, dim3(sms), W * 32, S::bytes(p, infos), s, p, infos ? 1 : 0);
  if (rc != ATTN_OK || p.rec) return rc;
  // few items: each has many pieces, and its rows go to blocks of their own
  const long long items = static_cast<long long>(p.n_seqs) * p.hk;
  return launch_after(join, dim3(sms * W, items * 8 < sms * W ? 4 : 1), 256, 0, s, p);
}

// warps: of a CTA, 4, 8 or (head dim 64) 12; beside the plan of thousands of sequences as many as the
// largest calls have.
int paged_rows8_launch(PagedParams &p, int d, int warps, cudaStream_t s) {
  const bool many = p.n_seqs > 1024, e4m3 = p.format == ATTN_CODES_E4M3;
  constexpr int I8 = ATTN_CODES_INT8, E4 = ATTN_CODES_E4M3;
  if (d == 128) {
    if (many) return e4m3 ? launch_rows8<128, 2, E4, 8>(p, s) : launch_rows8<128, 2, I8, 8>(p, s);
    if (warps == 4) return e4m3 ? launch_rows8<128, 3, E4, 4>(p, s) : launch_rows8<128, 3, I8, 4>(p, s);
    return e4m3 ? launch_rows8<128, 3, E4, 8>(p, s) : launch_rows8<128, 3, I8, 8>(p, s);
  }
  if (many) return e4m3 ? launch_rows8<64, 2, E4, 12>(p, s) : launch_rows8<64, 2, I8, 12>(p, s);
  if (warps == 4) return e4m3 ? launch_rows8<64, 4, E4, 4>(p, s) : launch_rows8<64, 4, I8, 4>(p, s);
  if (warps == 8) return e4m3 ? launch_rows8<64, 4, E4, 8>(p, s) : launch_rows8<64, 4, I8, 8>(p, s);
  return e4m3 ? launch_rows8<64, 3, E4, 12>(p, s) : launch_rows8<64, 3, I8, 12>(p, s);
}

}  // namespace attn
