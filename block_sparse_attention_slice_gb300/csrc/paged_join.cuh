// Joining the pieces of the items that cross span boundaries.
#pragma once
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "launch.cuh"
#include "paged_plan.cuh"

namespace attn {

// A running summary over pieces of one row, held by LN lanes: each has V columns
// of O, in words of 4 that lie 4 * LN apart.
template <int D, int LANES>
struct Gather {
  static constexpr int LN = LANES, V = D / LN, BATCH = 4;
  float m = -INFINITY, l = 0.f, acc[V];
  __device__ __forceinline__ Gather() {
#pragma unroll
    for (int c = 0; c < V; ++c) acc[c] = 0.f;
  }
  static __device__ __forceinline__ int lane() { return threadIdx.x & (LN - 1); }
  // the first column of word c / 4
  static __device__ __forceinline__ int column(int c) { return c * LN + lane() * 4; }
  static __device__ __forceinline__ void load(float (&y)[V], const float *src) {
#pragma unroll
    for (int c = 0; c < V; c += 4) {
      const float4 z = *reinterpret_cast<const float4 *>(src + column(c));
      y[c] = z.x, y[c + 1] = z.y, y[c + 2] = z.z, y[c + 3] = z.w;
    }
  }
  // Sets the sum of n <= 4 pieces: every lane reads their (m, l) itself, all
  // loads at once, and no shuffle is needed.
  template <typename FO, typename FM>
  __device__ __forceinline__ void few(int n, FO o_of, FM ml_of) {
    float2 ml[4];
    float y[4][V];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < n) {
        ml[k] = *reinterpret_cast<const float2 *>(ml_of(k));
        load(y[k], o_of(k));
      }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < n) m = fmaxf(m, ml[k].x);
    const float mb = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < n) {
        const float f = exp2f(ml[k].x - mb);
        l = fmaf(f, ml[k].y, l);
#pragma unroll
        for (int c = 0; c < V; ++c) acc[c] = fmaf(f, y[k][c], acc[c]);
      }
  }
  // Adds n <= LN pieces in order; o_of(i) is the address of piece i's O row,
  // and lane i has its (m, l).  The first rows are requested before the
  // weights that they wait for are known.  All rows of a warp together, most
  // being the largest of their n.
  template <typename F>
  __device__ __forceinline__ void add(int n, int most, float2 ml, F o_of) {
    float y[BATCH][V];
    auto fetch = [&](int k0) {
#pragma unroll
      for (int k = 0; k < BATCH; ++k)
        if (k0 + k < n) load(y[k], o_of(k0 + k));
    };
    fetch(0);
    const int i = lane();
    float top = i < n ? ml.x : -INFINITY;
#pragma unroll
    for (int o = LN / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    top = fmaxf(top, m);
    const float mb = top == -INFINITY ? 0.f : top, old = exp2f(m - mb);
    const float f = i < n ? exp2f(ml.x - mb) : 0.f;
    float s = i < n ? f * ml.y : 0.f;
#pragma unroll
    for (int o = LN / 2; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    m = top;
    l = l * old + s;
#pragma unroll
    for (int c = 0; c < V; ++c) acc[c] *= old;
    for (int k0 = 0; k0 < most; k0 += BATCH) {
      if (k0) fetch(k0);
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        const float g = __shfl_sync(0xffffffffu, f, k0 + k, LN);
        if (k0 + k < n) {
#pragma unroll
          for (int c = 0; c < V; ++c) acc[c] = fmaf(g, y[k][c], acc[c]);
        }
      }
    }
  }
  // Writes the finished row, and its lse.
  __device__ __forceinline__ void store(const PagedParams &p, long long row, int t, int head) const {
    float fo, lse;
    row_final(m, l, fo, lse);
#pragma unroll
    for (int c = 0; c < V; c += 4) {
      const long long at = row * D + column(c);
      const float y[4] = {finished(acc[c], fo), finished(acc[c + 1], fo), finished(acc[c + 2], fo), finished(acc[c + 3], fo)};
      if (p.out_f32)
        *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) =
            make_float4(y[0], y[1], y[2], y[3]);
      else
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + at) =
            make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
    }
    if (lane() == 0) p.lse[static_cast<long long>(head) * p.n_tokens + t] = lse;
  }
};

// Merges the pieces of the items that cross span boundaries: block x looks at
// what worker x left and, where an item begins there and goes on, merges that
// item's rows (blockIdx.y of gridDim.y takes its part of them).  Few pieces:
// a group of lanes a row.  Many (a long sequence alone in the batch): the
// block's groups share a row's pieces and add their sums.  Pieces are added in a
// fixed order, so results do not vary from run to run.
// Bound by L2, by its own instructions where there are many rows and by latency
// where there are few: its pieces were written just before.  Hence 16 lanes a row
// behind the tiles' 256 rows (prompt pieces, 152 spans: 12 us with 32 lanes, 8
// with 16) and, at head dim 128, 32 behind items of up to 16 rows, which leave
// half of the groups without a row (1 us less of a call of 120).  One sequence:
// 3 us.
// PACKED: rows stand as they are counted; else 128 / G whole tokens to each
// 128 rows.
template <int D, int TILE_ROWS, bool PACKED>
__global__ void __launch_bounds__(256, 4) paged_join_kernel(const PagedParams p) {
  using G = Gather<D, PACKED ? D / 4 : 16>;
  constexpr int NG = 256 / G::LN;
  __shared__ __align__(16) float red[NG][D + 4];
  // The tiles of codes take an SM's whole register file.  Started beside a join they are
  // slower throughout (back to back 275 us a call, 238 behind its end).
  if (PACKED || !p.bits8) admit_next();
  after_previous();
  const Cut cut = p.cuts[blockIdx.x];
  if (cut.rows == 0) return;
  const int grp = threadIdx.x / G::LN, lane = G::lane(), np = cut.np;
  const int per128 = PACKED ? 128 : 128 / p.G * p.G;
  auto place = [&](int i, int r) -> long long {
    return ((static_cast<long long>(blockIdx.x) + i * p.hp) * 2 + (i == 0 ? cut.slot0 : 0)) * TILE_ROWS +
           (PACKED || per128 == 128 ? r : r + r / per128 * (128 - per128));
  };
  auto finish = [&](int r, const G &g) {
    const int x = cut.x0 + r, t = x / p.G, head = cut.h * p.G + x - t * p.G;
    g.store(p, static_cast<long long>(cut.q0 + t) * p.hq + head, cut.q0 + t, head);
  };
  if (np <= 4) {
    for (int r = blockIdx.y * NG + grp; r < cut.rows; r += gridDim.y * NG) {
      G g;
      g.few(np, [&](int k) { return p.part_o + place(k, r) * D; }, [&](int k) { return p.part_ml + place(k, r) * 2; });
      finish(r, g);
    }
    return;
  }
  if (np <= NG) {
    for (int r0 = blockIdx.y * NG; r0 < cut.rows; r0 += gridDim.y * NG) {
      const int r = min(r0 + grp, cut.rows - 1);
      G g;
      float2 ml = make_float2(-INFINITY, 0.f);
      if (lane < np) ml = *reinterpret_cast<const float2 *>(p.part_ml + place(lane, r) * 2);
      g.add(np, np, ml, [&](int k) { return p.part_o + place(k, r) * D; });
      if (r0 + grp < cut.rows) finish(r, g);
    }
    return;
  }
  for (int r = blockIdx.y; r < cut.rows; r += gridDim.y) {
    // this group's pieces: grp, grp + NG, ...
    G g;
    for (int base = 0; base < np; base += G::LN * NG) {
      const int n = min(G::LN, max(0, np - base - grp + NG - 1) / NG), most = min(G::LN, (np - base + NG - 1) / NG);
      float2 ml = make_float2(-INFINITY, 0.f);
      if (lane < n) ml = *reinterpret_cast<const float2 *>(p.part_ml + place(base + grp + lane * NG, r) * 2);
      g.add(n, most, ml, [&](int k) { return p.part_o + place(base + grp + k * NG, r) * D; });
    }
#pragma unroll
    for (int c = 0; c < G::V; c += 4)
      *reinterpret_cast<float4 *>(&red[grp][G::column(c)]) = make_float4(g.acc[c], g.acc[c + 1], g.acc[c + 2], g.acc[c + 3]);
    if (lane == 0) {
      red[grp][D] = g.m;
      red[grp][D + 1] = g.l;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
      G all;
      float2 ml = make_float2(-INFINITY, 0.f);
      if (lane < NG) ml = make_float2(red[lane][D], red[lane][D + 1]);
      all.add(NG, NG, ml, [&](int k) -> const float * { return red[k]; });
      if (grp == 0) finish(r, all);
    }
    __syncthreads();
  }
}

// The largest i < n with a[i] <= x, where a does not decrease; 0 if there is none.
__device__ __forceinline__ int last_not_above(const int32_t *a, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Whether a record names pieces that the pass has.
__device__ __forceinline__ bool in_bounds(const Rec4 &r, const PagedParams &p, int rows) {
  const long long workers = static_cast<long long>(p.n_spans) * p.hp;
  return r.np <= 0 || (r.np <= p.n_spans && r.worker >= 0 && r.worker + (r.np - 1ll) * p.hp < workers && (r.slot0 & ~1) == 0 &&
                       r.row >= 0 && r.row < rows);
}

// Merges what two passes over the same rows left, the prefix's and that of
// what follows it: half a warp a row.  A row's records were written in this call
// exactly if the row belongs to a sequence (and to a group), which is looked
// up here, while the passes still run, rather than having the records cleared
// before them.  6 us for 6400 rows of 64 columns (7 with a warp a row), 9 for
// 8192 of 128.
template <int D>
__global__ void __launch_bounds__(256, D == 128 ? 3 : 4) paged_join_pair_kernel(const PagedParams pre, const PagedParams p,
                                                                 const int pre_rows, const int rows) {
  using G = Gather<D, 16>;
  admit_next();
  const int lane = G::lane();
  const long long row = static_cast<long long>(blockIdx.x) * (256 / G::LN) + threadIdx.x / G::LN;
  const int t = static_cast<int>(row / p.hq);
  bool mine = false, grouped = false;
  if (t < p.n_tokens) {
    const int b = p.q_ptr ? last_not_above(p.q_ptr, p.n_seqs, t) : t;
    const SeqInfo s = seq_info(p, b);
    mine = t >= s.q0 && t < s.q0 + s.nq;
    const SeqInfo g = seq_info(pre, last_not_above(pre.group_ptr, pre.n_seqs, b));
    grouped = t >= g.q0 && t < g.q0 + g.nq;
  }
  after_previous();
  if (!__any_sync(0xffffffffu, mine)) return;      // of no sequence: left as they are
  Rec4 a{0, 0, REC_EMPTY, 0}, b = a;
  if (mine) b = p.rec[row];
  if (mine && grouped) a = pre.rec[row];
  // a pass that gave up (a bounded wait ran out) left some records unwritten
  if (!in_bounds(a, pre, pre_rows)) a.np = REC_EMPTY;
  if (!in_bounds(b, p, rows)) b.np = REC_EMPTY;
  const int na = a.np < 0 ? 0 : a.np ? a.np : 1, nb = b.np < 0 ? 0 : b.np ? b.np : 1, np = na + nb;
  const int most = __reduce_max_sync(0xffffffffu, np);
  // row of piece i in its pass's pieces, or (np = 0) in the dense arrays
  auto place = [&](int i, bool &first, bool &dense) -> long long {
    first = i < na;
    const Rec4 &r = first ? a : b;
    const int k = first ? i : i - na;
    dense = r.np == 0;
    if (dense) return row;
    return ((static_cast<long long>(r.worker) + k * (first ? pre.hp : p.hp)) * 2 + (k == 0 ? r.slot0 : 0)) *
               (first ? pre_rows : rows) + r.row;
  };
  G g;
  for (int base = 0; base < most; base += G::LN) {
    float2 ml = make_float2(-INFINITY, 0.f);
    if (base + lane < np) {
      bool first, dense;
      const long long at = place(base + lane, first, dense);
      const PagedParams &x = first ? pre : p;
      ml = *reinterpret_cast<const float2 *>((dense ? x.dense_ml : x.part_ml) + at * 2);
    }
    g.add(max(0, min(G::LN, np - base)), min(G::LN, most - base), ml, [&](int k) -> const float * {
      bool first, dense;
      const long long at = place(base + k, first, dense);
      const PagedParams &x = first ? pre : p;
      return (dense ? x.dense_o : x.part_o) + at * D;
    });
  }
  if (mine) g.store(p, row, t, static_cast<int>(row - static_cast<long long>(t) * p.hq));
}

}  // namespace attn
