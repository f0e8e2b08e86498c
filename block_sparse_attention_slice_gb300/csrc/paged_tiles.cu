// Attention over a paged cache for many rows per key/value head: prompts taken
// in pieces, tokens verified together, and a shared prefix against all the
// rows of its group.  tcgen05 matrix instructions with tensor-memory
// accumulators, pages fetched by TMA.
//
// A row tile is 128 rows of tensor memory: TPT = 128 / G whole tokens with the
// G query heads of one key/value head (one 3-D TMA box of the query tensor
// packs them).  TILES = 2: an item is two row tiles that share every key tile,
// and the tensor core works on one while the softmax warps of the other run
// (the order of attn_fwd: PV_0(j), QK_0(j+1), PV_1(j), QK_1(j+1)).  TILES = 1,
// for items of at most TPT tokens: one row tile with two score buffers, QK(j+1)
// issued before softmax(j) ends, and the 128 keys of a tile shared by two
// softmax groups of 64, each with its own maximum, sum and O, which are merged
// when the segment ends: with few rows a step is one warp's pass over a row of
// scores, and half the row took 1 to 6 % off calls of 24 to 128 rows against one
// group for the whole tile (1 % more on very long calls at head dim 64).
//
// What bounds it.  Rows that fill their tiles: the chain of products and softmax
// that attn_fwd has.  4 x 1021 new tokens, window 4096, 32 query and 8 key/value
// heads of 128 columns: 159 us, 73 steps a CTA of 256 rows by 128 keys at 1.56 us
// (1.6 PFLOP/s over all SMs), and around them 10 us before the first product, 4.4
// at a change of item, 8 for the join.  The lane that issues is busy nearly all of
// a step: a commit takes it some 95 cycles, an instruction what the tensor core
// does.  A 128-key step of TILES = 1 at head dim 64 takes 0.8 to 0.85 us, of which
// the softmax of 64 columns is 0.6 (100 rows, 16384 keys, 16 heads, 4 groups: 34
// us on all SMs).
//
// One persistent CTA per SM takes an equal span of the flat list of 128-key
// tiles (paged_plan.cuh); pieces of items that cross spans are joined by
// paged_join_kernel.  Warps: two groups of 4 softmax warps (thread = row = tensor
// memory lane), a producer warp (walks the list, publishes each segment to the
// others, fetches Q, K and V; one lane per page of a tile) and a warp that
// issues the matrix instructions.
//
// Keys that no row of an item sees (behind the sequence's end, before the
// window) must not meet the zero weights of the P V product, whatever memory
// holds there: whole pages of them are fetched from outside the tensor map,
// which reads as zeros, and their rows of V in pages that are fetched are zeroed
// in shared memory by the softmax warps of row tile 0 before they let the
// product begin.
//
// Numerics as in paged_rows.cu: 32-bit scores, maxima, sums and O; P rounded
// to bf16 (half a step, 2^-8 of each weight either way) as the operand that the
// tensor core takes.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <mutex>

#include "attn_internal.h"
#include "paged_join.cuh"
#include "paged_plan.cuh"

namespace attn {

constexpr int PT_KL = 7, PT_BN = 128, PT_IQ = 4;
constexpr float PT_TAU = 8.0f;

template <int D, int TILES>
struct TileLayout {
  static constexpr int NS = D == 64 ? 10 : TILES == 2 ? 4 : 5;   // K/V ring slots: 128 to 160 KB
  static constexpr int HALF = 128 * 64 * 2, NHALF = D / 64, TILE = NHALF * HALF;
  static constexpr int Q_OFF = 0, KV_OFF = TILES * TILE, SEG_OFF = KV_OFF + NS * TILE;
  static constexpr int BAR_OFF = SEG_OFF + PT_IQ * 64;
  static constexpr int B_Q = 0, B_QE = 1, B_FULL = 2, B_EMPTY = B_FULL + NS, B_S = B_EMPTY + NS, B_P = B_S + 2,
                       B_O = B_P + 2, B_IF = B_O + TILES, B_IE = B_IF + PT_IQ, B_DRAIN = B_IE + PT_IQ,
                       B_V = B_DRAIN + 1, B_X = B_V + 1, NBAR = B_X + 2;
  static constexpr int MISC_OFF = BAR_OFF + NBAR * 8;
  static constexpr int XML_OFF = MISC_OFF + 16;               // TILES = 1: (m, l) of both groups
  static constexpr int SCAN_OFF = XML_OFF + (TILES == 1 ? 2 * 128 * 8 : 0);
  static constexpr int FIRST_OFF = SCAN_OFF + 16 * 8;
  static constexpr int THREADS = 256 + 64;
  static size_t bytes(const PagedParams &p, bool infos) {
    return 1024 + FIRST_OFF + (p.warp_plan ? THREADS / 32 * static_cast<size_t>(PLAN_WARP)
                                           : 8ull * (p.n_seqs + 1) + (infos ? sizeof(SeqInfo) * p.n_seqs : 0));
  }
  static_assert(PT_IQ * 64 >= THREADS / 32 * 16, "my_sms puts its sums where the segments will be");
  static_assert(MISC_OFF % 8 == 0 && (TILES == 1 || NS % 2 == 0), "alignment; keys in even slots");
};

// Transposes 4 x 4 words of 16 bytes among four neighbouring lanes: lane q's
// word k becomes lane k's word q.
__device__ __forceinline__ void exchange4(uint4 (&w)[4], int q) {
#pragma unroll
  for (int s = 1; s < 4; s <<= 1) {
    const bool up = q & s;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k & s) continue;
      uint4 &lo = w[k], &hi = w[k | s];
      const uint4 give = up ? lo : hi;
      uint4 got;
      got.x = __shfl_xor_sync(0xffffffffu, give.x, s);
      got.y = __shfl_xor_sync(0xffffffffu, give.y, s);
      got.z = __shfl_xor_sync(0xffffffffu, give.z, s);
      got.w = __shfl_xor_sync(0xffffffffu, give.w, s);
      if (up) lo = got;
      else hi = got;
    }
  }
}

// The end of a launch that gave up: lets the loads in flight, the last of nq into
// Q and of ld into the ring, land before the CTA retires.  Called where every role
// has come to its end: the producer may have issued its last loads before another
// role's wait ran out.
__device__ __noinline__ void land_loads(uint32_t q_full, uint32_t ring_full, uint32_t ns, uint32_t nq, uint32_t ld) {
  if (nq > 0) wait_drain(q_full, (nq - 1) & 1, 20000000ull);
  for (uint32_t i = ld > ns ? ld - ns : 0; i < ld; ++i) wait_drain(ring_full + 8 * (i % ns), (i / ns) & 1, 20000000ull);
}

// Zeros over what this thread's row was given, if it sees nothing (`none`): the
// products of its zero weights are not zero where a value that other rows see is
// not finite.  TILES = 1: over the group's half of the columns.  A warp together,
// behind its stores and out of line: that costs a call of 156.5 us 1.2, a choice
// for each column in the stores cost it 5.
template <int D, int TILES>
__device__ __noinline__ void zero_row(const PagedParams &p, bool none, long long row, int grp) {
  __syncwarp();
  const int bytes = (TILES == 1 ? D / 2 : D) * (p.out_f32 ? 4 : 2);
  uint8_t *at = static_cast<uint8_t *>(p.out) + row * (D * (p.out_f32 ? 4 : 2)) + (TILES == 1 ? grp * bytes : 0);
  for (int x = none ? 0 : bytes; x < bytes; x += 16) *reinterpret_cast<uint4 *>(at + x) = make_uint4(0u, 0u, 0u, 0u);
  __syncwarp();
}

// What the producer publishes of a segment: a run of key tiles of one item.
struct Seg {
  int tok0, ntok, h, pos0, len, ns, w0, i0, i1;
  int out;              // 0 finished here, 1 / 2 piece slot + 1, -1 no more
  int np, slot0;        // of an item that begins here (i0 = 0): see Rec4
  int rot;              // its key tiles are taken in the order i0 + rot, .., i1 - 1, i0, .., i0 + rot - 1
  // the j-th key tile (of 128 keys) of the segment
  static __device__ __forceinline__ int key_tile(int j, int i0, int i1, int rot, const Span &sp) {
    const int i = i0 + rot + j;
    return sp.tile(i < i1 ? i : i - (i1 - i0));
  }
};
static_assert(sizeof(Seg) <= 64, "segment record");

template <int D, int TILES>
__global__ void __launch_bounds__(TileLayout<D, TILES>::THREADS, 1)
    paged_tiles_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const PagedParams p, const int tpt,
                       const int keep_infos) {
  using L = TileLayout<D, TILES>;
  constexpr int NS = L::NS;
  extern __shared__ uint8_t tiles_smem[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(tiles_smem) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_u32(smem);
  auto bar = [&](int i) -> uint32_t { return sb + L::BAR_OFF + 8u * i; };
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::MISC_OFF);
  volatile int *abort = reinterpret_cast<volatile int *>(smem + L::MISC_OFF + 4);
  volatile uint32_t *loads = reinterpret_cast<volatile uint32_t *>(smem + L::MISC_OFF + 8);   // of Q and of K/V, in the end
  volatile Seg *segs = reinterpret_cast<volatile Seg *>(smem + L::SEG_OFF);   // 64 bytes apart
  auto seg_at = [&](int s) -> volatile Seg * {
    return reinterpret_cast<volatile Seg *>(reinterpret_cast<volatile uint8_t *>(segs) + 64 * s);
  };
  long long *scan = reinterpret_cast<long long *>(smem + L::SCAN_OFF);
  long long *first = reinterpret_cast<long long *>(smem + L::FIRST_OFF);
  SeqInfo *info = keep_infos ? reinterpret_cast<SeqInfo *>(first + p.n_seqs + 1) : nullptr;
  const uint32_t q_smem = sb + L::Q_OFF, kv_smem = sb + L::KV_OFF;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tpi = tpt * TILES;
  const uint64_t lim = p.wait_ns;
  constexpr int WP = 8, WM = 9;       // producer, issuer

  int sms = gridDim.x;
  if (p.share.side) {
    if (!p.wait_end) after_previous();
    admit_next();
    sms = my_sms<L::THREADS>(p, sms, reinterpret_cast<longlong2 *>(smem + L::SEG_OFF));      // no segment is published yet
    if (static_cast<int>(blockIdx.x) >= sms) {
      end_after_previous(p);
      return;
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    mbar_init(bar(L::B_Q), 1);
    mbar_init(bar(L::B_QE), 1);
    for (int s = 0; s < NS; ++s) {
      mbar_init(bar(L::B_FULL + s), 1);
      mbar_init(bar(L::B_EMPTY + s), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(L::B_S + t), 1);
      mbar_init(bar(L::B_P + t), TILES == 1 ? 256 : 128);
      mbar_init(bar(L::B_X + t), 256);
    }
    for (int t = 0; t < TILES; ++t) mbar_init(bar(L::B_O + t), 1);
    for (int u = 0; u < PT_IQ; ++u) {
      mbar_init(bar(L::B_IF + u), 1);
      mbar_init(bar(L::B_IE + u), 9);
    }
    mbar_init(bar(L::B_DRAIN), 1);
    mbar_init(bar(L::B_V), 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == WM) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  if (warp == WP && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (!p.wait_end) after_previous();
  admit_next();
  if (TILES == 1 && p.warp_plan) make_warp_plan<0, PT_KL>(p, tpi, smem + L::FIRST_OFF + warp * PLAN_WARP, first, info);
  else make_plan<0, PT_KL, L::THREADS>(p, tpi, first, info, scan);
  finish_empty<D, 0, PT_KL>(p, info, tpi, sms);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int n_spans = p.share.side ? sms / p.hp : p.n_spans;
  const long long total = first[p.n_seqs], span = span_of(total, n_spans);
  const int mine = blockIdx.x / p.hp, sub = blockIdx.x - mine * p.hp;      // span, and head of a group
  const long long from = mine < n_spans ? mine * span : total, to = min(total, from + span);

  if (warp == WP) {
    // -------------------------------------------------------------- producer
    uint32_t ld = 0, nseg = 0;
    bool ok = true;
    long long at = from;
    Walk<0, PT_KL> w;
    // stands if the launch gives up, too: the join then reads no stale record
    if (lane == 0 && !p.rec) p.cuts[blockIdx.x] = Cut{};
    if (at < to) w.seek(p, first, info, tpi, at);
    const int R = min(1 << p.page_shift, 128), ppt = 128 / R, page_mask = (1 << p.page_shift) - 1;
    while (ok) {
      const int qs = nseg % PT_IQ;
      if (nseg >= PT_IQ && !wait_all(bar(L::B_IE + qs), (nseg / PT_IQ - 1) & 1, abort, lim)) break;
      const bool more = at < to;
      int i1 = 0;
      // Row tiles of one group read the same keys.  Taking key tile k of an item
      // at the time k mod span lets the CTAs that share it read it together, so
      // that all but the first find it in L2.
      int rot = 0;
      if (more) {
        i1 = static_cast<int>(min(static_cast<long long>(w.sp.n), w.i + (to - at)));
        if (!p.causal) {
          const int ahead = static_cast<int>((span - w.i % span) % span);
          rot = w.i + ahead < i1 ? ahead : 0;
        }
      }
      if (!more) {
        if (lane == 0) {
          seg_at(qs)->out = -1;
          mbar_arrive(bar(L::B_IF + qs));
        }
        __syncwarp();
        break;
      }
      // Q of the segment's tokens
      if (nseg > 0 && !wait_all(bar(L::B_QE), (nseg - 1) & 1, abort, lim)) break;
      const int tok0 = w.s.q0 + w.rt * tpi;
      if (lane == 0) {
        mbar_arrive_expect_tx(bar(L::B_Q), TILES * L::NHALF * tpt * p.G * 128);
        for (int t = 0; t < TILES; ++t)
          for (int hh = 0; hh < L::NHALF; ++hh)
            tma_load_3d(q_smem + t * L::TILE + hh * L::HALF, &tm_q, bar(L::B_Q), hh * 64, (w.h * p.hp + sub) * p.G, tok0 + t * tpt);
      }
      ++nseg;
      // keys that some row sees: below `end`, at least `lo` or a first token
      const int tl = min(tpi, w.s.nq - w.rt * tpi) - 1, pos0 = w.s.len - w.s.nq + w.rt * tpi;
      const int end = p.causal ? pos0 + tl + 1 : w.s.len, lo = p.causal && p.window > 0 ? max(0, pos0 - p.window + 1) : 0;
      const long long row = w.s.slot * p.table_stride;
      const int i0 = w.i, steps = i1 - i0;
      // this lane's page of the j-th key tile, as the table has it; NOT_SEEN:
      // nothing to fetch.  Requested a tile ahead and looked at only when used,
      // or each tile would cost the latency of its table entry.
      constexpr int NOT_SEEN = INT_MIN;
      auto look_up = [&](int j, int &tok) -> int {
        const int k0 = (Seg::key_tile(j, i0, i1, rot, w.sp) << PT_KL) + lane * R;
        tok = k0 & page_mask;
        const bool seen = lane < ppt && k0 < end && (k0 + R > lo || k0 < p.sinks);
        return seen ? p.table[row + (k0 >> p.page_shift)] : NOT_SEEN;
      };
      auto checked = [&](int e) -> int {      // n_pages: zeros
        if (e >= 0 && e < p.n_pages) return e;
        if (e != NOT_SEEN) paged_fail(p, ATTN_ERR_INVALID_ARG);
        return p.n_pages;
      };
      int tok_next = 0, raw_next = look_up(0, tok_next);
      // what the others need to know; by now Q and the first page are on their way
      if (lane == 0) {
        volatile Seg *s = seg_at(qs);
        s->tok0 = tok0;
        s->ntok = tl + 1;
        s->h = w.h * p.hp + sub;
        s->pos0 = pos0;
        s->len = w.s.len;
        s->ns = w.sp.ns;
        s->w0 = w.sp.w0;
        s->i0 = i0;
        s->i1 = i1;
        s->out = i0 == 0 && i1 == w.sp.n ? 0 : at == from ? 1 : 2;
        int np, slot0;
        item_pieces(at - i0, w.sp.n, mine, span, from, np, slot0);
        s->np = np;
        s->slot0 = slot0;
        s->rot = rot;
        mbar_arrive(bar(L::B_IF + qs));
      }
      __syncwarp();
      // The tile of this lane's page into the next ring slot.  With two row tiles
      // the scores of K(j+1) follow the products of V(j), which lies before it in
      // the ring (NS is even): once they are done, both slots are free, by one
      // commit (1 % of the call).
      auto load = [&](const CUtensorMap *tm, int tok, int page, bool values) {
        const int slot = ld % NS;
        const uint32_t was = ld - NS + (TILES == 2 && values ? 1 : 0);
        if (ld >= NS && !wait_all(bar(L::B_EMPTY + was % NS), (was / NS) & 1, abort, lim)) {
          ok = false;
          return;
        }
        // failure-path test only: every CTA leaves its second load out, so that
        // the issuer's bounded wait for it runs out
        if (p.test_stall && ld == 1) {
          ++ld;
          return;
        }
        if (lane == 0) mbar_arrive_expect_tx(bar(L::B_FULL + slot), L::TILE);
        __syncwarp();
        if (lane < ppt)
          for (int hh = 0; hh < L::NHALF; ++hh)
            tma_load_4d(kv_smem + slot * L::TILE + hh * L::HALF + lane * R * 128, tm, bar(L::B_FULL + slot), hh * 64, tok,
                        w.h * p.hp + sub, page);
        ++ld;
      };
      // In the order in which the tensor core takes them, so that no slot waits
      // behind one that is needed later: K_0 V_0 K_1 V_1 .. for two row tiles,
      // K_0 K_1 V_0 K_2 V_1 .. for one.
      int tok = tok_next, page = checked(raw_next);
      if (steps > 1) raw_next = look_up(1, tok_next);
      if (TILES == 1) load(&tm_k, tok, page, false);
      for (int j = 0; j < steps && ok; ++j) {
        int tok1 = 0, page1 = 0;
        if (j + 1 < steps) {
          page1 = checked(raw_next);
          tok1 = tok_next;
          if (j + 2 < steps) raw_next = look_up(j + 2, tok_next);
        }
        if (TILES == 2) load(&tm_k, tok, page, false);
        if (TILES == 1 && j + 1 < steps) load(&tm_k, tok1, page1, false);
        if (ok) load(&tm_v, tok, page, true);
        tok = tok1;
        page = page1;
      }
      if (!ok) break;
      at += steps;
      w.i = i1 - 1;
      if (at == to && lane == 0 && !p.rec) leave_cut<0, PT_KL>(p, w, tpi, w.h * p.hp + sub, blockIdx.x, mine, span, from, to);
      if (at < to) w.next(p, first, info, tpi);
    }
    if (lane == 0) {
      loads[0] = nseg;
      loads[1] = ld;
    }
    __syncwarp();
  } else if (warp == WM) {
    // ---------------------------------------------------------------- issuer
    constexpr uint32_t IDESC_QK = idesc_bf16_f32(128, PT_BN, 0), IDESC_PV = idesc_bf16_f32(128, D, 1);
    // Descriptors as a constant high word and a low word (address and leading
    // offset, in units of 16 bytes) to which each instruction adds a constant:
    // whole descriptors cost the issuing lane more than the tensor core took (the
    // call above took 167 us, not 158).
    const uint32_t q_lo = desc_lo(q_smem, 16), k_lo = desc_lo(kv_smem, 16), v_lo = desc_lo(kv_smem, L::HALF);
    auto issue_qk = [=](int t, int sbuf, int slot) {
      const uint32_t a = q_lo + t * (L::TILE >> 4), b = k_lo + slot * (L::TILE >> 4), d = tmem + sbuf * 128;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk >> 2) * L::HALF + (kk & 3) * 32) >> 4;
        mma_ss_lo(d, a + off, b + off, IDESC_QK, kk > 0);
      }
    };
    // keys kk0 * 16 on, n * 16 of them
    auto issue_pv = [=](int o, int sbuf, int slot, int kk0, int n, bool start) {
      const uint32_t b = v_lo + slot * (L::TILE >> 4) + kk0 * (16 * 128 >> 4), d = tmem + 256 + o * 128, a = tmem + sbuf * 128 + kk0 * 16;
#pragma unroll
      for (int kk = 0; kk < n; ++kk) mma_ts_lo(d, a + kk * 8, b + kk * (16 * 128 >> 4), IDESC_PV, (start && kk == 0) ? 0u : 1u);
    };
    if (lane == 0) {
      // ring position as (slot, phase), advanced without divisions: between
      // groups of matrix instructions this lane's time is the tensor core's
      struct Pos {
        uint32_t slot, ph;
        __device__ __forceinline__ void next() {
          if (++slot == static_cast<uint32_t>(NS)) {
            slot = 0;
            ph ^= 1u;
          }
        }
      };
      Pos k{0, 0};
      uint32_t step = 0, nseg = 0;
      auto wait = [&](uint32_t b, uint32_t ph) { return mbar_wait_bounded(b, ph, abort, lim); };
      // both phases looked at once; the bounded waits only where one is not complete
      auto wait2 = [&](uint32_t a, uint32_t pa, uint32_t b, uint32_t pb) {
        const bool x = mbar_try_wait(a, pa), y = mbar_try_wait(b, pb);
        return (x || wait(a, pa)) && (y || wait(b, pb));
      };
      bool ok = true;
      while (ok) {
        const int qs = nseg % PT_IQ;
        if (!wait(bar(L::B_IF + qs), (nseg / PT_IQ) & 1)) break;
        volatile Seg *s = seg_at(qs);
        const int out = s->out, n = s->i1 - s->i0;
        mbar_arrive(bar(L::B_IE + qs));
        if (out < 0) break;
        if (!wait2(bar(L::B_Q), nseg & 1, bar(L::B_FULL + k.slot), k.ph)) break;
        ++nseg;
        tc_fence_after();
        if constexpr (TILES == 1) {
          // scores of key tile j go to buffer (step + j) & 1
          auto qk = [&](int j, uint32_t buf) {
            issue_qk(0, buf, k.slot);
            mma_commit(bar(L::B_S + buf));
            mma_commit(bar(L::B_EMPTY + k.slot));
            if (j + 1 == n) mma_commit(bar(L::B_QE));
            k.next();
          };
          qk(0, step & 1);
          for (int j = 0; j < n; ++j, ++step) {
            if (j + 1 < n) {
              if (!wait(bar(L::B_FULL + k.slot), k.ph)) {
                ok = false;
                break;
              }
              tc_fence_after();
              qk(j + 1, (step + 1) & 1);
            }
            if (!wait2(bar(L::B_FULL + k.slot), k.ph, bar(L::B_P + (step & 1)), (step >> 1) & 1)) {
              ok = false;
              break;
            }
            tc_fence_after();
            // each group's 64 keys into its own O
            issue_pv(0, step & 1, k.slot, 0, 4, j == 0);
            issue_pv(1, step & 1, k.slot, 4, 4, j == 0);
            mma_commit(bar(L::B_EMPTY + k.slot));
            mma_commit(bar(L::B_V));
            if (j + 1 == n) mma_commit(bar(L::B_O));
            k.next();
          }
        } else {
          issue_qk(0, 0, k.slot);
          mma_commit(bar(L::B_S + 0));
          issue_qk(1, 1, k.slot);
          mma_commit(bar(L::B_S + 1));
          mma_commit(bar(L::B_EMPTY + k.slot));
          if (n == 1) mma_commit(bar(L::B_QE));
          for (int j = 0; j < n; ++j, ++step) {
            const bool more = j + 1 < n;
            Pos v = k;
            v.next();
            k = v;
            k.next();
            if (!wait2(bar(L::B_FULL + v.slot), v.ph, bar(L::B_P + 0), step & 1)) {
              ok = false;
              break;
            }
            tc_fence_after();
            issue_pv(0, 0, v.slot, 0, 8, j == 0);
            if (!more) mma_commit(bar(L::B_O + 0));
            bool have_p1 = false;
            if (more) {
              const bool have_k = mbar_try_wait(bar(L::B_FULL + k.slot), k.ph);
              have_p1 = mbar_test_wait(bar(L::B_P + 1), step & 1);
              if (!have_k && !wait(bar(L::B_FULL + k.slot), k.ph)) {
                ok = false;
                break;
              }
              tc_fence_after();
              issue_qk(0, 0, k.slot);
              mma_commit(bar(L::B_S + 0));
            }
            if (!have_p1 && !wait(bar(L::B_P + 1), step & 1)) {
              ok = false;
              break;
            }
            tc_fence_after();
            issue_pv(1, 1, v.slot, 0, 8, j == 0);
            if (!more) {
              mma_commit(bar(L::B_O + 1));
            } else {
              issue_qk(1, 1, k.slot);
              mma_commit(bar(L::B_S + 1));
              mma_commit(bar(L::B_EMPTY + k.slot));
              if (j + 2 == n) mma_commit(bar(L::B_QE));
            }
          }
        }
      }
      // all matrix instructions are done before tensor memory is freed
      mma_commit(bar(L::B_DRAIN));
      wait_drain(bar(L::B_DRAIN), 0, 20000000ull);
    }
    __syncwarp();
  } else {
    // --------------------------------------------------------------- softmax
    // grp: softmax group and its O; t: row tile.  A group takes NC columns of a
    // tile's scores.
    constexpr int NC = TILES == 1 ? 64 : 128;
    const int grp = warp >> 2, t = TILES == 1 ? 0 : grp, wl = warp & 3, r = wl * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(wl * 32) << 16;
    const uint32_t tO = tmem + lane_off + 256 + grp * 128;
    float2 *xml = reinterpret_cast<float2 *>(smem + L::XML_OFF);
    const float sl2 = p.scale_log2;
    const int tl = r / p.G, g = r - tl * p.G;               // token and head of this row in its tile
    uint32_t step = 0, nseg = 0;
    bool ok = true;
    while (ok) {
      const int qs = nseg % PT_IQ;
      if (!wait_all(bar(L::B_IF + qs), (nseg / PT_IQ) & 1, abort, lim)) break;
      volatile Seg *s = seg_at(qs);
      const int out = s->out, tok0 = s->tok0 + t * tpt, ntok = min(tpt, s->ntok - t * tpt), h = s->h, pos0 = s->pos0 + t * tpt,
                len = s->len, i0 = s->i0, i1 = s->i1, np = s->np, slot0 = s->slot0, rot = s->rot;
      const Span sp{s->ns, s->w0, 0};
      const int it_ntok = s->ntok;         // of both row tiles
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::B_IE + qs));
      if (out < 0) break;
      const bool live = tl < ntok, idle = wl * 32 >= ntok * p.G;    // idle: none of the warp's rows is live
      const int hi = p.causal ? pos0 + tl + 1 : len;               // this row sees keys [lo, hi) and the first ones
      const int lo = p.causal && p.window > 0 ? hi - p.window : 0;
      const int all_hi = p.causal ? pos0 + 1 : len, all_lo = p.causal && p.window > 0 ? pos0 + ntok - p.window : 0;
      float m_ref = -INFINITY, l = 0.f;
      for (int j = 0; j < i1 - i0; ++j, ++step) {
        const int u = TILES == 1 ? step & 1 : t;
        const uint32_t ph = TILES == 1 ? (step >> 1) & 1 : step & 1;
        const uint32_t tS = tmem + lane_off + u * 128 + (TILES == 1 ? grp * 64 : 0);
        const int c0 = Seg::key_tile(j, i0, i1, rot, sp) << PT_KL;
        const bool masked = c0 + 128 > all_hi || (c0 < all_lo && c0 + 128 > p.sinks);
        uint32_t w[4] = {0u, 0u, 0u, 0u};
        bool clear = false;
        if (masked) {
          or_span(max(lo, 0), hi, c0, w);
          if (lo > 0) or_span(0, min(p.sinks, hi), c0, w);
          // does the tile hold keys that no row of the item sees?
          const int it_end = p.causal ? pos0 + it_ntok : len, it_lo = p.causal && p.window > 0 ? pos0 - p.window + 1 : 0;
          clear = grp == 0 && (c0 + 128 > it_end || (c0 < it_lo && c0 + 128 > p.sinks));
        }
        if (!wait_all(bar(L::B_S + u), ph, abort, lim)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (!idle) {
          float x[NC];
          {
            uint32_t y[NC];
#pragma unroll
            for (int c = 0; c < NC / 32; ++c) tmem_ld32(tS + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&y[c * 32]));
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < NC; ++k) {
              asm volatile("" : "+r"(y[k]));
              x[k] = __uint_as_float(y[k]);
            }
          }
          if (masked) {
            if (TILES == 1 && grp == 1) {
              w[0] = w[2];
              w[1] = w[3];
            }
#pragma unroll
            for (int k = 0; k < NC; ++k)
              if (!((w[k >> 5] >> (k & 31)) & 1u)) x[k] = -INFINITY;
          }
          float m4[4];
#pragma unroll
          for (int v = 0; v < 4; ++v) m4[v] = fmaxf(x[2 * v], x[2 * v + 1]);
#pragma unroll
          for (int k = 8; k < NC; k += 8) {
#pragma unroll
            for (int v = 0; v < 4; ++v) m4[v] = max3f(m4[v], x[k + 2 * v], x[k + 2 * v + 1]);
          }
          const float mx = max3f(m4[0], m4[1], fmaxf(m4[2], m4[3])) * sl2;
          const float m_old = m_ref;
          const bool grow = mx > m_ref + PT_TAU;
          if (grow) m_ref = mx;
          const float factor = grow ? ex2_approx(m_old - m_ref) : 1.f;
          l *= factor;
          const float mb = m_ref == -INFINITY ? 0.f : m_ref;
          const uint64_t sc2 = f2_make(sl2, sl2), nb2 = f2_make(-mb, -mb);
          uint64_t l2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
          for (int c = 0; c < NC / 32; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              float a0, a1;
              f2_split(f2_fma(f2_make(x[c * 32 + 2 * k], x[c * 32 + 2 * k + 1]), sc2, nb2), a0, a1);
              a0 = ex2_approx(a0);
              a1 = ex2_approx(a1);
              l2[k & 3] = f2_add(l2[k & 3], f2_make(a0, a1));
              pk[k] = pack_bf16x2(a0, a1);
            }
            tmem_st16(tS + c * 16, pk);
          }
          float a0, a1;
          f2_split(f2_add(f2_add(l2[0], l2[1]), f2_add(l2[2], l2[3])), a0, a1);
          l += a0 + a1;
          const bool rescale = grow && m_old != -INFINITY && j > 0;
          if (__any_sync(0xffffffffu, rescale)) {
            // PV(i-1) has to be done before O is rescaled: with one row tile
            // S(i) does not say so, its QK was issued before that product
            if (TILES == 1 && !wait_all(bar(L::B_V), (step - 1) & 1, abort, lim)) {
              ok = false;
              break;
            }
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t y[32];
              tmem_ld32_wait(tO + c * 32, y);
#pragma unroll
              for (int k = 0; k < 32; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * factor);
              tmem_st32(tO + c * 32, y);
            }
          }
          tmem_wait_st();
        }
        if (clear) {
          // their rows of V become zeros before the product that P's arrival admits
          const int it_end = p.causal ? pos0 + it_ntok : len, it_lo = p.causal && p.window > 0 ? pos0 - p.window + 1 : 0;
          const uint32_t pos = 2 * step + (TILES == 1 && j + 1 < i1 - i0 ? 2 : 1), slot = pos % NS;
          if (!wait_all(bar(L::B_FULL + slot), (pos / NS) & 1, abort, lim)) {
            ok = false;
            break;
          }
#pragma unroll 1
          for (int x = r * 16; x < 128 * 128; x += 128 * 16) {
            const int key = c0 + (x >> 7);
            if (key < it_end && (key >= it_lo || key < p.sinks)) continue;
            for (int hh = 0; hh < L::NHALF; ++hh)
              st_shared_v4(kv_smem + slot * L::TILE + hh * L::HALF + x, make_uint4(0u, 0u, 0u, 0u));
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        mbar_arrive(bar(L::B_P + u));
      }
      if (!ok) break;
      if (!wait_all(bar(L::B_O + t), nseg & 1, abort, lim)) break;
      // TILES = 1: both groups learn each other's (m, l); each then merges and
      // stores its half of the columns
      float f0 = 1.f, f1 = 0.f;
      if constexpr (TILES == 1) {
        xml[grp * 128 + r] = make_float2(m_ref, l);
        mbar_arrive(bar(L::B_X + 0));
        if (!wait_all(bar(L::B_X + 0), nseg & 1, abort, lim)) break;
        const float2 a = xml[r], b = xml[128 + r];
        m_ref = fmaxf(a.x, b.x);
        const float mb = m_ref == -INFINITY ? 0.f : m_ref;
        f0 = ex2_approx(a.x - mb);
        f1 = ex2_approx(b.x - mb);
        l = a.y * f0 + b.y * f1;
      }
      ++nseg;
      tc_fence_after();
      if (!idle) {
        // Four lanes exchange 16-byte words so that each row leaves in 64-byte
        // runs: a lane alone has 16 bytes of 32 different rows an instruction,
        // half sectors that L2 has to merge.  Faster than that by no more than
        // the noise; a segment's epilogue takes 2.1 us to bf16 and 3.7 to f32 pieces.
        const int q4 = lane & 3;
        const bool final = out == 0 && !p.rec, f32 = !final || p.out_f32;
        float fo = 1.f, lse;
        const bool tell = TILES == 2 || grp == 0;
        if (live) {
          const long long row = static_cast<long long>(tok0 + tl) * p.hq + h * p.G + g;
          if (final) {
            row_final(m_ref, l, fo, lse);
            if (tell) p.lse[static_cast<long long>(h * p.G + g) * p.n_tokens + tok0 + tl] = lse;
          } else if (tell) {
            const long long pr = (static_cast<long long>(blockIdx.x) * 2 + out - 1) * (TILES * 128) + t * 128 + r;
            *reinterpret_cast<float2 *>(out ? p.part_ml + pr * 2 : p.dense_ml + row * 2) = make_float2(m_ref, l);
          }
          if (p.rec && i0 == 0 && tell) p.rec[row] = Rec4{static_cast<int>(blockIdx.x), slot0, np, t * 128 + r};
        }
        uint8_t *dst[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int x = r - q4 + k, xt = x / p.G;
          const long long row = static_cast<long long>(tok0 + xt) * p.hq + h * p.G + x - xt * p.G;
          const long long pr = (static_cast<long long>(blockIdx.x) * 2 + out - 1) * (TILES * 128) + t * 128 + x;
          uint8_t *base = static_cast<uint8_t *>(final ? p.out : out ? static_cast<void *>(p.part_o) : static_cast<void *>(p.dense_o));
          dst[k] = xt < ntok ? base + (out ? pr : row) * (D * (f32 ? 4 : 2)) + q4 * 16 : nullptr;
        }
#pragma unroll 1
        for (int c = TILES == 1 ? grp * (D / 64) : 0; c < (TILES == 1 ? (grp + 1) * (D / 64) : D / 32); ++c) {
          uint32_t y[32];
          if constexpr (TILES == 1) {
            uint32_t z[32];
            tmem_ld32(tmem + lane_off + 256 + c * 32, y);
            tmem_ld32(tmem + lane_off + 384 + c * 32, z);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              asm volatile("" : "+r"(y[k]), "+r"(z[k]));
              y[k] = __float_as_uint(fmaf(__uint_as_float(y[k]), f0, __uint_as_float(z[k]) * f1));
            }
          } else {
            tmem_ld32_wait(tO + c * 32, y);
          }
          if (f32) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint4 w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t *z = y + half * 16 + 4 * k;
                w[k] = make_uint4(__float_as_uint(__uint_as_float(z[0]) * fo), __float_as_uint(__uint_as_float(z[1]) * fo),
                                  __float_as_uint(__uint_as_float(z[2]) * fo), __float_as_uint(__uint_as_float(z[3]) * fo));
              }
              exchange4(w, q4);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (dst[k]) *reinterpret_cast<uint4 *>(dst[k] + c * 128 + half * 64) = w[k];
            }
          } else {
            uint4 w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t *z = y + 8 * k;
              auto two = [&](int e) { return pack_bf16x2(__uint_as_float(z[e]) * fo, __uint_as_float(z[e + 1]) * fo); };
              w[k] = make_uint4(two(0), two(2), two(4), two(6));
            }
            exchange4(w, q4);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (dst[k]) *reinterpret_cast<uint4 *>(dst[k] + c * 64) = w[k];
          }
        }
        if (final && pos0 < 0)      // the tile's first tokens stand before the sequence's first key
          zero_row<D, TILES>(p, live && pos0 + tl < 0, static_cast<long long>(tok0 + tl) * p.hq + h * p.G + g, grp);
      }
      tc_fence_before();      // O is read before the next segment's first product
      if constexpr (TILES == 1) {
        // both O by both groups
        mbar_arrive(bar(L::B_X + 1));
        if (!wait_all(bar(L::B_X + 1), (nseg - 1) & 1, abort, lim)) break;
        tc_fence_after();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == WM) tmem_dealloc(tmem, 512);
  if (threadIdx.x == 0 && *abort) {
    paged_fail(p, ATTN_ERR_TIMEOUT);
    land_loads(bar(L::B_Q), bar(L::B_FULL), NS, loads[0], loads[1]);
  }
  end_after_previous(p);
}

// ---------------------------------------------------------------------- host

namespace {

int encode(CUtensorMap *m, const void *base, int rank, const cuuint64_t *dims, const cuuint64_t *strides, const cuuint32_t *box) {
  auto enc = tma_encode_fn();
  if (!enc) return ATTN_ERR_CUDA;
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(base), dims, strides, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? ATTN_OK
             : ATTN_ERR_UNSUPPORTED;
}

template <int D, int TILES>
int launch_tiles(PagedParams &p, const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, cudaStream_t s) {
  using L = TileLayout<D, TILES>;
  const int tpt = 128 / p.G;
  p.warp_plan = TILES == 1 && p.n_seqs <= 32 && (!p.causal || p.n_tokens <= 64ll * tpt);
  if (L::bytes(p, false) > kSmemMax) return ATTN_ERR_UNSUPPORTED;    // above 4000 sequences
  constexpr int kDev = 64;
  static bool done[kDev] = {};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDev) return ATTN_ERR_CUDA;
  auto kern = paged_tiles_kernel<D, TILES>;
  auto join = paged_join_kernel<D, TILES * 128, false>;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (raise_smem(kern, kSmemMax, &done[dev]) != ATTN_OK) return ATTN_ERR_CUDA;
  }
  const int sms = device_sm_count();
  if (sms <= 0) return ATTN_ERR_CUDA;
  p.hp = paged_tiles_heads(sms, p.hk);
  p.n_spans = sms / p.hp;
  p.part_ml = p.part_o + paged_piece_floats(TILES * 128, D);
  p.cuts = reinterpret_cast<Cut *>(p.part_ml + static_cast<size_t>(sms) * 2 * TILES * 128 * 2);
  const bool infos = L::bytes(p, true) <= kSmemMax;
  const int rc = launch_after(kern, dim3(sms), L::THREADS, L::bytes(p, infos), s, mq, mk, mv, p, tpt, infos ? 1 : 0);
  if (rc != ATTN_OK || p.rec) return rc;
  return launch_after(join, dim3(sms, TILES * 8), 256, 0, s, p);
}

}  // namespace

// Heads side by side: as many as divide them while that leaves no more than a
// few SMs idle.
int paged_tiles_heads(int sms, int hk) {
  int hp = 1;
  while (hp < 8 && hk % (2 * hp) == 0 && sms % (2 * hp) <= sms / 32) hp *= 2;
  return hp;
}

size_t paged_tiles_workspace(int d) {
  const int sms = device_sm_count();
  return sms <= 0 ? 0 : static_cast<size_t>(sms) * (2 * 256 * (d + 2) * sizeof(float) + sizeof(Cut));
}

// UNSUPPORTED, with nothing launched, where the tensor maps cannot say the
// layout (more than 128 query heads a key/value head, strides of zero).
int paged_tiles_launch(PagedParams &p, int d, int tokens, cudaStream_t s, int *tile_rows) {
  if (p.G > 128) return ATTN_ERR_UNSUPPORTED;
  // ATTN_TEST_STALL_PAGED=1 in the environment: the launch ends by its bounded
  // waits running out, which is how the tests drive its abort path
  const char *stall = std::getenv("ATTN_TEST_STALL_PAGED");
  p.test_stall = stall && stall[0] == '1';
  const int page = 1 << p.page_shift, tpt = 128 / p.G;
  CUtensorMap mq, mk, mv;
  int rc;
  {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(p.hq), static_cast<cuuint64_t>(p.n_tokens)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(p.hq) * d * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(p.G), static_cast<cuuint32_t>(tpt)};
    if ((rc = encode(&mq, p.q, 3, dims, strides, box)) != ATTN_OK) return rc;
  }
  {
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(page), static_cast<cuuint64_t>(p.hk),
                                static_cast<cuuint64_t>(p.n_pages)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(p.token_stride) * 2, static_cast<cuuint64_t>(p.head_stride) * 2,
                                   static_cast<cuuint64_t>(p.page_stride) * 2};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(page < 128 ? page : 128), 1, 1};
    if ((rc = encode(&mk, p.k, 4, dims, strides, box)) != ATTN_OK) return rc;
    if ((rc = encode(&mv, p.v, 4, dims, strides, box)) != ATTN_OK) return rc;
  }
  const bool two = tokens > tpt;
  *tile_rows = two ? 256 : 128;
  if (d == 128) return two ? launch_tiles<128, 2>(p, mq, mk, mv, s) : launch_tiles<128, 1>(p, mq, mk, mv, s);
  return two ? launch_tiles<64, 2>(p, mq, mk, mv, s) : launch_tiles<64, 1>(p, mq, mk, mv, s);
}

}  // namespace attn
