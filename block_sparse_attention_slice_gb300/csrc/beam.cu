// A beam search's step: the best continuations of each prompt, and the beams' states
// brought into their order.
//
// A continuation's score is c_b + logit, with c_b = score_b - ln sum exp(logit): of one
// beam's continuations the best are those of its largest logits, so one pass over the
// logits gives both the sum and, for every part of a row, its `keep` largest.  The rest
// is small: a block a prompt adds the parts' sums, compares the parts' best as 64-bit
// scores and keeps the best of them all.
//
// beam_scan_kernel: a warp takes a part of a row as a stream, keeps the running maximum and
// sum of each lane, and the best so far, one or two a lane in their order.  16 bytes are
// looked into only where their largest value beats the last of them, which gets rare: 512
// rows of 131072 bf16 take 37 us (a block a part, its threshold by an exchange and its
// candidates ranked in shared memory, took half as long again).  The first
// words have a threshold of their own, the `keep`-th of the lanes' largest values.  Values are
// compared as whole numbers in the order of the floats, -0 as 0.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/attn_beam.h"
#include "attn_device.cuh"
#include "attn_internal.h"
#include "launch.cuh"

namespace attn {

namespace {

constexpr int BS_T = 256;            // threads of a scanning block
constexpr int BS_REGS = 16;          // words of 4 bytes that a lane of it takes at a time, in groups of 4
constexpr int BP_T = 256;            // of a choosing block
constexpr int BP_CAP = 1024;

// The order of the floats as whole numbers; -inf is 0x007fffff, 0 stands for no value.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return max((b & 0x80000000u) ? ~b : b | 0x80000000u, 1u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ unsigned long long key_of(double x) {
  const unsigned long long b = static_cast<unsigned long long>(__double_as_longlong(x)), top = 1ull << 63;
  return b >= top ? b == top ? top : ~b : b | top;
}
__device__ __forceinline__ double value_of(unsigned long long k) {
  return __longlong_as_double(static_cast<long long>((k >> 63) ? k ^ 1ull << 63 : ~k));
}

// A key, not 0, that at least min(keep, keys there are) of the block's keys reach, given
// the largest of each thread's (0: none), of which the first `active` have some;
// keep <= 64.  `sums` has a place a warp.
template <int T>
__device__ __forceinline__ unsigned long long threshold(unsigned long long top, int keep, int active, unsigned long long *sums) {
  // groups of as many threads as leave `keep` of them, a warp at most
  int width = 32;
  while (width > 1 && active < keep * width) width >>= 1;
  for (int o = 1; o < width; o <<= 1) {
    const unsigned long long a = __shfl_xor_sync(0xffffffffu, top, o);
    top = a > top ? a : top;
  }
  if (static_cast<int>(threadIdx.x & ~(width - 1)) >= active) top = ~0ull;
  for (int o = width; o < 32; o <<= 1) {
    const unsigned long long a = __shfl_xor_sync(0xffffffffu, top, o);
    top = a < top ? a : top;
  }
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < T / 32; ++w) top = sums[w] < top ? sums[w] : top;
  return top < 1 || active < keep ? 1 : top;
}

// Whether (a, i) stands before (b, j).
template <typename K>
__device__ __forceinline__ bool before(K a, int i, K b, int j) {
  return a > b || (a == b && i < j);
}

// The best of (k, i) over the block, for every thread; equal ones by the lowest i.
template <int T, typename K>
__device__ __forceinline__ void block_best(K &k, int &i, K *ks, int *is) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const K a = __shfl_xor_sync(0xffffffffu, k, o);
    const int j = __shfl_xor_sync(0xffffffffu, i, o);
    if (before(a, j, k, i)) k = a, i = j;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) ks[threadIdx.x >> 5] = k, is[threadIdx.x >> 5] = i;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < T / 32; ++w)
    if (before(ks[w], is[w], k, i)) k = ks[w], i = is[w];
}

// Writes the best of n listed keys: a warp takes an entry at a time and counts those that
// stand before it, 32 together.
template <int T, typename B, typename W>
__device__ __forceinline__ void rank_list(int n, int keep, B stands_before, W write) {
  const int lane = threadIdx.x & 31;
  for (int i = threadIdx.x >> 5; i < n; i += T / 32) {
    int rank = 0;
    if (n <= 32) {
      rank = __popc(__ballot_sync(0xffffffffu, lane < n && stands_before(lane, i)));
      if (lane == 0 && rank < keep) write(rank, i);
      continue;
    }
    for (int j0 = 0; j0 < n && rank < keep; j0 += 32) rank += __popc(__ballot_sync(0xffffffffu, j0 + lane < n && stands_before(j0 + lane, i)));
    if (lane == 0 && rank < keep) write(rank, i);
  }
}

struct ScanParams {
  const void *logits;
  const uint8_t *done;
  long long row_stride;      // elements
  int vocab, splits, keep, units, rest, parts;       // a part: `units` of the row, the first `rest` of a row one more; parts: of all rows
  float2 *ms;                // [rows][splits]: maximum, sum of exp(x - maximum)
  uint32_t *keys;            // [rows][splits][keep], best first
  int *ids;                  // their tokens; -1: none
};

// A lane's logits: units of UNIT bytes, N values each, in registers of V values.
template <typename E, int UNIT>
struct Vec {
  static constexpr int N = UNIT / static_cast<int>(sizeof(E)), V = UNIT == 2 ? 1 : 4 / static_cast<int>(sizeof(E));
  static constexpr int REGS = N / V, UNITS = BS_REGS / REGS;      // registers of a unit; units of a lane
  static constexpr uint32_t NONE = sizeof(E) == 4 ? 0xff800000u : V == 2 ? 0xff80ff80u : 0xff80u;      // -inf
  // value e of a register
  static __device__ __forceinline__ float get(uint32_t x, int e) {
    return __uint_as_float(sizeof(E) == 4 ? x : e ? x & 0xffff0000u : x << 16);
  }
  // the largest of 4 registers; a NaN is passed by
  static __device__ __forceinline__ float top(const uint32_t *x) {
    if constexpr (V == 1) {
      return fmaxf(max3f(get(x[0], 0), get(x[1], 0), get(x[2], 0)), get(x[3], 0));
    } else {
      uint32_t a, b;
      asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(x[0]), "r"(x[1]));
      asm("max.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(x[2]), "r"(x[3]));
      asm("max.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
      return fmaxf(get(a, 0), get(a, 1));
    }
  }
  // the unit at p, which is aligned to it
  static __device__ __forceinline__ void load(const E *p, uint32_t *x) {
    if constexpr (UNIT == 16) {
      const uint4 w = __ldcs(reinterpret_cast<const uint4 *>(p));
      x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w;
    } else if constexpr (UNIT == 4) {
      x[0] = __ldcs(reinterpret_cast<const uint32_t *>(p));
    } else {
      x[0] = __ldcs(reinterpret_cast<const uint16_t *>(p));
    }
  }
  static __device__ __forceinline__ uint32_t bits(const E *p) {
    if constexpr (sizeof(E) == 4) return __float_as_uint(*p);
    else return *p;
  }
};

// The best `keep` so far of a warp's part: place lane + 32 i of their order is best i of a
// lane; key 0: none.
template <int R>
struct Best {
  uint32_t k[R];
  int id[R];
  __device__ __forceinline__ Best() {
#pragma unroll
    for (int i = 0; i < R; ++i) k[i] = 0, id[i] = INT_MAX;
  }
  // the last of them: what a new one has to beat
  __device__ __forceinline__ void last(int keep, uint32_t &lk, int &li) const {
    const int i = R == 2 && keep > 32;
    lk = __shfl_sync(0xffffffffu, i ? k[R - 1] : k[0], (keep - 1) & 31);
    li = __shfl_sync(0xffffffffu, i ? id[R - 1] : id[0], (keep - 1) & 31);
  }
  __device__ __forceinline__ void insert(uint32_t ck, int ci) {
    const int lane = threadIdx.x & 31;
    int at = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) at += __popc(__ballot_sync(0xffffffffu, before(k[i], id[i], ck, ci)));
#pragma unroll
    for (int i = R - 1; i >= 0; --i) {
      uint32_t pk = __shfl_up_sync(0xffffffffu, k[i], 1);
      int pi = __shfl_up_sync(0xffffffffu, id[i], 1);
      if (i > 0) {
        const uint32_t ok = __shfl_sync(0xffffffffu, k[i - 1], 31);
        const int oi = __shfl_sync(0xffffffffu, id[i - 1], 31);
        if (lane == 0) pk = ok, pi = oi;
      }
      const int place = lane + 32 * i;
      if (place > at) k[i] = pk, id[i] = pi;
      if (place == at) k[i] = ck, id[i] = ci;
    }
  }
};

// E: the logits' type; R: best a lane.  A row is taken by its units of UNIT bytes wherever it
// begins; of a unit that the row's ends cut the values outside count as -inf and are no
// candidates.  A unit divides the distance of two rows, so that all rows are cut alike: equal rows have
// equal sums to the last bit, whatever their addresses, and their beams stand in order.  The choice
// for 64 prompts of 8 beams, bf16: 131072 tokens in units of 16 bytes 47.2 us, 131070 in units of 4 47.4,
// 131071 in units of 2 56.6; 24 of 5, f32: 100004 and 100003 tokens 26.0, 25.2.
template <typename E, int UNIT, int R>
__global__ void __launch_bounds__(BS_T, 3) beam_scan_kernel(const ScanParams p) {
  using X = Vec<E, UNIT>;
  constexpr int N = X::N, V = X::V, Q = X::REGS, W = X::UNITS, STEP = 32 * W;
  after_previous();
  admit_next();
  const int lane = threadIdx.x & 31;
  const int at = blockIdx.x * (BS_T / 32) + (threadIdx.x >> 5);
  if (at >= p.parts) return;
  const int row = at / p.splits, split = at - row * p.splits;
  if (p.done && p.done[row]) return;
  const E *base = static_cast<const E *>(p.logits) + row * p.row_stride;
  const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(base) & (UNIT - 1)) / sizeof(E));
  const int begin = split * p.units + min(split, p.rest), end = begin + p.units + (split < p.rest);
  // units u of them, u = from + 32 i + lane
  auto load = [&](int from, uint32_t (&x)[BS_REGS]) {
    const bool inner = from > 0 && (from + STEP) * N - skew <= p.vocab && from + STEP <= end;
    if (inner) {
      const E *src = base - skew + (static_cast<long long>(from) + lane) * N;
#pragma unroll
      for (int i = 0; i < W; ++i) X::load(src + 32 * i * N, x + Q * i);
      return;
    }
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const int u = from + 32 * i + lane;
      const long long v = u < end ? static_cast<long long>(u) * N - skew : p.vocab;
      if (v >= 0 && v + N <= p.vocab) {
        X::load(base + v, x + Q * i);
        continue;
      }
#pragma unroll
      for (int k = 0; k < Q; ++k) {
        uint32_t z = X::NONE;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const long long y = v + k * V + e;
          const int by = 32 / V * e;
          if (y >= 0 && y < p.vocab) z = V == 1 ? X::bits(base + y) : (z & ~(0xffffu << by)) | X::bits(base + y) << by;
        }
        x[Q * i + k] = z;
      }
    }
  };
  uint32_t next[BS_REGS];
  load(begin, next);
  Best<R> best;
  uint32_t last_k = 0;       // what a candidate has to beat: this key, with a lower token
  int last_i = INT_MAX;
  float m = -INFINITY, s = 0.f;
  bool first = true;
  for (int from = begin; from < end; from += STEP) {
    uint32_t x[BS_REGS];
#pragma unroll
    for (int i = 0; i < BS_REGS; ++i) x[i] = next[i];
    if (from + STEP < end) load(from + STEP, next);
    // maximum (a NaN is passed by, and spoils the sum)
    float mw[BS_REGS / 4];
#pragma unroll
    for (int i = 0; i < BS_REGS / 4; ++i) mw[i] = X::top(x + 4 * i);
    const float top = fmaxf(fmaxf(mw[0], mw[1]), fmaxf(mw[2], mw[3]));
    static_assert(BS_REGS == 16, "the maximum of a lane's groups");
    const uint32_t key = key_of(top);
    // tokens ascend: what is equal to the last of the best comes behind it
    uint32_t least = max(last_k, last_k + 1);
    if (first) {
      // the `keep`-th of the lanes' largest: `keep` values reach it, and few more (equal ones
      // leave together, so that it may be less); of fewer lanes every value counts
      uint32_t k = key;
      least = p.keep <= 32 ? 0xffffffffu : 0u;
      for (int i = 0; i < p.keep && least; ++i) {
        least = __reduce_max_sync(0xffffffffu, k);
        if (k == least) k = 0u;
      }
    }
    if (__any_sync(0xffffffffu, key >= least)) {
#pragma unroll
      for (int g = 0; g < BS_REGS / 4; ++g) {
        for (unsigned hot = __ballot_sync(0xffffffffu, key_of(mw[g]) >= least); hot; hot &= hot - 1) {
          // the group's values to as many lanes
          const int src = __ffs(hot) - 1;
          const uint32_t y0 = __shfl_sync(0xffffffffu, x[4 * g], src), y1 = __shfl_sync(0xffffffffu, x[4 * g + 1], src),
                         y2 = __shfl_sync(0xffffffffu, x[4 * g + 2], src), y3 = __shfl_sync(0xffffffffu, x[4 * g + 3], src);
          const int part = lane / V;
          const uint32_t k = key_of(X::get(part & 2 ? (part & 1 ? y3 : y2) : (part & 1 ? y1 : y0), lane % V));
          const int unit = from + 32 * ((4 * g + part) / Q) + src;
          const long long token = static_cast<long long>(unit) * N - skew + lane % N;
          const int id = static_cast<int>(token);
          const bool there = lane < 4 * V && unit < end && token >= 0 && token < p.vocab && k >= least;
          for (unsigned c = __ballot_sync(0xffffffffu, there && before(k, id, last_k, last_i)); c; c &= c - 1) {
            const int e = __ffs(c) - 1;
            const uint32_t ck = __shfl_sync(0xffffffffu, k, e);
            const int ci = __shfl_sync(0xffffffffu, id, e);
            if (!before(ck, ci, last_k, last_i)) continue;       // the ones before it left no room
            best.insert(ck, ci);
            best.last(p.keep, last_k, last_i);
          }
        }
        // a group's tokens stand behind those of the one before, in no order of their own
        least = max(least, max(last_k, last_k + 1));
      }
    }
    first = false;
    // the lane's maximum and sum
    const float to = fmaxf(m, top), mb = to == -INFINITY ? 0.f : to;
    s *= ex2_approx((m - mb) * 1.44269504f);
    m = to;
    const uint64_t nm = f2_make(-mb, -mb), c2 = f2_make(1.44269504f, 1.44269504f);
    uint64_t s2 = 0ull;
#pragma unroll
    for (int e = 0; e < BS_REGS * V; e += 2) {
      float a, b;
      f2_split(f2_mul(f2_add(f2_make(X::get(x[e / V], e % V), X::get(x[(e + 1) / V], (e + 1) % V)), nm), c2), a, b);
      s2 = f2_add(s2, f2_make(ex2_approx(a), ex2_approx(b)));
    }
    float a, b;
    f2_split(s2, a, b);
    s += a + b;
  }
  float most = m;
#pragma unroll
  for (int o = 16; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  s *= ex2_approx((m - (most == -INFINITY ? 0.f : most)) * 1.44269504f);
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) p.ms[at] = make_float2(most, s);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int place = lane + 32 * i;
    if (place >= p.keep) continue;
    p.keys[static_cast<long long>(at) * p.keep + place] = best.k[i];
    p.ids[static_cast<long long>(at) * p.keep + place] = best.k[i] ? best.id[i] : -1;
  }
}

struct PickParams {
  const float *scores;
  const uint8_t *done;
  const int32_t *slots;
  const float2 *ms;
  const uint32_t *keys;
  const int *ids;
  int beams, vocab, splits, keep, eos;
  float *out_scores;
  int32_t *out_parents, *out_tokens, *out_src;
  uint8_t *out_done;
};

// One block a group, 10 us behind its scan for 24 and for 64 groups (9.4 alone): dependent loads, the
// sums in 64 bits, one exchange and the ranks of what is left.  Continuations are the parts' best, and of a beam that offers
// nothing the first `keep` by their place, at -inf (of one that has ended its eos, then
// those), so that the choice needs no other rule.
__global__ void __launch_bounds__(BP_T) beam_pick_kernel(const PickParams p) {
  __shared__ double offset[ATTN_BEAM_MAX];      // score - ln sum; NaN: the beam offers nothing but -inf
  __shared__ unsigned long long sums[BP_T / 32];
  __shared__ int isum[BP_T / 32];
  __shared__ unsigned long long list_k[BP_CAP];
  __shared__ int list_b[BP_CAP], list_v[BP_CAP];
  __shared__ int listed, source[ATTN_BEAM_MAX];
  __shared__ bool ended[ATTN_BEAM_MAX];
  after_previous();
  admit_next();
  const int g = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, per = p.splits * p.keep, n = p.beams * per;
  if (threadIdx.x == 0) listed = 0;
  // a thread's first candidates are on their way while the beams' sums are made
  // In the order beam, part, rank: neighbours are of different beams and parts, so that
  // every group of threads has good ones.
  auto entry = [&](int c) { return (c % p.splits) * p.keep + c / p.splits; };
  constexpr int HELD = 4;
  int hb[HELD], hv[HELD];
  uint32_t hx[HELD];
  int hc[HELD];
  const int c_step = BP_T / p.beams, b_step = BP_T - c_step * p.beams;
#pragma unroll
  for (int i = 0; i < HELD; ++i) {
    if (i == 0) {
      hc[0] = threadIdx.x / p.beams;
      hb[0] = threadIdx.x - hc[0] * p.beams;
    } else {
      const int b = hb[i - 1] + b_step;
      hb[i] = b - (b >= p.beams ? p.beams : 0);
      hc[i] = hc[i - 1] + c_step + (b >= p.beams);
    }
    hv[i] = -1;
    hx[i] = 0;
    if (static_cast<int>(threadIdx.x) + i * BP_T < n) {
      const long long at = (static_cast<long long>(g) * p.beams + hb[i]) * per + entry(hc[i]);
      hv[i] = p.ids[at];
      hx[i] = p.keys[at];
    }
  }
  for (int b = warp; b < p.beams; b += BP_T / 32) {
    const long long row = static_cast<long long>(g) * p.beams + b;
    double c = __longlong_as_double(0x7ff8000000000000ll);
    // all that is read of a beam is asked for at once
    const float2 y0 = lane < p.splits ? p.ms[row * p.splits + lane] : make_float2(-INFINITY, 0.f);
    const float score = p.scores[row];
    const bool over = p.done && p.done[row];
    const int from = p.slots ? p.slots[row] : static_cast<int>(row);
    if (lane == 0) ended[b] = over, source[b] = from;
    if (!over && score > -INFINITY && score < INFINITY) {
      // the parts' sums brought to the largest maximum
      float m = -INFINITY, s = 0.f;
      for (int i0 = 0; i0 < p.splits; i0 += 32) {
        const float2 y = i0 == 0 ? y0 : i0 + lane < p.splits ? p.ms[row * p.splits + i0 + lane] : make_float2(-INFINITY, 0.f);
        float top = y.x;
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        top = fmaxf(top, m);
        const float mb = top == -INFINITY ? 0.f : top;
        // a part of -inf alone has the sum 0; one with a NaN keeps it
        s = s * ex2_approx((m - mb) * 1.44269504f) + y.y * (y.x == -INFINITY ? 0.f : ex2_approx((y.x - mb) * 1.44269504f));
        m = top;
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      // ln s = e ln 2 + ln f with f in [3/4, 3/2): to 2^-24 of 1, not of ln s; few
      // operations in 64 bits, which take a warp 16 cycles each here
      const int e = static_cast<int>(__float_as_uint(s) - 0x3f400000u) >> 23;
      const float f = __uint_as_float(__float_as_uint(s) - (static_cast<uint32_t>(e) << 23));
      if (s > 0.f && s < INFINITY)
        c = static_cast<double>(score) - (static_cast<double>(m) + (e * 0.69314718055994530942 + static_cast<double>(log1pf(f - 1.f))));
      if (!(c > -INFINITY && c < INFINITY)) c = __longlong_as_double(0x7ff8000000000000ll);
    }
    if (lane == 0) offset[b] = c;
  }
  __syncthreads();
  // Continuation j: its score as a key (0: none), beam and token.
  auto score_of = [&](int i, int b, uint32_t x, int &v) -> unsigned long long {
    const long long row = static_cast<long long>(g) * p.beams + b;
    const double c = offset[b];
    if (c == c) return v >= 0 ? key_of(c + static_cast<double>(value_of(x))) : 0ull;
    unsigned long long k = 0;
    if (i < p.keep) {
      const float score = p.scores[row];
      const bool over = ended[b] && score > -INFINITY && score < INFINITY;
      if (over && i == 0) {
        v = p.eos;
        k = key_of(static_cast<double>(score));
      } else {
        v = over ? i - 1 + (i - 1 >= p.eos) : i;
        if (v < p.vocab) k = key_of(-static_cast<double>(INFINITY));
      }
    }
    return k;
  };
  auto get = [&](int j, unsigned long long &k, int &b, int &v) {
    const int i = j / p.beams;
    b = j - i * p.beams;
    const long long at = (static_cast<long long>(g) * p.beams + b) * per + entry(i);
    v = p.ids[at];
    k = score_of(i, b, p.keys[at], v);
  };
  unsigned long long hk[HELD], top = 0;
#pragma unroll
  for (int i = 0; i < HELD; ++i) {
    hk[i] = static_cast<int>(threadIdx.x) + i * BP_T < n ? score_of(hc[i], hb[i], hx[i], hv[i]) : 0ull;
    top = hk[i] > top ? hk[i] : top;
  }
  for (int j = threadIdx.x + HELD * BP_T; j < n; j += BP_T) {
    unsigned long long k;
    int b, v;
    get(j, k, b, v);
    top = k > top ? k : top;
  }
  const unsigned long long least = threshold<BP_T>(top, p.keep, min(BP_T, n), sums);
  auto list = [&](unsigned long long k, int b, int v) {
    if (k < least) return;
    const int at = atomicAdd(&listed, 1);
    if (at < BP_CAP) list_k[at] = k, list_b[at] = b, list_v[at] = v;
  };
#pragma unroll
  for (int i = 0; i < HELD; ++i) list(hk[i], hb[i], hv[i]);
  for (int j = threadIdx.x + HELD * BP_T; j < n; j += BP_T) {
    unsigned long long k;
    int b, v;
    get(j, k, b, v);
    list(k, b, v);
  }
  __syncthreads();
  auto write = [&](int r, unsigned long long k, int b, int v) {
    const long long to = static_cast<long long>(g) * p.keep + r, row = static_cast<long long>(g) * p.beams + b;
    p.out_scores[to] = static_cast<float>(value_of(k));
    p.out_parents[to] = static_cast<int32_t>(row);
    p.out_tokens[to] = v;
    if (p.out_done) p.out_done[to] = ended[b] || v == p.eos;
    if (p.out_src) p.out_src[to] = source[b];
  };
  const int m = listed;
  if (m <= BP_CAP) {
    rank_list<BP_T>(
        m, p.keep,
        [&](int x, int y) {
          return list_k[x] > list_k[y] || (list_k[x] == list_k[y] && (list_b[x] < list_b[y] || (list_b[x] == list_b[y] && list_v[x] < list_v[y])));
        },
        [&](int rank, int i) { write(rank, list_k[i], list_b[i], list_v[i]); });
    return;
  }
  unsigned long long last_k = ~0ull;
  long long last_at = -1;
  for (int r = 0; r < p.keep; ++r) {
    // beams first, then tokens: two rounds find the place of the best that is left
    unsigned long long k = 0;
    int b = INT_MAX, v = INT_MAX;
    for (int j = threadIdx.x; j < n; j += BP_T) {
      unsigned long long y;
      int c, w;
      get(j, y, c, w);
      const long long at = static_cast<long long>(c) * p.vocab + w;
      if (y && (y < last_k || (y == last_k && at > last_at)) && (y > k || (y == k && (c < b || (c == b && w < v))))) k = y, b = c, v = w;
    }
    unsigned long long bk = k;
    int bb = b;
    block_best<BP_T>(bk, bb, sums, isum);
    int bv = k == bk && b == bb ? v : INT_MAX;
    unsigned long long one = k == bk && b == bb ? 1 : 0;
    block_best<BP_T>(one, bv, sums, isum);
    if (threadIdx.x == 0) write(r, bk, bb, bv);
    last_k = bk;
    last_at = static_cast<long long>(bb) * p.vocab + bv;
  }
}

// -------------------------------------------------------------------- reorder

struct State {
  uint8_t *at;
  long long stride, bytes;   // from row to row, of a row
  int loose, first;          // not in words of 16 bytes; the state's first unit
};
struct ReorderParams {
  State s[ATTN_BEAM_MAX_STATES];
  const int32_t *parents;
  int n_states, groups, beams, units;
  unsigned int *status;
};
constexpr int RE_T = 256;
// Bytes of a row that a unit moves: a word of 16 bytes a thread; or a power of two that leaves
// all rows room for 32 KB.
__host__ __device__ __forceinline__ int unit_bytes(bool loose, int beams) {
  return !loose ? RE_T * 16 : beams <= 16 ? 2048 : beams <= 32 ? 1024 : 512;
}
// A row of it in shared memory lies as in memory, up to 15 bytes behind a word's beginning.
__host__ __device__ __forceinline__ int run_pitch(int beams) { return unit_bytes(true, beams) + 32; }

// All parents' words of one column of a group, then all rows': the column is this
// thread's alone, so the rows may change places in memory.  Rows that stay are not
// touched.  64 groups of 8 rows of 139 KB: 15.3 us a call, the most part from and to L2.
template <int MOST>
__device__ __forceinline__ void move_column(uint8_t *base, long long stride, const int *par, int beams) {
  uint4 x[MOST];
#pragma unroll
  for (int b = 0; b < MOST; ++b)
    if (b < beams && par[b] != b) x[b] = *reinterpret_cast<const uint4 *>(base + par[b] * stride);
#pragma unroll
  for (int b = 0; b < MOST; ++b)
    if (b < beams && par[b] != b) *reinterpret_cast<uint4 *>(base + b * stride) = x[b];
}

// Words of 16 bytes that lie wholly in n bytes that begin `skew` behind a word: of `head`
// bytes before the first, and how many.
__device__ __forceinline__ int whole_words(int n, int skew, int &head) {
  head = min((16 - skew) & 15, n);
  return (n - head) >> 4;
}

// The same for `n` bytes of rows at any address, or of more than 16 beams, through shared
// memory: words of 16 bytes where they lie in memory, read as they are and written as two of
// them shifted into the new row's place.  (24 groups of 5 rows of 100003 bytes: 8.9 us a
// call, 12.3 alone with cold caches; words of 4 bytes, whose instructions bound it, took twice that, bytes four times as long again.)  The bytes at the
// ends of the run are moved alone, those outside it neither read nor written.
__device__ __forceinline__ void move_run(uint8_t *base, long long stride, int n, const int *par, const int *used, int n_used, int beams, uint8_t *buf) {
  constexpr int BATCH = 4;
  const int pitch = run_pitch(beams), slots = unit_bytes(true, beams) / 16, shift = 31 - __clz(slots);
  auto skew_of = [&](int row) { return static_cast<int>(reinterpret_cast<uintptr_t>(base + row * stride) & 15); };
  for (int i0 = threadIdx.x; i0 < n_used << shift; i0 += RE_T * BATCH) {
    uint4 w[BATCH];
    uint8_t *to[BATCH];
#pragma unroll
    for (int q = 0; q < BATCH; ++q) {
      const int i = i0 + q * RE_T, x = i >> shift, j = i & (slots - 1);
      to[q] = nullptr;
      if (x >= n_used) continue;
      const int row = used[x], skew = skew_of(row);
      int head;
      if (j >= whole_words(n, skew, head)) continue;
      w[q] = *reinterpret_cast<const uint4 *>(base + row * stride + head + 16 * j);
      to[q] = buf + row * pitch + skew + head + 16 * j;
    }
#pragma unroll
    for (int q = 0; q < BATCH; ++q)
      if (to[q]) *reinterpret_cast<uint4 *>(to[q]) = w[q];
  }
  // place e of 32 of the bytes before and behind the whole words; -1: none
  auto end_byte = [&](int e, int skew) -> int {
    int head;
    const int behind = 16 * whole_words(n, skew, head) + head + e - 16;
    return e < 16 ? (e < head ? e : -1) : behind < n ? behind : -1;
  };
  for (int i = threadIdx.x; i < n_used * 32; i += RE_T) {
    const int row = used[i >> 5], skew = skew_of(row), t = end_byte(i & 31, skew);
    if (t >= 0) buf[row * pitch + skew + t] = base[row * stride + t];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < beams << shift; i += RE_T) {
    const int row = i >> shift, j = i & (slots - 1), from = par[row];
    if (from == row) continue;
    int head;
    if (j >= whole_words(n, skew_of(row), head)) continue;
    const int at = skew_of(from) + head + 16 * j;
    const uint4 *src = reinterpret_cast<const uint4 *>(buf + from * pitch + (at & ~15));
    const uint4 a = src[0], b = at & 15 ? src[1] : make_uint4(0u, 0u, 0u, 0u);
    // of the eight words the four from at / 4 on, and one more
    const bool two = at & 8, one = at & 4;
    const uint32_t x0 = two ? a.z : a.x, x1 = two ? a.w : a.y, x2 = two ? b.x : a.z, x3 = two ? b.y : a.w, x4 = two ? b.z : b.x, x5 = two ? b.w : b.y;
    const uint32_t y0 = one ? x1 : x0, y1 = one ? x2 : x1, y2 = one ? x3 : x2, y3 = one ? x4 : x3, y4 = one ? x5 : x4;
    const int by = 8 * (at & 3);
    *reinterpret_cast<uint4 *>(base + row * stride + head + 16 * j) =
        make_uint4(__funnelshift_r(y0, y1, by), __funnelshift_r(y1, y2, by), __funnelshift_r(y2, y3, by), __funnelshift_r(y3, y4, by));
  }
  for (int i = threadIdx.x; i < beams * 32; i += RE_T) {
    const int row = i >> 5, from = par[row], t = end_byte(i & 31, skew_of(row));
    if (from != row && t >= 0) base[row * stride + t] = buf[from * pitch + skew_of(from) + t];
  }
}

// RUNS: some state is loose; 64 registers then, for more blocks an SM (runs of 5 rows: 15.6, 10.7
// us when that was chosen), which columns of 8 rows would pay for (15.0, 24.5).
template <int MOST, bool RUNS>
__global__ void __launch_bounds__(RE_T, !RUNS ? 1 : MOST <= 8 ? 4 : 2) beam_reorder_kernel(const __grid_constant__ ReorderParams p) {
  __shared__ int par[ATTN_BEAM_MAX], used[ATTN_BEAM_MAX], n_used;
  extern __shared__ uint4 runs[];       // run_pitch(beams) bytes a row, where some state is loose
  after_previous();
  admit_next();
  int s = 0;
  for (int u = blockIdx.x; u < p.units; u += gridDim.x) {
    while (s + 1 < p.n_states && u >= p.s[s + 1].first) ++s;
    const State &st = p.s[s];
    const int each = unit_bytes(st.loose, p.beams);
    const long long per = (st.bytes + each - 1) / each, g = (u - st.first) / per, row0 = g * p.beams;
    const long long at = (u - st.first - g * per) * each;
    __syncthreads();
    const int b = threadIdx.x;
    int off = 0;
    if (b < p.beams) {
      const long long a = p.parents[row0 + b] - row0;
      off = a < 0 || a >= p.beams;
      par[b] = off ? b : static_cast<int>(a);
    }
    if (__syncthreads_or(off)) {
      if (threadIdx.x == 0) atomicCAS(p.status, 0u, static_cast<unsigned>(ATTN_ERR_INVALID_ARG));
      continue;
    }
    uint8_t *base = st.at + row0 * st.stride + at;
    if (!RUNS || !st.loose) {
      if (at + 16 * threadIdx.x < st.bytes) move_column<MOST>(base + 16 * threadIdx.x, st.stride, par, p.beams);
    } else {
      if (b < 32) {          // the rows that others become
        int count = 0;
        for (int r0 = 0; r0 < p.beams; r0 += 32) {
          const int r = r0 + b;
          bool on = false;
          for (int k = 0; k < p.beams; ++k) on |= r < p.beams && k != r && par[k] == r;
          const unsigned all = __ballot_sync(0xffffffffu, on);
          if (on) used[count + __popc(all & ((1u << b) - 1))] = r;
          count += __popc(all);
        }
        if (b == 0) n_used = count;
      }
      __syncthreads();
      move_run(base, st.stride, static_cast<int>(min(static_cast<long long>(each), st.bytes - at)), par, used, n_used, p.beams, reinterpret_cast<uint8_t *>(runs));
    }
  }
}

// Parts of a row, a warp each: as many as fill the SMs with 24 warps (64 prompts of 8 beams
// and 131072 tokens, the whole step when that was chosen: 63.6 us; 20 warps 69.3; 32, of 64 registers a thread, 72.1),
// of what a warp takes at a time at least.  n: values of a unit; units: of a row, wherever it
// begins.  Not more than leave a group's choice 16384 candidates.
int splits_of(int groups, int beams, int vocab, int keep, int n, int per_lane, int sms, int *units) {
  *units = (vocab + 2 * n - 2) / n;
  const int step = 32 * per_lane / n, most = (*units + step - 1) / step;
  return std::max(1, std::min({most, sms * 24 / std::max(groups * beams, 1), 16384 / (beams * keep)}));
}

// The scans: `n` values of a unit of `unit` bytes, a lane takes `per_lane` at a time; with one best a
// lane and with two.
struct Scan {
  int dtype, unit, n, per_lane;
  void (*few)(const ScanParams), (*many)(const ScanParams);
};
template <typename E, int UNIT>
constexpr Scan scan_of(int dtype) {
  using X = Vec<E, UNIT>;
  return Scan{dtype, UNIT, X::N, X::N * X::UNITS, beam_scan_kernel<E, UNIT, 1>, beam_scan_kernel<E, UNIT, 2>};
}
// by type, the widest first
const Scan kScans[] = {scan_of<float, 16>(ATTN_DTYPE_F32), scan_of<float, 4>(ATTN_DTYPE_F32), scan_of<uint16_t, 16>(ATTN_DTYPE_BF16),
                       scan_of<uint16_t, 4>(ATTN_DTYPE_BF16), scan_of<uint16_t, 2>(ATTN_DTYPE_BF16)};

int check_beams(int groups, int beams, int vocab, int keep) {
  if (groups < 0 || beams < 1 || vocab < 1 || keep < 1) return ATTN_ERR_INVALID_ARG;
  if (beams > ATTN_BEAM_MAX || keep > ATTN_BEAM_MAX || static_cast<int64_t>(groups) * beams >= (1 << 24) || vocab > (1 << 30)) return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" {

int attn_beam_workspace_bytes(int groups, int beams, int vocab, int keep, size_t *bytes) {
  if (!bytes) return ATTN_ERR_INVALID_ARG;
  const int rc = check_beams(groups, beams, vocab, keep);
  if (rc != ATTN_OK) return rc;
  const int sms = device_sm_count();
  if (sms <= 0) return ATTN_ERR_CUDA;
  size_t most = 0;
  for (const Scan &x : kScans) {
    int units;
    const size_t parts = static_cast<size_t>(groups) * beams * splits_of(groups, beams, vocab, keep, x.n, x.per_lane, sms, &units);
    const size_t need = up256(parts * 8) + 2 * up256(parts * keep * 4);
    most = need > most ? need : most;
  }
  *bytes = most;
  return ATTN_OK;
}

int attn_beam_select(const void *logits, int logits_dtype, int64_t row_stride, int groups, int beams, int vocab, const float *scores,
                     const uint8_t *done, int eos, const int32_t *slots, int keep, float *out_scores, int32_t *out_parents,
                     int32_t *out_tokens, uint8_t *out_done, int32_t *out_src, void *d_ws, size_t ws_bytes, attn_stream_t stream) {
  if (logits_dtype != ATTN_DTYPE_F32 && logits_dtype != ATTN_DTYPE_BF16) return ATTN_ERR_INVALID_ARG;
  int rc = check_beams(groups, beams, vocab, keep);
  if (rc != ATTN_OK) return rc;
  if (static_cast<int64_t>(beams) * vocab < keep || eos < -1 || eos >= vocab || (done && eos < 0)) return ATTN_ERR_INVALID_ARG;
  if (row_stride < vocab) return ATTN_ERR_INVALID_ARG;
  if (groups == 0) return ATTN_OK;
  if (!logits || !scores || !out_scores || !out_parents || !out_tokens || !d_ws) return ATTN_ERR_INVALID_ARG;
  const int esize = logits_dtype == ATTN_DTYPE_F32 ? 4 : 2;
  auto off = [](const void *x, int to) { return (reinterpret_cast<uintptr_t>(x) & (to - 1)) != 0; };
  if (off(logits, esize) || off(scores, 4) || off(slots, 4) || off(out_scores, 4) || off(out_parents, 4) || off(out_tokens, 4) ||
      off(out_src, 4) || off(d_ws, 16))
    return ATTN_ERR_UNSUPPORTED;
  size_t need = 0;
  if ((rc = attn_beam_workspace_bytes(groups, beams, vocab, keep, &need)) != ATTN_OK) return rc;
  if (ws_bytes < need) return ATTN_ERR_CAPACITY;
  const int rows = groups * beams;
  const int sms = device_sm_count();
  if (sms <= 0) return ATTN_ERR_CUDA;
  // the first whose units divide the distance of two beams' rows
  const Scan *x = kScans;
  while (x->dtype != logits_dtype || (beams > 1 && row_stride * esize % x->unit)) ++x;
  int units;
  const int splits = splits_of(groups, beams, vocab, keep, x->n, x->per_lane, sms, &units);
  const size_t parts = static_cast<size_t>(rows) * splits;
  if (parts >= (size_t(1) << 30) || static_cast<int64_t>(beams) * splits * keep >= INT_MAX) return ATTN_ERR_UNSUPPORTED;
  uint8_t *ws = static_cast<uint8_t *>(d_ws);
  float2 *ms = reinterpret_cast<float2 *>(ws);
  uint32_t *keys = reinterpret_cast<uint32_t *>(ws + up256(parts * 8));
  int *ids = reinterpret_cast<int *>(ws + up256(parts * 8) + up256(parts * keep * 4));
  const ScanParams sp{logits, done, row_stride, vocab, splits, keep, units / splits, units % splits, static_cast<int>(parts), ms, keys, ids};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  auto scan = keep <= 32 ? x->few : x->many;
  const unsigned grid = static_cast<unsigned>((parts + BS_T / 32 - 1) / (BS_T / 32));
  if ((rc = launch_after(scan, dim3(grid), BS_T, 0, s, sp)) != ATTN_OK) return rc;
  const PickParams pp{scores, done, slots, ms, keys, ids, beams, vocab, splits, keep, eos, out_scores, out_parents, out_tokens, out_src, out_done};
  return launch_after(beam_pick_kernel, dim3(groups), BP_T, 0, s, pp);
}

int attn_beam_reorder(void *const *h_states, const int64_t *h_row_bytes, const int64_t *h_row_strides, int n_states, const int32_t *parents,
                      int groups, int beams, attn_stream_t stream) {
  if (n_states < 0 || groups < 0 || beams < 1 || (n_states > 0 && (!h_states || !h_row_bytes || !h_row_strides))) return ATTN_ERR_INVALID_ARG;
  if (n_states > ATTN_BEAM_MAX_STATES || beams > ATTN_BEAM_MAX || static_cast<int64_t>(groups) * beams >= (1 << 24)) return ATTN_ERR_UNSUPPORTED;
  if (groups > 0 && !parents) return ATTN_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(parents) & 3) return ATTN_ERR_UNSUPPORTED;
  ReorderParams p;
  std::memset(&p, 0, sizeof(p));
  int64_t units = 0;
  bool runs = false;
  for (int i = 0; i < n_states; ++i) {
    const int64_t bytes = h_row_bytes[i], stride = h_row_strides[i];
    if (bytes < 0 || stride < bytes) return ATTN_ERR_INVALID_ARG;
    if (bytes == 0 || groups == 0) continue;
    if (!h_states[i]) return ATTN_ERR_INVALID_ARG;
    for (int j = 0; j < p.n_states; ++j)
      if (p.s[j].at == h_states[i]) return ATTN_ERR_INVALID_ARG;
    const uint64_t all = reinterpret_cast<uintptr_t>(h_states[i]) | static_cast<uint64_t>(bytes) | static_cast<uint64_t>(stride);
    const int loose = (all & 15) || beams > 16;
    runs |= loose;
    const int64_t each = unit_bytes(loose, beams);
    p.s[p.n_states++] = State{static_cast<uint8_t *>(h_states[i]), stride, bytes, loose, static_cast<int>(units)};
    units += (bytes + each - 1) / each * groups;
    if (units >= INT_MAX) return ATTN_ERR_UNSUPPORTED;
  }
  if (units == 0) return ATTN_OK;
  p.parents = parents;
  p.groups = groups;
  p.beams = beams;
  p.units = static_cast<int>(units);
  if (!(p.status = paged_status())) return ATTN_ERR_CUDA;
  const int sms = device_sm_count();
  if (sms <= 0) return ATTN_ERR_CUDA;
  auto kern = runs ? beams <= 4 ? beam_reorder_kernel<4, true> : beams <= 8 ? beam_reorder_kernel<8, true> : beam_reorder_kernel<16, true>
                   : beams <= 4 ? beam_reorder_kernel<4, false> : beams <= 8 ? beam_reorder_kernel<8, false> : beam_reorder_kernel<16, false>;
  const int64_t grid = sms * 16;
  return launch_after(kern, dim3(static_cast<unsigned>(units < grid ? units : grid)), RE_T, runs ? beams * run_pitch(beams) : 0, reinterpret_cast<cudaStream_t>(stream), p);
}

}  // extern "C"
