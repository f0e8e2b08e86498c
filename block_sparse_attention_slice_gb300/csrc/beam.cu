// A beam search's step: the best continuations of each prompt, and the beams' states
// brought into their order.
//
// A continuation's score is c_b + logit, with c_b = score_b - ln sum exp(logit): of one
// beam's continuations the best are those of its largest logits, so one pass over the
// logits gives both the sum and, for every part of a row, its `keep` largest.  The rest
// is small: a block a prompt adds the parts' sums in 64 bits, compares the parts' best
// as 64-bit scores and keeps the best of them all.
//
// beam_scan_kernel: a block holds a part of a row in registers (its logits are read
// once) and has from it maximum, sum and the best.  For those it finds a threshold that
// `keep` values reach by bisection on the threads' maxima: `keep` threads whose maximum
// reaches it have as many values that do, and few others are there.  What reaches it
// goes to a list in shared memory and is ranked there.  Values are compared as whole
// numbers in the order of the floats.  Where the list overflows (values that are equal by
// the thousand, as where most of a vocabulary is ruled out) the best are taken one by one.
#include <cuda_runtime.h>

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
constexpr int BS_CAP = 1024;         // places of its list
constexpr int BP_T = 256;            // of a choosing block
constexpr int BP_CAP = 1024;

// The order of the floats as whole numbers; -inf is 0x007fffff, 0 stands for no value.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return max((b & 0x80000000u) ? ~b : b | 0x80000000u, 1u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ unsigned long long key_of(double x) {
  const unsigned long long b = static_cast<unsigned long long>(__double_as_longlong(x));
  return (b >> 63) ? ~b : b | 1ull << 63;
}
__device__ __forceinline__ double value_of(unsigned long long k) {
  return __longlong_as_double(static_cast<long long>((k >> 63) ? k ^ 1ull << 63 : ~k));
}

// A threshold that at least min(keep, values there are) of the block's `top`, one a
// thread, reach, and not many more: bisection between the largest and the smallest.
template <int T, typename K>
__device__ __forceinline__ K threshold(K top, int keep, K *sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  K hi = top, lo = top;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const K a = __shfl_xor_sync(0xffffffffu, hi, o), b = __shfl_xor_sync(0xffffffffu, lo, o);
    hi = a > hi ? a : hi;
    lo = b < lo ? b : lo;
  }
  if (lane == 0) sums[2 * warp] = hi, sums[2 * warp + 1] = lo;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < T / 32; ++w) {
    hi = sums[2 * w] > hi ? sums[2 * w] : hi;
    lo = sums[2 * w + 1] < lo ? sums[2 * w + 1] : lo;
  }
  // all reach lo; fewer than keep reach hi + 1
  if (lo < 1) lo = 1;
  while (lo < hi) {
    const K mid = lo + (hi - lo + 1) / 2;
    const int n = __syncthreads_count(top >= mid);
    if (n >= keep) {
      lo = mid;
      if (n <= keep + keep / 2) break;
    } else {
      hi = mid - 1;
    }
  }
  return lo;
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

struct ScanParams {
  const void *logits;
  const uint8_t *done;
  long long row_stride;      // elements
  int vocab, splits, keep;
  float2 *ms;                // [rows][splits]: maximum, sum of exp(x - maximum)
  uint32_t *keys;            // [rows][splits][keep], best first
  int *ids;                  // their tokens; -1: none
};

template <typename E>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4 &w, float *x) {
    x[0] = __uint_as_float(w.x), x[1] = __uint_as_float(w.y), x[2] = __uint_as_float(w.z), x[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ float one(const float *p) { return *p; }
};
template <>
struct Vec<uint16_t> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4 &w, float *x) {
    const uint32_t y[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(y[i] << 16), x[2 * i + 1] = __uint_as_float(y[i] & 0xffff0000u);
  }
  static __device__ __forceinline__ float one(const uint16_t *p) { return __uint_as_float(static_cast<uint32_t>(*p) << 16); }
};

// Bound by HBM where there are many rows.  E: the logits' type; PER values a thread.
// A row is taken by its 16-byte words wherever it begins: a word that the row's ends cut
// is read value by value.
template <typename E, int PER>
__global__ void __launch_bounds__(BS_T) beam_scan_kernel(const ScanParams p) {
  constexpr int N = Vec<E>::N, WORDS = PER / N;
  __shared__ uint32_t sums[2 * BS_T / 32];
  __shared__ float part[BS_T / 32];
  __shared__ uint32_t list_k[BS_CAP];
  __shared__ int list_i[BS_CAP];
  __shared__ int listed;
  after_previous();
  admit_next();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long row = blockIdx.x / p.splits;
  const int split = static_cast<int>(blockIdx.x - row * p.splits);
  if (p.done && p.done[row]) return;
  const E *base = static_cast<const E *>(p.logits) + row * p.row_stride;
  const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(base) & 15) / sizeof(E));
  const E *aligned = base - skew;            // not read before base
  float x[PER];
#pragma unroll
  for (int w = 0; w < WORDS; ++w) {
    // the word's first value is number v of the row
    const long long v = (static_cast<long long>(split) * (BS_T * WORDS) + w * BS_T + threadIdx.x) * N - skew;
    if (v >= 0 && v + N <= p.vocab) {
      Vec<E>::unpack(__ldcs(reinterpret_cast<const uint4 *>(aligned + skew + v)), x + w * N);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) x[w * N + e] = v + e >= 0 && v + e < p.vocab ? Vec<E>::one(base + v + e) : 0.f;
    }
  }
  auto id_of = [&](int w, int e) -> long long {
    return (static_cast<long long>(split) * (BS_T * WORDS) + w * BS_T + threadIdx.x) * N - skew + e;
  };
  auto there = [&](int w, int e) {
    const long long v = id_of(w, e);
    return v >= 0 && v < p.vocab;
  };
  if (threadIdx.x == 0) listed = 0;
  // maximum (a NaN is passed by, and spoils the sum), this thread's best
  float m = -INFINITY;
  uint32_t top = 0;
#pragma unroll
  for (int w = 0; w < WORDS; ++w)
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (there(w, e)) {
        m = fmaxf(m, x[w * N + e]);
        top = max(top, key_of(x[w * N + e]));
      }
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) part[warp] = m;
  const uint32_t least = threshold<BS_T>(top, p.keep, sums);      // has a barrier
#pragma unroll
  for (int w = 0; w < BS_T / 32; ++w) m = fmaxf(m, part[w]);
  __syncthreads();
  const float mb = m == -INFINITY ? 0.f : m;
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < WORDS; ++w) {
    float t = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (there(w, e)) {
        const float y = x[w * N + e];
        t += ex2_approx((y - mb) * 1.44269504f);
        if (key_of(y) >= least) {
          const int at = atomicAdd(&listed, 1);
          if (at < BS_CAP) {
            list_k[at] = key_of(y);
            list_i[at] = static_cast<int>(id_of(w, e));
          }
        }
      }
    s += t;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) part[warp] = s;
  __syncthreads();
  const long long at = row * p.splits + split;
  if (threadIdx.x == 0) {
    s = 0.f;
#pragma unroll
    for (int w = 0; w < BS_T / 32; ++w) s += part[w];
    p.ms[at] = make_float2(m, s);
  }
  uint32_t *keys = p.keys + at * p.keep;
  int *ids = p.ids + at * p.keep;
  const int n = listed;
  if (n <= BS_CAP) {
    for (int i = threadIdx.x; i < n; i += BS_T) {
      const uint32_t k = list_k[i];
      const int id = list_i[i];
      int rank = 0;
      for (int j = 0; j < n && rank < p.keep; ++j) rank += before(list_k[j], list_i[j], k, id);
      if (rank < p.keep) keys[rank] = k, ids[rank] = id;
    }
    for (int i = n + threadIdx.x; i < p.keep; i += BS_T) ids[i] = -1;
    return;
  }
  uint32_t last_k = 0xffffffffu;
  int last_i = -1;
  for (int r = 0; r < p.keep; ++r) {      // more than `keep` values are there
    uint32_t k = 0;
    int id = INT_MAX;
#pragma unroll
    for (int w = 0; w < WORDS; ++w)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const uint32_t a = key_of(x[w * N + e]);
        const int i = static_cast<int>(id_of(w, e));
        if (there(w, e) && before(last_k, last_i, a, i) && before(a, i, k, id)) k = a, id = i;
      }
    block_best<BS_T>(k, id, sums, reinterpret_cast<int *>(part));
    if (threadIdx.x == 0) keys[r] = k, ids[r] = id;
    last_k = k;
    last_i = id;
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

// One block a group.  Continuations are the parts' best, and of a beam that offers
// nothing the first `keep` by their place, at -inf (of one that has ended its eos, then
// those), so that the choice needs no other rule.
__global__ void __launch_bounds__(BP_T) beam_pick_kernel(const PickParams p) {
  __shared__ double offset[ATTN_BEAM_MAX];      // score - ln sum; NaN: the beam offers nothing but -inf
  __shared__ unsigned long long sums[2 * BP_T / 32];
  __shared__ int isum[BP_T / 32];
  __shared__ unsigned long long list_k[BP_CAP];
  __shared__ int list_i[BP_CAP];
  __shared__ int listed;
  after_previous();
  admit_next();
  const int g = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, per = p.splits * p.keep, n = p.beams * per;
  if (threadIdx.x == 0) listed = 0;
  for (int b = warp; b < p.beams; b += BP_T / 32) {
    const long long row = static_cast<long long>(g) * p.beams + b;
    double c = __longlong_as_double(0x7ff8000000000000ll);
    const float score = p.scores[row];
    if (!(p.done && p.done[row]) && score > -INFINITY && score < INFINITY) {
      float m = -INFINITY;
      for (int i = lane; i < p.splits; i += 32) m = fmaxf(m, p.ms[row * p.splits + i].x);
#pragma unroll
      for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      double s = 0.0;
      for (int i = lane; i < p.splits; i += 32) {
        const float2 y = p.ms[row * p.splits + i];
        // a part of -inf alone has the sum 0; one with a NaN keeps it
        s += y.x == -INFINITY ? static_cast<double>(y.y) * 0.0 : static_cast<double>(y.y) * exp(static_cast<double>(y.x) - static_cast<double>(m));
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      c = static_cast<double>(score) - (static_cast<double>(m) + log(s));
      if (!(c > -INFINITY && c < INFINITY)) c = __longlong_as_double(0x7ff8000000000000ll);
    }
    if (lane == 0) offset[b] = c;
  }
  __syncthreads();
  // continuation j: its score as a key (0: none) and its place, kept as beam and token
  auto get = [&](int j, unsigned long long &k, int &b, int &v) {
    b = j / per;
    const long long row = static_cast<long long>(g) * p.beams + b;
    const int i = j - b * per;
    const double c = offset[b];
    k = 0;
    v = 0;
    if (c == c) {
      v = p.ids[row * per + i];
      if (v >= 0) k = key_of(c + static_cast<double>(value_of(p.keys[row * per + i])));
    } else if (i < p.keep) {
      const float score = p.scores[row];
      const bool ended = p.done && p.done[row] && score > -INFINITY && score < INFINITY;
      if (ended && i == 0) {
        v = p.eos;
        k = key_of(static_cast<double>(score));
      } else {
        v = ended ? i - 1 + (i - 1 >= p.eos) : i;
        if (v < p.vocab) k = key_of(-static_cast<double>(INFINITY));
      }
    }
  };
  unsigned long long top = 0;
  for (int j = threadIdx.x; j < n; j += BP_T) {
    unsigned long long k;
    int b, v;
    get(j, k, b, v);
    top = k > top ? k : top;
  }
  const unsigned long long least = threshold<BP_T>(top, p.keep, sums);
  for (int j = threadIdx.x; j < n; j += BP_T) {
    unsigned long long k;
    int b, v;
    get(j, k, b, v);
    if (k >= least && k) {
      const int at = atomicAdd(&listed, 1);
      if (at < BP_CAP) list_k[at] = k, list_i[at] = j;
    }
  }
  __syncthreads();
  auto write = [&](int r, unsigned long long k, int b, int v) {
    const long long to = static_cast<long long>(g) * p.keep + r, row = static_cast<long long>(g) * p.beams + b;
    p.out_scores[to] = static_cast<float>(value_of(k));
    p.out_parents[to] = static_cast<int32_t>(row);
    p.out_tokens[to] = v;
    if (p.out_done) p.out_done[to] = (p.done && p.done[row]) || v == p.eos;
    if (p.out_src) p.out_src[to] = p.slots ? p.slots[row] : static_cast<int32_t>(row);
  };
  const int m = listed;
  if (m <= BP_CAP) {
    for (int i = threadIdx.x; i < m; i += BP_T) {
      unsigned long long k;
      int b, v, rank = 0;
      get(list_i[i], k, b, v);
      for (int j = 0; j < m && rank < p.keep; ++j) {
        const unsigned long long a = list_k[j];
        if (a > k) {
          ++rank;
        } else if (a == k && j != i) {
          unsigned long long y;
          int c, w;
          get(list_i[j], y, c, w);
          rank += c < b || (c == b && w < v);
        }
      }
      if (rank < p.keep) write(rank, k, b, v);
    }
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
  long long stride;          // bytes from row to row
  long long words;           // of a row
  int word, first;           // bytes of a word; the state's first unit
};
struct ReorderParams {
  State s[ATTN_BEAM_MAX_STATES];
  const int32_t *parents;
  int n_states, groups, beams, units;
  unsigned int *status;
};
constexpr int RE_T = 256;

// All parents' words of one column of a group, then all rows': the column is this
// thread's alone, so the rows may change places in memory.  Rows that stay are not
// touched.
template <typename W, int MOST>
__device__ __forceinline__ void move_column(const State &s, long long row0, long long word, const int *par, int beams) {
  W x[MOST];
  uint8_t *base = s.at + row0 * s.stride + word * sizeof(W);
#pragma unroll
  for (int b = 0; b < MOST; ++b)
    if (b < beams && par[b] != b) x[b] = *reinterpret_cast<const W *>(base + par[b] * s.stride);
#pragma unroll
  for (int b = 0; b < MOST; ++b)
    if (b < beams && par[b] != b) *reinterpret_cast<W *>(base + b * s.stride) = x[b];
}

template <int MOST>
__global__ void __launch_bounds__(RE_T) beam_reorder_kernel(const __grid_constant__ ReorderParams p) {
  __shared__ int par[ATTN_BEAM_MAX];
  after_previous();
  admit_next();
  int s = 0;
  for (int u = blockIdx.x; u < p.units; u += gridDim.x) {
    while (s + 1 < p.n_states && u >= p.s[s + 1].first) ++s;
    const State &st = p.s[s];
    const int per = static_cast<int>((st.words + RE_T - 1) / RE_T), g = (u - st.first) / per;
    const long long word = static_cast<long long>(u - st.first - g * per) * RE_T + threadIdx.x, row0 = static_cast<long long>(g) * p.beams;
    __syncthreads();
    int off = 0;
    if (threadIdx.x < static_cast<unsigned>(p.beams)) {
      const long long a = p.parents[row0 + threadIdx.x] - row0;
      off = a < 0 || a >= p.beams;
      par[threadIdx.x] = off ? static_cast<int>(threadIdx.x) : static_cast<int>(a);
    }
    if (__syncthreads_or(off)) {
      if (threadIdx.x == 0) atomicCAS(p.status, 0u, static_cast<unsigned>(ATTN_ERR_INVALID_ARG));
      continue;
    }
    if (word >= st.words) continue;
    if (MOST <= 16 && st.word == 16) move_column<uint4, MOST <= 16 ? MOST : 1>(st, row0, word, par, p.beams);
    else if (st.word == 4) move_column<uint32_t, MOST>(st, row0, word, par, p.beams);
    else move_column<uint8_t, MOST>(st, row0, word, par, p.beams);
  }
}

int splits_of(int rows, int vocab, int dtype, int *per) {
  // 8 values a thread where 32 would leave SMs without a block
  const int n = dtype == ATTN_DTYPE_F32 ? 4 : 8;
  auto parts = [&](int each) { return static_cast<int>((static_cast<long long>(vocab) + n - 1 + BS_T * each - 1) / (BS_T * each)); };
  *per = static_cast<long long>(rows) * parts(32) >= 2 * 152 ? 32 : 8;
  return parts(*per);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" {

int attn_beam_workspace_bytes(int groups, int beams, int vocab, int keep, size_t *bytes) {
  if (!bytes || groups < 0 || beams < 1 || vocab < 1 || keep < 1) return ATTN_ERR_INVALID_ARG;
  if (beams > ATTN_BEAM_MAX || keep > ATTN_BEAM_MAX || static_cast<int64_t>(groups) * beams >= (1 << 24)) return ATTN_ERR_UNSUPPORTED;
  size_t most = 0;
  for (int dtype : {ATTN_DTYPE_F32, ATTN_DTYPE_BF16}) {
    int per;
    const size_t parts = static_cast<size_t>(groups) * beams * splits_of(groups * beams, vocab, dtype, &per);
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
  size_t need = 0;
  int rc = attn_beam_workspace_bytes(groups, beams, vocab, keep, &need);
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
  if (ws_bytes < need) return ATTN_ERR_CAPACITY;
  const int rows = groups * beams;
  int per;
  const int splits = splits_of(rows, vocab, logits_dtype, &per);
  const size_t parts = static_cast<size_t>(rows) * splits;
  if (parts >= (size_t(1) << 31) || static_cast<int64_t>(beams) * splits * keep >= INT_MAX) return ATTN_ERR_UNSUPPORTED;
  uint8_t *ws = static_cast<uint8_t *>(d_ws);
  float2 *ms = reinterpret_cast<float2 *>(ws);
  uint32_t *keys = reinterpret_cast<uint32_t *>(ws + up256(parts * 8));
  int *ids = reinterpret_cast<int *>(ws + up256(parts * 8) + up256(parts * keep * 4));
  const ScanParams sp{logits, done, row_stride, vocab, splits, keep, ms, keys, ids};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  auto scan = logits_dtype == ATTN_DTYPE_F32 ? (per == 32 ? beam_scan_kernel<float, 32> : beam_scan_kernel<float, 8>)
                                             : (per == 32 ? beam_scan_kernel<uint16_t, 32> : beam_scan_kernel<uint16_t, 8>);
  if ((rc = launch_after(scan, dim3(static_cast<unsigned>(parts)), BS_T, 0, s, sp)) != ATTN_OK) return rc;
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
  for (int i = 0; i < n_states; ++i) {
    const int64_t bytes = h_row_bytes[i], stride = h_row_strides[i];
    if (bytes < 0 || stride < bytes) return ATTN_ERR_INVALID_ARG;
    if (bytes == 0 || groups == 0) continue;
    if (!h_states[i]) return ATTN_ERR_INVALID_ARG;
    const uint64_t all = reinterpret_cast<uintptr_t>(h_states[i]) | static_cast<uint64_t>(bytes) | static_cast<uint64_t>(stride);
    const int word = !(all & 15) && beams <= 16 ? 16 : !(all & 3) ? 4 : 1;
    p.s[p.n_states++] = State{static_cast<uint8_t *>(h_states[i]), stride, bytes / word, word, static_cast<int>(units)};
    units += (bytes / word + RE_T - 1) / RE_T * groups;
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
  auto kern = beams <= 4 ? beam_reorder_kernel<4> : beams <= 8 ? beam_reorder_kernel<8> : beams <= 16 ? beam_reorder_kernel<16> : beam_reorder_kernel<64>;
  const int64_t grid = sms * 16;
  return launch_after(kern, dim3(static_cast<unsigned>(units < grid ? units : grid)), RE_T, 0, reinterpret_cast<cudaStream_t>(stream), p);
}

}  // extern "C"
