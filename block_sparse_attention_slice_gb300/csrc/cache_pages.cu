// Pages of a key/value cache: growing, forking, freeing, trimming and
// compacting the page table, writing tokens and copying pages.
//
// The table operations are integer work on a few hundred KB, so what they cost
// is launches and waits, not bytes: each is ONE launch of one cluster of 8 CTAs
// of 1024 threads, whose hardware barrier (about a microsecond for both halves)
// takes the place of grid barriers or further launches, and whose distributed
// shared memory carries the counts between CTAs.  Nothing is kept between
// calls.  32 rows of up to 128 pages fork in 8 us, 64 rows free and extend in 5
// and 6; half a million pages take 68 us to free and extend, 137 to fork, bound
// by the cluster's 8 SMs.  Clusters of 1, 2 or 4 CTAs gave the small calls 1 us
// and the large ones up to 8 times their time.  Work over the sequences of a list
// is flattened: a block-wide prefix sum of their page counts, then every thread
// takes flat indices 8192 apart and finds its sequence by bisection in shared
// memory, so one long sequence costs no more than many short ones.  Results are
// exact and do not depend on the order of atomics: adding and subtracting counts
// commutes, and fresh pages are chosen from the counts as they stood before the
// call.
//
// A call either does all it was asked for or, when a list names a row out of
// range or twice, or free pages or table columns run out, changes nothing and
// leaves the reason for attn_last_device_error().
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "../../include/attn_paged.h"
#include "attn_device.cuh"
#include "attn_internal.h"
#include "launch.cuh"

namespace attn {

constexpr int CC = 8, CT = 1024, CALL = CC * CT;   // CTAs, threads of each, of all

struct CacheParams {
  int32_t *table, *lens, *refs;
  long long stride;
  int n_slots, max_pages, n_pages, shift;
  const int32_t *a, *b;         // lists of the call
  int n;
  int window, sinks;
  int32_t *copies;              // count, src[cap], dst[cap]
  int cap;
  int32_t *ws;
  unsigned int *status;
};

struct CacheSmem {
  int scan[33];
  int count[CC];                // one number of every CTA, written by each into all
  int count2[CC];
  int bad;
};

__device__ __forceinline__ int pages_of(const CacheParams &p, int len) {
  return static_cast<int>((static_cast<long long>(len) + (1 << p.shift) - 1) >> p.shift);
}

// Exclusive prefix sum of x over the block; the total in `sum`.
__device__ inline int block_scan(CacheSmem &s, int x, int &sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  __syncthreads();
  if (lane == 31) s.scan[warp] = y;
  __syncthreads();
  if (warp == 0) {
    int w = s.scan[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += z;
    }
    s.scan[lane] = w;
  }
  __syncthreads();
  sum = s.scan[31];
  return y - x + (warp ? s.scan[warp - 1] : 0);
}

// first[i] = sum of count(0..i-1) for i in 0..n, in shared memory.
template <typename F>
__device__ inline int list_scan(CacheSmem &s, int n, int *first, F count) {
  int base = 0;
  for (int i0 = 0; i0 < n; i0 += CT) {
    const int i = i0 + threadIdx.x;
    int sum;
    const int x = block_scan(s, i < n ? count(i) : 0, sum);
    if (i < n) first[i] = base + x;
    base += sum;
  }
  if (threadIdx.x == 0) first[n] = base;
  __syncthreads();
  return base;
}

// i with first[i] <= x < first[i + 1]
__device__ __forceinline__ int list_find(const int *first, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The barrier in two halves: no CTA's shared memory is written to by another
// before all have started (arrive at the start, wait before the first write).
__device__ __forceinline__ void cluster_started() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait_started() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Gives every CTA of the cluster this one's x; ends with the cluster's barrier.
__device__ inline void share_count(int *count, int x, int rank) {
  if (threadIdx.x < CC)
    st_shared_cluster_u32(mapa_shared(smem_u32(count + rank), threadIdx.x), static_cast<uint32_t>(x));
  cluster_sync();
}

// This CTA's share of the pages, a multiple of 4 pages but for the last.
__device__ __forceinline__ void page_share(const CacheParams &p, int rank, int &from, int &to) {
  const int per = (((p.n_pages + CC - 1) / CC) + 3) & ~3;
  from = static_cast<int>(min(static_cast<long long>(rank) * per, static_cast<long long>(p.n_pages)));
  to = static_cast<int>(min(static_cast<long long>(from) + per, static_cast<long long>(p.n_pages)));
}

// Bits of `want(page, refs)` for the 4 pages from page x on (those below `to`).
template <typename F>
__device__ __forceinline__ unsigned page_bits(const CacheParams &p, int x, int to, F want) {
  unsigned m = 0;
  if (x + 4 <= to && (reinterpret_cast<uintptr_t>(p.refs + x) & 15) == 0) {
    const int4 r = *reinterpret_cast<const int4 *>(p.refs + x);
    m = (want(x, r.x) ? 1u : 0u) | (want(x + 1, r.y) ? 2u : 0u) | (want(x + 2, r.z) ? 4u : 0u) |
        (want(x + 3, r.w) ? 8u : 0u);
  } else {
    for (int k = 0; k < 4; ++k)
      if (x + k < to && want(x + k, p.refs[x + k])) m |= 1u << k;
  }
  return m;
}

template <typename F>
__device__ inline int count_pages(CacheSmem &s, const CacheParams &p, int from, int to, F want) {
  int c = 0, sum;
  for (int x = from + 4 * threadIdx.x; x < to; x += 4 * CT) c += __popc(page_bits(p, x, to, want));
  block_scan(s, c, sum);
  return sum;
}

// emit(rank, page) for the wanted pages of this CTA's share in ascending
// order, ranks from `rank` on and below `limit`.
template <typename F, typename E>
__device__ inline void rank_pages(CacheSmem &s, const CacheParams &p, int from, int to, int rank, int limit, F want,
                                  E emit) {
  for (int x0 = from; x0 < to && rank < limit; x0 += 4 * CT) {
    const int x = x0 + 4 * threadIdx.x;
    unsigned m = x < to ? page_bits(p, x, to, want) : 0u;
    int sum;
    int r = rank + block_scan(s, __popc(m), sum);
    for (; m && r < limit; ++r) {
      const int k = __ffs(m) - 1;
      m &= m - 1;
      emit(r, x + k);
    }
    rank += sum;
  }
}

// The list's rows are in range and named once each (by the set of bits `seen`
// over the slots, cleared here); every CTA comes to the same answer.
__device__ inline void check_rows(CacheSmem &s, const CacheParams &p, const int32_t *list, uint32_t *seen) {
  for (int i = threadIdx.x; i < (p.n_slots + 31) / 32; i += CT) seen[i] = 0;
  if (threadIdx.x == 0) s.bad = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < p.n; i += CT) {
    const int x = list[i];
    if (x < 0 || x >= p.n_slots || (atomicOr(&seen[x >> 5], 1u << (x & 31)) >> (x & 31) & 1u)) s.bad = 1;
  }
  __syncthreads();
}

__device__ __forceinline__ bool good_len(const CacheParams &p, int len) {
  return len >= 0 && len <= (static_cast<long long>(p.max_pages) << p.shift);
}

__device__ __forceinline__ void refuse(const CacheParams &p, int rank, unsigned code) {
  if (rank == 0 && threadIdx.x == 0) {
    atomicCAS(p.status, 0u, code);
    if (p.copies) p.copies[0] = 0;
  }
}

// Drops one holder of a page.
__device__ __forceinline__ void drop(const CacheParams &p, int page) {
  if (page < 0) return;                       // given back already
  if (page < p.n_pages) atomicSub(p.refs + page, 1);
  else atomicCAS(p.status, 0u, static_cast<unsigned>(ATTN_ERR_INVALID_ARG));
}

// Reads what the kernel will need first, all at once: list entries, the lengths
// they name and this CTA's first page counts.  The reads that follow, one after
// the other, then find them in L1.
struct Ahead {
  int x[3] = {0, 0, 0};
  int4 refs = {0, 0, 0, 0};
  __device__ __forceinline__ Ahead(const CacheParams &p, int page_from, int page_to) {
    const int i = threadIdx.x, page = page_from + 4 * i;
    if (page + 4 <= page_to && (reinterpret_cast<uintptr_t>(p.refs + page) & 15) == 0)
      refs = *reinterpret_cast<const int4 *>(p.refs + page);
    if (i < p.n) {
      const int a = p.a ? p.a[i] : i, b = p.b ? p.b[i] : -1;
      x[0] = b;
      if (a >= 0 && a < p.n_slots) x[1] = p.lens[a];
      if (p.copies && b >= 0 && b < p.n_slots) x[2] = p.lens[b];
    }
  }
  __device__ __forceinline__ void arrived() {
    asm volatile("" ::"r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(refs.x), "r"(refs.y), "r"(refs.z), "r"(refs.w) : "memory");
  }
};

extern __shared__ __align__(16) int cache_smem[];

// ---------------------------------------------------------------- extend

__global__ void __cluster_dims__(CC, 1, 1) __launch_bounds__(CT, 1) cache_extend_kernel(const CacheParams p) {
  after_previous();
  admit_next();
  __shared__ CacheSmem s;
  cluster_started();
  const int rank = cluster_ctarank();
  int from, to;
  page_share(p, rank, from, to);
  Ahead ahead(p, from, to);
  int *first = cache_smem, *have = first + p.n + 1;
  uint32_t *seen = reinterpret_cast<uint32_t *>(have + p.n);
  check_rows(s, p, p.a, seen);
  ahead.arrived();
  unsigned code = s.bad ? ATTN_ERR_INVALID_ARG : 0u;
  if (code == 0) {
    __shared__ int full;
    if (threadIdx.x == 0) full = 0;
    __syncthreads();
    list_scan(s, p.n, first, [&](int i) {
      const int len = p.lens[p.a[i]], add = p.b[i];
      have[i] = pages_of(p, max(len, 0));
      if (add < 0 || !good_len(p, len)) {
        s.bad = 1;
        return 0;
      }
      const long long to = static_cast<long long>(len) + add;
      if (to > (static_cast<long long>(p.max_pages) << p.shift)) {
        full = 1;
        return 0;
      }
      return pages_of(p, static_cast<int>(to)) - have[i];
    });
    code = s.bad ? ATTN_ERR_INVALID_ARG : full ? ATTN_ERR_CAPACITY : 0u;
  }
  auto is_free = [](int, int r) { return r == 0; };
  const int mine = code ? 0 : count_pages(s, p, from, to, is_free);
  cluster_wait_started();
  share_count(s.count, mine, rank);          // every CTA has read the lengths by now
  if (code == 0) {
    int before = 0, total = 0;
    for (int c = 0; c < CC; ++c) {
      before += c < rank ? s.count[c] : 0;
      total += s.count[c];
    }
    const int want = first[p.n];
    if (total < want) {
      code = ATTN_ERR_CAPACITY;
    } else {
      rank_pages(s, p, from, to, before, want, is_free, [&](int r, int page) {
        const int i = list_find(first, p.n, r);
        p.table[p.a[i] * p.stride + have[i] + r - first[i]] = page;
        p.refs[page] = 1;
      });
      if (rank == 0)
        for (int i = threadIdx.x; i < p.n; i += CT) p.lens[p.a[i]] += p.b[i];
    }
  }
  if (code) refuse(p, rank, code);
}

// ---------------------------------------------------------------- free, trim

// TRIM false: all pages of the list's rows.  TRIM true: those behind the first
// tokens that no token at position len - 1 or later sees.
template <bool TRIM>
__global__ void __cluster_dims__(CC, 1, 1) __launch_bounds__(CT, 1) cache_free_kernel(const CacheParams p) {
  after_previous();
  admit_next();
  __shared__ CacheSmem s;
  const int rank = cluster_ctarank();
  Ahead ahead(p, 0, 0);
  int *first = cache_smem;
  uint32_t *seen = reinterpret_cast<uint32_t *>(first + p.n + 1);
  if (p.a) {
    check_rows(s, p, p.a, seen);
  } else {
    if (threadIdx.x == 0) s.bad = 0;
    __syncthreads();
  }
  ahead.arrived();
  auto slot = [&](int i) { return p.a ? p.a[i] : i; };
  auto begin = [&]() { return TRIM ? pages_of(p, p.sinks) : 0; };
  // Read by every thread before any writes it again below: a thread that saw a
  // bad length flagged here would pass by the barriers that the others wait at.
  const bool listed = !s.bad;
  __syncthreads();
  if (listed)
    list_scan(s, p.n, first, [&](int i) {
      const int len = p.lens[slot(i)];
      if (!good_len(p, len)) {
        s.bad = 1;
        return 0;
      }
      if (!TRIM) return pages_of(p, len);
      return max(0, (max(0, len - p.window) >> p.shift) - begin());
    });
  const bool bad = s.bad;
  cluster_sync();                            // every CTA has read the lengths
  if (bad) {
    refuse(p, rank, ATTN_ERR_INVALID_ARG);
    return;
  }
  const int total = first[p.n], j0 = begin();
  for (int x = rank * CT + threadIdx.x; x < total; x += CALL) {
    const int i = list_find(first, p.n, x);
    int32_t *e = p.table + slot(i) * p.stride + j0 + x - first[i];
    const int page = *e;
    *e = -1;
    drop(p, page);
  }
  if (!TRIM && rank == 0)
    for (int i = threadIdx.x; i < p.n; i += CT) p.lens[slot(i)] = 0;
}

// ---------------------------------------------------------------- fork

// All rows of the list at once, as they stood before the call: row b[i]
// becomes a copy of row a[i].  Rows are read into the workspace (a row may be
// a source and be replaced), fresh pages are chosen, then the barrier, then
// rows and counts are written.
__global__ void __cluster_dims__(CC, 1, 1) __launch_bounds__(CT, 1) cache_fork_kernel(const CacheParams p) {
  after_previous();
  admit_next();
  __shared__ CacheSmem s;
  cluster_started();
  const int rank = cluster_ctarank(), n = p.n;
  int *first = cache_smem;                   // [n + 1] row entries to write
  int *rank_of = first + n + 1;              // [n + 1] copies before child i
  int *len = rank_of + n + 1;                // [n] of the source
  int *heir = len + n;                       // [n_slots] first child of each source
  uint32_t *seen = reinterpret_cast<uint32_t *>(heir + p.n_slots);
  int32_t *fresh = p.ws, *rows = p.ws + n;
  int from, to;
  page_share(p, rank, from, to);
  Ahead ahead(p, from, to);
  check_rows(s, p, p.b, seen);               // seen: the rows that are replaced
  ahead.arrived();
  for (int i = threadIdx.x; i < p.n_slots; i += CT) heir[i] = INT_MAX;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += CT) {
    const int a = p.a[i];
    if (a < 0 || a >= p.n_slots) {
      s.bad = 1;
    } else {
      len[i] = p.lens[a];
      if (!good_len(p, len[i])) s.bad = 1;
      atomicMin(&heir[a], i);
    }
  }
  __syncthreads();
  unsigned code = s.bad ? ATTN_ERR_INVALID_ARG : 0u;
  // the partial page stays with the source, or with its first child where the source is replaced
  auto part = [&](int i) { return (len[i] & ((1 << p.shift) - 1)) != 0; };
  auto copied = [&](int i) {
    const int a = p.a[i];
    return part(i) && !((seen[a >> 5] >> (a & 31) & 1u) && heir[a] == i);
  };
  int want = 0;
  if (code == 0) {
    want = list_scan(s, n, rank_of, [&](int i) { return copied(i) ? 1 : 0; });
    list_scan(s, n, first, [&](int i) {
      const int old = p.lens[p.b[i]];
      if (!good_len(p, old)) s.bad = 1;
      return max(pages_of(p, len[i]), pages_of(p, max(0, min(old, p.max_pages << p.shift))));
    });
    if (s.bad) code = ATTN_ERR_INVALID_ARG;
    else if (want > p.cap) code = ATTN_ERR_CAPACITY;
  }
  auto is_free = [](int, int r) { return r == 0; };
  const int mine = code ? 0 : count_pages(s, p, from, to, is_free);
  cluster_wait_started();
  share_count(s.count, mine, rank);
  if (code == 0) {
    int before = 0, total = 0;
    for (int c = 0; c < CC; ++c) {
      before += c < rank ? s.count[c] : 0;
      total += s.count[c];
    }
    if (total < want) code = ATTN_ERR_CAPACITY;
    else
      rank_pages(s, p, from, to, before, want, is_free, [&](int r, int page) { fresh[r] = page; });
  }
  const int total = code ? 0 : first[n], x0 = rank * CT + threadIdx.x;
  // the thread's first entry waits for the barrier in registers, others in the workspace
  int i0 = 0, page0 = -1, old0 = -1;
  if (x0 < total) {
    i0 = list_find(first, n, x0);
    const int j = x0 - first[i0];
    if (j < pages_of(p, len[i0])) page0 = p.table[p.a[i0] * p.stride + j];
    old0 = p.table[p.b[i0] * p.stride + j];
  }
  for (int x = x0 + CALL; x < total; x += CALL) {
    const int i = list_find(first, n, x), j = x - first[i];
    if (j < pages_of(p, len[i])) rows[x] = p.table[p.a[i] * p.stride + j];
  }
  cluster_sync();
  if (code) {
    refuse(p, rank, code);
    return;
  }
  for (int x = x0; x < total; x += CALL) {
    const int i = x == x0 ? i0 : list_find(first, n, x), j = x - first[i], np = pages_of(p, len[i]);
    int32_t *e = p.table + p.b[i] * p.stride + j;
    const int old = x == x0 ? old0 : *e;
    int page = -1;
    if (j < np) {
      page = x == x0 ? page0 : rows[x];
      if (j == np - 1 && copied(i)) {
        const int r = rank_of[i];
        p.copies[1 + r] = page;
        page = fresh[r];
        p.copies[1 + p.cap + r] = page;
        p.refs[page] = 1;
      } else if (page >= p.n_pages) {
        atomicCAS(p.status, 0u, static_cast<unsigned>(ATTN_ERR_INVALID_ARG));
        page = -1;
      } else if (page >= 0) {
        atomicAdd(p.refs + page, 1);
      }
    }
    *e = page;
    drop(p, old);
  }
  for (int r = want + rank * CT + threadIdx.x; r < p.cap; r += CALL) p.copies[1 + r] = p.copies[1 + p.cap + r] = -1;
  if (rank == 0) {
    for (int i = threadIdx.x; i < n; i += CT) p.lens[p.b[i]] = len[i];
    if (threadIdx.x == 0) p.copies[0] = want;
  }
}

// ---------------------------------------------------------------- compact

// Pages in use move to the lowest indices: those at `used` and above, in
// ascending order, into the free ones below it, in ascending order.
__global__ void __cluster_dims__(CC, 1, 1) __launch_bounds__(CT, 1) cache_compact_kernel(const CacheParams p) {
  after_previous();
  admit_next();
  __shared__ CacheSmem s;
  cluster_started();
  const int rank = cluster_ctarank();
  int *first = cache_smem;                   // [n_slots + 1]
  int32_t *moved = p.ws;                     // [n_pages] where a page at `used` or above goes
  int32_t *src = p.copies + 1, *dst = src + p.cap;
  int from, to;
  page_share(p, rank, from, to);
  Ahead ahead(p, from, to);
  if (threadIdx.x == 0) s.bad = 0;
  __syncthreads();
  ahead.arrived();
  list_scan(s, p.n_slots, first, [&](int i) {
    const int len = p.lens[i];
    if (!good_len(p, len)) {
      s.bad = 1;
      return 0;
    }
    return pages_of(p, len);
  });
  const int in_use = count_pages(s, p, from, to, [](int, int r) { return r != 0; });
  cluster_wait_started();
  share_count(s.count, in_use, rank);
  int used = 0;
  for (int c = 0; c < CC; ++c) used += s.count[c];
  auto high = [used](int x, int r) { return r != 0 && x >= used; };
  auto hole = [used](int x, int r) { return r == 0 && x < used; };
  share_count(s.count2, count_pages(s, p, from, to, high), rank);
  // holes below `used` before this CTA: pages below it less those in use
  int high_before = 0, moves = 0, hole_before = min(from, used);
  for (int c = 0; c < CC; ++c) {
    moves += s.count2[c];
    if (c < rank) {
      high_before += s.count2[c];
      hole_before -= s.count[c] - s.count2[c];
    }
  }
  const unsigned code = s.bad ? ATTN_ERR_INVALID_ARG : moves > p.cap ? ATTN_ERR_CAPACITY : 0u;
  if (code) {
    refuse(p, rank, code);
    return;                                  // all CTAs alike, and none is written to any more
  }
  rank_pages(s, p, from, to, high_before, moves, high, [&](int r, int page) { src[r] = page; });
  rank_pages(s, p, from, to, hole_before, moves, hole, [&](int r, int page) { dst[r] = page; });
  for (int x = max(from, used) + threadIdx.x; x < to; x += CT) moved[x] = -1;
  cluster_sync();
  for (int r = rank * CT + threadIdx.x; r < moves; r += CALL) {
    const int a = src[r], b = dst[r];
    moved[a] = b;
    p.refs[b] = p.refs[a];
    p.refs[a] = 0;
  }
  for (int r = moves + rank * CT + threadIdx.x; r < p.cap; r += CALL) src[r] = dst[r] = -1;
  if (rank == 0 && threadIdx.x == 0) p.copies[0] = moves;
  cluster_sync();
  const int total = first[p.n_slots];
  for (int x = rank * CT + threadIdx.x; x < total; x += CALL) {
    const int i = list_find(first, p.n_slots, x);
    int32_t *e = p.table + i * p.stride + x - first[i];
    const int page = *e;
    if (page < used) continue;
    const int to_page = page < p.n_pages ? moved[page] : -1;
    if (to_page >= 0) *e = to_page;
    else atomicCAS(p.status, 0u, static_cast<unsigned>(ATTN_ERR_INVALID_ARG));   // in the table, but not counted
  }
}

// ---------------------------------------------------------------- copy, write

struct CopyParams {
  uint8_t *pool[ATTN_CACHE_MAX_POOLS];
  const int32_t *copies;
  long long page_stride;        // bytes
  int n_pools, cap, n_pages, chunks, tail;   // chunks of CHUNK bytes a page, the last of `tail` 16-byte words
  unsigned int *status;
};

constexpr int COPY_T = 256, COPY_U = 4, COPY_CHUNK = COPY_T * COPY_U * 16;

// Streams pages: a unit is 16 KB of one page of one pool, four 16-byte words a
// thread, all loaded before the first is stored.  Bound by HBM: 1570 pages of
// 128 KB in 4 pools, 1646 MB read and written, in 265 us (6.2 TB/s; a plain copy
// of as many bytes takes 240).  Bulk copies through shared memory took
// 263 to 267, 8 words a thread 262 here and 7 % more on a fragmented pool.
// Stores that leave the pages in L2: what is copied is read next (a compaction and
// an admission behind it 311 -> 307 us, a beam search's step 11.1 -> 11.0).
__global__ void __launch_bounds__(COPY_T) cache_copy_kernel(const __grid_constant__ CopyParams p) {
  after_previous();
  admit_next();
  const int count = min(max(p.copies[0], 0), p.cap);
  const long long units = static_cast<long long>(count) * p.chunks * p.n_pools;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const int c = static_cast<int>(u % p.chunks);
    const long long y = u / p.chunks;
    const int pool = static_cast<int>(y % p.n_pools), r = static_cast<int>(y / p.n_pools);
    const int a = p.copies[1 + r], b = p.copies[1 + p.cap + r];
    if (a < 0 || b < 0 || a >= p.n_pages || b >= p.n_pages) {
      if (threadIdx.x == 0) atomicCAS(p.status, 0u, static_cast<unsigned>(ATTN_ERR_INVALID_ARG));
      continue;
    }
    const int words = c == p.chunks - 1 ? p.tail : COPY_CHUNK / 16;
    const int4 *src = reinterpret_cast<const int4 *>(p.pool[pool] + a * p.page_stride + static_cast<long long>(c) * COPY_CHUNK);
    int4 *dst = reinterpret_cast<int4 *>(p.pool[pool] + b * p.page_stride + static_cast<long long>(c) * COPY_CHUNK);
    int4 x[COPY_U];
#pragma unroll
    for (int k = 0; k < COPY_U; ++k)
      if (k * COPY_T + threadIdx.x < words) x[k] = __ldcs(src + k * COPY_T + threadIdx.x);
#pragma unroll
    for (int k = 0; k < COPY_U; ++k)
      if (k * COPY_T + threadIdx.x < words) dst[k * COPY_T + threadIdx.x] = x[k];
  }
}

struct WriteParams {
  uint16_t *k, *v;
  const uint16_t *k_new, *v_new;
  const int32_t *q_ptr, *seqs, *lens, *table;
  long long table_stride, page_stride, token_stride, head_stride, new_token, new_head;   // elements
  int n_tokens, n_seqs, n_slots, max_pages, n_pages, shift, hk, words, run;   // words: 16-byte words of a head's row
  unsigned int *status;
};

// A warp takes p.run tokens at a time: 2 where that leaves every SM 32 warps, else
// 1.  Its lanes find the tokens' sequences and pages, a token a lane, then move
// token after token together, a token's 16-byte words (WRITE_WORDS a lane, keys and
// values) all loaded before the first is stored.  Bound by HBM: 43200 tokens of 8
// heads of 128 read and written (354 MB) in 58 us, 6.1 TB/s; word by word 61, one
// token at a time 59.5, four 57.4 but more where the tokens are still in L2
// (48.4 us of a server's round of arrivals with two, 49.1 with one, 49.9 with four).
constexpr int WRITE_WORDS = 4;
__global__ void __launch_bounds__(256) cache_write_kernel(const WriteParams p) {
  after_previous();
  admit_next();
  const int lane = threadIdx.x & 31, all = p.hk * p.words;
  const long long warp = blockIdx.x * 8ll + (threadIdx.x >> 5), warps = gridDim.x * 8ll;
  for (long long t0 = warp * p.run; t0 < p.n_tokens; t0 += warps * p.run) {
    const int t = static_cast<int>(t0) + lane;
    long long at = -1;                            // where the token's rows go; -1: it is not written
    if (lane < p.run && t < p.n_tokens) {
      int b = t, q0 = t, q1 = t + 1;
      if (p.q_ptr) {
        // the largest b < n_seqs with q_ptr[b] <= t
        b = 0;
        for (int hi = p.n_seqs; hi - b > 1;) {
          const int mid = (b + hi) >> 1;
          if (p.q_ptr[mid] <= t) b = mid;
          else hi = mid;
        }
        q0 = p.q_ptr[b];
        q1 = p.q_ptr[b + 1];
      }
      if (t >= q0 && t < q1) {                    // else of no sequence
        const int slot = p.seqs ? p.seqs[b] : b;
        bool good = slot >= 0 && slot < p.n_slots && q0 >= 0 && q1 <= p.n_tokens;
        if (good) {
          const int pos = p.lens[slot] - (q1 - t);
          good = pos >= 0 && (pos >> p.shift) < p.max_pages;
          if (good) {
            const int page = p.table[slot * p.table_stride + (pos >> p.shift)];
            good = page >= 0 && page < p.n_pages;
            at = page * p.page_stride + (pos & ((1 << p.shift) - 1)) * p.token_stride;
          }
        }
        if (!good) {
          at = -1;
          atomicCAS(p.status, 0u, static_cast<unsigned>(ATTN_ERR_INVALID_ARG));
        }
      }
    }
    __syncwarp();
    const int n = static_cast<int>(min(static_cast<long long>(p.run), p.n_tokens - t0));
    for (int i = 0; i < n; ++i) {
      const long long to = __shfl_sync(0xffffffffu, at, i);
      if (to < 0) continue;
      const long long from = (t0 + i) * p.new_token;
      for (int w0 = lane; w0 < all; w0 += 32 * WRITE_WORDS) {
        int4 x[WRITE_WORDS], y[WRITE_WORDS];
#pragma unroll
        for (int k = 0; k < WRITE_WORDS; ++k) {
          const int w = w0 + 32 * k, h = w / p.words, c = (w - h * p.words) * 8;
          if (w < all) {
            x[k] = __ldcs(reinterpret_cast<const int4 *>(p.k_new + from + h * p.new_head + c));
            y[k] = __ldcs(reinterpret_cast<const int4 *>(p.v_new + from + h * p.new_head + c));
          }
        }
#pragma unroll
        for (int k = 0; k < WRITE_WORDS; ++k) {
          const int w = w0 + 32 * k, h = w / p.words, c = (w - h * p.words) * 8;
          if (w < all) {
            *reinterpret_cast<int4 *>(p.k + to + h * p.head_stride + c) = x[k];
            *reinterpret_cast<int4 *>(p.v + to + h * p.head_stride + c) = y[k];
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------- host

namespace {

int cache_check(const attn_cache_t *c, CacheParams *p) {
  std::memset(p, 0, sizeof(*p));
  if (!c || !c->table || !c->seq_lens || !c->refs) return ATTN_ERR_INVALID_ARG;
  if (c->n_slots < 1 || c->max_pages < 1 || c->n_pages < 1 || c->table_stride < c->max_pages) return ATTN_ERR_INVALID_ARG;
  if (c->page_size < 16 || (c->page_size & (c->page_size - 1))) return ATTN_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(c->max_pages) * c->page_size > ATTN_PAGED_MAX_LEN || c->n_slots > ATTN_CACHE_MAX_SLOTS ||
      c->n_pages > ATTN_CACHE_MAX_PAGES || static_cast<int64_t>(c->n_slots) * c->max_pages >= (int64_t(1) << 31))
    return ATTN_ERR_UNSUPPORTED;
  p->table = c->table;
  p->lens = c->seq_lens;
  p->refs = c->refs;
  p->stride = c->table_stride;
  p->n_slots = c->n_slots;
  p->max_pages = c->max_pages;
  p->n_pages = c->n_pages;
  while ((1 << p->shift) < c->page_size) ++p->shift;
  return ATTN_OK;
}

int list_check(CacheParams *p, const int32_t *a, const int32_t *b, bool two, int n) {
  if (n < 0 || (n > 0 && (!a || (two && !b)))) return ATTN_ERR_INVALID_ARG;
  if (n > ATTN_PAGED_MAX_SEQS) return ATTN_ERR_UNSUPPORTED;
  if (n > p->n_slots) return ATTN_ERR_INVALID_ARG;     // a row is named once at most
  p->a = a;
  p->b = b;
  p->n = n;
  return ATTN_OK;
}

constexpr int kDev = 64;

int cache_launch(void (*kern)(const CacheParams), bool (&done)[kDev], CacheParams p, size_t smem, cudaStream_t s) {
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDev) return ATTN_ERR_CUDA;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev]) {
      if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024) != cudaSuccess)
        return ATTN_ERR_CUDA;
      done[dev] = true;
    }
  }
  if (!(p.status = paged_status())) return ATTN_ERR_CUDA;
  return launch_after(kern, dim3(CC), CT, smem, s, p);
}

size_t bits(int n_slots) { return 4ull * ((n_slots + 31) / 32); }

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" {

int attn_cache_extend(const attn_cache_t *cache, const int32_t *seqs, const int32_t *counts, int n, attn_stream_t stream) {
  CacheParams p;
  int rc;
  if ((rc = cache_check(cache, &p)) != ATTN_OK || (rc = list_check(&p, seqs, counts, true, n)) != ATTN_OK) return rc;
  if (n == 0) return ATTN_OK;
  static bool done[kDev];
  return cache_launch(cache_extend_kernel, done, p, 4ull * (2 * n + 1) + bits(p.n_slots), reinterpret_cast<cudaStream_t>(stream));
}

int attn_cache_free(const attn_cache_t *cache, const int32_t *seqs, int n, attn_stream_t stream) {
  CacheParams p;
  int rc;
  if ((rc = cache_check(cache, &p)) != ATTN_OK || (rc = list_check(&p, seqs, nullptr, false, n)) != ATTN_OK) return rc;
  if (n == 0) return ATTN_OK;
  static bool done[kDev];
  return cache_launch(cache_free_kernel<false>, done, p, 4ull * (n + 1) + bits(p.n_slots), reinterpret_cast<cudaStream_t>(stream));
}

int attn_cache_trim(const attn_cache_t *cache, const int32_t *seqs, int n, int window, int sinks, attn_stream_t stream) {
  CacheParams p;
  int rc;
  if (window < 1 || sinks < 0) return ATTN_ERR_INVALID_ARG;
  if ((rc = cache_check(cache, &p)) != ATTN_OK) return rc;
  if (seqs) {
    if ((rc = list_check(&p, seqs, nullptr, false, n)) != ATTN_OK) return rc;
  } else {
    if (n != p.n_slots) return ATTN_ERR_INVALID_ARG;
    p.n = n;
  }
  if (n == 0) return ATTN_OK;
  p.window = window < ATTN_PAGED_MAX_LEN ? window : ATTN_PAGED_MAX_LEN;
  p.sinks = sinks < ATTN_PAGED_MAX_LEN ? sinks : ATTN_PAGED_MAX_LEN;
  static bool done[kDev];
  return cache_launch(cache_free_kernel<true>, done, p, 4ull * (p.n + 1) + bits(p.n_slots), reinterpret_cast<cudaStream_t>(stream));
}

int attn_cache_workspace_bytes(const attn_cache_t *cache, int n, size_t *bytes) {
  CacheParams p;
  int rc;
  if (!bytes || n < 0) return ATTN_ERR_INVALID_ARG;
  if ((rc = cache_check(cache, &p)) != ATTN_OK) return rc;
  if (n > ATTN_PAGED_MAX_SEQS) return ATTN_ERR_UNSUPPORTED;
  const size_t fork = 4ull * n * (static_cast<size_t>(p.max_pages) + 1), compact = 4ull * p.n_pages;
  *bytes = fork > compact ? fork : compact;
  return ATTN_OK;
}

int attn_cache_fork(const attn_cache_t *cache, const int32_t *src, const int32_t *dst, int n, int32_t *copies, int cap,
                    void *d_ws, size_t ws_bytes, attn_stream_t stream) {
  CacheParams p;
  int rc;
  if ((rc = cache_check(cache, &p)) != ATTN_OK || (rc = list_check(&p, src, dst, true, n)) != ATTN_OK) return rc;
  if (!copies || cap < 0) return ATTN_ERR_INVALID_ARG;
  if (n > 0 && !d_ws) return ATTN_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(d_ws) & 3) return ATTN_ERR_UNSUPPORTED;
  if (ws_bytes < 4ull * n * (static_cast<size_t>(p.max_pages) + 1)) return ATTN_ERR_CAPACITY;
  p.copies = copies;
  p.cap = cap;
  p.ws = static_cast<int32_t *>(d_ws);
  static bool done[kDev];
  return cache_launch(cache_fork_kernel, done, p, 4ull * (3 * n + 2 + p.n_slots) + bits(p.n_slots),
                      reinterpret_cast<cudaStream_t>(stream));
}

int attn_cache_compact(const attn_cache_t *cache, int32_t *copies, int cap, void *d_ws, size_t ws_bytes, attn_stream_t stream) {
  CacheParams p;
  int rc;
  if ((rc = cache_check(cache, &p)) != ATTN_OK) return rc;
  if (!copies || cap < 0 || !d_ws) return ATTN_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(d_ws) & 3) return ATTN_ERR_UNSUPPORTED;
  if (ws_bytes < 4ull * p.n_pages) return ATTN_ERR_CAPACITY;
  p.copies = copies;
  p.cap = cap;
  p.ws = static_cast<int32_t *>(d_ws);
  static bool done[kDev];
  return cache_launch(cache_compact_kernel, done, p, 4ull * (p.n_slots + 1), reinterpret_cast<cudaStream_t>(stream));
}

int attn_cache_copy_pages(void *const *h_pools, int n_pools, size_t page_bytes, size_t page_stride_bytes, int n_pages,
                          const int32_t *copies, int cap, attn_stream_t stream) {
  if (n_pools < 0 || (n_pools > 0 && !h_pools) || n_pages < 1 || !copies || cap < 0) return ATTN_ERR_INVALID_ARG;
  if (n_pools > ATTN_CACHE_MAX_POOLS || page_bytes >= (size_t(1) << 31)) return ATTN_ERR_UNSUPPORTED;
  if (page_bytes == 0 || page_stride_bytes < page_bytes) return ATTN_ERR_INVALID_ARG;
  if ((page_bytes | page_stride_bytes) & 15) return ATTN_ERR_UNSUPPORTED;
  CopyParams p;
  std::memset(&p, 0, sizeof(p));
  for (int i = 0; i < n_pools; ++i) {
    if (!h_pools[i]) return ATTN_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(h_pools[i]) & 15) return ATTN_ERR_UNSUPPORTED;
    p.pool[i] = static_cast<uint8_t *>(h_pools[i]);
  }
  if (n_pools == 0 || cap == 0) return ATTN_OK;
  p.copies = copies;
  p.page_stride = static_cast<long long>(page_stride_bytes);
  p.n_pools = n_pools;
  p.cap = cap;
  p.n_pages = n_pages;
  p.chunks = static_cast<int>((page_bytes + COPY_CHUNK - 1) / COPY_CHUNK);
  p.tail = static_cast<int>((page_bytes - static_cast<size_t>(p.chunks - 1) * COPY_CHUNK) / 16);
  if (!(p.status = paged_status())) return ATTN_ERR_CUDA;
  const int sms = device_sm_count();
  if (sms <= 0) return ATTN_ERR_CUDA;
  const long long most = static_cast<long long>(cap) * p.chunks * n_pools, grid = sms * 8;
  return launch_after(cache_copy_kernel, dim3(static_cast<unsigned>(most < grid ? most : grid)), COPY_T, 0,
                      reinterpret_cast<cudaStream_t>(stream), p);
}

int attn_cache_write(const attn_pages_t *pages, const attn_seqs_t *seqs, const int32_t *q_ptr, const void *k_new,
                     const void *v_new, int n_tokens, int64_t new_token_stride, int64_t new_head_stride,
                     attn_stream_t stream) {
  int shift = 0, rc;
  if (n_tokens < 0) return ATTN_ERR_INVALID_ARG;
  if ((rc = paged_check_pages(pages, &shift)) != ATTN_OK || (rc = paged_check_seqs(seqs, pages->page_size)) != ATTN_OK) return rc;
  if (!q_ptr && n_tokens != seqs->n_seqs) return ATTN_ERR_INVALID_ARG;
  if (n_tokens == 0 || seqs->n_seqs == 0) return ATTN_OK;
  if (!k_new || !v_new) return ATTN_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(k_new) | reinterpret_cast<uintptr_t>(v_new)) & 15) return ATTN_ERR_UNSUPPORTED;
  if ((new_token_stride | new_head_stride) & 7 || new_token_stride < 0 || new_head_stride < 0) return ATTN_ERR_UNSUPPORTED;
  // one place of memory seen as several is fine to read, not to write
  if ((pages->page_stride == 0 && pages->n_pages > 1) || pages->token_stride == 0 || (pages->head_stride == 0 && pages->hk > 1))
    return ATTN_ERR_UNSUPPORTED;
  if (n_tokens > ATTN_PAGED_MAX_LEN) return ATTN_ERR_UNSUPPORTED;
  WriteParams p;
  p.k = static_cast<uint16_t *>(const_cast<void *>(pages->k));
  p.v = static_cast<uint16_t *>(const_cast<void *>(pages->v));
  p.k_new = static_cast<const uint16_t *>(k_new);
  p.v_new = static_cast<const uint16_t *>(v_new);
  p.q_ptr = q_ptr;
  p.seqs = seqs->seqs;
  p.lens = seqs->seq_lens;
  p.table = seqs->table;
  p.table_stride = seqs->table_stride;
  p.page_stride = pages->page_stride;
  p.token_stride = pages->token_stride;
  p.head_stride = pages->head_stride;
  p.new_token = new_token_stride;
  p.new_head = new_head_stride;
  p.n_tokens = n_tokens;
  p.n_seqs = seqs->n_seqs;
  p.n_slots = seqs->n_slots;
  p.max_pages = seqs->max_pages;
  p.n_pages = pages->n_pages;
  p.shift = shift;
  p.hk = pages->hk;
  p.words = pages->d / 8;
  if (!(p.status = paged_status())) return ATTN_ERR_CUDA;
  const int sms = device_sm_count();
  if (sms <= 0) return ATTN_ERR_CUDA;
  p.run = n_tokens >= sms * 64 ? 2 : 1;
  const int blocks = (n_tokens + 8 * p.run - 1) / (8 * p.run), grid = sms * 8;
  return launch_after(cache_write_kernel, dim3(blocks < grid ? blocks : grid), 256, 0,
                      reinterpret_cast<cudaStream_t>(stream), p);
}

}  // extern "C"
