// Tokens of the cache as rows: new ones written to pages in 8 bits, cached ones read
// back from pages of either kind.
//
// A head's row becomes codes with one scale: a = max |x| over it, scale = a / M
// (M = 127 for int8, 448 for e4m3), code = x M / a rounded to the nearest code,
// halfway ones to the even.  That rounding is exact: x and a are bf16, of 8
// significant bits, so a quotient x M / a that is not halfway between two codes is
// further from it than 2^-20 of itself, and one that is halfway is an f32 number.  So M / a
// is taken as hi + lo, a quotient and what its remainder leaves (to 2^-40 of it, once a
// row), and x hi + x lo by one product and one fused addition: where the quotient is an f32
// number that is the number.  A division a value took the kernel twice its time, a
// correction by each value's own remainder 2 % more.  a is brought to [1, 2) first, by a power of two,
// so that nothing overflows.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "attn_device.cuh"
#include "attn_internal.h"
#include "codes.cuh"
#include "launch.cuh"
#include "ptx.cuh"

namespace attn {

namespace {

enum { FROM_BF16 = -1 };       // of pages that hold bf16; else ATTN_CODES_*

struct TokenParams {
  uint8_t *k, *v;                       // pages
  float *k_scales, *v_scales;
  const uint16_t *k_new, *v_new;        // write
  uint8_t *k_out, *v_out;               // read
  const int32_t *q_ptr, *seqs, *lens, *table;
  long long table_stride, page_stride, token_stride, head_stride, scale_page, scale_token, scale_head, new_token, new_head;   // elements
  int n_tokens, n_seqs, n_slots, max_pages, n_pages, shift, hk, words, run;   // words: a head's row in words of 8 values
  uint32_t per_token, per_head;      // 2^32 / (hk words) and 2^32 / words, rounded up
  unsigned int *status;
};

// Where token t's rows and scales begin in the pages; at -1: of no sequence, or out of
// range (then the status says so).
struct Place {
  long long at, scales;
};
__device__ __forceinline__ Place place_of(const TokenParams &p, int t) {
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
  if (t < q0 || t >= q1) return Place{-1, 0};
  const int slot = p.seqs ? p.seqs[b] : b;
  if (slot >= 0 && slot < p.n_slots && q0 >= 0 && q1 <= p.n_tokens) {
    const int pos = p.lens[slot] - (q1 - t);
    if (pos >= 0 && (pos >> p.shift) < p.max_pages) {
      const int page = p.table[slot * p.table_stride + (pos >> p.shift)], row = pos & ((1 << p.shift) - 1);
      if (page >= 0 && page < p.n_pages) return Place{page * p.page_stride + row * p.token_stride, page * p.scale_page + row * p.scale_token};
    }
  }
  atomicCAS(p.status, 0u, static_cast<unsigned>(ATTN_ERR_INVALID_ARG));
  return Place{-1, 0};
}

__device__ __forceinline__ float bf16_of(uint32_t half) { return __uint_as_float(half << 16); }

// On pairs, subnormal numbers as they are.
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// Codes of 8 values (16 bytes of bf16), given the bit pattern of the row's
// largest magnitude; lowest byte first.
template <int FMT>
__device__ __forceinline__ uint2 encode8(const int4 &x, uint32_t top) {
  constexpr float M = FMT == ATTN_CODES_INT8 ? 127.f : 448.f;
  if (top == 0 || top >= 0x7f80u) return make_uint2(0u, 0u);
  const float a = bf16_of(top);
  // 2^(127 - exponent), as far as M times it stays finite
  const float f = __uint_as_float(static_cast<uint32_t>(min(max(254 - static_cast<int>(top >> 7), 1), 240)) << 23);
  const float den = a * f;
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(den));
  const float hi = M * inv, lo = __fmaf_rn(-hi, den, M) * inv;
  const uint64_t f2 = f2_make(f, f), hi2 = f2_make(hi, hi), lo2 = f2_make(lo, lo);
  const uint32_t w[4] = {static_cast<uint32_t>(x.x), static_cast<uint32_t>(x.y), static_cast<uint32_t>(x.z), static_cast<uint32_t>(x.w)};
  uint32_t out[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float y[4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint64_t v = mul2(f2_make(__uint_as_float(w[2 * i + e] << 16), __uint_as_float(w[2 * i + e] & 0xffff0000u)), f2);
      f2_split(fma2(v, hi2, mul2(v, lo2)), y[2 * e], y[2 * e + 1]);
    }
    if constexpr (FMT == ATTN_CODES_INT8) {
      // 1.5 2^23 + y has the nearest whole number, the even one of two, in its low byte
      constexpr float kWhole = 12582912.f;
      const uint32_t lo = __byte_perm(__float_as_uint(y[0] + kWhole), __float_as_uint(y[1] + kWhole), 0x0040),
                     hi = __byte_perm(__float_as_uint(y[2] + kWhole), __float_as_uint(y[3] + kWhole), 0x0040);
      out[i] = __byte_perm(lo, hi, 0x5410);
    } else {
      asm("{\n\t.reg .b16 l, h;\n\t"
          "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
          "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
          "mov.b32 %0, {l, h};\n\t}"
          : "=r"(out[i])
          : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]));
    }
  }
  return make_uint2(out[0], out[1]);
}

// a / M of the largest magnitude's bit pattern, rounded once: the quotient corrected by its
// remainder is that for all 128 significands of bf16; a division where it is subnormal.
template <int FMT>
__device__ __forceinline__ float scale_of(uint32_t top) {
  constexpr float M = FMT == ATTN_CODES_INT8 ? 127.f : 448.f, inv = 1.f / M;
  if (top >= 0x7f80u) return __uint_as_float(0x7fffffffu);
  const float a = bf16_of(top), q = a * inv;
  return top < 0x0800u ? __fdiv_rn(a, M) : __fmaf_rn(__fmaf_rn(-q, M, a), inv, q);
}

// The larger of two pairs of magnitudes; one that is no number counts as the largest of all.
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Largest magnitude, as a bit pattern, of 8 values.
__device__ __forceinline__ uint32_t top8(const int4 &x) {
  const uint32_t m = 0x7fff7fffu;
  const uint32_t a = larger(larger(x.x & m, x.y & m), larger(x.z & m, x.w & m));
  return max(a & 0xffffu, a >> 16);
}

constexpr int TOKEN_WORDS = 4, MAX_HEADS = 1024;

// A warp takes p.run tokens at a time: its lanes find their places, a token a lane, then
// the tokens' words of 8 values, one after the other, are shared out to them, up to
// TOKEN_WORDS of keys and of values each.  f(word) is called by all lanes together;
// word(k, ..), k < TOKEN_WORDS, too, gives token, place, head and first column, and whether
// there is such a word of a token that has a place.
template <typename F>
__device__ __forceinline__ void for_words(const TokenParams &p, F f) {
  const int lane = threadIdx.x & 31, all = p.hk * p.words;
  const long long warp = blockIdx.x * 8ll + (threadIdx.x >> 5), warps = gridDim.x * 8ll;
  for (long long t0 = warp * p.run; t0 < p.n_tokens; t0 += warps * p.run) {
    Place mine{-1, 0};
    if (lane < p.run && t0 + lane < p.n_tokens) mine = place_of(p, static_cast<int>(t0) + lane);
    __syncwarp();
    const int n = static_cast<int>(min(static_cast<long long>(p.run), p.n_tokens - t0)) * all;
    for (int w0 = lane; w0 - lane < n; w0 += 32 * TOKEN_WORDS)
      f([&](int k, long long &t, Place &to, int &h, int &c) -> bool {
        const int x = min(w0 + 32 * k, n - 1), i = static_cast<int>(__umulhi(x, p.per_token)), w = x - i * all;
        h = static_cast<int>(__umulhi(w, p.per_head));
        c = (w - h * p.words) * 8;
        t = t0 + i;
        to.at = __shfl_sync(0xffffffffu, mine.at, i);
        to.scales = __shfl_sync(0xffffffffu, mine.scales, i);
        return w0 + 32 * k < n && to.at >= 0;
      });
  }
}

// The 8 or 16 lanes of a head's row find its largest value together, keys and values by one
// exchange.  BLOCKS an SM: of a call that fills the GPU 4, of 64 registers a thread (24 prompts of up to 8192
// tokens: 53.8 us, 56.6 with 74); one that does not is over sooner without that limit (64 tokens
// 4.15 us, 4.4 with it).
template <int FMT, int BLOCKS>
__global__ void __launch_bounds__(256, BLOCKS) cache_encode_kernel(const TokenParams p) {
  after_previous();
  admit_next();
  for_words(p, [&](auto word) {
    int4 x[TOKEN_WORDS], y[TOKEN_WORDS];
    long long to[TOKEN_WORDS], sto[TOKEN_WORDS];       // -1: none; none of this lane's
#pragma unroll
    for (int k = 0; k < TOKEN_WORDS; ++k) {
      long long t;
      Place at;
      int h, c;
      const bool on = word(k, t, at, h, c);
      x[k] = y[k] = make_int4(0, 0, 0, 0);
      to[k] = sto[k] = -1;
      if (on) {
        x[k] = __ldcs(reinterpret_cast<const int4 *>(p.k_new + t * p.new_token + h * p.new_head + c));
        y[k] = __ldcs(reinterpret_cast<const int4 *>(p.v_new + t * p.new_token + h * p.new_head + c));
        to[k] = at.at + h * p.head_stride + c;
        if (c == 0) sto[k] = at.scales + h * p.scale_head;
      }
    }
#pragma unroll
    for (int k = 0; k < TOKEN_WORDS; ++k) {
      uint32_t top = top8(x[k]) | top8(y[k]) << 16;
#pragma unroll
      for (int s = 1; s < 8; s <<= 1) top = larger(top, __shfl_xor_sync(0xffffffffu, top, s));
      if (p.words == 16) top = larger(top, __shfl_xor_sync(0xffffffffu, top, 8));
      if (to[k] >= 0) {
        *reinterpret_cast<uint2 *>(p.k + to[k]) = encode8<FMT>(x[k], top & 0xffffu);
        *reinterpret_cast<uint2 *>(p.v + to[k]) = encode8<FMT>(y[k], top >> 16);
        if (sto[k] >= 0) {
          p.k_scales[sto[k]] = scale_of<FMT>(top & 0xffffu);
          p.v_scales[sto[k]] = scale_of<FMT>(top >> 16);
        }
      }
    }
  });
}

// 8 values as f32.
template <int FMT>
struct Word {
  uint2 codes;
  float scale;
  __device__ __forceinline__ void load(const uint8_t *pages, const float *scales, long long at, long long sat) {
    codes = *reinterpret_cast<const uint2 *>(pages + at);
    scale = scales[sat];
  }
  __device__ __forceinline__ void values(float (&y)[8]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t a, b;
      F16Codes<FMT>::unpack(i ? codes.y : codes.x, a, b);
      auto two = [](uint32_t h, float &lo, float &hi) {
        asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}" : "=f"(lo), "=f"(hi) : "r"(h));
      };
      two(a, y[4 * i + F16Codes<FMT>::A0], y[4 * i + F16Codes<FMT>::A1]);
      two(b, y[4 * i + F16Codes<FMT>::B0], y[4 * i + F16Codes<FMT>::B1]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] *= scale;
  }
};
template <>
struct Word<FROM_BF16> {
  int4 x;
  __device__ __forceinline__ void load(const uint8_t *pages, const float *, long long at, long long) {
    x = *reinterpret_cast<const int4 *>(pages + 2 * at);
  }
  __device__ __forceinline__ void values(float (&y)[8]) const {
    const uint32_t w[4] = {static_cast<uint32_t>(x.x), static_cast<uint32_t>(x.y), static_cast<uint32_t>(x.z), static_cast<uint32_t>(x.w)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[2 * i] = __uint_as_float(w[i] << 16);
      y[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};

template <bool F32>
__device__ __forceinline__ void store8(uint8_t *out, long long at, const float (&y)[8]) {
  if constexpr (F32) {
    float4 *to = reinterpret_cast<float4 *>(out + 4 * at);
    __stcs(to, make_float4(y[0], y[1], y[2], y[3]));
    __stcs(to + 1, make_float4(y[4], y[5], y[6], y[7]));
  } else {
    __stcs(reinterpret_cast<uint4 *>(out + 2 * at),
           make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7])));
  }
}

template <int FMT, bool F32>
__global__ void __launch_bounds__(256) cache_read_kernel(const TokenParams p) {
  after_previous();
  admit_next();
  for_words(p, [&](auto word) {
    Word<FMT> x[TOKEN_WORDS], y[TOKEN_WORDS];
    long long to[TOKEN_WORDS];
#pragma unroll
    for (int k = 0; k < TOKEN_WORDS; ++k) {
      long long t;
      Place at;
      int h, c;
      const bool on = word(k, t, at, h, c);
      to[k] = on ? (t * p.hk + h) * (p.words * 8) + c : -1;
      if (on) {
        const long long from = at.at + h * p.head_stride + c, scale = at.scales + h * p.scale_head;
        x[k].load(p.k, p.k_scales, from, scale);
        y[k].load(p.v, p.v_scales, from, scale);
      }
    }
#pragma unroll
    for (int k = 0; k < TOKEN_WORDS; ++k) {
      if (to[k] >= 0) {
        float z[8];
        x[k].values(z);
        store8<F32>(p.k_out, to[k], z);
        y[k].values(z);
        store8<F32>(p.v_out, to[k], z);
      }
    }
  });
}

TokenParams token_params(const attn_pages_t *g, const attn_pages8_t *g8, const attn_seqs_t *s, const int32_t *q_ptr, int n_tokens, int shift) {
  TokenParams p;
  std::memset(&p, 0, sizeof(p));
  p.k = static_cast<uint8_t *>(const_cast<void *>(g->k));
  p.v = static_cast<uint8_t *>(const_cast<void *>(g->v));
  p.q_ptr = q_ptr;
  p.seqs = s->seqs;
  p.lens = s->seq_lens;
  p.table = s->table;
  p.table_stride = s->table_stride;
  p.page_stride = g->page_stride;
  p.token_stride = g->token_stride;
  p.head_stride = g->head_stride;
  if (g8) {
    p.k_scales = const_cast<float *>(g8->k_scales);
    p.v_scales = const_cast<float *>(g8->v_scales);
    p.scale_page = g8->scale_page_stride;
    p.scale_token = g8->scale_token_stride;
    p.scale_head = g8->scale_head_stride;
  }
  p.n_tokens = n_tokens;
  p.n_seqs = s->n_seqs;
  p.n_slots = s->n_slots;
  p.max_pages = s->max_pages;
  p.n_pages = g->n_pages;
  p.shift = shift;
  p.hk = g->hk;
  p.words = g->d / 8;
  // x / n for x < 4 n (a warp's tokens) is the upper half of x times this: right where
  // 4 n^2 < 2^32, and n is 16 MAX_HEADS at most
  p.per_token = static_cast<uint32_t>(((uint64_t(1) << 32) + p.hk * p.words - 1) / (p.hk * p.words));
  p.per_head = static_cast<uint32_t>(((uint64_t(1) << 32) + p.words - 1) / p.words);
  return p;
}

// kern: of a call of few tokens and of one that fills the GPU, which gets `per_sm` blocks an SM.
int launch_tokens(void (*few)(const TokenParams), void (*kern)(const TokenParams), int per_sm, TokenParams &p, attn_stream_t stream) {
  if (!(p.status = paged_status())) return ATTN_ERR_CUDA;
  const int sms = device_sm_count();
  if (sms <= 0) return ATTN_ERR_CUDA;
  // as many tokens a warp as leave every SM 32 warps, up to 4 (2, 4, 8, 16: 24 prompts written in
  // 63.1, 61.5, 68.3, 68.3 us, a batch of 32 sequences read back in 79.3, 64.2, 67.1, 63.4)
  p.run = std::max(1, std::min(4, p.n_tokens / (sms * 32)));        // 4: see token_params
  const int blocks = (p.n_tokens + 8 * p.run - 1) / (8 * p.run), grid = sms * per_sm;
  return launch_after(blocks < grid ? few : kern, dim3(blocks < grid ? blocks : grid), 256, 0, reinterpret_cast<cudaStream_t>(stream), p);
}

// What reads and writes of tokens share; *go: there is something to do.
int check_tokens(const attn_seqs_t *seqs, int page_size, int hk, const int32_t *q_ptr, int n_tokens, bool *go) {
  *go = false;
  if (n_tokens < 0) return ATTN_ERR_INVALID_ARG;
  const int rc = paged_check_seqs(seqs, page_size);
  if (rc != ATTN_OK) return rc;
  if (!q_ptr && n_tokens != seqs->n_seqs) return ATTN_ERR_INVALID_ARG;
  if (n_tokens > ATTN_PAGED_MAX_LEN || hk > MAX_HEADS) return ATTN_ERR_UNSUPPORTED;
  *go = n_tokens > 0 && seqs->n_seqs > 0;
  return ATTN_OK;
}

int read_tokens(const attn_pages_t *g, const attn_pages8_t *g8, const attn_seqs_t *seqs, const int32_t *q_ptr, int n_tokens, void *k_out,
                void *v_out, int out_dtype, int shift, attn_stream_t stream) {
  bool go;
  const int rc = check_tokens(seqs, g->page_size, g->hk, q_ptr, n_tokens, &go);
  if (rc != ATTN_OK) return rc;
  if (out_dtype != ATTN_DTYPE_BF16 && out_dtype != ATTN_DTYPE_F32) return ATTN_ERR_INVALID_ARG;
  if (!go) return ATTN_OK;
  if (!k_out || !v_out) return ATTN_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & 15) return ATTN_ERR_UNSUPPORTED;
  TokenParams p = token_params(g, g8, seqs, q_ptr, n_tokens, shift);
  p.k_out = static_cast<uint8_t *>(k_out);
  p.v_out = static_cast<uint8_t *>(v_out);
  const bool f32 = out_dtype == ATTN_DTYPE_F32;
  // 8 blocks an SM, two times the 4 that it holds at once (4: a batch of 32 sequences 67.2 us, 65.3)
  auto read = [&](void (*kern)(const TokenParams)) { return launch_tokens(kern, kern, 8, p, stream); };
  if (!g8) return read(f32 ? cache_read_kernel<FROM_BF16, true> : cache_read_kernel<FROM_BF16, false>);
  if (g8->format == ATTN_CODES_INT8) return read(f32 ? cache_read_kernel<ATTN_CODES_INT8, true> : cache_read_kernel<ATTN_CODES_INT8, false>);
  return read(f32 ? cache_read_kernel<ATTN_CODES_E4M3, true> : cache_read_kernel<ATTN_CODES_E4M3, false>);
}

}  // namespace

int paged_check_pages8(const attn_pages8_t *g, int *shift) {
  if (!g) return ATTN_ERR_INVALID_ARG;
  const int rc = paged_check_pages(&g->pages, shift);
  if (rc != ATTN_OK) return rc;
  if (!g->k_scales || !g->v_scales || (g->format != ATTN_CODES_INT8 && g->format != ATTN_CODES_E4M3)) return ATTN_ERR_INVALID_ARG;
  if ((g->pages.page_stride | g->pages.token_stride | g->pages.head_stride) & 15) return ATTN_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(g->k_scales) | reinterpret_cast<uintptr_t>(g->v_scales)) & 3) return ATTN_ERR_UNSUPPORTED;
  if (g->scale_page_stride < 0 || g->scale_token_stride < 0 || g->scale_head_stride < 0) return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

}  // namespace attn

using namespace attn;

extern "C" {

int attn_cache8_write(const attn_pages8_t *pages, const attn_seqs_t *seqs, const int32_t *q_ptr, const void *k_new, const void *v_new,
                      int n_tokens, int64_t new_token_stride, int64_t new_head_stride, attn_stream_t stream) {
  int shift = 0, rc;
  bool go;
  if ((rc = paged_check_pages8(pages, &shift)) != ATTN_OK) return rc;
  if ((rc = check_tokens(seqs, pages->pages.page_size, pages->pages.hk, q_ptr, n_tokens, &go)) != ATTN_OK || !go) return rc;
  if (!k_new || !v_new) return ATTN_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(k_new) | reinterpret_cast<uintptr_t>(v_new)) & 15) return ATTN_ERR_UNSUPPORTED;
  if ((new_token_stride | new_head_stride) & 7 || new_token_stride < 0 || new_head_stride < 0) return ATTN_ERR_UNSUPPORTED;
  // one place of memory seen as several is fine to read, not to write
  const attn_pages_t &g = pages->pages;
  if ((g.n_pages > 1 && (g.page_stride == 0 || pages->scale_page_stride == 0)) || g.token_stride == 0 || pages->scale_token_stride == 0 ||
      (g.hk > 1 && (g.head_stride == 0 || pages->scale_head_stride == 0)))
    return ATTN_ERR_UNSUPPORTED;
  TokenParams p = token_params(&g, pages, seqs, q_ptr, n_tokens, shift);
  p.k_new = static_cast<const uint16_t *>(k_new);
  p.v_new = static_cast<const uint16_t *>(v_new);
  p.new_token = new_token_stride;
  p.new_head = new_head_stride;
  constexpr int I8 = ATTN_CODES_INT8, E4 = ATTN_CODES_E4M3;
  if (pages->format == I8) return launch_tokens(cache_encode_kernel<I8, 1>, cache_encode_kernel<I8, 4>, 4, p, stream);
  return launch_tokens(cache_encode_kernel<E4, 1>, cache_encode_kernel<E4, 4>, 4, p, stream);
}

int attn_cache8_read(const attn_pages8_t *pages, const attn_seqs_t *seqs, const int32_t *q_ptr, int n_tokens, void *k_out, void *v_out,
                     int out_dtype, attn_stream_t stream) {
  int shift = 0;
  const int rc = paged_check_pages8(pages, &shift);
  return rc != ATTN_OK ? rc : read_tokens(&pages->pages, pages, seqs, q_ptr, n_tokens, k_out, v_out, out_dtype, shift, stream);
}

int attn_cache_read(const attn_pages_t *pages, const attn_seqs_t *seqs, const int32_t *q_ptr, int n_tokens, void *k_out, void *v_out,
                    int out_dtype, attn_stream_t stream) {
  int shift = 0;
  const int rc = paged_check_pages(pages, &shift);
  return rc != ATTN_OK ? rc : read_tokens(pages, nullptr, seqs, q_ptr, n_tokens, k_out, v_out, out_dtype, shift, stream);
}

}  // extern "C"
