// The 4-bit K/V cache: its format, storing tokens and reading them back.
//
// 16 neighbouring values of a head share a scale.  The scale is a byte b that
// stands for the IEEE half with bits b << 7 (5 exponent bits, 3 mantissa bits,
// no sign): the smallest one with 6 scale >= max|x|, at most 10240 (so that
// 6 * 10240 = 61440 is still an fp16 value).  A code is 4 bits, sign and
// magnitude {0, .5, 1, 1.5, 2, 3, 4, 6} (e2m1): the nearest to x / scale, ties
// to the even code.  A code times a scale has at most 6 significant bits, so
// the attention's fp16 operands hold it exactly: nothing is rounded after
// storing.  4.5 bits a value.
//
// A record holds 8 tokens of one KV head (the routed attention's group):
//   K codes [8][d/2], V codes [8][d/2] (dim 2i in the low nibble of byte i),
//   K scales [8][d/16], V scales [8][d/16]                  = 9 d bytes,
// one contiguous span whose size is a multiple of 16 bytes, so one bulk copy
// fetches a group's K and V.  A page is [KV head][page_tokens / 8] records: a
// head's tokens of a page are contiguous too.
#pragma once
#include <cuda_fp16.h>
#include "common.cuh"
#include "tc.cuh"

namespace hga {

constexpr int kQ4MaxScale = 226;            // the byte of 10240
constexpr float kQ4MaxValue = 61440.0f;

__host__ __device__ constexpr int q4_record_bytes(int d) { return 9 * d; }

struct Q4Cache {
  char* base;                // the plane's pages
  int64_t page_bytes;
  const int32_t* table;      // [n_rows][row_pages]
  const int32_t* len;        // [n_rows]
  int n_pages, n_rows, row_pages, page_recs, page_tokens, Hkv;
  uint32_t page_recs_inv;    // 2^32 / page_recs, rounded up (page_recs = 1: 2^32 - 1)
};

struct Q4BatchArgs {
  const int32_t* rows;       // [n_seq] table rows, < 0 = inactive
  const int32_t* off;        // [n_seq + 1], null: one token each
  int n_seq;
};

__device__ __forceinline__ bool q4_has_tokens(const Q4BatchArgs& b, int s) {
  return !b.off || b.off[s + 1] > b.off[s];
}

// Where a token of the batch lives: its table row and position; false where
// it belongs to no sequence (behind the last one, or an inactive one).
__device__ __forceinline__ bool q4_locate(const Q4Cache& c, const Q4BatchArgs& b, int64_t tok,
                                          int* row, int* pos) {
  int s, n, j;
  if (b.off) {
    // last sequence whose start is at or before the token
    int lo = 0, hi = b.n_seq;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (b.off[mid + 1] <= tok) lo = mid + 1;
      else hi = mid;
    }
    s = lo;
    if (s >= b.n_seq) return false;
    const int o = b.off[s];
    if (tok < o) return false;
    n = b.off[s + 1] - o;
    j = (int)(tok - o);
  } else {
    if (tok >= b.n_seq) return false;
    s = (int)tok;
    n = 1;
    j = 0;
  }
  const int r = b.rows[s];
  if (r < 0) return false;
  if (r >= c.n_rows) {
    report(HGA_ERR_DEVICE_CHECK);
    return false;
  }
  *row = r;
  *pos = c.len[r] - n + j;
  return true;
}

// The record of (row, position, head), or null (reported) where the page table
// names none.
__device__ __forceinline__ char* q4_record(const Q4Cache& c, int row, int pos, int h, int rec) {
  if (pos < 0 || pos >= (int64_t)c.row_pages * c.page_tokens) {
    report(HGA_ERR_DEVICE_CHECK);
    return nullptr;
  }
  const int col = pos / c.page_tokens;
  const int pg = c.table[(int64_t)row * c.row_pages + col];
  if (pg < 0 || pg >= c.n_pages) {
    report(HGA_ERR_DEVICE_CHECK);
    return nullptr;
  }
  const int in = (pos - col * c.page_tokens) >> 3;
  return c.base + pg * c.page_bytes + ((int64_t)h * c.page_recs + in) * rec;
}

__device__ __forceinline__ float q4_scale(int b) {
  return __half2float(__ushort_as_half((unsigned short)(b << 7)));
}

// Smallest scale byte with 6 scale >= m, m in [0, 61440].  A byte is a half's
// upper bits, so it is m / 6 rounded up, twice.  bf16: m has 8 bits, so m / 6 is a
// scale's value or at least 2^-10 of itself away from one, and the product may
// be too small by 2^-20 (checked for every m).  fp32: the guess is compared.
template <typename T>
__device__ __forceinline__ int q4_scale_byte(float m) {
  constexpr float kSixth = sizeof(T) == 2 ? 0.16666667f * (1.f - 0x1p-20f) : 0.16666667f;
  int b = min((__half_as_ushort(__float2half_ru(m * kSixth)) + 127) >> 7, kQ4MaxScale);
  if constexpr (sizeof(T) == 4) {
    while (b > 0 && 6.0f * q4_scale(b - 1) >= m) --b;
    while (b < kQ4MaxScale && 6.0f * q4_scale(b) < m) ++b;
  }
  return b;
}

// Codes of eight values already divided by their scale (the first one in the
// low nibble).
__device__ __forceinline__ uint32_t q4_code8(const float* f) {
  uint32_t r;
  asm("{\n .reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(r)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return r;
}

// Eight values (half of a scale's 16; the thread beside has the others, lane
// ^ 1) -> four code bytes and the scale byte.  Called by whole warps; a thread
// that is not live reads nothing.
//
// The maximum is taken over the magnitudes' bits, where infinities and NaN come
// last.  x / s has to be exact where it is a tie of the code grid.  fp32: a
// correctly rounded quotient is enough, x has 24 bits and s 4, so a quotient
// that is no tie lies more than half an ulp of the tie away from it.  bf16: a
// product with 1/s (together good to 2^-21 of at most 7) whose error is taken off
// by rounding to a multiple of 2^-12: |x / s - tie| is 0 or at least 2^-10.
template <typename T>
__device__ __forceinline__ uint32_t q4_encode8(const T* src, bool live, int* scale, bool* bad) {
  float f[8];
  uint32_t top = 0;
  if constexpr (sizeof(T) == 2) {
    const uint4 raw = live ? *reinterpret_cast<const uint4*>(src) : make_uint4(0, 0, 0, 0);
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      top = __vmaxu2(top, w[i] & 0x7fff7fffu);
    }
    top = max(top << 16, top & 0xffff0000u);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 r = live ? reinterpret_cast<const float4*>(src)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
      f[4 * i] = r.x; f[4 * i + 1] = r.y; f[4 * i + 2] = r.z; f[4 * i + 3] = r.w;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(f[i]) & 0x7fffffffu);
  }
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  float m = __uint_as_float(top);
  const bool over = !(m <= kQ4MaxValue);
  if (__any_sync(0xffffffffu, over)) {
    *bad |= over;
    m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      f[i] = f[i] == f[i] ? fminf(fmaxf(f[i], -kQ4MaxValue), kQ4MaxValue) : 0.f;
      m = fmaxf(m, fabsf(f[i]));
    }
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  }
  const int b = q4_scale_byte<T>(m);
  *scale = b;
  const float s = b == 0 ? 1.f : q4_scale(b);   // 0: every value is 0
  if constexpr (sizeof(T) == 2) {
    const float inv = __fdividef(1.0f, s);
    const uint64_t inv2 = tc::pk2(inv, inv), up = tc::pk2(2048.f, 2048.f), down = tc::pk2(-2048.f, -2048.f);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      tc::unpk2(tc::fadd2(tc::ffma2(tc::pk2(f[2 * i], f[2 * i + 1]), inv2, up), down), f[2 * i],
                f[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __fdiv_rn(f[i], s);
  }
  return q4_code8(f);
}

// Eight codes (one word) -> four pairs of fp16.
__device__ __forceinline__ void q4_unpack8(uint32_t w, uint32_t* h) {
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t q4_mul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// ---------------------------------------------------------------- append

constexpr int kQ4Threads = 256;
constexpr int kQ4BlockTok = 32;             // most tokens of a block

struct Q4IoArgs {
  Q4Cache c;
  Q4BatchArgs b;
  const void *k, *v;         // append: the tokens; read: where they go
  int64_t k_tok, k_head, v_tok, v_head;   // strides in elements
  int64_t n_tok;
  int toks;                  // tokens of a block
  int D;
};

template <typename T>
__device__ __forceinline__ void q4_load16(const T* p, float* f) {
  if constexpr (sizeof(T) == 2) {
    const uint4 r[2] = {reinterpret_cast<const uint4*>(p)[0], reinterpret_cast<const uint4*>(p)[1]};
    const uint32_t w[8] = {r[0].x, r[0].y, r[0].z, r[0].w, r[1].x, r[1].y, r[1].z, r[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 r = reinterpret_cast<const float4*>(p)[i];
      f[4 * i] = r.x; f[4 * i + 1] = r.y; f[4 * i + 2] = r.z; f[4 * i + 3] = r.w;
    }
  }
}

// A block's tokens: where their records are, looked up once by one thread each
// (a thread of the loop below handles 16 values, for which the search of the
// sequence and the page would cost more than the values).  off < 0: no token.
struct Q4BlockTokens {
  int64_t off[kQ4BlockTok];  // the record of KV head 0, in bytes from the plane's first page
  int r[kQ4BlockTok];        // row within the record
};
__device__ __forceinline__ void q4_block_tokens(const Q4IoArgs& a, int64_t t0, int nt,
                                                Q4BlockTokens* s) {
  for (int i = threadIdx.x; i < nt; i += kQ4Threads) {
    int row, pos;
    char* rec = nullptr;
    if (q4_locate(a.c, a.b, t0 + i, &row, &pos)) rec = q4_record(a.c, row, pos, 0, q4_record_bytes(a.D));
    s->off[i] = rec ? rec - a.c.base : -1;
    s->r[i] = pos & 7;
  }
  __syncthreads();
}

// One thread per 8 values of K and the same 8 of V, so that a warp's 16-byte
// loads are contiguous; the two threads of a scale exchange their maxima.
// It reads 4 d and writes 9 d / 8 bytes per token and head.  Bound: a block's one
// chain (places of its tokens, a barrier, loads, encoding) beside the issue slots
// (65 % taken, ALU 57 %, HBM 40 %): 32768 tokens, 8 heads of 128, bf16: 43 us.
template <typename T>
__global__ void __launch_bounds__(kQ4Threads) q4_append_kernel(const Q4IoArgs a) {
  __shared__ Q4BlockTokens tok;
  griddep_wait();
  const int64_t t0 = (int64_t)blockIdx.x * a.toks;
  const int nt = (int)min((int64_t)a.toks, a.n_tok - t0);
  q4_block_tokens(a, t0, nt, &tok);
  const int half = a.D >> 1, log_nv = a.D == 128 ? 4 : 3, nb = a.D >> 4;
  const int hb = a.c.Hkv << log_nv;                 // threads of a token
  bool bad = false;
  // a row named by two sequences that have tokens would be written twice:
  // reported.  A block compares its sequences with those before them, a thread
  // every 256th (the call for 1000 generated tokens takes 5.1 us; with a thread a
  // sequence, which has all before it to read, it took 43).
  for (int i = blockIdx.x; i < a.b.n_seq; i += gridDim.x) {
    const int row = a.b.rows[i];
    if (row < 0 || !q4_has_tokens(a.b, i)) continue;
    for (int j = threadIdx.x; j < i; j += kQ4Threads)
      if (a.b.rows[j] == row && q4_has_tokens(a.b, j)) bad = true;
  }
  const int dt = kQ4Threads / hb, dx = kQ4Threads % hb;
  int t = threadIdx.x / hb, x = threadIdx.x % hb;
  const int turns = (nt * hb + kQ4Threads - 1) / kQ4Threads;   // whole warps: the maxima are exchanged
  for (int i = 0; i < turns; ++i) {
    const bool live = t < nt && tok.off[t] >= 0;
    const int tt = live ? t : 0;
    const int h = x >> log_nv, v8 = x & ((1 << log_nv) - 1), r = tok.r[tt];
    char* rec = a.c.base + tok.off[tt] + (int64_t)h * a.c.page_recs * q4_record_bytes(a.D);
    int ks, vs;
    const uint32_t kc = q4_encode8(
        static_cast<const T*>(a.k) + (t0 + tt) * a.k_tok + h * a.k_head + v8 * 8, live, &ks, &bad);
    const uint32_t vc = q4_encode8(
        static_cast<const T*>(a.v) + (t0 + tt) * a.v_tok + h * a.v_head + v8 * 8, live, &vs, &bad);
    if (live) {
      *reinterpret_cast<uint32_t*>(rec + r * half + v8 * 4) = kc;
      *reinterpret_cast<uint32_t*>(rec + 8 * half + r * half + v8 * 4) = vc;
      // the even thread has K's scale, the odd one V's
      const int sb = r * nb + (v8 >> 1);
      if (v8 & 1) rec[16 * half + 8 * nb + sb] = (char)vs;
      else rec[16 * half + sb] = (char)ks;
    }
    t += dt + (x + dx >= hb);
    x = x + dx >= hb ? x + dx - hb : x + dx;
  }
  if (bad) report(HGA_ERR_DEVICE_CHECK);
  griddep_launch();
}

// ---------------------------------------------------------------- read

// 8 codes -> 16 bytes of fp16 or bf16 or 32 of fp32, exact.
template <typename T>
__device__ __forceinline__ void q4_decode8(uint32_t codes, int scale, T* out) {
  const uint32_t s2 = (uint32_t)scale * 0x00800080u;
  uint32_t h[4];
  q4_unpack8(codes, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = q4_mul2(h[i], s2);
  if constexpr (std::is_same<T, __half>::value) {
    *reinterpret_cast<uint4*>(out) = make_uint4(h[0], h[1], h[2], h[3]);
  } else {
    float2 f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __half22float2(*reinterpret_cast<__half2*>(&h[i]));
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = tc::pack_bf162(f[i].x, f[i].y);
      *reinterpret_cast<uint4*>(out) = make_uint4(h[0], h[1], h[2], h[3]);
    } else {
      reinterpret_cast<float4*>(out)[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
      reinterpret_cast<float4*>(out)[1] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
    }
  }
}

// The batch's tokens back as the values their codes stand for, in TK and TV.
// One thread per 8 values of K and of V: contiguous 16-byte stores.  Bound: the
// latency of the look-up and the small loads (the largest stall; issue slots 55 %,
// HBM 39 %): 32768 tokens, 8 heads of 128: 36 us.
template <typename TK, typename TV>
__global__ void __launch_bounds__(kQ4Threads) q4_read_kernel(const Q4IoArgs a) {
  __shared__ Q4BlockTokens tok;
  griddep_wait();
  const int64_t t0 = (int64_t)blockIdx.x * a.toks;
  const int nt = (int)min((int64_t)a.toks, a.n_tok - t0);
  q4_block_tokens(a, t0, nt, &tok);
  const int half = a.D >> 1, log_nv = a.D == 128 ? 4 : 3, nb = a.D >> 4;
  const int hb = a.c.Hkv << log_nv;
  const int dt = kQ4Threads / hb, dx = kQ4Threads % hb;
  int t = threadIdx.x / hb, x = threadIdx.x % hb;
#pragma unroll 2
  for (; t < nt; t += dt + (x + dx >= hb), x = x + dx >= hb ? x + dx - hb : x + dx) {
    if (tok.off[t] < 0) continue;
    const int h = x >> log_nv, v8 = x & ((1 << log_nv) - 1), r = tok.r[t];
    const char* rec = a.c.base + tok.off[t] + (int64_t)h * a.c.page_recs * q4_record_bytes(a.D);
    const uint32_t kc = *reinterpret_cast<const uint32_t*>(rec + r * half + v8 * 4);
    const uint32_t vc = *reinterpret_cast<const uint32_t*>(rec + 8 * half + r * half + v8 * 4);
    const int sb = 16 * half + r * nb + (v8 >> 1);
    const int ks = (unsigned char)rec[sb], vs = (unsigned char)rec[sb + 8 * nb];
    q4_decode8(kc, ks, (TK*)a.k + (t0 + t) * a.k_tok + h * a.k_head + v8 * 8);
    q4_decode8(vc, vs, (TV*)a.v + (t0 + t) * a.v_tok + h * a.v_head + v8 * 8);
  }
  griddep_launch();
}

}  // namespace hga
