// The quantised paged cache: writing new tokens and reading tokens back.
//
// Append, per row (token, head) of D values x of K and of V:
//   amax = max |x|,  scale = fl32(amax / top),  code = round(x * top / amax),
// top = 127 and round to the nearest integer for INT8, top = 448 and round to
// the nearest code for E4M3; ties to even, the quotient taken as exact.  A row
// of zeros has scale 0 and codes 0; a row with an infinity or a NaN has scale
// NaN and codes 0, so that it reads back as NaN and spoils what attends to it.
//
// The quotient: inv + rest is top / amax to 2^-45 (relative) for amax below 2^112, and to less and less above,
// where rest is subnormal: 2^-29 at the largest BF16 values.  So t = fma(x, inv, x * rest) is q = x * top / amax to less
// than half an FP32 step before its one rounding: a q that is an FP32 value, as every half-way point between two codes
// is, is t itself, and any other t is within 2^-23 of q.  With 8
// significant bits in x and in amax, a q that is not half-way between two codes
// is at least 2^-16 away from half-way (INT8: |254 xm - a (2k+1) 2^s| >= 1 over
// a (2k+1) 2^s <= 2^16; E4M3: the denominator is at most 2^13), so t is half-way
// exactly where q is and on q's side of it elsewhere: the code is that of the exact
// quotient, without a division per element.
//
// Read: bf16(fl32(code * scale)).
//
// Both are bound by HBM: 3 bytes per element and 4 per row.  Four threads share
// a row, so that its lookups and scale cost little per element, and eight
// neighbouring tokens of a head lie in one warp: their scales are one 32-byte
// sector and their codes are contiguous in the page.  Measured on B200: append of
// 16 prompts of 37..8192 tokens, 8 heads of 128, 80 to 90 us by the box (68 at the copy rate; with a thread per row and a
// division per element 168); read of 4 contexts of 1000..37810, 107 us (102; 162 with a thread per row).
#include "cache_codes.cuh"
#include "cache_common.cuh"

namespace sage {
namespace {

using cattn::add2;
using cattn::fma2;
using cattn::mul2;
using cattn::pair;
using cattn::unpair;

constexpr int kCacheThreads = 256;

constexpr int kLanes = 4;                          // threads of a row
constexpr int kPerBlock = kCacheThreads / kLanes;  // rows of a block at a time

__device__ __forceinline__ uint32_t pack_bf16(float2 v) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(v.y), "f"(v.x));
  return r;
}

// Token n and head h of row r of a sequence: groups of 2^gs tokens, head by head.
struct TokenHead {
  int64_t n;
  int h;
};
__device__ __forceinline__ TokenHead token_head(int64_t r, int H, int gs) {
  const int64_t g = r >> gs;
  const int64_t q = g < 0x80000000ll ? (unsigned)g / (unsigned)H : g / H;
  return {(q << gs) + (r & ((1 << gs) - 1)), (int)(g - q * H)};
}

// Codes of 8 BF16 values.
__device__ __forceinline__ uint2 codes8(uint4 u, uint64_t inv, uint64_t rest, bool int8) {
  const uint32_t xw[4] = {u.x, u.y, u.z, u.w};
  uint32_t h[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint64_t x = pair(__uint_as_float(xw[e] << 16), __uint_as_float(xw[e] & 0xFFFF0000u));
    uint64_t t = fma2(x, inv, mul2(x, rest));
    if (int8) {
      // 1.5 * 2^23 + t rounds to an integer, ties to even; its low byte is the code
      t = add2(t, pair(12582912.0f, 12582912.0f));
      const float2 f = unpair(t);
      h[e] = __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x0040);
    } else {
      const float2 f = unpair(t);
      h[e] = e4m3x2(f.x, f.y);
    }
  }
  return make_uint2(__byte_perm(h[0], h[1], 0x5410), __byte_perm(h[2], h[3], 0x5410));
}

// grid (rows of a sequence, B); ROWS rows per thread, their loads issued together.
template <int D, int ROWS>
__global__ void __launch_bounds__(kCacheThreads) cache_append_kernel(const AppendArgs a, int gs) {
  constexpr int CH = D / (8 * kLanes);  // chunks of 8 values of a thread: 8 (lane + 4 j) ..
  const int b = blockIdx.y, lane = threadIdx.x % kLanes;
  const int64_t r0 = (int64_t)blockIdx.x * (kPerBlock * ROWS) + threadIdx.x / kLanes;
  begin_dependent();
  int count = a.N;
  if (a.count) {
    count = a.count[b];
    if ((count < 0 || count > a.N) && r0 == 0 && lane == 0) flag_bad(a.c.status, kWhereAppend);
    count = max(min(count, a.N), 0);
  }
  const int64_t rows = (((int64_t)count + (1 << gs) - 1) >> gs << gs) * a.c.H;
  if ((int64_t)blockIdx.x * (kPerBlock * ROWS) >= rows) return;
  const int64_t start = a.start ? a.start[b] : 0;
  uint4 u[2][ROWS][CH];
  int64_t row[ROWS];
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
    const TokenHead t = token_head(r0 + k * kPerBlock, a.c.H, gs);
    const bool on = t.n < count;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        u[i][k][j] = make_uint4(0, 0, 0, 0);
        if (on)
          u[i][k][j] = *reinterpret_cast<const uint4*>(a.x[i] + b * a.sb[i] + t.n * a.sn[i] + t.h * a.sh[i] +
                                                       8 * (lane + kLanes * j));
      }
    row[k] = on ? cache_row(a.c, b, t.h, start + t.n) : -1;
    if (on && row[k] < 0 && lane == 0) flag_bad(a.c.status, kWhereAppend);
  }
#pragma unroll
  for (int k = 0; k < ROWS; ++k)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool int8 = a.c.format[i] == SAGE_CACHE_INT8;
      const float lim = int8 ? 127.0f : 448.0f;
      // the magnitude's bits order like its value, infinities and NaN above all
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        const uint4 v = u[i][k][j];
        top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                     __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
      }
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
      top = max(top & 0xFFFFu, top >> 16);
      if (row[k] < 0) continue;
      uint8_t* codes = a.c.codes[i] + row[k] * D + 8 * lane;
      float scale;
      if (top == 0 || top >= 0x7F80u) {
        scale = top == 0 ? 0.0f : __uint_as_float(0x7FC00000u);
#pragma unroll
        for (int j = 0; j < CH; ++j) *reinterpret_cast<uint2*>(codes + 8 * kLanes * j) = make_uint2(0, 0);
      } else {
        const float amax = __uint_as_float(top << 16);
        scale = __fdiv_rn(amax, lim);
        // 2^60 / amax and x 2^-60 where lim / amax would overflow: both exact
        const float pre = top < 0x1000u ? 0x1p60f : 1.0f;  // amax below 2^-95
        const float up = amax * pre, inv = __fdiv_rn(lim, up), rest = __fdiv_rn(fmaf(-inv, up, lim), up);
#pragma unroll
        for (int j = 0; j < CH; ++j) {
          uint4 v = u[i][k][j];
          if (top < 0x1000u) {
            uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = pack_bf16(make_float2(__uint_as_float(w[e] << 16) * pre, __uint_as_float(w[e] & 0xFFFF0000u) * pre));
          }
          *reinterpret_cast<uint2*>(codes + 8 * kLanes * j) = codes8(v, pair(inv, inv), pair(rest, rest), int8);
        }
      }
      if (lane == 0) a.c.scale[i][row[k]] = scale;
    }
}

// Four codes -> four BF16 values.
__device__ __forceinline__ uint2 values4(uint32_t w, uint64_t scale, bool int8) {
  uint64_t lo, hi;
  if (int8) {
    // 0x4B000000 | (code + 128) is 2^23 + 128 + code
    const uint32_t u = w ^ 0x80808080u, k = 0x4B000000u;
    const uint64_t bias = pair(-8388736.0f, -8388736.0f);
    lo = add2(pair(__uint_as_float(__byte_perm(u, k, 0x7540)), __uint_as_float(__byte_perm(u, k, 0x7541))), bias);
    hi = add2(pair(__uint_as_float(__byte_perm(u, k, 0x7542)), __uint_as_float(__byte_perm(u, k, 0x7543))), bias);
  } else {
    uint32_t a, b;
    asm("{.reg .b16 lo, hi; mov.b32 {lo, hi}, %2; cvt.rn.f16x2.e4m3x2 %0, lo; cvt.rn.f16x2.e4m3x2 %1, hi;}"
        : "=r"(a), "=r"(b)
        : "r"(w));
    float f[4];
    asm("{.reg .b16 lo, hi; mov.b32 {lo, hi}, %2; cvt.f32.f16 %0, lo; cvt.f32.f16 %1, hi;}" : "=f"(f[0]), "=f"(f[1]) : "r"(a));
    asm("{.reg .b16 lo, hi; mov.b32 {lo, hi}, %2; cvt.f32.f16 %0, lo; cvt.f32.f16 %1, hi;}" : "=f"(f[2]), "=f"(f[3]) : "r"(b));
    lo = pair(f[0], f[1]);
    hi = pair(f[2], f[3]);
  }
  return make_uint2(pack_bf16(unpair(mul2(lo, scale))), pack_bf16(unpair(mul2(hi, scale))));
}

template <int D, int ROWS>
__global__ void __launch_bounds__(kCacheThreads) cache_read_kernel(const ReadArgs a, int gs) {
  constexpr int CH = D / (8 * kLanes);
  const int b = blockIdx.y, lane = threadIdx.x % kLanes;
  const int64_t r0 = (int64_t)blockIdx.x * (kPerBlock * ROWS) + threadIdx.x / kLanes;
  begin_dependent();
  int count = a.N;
  if (a.count) {
    count = a.count[b];
    if ((count < 0 || count > a.N) && r0 == 0 && lane == 0) flag_bad(a.c.status, kWhereRead);
    count = max(min(count, a.N), 0);
  }
  const int64_t rows = (((int64_t)count + (1 << gs) - 1) >> gs << gs) * a.c.H;
  if (r0 >= rows) return;
  const int64_t start = a.start ? a.start[b] : 0;
  uint2 w[2][ROWS][CH];
  float scale[2][ROWS];
  int64_t row[ROWS];
  TokenHead t[ROWS];
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
    t[k] = token_head(r0 + k * kPerBlock, a.c.H, gs);
    row[k] = -1;
    if (t[k].n < count) {
      row[k] = cache_row(a.c, b, t[k].h, start + t[k].n);
      if (row[k] < 0 && lane == 0) flag_bad(a.c.status, kWhereRead);
    }
  }
#pragma unroll
  for (int k = 0; k < ROWS; ++k)
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (row[k] >= 0 && a.y[i]) {
#pragma unroll
        for (int j = 0; j < CH; ++j)
          w[i][k][j] = *reinterpret_cast<const uint2*>(a.c.codes[i] + row[k] * D + 8 * (lane + kLanes * j));
        scale[i][k] = a.c.scale[i][row[k]];
      }
#pragma unroll
  for (int k = 0; k < ROWS; ++k)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (row[k] < 0 || !a.y[i]) continue;
      const bool int8 = a.c.format[i] == SAGE_CACHE_INT8;
      const uint64_t s = pair(scale[i][k], scale[i][k]);
      uint16_t* y = a.y[i] + b * a.yb[i] + t[k].n * a.yn[i] + t[k].h * a.yh[i] + 8 * lane;
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        const uint2 lo = values4(w[i][k][j].x, s, int8), hi = values4(w[i][k][j].y, s, int8);
        *reinterpret_cast<uint4*>(y + 8 * kLanes * j) = make_uint4(lo.x, lo.y, hi.x, hi.y);
      }
    }
}

// Tokens of a group of rows: eight, or one where there are not as many (a
// decode step's rows then fill the blocks).
int group_shift(int N) { return N >= 8 ? 3 : 0; }
dim3 rows_grid(int N, int H, int per_block, int B) {
  const int gs = group_shift(N);
  const int64_t rows = (((int64_t)N + (1 << gs) - 1) >> gs << gs) * H;
  return dim3((unsigned)((rows + per_block - 1) / per_block), B);
}

}  // namespace

int launch_cache_append(const AppendArgs& a, cudaStream_t s) {
  const int gs = group_shift(a.N);
  return a.c.D == 128 ? launch_dependent(cache_append_kernel<128, 1>, rows_grid(a.N, a.c.H, kPerBlock, a.B),
                                         kCacheThreads, 0, s, a, gs)
                      : launch_dependent(cache_append_kernel<64, 2>, rows_grid(a.N, a.c.H, 2 * kPerBlock, a.B),
                                         kCacheThreads, 0, s, a, gs);
}

int launch_cache_read(const ReadArgs& a, cudaStream_t s) {
  const int gs = group_shift(a.N);
  return a.c.D == 128 ? launch_dependent(cache_read_kernel<128, 1>, rows_grid(a.N, a.c.H, kPerBlock, a.B),
                                         kCacheThreads, 0, s, a, gs)
                      : launch_dependent(cache_read_kernel<64, 2>, rows_grid(a.N, a.c.H, 2 * kPerBlock, a.B),
                                         kCacheThreads, 0, s, a, gs);
}

}  // namespace sage
