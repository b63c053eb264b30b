// The quantised paged cache: writing new tokens and reading tokens back.
//
// Append, per row (token, head) of D values x of K and of V:
//   amax = max |x|,  scale = fl32(amax / top),  code = round(x * top / amax),
// top = 127 and round to the nearest integer for INT8, top = 448 and round to
// the nearest code for E4M3; ties to even, the quotient taken as exact.  A row
// of zeros has scale 0 and codes 0; a row with an infinity or a NaN has scale
// NaN and codes 0, so that it reads back as NaN and spoils what attends to it.
//
// The quotient: t = fl32(x * fl32(top / amax)) is within 2^-22 of
// q = x * top / amax (relative).  With 8 significant bits in x and in amax, a q
// that is not half-way between two codes is at least 2^-16 away from half-way
// (INT8: |254 xm - a (2k+1) 2^s| >= 1 over a (2k+1) 2^s <= 2^16; E4M3: the
// denominator is at most 2^13).  Rounding t to 18 bits therefore gives half-way
// where q is half-way and stays on q's side where it is not, and the code is
// that of the exact quotient without a division per element.
//
// Read: bf16(fl32(code * scale)).
//
// Both are bound by HBM: 3 bytes per element and 4 per row.
#include "cache_common.cuh"

namespace sage {
namespace {

constexpr int kCacheThreads = 256;

// 16-bit codes -> two floats.
__device__ __forceinline__ float2 e4m3x2_to_f32(uint16_t w) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(w));
  float2 r;
  asm("{.reg .b16 lo, hi; mov.b32 {lo, hi}, %2; cvt.f32.f16 %0, lo; cvt.f32.f16 %1, hi;}" : "=f"(r.x), "=f"(r.y) : "r"(h));
  return r;
}

// t to 18 significant bits, nearest (half-way cases upwards in magnitude: no
// half-way point of a code needs more than 9 bits, so they do not matter).
__device__ __forceinline__ float snap18(float t) { return __uint_as_float((__float_as_uint(t) + 0x20u) & ~0x3Fu); }

// Codes of 8 values (two words) with the row's factors.
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float pre, float inv, bool int8) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float t[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) t[e] = snap18(__fmul_rn(__fmul_rn(x[4 * i + e], pre), inv));
    if (int8)
      w[i] = (__float2int_rn(t[0]) & 0xFF) | (__float2int_rn(t[1]) & 0xFF) << 8 | (__float2int_rn(t[2]) & 0xFF) << 16 |
             (uint32_t)__float2int_rn(t[3]) << 24;
    else
      w[i] = (uint32_t)e4m3x2(t[0], t[1]) | (uint32_t)e4m3x2(t[2], t[3]) << 16;
  }
  return make_uint2(w[0], w[1]);
}

// D/8 threads per row, 8 values each; grid (rows of a sequence, B).
template <int D>
__global__ void __launch_bounds__(kCacheThreads) cache_append_kernel(const AppendArgs a) {
  constexpr int LPR = D / 8;
  const int b = blockIdx.y;
  const int64_t r = (int64_t)blockIdx.x * (kCacheThreads / LPR) + threadIdx.x / LPR;
  const int64_t n = r / a.c.H;
  const int h = (int)(r % a.c.H), lane = threadIdx.x % LPR;
  int count = a.N;
  if (a.count) {
    count = a.count[b];
    if ((count < 0 || count > a.N) && r == 0 && lane == 0) flag_bad(a.c.status, kWhereAppend);
    count = min(count, a.N);
  }
  const bool on = n < count;
  int64_t row = -1;
  if (on) {
    row = cache_row(a.c, b, h, (a.start ? a.start[b] : 0) + n);
    if (row < 0 && lane == 0) flag_bad(a.c.status, kWhereAppend);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint4 u = make_uint4(0, 0, 0, 0);
    if (row >= 0) u = *reinterpret_cast<const uint4*>(a.x[i] + b * a.sb[i] + n * a.sn[i] + h * a.sh[i] + 8 * lane);
    const uint32_t xw[4] = {u.x, u.y, u.z, u.w};
    // the magnitude's bits order like its value, infinities and NaN above all
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) top = max(top, max(xw[e] & 0x7FFFu, (xw[e] >> 16) & 0x7FFFu));
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (row < 0) continue;
    const bool int8 = a.c.format[i] == SAGE_CACHE_INT8;
    const float lim = int8 ? 127.0f : 448.0f;
    const bool bad = top >= 0x7F80u, none = bad || top == 0;
    const float amax = __uint_as_float(top << 16);
    // a tiny amax is scaled up first (exactly), so that top / amax stays finite
    const float pre = amax < 0x1p-100f ? 0x1p60f : 1.0f;
    const float inv = none ? 0.0f : __fdiv_rn(lim, amax * pre);
    float x[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = bad ? 0.0f : __uint_as_float(xw[e] << 16);
      x[2 * e + 1] = bad ? 0.0f : __uint_as_float(xw[e] & 0xFFFF0000u);
    }
    *reinterpret_cast<uint2*>(a.c.codes[i] + row * D + 8 * lane) = codes8(x, pre, inv, int8);
    if (lane == 0) a.c.scale[i][row] = bad ? __uint_as_float(0x7FC00000u) : __fdiv_rn(amax, lim);
  }
}

template <int D>
__global__ void __launch_bounds__(kCacheThreads) cache_read_kernel(const ReadArgs a) {
  constexpr int LPR = D / 8;
  const int b = blockIdx.y;
  const int64_t r = (int64_t)blockIdx.x * (kCacheThreads / LPR) + threadIdx.x / LPR;
  const int64_t n = r / a.c.H;
  const int h = (int)(r % a.c.H), lane = threadIdx.x % LPR;
  int count = a.N;
  if (a.count) {
    count = a.count[b];
    if ((count < 0 || count > a.N) && r == 0 && lane == 0) flag_bad(a.c.status, kWhereRead);
    count = min(count, a.N);
  }
  if (n >= count) return;
  const int64_t row = cache_row(a.c, b, h, (a.start ? a.start[b] : 0) + n);
  if (row < 0) {
    if (lane == 0) flag_bad(a.c.status, kWhereRead);
    return;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (!a.y[i]) continue;
    const uint2 w = *reinterpret_cast<const uint2*>(a.c.codes[i] + row * D + 8 * lane);
    const float scale = a.c.scale[i][row];
    const uint32_t cw[2] = {w.x, w.y};
    uint32_t yw[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t two = cw[e >> 1] >> (16 * (e & 1));
      float2 f;
      if (a.c.format[i] == SAGE_CACHE_INT8) f = make_float2((float)(int8_t)(two & 0xFF), (float)(int8_t)((two >> 8) & 0xFF));
      else f = e4m3x2_to_f32((uint16_t)two);
      yw[e] = (uint32_t)f32_to_bf16_rn(__fmul_rn(f.x, scale)) | (uint32_t)f32_to_bf16_rn(__fmul_rn(f.y, scale)) << 16;
    }
    *reinterpret_cast<uint4*>(a.y[i] + b * a.yb[i] + n * a.yn[i] + h * a.yh[i] + 8 * lane) =
        make_uint4(yw[0], yw[1], yw[2], yw[3]);
  }
}

dim3 rows_grid(int64_t rows, int per_block, int B) { return dim3((unsigned)((rows + per_block - 1) / per_block), B); }

}  // namespace

int launch_cache_append(const AppendArgs& a, cudaStream_t s) {
  const int per = kCacheThreads / (a.c.D / 8);
  const dim3 grid = rows_grid((int64_t)a.N * a.c.H, per, a.B);
  if (a.c.D == 128) cache_append_kernel<128><<<grid, kCacheThreads, 0, s>>>(a);
  else cache_append_kernel<64><<<grid, kCacheThreads, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? SAGE_OK : SAGE_ERR_CUDA;
}

int launch_cache_read(const ReadArgs& a, cudaStream_t s) {
  const int per = kCacheThreads / (a.c.D / 8);
  const dim3 grid = rows_grid((int64_t)a.N * a.c.H, per, a.B);
  if (a.c.D == 128) cache_read_kernel<128><<<grid, kCacheThreads, 0, s>>>(a);
  else cache_read_kernel<64><<<grid, kCacheThreads, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? SAGE_OK : SAGE_ERR_CUDA;
}

}  // namespace sage
