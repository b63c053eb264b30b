// Division of the cache attention's work among CTAs, and the joining of the
// parts, shared by its kernels.
//
// The work is a list of tiles of TILE keys: sequence by sequence, head by
// head, row tile by row tile (a unit: R of the count*G rows that share a head
// of the cache), tile by tile.  Every CTA takes one equal stretch of the list,
// whatever the lengths of the sequences: a unit that a stretch holds whole is
// finished there, one that is cut leaves a part (FP32 sums with their offset
// and denominator) per CTA, and the joining kernel adds the parts in list
// order.  A CTA leaves at most two parts: slot 0 for a unit that began before
// its stretch, slot 1 for one that begins in it and goes on behind it.  The
// lengths are read on the device, so a captured launch follows them.
#pragma once
#include "cache_codes.cuh"
#include "cache_common.cuh"

namespace sage {
namespace cattn {

struct Seq {
  int ctx, cnt;      // context and drafted tokens
  unsigned n;        // tiles of a unit
  unsigned rt;       // row tiles
  unsigned per;      // tiles of all its units (the launch checks that the list stays below 2^31)
};

template <int TILE, int R>
__device__ __forceinline__ Seq seq_of(const CacheAttnArgs& a, int b) {
  Seq s;
  s.ctx = max(a.context[b], 0);
  s.cnt = a.count ? min(max(a.count[b], 0), a.T) : a.T;
  const unsigned cap = (unsigned)a.c.table_pages << a.c.page_shift;
  s.n = (min((unsigned)s.ctx + (unsigned)s.cnt, cap) + TILE - 1) / TILE;
  s.rt = (s.cnt * a.G + R - 1) / R;
  s.per = a.c.H * s.rt * s.n;
  return s;
}

// A place in the list: the sequence b whose tiles begin at `base`.
struct Place {
  unsigned base;
  int b;
  Seq s;
};
// Moves on to the sequence of tile idx (idx >= base, below the list's end).
template <int TILE, int R>
__device__ __forceinline__ void go_to(const CacheAttnArgs& a, Place& p, unsigned idx) {
  while (idx >= p.base + p.s.per) {
    p.base += p.s.per;
    ++p.b;
    p.s = seq_of<TILE, R>(a, p.b);
  }
}
struct Unit {
  int h, rt;       // head of the cache, row tile
  unsigned start;  // list index of its first tile
};
__device__ __forceinline__ Unit unit_of(const Place& p, unsigned idx) {
  const unsigned u = (idx - p.base) / p.s.n;
  Unit r;
  r.rt = (int)(u % p.s.rt);
  r.h = (int)(u / p.s.rt);
  r.start = p.base + u * p.s.n;
  return r;
}

constexpr unsigned kMaxParts = 32;  // of a unit of many rows

// The stretch [s, e) of CTA `cta` of `ctas`, and the place of a tile in it.
// Every warp finds it for itself, 32 sequences at a time, which needs no
// barrier.  STEP: stretches are multiples of it.
struct Stretch {
  unsigned s, e, share, total;
  Seq own;  // sequence `lane`, for place_of (a second load would be another trip to L2)
};
template <int TILE, int R, int STEP>
__device__ __forceinline__ Stretch find_stretch(const CacheAttnArgs& a, int cta, int ctas) {
  const int lane = threadIdx.x & 31;
  Stretch t;
  t.own.ctx = t.own.cnt = 0;
  t.own.n = t.own.rt = 1;
  t.own.per = 0;
  if (lane < a.B) t.own = seq_of<TILE, R>(a, lane);
  unsigned sum = t.own.per, longest = t.own.per ? t.own.n : 0;  // a sequence without rows has no unit
  for (int b = lane + 32; b < a.B; b += 32) {
    const Seq s = seq_of<TILE, R>(a, b);
    sum += s.per;
    if (s.per) longest = max(longest, s.n);
  }
  t.total = __reduce_add_sync(0xffffffffu, sum);
  t.share = max((t.total + ctas * STEP - 1) / (ctas * STEP), 1u) * STEP;
  // Many rows: a part of a unit is up to 64 KB, and the join reads all parts of a unit in one block per 8 rows, so a
  // short list is cut into fewer.  Measured on B200 (us, one unit of 128 rows over 128 tiles of 64 keys): 128 parts
  // 56, 43 33.5, 32 28.9, 22 30.4; units of 2 tiles are cut in two as before.
  if (R >= 64) t.share = max(t.share, (__reduce_max_sync(0xffffffffu, longest) + kMaxParts - 1) / kMaxParts);
  t.s = min((unsigned)cta * t.share, t.total);
  t.e = min(t.s + t.share, t.total);
  return t;
}
template <int TILE, int R>
__device__ __forceinline__ Place place_of(const CacheAttnArgs& a, const Seq& own, unsigned idx) {
  const int lane = threadIdx.x & 31;
  Place p;
  p.base = 0;
  p.b = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    Seq s = own;
    if (b0 > 0) {
      s.per = 0;
      if (b0 + lane < a.B) s = seq_of<TILE, R>(a, b0 + lane);
    }
    unsigned incl = s.per;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned w = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += w;
    }
    const unsigned here = __ballot_sync(0xffffffffu, idx < p.base + incl);
    if (here) {  // the first lane whose sum passes idx
      const int l = __ffs(here) - 1;
      p.b = b0 + l;
      p.base += __shfl_sync(0xffffffffu, incl - s.per, l);
      p.s.ctx = __shfl_sync(0xffffffffu, s.ctx, l);
      p.s.cnt = __shfl_sync(0xffffffffu, s.cnt, l);
      p.s.n = __shfl_sync(0xffffffffu, s.n, l);
      p.s.rt = __shfl_sync(0xffffffffu, s.rt, l);
      p.s.per = __shfl_sync(0xffffffffu, s.per, l);
      return p;
    }
    p.base += __shfl_sync(0xffffffffu, incl, 31);
  }
  return p;  // not reached for idx below the list's end
}

// The longest list that the arguments allow, in tiles; it has to stay below 2^31.
template <int TILE, int R>
inline double longest_list(const CacheAttnArgs& a) {
  const double n = (((double)a.c.table_pages * (1 << a.c.page_shift)) + TILE - 1) / TILE;
  return n * a.B * a.c.H * ((a.T * a.G + R - 1) / R);
}
template <int TILE, int R>
inline bool list_fits(const CacheAttnArgs& a) { return longest_list<TILE, R>(a) < 2147483648.0; }

// begin_dependent, also for codes that a kernel before wrote by ordinary stores and TMA reads.
__device__ __forceinline__ void begin_dependent_tma() {
  begin_dependent();
  asm volatile("fence.proxy.async;" ::: "memory");
}

constexpr int kMaxCtas = 148;  // one per SM
constexpr int kMaxRows = 128;  // of a unit
constexpr size_t kPartBytes = (size_t)2 * kMaxCtas * (kMaxRows * 128 + 2 * kMaxRows) * sizeof(float);

// What the join needs of the unit that begins in a CTA's stretch and goes on behind it; parts 0: there is none.  The main
// kernel leaves one for each CTA behind its parts in the workspace: what the lengths were is known to it alone, since the join
// starts before it may read what was written in front of the main kernel.
struct alignas(16) CutUnit {
  int parts, b, h, row0, rows;
};
constexpr size_t kCutBytes = kMaxCtas * sizeof(CutUnit);
static_assert(kPartBytes % alignof(CutUnit) == 0, "the records lie behind the parts");
__device__ __forceinline__ CutUnit* cut_unit(const CacheAttnArgs& a, int cta) {
  return reinterpret_cast<CutUnit*>(static_cast<char*>(a.workspace) + kPartBytes) + cta;
}

// Parts in the workspace: [2 * CTA + slot] of R x D sums, R offsets, R denominators.
template <int R, int D>
__device__ __forceinline__ float* part_of(const CacheAttnArgs& a, int cta, int slot) {
  return static_cast<float*>(a.workspace) + (size_t)(2 * cta + slot) * (R * D + 2 * R);
}

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2f(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A finished row of the output, and four columns of one.
struct OutRow {
  uint16_t* p;
  __device__ __forceinline__ OutRow(const CacheAttnArgs& a, int b, int h, int row)
      : p(a.out + b * a.ob + (row / a.G) * a.on + (h * a.G + row % a.G) * a.oh) {}
};
__device__ __forceinline__ void store_out(const CacheAttnArgs& a, int b, int h, int row, int col, float4 o, float inv) {
  const OutRow to(a, b, h, row);
  *reinterpret_cast<uint2*>(to.p + col) = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
}
// 1 / l and the row's lse; a row that saw nothing has l = 0.
__device__ __forceinline__ float row_inverse(float l) { return l == 0.0f ? 0.0f : __frcp_rn(l); }
__device__ __forceinline__ void store_lse(const CacheAttnArgs& a, int b, int h, int row, float c, float l) {
  if (!a.lse) return;
  const int t = row / a.G, hq = h * a.G + row % a.G;
  const Mass m = normalised(c, l, 0);
  a.lse[((int64_t)b * a.T + t) * a.Hq + hq] = l == 0.0f ? -INFINITY : (m.c + log2f(m.l)) * 0.693147180559945f;
}

// Joins the parts of the unit that begins in CTA blockIdx.x's stretch and is
// cut by its end; blockIdx.y takes kRows of its rows.  Threads beyond a float4 of each share the
// parts, group by group in list order, so the sums have one order.  The blocks
// become resident while the CTAs of the main kernel end, and read nothing before those have.
template <int R, int D>
struct Join {
  // few rows: more threads for each, since one unit may have a part in every CTA; many: a grid that stays within a
  // resident wave
  static constexpr int kRows = R >= 64 ? 8 : 4, kThreads = 256, kItems = kRows * D / 4, kGroups = kThreads / kItems;
  static_assert(kThreads % kItems == 0 && R % kRows == 0, "whole groups and blocks");
};
template <int R, int D>
__global__ void __launch_bounds__(256) cache_attn_join_kernel(const CacheAttnArgs a) {
  using J = Join<R, D>;
  constexpr int RB = J::kRows, V4 = D / 4;
  __shared__ float c_s[RB][kMaxCtas], l_s[RB][kMaxCtas];  // offsets, then weights; denominators
  __shared__ float c_row[RB], l_row[RB];
  __shared__ float4 o_s[J::kGroups > 1 ? J::kThreads : 1];
  begin_dependent();
  const int first = blockIdx.x, r0 = blockIdx.y * RB;
  const CutUnit u = *cut_unit(a, first);
  const int np = u.parts, nr = min(RB, u.rows - r0);
  if (np == 0 || nr <= 0) return;
  auto part = [&](int i) { return part_of<R, D>(a, first + i, i == 0 ? 1 : 0); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < np * RB; i += J::kThreads) {
    const int k = i / RB, r = i % RB;
    if (r < nr) {
      c_s[r][k] = part(k)[R * D + r0 + r];
      l_s[r][k] = part(k)[R * D + R + r0 + r];
    }
  }
  __syncthreads();
  if (warp < nr) {
    const int r = warp;
    float c = -INFINITY, l = 0.0f;
    for (int k = lane; k < np; k += 32) c = fmaxf(c, c_s[r][k]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) c = fmaxf(c, __shfl_xor_sync(0xffffffffu, c, o));
    for (int k = lane; k < np; k += 32) {
      const float f = c_s[r][k] == -INFINITY ? 0.0f : ex2f(c_s[r][k] - c);
      l += l_s[r][k] * f;
      c_s[r][k] = f;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) {
      c_row[r] = c;
      l_row[r] = l;
    }
  }
  __syncthreads();
  const int i4 = threadIdx.x % J::kItems, group = threadIdx.x / J::kItems, r = i4 / V4, col = 4 * (i4 % V4);
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (r < nr) {
#pragma unroll 8
    for (int k = group; k < np; k += J::kGroups) {
      const float f = c_s[r][k];
      const float4 x = *reinterpret_cast<const float4*>(part(k) + (r0 + r) * D + col);
      o.x += x.x * f; o.y += x.y * f; o.z += x.z * f; o.w += x.w * f;
    }
  }
  if (J::kGroups > 1) {
    o_s[threadIdx.x] = o;
    __syncthreads();
    if (group) return;
#pragma unroll
    for (int k = 1; k < J::kGroups; ++k) {
      const float4 x = o_s[k * J::kItems + i4];
      o.x += x.x; o.y += x.y; o.z += x.z; o.w += x.w;
    }
  }
  if (r >= nr) return;
  store_out(a, u.b, u.h, u.row0 + r0 + r, col, o, row_inverse(l_row[r]));
  if (col == 0) store_lse(a, u.b, u.h, u.row0 + r0 + r, c_row[r], l_row[r]);
}

template <int TILE, int R, int D, int STEP>
int launch_join(const CacheAttnArgs& a, cudaStream_t s) {
  using J = Join<R, D>;
  const int rows = min(R, a.T * a.G);                                                // of the fullest unit
  const int ctas = (int)fmin(kMaxCtas, ceil(longest_list<TILE, R>(a) / STEP));  // that can have a stretch
  return launch_dependent(cache_attn_join_kernel<R, D>, dim3(ctas, (rows + J::kRows - 1) / J::kRows), J::kThreads, 0, s, a);
}

}  // namespace cattn
}  // namespace sage
