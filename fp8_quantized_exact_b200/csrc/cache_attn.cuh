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
#include "cache_common.cuh"

namespace sage {
namespace cattn {

struct Seq {
  int ctx, cnt;     // context and drafted tokens
  int n;            // tiles
  int rt;           // row tiles
  long long per;    // tiles of all its units
};

template <int TILE, int R>
__device__ __forceinline__ Seq seq_of(const CacheAttnArgs& a, int b) {
  Seq s;
  s.ctx = max(__ldg(a.context + b), 0);
  s.cnt = a.count ? min(max(__ldg(a.count + b), 0), a.T) : a.T;
  const long long cap = (long long)a.c.table_pages << a.c.page_shift;
  s.n = (int)((min((long long)s.ctx + s.cnt, cap) + TILE - 1) / TILE);
  s.rt = (s.cnt * a.G + R - 1) / R;
  s.per = (long long)a.c.H * s.rt * s.n;
  return s;
}

// A place in the list: the sequence b whose tiles begin at `base`.
struct Place {
  long long base;
  int b;
  Seq s;
};
// Moves on to the sequence of tile idx (idx >= base, below the list's end).
template <int TILE, int R>
__device__ __forceinline__ void go_to(const CacheAttnArgs& a, Place& p, long long idx) {
  while (idx >= p.base + p.s.per) {
    p.base += p.s.per;
    ++p.b;
    p.s = seq_of<TILE, R>(a, p.b);
  }
}
struct Unit {
  int h, rt;         // head of the cache, row tile
  long long start;   // list index of its first tile
};
__device__ __forceinline__ Unit unit_of(const Place& p, long long idx) {
  const unsigned long long u = (unsigned long long)(idx - p.base) / (unsigned)p.s.n;
  Unit r;
  r.rt = (int)(u % (unsigned)p.s.rt);
  r.h = (int)(u / (unsigned)p.s.rt);
  r.start = p.base + (long long)u * p.s.n;
  return r;
}

// The stretch [s, e) of CTA `cta` of at most `ctas`, by a whole block (THREADS
// threads): lengths are summed and searched THREADS sequences at a time.
// STEP: stretches are multiples of it (what a CTA does at once).
struct Stretch {
  long long s, e, share, total;
  Place p;
};
struct StretchSmem {
  long long warp_sum[32];
  long long base;
  int b;
};
template <int TILE, int R, int THREADS, int STEP>
__device__ __forceinline__ Stretch find_stretch(const CacheAttnArgs& a, int cta, int ctas, StretchSmem& sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // inclusive sum over the block of one value per thread, and the total
  auto block_scan = [&](long long v, long long& total) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long w = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += w;
    }
    __syncthreads();
    if (lane == 31) sm.warp_sum[warp] = v;
    __syncthreads();
    long long before = 0;
    total = 0;
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) before += sm.warp_sum[w];
      total += sm.warp_sum[w];
    }
    return v + before;
  };
  auto tiles = [&](int b) { return b < a.B ? seq_of<TILE, R>(a, b).per : 0; };
  Stretch t;
  t.total = 0;
  long long mine = tiles(threadIdx.x), incl = 0, part;
  for (int b0 = 0; b0 < a.B; b0 += THREADS) {
    incl = block_scan(b0 == 0 ? mine : tiles(b0 + threadIdx.x), part);
    t.total += part;
  }
  t.share = (t.total + ctas - 1) / ctas;
  t.share = max((t.share + STEP - 1) / STEP, 1ll) * STEP;
  t.s = min(cta * t.share, t.total);
  t.e = min(t.s + t.share, t.total);
  t.p.base = 0;
  t.p.b = 0;
  if (t.s < t.e) {
    long long before = 0;
    for (int b0 = 0; b0 < a.B; b0 += THREADS) {
      if (a.B > THREADS) {  // otherwise the one block of sums is still here
        mine = tiles(b0 + threadIdx.x);
        incl = block_scan(mine, part);
      } else {
        part = t.total;
      }
      if (t.s >= before + incl - mine && t.s < before + incl) {
        sm.base = before + incl - mine;
        sm.b = b0 + threadIdx.x;
      }
      before += part;
      if (before > t.s) break;
    }
    __syncthreads();
    t.p.base = sm.base;
    t.p.b = sm.b;
    t.p.s = seq_of<TILE, R>(a, t.p.b);
  }
  return t;
}

constexpr int kMaxCtas = 148;  // one per SM
constexpr int kMaxRows = 128;  // of a unit
constexpr size_t kCtaPartBytes = (size_t)2 * kMaxCtas * (kMaxRows * 128 + 2 * kMaxRows) * sizeof(float);

// Parts of the CTAs: [2 * CTA + slot] of R x D sums, R offsets, R denominators;
// behind them, where warps leave parts too, [2 * warp of the grid + slot] of R x D sums.
template <int R, int D>
__device__ __forceinline__ float* warp_part(const CacheAttnArgs& a, int warp, int slot) {
  return static_cast<float*>(a.workspace) + kCtaPartBytes / sizeof(float) + (size_t)(2 * warp + slot) * (R * D);
}
template <int R, int D>
__device__ __forceinline__ float* part_of(const CacheAttnArgs& a, int cta, int slot) {
  return static_cast<float*>(a.workspace) + (size_t)(2 * cta + slot) * (R * D + 2 * R);
}

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
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
  a.lse[((int64_t)b * a.T + t) * a.Hq + hq] = l == 0.0f ? -INFINITY : (c + log2f(l)) * 0.693147180559945f;
}

// Joins the parts of the unit that begins in CTA blockIdx.x's stretch and is
// cut by its end; blockIdx.y of gridDim.y takes a share of the columns.
template <int TILE, int R, int D, int STEP, int THREADS>
__global__ void __launch_bounds__(THREADS) cache_attn_join_kernel(const CacheAttnArgs a, int ctas) {
  __shared__ StretchSmem sm;
  __shared__ float c_row[R], l_row[R];
  const Stretch st = find_stretch<TILE, R, THREADS, STEP>(a, blockIdx.x, ctas, sm);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // from here on the parts are written
  if (st.s >= st.e) return;
  Place p = st.p;
  go_to<TILE, R>(a, p, st.e - 1);
  const Unit u = unit_of(p, st.e - 1);
  const long long end = u.start + p.s.n;
  if (u.start < st.s || end <= st.e) return;
  const int last = (int)((end - 1) / st.share);
  const int rows = min(R, p.s.cnt * a.G - u.rt * R);
  auto part = [&](int i) { return part_of<R, D>(a, i, i == (int)blockIdx.x ? 1 : 0); };
  for (int r = threadIdx.x; r < rows; r += THREADS) {
    float c = -INFINITY, l = 0.0f;
    for (int i = blockIdx.x; i <= last; ++i) c = fmaxf(c, part(i)[R * D + r]);
    for (int i = blockIdx.x; i <= last; ++i) {
      const float ci = part(i)[R * D + r];
      l += part(i)[R * D + R + r] * (ci == -INFINITY ? 0.0f : ex2f(ci - c));
    }
    c_row[r] = c;
    l_row[r] = l;
    if (blockIdx.y == 0) store_lse(a, p.b, u.h, u.rt * R + r, c, l);
  }
  __syncthreads();
  constexpr int V4 = D / 4;
  for (int i4 = blockIdx.y * THREADS + threadIdx.x; i4 < rows * V4; i4 += gridDim.y * THREADS) {
    const int r = i4 / V4, col = 4 * (i4 % V4);
    const float c = c_row[r];
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int i = blockIdx.x; i <= last; ++i) {
      const float ci = part(i)[R * D + r];
      const float f = ci == -INFINITY ? 0.0f : ex2f(ci - c);
      const float4 x = *reinterpret_cast<const float4*>(part(i) + r * D + col);
      o.x += x.x * f; o.y += x.y * f; o.z += x.z * f; o.w += x.w * f;
    }
    store_out(a, p.b, u.h, u.rt * R + r, col, o, row_inverse(l_row[r]));
  }
}

}  // namespace cattn
}  // namespace sage
