// Attention of new or drafted tokens over the quantised paged cache.
//
// Row (b, t, h) of Q sees slots 0 .. context[b]-1 of its sequence, and slot
// context[b] + j of the drafted tokens where bit j of its mask is set:
//   s_j = (q . k_j) * kscale_j * sm_scale,  out = sum_j softmax(s)_j v_j vscale_j,
//   lse = ln sum_j exp(s_j);  a row that sees nothing has out = 0, lse = -inf.
//
// The count*G rows that share a head of the cache are the M side of
// m16n8k16 FP16 MMAs with FP32 sums, MT tiles of 16 rows at a time, so that
// every code is read and converted once for all of them.  The codes are exact
// in FP16.  Q is FP16 too: a row is scaled by a power of two that brings its
// largest value to 2^13, which leaves its BF16 values exact down to 2^-27 of
// the largest.
//
// Online softmax per row in base 2 with the running maximum c: FP32 sums
// l += p_j and O += w_j code_j, p_j = 2^(s_j - c) and w_j = p_j vscale_j 2^-E
// rounded to FP16 (2^-11) for the PV MMA.  E is an integer per row with 2^E
// at or above the largest V scale that the row has seen, so that w_j is at most
// 1; it is per row because a token that only other rows see may have any scale.
//
// Eight warps per CTA, one CTA per SM.  A warp takes every eighth tile of 16
// keys of the CTA's stretch of the work list and runs alone: lane 0 keeps its
// ring of K and V tiles (2 KB each at D = 128) filled by TMA, several tiles
// ahead and across units, and the warps meet only where a unit ends, to join
// their rows in shared memory.  16 keys are the smallest page, so a tile never
// crosses one.
#include "cache_attn.cuh"
#include "tc_prims.cuh"

namespace sage {
namespace {

using namespace cattn;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 16;       // keys
constexpr int kMaxCtas = 148;   // one per SM

// n index of an 8-key MMA tile -> key.  Keys of neighbouring n differ in bits
// 0 and 2, so the 16-byte shared-memory reads of two rows fall on different
// banks under both swizzles (64- and 128-byte rows).
__device__ __forceinline__ int key_of(int n) { return (n >> 1) ^ ((n & 1) ? 5 : 0); }

// Four codes -> bytes 0 and 2, and bytes 1 and 3, as FP16 pairs.
template <int F>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& even, uint32_t& odd) {
  if (F == SAGE_CACHE_INT8) {
    // 0x6400 | (code + 128) is 1024 + 128 + code in FP16
    const uint32_t e = (w & 0x00FF00FFu) ^ 0x64806480u, o = ((w >> 8) & 0x00FF00FFu) ^ 0x64806480u;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(even) : "r"(e), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(odd) : "r"(o), "r"(0x64806480u));
  } else {
    const uint32_t p = __byte_perm(w, 0, 0x3120);
    asm("{.reg .b16 lo, hi; mov.b32 {lo, hi}, %2; cvt.rn.f16x2.e4m3x2 %0, lo; cvt.rn.f16x2.e4m3x2 %1, hi;}"
        : "=r"(even), "=r"(odd)
        : "r"(p));
  }
}

// Unused slots hold any bytes: E4M3 NaN codes become 0 (their weight is 0).
template <int F>
__device__ __forceinline__ uint32_t no_nan(uint32_t w) {
  return F == SAGE_CACHE_E4M3 ? w & ~__vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu) : w;
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int D>
__device__ __forceinline__ uint32_t swizzled(int key, int chunk) {
  return key * D + ((D == 128 ? chunk ^ (key & 7) : chunk ^ ((key >> 1) & 3)) << 4);
}

template <int D, int MT>
struct Smem {
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr int kFrags = MT * (D / 8) * 4;  // FP32 sums per lane
  alignas(1024) uint8_t k[kWarps][kStages][kTile * D];
  alignas(1024) uint8_t v[kWarps][kStages][kTile * D];
  float join[kWarps / 2][kFrags][32];
  uint4 q[MT > 1 ? MT : 1][D / 16][32];  // MT > 1: Q fragments
  float f[16 * MT];
  float c[kWarps][16 * MT], l[kWarps][16 * MT];
  uint64_t full[kWarps][kStages];
  StretchSmem stretch;
};

// Running state of the thread's two rows (g and g + 8) of one 16-row tile.
struct Rows {
  float M[2], c[2], l[2];
  int E[2];
};

template <int D, int MT, int KF, int VF>
__global__ void __launch_bounds__(kThreads, 1)
    cache_attn_mma_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                          const CacheAttnArgs a) {
  constexpr int R = 16 * MT, KS = D / 16;  // rows of a unit, k steps of QK
  constexpr int S = Smem<D, MT>::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem<D, MT>& sm = *reinterpret_cast<Smem<D, MT>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c4 = lane & 3;

  if (threadIdx.x < kWarps * S) tc::mbar_init(&sm.full[0][0] + threadIdx.x, 1);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x == 0)  // lengths that cannot be
    for (int b = threadIdx.x; b < a.B; b += kThreads) {
      const int ctx = a.context[b], cnt = a.count ? a.count[b] : a.T;
      if (ctx < 0 || cnt < 0 || cnt > a.T ||
          (long long)ctx + cnt > ((long long)a.c.table_pages << a.c.page_shift))
        flag_bad(a.c.status, kWhereAttn);
    }
  const Stretch st = find_stretch<kTile, R, kThreads, kWarps>(a, blockIdx.x, gridDim.x, sm.stretch);
  __syncthreads();
  if (st.s >= st.e) return;

  // ---- this warp's tiles: list indices first, first + 8, ...; nt of them
  const long long first = st.s + warp;
  const int nt = first < st.e ? (int)((st.e - first + kWarps - 1) / kWarps) : 0;
  // cache rows (of head h, from the tile's first key on) of tiles 32 blk + lane: this block of 32 and the next
  Place walk = st.p;
  auto rows_of_block = [&](int blk) -> int {
    const long long idx = first + (long long)kWarps * (32 * blk + lane);
    if (idx >= st.e) return -1;
    go_to<kTile, R>(a, walk, idx);
    const Unit u = unit_of(walk, idx);
    const int64_t row = cache_row(a.c, walk.b, u.h, (idx - u.start) * kTile);
    if (row < 0) flag_bad(a.c.status, kWhereAttn);
    return (int)row;
  };
  int block = 0, rows_a = rows_of_block(0), rows_b = nt > 32 ? rows_of_block(1) : -1;
  auto row_of = [&](int i) { return __shfl_sync(0xffffffffu, (i >> 5) == block ? rows_a : rows_b, i & 31); };
  auto issue = [&](int i) {
    const int row = row_of(i), s = i % S;
    if (row >= 0 && lane == 0) {
      tc::mbar_expect_tx(&sm.full[warp][s], 2 * kTile * D);
      tc::tma_load_3d(sm.k[warp][s], &tm_k, 0, row, 0, &sm.full[warp][s]);
      tc::tma_load_3d(sm.v[warp][s], &tm_v, 0, row, 0, &sm.full[warp][s]);
    }
  };
  // the tile's K scales in lanes 0-15, its V scales in lanes 16-31
  auto scales_of = [&](int i) -> float {
    const int row = row_of(i);
    return row < 0 ? 0.0f : __ldg(lane < 16 ? a.c.scale[0] + row + lane : a.c.scale[1] + row + (lane - 16));
  };
  int issued = min(S, nt);
  for (int i = 0; i < issued; ++i) issue(i);
  float sc_next = nt > 0 ? scales_of(0) : 0.0f;
  uint32_t phase = 0;
  bool dead = false;  // a TMA tile that never came: nothing more is issued or computed
  int abort_flag = 0;

  const uint32_t kbase = smem_u32(sm.k[warp][0]), vbase = smem_u32(sm.v[warp][0]);
  const int vkey = 8 * ((lane >> 3) & 1) + key_of(lane & 7), vchunk = lane >> 4;  // this lane's ldmatrix row

  Place at = st.p;
  int i = 0;
  for (long long seg = st.s; seg < st.e;) {
    go_to<kTile, R>(a, at, seg);
    const Unit u = unit_of(at, seg);
    const int b = at.b, h = u.h, row0 = u.rt * R;
    const int ctx = at.s.ctx, cnt = at.s.cnt, rows = min(R, cnt * a.G - row0);
    const long long unit_end = u.start + at.s.n, seg_end = min(unit_end, st.e);
    const int i_end = seg_end > first ? (int)((seg_end - first + kWarps - 1) / kWarps) : 0;

    // ---- Q rows as A fragments: of k step 4x + i, k = 2c, 2c+1 and 2c+8, 2c+9 are channels 64x + 16c + 4i + 0, 2
    // and + 1, 3, the bytes 0, 2 and 1, 3 of the K words
    uint32_t qf[MT == 1 ? KS : 1][4];
    float f[MT][2];
    auto load_q = [&](int mt, auto&& put) {
      uint32_t w[2][D / 8];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int lr = 16 * mt + g + 8 * r;
        const bool on = lr < rows;
        const int t = (row0 + lr) / a.G, hq = h * a.G + (row0 + lr) % a.G;
        const uint16_t* q = a.q + b * a.qb + t * a.qn + hq * a.qh + 16 * c4;
        uint32_t top = 0;
#pragma unroll
        for (int x = 0; x < D / 64; ++x)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (on) v = __ldg(reinterpret_cast<const uint4*>(q + 64 * x + 8 * y));
            const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              w[r][8 * x + 4 * y + e] = vw[e];
              top = max(top, max(vw[e] & 0x7FFFu, (vw[e] >> 16) & 0x7FFFu));
            }
          }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int eq = (top == 0 || top >= 0x7F80u) ? 0 : max((int)(top >> 7) - 127 - 13, -110);
        const float down = __int_as_float((127 - eq) << 23);
        f[mt][r] = fmaxf(a.sl2 * __int_as_float((127 + eq) << 23), 1.17549435e-38f);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const uint32_t w0 = w[r][2 * s], w1 = w[r][2 * s + 1];  // channels 4s .. 4s + 3 of this lane's
          put(s, r, pack_f16x2(__uint_as_float(w0 << 16) * down, __uint_as_float(w1 << 16) * down),
              pack_f16x2(__uint_as_float(w0 & 0xFFFF0000u) * down, __uint_as_float(w1 & 0xFFFF0000u) * down));
        }
      }
    };
    if constexpr (MT == 1) {
      load_q(0, [&](int s, int r, uint32_t even, uint32_t odd) { qf[s][r] = even; qf[s][2 + r] = odd; });
    } else {
      if (warp < MT) {
        load_q(warp % MT, [&](int s, int r, uint32_t even, uint32_t odd) {
          uint32_t* to = reinterpret_cast<uint32_t*>(&sm.q[warp % MT][s][lane]);
          to[r] = even;
          to[2 + r] = odd;
        });
      }
    }
    float o[MT][D / 8][4];
    Rows rs[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        rs[mt].M[r] = -INFINITY;
        rs[mt].c[r] = 0.0f;
        rs[mt].l[r] = 0.0f;
        rs[mt].E[r] = -126;
      }
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][n][e] = 0.0f;
    }
    if constexpr (MT > 1) {
      if (warp < MT && c4 == 0) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
          if (mt == warp) { sm.f[16 * mt + g] = f[mt][0]; sm.f[16 * mt + g + 8] = f[mt][1]; }
      }
      __syncthreads();
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) { f[mt][0] = sm.f[16 * mt + g]; f[mt][1] = sm.f[16 * mt + g + 8]; }
    }

    // ---- one tile of 16 keys from slot `slot0` on
    auto tile = [&](auto masked_tag, uint32_t ks_addr, uint32_t vs_addr, float sc, int64_t slot0) {
      constexpr bool MASKED = decltype(masked_tag)::value;
      float s[MT][2][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[mt][j][e] = 0.0f;
#pragma unroll
      for (int x = 0; x < D / 64; ++x) {
        uint4 kw[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) kw[j] = lds128(ks_addr + swizzled<D>(8 * j + key_of(g), 4 * x + c4));
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          uint32_t qa[MT][4];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            if constexpr (MT == 1) {
#pragma unroll
              for (int e = 0; e < 4; ++e) qa[mt][e] = qf[4 * x + y][e];
            } else {
              const uint4 v = sm.q[mt][4 * x + y][lane];
              qa[mt][0] = v.x; qa[mt][1] = v.y; qa[mt][2] = v.z; qa[mt][3] = v.w;
            }
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t w = y == 0 ? kw[j].x : y == 1 ? kw[j].y : y == 2 ? kw[j].z : kw[j].w;
            uint32_t b0, b1;
            codes_to_f16<KF>(w, b0, b1);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) mma16816(s[mt][j], qa[mt], b0, b1);
          }
        }
      }
      float ksc[2][2], vsc[2][2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int key = 8 * j + (e ? c4 ^ 5 : c4);
          ksc[j][e] = __shfl_sync(0xffffffffu, sc, key);
          vsc[j][e] = __shfl_sync(0xffffffffu, sc, 16 + key);
        }
      uint32_t pa[MT][4];
      float al[MT][2];
      bool moved = false;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        Rows& q = rs[mt];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float x[2][2], vv[2][2];
          float top = -INFINITY, vmax = 0.0f;
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              x[j][e] = s[mt][j][2 * r + e] * ksc[j][e];
              vv[j][e] = vsc[j][e];
              if (MASKED) {
                const int64_t slot = slot0 + 8 * j + (e ? c4 ^ 5 : c4);
                bool seen = slot < ctx;
                const int lr = 16 * mt + g + 8 * r;
                if (!seen && slot < (int64_t)ctx + cnt && lr < rows) {
                  const int d = (int)(slot - ctx), t = (row0 + lr) / a.G;
                  seen = a.mask ? (__ldg(a.mask + ((int64_t)b * a.T + t) * ((a.T + 31) / 32) + d / 32) >> (d % 32)) & 1u
                                : d <= t;
                }
                if (!seen) { x[j][e] = -INFINITY; vv[j][e] = 0.0f; }
              }
              top = fmaxf(top, x[j][e]);
              vmax = fmaxf(vmax, vv[j][e]);
            }
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, 2));
          const float M = fmaxf(q.M[r], top);
          const int E = min(max(q.E[r], (__float_as_int(vmax) >> 23) - 126), 126);
          const float c = M == -INFINITY ? 0.0f : M * f[mt][r], down = __int_as_float((127 - E) << 23);
          const float al_l = q.M[r] == -INFINITY ? 0.0f : ex2f(q.c[r] - c);
          al[mt][r] = E == q.E[r] ? al_l : al_l * ex2f((float)(q.E[r] - E));
          moved |= al[mt][r] != 1.0f;
          float w[2][2], sum = 0.0f;
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float p = ex2f(fmaf(x[j][e], f[mt][r], -c));
              sum += p;
              w[j][e] = p * (vv[j][e] * down);
            }
          q.l[r] = q.l[r] * al_l + sum;
          q.M[r] = M; q.E[r] = E; q.c[r] = c;
          pa[mt][r] = pack_f16x2(w[0][0], w[0][1]);
          pa[mt][2 + r] = pack_f16x2(w[1][0], w[1][1]);
        }
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[mt][n][e] *= al[mt][e >> 1];
      }
#pragma unroll
      for (int x = 0; x < D / 16; x += 2) {
        uint32_t vw[4];
        ldmatrix_x4_trans(vs_addr + swizzled<D>(vkey, x + vchunk), vw);
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          uint32_t e0, o0, e1, o1;
          codes_to_f16<VF>(MASKED ? no_nan<VF>(vw[2 * y]) : vw[2 * y], e0, o0);
          codes_to_f16<VF>(MASKED ? no_nan<VF>(vw[2 * y + 1]) : vw[2 * y + 1], e1, o1);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            mma16816(o[mt][2 * (x + y)], pa[mt], e0, e1);
            mma16816(o[mt][2 * (x + y) + 1], pa[mt], o0, o1);
          }
        }
      }
    };

    for (; i < i_end; ++i) {
      const int row = row_of(i), s = i % S;
      const float sc = sc_next;
      if (i + 1 < nt) sc_next = scales_of(i + 1);
      if (row >= 0 && i < issued) {
        if (!tc::wait_bounded(&sm.full[warp][s], (phase >> s) & 1u, &abort_flag, a.c.status, kWhereAttn,
                              kDefaultWaitLimit, false))
          dead = true;
        phase ^= 1u << s;
        dead = __any_sync(0xffffffffu, dead);
        if (!dead) {
          const int64_t slot0 = (first + (long long)kWarps * i - u.start) * kTile;
          const uint32_t ka = kbase + s * kTile * D, va = vbase + s * kTile * D;
          if (slot0 + kTile <= ctx) tile(std::false_type{}, ka, va, sc, slot0);
          else tile(std::true_type{}, ka, va, sc, slot0);
        }
      }
      __syncwarp();
      if (issued < nt && !dead) issue(issued++);
      if ((i & 31) == 31) {
        ++block;
        rows_a = rows_b;
        rows_b = nt > 32 * (block + 1) ? rows_of_block(block + 1) : -1;
      }
    }

    // ---- join the warps' rows
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float l = rs[mt].l[r];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (c4 == 0) {
          sm.c[warp][16 * mt + g + 8 * r] = rs[mt].M[r] == -INFINITY ? -INFINITY : rs[mt].c[r];
          sm.l[warp][16 * mt + g + 8 * r] = l;
        }
      }
    __syncthreads();
    float cmax[MT][2], lsum[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int lr = 16 * mt + g + 8 * r;
        float c = -INFINITY, l = 0.0f, mine = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) c = fmaxf(c, sm.c[w][lr]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float cw = sm.c[w][lr], fw = cw == -INFINITY ? 0.0f : ex2f(cw - c);
          l += sm.l[w][lr] * fw;
          if (w == warp) mine = fw;
        }
        cmax[mt][r] = c;
        lsum[mt][r] = l;
        mine *= __int_as_float((127 + rs[mt].E[r]) << 23);
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
          o[mt][n][2 * r] *= mine;
          o[mt][n][2 * r + 1] *= mine;
        }
      }
    if (warp >= kWarps / 2) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) sm.join[warp - kWarps / 2][(mt * (D / 8) + n) * 4 + e][lane] = o[mt][n][e];
    }
    __syncthreads();
    if (warp < kWarps / 2) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) sm.join[warp][(mt * (D / 8) + n) * 4 + e][lane] += o[mt][n][e];
    }
    __syncthreads();
    const bool whole = seg == u.start && seg_end == unit_end;
    float* part = part_of<R, D>(a, blockIdx.x, seg == u.start ? 1 : 0);
    // 16 columns of 16 rows at a time: even columns in fragment 2x, odd ones in 2x + 1
#pragma unroll
    for (int it = 0; it < (MT * D / 16 + kWarps - 1) / kWarps; ++it) {
      const int item = it * kWarps + warp;
      if (item < MT * D / 16) {
        const int mt = item / (D / 16), x = item % (D / 16);
        float v[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int fr = (mt * (D / 8) + 2 * x + n) * 4 + e;
            v[n][e] = (sm.join[0][fr][lane] + sm.join[1][fr][lane]) + (sm.join[2][fr][lane] + sm.join[3][fr][lane]);
          }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int lr = 16 * mt + g + 8 * r, col = 16 * x + 4 * c4;
          const float4 ov = make_float4(v[0][2 * r], v[1][2 * r], v[0][2 * r + 1], v[1][2 * r + 1]);
          float cc = cmax[0][r], ll = lsum[0][r];
#pragma unroll
          for (int k = 1; k < MT; ++k)
            if (k == mt) { cc = cmax[k][r]; ll = lsum[k][r]; }
          if (lr < rows) {
            if (whole) {
              store_out(a, b, h, row0 + lr, col, ov, row_inverse(ll));
              if (x == 0 && c4 == 0) store_lse(a, b, h, row0 + lr, cc, ll);
            } else {
              *reinterpret_cast<float4*>(part + lr * D + col) = ov;
              if (x == 0 && c4 == 0) { part[R * D + lr] = cc; part[R * D + R + lr] = ll; }
            }
          }
        }
      }
    }
    __syncthreads();
    seg = seg_end;
  }
}

template <int D, int MT, int KF, int VF>
int launch_mma(const CacheAttnArgs& a, cudaStream_t s) {
  constexpr int R = 16 * MT;
  const uint64_t rows = (uint64_t)a.c.pages * a.c.H << a.c.page_shift;
  CUtensorMap mk, mv;
  if (!tc::make_map(&mk, a.c.codes[0], D, rows, 1, D, rows * D, D, kTile) ||
      !tc::make_map(&mv, a.c.codes[1], D, rows, 1, D, rows * D, D, kTile))
    return SAGE_ERR_CUDA;
  auto* fn = cache_attn_mma_kernel<D, MT, KF, VF>;
  const size_t smem = sizeof(Smem<D, MT>) + 1024;
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return SAGE_ERR_CUDA;
  fn<<<kMaxCtas, kThreads, smem, s>>>(mk, mv, a);
  if (cudaGetLastError() != cudaSuccess) return SAGE_ERR_CUDA;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kMaxCtas, 2);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_attn_join_kernel<kTile, R, D, kWarps, 256>, a, kMaxCtas) == cudaSuccess
             ? SAGE_OK
             : SAGE_ERR_CUDA;
}

template <int D, int MT>
int by_format(const CacheAttnArgs& a, cudaStream_t s) {
  const bool k8 = a.c.format[0] == SAGE_CACHE_INT8, v8 = a.c.format[1] == SAGE_CACHE_INT8;
  if (k8) return v8 ? launch_mma<D, MT, SAGE_CACHE_INT8, SAGE_CACHE_INT8>(a, s) : launch_mma<D, MT, SAGE_CACHE_INT8, SAGE_CACHE_E4M3>(a, s);
  return v8 ? launch_mma<D, MT, SAGE_CACHE_E4M3, SAGE_CACHE_INT8>(a, s) : launch_mma<D, MT, SAGE_CACHE_E4M3, SAGE_CACHE_E4M3>(a, s);
}

}  // namespace

size_t cache_attn_workspace_bytes() { return (size_t)2 * kMaxCtas * (32 * 128 + 2 * 32) * sizeof(float); }

int launch_cache_attn(const CacheAttnArgs& a, cudaStream_t s) {
  const bool one = a.T * a.G <= 16;
  if (a.c.D == 128) return one ? by_format<128, 1>(a, s) : by_format<128, 2>(a, s);
  return one ? by_format<64, 1>(a, s) : by_format<64, 2>(a, s);
}

}  // namespace sage
