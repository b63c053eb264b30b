// Attention of new or drafted tokens over the quantised paged cache.
//
// Row (b, t, h) of Q sees slots 0 .. context[b]-1 of its sequence, and slot
// context[b] + j of the drafted tokens where bit j of its mask is set:
//   s_j = (q . k_j) * kscale_j * sm_scale,  out = sum_j softmax(s)_j v_j vscale_j,
//   lse = ln sum_j exp(s_j);  a row that sees nothing has out = 0, lse = -inf.
//
// Transposed products: S^T = K Q^T and O^T = V^T P^T as m16n8k16 FP16 MMAs
// with FP32 sums, the codes (exact in FP16) as the A operand and NT groups of 8
// of the count*G rows that share a head as the B operand, so that a decode step
// of up to 8 query heads per head wastes no MMA and every code is read and
// converted once for all rows.  Q is FP16 too: a row is scaled by a power of two
// that brings its largest value to 2^13, which leaves its BF16 values exact
// down to 2^-27 of the largest.
//
// Online softmax per row in base 2: FP32 sums l += p_j and O += w_j code_j,
// p_j = 2^(s_j - c) and w_j = p_j vscale_j 2^-E rounded to FP16 (2^-11), for which
// c keeps the row's largest weight near 2^8 (cache_codes.cuh says why).  c is set
// again only when a score passes it by more than 15 or a V scale passes 2^E, which
// one vote per tile finds out: later tiles need no reduction across lanes.  E is an
// integer per row with 2^E at or above the largest V scale that the row has seen; it
// is per row because a token that only other rows see may have any scale.  When E
// grows, c falls by as much, which leaves the unit of O.
//
// One CTA per SM.  A CTA's stretch of the work list is cut once more, into one
// stretch per warp, and the warps run alone: lane 0 keeps its ring of K and V
// tiles of 32 keys filled by TMA, ahead and across units; a unit that lies
// within the warp's stretch is finished from its registers, one that is cut
// leaves a part in shared memory, and the CTA joins its warps' parts once, at its
// end.  A tile is two boxes of 16 keys, the smallest page, so a box never crosses
// one.
#include "cache_attn.cuh"
#include "cache_codes.cuh"
#include "tc_prims.cuh"

namespace sage {
namespace {

using namespace cattn;

constexpr int kTile = 32, kBox = 16;  // keys

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Launch shape by D and the number of 8-row groups.  A tile of D = 64 is half the work between the same waits, so more
// warps run beside each other: 12 are three for each quarter of the SM, which 168 registers allow.  Measured on B200
// (us, D = 64; one context of 151241 at 4 rows per head, 16 contexts of 500..16384 at 16 and 48): 10, 12, 14, 16, 20
// warps 49.4, 44.4, 47.3, 46.4, 74.7 at 4 rows; 8 and 12 warps 71 and 66 at 16 rows, 159 and 142 at 48.  D = 128 at 4 rows
// (64 contexts of 1..8192): 8, 10, 11 warps 127, 122, 125; shared memory ends there.
template <int D, int NT>
struct Shape {
  static constexpr int kWarps = D == 64 ? 12 : NT == 1 ? 10 : 8;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kRegs = D == 64 ? (NT == 1 ? 144 : 168) : NT == 1 ? 168 : 224;
  static constexpr int kStages = D == 64 ? 3 : 2;
  static_assert(kStages * kTile * D >= 8 * NT * D * 4, "a part fits a warp's ring of K");
};

// The last unit of a warp's stretch, and the first of the CTA's: what the CTA's
// join needs of it.  slot -1: the warp left no such part.
struct Cut {
  unsigned start, end;  // of the unit, in the list
  int slot, b, h, row0, rows;
  const float* sums;
};

template <int D, int NT>
struct Smem {
  using Sh = Shape<D, NT>;
  alignas(1024) uint8_t k[Sh::kWarps][Sh::kStages][kTile * D];
  alignas(1024) uint8_t v[Sh::kWarps][Sh::kStages][kTile * D];
  float head[Sh::kWarps][8 * NT * D];  // sums of slot 0, where the stretch goes on behind them; the others lie in the ring of K
  float c[Sh::kWarps][2][8 * NT], l[Sh::kWarps][2][8 * NT];  // of the parts
  Cut cut[Sh::kWarps + 1];  // [w]: a unit that begins in warp w's stretch and goes on; [kWarps]: one that began before the CTA's
  const float* at0[Sh::kWarps];  // sums of slot 0
  uint64_t full[Sh::kWarps][Sh::kStages];
};

// Running state of the thread's rows 8 nt + 2c and 8 nt + 2c + 1.
struct Rows {
  uint64_t l, f, nc, down;  // pairs: sum, score factor, -c, 2^-E
  float thr[2];             // raw score above which c is raised; -inf: nothing seen yet
};

template <int D, int NT, int KF, int VF>
__global__ void __maxnreg__((Shape<D, NT>::kRegs))
    cache_attn_mma_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                          const CacheAttnArgs a) {
  using Sh = Shape<D, NT>;
  constexpr int R = 8 * NT, KS = D / 16, S = Sh::kStages, W = Sh::kWarps, XV = D / 16;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem<D, NT>& sm = *reinterpret_cast<Smem<D, NT>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c4 = lane & 3;

  if (lane == 0) {
    for (int s = 0; s < S; ++s) tc::mbar_init(&sm.full[warp][s], 1);
    sm.cut[warp].slot = -1;
    if (warp == 0) sm.cut[W].slot = -1;
  }
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  __syncwarp();
  begin_dependent_tma();
  const Stretch st = find_stretch<kTile, R, W>(a, blockIdx.x, gridDim.x);
  if (blockIdx.x == 0)  // lengths that cannot be
    for (int b = threadIdx.x; b < a.B; b += Sh::kThreads) {
      const int ctx = a.context[b], cnt = a.count ? a.count[b] : a.T;
      if (ctx < 0 || cnt < 0 || cnt > a.T ||
          (long long)ctx + cnt > ((long long)a.c.table_pages << a.c.page_shift))
        flag_bad(a.c.status, kWhereAttn);
    }
  if (threadIdx.x == 0) cut_unit(a, blockIdx.x)->parts = 0;  // behind the wait: the join of a call before may read its own until then
  if (st.s >= st.e) return;

  // ---- this warp's tiles: list indices [first, last)
  const unsigned share = st.share / W, first = min(st.s + warp * share, st.e), last = min(first + share, st.e);
  const int n_tiles = (int)(last - first);
  const Place begin = n_tiles > 0 ? place_of<kTile, R>(a, st.own, first) : Place{};
  // cache rows of the two boxes of tiles 32 blk + lane, -1 for a box without keys: this block of 32 tiles and the next
  Place walk = begin;
  auto rows_of_block = [&](int blk, int& r0, int& r1) {
    r0 = r1 = -1;
    const unsigned idx = first + 32 * blk + lane;
    if (idx >= last) return;
    go_to<kTile, R>(a, walk, idx);
    const Unit u = unit_of(walk, idx);
    const int64_t slot = (int64_t)(idx - u.start) * kTile, end = (int64_t)walk.s.ctx + walk.s.cnt;
    r0 = (int)cache_row(a.c, walk.b, u.h, slot);
    if (r0 < 0) flag_bad(a.c.status, kWhereAttn);
    if (slot + kBox < end) {
      r1 = (int)cache_row(a.c, walk.b, u.h, slot + kBox);
      if (r1 < 0) flag_bad(a.c.status, kWhereAttn);
    }
  };
  int block = 0, ra0 = -1, ra1 = -1, rb0 = -1, rb1 = -1;
  if (n_tiles > 0) rows_of_block(0, ra0, ra1);
  if (n_tiles > 32) rows_of_block(1, rb0, rb1);
  auto row0_of = [&](int i) { return __shfl_sync(0xffffffffu, (i >> 5) == block ? ra0 : rb0, i & 31); };
  auto row1_of = [&](int i) { return __shfl_sync(0xffffffffu, (i >> 5) == block ? ra1 : rb1, i & 31); };
  auto issue = [&](int i) {
    const int r0 = row0_of(i), r1 = row1_of(i), s = i % S;
    if (i == a.stall_tile) return;  // test hook
    if (lane == 0 && (r0 >= 0 || r1 >= 0)) {
      uint64_t* bar = &sm.full[warp][s];
      tc::mbar_expect_tx(bar, (r0 >= 0 && r1 >= 0 ? 4 : 2) * kBox * D);
      if (r0 >= 0) {
        tc::tma_load_3d(sm.k[warp][s], &tm_k, 0, r0, 0, bar);
        tc::tma_load_3d(sm.v[warp][s], &tm_v, 0, r0, 0, bar);
      }
      if (r1 >= 0) {
        tc::tma_load_3d(sm.k[warp][s] + kBox * D, &tm_k, 0, r1, 0, bar);
        tc::tma_load_3d(sm.v[warp][s] + kBox * D, &tm_v, 0, r1, 0, bar);
      }
    }
  };
  // the scales of the tile's key `lane`
  auto scales_of = [&](int i, float& ks, float& vs) {
    const int r0 = row0_of(i), r1 = row1_of(i), row = lane < kBox ? r0 : r1;
    ks = row < 0 ? 0.0f : a.c.scale[0][row + (lane & 15)];
    vs = row < 0 ? 0.0f : a.c.scale[1][row + (lane & 15)];
  };
  int issued = min(S, n_tiles);
  for (int i = 0; i < issued; ++i) issue(i);
  float ks_next = 0.0f, vs_next = 0.0f;
  if (n_tiles > 0) scales_of(0, ks_next, vs_next);
  uint32_t phase = 0;
  bool dead = false;  // a TMA tile that never came: nothing more is issued or computed
  int abort_flag = 0;

  const uint32_t kbase = smem_u32(sm.k[warp][0]), vbase = smem_u32(sm.v[warp][0]);
  // this lane's 16-byte reads: K row key_of(g), V row of its ldmatrix matrix
  const uint32_t ksw = swizzled<D>(key_of(g), c4);
  const int vkey = 8 * ((lane >> 3) & 1) + key_of(lane & 7), vchunk = lane >> 4;

  Place at = begin;
  int i = 0;
  for (unsigned seg = first; seg < last;) {
    go_to<kTile, R>(a, at, seg);
    const Unit u = unit_of(at, seg);
    const int b = at.b, h = u.h, row0 = u.rt * R;
    const int ctx = at.s.ctx, cnt = at.s.cnt, rows = min(R, cnt * a.G - row0);
    const unsigned unit_end = u.start + at.s.n, seg_end = min(unit_end, last);
    const int i_end = (int)(seg_end - first);

    // ---- Q rows as B fragments: of k step 4x + y, k = 2c, 2c+1 and 2c+8, 2c+9 are channels 64x + 16c + 4y + 0, 2
    // and + 1, 3, the bytes 0, 2 and 1, 3 of the K words
    uint2 qf[NT][KS];
    Rows rs[NT];
    auto load_q = [&](int nt, auto&& put) -> float {
      uint32_t w[D / 8];
      const int lr = 8 * nt + g;
      const int t = (row0 + lr) / a.G, hq = h * a.G + (row0 + lr) % a.G;
      const uint16_t* q = a.q + b * a.qb + t * a.qn + hq * a.qh + 16 * c4;
      uint32_t top = 0;
#pragma unroll
      for (int x = 0; x < D / 64; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (lr < rows) v = *reinterpret_cast<const uint4*>(q + 64 * x + 8 * y);
          const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            w[8 * x + 4 * y + e] = vw[e];
            top = max(top, max(vw[e] & 0x7FFFu, (vw[e] >> 16) & 0x7FFFu));
          }
        }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int eq = q_exponent(top);
      const float down = q_down(top, eq);
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const uint32_t w0 = w[2 * s], w1 = w[2 * s + 1];
        put(s, make_uint2(pack_f16x2(__uint_as_float(w0 << 16) * down, __uint_as_float(w1 << 16) * down),
                          pack_f16x2(__uint_as_float(w0 & 0xFFFF0000u) * down, __uint_as_float(w1 & 0xFFFF0000u) * down)));
      }
      return q_factor(eq);
    };
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float f = load_q(nt, [&](int s, uint2 v) { qf[nt][s] = v; });
      rs[nt].f = pair(__shfl_sync(0xffffffffu, f, 8 * c4), __shfl_sync(0xffffffffu, f, 8 * c4 + 4));
    }
    float o[NT][XV][4];
    float vlim = 1.17549435e-38f;  // the smallest 2^E of the thread's rows
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      rs[nt].l = rs[nt].nc = 0;
      rs[nt].down = pair(0x1p126f, 0x1p126f);
      rs[nt].thr[0] = rs[nt].thr[1] = -INFINITY;
#pragma unroll
      for (int x = 0; x < XV; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][x][e] = 0.0f;
    }

    // ---- one tile of 32 keys from slot `slot0` on; box0, box1: it holds the keys of that box
    auto tile = [&](auto masked_tag, uint32_t ka, uint32_t va, float ks, float vs, int64_t slot0, bool box0, bool box1) {
      constexpr bool MASKED = decltype(masked_tag)::value;
      float s[2][NT][4];  // keys 16 hf + key_of(g), + 8; rows 2c, 2c + 1
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[hf][nt][e] = 0.0f;
#pragma unroll
      for (int x = 0; x < D / 64; ++x) {
        uint4 kw[2][2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int j = 0; j < 2; ++j) kw[hf][j] = lds128((ka + (16 * hf + 8 * j) * D + ksw) ^ (64 * x));
#pragma unroll
        for (int y = 0; y < 4; ++y) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            uint32_t fa[4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint4& k4 = kw[hf][j];
              codes_to_f16<KF>(y == 0 ? k4.x : y == 1 ? k4.y : y == 2 ? k4.z : k4.w, fa[j], fa[2 + j]);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816(s[hf][nt], fa, qf[nt][4 * x + y].x, qf[nt][4 * x + y].y);
          }
        }
      }
      float vsc[2][2], vtop = 0.0f;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int key = 16 * hf + 8 * j + key_of(g);
          const float kk = __shfl_sync(0xffffffffu, ks, key);
          vsc[hf][j] = __shfl_sync(0xffffffffu, vs, key);
          if (!MASKED) vtop = fmaxf(vtop, vsc[hf][j]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float2 x = unpair(mul2(pair(s[hf][nt][2 * j], s[hf][nt][2 * j + 1]), pair(kk, kk)));
            s[hf][nt][2 * j] = x.x;
            s[hf][nt][2 * j + 1] = x.y;
          }
        }
      // a masked tile: which of its scores the rows see
      uint32_t seen = 0xFFFFFFFFu;  // bit (nt * 8 + hf * 4 + j * 2 + e)
      if (MASKED) {
        seen = 0;
        const int64_t d0 = slot0 - ctx;  // drafted token of the tile's first key (below 0: context)
        const bool drafts = d0 < cnt && d0 > -kTile;
        const int lo = (int)max(d0, (int64_t)0), hi = drafts ? min((int)(d0 + kTile), cnt) : lo;  // drafted tokens [lo, hi)
        const int words = (a.T + 31) / 32, w0 = lo / 32;
        uint32_t m[NT][2][2];  // the rows' mask words of lo and behind, all loads before the first use
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int lr = 8 * nt + 2 * c4 + e, t = (row0 + lr) / a.G;
#pragma unroll
            for (int w = 0; w < 2; ++w)
              m[nt][e][w] = a.mask && drafts && lr < rows && w0 + w < words
                                ? a.mask[((int64_t)b * a.T + t) * words + w0 + w] : 0u;
          }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int lr = 8 * nt + 2 * c4 + e, t = (row0 + lr) / a.G;
            uint32_t bits = d0 <= -kTile ? ~0u : d0 >= 0 ? 0u : ~0u >> (int)(kTile + d0);  // the tile's keys
            if (drafts && lr < rows) {
              uint32_t draft = a.mask ? __funnelshift_r(m[nt][e][0], m[nt][e][1], lo)
                                      : t < lo ? 0u : t - lo >= 31 ? ~0u : (2u << (t - lo)) - 1;
              if (hi - lo < 32) draft &= (1u << (hi - lo)) - 1;
              bits |= draft << (int)(lo - d0);
            }
            if (!box0) bits &= 0xFFFF0000u;
            if (!box1) bits &= 0x0000FFFFu;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                if ((bits >> (16 * hf + 8 * j + key_of(g))) & 1u) seen |= 1u << (nt * 8 + hf * 4 + j * 2 + e);
                else s[hf][nt][2 * j + e] = -INFINITY;
              }
          }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int j = 0; j < 2; ++j)  // a key that one of the thread's rows sees
            if (seen & (0x03030303u << (hf * 4 + j * 2))) vtop = fmaxf(vtop, vsc[hf][j]);
      }
      bool up = vtop > vlim;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          up |= fmaxf(fmaxf(s[0][nt][e], s[0][nt][2 + e]), fmaxf(s[1][nt][e], s[1][nt][2 + e])) > rs[nt].thr[e];
      if (__any_sync(0xffffffffu, up)) {
        vlim = INFINITY;
        if (!MASKED) {
#pragma unroll
          for (int k = 4; k < 32; k <<= 1) vtop = fmaxf(vtop, __shfl_xor_sync(0xffffffffu, vtop, k));
        }
        float lv[2][2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int j = 0; j < 2; ++j) lv[hf][j] = lg2f(vsc[hf][j]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float al_o[2], al_l[2], nc[2], dn[2];
          const float2 f = unpair(rs[nt].f), nc_old = unpair(rs[nt].nc), dn_old = unpair(rs[nt].down);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = -INFINITY, weight = -INFINITY, vm = vtop;  // vm: the largest V scale that the row sees
            if (MASKED) {
              vm = 0.0f;
#pragma unroll
              for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                  if ((seen >> (nt * 8 + hf * 4 + j * 2 + e)) & 1u) vm = fmaxf(vm, vsc[hf][j]);
#pragma unroll
              for (int k = 4; k < 32; k <<= 1) vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, k));
            }
            const float fe = e ? f.y : f.x, c_old = -(e ? nc_old.y : nc_old.x), d_old = e ? dn_old.y : dn_old.x;
            const int E_old = 127 - (__float_as_int(d_old) >> 23);
            const int E = min(max(E_old, (__float_as_int(vm) >> 23) - 126), 126);
            dn[e] = __int_as_float((127 - E) << 23);
            vlim = fminf(vlim, __int_as_float((127 + E) << 23));
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
              for (int j = 0; j < 2; ++j) {  // a score that the row does not see is -infinity
                top = fmaxf(top, s[hf][nt][2 * j + e]);
                weight = fmaxf(weight, __fmaf_ru(s[hf][nt][2 * j + e], fe, lv[hf][j]));
              }
#pragma unroll
            for (int k = 4; k < 32; k <<= 1) {
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
              weight = fmaxf(weight, __shfl_xor_sync(0xffffffffu, weight, k));
            }
            const bool none = rs[nt].thr[e] == -INFINITY;
            float c = top == -INFINITY ? (none ? 0.0f : -INFINITY) : tile_offset(top * fe, weight, E);
            if (__any_sync(0xffffffffu, !none && E != E_old)) {
              const float2 l2 = unpair(rs[nt].l);
              float mass = e ? l2.y : l2.x;
#pragma unroll
              for (int k = 4; k < 32; k <<= 1) mass += __shfl_xor_sync(0xffffffffu, mass, k);
              if (!none) c = fmaxf(c, kept_offset(c_old, E - E_old, mass));
            } else if (!none) {
              c = fmaxf(c, c_old);
            }
            al_l[e] = none ? 0.0f : ex2f(c_old - c);
            al_o[e] = none ? 0.0f : ex2f((c_old - c) + (float)(E_old - E));
            if (!none || top != -INFINITY) rs[nt].thr[e] = __fadd_rd(c, kLimit) / fe;
            nc[e] = -c;
          }
          rs[nt].nc = pair(nc[0], nc[1]);
          rs[nt].down = pair(dn[0], dn[1]);
          rs[nt].l = mul2(rs[nt].l, pair(al_l[0], al_l[1]));
#pragma unroll
          for (int x = 0; x < XV; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nt][x][e] *= al_o[e & 1];
        }
      }
      uint32_t pb[2][NT][2];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float2 x = unpair(fma2(pair(s[hf][nt][2 * j], s[hf][nt][2 * j + 1]), rs[nt].f, rs[nt].nc));
            const uint64_t p = pair(ex2f(x.x), ex2f(x.y));
            rs[nt].l = add2(rs[nt].l, p);
            const float2 w = unpair(mul2(p, mul2(pair(vsc[hf][j], vsc[hf][j]), rs[nt].down)));
            if (MASKED) {
              const uint32_t on = seen >> (nt * 8 + hf * 4 + j * 2);
              pb[hf][nt][j] = transpose8x8(pack_f16x2(on & 1u ? w.x : 0.0f, on & 2u ? w.y : 0.0f));
            } else {
              pb[hf][nt][j] = transpose8x8(pack_f16x2(w.x, w.y));
            }
          }
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int x = 0; x < XV; x += 2) {
          uint32_t vw[4];
          ldmatrix_x4_trans(va + 16 * hf * D + swizzled<D>(vkey, x + vchunk), vw);
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            uint32_t fa[4];
            codes_to_f16<VF>(MASKED ? no_nan<VF>(vw[2 * y]) : vw[2 * y], fa[0], fa[1]);
            codes_to_f16<VF>(MASKED ? no_nan<VF>(vw[2 * y + 1]) : vw[2 * y + 1], fa[2], fa[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816(o[nt][x + y], fa, pb[hf][nt][0], pb[hf][nt][1]);
          }
        }
    };

    for (; i < i_end; ++i) {
      const int r0 = row0_of(i), r1 = row1_of(i), s = i % S;
      const float ks = ks_next * a.sl2, vs = vs_next;  // multiplied here: at the load it would wait for it
      if (i + 1 < n_tiles) scales_of(i + 1, ks_next, vs_next);
      if ((r0 >= 0 || r1 >= 0) && i < issued) {
        if (!tc::wait_bounded(&sm.full[warp][s], (phase >> s) & 1u, &abort_flag, a.c.status, kWhereAttn,
                              a.wait_limit, false))
          dead = true;
        phase ^= 1u << s;
        dead = __any_sync(0xffffffffu, dead);
        if (!dead) {
          const int64_t slot0 = (int64_t)(first + i - u.start) * kTile;
          const uint32_t ka = kbase + s * kTile * D, va = vbase + s * kTile * D;
          if (slot0 + kTile <= ctx && r0 >= 0 && r1 >= 0) tile(std::false_type{}, ka, va, ks, vs, slot0, true, true);
          else tile(std::true_type{}, ka, va, ks, vs, slot0, r0 >= 0, r1 >= 0);
        }
      }
      __syncwarp();
      if (issued < n_tiles && !dead) issue(issued++);
      if ((i & 31) == 31) {
        ++block;
        ra0 = rb0;
        ra1 = rb1;
        if (n_tiles > 32 * (block + 1)) rows_of_block(block + 1, rb0, rb1);
      }
    }

    // ---- the unit's rows, or this warp's part of them
    const bool whole = seg == u.start && seg_end == unit_end;
    const int slot = seg == u.start ? 1 : 0;
    // a warp's last part lies in its ring, which is used up
    float* part = seg_end == last ? reinterpret_cast<float*>(sm.k[warp][0]) : sm.head[warp];
    if (!whole) __syncwarp();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float2 l2 = unpair(rs[nt].l);
      const float2 nc = unpair(rs[nt].nc), dn = unpair(rs[nt].down);
#pragma unroll
      for (int k = 4; k < 32; k <<= 1) {
        l2.x += __shfl_xor_sync(0xffffffffu, l2.x, k);
        l2.y += __shfl_xor_sync(0xffffffffu, l2.y, k);
      }
      // elements 0, 2 are columns 2g, 2g + 1 of row 2c, elements 1, 3 of row 2c + 1
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int lr = 8 * nt + 2 * c4 + e;
        const float up = __int_as_float((254 << 23) - __float_as_int(e ? dn.y : dn.x));  // 2^E
        const Mass m = normalised(rs[nt].thr[e] == -INFINITY ? -INFINITY : -(e ? nc.y : nc.x), e ? l2.y : l2.x, kPartBias);
        if (lr >= rows) continue;
        if (whole) {
          const OutRow to(a, b, h, row0 + lr);
          const float f = m.g * row_inverse(m.l);
#pragma unroll
          for (int x = 0; x < XV; ++x)
            *reinterpret_cast<uint32_t*>(to.p + 16 * x + 2 * g) =
                pack_bf16x2(o[nt][x][e] * f * up, o[nt][x][2 + e] * f * up);
          if (g == 0) store_lse(a, b, h, row0 + lr, m.c, m.l);
        } else {
#pragma unroll
          for (int x = 0; x < XV; ++x)
            *reinterpret_cast<float2*>(part + lr * D + 16 * x + 2 * g) =
                make_float2(o[nt][x][e] * m.g * up, o[nt][x][2 + e] * m.g * up);
          if (g == 0) {
            sm.c[warp][slot][lr] = m.c;
            sm.l[warp][slot][lr] = m.l;
          }
        }
      }
    }
    if (!whole && lane == 0 && (slot == 1 || warp == 0)) {
      Cut& k = sm.cut[slot == 1 ? warp : W];
      k.start = u.start;
      k.end = unit_end;
      k.b = b; k.h = h; k.row0 = row0; k.rows = rows;
      k.slot = slot;
      k.sums = part;
    }
    if (!whole && lane == 0 && slot == 0) sm.at0[warp] = part;
    seg = seg_end;
  }

  // ---- join the parts of the units that the warps' borders cut
  __syncthreads();
  constexpr int V4 = D / 4;
  for (int item = threadIdx.x / V4; item < (W + 1) * R; item += Sh::kThreads / V4) {
    const int r = item % R, col = 4 * (threadIdx.x % V4);
    const Cut& cut = sm.cut[item / R];
    if (cut.slot < 0 || r >= cut.rows) continue;
    const int w0 = item / R == W ? 0 : item / R;
    int w1 = w0 + 1;  // parts: (w0, its slot), then slot 0 of the warps up to w1
    while (w1 < W && st.s + w1 * share < min(cut.end, st.e)) ++w1;
    float c = sm.c[w0][cut.slot][r], l = 0.0f;
    for (int w = w0 + 1; w < w1; ++w) c = fmaxf(c, sm.c[w][0][r]);
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int w = w0; w < w1; ++w) {
      const int slot = w == w0 ? cut.slot : 0;
      const float cw = sm.c[w][slot][r], f = cw == -INFINITY ? 0.0f : ex2f(cw - c);
      const float4 x = *reinterpret_cast<const float4*>((w == w0 ? cut.sums : sm.at0[w]) + r * D + col);
      l += sm.l[w][slot][r] * f;
      o.x += x.x * f; o.y += x.y * f; o.z += x.z * f; o.w += x.w * f;
    }
    if (cut.start >= st.s && cut.end <= st.e) {
      store_out(a, cut.b, cut.h, cut.row0 + r, col, o, row_inverse(l));
      if (col == 0) store_lse(a, cut.b, cut.h, cut.row0 + r, c, l);
    } else {
      float* to = part_of<R, D>(a, blockIdx.x, cut.start < st.s ? 0 : 1);
      *reinterpret_cast<float4*>(to + r * D + col) = o;
      if (col == 0) { to[R * D + r] = c; to[R * D + R + r] = l; }
      if (col == 0 && r == 0 && cut.start >= st.s)
        *cut_unit(a, blockIdx.x) = CutUnit{(int)((cut.end - 1) / st.share - blockIdx.x) + 1, cut.b, cut.h, cut.row0, cut.rows};
    }
  }
}

template <int D, int NT, int KF, int VF>
int launch_mma(const CacheAttnArgs& a, cudaStream_t s) {
  using Sh = Shape<D, NT>;
  if (!list_fits<kTile, 8 * NT>(a)) return SAGE_ERR_UNSUPPORTED;
  const uint64_t rows = (uint64_t)a.c.pages * a.c.H << a.c.page_shift;
  CUtensorMap mk, mv;
  if (!tc::make_map(&mk, a.c.codes[0], D, rows, 1, D, rows * D, D, kBox) ||
      !tc::make_map(&mv, a.c.codes[1], D, rows, 1, D, rows * D, D, kBox))
    return SAGE_ERR_CUDA;
  auto* fn = cache_attn_mma_kernel<D, NT, KF, VF>;
  constexpr size_t smem = sizeof(Smem<D, NT>) + 1024;
  static_assert(smem <= 227 * 1024, "shared memory of one CTA");
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return SAGE_ERR_CUDA;
  if (const int rc = launch_dependent(fn, dim3(kMaxCtas), Sh::kThreads, smem, s, mk, mv, a)) return rc;
  return launch_join<kTile, 8 * NT, D, Sh::kWarps>(a, s);
}

template <int D, int NT>
int by_format(const CacheAttnArgs& a, cudaStream_t s) {
  const bool k8 = a.c.format[0] == SAGE_CACHE_INT8, v8 = a.c.format[1] == SAGE_CACHE_INT8;
  if (k8) return v8 ? launch_mma<D, NT, SAGE_CACHE_INT8, SAGE_CACHE_INT8>(a, s) : launch_mma<D, NT, SAGE_CACHE_INT8, SAGE_CACHE_E4M3>(a, s);
  return v8 ? launch_mma<D, NT, SAGE_CACHE_E4M3, SAGE_CACHE_INT8>(a, s) : launch_mma<D, NT, SAGE_CACHE_E4M3, SAGE_CACHE_E4M3>(a, s);
}

template <int D>
int by_rows(const CacheAttnArgs& a, cudaStream_t s) {
  const int rows = a.T * a.G;
  return rows <= 8 ? by_format<D, 1>(a, s) : by_format<D, 2>(a, s);
}

}  // namespace

size_t cache_attn_workspace_bytes() { return kPartBytes + kCutBytes; }

int launch_cache_attn(const CacheAttnArgs& a, cudaStream_t s) {
  // The tcgen05 variant takes 128 rows at once at nearly the time of 16; this one reads and converts the cache again for
  // each 16.  Measured on B200 (us here against there, cold L2, 16 sequences of 500..16384, 8 heads): D = 128: 16 rows
  // 101 / 167, 32 rows 169 / 169, 40 rows 220 / 169; D = 64: 32 rows 105 / 154, 48 rows 132 / 157, 56 rows 161 / 157.
  if (a.T * a.G > (a.c.D == 128 ? 32 : 48)) return launch_cache_attn_tc(a, s);
  return a.c.D == 128 ? by_rows<128>(a, s) : by_rows<64>(a, s);
}

}  // namespace sage
