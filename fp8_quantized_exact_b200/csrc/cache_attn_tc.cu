// Attention of drafted tokens over the quantised paged cache with many rows per
// head of the cache: tcgen05 FP16 MMAs with FP32 sums in tensor memory.
//
// The mathematics is that of cache_attn.cu: S = Q K^T and O = P V with the codes
// exact in FP16, Q rows scaled by a power of two, FP32 statistics, a lazily
// raised offset c, probabilities times V scales 2^-E rounded to FP16.  Here a
// unit is up to 128 rows, the M of the MMAs, and a tile is 64 keys.
//
// One CTA per SM, with fixed roles:
//   warps 0-3, 4-7   two independent softmax streams, on alternate tiles, each
//                    with its own O accumulator and its own c, l and E (joined at the
//                    end of the unit, like split keys): one stream's softmax runs
//                    beside the other's MMAs and nothing is handed over.  A thread
//                    owns a row.  It also converts half of the row's Q at the
//                    start of a unit and stores half of its output at the end, and
//                    multiplies its O row when c or E is raised, which is rare.
//   warps 8-15       converters: raw K and V codes of a tile -> FP16 tiles in the
//                    128-byte swizzle that the MMAs read (K K-major, V MN-major).
//   warps 16, 17     TMA producers of raw K and V tiles (one box per page that the
//                    tile touches) and of their scales (bulk copies).
//   warps 18, 19     QK and PV issuers; P is the TMEM A operand of PV.
// Channels are in the order 0, 2, 1, 3 within each four, in Q, K and V alike, as the
// conversion yields them; the output undoes it.
//
// Every wait is bounded; one that runs out records SAGE_ERR_TIMEOUT, raises the
// CTA's abort flag, and every role leaves its loop and drains what it has in flight.
#include "cache_attn.cuh"
#include "cache_codes.cuh"
#include "tc_prims.cuh"

namespace sage {
namespace {

using namespace cattn;
using namespace tc;

constexpr int kRowsT = 128, kTileT = 64;
constexpr int kConv0 = 8, kConvWarps = 8, kLoadK = kConv0 + kConvWarps, kLoadV = kLoadK + 1, kQkWarpT = kLoadK + 2,
              kPvWarpT = kLoadK + 3;
constexpr int kThreadsT = 32 * (kPvWarpT + 1);
constexpr int kKStages = 2, kVStages = 4;
constexpr int kScales = 16;    // scale ring: softmax has read a tile's slot before its successor's loads are issued
constexpr uint32_t kColsT = 512, kColOT = 256;  // TMEM: S buffers [stream][2] of 64 columns, then O of each stream

template <int D>
struct SmemT {
  static constexpr int kRaw = D == 128 ? 5 : 8;
  alignas(1024) uint8_t q[kRowsT * D * 2];
  alignas(1024) uint8_t k[kKStages][kTileT * D * 2];
  alignas(1024) uint8_t v[kVStages][kTileT * D * 2];
  alignas(1024) uint8_t raw[kRaw][2][kTileT * D];
  alignas(128) float scale[kScales][2][kTileT];
  alignas(16) float vd[kScales][kTileT];  // V scales times 2^-E of the tile (tiles that every row sees whole)
  int e[kScales];                       // that E
  uint32_t amax[2][kRowsT];             // of the halves of Q's rows
  float c[2][kRowsT], l[2][kRowsT], up[2][kRowsT];  // what the streams exchange at a unit's end
  int flags[kScales];                   // bits 0-3: the 16-key groups that hold keys; bit 4: not every row sees every key; bit 5: a unit's first tile
  uint64_t raw_full[kRaw], raw_empty[kRaw];
  uint64_t k_full[kKStages], k_empty[kKStages], v_full[kVStages], v_empty[kVStages];
  uint64_t s_full[2][2], p_full[2][2], o_done[2][2];  // [stream][its tiles mod 2]
  uint64_t q_full, swap, drain[2];
  uint32_t tmem_base;
  int abort_flag;
};
constexpr int kMasked = 16, kFirst = 32;

// E for a largest V scale, by its bits (NaN left out by the callers): 2^E is above it.
__device__ __forceinline__ int v_exponent(uint32_t bits) { return min((int)(bits >> 23) - 126, 126); }

// Descriptor of a 128-byte-swizzled tile: `lbo` and `sbo` in bytes.
__device__ __forceinline__ uint64_t desc128(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | (uint64_t)(lbo >> 4) << 16 | (uint64_t)(sbo >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// FP16 x FP16 -> FP32, M = 128; `mn` where B is MN-major.
__host__ __device__ constexpr uint32_t idesc_f16(int n, bool mn) {
  return (1u << 4) | (mn ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kRowsT >> 4) << 24);
}
// The issuing warps run converged and predicate the instruction itself on the
// one lane `on`, so that the operands stay in uniform registers: inside a branch
// on the lane each MMA took about 80 cycles to issue.
__device__ __forceinline__ void mma_f16_ss(uint32_t on, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{.reg .pred p, q; setp.ne.b32 p, %4, 0; setp.ne.b32 q, %5, 0;"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(on)
      : "memory");
}
__device__ __forceinline__ void mma_f16_ts(uint32_t on, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{.reg .pred p, q; setp.ne.b32 p, %4, 0; setp.ne.b32 q, %5, 0;"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(on)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t on, uint64_t* b) {
  asm volatile(
      "{.reg .pred q; setp.ne.b32 q, %1, 0;"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];}" ::"r"(smem_u32(b)),
      "r"(on)
      : "memory");
}
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// One 64-key tile of raw codes -> FP16 in the MMA layout: 64-channel blocks of
// [key][128 bytes].  Warp w of the converters takes the keys 8 w .. 8 w + 7.
template <int D, int F>
__device__ __forceinline__ void convert(uint32_t raw, uint32_t to, int w, int lane, bool clean) {
  const int c = lane & 3, key = 8 * w + key_of(lane >> 2);
  uint4 in[D / 64];
#pragma unroll
  for (int x = 0; x < D / 64; ++x) in[x] = lds128(raw + swizzled<D>(key, 4 * x + c));
  if (F == SAGE_CACHE_E4M3 && clean) {
#pragma unroll
    for (int x = 0; x < D / 64; ++x)
      in[x] = make_uint4(no_nan<F>(in[x].x), no_nan<F>(in[x].y), no_nan<F>(in[x].z), no_nan<F>(in[x].w));
  }
#pragma unroll
  for (int x = 0; x < D / 64; ++x) {
    uint32_t o[8];
    const uint32_t iw[4] = {in[x].x, in[x].y, in[x].z, in[x].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) codes_to_f16<F>(iw[e], o[2 * e], o[2 * e + 1]);
    const uint32_t row = to + x * (kTileT * 128) + key * 128;
    sts128(row + (((2 * c) ^ (key & 7)) << 4), o[0], o[1], o[2], o[3]);
    sts128(row + (((2 * c + 1) ^ (key & 7)) << 4), o[4], o[5], o[6], o[7]);
  }
}

template <int D, int KF, int VF>
__global__ void __launch_bounds__(kThreadsT, 1)
    cache_attn_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                         const CacheAttnArgs a) {
  constexpr int NR = SmemT<D>::kRaw, DH = D / 2, BLK = kTileT * 128;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  SmemT<D>& sm = *reinterpret_cast<SmemT<D>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &sm.abort_flag;
  DeviceStatus* status = a.c.status;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Stretch st = find_stretch<kTileT, kRowsT, 1>(a, blockIdx.x, gridDim.x);
  if (blockIdx.x == 0)  // lengths that cannot be
    for (int b = threadIdx.x; b < a.B; b += kThreadsT) {
      const int ctx = a.context[b], cnt = a.count ? a.count[b] : a.T;
      if (ctx < 0 || cnt < 0 || cnt > a.T ||
          (long long)ctx + cnt > ((long long)a.c.table_pages << a.c.page_shift))
        flag_bad(status, kWhereAttn);
    }
  if (st.s >= st.e) return;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NR; ++s) {
      mbar_init(&sm.raw_full[s], 2);  // both producers
      mbar_init(&sm.raw_empty[s], kConvWarps);
    }
    for (int s = 0; s < kKStages; ++s) {
      mbar_init(&sm.k_full[s], kConvWarps);
      mbar_init(&sm.k_empty[s], 1);
    }
    for (int s = 0; s < kVStages; ++s) {
      mbar_init(&sm.v_full[s], kConvWarps);
      mbar_init(&sm.v_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      for (int k = 0; k < 2; ++k) {
        mbar_init(&sm.s_full[s][k], 1);
        mbar_init(&sm.p_full[s][k], 4);
        mbar_init(&sm.o_done[s][k], 1);
      }
    }
    mbar_init(&sm.q_full, 256);
    mbar_init(&sm.swap, 256);
    mbar_init(&sm.drain[0], 1);
    mbar_init(&sm.drain[1], 1);
    sm.abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kQkWarpT) tmem_alloc(&sm.tmem_base, kColsT);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  const int n_tiles = (int)(st.e - st.s);
  // the phase of number `phase` of a barrier, by a whole warp
  auto wait = [&](uint64_t* bar, uint32_t phase, int where) -> bool {
    return __all_sync(0xffffffffu, wait_bounded(bar, phase & 1u, abort_flag, status, 100 + where, kDefaultWaitLimit));
  };

  if (warp < kConv0) {
    // ------------------------------------------------------ softmax streams
    const int sid = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16), col_o = lanes + kColOT + sid * D;
    float* vd = sm.vd[warp];
    uint32_t swaps = 0;
    bool ok = true;
    Place at = place_of<kTileT, kRowsT>(a, st.s);
    for (unsigned seg = st.s; ok && seg < st.e;) {
      go_to<kTileT, kRowsT>(a, at, seg);
      const Unit u = unit_of(at, seg);
      const int b = at.b, h = u.h, row0 = u.rt * kRowsT, ctx = at.s.ctx, cnt = at.s.cnt;
      const int rows = min(kRowsT, cnt * a.G - row0);
      const unsigned unit_end = u.start + at.s.n, seg_end = min(unit_end, st.e);
      const int token = min((row0 + row) / a.G, a.T - 1);
      const bool idle = (warp & 3) * 32 >= rows;  // no row of this warp

      // ---- this thread's half of its Q row: FP16, channels 0, 2, 1, 3 of each four, 128-byte swizzle
      float f;
      {
        uint4 w[DH / 8];
        uint32_t top = 0;
        const uint16_t* q = a.q + b * a.qb + token * a.qn + (h * a.G + (row0 + row) % a.G) * a.qh + sid * DH;
#pragma unroll
        for (int x = 0; x < DH / 8; ++x) {
          w[x] = make_uint4(0, 0, 0, 0);
          if (row < rows) w[x] = __ldg(reinterpret_cast<const uint4*>(q + 8 * x));
          const uint32_t ww[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) top = max(top, max(ww[e] & 0x7FFFu, (ww[e] >> 16) & 0x7FFFu));
        }
        sm.amax[sid][row] = top;
        mbar_arrive(&sm.swap);
        // past this wait every thread has finished the unit before, whose QK MMAs are done
        if (!(ok = wait(&sm.swap, swaps++, 0))) break;
        top = max(top, sm.amax[sid ^ 1][row]);
        const int eq = q_exponent(top);
        const float down = __int_as_float((127 - eq) << 23);
        f = q_factor(a.sl2, eq);
        const uint32_t qa = smem_u32(sm.q) + row * 128;
#pragma unroll
        for (int x = 0; x < DH / 8; ++x) {
          const uint32_t ww[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            o[e] = pack_f16x2(__uint_as_float(ww[e] << 16) * down, __uint_as_float(ww[e + 1] << 16) * down);
            o[e + 1] = pack_f16x2(__uint_as_float(ww[e] & 0xFFFF0000u) * down, __uint_as_float(ww[e + 1] & 0xFFFF0000u) * down);
          }
          const int ch = sid * (DH / 8) + x;  // 16-byte chunk of the row
          sts128(qa + (ch >> 3) * (kRowsT * 128) + (((ch & 7) ^ (row & 7)) << 4), o[0], o[1], o[2], o[3]);
        }
        fence_async_smem();
        tc_fence_before();
        mbar_arrive(&sm.q_full);
      }
      const uint64_t f2 = pair(f, f);
      float c = 0.0f;
      bool none = true;  // nothing seen yet
      uint64_t l0 = 0, l1 = 0;
      int E = -126;
      bool fresh = true;  // no PV of this unit yet: the accumulator holds nothing

      // one tile; first and later ones, seen whole by every row or masked
      auto tile = [&](auto masked_tag, uint32_t cols, int slot, int k, uint64_t seen, int E_new) {
        constexpr bool MASKED = decltype(masked_tag)::value;
        const float* ks = sm.scale[slot][0];
        const float* vs = MASKED ? sm.scale[slot][1] : sm.vd[slot];
        const float down = __int_as_float((127 - E_new) << 23);
        // c is raised until a row has seen something, with E, and where the sum of a tile's p passes 2^14 (so that FP16 holds each of
        // them); the tile is then done again
        bool raise = MASKED || __any_sync(0xffffffffu, none || E_new != E);
        uint32_t p[32];
        uint64_t s0, s1;
        for (;;) {
          uint32_t sa[16], sb[16];
          if (raise) {
            float top = -INFINITY;
#pragma unroll
            for (int j0 = 0; j0 < 64; j0 += 16) {
              tmem_ld16(cols + j0, sa);
              tmem_wait_ld16(sa);
#pragma unroll
              for (int j = 0; j < 16; j += 4) {
                const float4 kk = *reinterpret_cast<const float4*>(ks + j0 + j);
                const float x[4] = {__uint_as_float(sa[j]) * kk.x, __uint_as_float(sa[j + 1]) * kk.y,
                                    __uint_as_float(sa[j + 2]) * kk.z, __uint_as_float(sa[j + 3]) * kk.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (!MASKED || (seen >> (j0 + j + e)) & 1) top = fmaxf(top, x[e]);
              }
            }
            const float c_new = none ? (top == -INFINITY ? 0.0f : top * f) : fmaxf(c, top * f);
            const float al = none ? 0.0f : ex2(c - c_new), al_o = E_new == E ? al : al * ex2((float)(E - E_new));
            none = none && top == -INFINITY;
            c = c_new;
            E = E_new;
            l0 = mul2(l0, pair(al, al));
            l1 = mul2(l1, pair(al, al));
            if (!fresh && __any_sync(0xffffffffu, al_o != 1.0f)) {
              // the PV before is done first, then the accumulator's row is multiplied
              if (!(ok = wait(&sm.o_done[sid][(k - 1) & 1], (k - 1) >> 1, 3))) return;
              tc_fence_after();
#pragma unroll 1
              for (int x = 0; x < D; x += 16) {
                tmem_ld16(col_o + x, sa);
                tmem_wait_ld16(sa);
#pragma unroll
                for (int e = 0; e < 16; ++e) sa[e] = __float_as_uint(__uint_as_float(sa[e]) * al_o);
                tmem_st16(col_o + x, sa);
              }
            }
          }
          const uint64_t nc2 = pair(-c, -c);
          s0 = s1 = 0;
          // 16 keys from j0 on
          auto chunk = [&](const uint32_t (&sr)[16], int j0) {
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              const float4 kk = *reinterpret_cast<const float4*>(ks + j0 + j);
              float4 v = *reinterpret_cast<const float4*>(vs + j0 + j);
              uint64_t x0 = mul2(pair(__uint_as_float(sr[j]), __uint_as_float(sr[j + 1])), pair(kk.x, kk.y));
              uint64_t x1 = mul2(pair(__uint_as_float(sr[j + 2]), __uint_as_float(sr[j + 3])), pair(kk.z, kk.w));
              x0 = fma2(x0, f2, nc2);
              x1 = fma2(x1, f2, nc2);
              float2 a0 = unpair(x0), a1 = unpair(x1);
              if (MASKED) {
                const uint32_t on = (uint32_t)(seen >> (j0 + j));
                if (!(on & 1)) { a0.x = -INFINITY; v.x = 0.0f; }
                if (!(on & 2)) { a0.y = -INFINITY; v.y = 0.0f; }
                if (!(on & 4)) { a1.x = -INFINITY; v.z = 0.0f; }
                if (!(on & 8)) { a1.y = -INFINITY; v.w = 0.0f; }
                v.x *= down; v.y *= down; v.z *= down; v.w *= down;
              }
              const uint64_t p0 = pair(ex2(a0.x), ex2(a0.y)), p1 = pair(ex2(a1.x), ex2(a1.y));
              s0 = add2(s0, p0);
              s1 = add2(s1, p1);
              const float2 w0 = unpair(mul2(p0, pair(v.x, v.y))), w1 = unpair(mul2(p1, pair(v.z, v.w)));
              p[(j0 + j) / 2] = pack_f16x2(w0.x, w0.y);
              p[(j0 + j) / 2 + 1] = pack_f16x2(w1.x, w1.y);
            }
          };
          tmem_ld16(cols, sa);
          tmem_wait_ld16(sa);
          tmem_ld16(cols + 16, sb);
          chunk(sa, 0);
          tmem_wait_ld16(sb);
          tmem_ld16(cols + 32, sa);
          chunk(sb, 16);
          tmem_wait_ld16(sa);
          tmem_ld16(cols + 48, sb);
          chunk(sa, 32);
          tmem_wait_ld16(sb);
          chunk(sb, 48);
          if (raise) break;
          const float2 y = unpair(add2(s0, s1));
          raise = __any_sync(0xffffffffu, !(y.x + y.y <= 16384.0f));
          if (!raise) break;
        }
        l0 = add2(l0, s0);
        l1 = add2(l1, s1);
        tmem_st16(cols, *reinterpret_cast<const uint32_t(*)[16]>(&p[0]));
        tmem_st16(cols + 16, *reinterpret_cast<const uint32_t(*)[16]>(&p[16]));
        tmem_wait_st();
      };

      // ---- tiles of this stream
      int i = (int)(seg - st.s);
      i += (i & 1) ^ sid;
      for (; i < (int)(seg_end - st.s); i += 2) {
        const int k = i >> 1, buf = k & 1, slot = i & (kScales - 1);
        if (!(ok = wait(&sm.s_full[sid][buf], k >> 1, 2))) break;
        tc_fence_after();
        const uint32_t cols = lanes + (sid * 2 + buf) * 64;
        if (!idle) {
          const int flags = sm.flags[slot];
          if (!(flags & kMasked)) {
            tile(std::false_type{}, cols, slot, k, ~0ull, sm.e[slot]);
          } else {
            const int64_t slot0 = (int64_t)(st.s + i - u.start) * kTileT;
            const int64_t d0 = slot0 - ctx;  // drafted token of the tile's first key (below 0: context)
            uint64_t seen = d0 <= -64 ? ~0ull : d0 >= 0 ? 0ull : ~0ull >> (64 + d0);
            if (row < rows && d0 < cnt && d0 > -64) {
              const int lo = (int)max(d0, (int64_t)0), hi = min((int)(d0 + 64), cnt);  // drafted tokens [lo, hi)
              uint64_t bits = 0;  // of tokens lo, lo + 1, ...
              if (a.mask) {
                const int words = (a.T + 31) / 32;
                const uint32_t* m = a.mask + ((int64_t)b * a.T + token) * words;
                for (int w = lo / 32; w <= (hi - 1) / 32; ++w) {
                  const uint64_t word = __ldg(m + w);
                  bits |= 32 * w >= lo ? word << (32 * w - lo) : word >> (lo - 32 * w);
                }
              } else if (token >= lo) {
                bits = token - lo >= 63 ? ~0ull : (2ull << (token - lo)) - 1;
              }
              if (hi - lo < 64) bits &= (1ull << (hi - lo)) - 1;
              seen |= bits << (lo - (int)d0);
            }
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (!((flags >> x) & 1)) seen &= ~(0xFFFFull << (16 * x));
            float vm = 0.0f;
            for (int j = 0; j < 64; ++j)
              if ((seen >> j) & 1) vm = fmaxf(vm, sm.scale[slot][1][j]);
            tile(std::true_type{}, cols, slot, k, seen, max(E, v_exponent(__float_as_uint(vm))));
          }
          if (!ok) break;
        }
        fresh = false;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[sid][buf]);
      }
      if (!ok) break;

      // ---- the unit's end: wait for this stream's last PV, exchange the states, store half of the columns
      if (!fresh) {
        const int last = ((int)(seg_end - st.s) - 1 - sid) >> 1;  // the stream's tile before the end
        if (!(ok = wait(&sm.o_done[sid][last & 1], last >> 1, 4))) break;
      }
      float l;
      {
        const float2 x = unpair(l0), y = unpair(l1);
        l = (x.x + x.y) + (y.x + y.y);
      }
      sm.l[sid][row] = l;
      sm.c[sid][row] = none ? -INFINITY : c;
      sm.up[sid][row] = fresh ? 0.0f : __int_as_float((127 + E) << 23);  // 2^E; 0: the accumulator holds nothing
      tc_fence_before();
      mbar_arrive(&sm.swap);
      if (!(ok = wait(&sm.swap, swaps++, 5))) break;
      tc_fence_after();
      if (!idle) {
        const float ca = sm.c[0][row], cb = sm.c[1][row], cm = fmaxf(ca, cb);
        const float wa = ca == -INFINITY ? 0.0f : ex2(ca - cm), wb = cb == -INFINITY ? 0.0f : ex2(cb - cm);
        l = sm.l[0][row] * wa + sm.l[1][row] * wb;
        const bool has_a = sm.up[0][row] != 0.0f, has_b = sm.up[1][row] != 0.0f;
        const bool whole = seg == u.start && seg_end == unit_end, on = row < rows;
        const float inv = whole ? row_inverse(l) : 1.0f;
        const float fa = wa * sm.up[0][row] * inv, fb = wb * sm.up[1][row] * inv;
        const OutRow out(a, b, h, min(row0 + row, cnt * a.G - 1));
        float* part = part_of<kRowsT, D>(a, blockIdx.x, seg == u.start ? 1 : 0);
#pragma unroll 1
        for (int x = 0; x < DH; x += 16) {
          const int col = sid * DH + x;
          uint32_t oa[16], ob[16];
          tmem_ld16(lanes + kColOT + col, oa);
          tmem_ld16(lanes + kColOT + D + col, ob);
          tmem_wait_ld16(oa);
          tmem_wait_ld16(ob);
          float o[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            o[e] = (has_a ? __uint_as_float(oa[e]) * fa : 0.0f) + (has_b ? __uint_as_float(ob[e]) * fb : 0.0f);
          if (on && whole) {
#pragma unroll
            for (int e = 0; e < 16; e += 8)
              *reinterpret_cast<uint4*>(out.p + col + e) =
                  make_uint4(pack_bf16x2(o[e], o[e + 2]), pack_bf16x2(o[e + 1], o[e + 3]),
                             pack_bf16x2(o[e + 4], o[e + 6]), pack_bf16x2(o[e + 5], o[e + 7]));
          } else if (on) {
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              *reinterpret_cast<float4*>(part + row * D + col + e) = make_float4(o[e], o[e + 2], o[e + 1], o[e + 3]);
          }
        }
        if (on && sid == 0) {
          if (whole) {
            store_lse(a, b, h, row0 + row, cm, l);
          } else {
            part[kRowsT * D + row] = cm;
            part[kRowsT * D + kRowsT + row] = l;
          }
        }
      }
      tc_fence_before();
      seg = seg_end;
    }
  } else if (warp < kLoadK) {
    // ----------------------------------------------------------- converters
    const int w = warp - kConv0;
    int E = -126;  // of the tiles so far that every row sees whole
    for (int i = 0; i < n_tiles; ++i) {
      const int r = i % NR, slot = i & (kScales - 1);
      if (!wait(&sm.raw_full[r], i / NR, 6)) break;
      const int flags = sm.flags[slot];
      const bool clean = flags & kMasked;
      if (w == 0) {
        if (flags & kFirst) E = -126;
        if (!clean) {
          const float v0 = sm.scale[slot][1][lane], v1 = sm.scale[slot][1][lane + 32];
          E = max(E, v_exponent(__reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(fmaxf(v0, v1), 0.0f)))));
          const float down = __int_as_float((127 - E) << 23);
          sm.vd[slot][lane] = v0 * down;
          sm.vd[slot][lane + 32] = v1 * down;
          if (lane == 0) sm.e[slot] = E;
        }
      }
      if (!wait(&sm.k_empty[i % kKStages], (i / kKStages) ^ 1, 7)) break;
      convert<D, KF>(smem_u32(sm.raw[r][0]), smem_u32(sm.k[i % kKStages]), w, lane, false);
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.k_full[i % kKStages]);
      if (!wait(&sm.v_empty[i % kVStages], (i / kVStages) ^ 1, 8)) break;
      convert<D, VF>(smem_u32(sm.raw[r][1]), smem_u32(sm.v[i % kVStages]), w, lane, clean);
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sm.v_full[i % kVStages]);
        mbar_arrive(&sm.raw_empty[r]);
      }
    }
  } else if (warp <= kLoadV) {
    // ------------------------------------------------------------ producers
    // A tile's boxes are 16, 32 or 64 keys, what a page holds of it.  Lane 4 t + x looks up the row of group x of 16 keys
    // of tile t of the next eight; the first group of a box stands for it.
    const int side = warp - kLoadK, box = min(1 << a.c.page_shift, kTileT), per = box / 16;
    const CUtensorMap* map = side ? &tm_v : &tm_k;
    Place walk = place_of<kTileT, kRowsT>(a, st.s);
    int issued = 0, rows8 = -1;
    bool masked8 = false, first8 = false;
    for (int i = 0; i < n_tiles; ++i) {
      const int r = i % NR, slot = i & (kScales - 1);
      if ((i & 7) == 0) {
        const unsigned idx = st.s + i + (lane >> 2);
        rows8 = -1;
        masked8 = true;
        if (idx < st.e) {
          go_to<kTileT, kRowsT>(a, walk, idx);
          const Unit u = unit_of(walk, idx);
          const int64_t first = (int64_t)(idx - u.start) * kTileT, s = first + 16 * (lane & 3);
          masked8 = first + kTileT > walk.s.ctx;
          first8 = idx == max(u.start, st.s);
          if (s < (int64_t)walk.s.ctx + walk.s.cnt) {
            rows8 = (int)cache_row(a.c, walk.b, u.h, s);
            if (rows8 < 0) flag_bad(status, kWhereAttn);
          }
        }
      }
      const int row = __shfl_sync(0xffffffffu, rows8, 4 * (i & 7) + (lane & 3));
      const bool masked = __shfl_sync(0xffffffffu, masked8, 4 * (i & 7));
      const bool begins = __shfl_sync(0xffffffffu, first8, 4 * (i & 7));
      const uint32_t valid = __ballot_sync(0xffffffffu, lane < 4 && row >= 0);
      const uint32_t boxes = __ballot_sync(0xffffffffu, lane < 4 && row >= 0 && lane % per == 0);
      if (!wait(&sm.raw_empty[r], (i / NR) ^ 1, 9)) break;
      if (lane == 0) {
        if (side == 0) sm.flags[slot] = (int)valid | (masked || valid != 15u ? kMasked : 0) | (begins ? kFirst : 0);
        mbar_expect_tx(&sm.raw_full[r], __popc(boxes) * box * (D + 4));
      }
      __syncwarp();
      if ((boxes >> lane) & 1u) {
        tma_load_3d(sm.raw[r][side] + lane * 16 * D, map, 0, row, 0, &sm.raw_full[r]);
        bulk_load(&sm.scale[slot][side][lane * 16], a.c.scale[side] + row, box * 4, &sm.raw_full[r]);
      }
      issued = i + 1;
    }
    for (int i = max(0, issued - NR); i < issued; ++i)
      wait_bounded(&sm.raw_full[i % NR], (uint32_t)((i / NR) & 1), abort_flag, nullptr, 110, kDefaultWaitLimit, false);
  } else {
    // -------------------------------------------------------------- issuers
    const uint32_t leader = lane == 0;
    Place at = place_of<kTileT, kRowsT>(a, st.s);
    unsigned seg_end = st.s;  // of the unit that tile i belongs to
    int units = 0, begin = 0;
    for (int i = 0; i < n_tiles; ++i) {
      const int s = i & 1, k = i >> 1;
      const uint32_t sc = tmem + (s * 2 + (k & 1)) * 64;
      const bool next = st.s + i == seg_end;
      if (next) {
        go_to<kTileT, kRowsT>(a, at, st.s + i);
        const Unit u = unit_of(at, st.s + i);
        seg_end = min(u.start + at.s.n, st.e);
        begin = i;
      }
      if (warp == kQkWarpT) {
        // a new unit's Q; S buffer k & 1 of the stream: PV of the tile two back in the stream has read its P
        if (next && !wait(&sm.q_full, units++, 13)) break;
        if (k >= 2 && !wait(&sm.o_done[s][k & 1], (k >> 1) - 1, 14)) break;
        if (!wait(&sm.k_full[i % kKStages], i / kKStages, 15)) break;
        tc_fence_after();
        const uint64_t qd = desc128(smem_u32(sm.q), 16, 1024), kd = desc128(smem_u32(sm.k[i % kKStages]), 16, 1024);
#pragma unroll
        for (int x = 0; x < D / 16; ++x)
          mma_f16_ss(leader, sc, qd + (x / 4) * ((kRowsT * 128) >> 4) + 2 * (x % 4),
                     kd + (x / 4) * (BLK >> 4) + 2 * (x % 4), idesc_f16(kTileT, false), x > 0);
        commit(leader, &sm.s_full[s][k & 1]);
        commit(leader, &sm.k_empty[i % kKStages]);
      } else {
        if (!wait(&sm.v_full[i % kVStages], i / kVStages, 12) || !wait(&sm.p_full[s][k & 1], k >> 1, 11)) break;
        tc_fence_after();
        const uint64_t vd = desc128(smem_u32(sm.v[i % kVStages]), BLK, 1024);
        const uint32_t o = tmem + kColOT + s * D, more = i >= begin + 2;  // the unit's first tile of a stream starts its O
#pragma unroll
        for (int x = 0; x < kTileT / 16; ++x)
          mma_f16_ts(leader, o, sc + 8 * x, vd + x * (2048 >> 4), idesc_f16(D, true), x > 0 ? 1u : more);
        commit(leader, &sm.o_done[s][k & 1]);
        commit(leader, &sm.v_empty[i % kVStages]);
      }
    }
    __syncwarp();
    uint64_t* drain = &sm.drain[warp - kQkWarpT];
    commit(leader, drain);
    wait_bounded(drain, 0, abort_flag, nullptr, 116, kDefaultWaitLimit, false);
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kQkWarpT) tmem_free(tmem, kColsT);
}

template <int D, int KF, int VF>
int launch_tc(const CacheAttnArgs& a, cudaStream_t s) {
  if (!list_fits<kTileT, kRowsT>(a)) return SAGE_ERR_UNSUPPORTED;
  const uint64_t rows = (uint64_t)a.c.pages * a.c.H << a.c.page_shift;
  const uint32_t box = a.c.page_shift < 6 ? 1u << a.c.page_shift : kTileT;
  CUtensorMap mk, mv;
  if (!make_map(&mk, a.c.codes[0], D, rows, 1, D, rows * D, D, box) ||
      !make_map(&mv, a.c.codes[1], D, rows, 1, D, rows * D, D, box))
    return SAGE_ERR_CUDA;
  auto* fn = cache_attn_tc_kernel<D, KF, VF>;
  // more than half of an SM's shared memory: one CTA (and one request for all of the TMEM) per SM
  constexpr size_t need = sizeof(SmemT<D>) + 1024, smem = need > 120 * 1024 ? need : 120 * 1024;
  static_assert(smem <= 227 * 1024, "shared memory of one CTA");
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return SAGE_ERR_CUDA;
  fn<<<kMaxCtas, kThreadsT, smem, s>>>(mk, mv, a);
  if (cudaGetLastError() != cudaSuccess) return SAGE_ERR_CUDA;
  return launch_join<kTileT, kRowsT, D, 1>(a, s);
}

template <int D>
int by_format_tc(const CacheAttnArgs& a, cudaStream_t s) {
  const bool k8 = a.c.format[0] == SAGE_CACHE_INT8, v8 = a.c.format[1] == SAGE_CACHE_INT8;
  if (k8) return v8 ? launch_tc<D, SAGE_CACHE_INT8, SAGE_CACHE_INT8>(a, s) : launch_tc<D, SAGE_CACHE_INT8, SAGE_CACHE_E4M3>(a, s);
  return v8 ? launch_tc<D, SAGE_CACHE_E4M3, SAGE_CACHE_INT8>(a, s) : launch_tc<D, SAGE_CACHE_E4M3, SAGE_CACHE_E4M3>(a, s);
}

}  // namespace

int launch_cache_attn_tc(const CacheAttnArgs& a, cudaStream_t s) {
  return a.c.D == 128 ? by_format_tc<128>(a, s) : by_format_tc<64>(a, s);
}

}  // namespace sage
