// Attention of drafted tokens over the quantised paged cache with many rows per
// head of the cache: tcgen05 FP16 MMAs with FP32 sums in tensor memory.
//
// The mathematics is that of cache_attn.cu: S = Q K^T and O = P V with the codes
// exact in FP16, Q rows scaled by a power of two, FP32 statistics, a lazily
// set offset c, probabilities times V scales 2^-E rounded to FP16.  Here a
// unit is up to 128 rows, the M of the MMAs, and a tile is 64 keys.
//
// One CTA per SM, with fixed roles:
//   warps 0-3, 4-7   two independent softmax streams, on alternate tiles, each
//                    with its own O accumulator and its own c, l and E (joined at the
//                    end of the unit, like split keys): one stream's softmax runs
//                    beside the other's MMAs and nothing is handed over.  They work on
//                    S in MMA fragment order (a quarter of the keys of four rows
//                    per thread), write Q (half a row each) to TMEM at the start of a
//                    unit, store half of the output each at its end, and multiply their
//                    O rows when c or E is raised, which is rare.
//   warps 8-11       converters of K: raw codes of a tile -> an FP16 tile in the
//   warps 12-15      and of V: 128-byte swizzle that the MMAs read (V MN-major).
//   warps 16, 17     TMA producers of raw K and V tiles (one box per page that the
//                    tile touches) and of their scales (bulk copies).
//   warps 18, 19     QK and PV issuers; the A operands, Q and P, are in TMEM.
// What bounds it: the instructions and waits of the roles, not a pipe.  A tile of 64
// keys takes 1,600 (64 drafted tokens over 4 contexts of 20000..37810: tensor pipe 32% busy,
// issue slots 62%) to 1,900 cycles (21 over 16 of 500..16384: 27%, 53%) on an SM, with about 1,000
// instructions per scheduler, and little less at 16 rows; an M = 128 MMA costs its issuer about 65
// cycles for any N up to 128.  272 bytes of registers are spilled (96 a thread), mostly by the masked form.
// Four roles share the way of instructions to the SM, so their layout counts: see set_offsets and
// MaskedRows.  Tried and not kept, as factors of the time of 64 drafted
// tokens over 4 contexts of 20000..37810 (424 us then, 449 to 469 by the box now): pairs of tiles per QK MMA 1.27, P in
// columns of its own with Q in shared memory 1.05, one QK issuer per stream 1.25,
// both score loads of a half before one wait 1.12, two converter warps per side
// instead of four 1.22, 32x32b loads with every scale read by every thread 1.15.
// Channels are in the order 0, 2, 1, 3 within each four, in Q, K and V alike, as the
// conversion yields them; the output undoes it.
//
// Every wait is bounded; one that runs out records SAGE_ERR_TIMEOUT, raises the
// CTA's abort flag, and every role leaves its loop and drains what it has in flight.
#include <type_traits>

#include "cache_attn.cuh"
#include "cache_codes.cuh"
#include "tc_prims.cuh"

namespace sage {
namespace {

using namespace cattn;
using namespace tc;

constexpr int kRowsT = 128, kTileT = 64;
constexpr int kConvK = 8, kConvV = 12, kConvWarps = 4, kLoadK = 16, kLoadV = 17, kQkWarpT = 18, kPvWarpT = 19;
constexpr int kThreadsT = 32 * (kPvWarpT + 1);
constexpr int kKStages = 2, kVStages = 4;
constexpr int kScales = 16;    // scale ring: softmax has read a tile's slot before its successor's loads are issued
constexpr int kSBufs = 3;      // score buffers, tile i in i % 3
// TMEM columns: S (and P over it), Q, O of each stream
constexpr uint32_t kColsT = 512, kColQT = kSBufs * 64, kColOT = 256;

template <int D>
struct SmemT {
  static constexpr int kRaw = D == 128 ? 4 : 8;
  alignas(1024) uint8_t k[kKStages][kTileT * D * 2];
  alignas(1024) uint8_t v[kVStages][kTileT * D * 2];
  alignas(1024) uint8_t raw[kRaw][2][kTileT * D];
  alignas(128) float scale[kScales][2][kTileT];
  alignas(16) float vd[kScales][kTileT];  // V scales times 2^-E of the tile (tiles that every row sees whole)
  alignas(16) float lv[kScales][kTileT];  // log2 of the V scales
  int e[kScales];                       // that E
  uint32_t amax[2][kRowsT];             // of the halves of Q's rows
  float c[2][kRowsT], l[2][kRowsT], g[2][kRowsT], up[2][kRowsT];  // what the streams exchange at a unit's end
  int flags[kScales];                   // bits 0-3: the 16-key groups that hold keys; bit 4: not every row sees every key; bit 5: a unit's first tile
  uint64_t raw_full[kRaw], raw_empty[kRaw];
  uint64_t k_full[kKStages], k_empty[kKStages], v_full[kVStages], v_empty[kVStages];
  uint64_t s_full[kSBufs], p_full[kSBufs], o_done[kSBufs];
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
// TMEM in MMA fragment order: of 16 rows and blocks of 8 columns, thread (g, c)
// = (lane / 4, lane % 4) holds columns 2c, 2c + 1 of rows g and g + 8 (four
// registers a block); packed to 16 bits, two registers.  A thread then meets a
// quarter of a tile's keys in four rows instead of all keys in one, and reads a
// quarter of the scales from shared memory.
__device__ __forceinline__ void tmem_ld_frag4(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// Two blocks, waited for.
__device__ __forceinline__ void tmem_ld_frag2(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st_frag4(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_half8(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
constexpr uint32_t kLane16 = 16u << 16;  // rows 16-31 of a warp

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
// [key][128 bytes].  Each warp w of the converters takes 16 keys.
template <int D, int F>
__device__ __forceinline__ void convert(uint32_t raw, uint32_t to, int w, int lane, bool clean) {
  constexpr int KB = kTileT / (8 * kConvWarps);
  const int c = lane & 3;
  uint4 in[KB][D / 64];
#pragma unroll
  for (int kb = 0; kb < KB; ++kb)
#pragma unroll
    for (int x = 0; x < D / 64; ++x) in[kb][x] = lds128(raw + swizzled<D>(8 * (KB * w + kb) + key_of(lane >> 2), 4 * x + c));
  if (F == SAGE_CACHE_E4M3 && clean) {
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int x = 0; x < D / 64; ++x) {
        uint4& v = in[kb][x];
        v = make_uint4(no_nan<F>(v.x), no_nan<F>(v.y), no_nan<F>(v.z), no_nan<F>(v.w));
      }
  }
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) {
    const int key = 8 * (KB * w + kb) + key_of(lane >> 2);
#pragma unroll
    for (int x = 0; x < D / 64; ++x) {
      uint32_t o[8];
      const uint32_t iw[4] = {in[kb][x].x, in[kb][x].y, in[kb][x].z, in[kb][x].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) codes_to_f16<F>(iw[e], o[2 * e], o[2 * e + 1]);
      const uint32_t row = to + x * (kTileT * 128) + key * 128;
      sts128(row + (((2 * c) ^ (key & 7)) << 4), o[0], o[1], o[2], o[3]);
      sts128(row + (((2 * c + 1) ^ (key & 7)) << 4), o[4], o[5], o[6], o[7]);
    }
  }
}

// The offsets c of a thread's two rows (of 16, at TMEM columns `cols`) for a tile, the sums l in their unit, and the factors
// al of the accumulator's rows; `ks`, `lv`: the keys' score scales and log2 of their V scales; bit 16 q + 2 n + e of `seen`:
// row q sees key 8 n + 2 c4 + e; bit q of `none`: row q has seen nothing yet, of `found`: it has now.  Rare (a unit's first
// tile in each stream, a larger V scale), and it pays by its size: unrolled, or 32 keys at a time, its four
// copies cost the common path more (us, 21 drafted tokens over 16 contexts of 500..16384: 16 keys at a time 184, 8
// keys 190, 32 keys 193, unrolled 252).
struct Offsets {
  float c[2], l[2], al[2];
  uint32_t found;
};
__device__ __forceinline__ Offsets set_offsets(uint32_t cols, const float* ks, const float* lv, uint32_t seen, uint32_t none,
                                               float fr0, float fr1, const Offsets& was, int E0, int E1, int Ea, int Eb) {
  const float fr[2] = {fr0, fr1};
  const int E[2] = {E0, E1}, E_new[2] = {Ea, Eb};
  float top[2] = {-INFINITY, -INFINITY}, weight[2] = {-INFINITY, -INFINITY};
  uint32_t s[8];
#pragma unroll 1
  for (int cb = 0; cb < 4; ++cb) {
    tmem_ld_frag2(cols + 16 * cb, s);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const int n = 2 * cb + m;
      const float2 k2 = *reinterpret_cast<const float2*>(ks + 8 * n), v2 = *reinterpret_cast<const float2*>(lv + 8 * n);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if ((seen >> (16 * (e >> 1) + 2 * n + (e & 1))) & 1u) {
          const float x = __uint_as_float(s[4 * m + e]) * ((e & 1) ? k2.y : k2.x);
          top[e >> 1] = fmaxf(top[e >> 1], x);
          weight[e >> 1] = fmaxf(weight[e >> 1], __fmaf_ru(x, fr[e >> 1], (e & 1) ? v2.y : v2.x));
        }
    }
  }
  Offsets to;
  to.found = 0;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    float mass = was.l[q];
#pragma unroll
    for (int k = 1; k < 4; k <<= 1) {  // the four threads that share a row
      mass += __shfl_xor_sync(0xffffffffu, mass, k);
      top[q] = fmaxf(top[q], __shfl_xor_sync(0xffffffffu, top[q], k));
      weight[q] = fmaxf(weight[q], __shfl_xor_sync(0xffffffffu, weight[q], k));
    }
    const bool nothing = (none >> q) & 1u, some = top[q] != -INFINITY;
    const float kept = kept_offset(was.c[q], E_new[q] - E[q], mass);
    const float set = some ? tile_offset(top[q] * fr[q], weight[q], E_new[q]) : nothing ? 0.0f : kept;
    to.c[q] = nothing ? set : fmaxf(set, kept);
    to.l[q] = nothing ? 0.0f : was.l[q] * ex2(was.c[q] - to.c[q]);
    to.al[q] = nothing ? 0.0f : ex2((was.c[q] - to.c[q]) + (float)(E[q] - E_new[q]));
    if (some) to.found |= 1u << q;
  }
  return to;
}
// Multiplies a thread's two rows of an accumulator at TMEM columns `col` on.
template <int D>
__device__ __forceinline__ void multiply_rows(uint32_t col, float al0, float al1) {
  uint32_t s[16];
#pragma unroll 1
  for (int x = 0; x < D; x += 32) {
    tmem_ld_frag4(col + x, s);
    tmem_wait_ld16(s);
#pragma unroll
    for (int e = 0; e < 16; ++e) s[e] = __float_as_uint(__uint_as_float(s[e]) * ((e >> 1) & 1 ? al1 : al0));
    tmem_st_frag4(col + x, s);
  }
}

// What a softmax thread holds of its four fragment rows: row 8 r + g of the warp's 32, r = 0 .. 3.
struct RowState {
  float c[4], l[4];
  int E[4];
  uint32_t none;  // bit r: the row has seen nothing yet
};
struct TileOf {
  uint32_t cols, col_o;  // TMEM columns of the tile's scores and of the stream's accumulator
  int i;                 // the tile
  bool fresh;            // the accumulator holds nothing yet
  long long wait_limit;
  DeviceStatus* status;
};
// Softmax of half HV of a tile's rows, the thread's rows 2 HV and 2 HV + 1: scores -> weights over them in TMEM.  `seen` (a
// masked tile): bit 16 q + 2 n + e: its row 2 HV + q sees key 8 n + 2 c4 + e.  Ea, Eb: E of the rows from here on.
template <int D, bool MASKED, int HV>
__device__ __forceinline__ bool half(SmemT<D>& sm, RowState& st, const float (&fr)[4], const TileOf& at, uint32_t seen,
                                     int Ea, int Eb) {
  constexpr int r0 = 2 * HV;
  const int slot = at.i & (kScales - 1), c4 = threadIdx.x & 3;
  const float* ks = sm.scale[slot][0] + 2 * c4;
  const float* vs = (MASKED ? sm.scale[slot][1] : sm.vd[slot]) + 2 * c4;
  auto sees = [&](int q, int n, int e) { return !MASKED || ((seen >> (16 * q + 2 * n + e)) & 1u); };
  const uint32_t cols = at.cols + HV * kLane16;
  // c is set until a row has seen something, with E, and where a thread's sum of a tile's p passes what FP16 holds (so
  // that it holds each weight); the half is then done again
  bool raise = __any_sync(0xffffffffu, Ea != st.E[r0] || Eb != st.E[r0 + 1] || ((st.none >> r0) & 3u));
  uint32_t p[16];
  uint64_t sum[2];
  for (;;) {
    uint32_t s[16];
    if (raise) {
      const Offsets to = set_offsets(cols, ks, sm.lv[slot] + 2 * c4, MASKED ? seen : ~0u, (st.none >> r0) & 3u, fr[r0],
                                     fr[r0 + 1], {{st.c[r0], st.c[r0 + 1]}, {st.l[r0], st.l[r0 + 1]}, {}, 0}, st.E[r0],
                                     st.E[r0 + 1], Ea, Eb);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        st.c[r0 + q] = to.c[q];
        st.l[r0 + q] = to.l[q];
      }
      st.none &= ~(to.found << r0);
      st.E[r0] = Ea;
      st.E[r0 + 1] = Eb;
      if (!at.fresh && __any_sync(0xffffffffu, to.al[0] != 1.0f || to.al[1] != 1.0f)) {
        // the stream's PV before is done first, then the accumulator's rows are multiplied
        if (!__all_sync(0xffffffffu, wait_bounded(&sm.o_done[(at.i - 2) % kSBufs], ((at.i - 2) / kSBufs) & 1u,
                                                  &sm.abort_flag, at.status, 103, at.wait_limit)))
          return false;
        tc_fence_after();
        multiply_rows<D>(at.col_o + HV * kLane16, to.al[0], to.al[1]);
      }
    }
    sum[0] = sum[1] = 0;
#pragma unroll
    for (int cb = 0; cb < 2; ++cb) {
      tmem_ld_frag4(cols + 32 * cb, s);
      tmem_wait_ld16(s);
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int n = 4 * cb + m;
        const uint64_t kk = *reinterpret_cast<const uint64_t*>(ks + 8 * n), vv = *reinterpret_cast<const uint64_t*>(vs + 8 * n);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int r = r0 + q;
          const float2 x = unpair(mul2(pair(__uint_as_float(s[4 * m + 2 * q]), __uint_as_float(s[4 * m + 2 * q + 1])), kk));
          float2 y = make_float2(fmaf(x.x, fr[r], -st.c[r]), fmaf(x.y, fr[r], -st.c[r]));
          uint64_t v = vv;
          if (MASKED) {
            const float2 vm = unpair(v);
            const float down = __int_as_float((127 - st.E[r]) << 23);
            if (!sees(q, n, 0)) y.x = -INFINITY;
            if (!sees(q, n, 1)) y.y = -INFINITY;
            v = pair(sees(q, n, 0) ? vm.x * down : 0.0f, sees(q, n, 1) ? vm.y * down : 0.0f);
          }
          const uint64_t w = pair(ex2(y.x), ex2(y.y));
          sum[q] = add2(sum[q], w);
          const float2 z = unpair(mul2(w, v));
          p[2 * n + q] = pack_f16x2(z.x, z.y);
        }
      }
    }
    if (raise) break;
    const float2 y0 = unpair(sum[0]), y1 = unpair(sum[1]);
    raise = __any_sync(0xffffffffu, !(y0.x + y0.y <= 65504.0f) || !(y1.x + y1.y <= 65504.0f));
    if (!raise) break;
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const float2 y = unpair(sum[q]);
    st.l[r0 + q] += y.x + y.y;
  }
  tmem_st_half8(cols, p);
  return true;
}

// A tile that not every row sees whole: the drafted tokens, a unit's end, a page left out.  What it takes and returns is one
// block by value: with references the same instructions lay so that warps waited for instructions 2.5 times as long
// (1.33 against 0.53 stalls per issue) and 21 drafted tokens over 16 contexts of 500..16384 took 212 us instead of 183.
template <int D>
struct MaskedRows {
  SmemT<D>* sm;
  const CacheAttnArgs* a;
  TileOf at;
  RowState st;
  float fr[4];
  int b, row0, rows, ctx, cnt, wrow;
  int64_t slot0;  // the tile's first slot
  int flags;
  bool ok;
};
template <int D>
__device__ __forceinline__ MaskedRows<D> masked_tile(MaskedRows<D> t) {
  SmemT<D>& sm = *t.sm;
  const CacheAttnArgs& a = *t.a;
  const int lane = threadIdx.x & 31, g = lane >> 2, c4 = lane & 3, slot = t.at.i & (kScales - 1);
  const int64_t d0 = t.slot0 - t.ctx;  // drafted token of the tile's first key (below 0: context)
  const bool drafts = d0 < t.cnt && d0 > -kTileT;
  const int lo = (int)max(d0, (int64_t)0), hi = drafts ? min((int)(d0 + kTileT), t.cnt) : lo;  // drafted tokens [lo, hi)
  const int words = (a.T + 31) / 32, w0 = lo / 32, sh = lo % 32;
  uint32_t m[4][3];  // the t.rows' mask words of lo and behind, all loads before the first use
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int rw = t.wrow + g + 8 * r, tok = (t.row0 + rw) / a.G;
#pragma unroll
    for (int w = 0; w < 3; ++w)
      m[r][w] = a.mask && drafts && rw < t.rows && w0 + w < words ? a.mask[((int64_t)t.b * a.T + tok) * words + w0 + w] : 0u;
  }
  uint32_t mine[2] = {0, 0};
  int E_new[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    uint64_t seen = d0 <= -64 ? ~0ull : d0 >= 0 ? 0ull : ~0ull >> (64 + d0);
    if (t.wrow + g + 8 * r < t.rows && drafts) {
      const int tok = (t.row0 + t.wrow + g + 8 * r) / a.G;
      uint64_t bits = 0;  // of tokens lo, lo + 1, ...
      if (a.mask) {
        bits = (uint64_t)__funnelshift_r(m[r][1], m[r][2], sh) << 32 | __funnelshift_r(m[r][0], m[r][1], sh);
      } else if (tok >= lo) {
        bits = tok - lo >= 63 ? ~0ull : (2ull << (tok - lo)) - 1;
      }
      if (hi - lo < 64) bits &= (1ull << (hi - lo)) - 1;
      seen |= bits << (lo - (int)d0);
    }
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (!((t.flags >> x) & 1)) seen &= ~(0xFFFFull << (16 * x));
    float vm = 0.0f;
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const uint32_t two = (uint32_t)(seen >> (8 * n + 2 * c4)) & 3u;
      const float2 v = *reinterpret_cast<const float2*>(sm.scale[slot][1] + 8 * n + 2 * c4);
      if (two & 1) vm = fmaxf(vm, v.x);
      if (two & 2) vm = fmaxf(vm, v.y);
      mine[r >> 1] |= two << (16 * (r & 1) + 2 * n);
    }
    vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, 1));
    vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, 2));
    E_new[r] = max(t.st.E[r], v_exponent(__float_as_uint(vm)));
  }
  t.ok = half<D, true, 0>(sm, t.st, t.fr, t.at, mine[0], E_new[0], E_new[1]) &&
         half<D, true, 1>(sm, t.st, t.fr, t.at, mine[1], E_new[2], E_new[3]);
  return t;
}

template <int D, int KF, int VF>
__global__ void __launch_bounds__(kThreadsT, 1)
    cache_attn_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                         const __grid_constant__ CacheAttnArgs a) {
  constexpr int NR = SmemT<D>::kRaw, DH = D / 2, BLK = kTileT * 128;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  SmemT<D>& sm = *reinterpret_cast<SmemT<D>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &sm.abort_flag;
  DeviceStatus* status = a.c.status;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NR; ++s) {
      mbar_init(&sm.raw_full[s], 2);  // both producers
      mbar_init(&sm.raw_empty[s], 2 * kConvWarps);
    }
    for (int s = 0; s < kKStages; ++s) {
      mbar_init(&sm.k_full[s], kConvWarps);
      mbar_init(&sm.k_empty[s], 1);
    }
    for (int s = 0; s < kVStages; ++s) {
      mbar_init(&sm.v_full[s], kConvWarps);
      mbar_init(&sm.v_empty[s], 1);
    }
    for (int s = 0; s < kSBufs; ++s) {
      mbar_init(&sm.s_full[s], 1);
      mbar_init(&sm.p_full[s], 4);
      mbar_init(&sm.o_done[s], 1);
    }
    mbar_init(&sm.q_full, 256);
    mbar_init(&sm.swap, 256);
    mbar_init(&sm.drain[0], 1);
    mbar_init(&sm.drain[1], 1);
    sm.abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  begin_dependent_tma();
  const Stretch st = find_stretch<kTileT, kRowsT, 1>(a, blockIdx.x, gridDim.x);
  if (blockIdx.x == 0)  // lengths that cannot be
    for (int b = threadIdx.x; b < a.B; b += kThreadsT) {
      const int ctx = a.context[b], cnt = a.count ? a.count[b] : a.T;
      if (ctx < 0 || cnt < 0 || cnt > a.T ||
          (long long)ctx + cnt > ((long long)a.c.table_pages << a.c.page_shift))
        flag_bad(status, kWhereAttn);
    }
  if (threadIdx.x == 0) cut_unit(a, blockIdx.x)->parts = 0;  // behind the wait: the join of a call before may read its own until then
  if (st.s >= st.e) return;
  if (warp == kQkWarpT) tmem_alloc(&sm.tmem_base, kColsT);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  const int n_tiles = (int)(st.e - st.s);
  // the phase of number `phase` of a barrier, by a whole warp
  auto wait = [&](uint64_t* bar, uint32_t phase, int where) -> bool {
    return __all_sync(0xffffffffu, wait_bounded(bar, phase & 1u, abort_flag, status, 100 + where, a.wait_limit));
  };

  if (warp < kConvK) {
    // ------------------------------------------------------ softmax streams
    const int sid = warp >> 2, wrow = (warp & 3) * 32, row = wrow + lane, g = lane >> 2, c4 = lane & 3;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16), col_o = lanes + kColOT + sid * D;
    uint32_t swaps = 0;
    bool ok = true;
    Place at = place_of<kTileT, kRowsT>(a, st.own, st.s);
    for (unsigned seg = st.s; ok && seg < st.e;) {
      go_to<kTileT, kRowsT>(a, at, seg);
      const Unit u = unit_of(at, seg);
      const int b = at.b, h = u.h, row0 = u.rt * kRowsT, ctx = at.s.ctx, cnt = at.s.cnt;
      const int rows = min(kRowsT, cnt * a.G - row0);
      const unsigned unit_end = u.start + at.s.n, seg_end = min(unit_end, st.e);
      const bool idle = (warp & 3) * 32 >= rows;  // no row of this warp

      // ---- this thread's half of its Q row: FP16, channels 0, 2, 1, 3 of each four
      float f;
      {
        uint4 w[DH / 8];
        uint32_t top = 0;
        const uint16_t* q = a.q + b * a.qb + min((row0 + row) / a.G, a.T - 1) * a.qn + (h * a.G + (row0 + row) % a.G) * a.qh + sid * DH;
#pragma unroll
        for (int x = 0; x < DH / 8; ++x) {
          w[x] = make_uint4(0, 0, 0, 0);
          if (row < rows) w[x] = *reinterpret_cast<const uint4*>(q + 8 * x);
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
        const float down = q_down(top, eq);
        f = q_factor(eq);
#pragma unroll
        for (int x0 = 0; x0 < DH / 8; x0 += 4) {
          uint32_t o[16];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint32_t ww[4] = {w[x0 + x].x, w[x0 + x].y, w[x0 + x].z, w[x0 + x].w};
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              o[4 * x + e] = pack_f16x2(__uint_as_float(ww[e] << 16) * down, __uint_as_float(ww[e + 1] << 16) * down);
              o[4 * x + e + 1] =
                  pack_f16x2(__uint_as_float(ww[e] & 0xFFFF0000u) * down, __uint_as_float(ww[e + 1] & 0xFFFF0000u) * down);
            }
          }
          tmem_st16(lanes + kColQT + sid * (DH / 2) + 4 * x0, o);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&sm.q_full);
      }
      // From here on a thread works on its four fragment rows: row 8 r + g of the warp's 32, r = 0 .. 3.
      float fr[4];
      RowState st_rows;
      st_rows.none = 15;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        fr[r] = __shfl_sync(0xffffffffu, f, g + 8 * r);
        st_rows.c[r] = st_rows.l[r] = 0.0f;
        st_rows.E[r] = -126;
      }
      bool fresh = true;  // no PV of this unit yet: the accumulator holds nothing

      // ---- tiles of this stream
      int i = (int)(seg - st.s);
      i += (i & 1) ^ sid;
      for (; i < (int)(seg_end - st.s); i += 2) {
        const int buf = i % kSBufs, slot = i & (kScales - 1);
        if (!(ok = wait(&sm.s_full[buf], i / kSBufs, 2))) break;
        tc_fence_after();
        const uint32_t cols = lanes + buf * 64;
        if (!idle) {
          const int flags = sm.flags[slot];
          const TileOf at_tile{cols, col_o, i, fresh, a.wait_limit, status};
          if (!(flags & kMasked)) {
            const int E_new = sm.e[slot];
            ok = half<D, false, 0>(sm, st_rows, fr, at_tile, ~0u, E_new, E_new) &&
                 half<D, false, 1>(sm, st_rows, fr, at_tile, ~0u, E_new, E_new);
          } else {
            MaskedRows<D> m{&sm, &a, at_tile, st_rows, {fr[0], fr[1], fr[2], fr[3]}, b, row0, rows, ctx, cnt, wrow,
                            (int64_t)(st.s + i - u.start) * kTileT, flags, true};
            m = masked_tile<D>(m);
            st_rows = m.st;
            ok = m.ok;
          }
          if (!ok) break;
          tmem_wait_st();
        }
        fresh = false;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[buf]);
      }
      if (!ok) break;

      // ---- the unit's end: wait for this stream's last PV, exchange the states, store half of the columns
      if (!fresh) {
        int last = (int)(seg_end - st.s) - 1;  // the stream's last tile
        last -= (last & 1) ^ sid;
        if (!(ok = wait(&sm.o_done[last % kSBufs], last / kSBufs, 4))) break;
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float x = st_rows.l[r];
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        if (c4 == 0) {
          const int rw = wrow + g + 8 * r;
          const Mass m = normalised((st_rows.none >> r) & 1 ? -INFINITY : st_rows.c[r], x, kPartBias);
          sm.l[sid][rw] = m.l;
          sm.c[sid][rw] = m.c;
          sm.g[sid][rw] = m.g;
          sm.up[sid][rw] = fresh ? 0.0f : __int_as_float((127 + st_rows.E[r]) << 23);  // 2^E; 0: the accumulator holds nothing
        }
      }
      tc_fence_before();
      mbar_arrive(&sm.swap);
      if (!(ok = wait(&sm.swap, swaps++, 5))) break;
      tc_fence_after();
      if (!idle) {
        const float ca = sm.c[0][row], cb = sm.c[1][row], cm = fmaxf(ca, cb);
        const float wa = ca == -INFINITY ? 0.0f : ex2(ca - cm), wb = cb == -INFINITY ? 0.0f : ex2(cb - cm);
        const float lt = sm.l[0][row] * wa + sm.l[1][row] * wb;
        const bool has_a = sm.up[0][row] != 0.0f, has_b = sm.up[1][row] != 0.0f;
        const bool whole = seg == u.start && seg_end == unit_end, on = row < rows;
        const float inv = whole ? row_inverse(lt) : 1.0f;
        const float fa = sm.g[0][row] * wa * inv, fb = sm.g[1][row] * wb * inv, up_a = sm.up[0][row], up_b = sm.up[1][row];
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
            o[e] = (has_a ? __uint_as_float(oa[e]) * fa * up_a : 0.0f) + (has_b ? __uint_as_float(ob[e]) * fb * up_b : 0.0f);
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
            store_lse(a, b, h, row0 + row, cm, lt);
          } else {
            part[kRowsT * D + row] = cm;
            part[kRowsT * D + kRowsT + row] = lt;
            if (row == 0 && seg == u.start)
              *cut_unit(a, blockIdx.x) = CutUnit{(int)((unit_end - 1) / st.share - blockIdx.x) + 1, b, h, row0, rows};
          }
        }
      }
      tc_fence_before();
      seg = seg_end;
    }
  } else if (warp < kLoadK) {
    // ----------------------------------------------------------- converters
    // warps of K and of V, each at its own pace
    const bool is_v = warp >= kConvV;
    const int w = warp - (is_v ? kConvV : kConvK);
    int E = -126;  // of the unit's tiles so far; behind one with a draft or an end none follows that needs it
    for (int i = 0; i < n_tiles; ++i) {
      const int r = i % NR, slot = i & (kScales - 1);
      if (!wait(&sm.raw_full[r], i / NR, 6)) break;
      const int flags = sm.flags[slot];
      if (is_v) {
        if (!wait(&sm.v_empty[i % kVStages], (i / kVStages) ^ 1, 8)) break;
        convert<D, VF>(smem_u32(sm.raw[r][1]), smem_u32(sm.v[i % kVStages]), w, lane, flags & kMasked);
      } else {
        if (w == 1) {  // the softmax streams' scales, seen behind k_full: K's with the softmax scale, and V's with 2^-E
          sm.scale[slot][0][lane] *= a.sl2;
          sm.scale[slot][0][lane + 32] *= a.sl2;
        } else if (w == 0) {
          if (flags & kFirst) E = -126;
          float v0 = sm.scale[slot][1][lane], v1 = sm.scale[slot][1][lane + 32];
          if (!((flags >> (lane / 16)) & 1)) v0 = 0.0f;  // a group without keys: what the slot held before
          if (!((flags >> (2 + lane / 16)) & 1)) v1 = 0.0f;
          // with the tiles that have a page left out in the middle of a context, whose E the rows took for themselves
          E = max(E, v_exponent(__reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(fmaxf(v0, v1), 0.0f)))));
          if (!(flags & kMasked)) {
            const float down = __int_as_float((127 - E) << 23);
            sm.vd[slot][lane] = v0 * down;
            sm.vd[slot][lane + 32] = v1 * down;
            if (lane == 0) sm.e[slot] = E;
          }
        } else if (w == 2) {
          sm.lv[slot][lane] = lg2f(sm.scale[slot][1][lane]);
          sm.lv[slot][lane + 32] = lg2f(sm.scale[slot][1][lane + 32]);
        }
        if (!wait(&sm.k_empty[i % kKStages], (i / kKStages) ^ 1, 7)) break;
        convert<D, KF>(smem_u32(sm.raw[r][0]), smem_u32(sm.k[i % kKStages]), w, lane, false);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(is_v ? &sm.v_full[i % kVStages] : &sm.k_full[i % kKStages]);
        mbar_arrive(&sm.raw_empty[r]);
      }
    }
  } else if (warp <= kLoadV) {
    // ------------------------------------------------------------ producers
    // A tile's boxes are 16, 32 or 64 keys, what a page holds of it.  Lane 4 t + x looks up the row of group x of 16 keys
    // of tile t of the next eight; the first group of a box stands for it.
    const int side = warp - kLoadK, box = min(1 << a.c.page_shift, kTileT), per = box / 16;
    const CUtensorMap* map = side ? &tm_v : &tm_k;
    Place walk = place_of<kTileT, kRowsT>(a, st.own, st.s);
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
      if (i == a.stall_tile) break;  // test hook: nothing comes from here on
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
      wait_bounded(&sm.raw_full[i % NR], (uint32_t)((i / NR) & 1), abort_flag, nullptr, 110, a.wait_limit, false);
  } else {
    // -------------------------------------------------------------- issuers
    const uint32_t leader = lane == 0;
    Place at = place_of<kTileT, kRowsT>(a, st.own, st.s);
    unsigned seg_end = st.s;  // of the unit that tile i belongs to
    int units = 0, begin = 0;
    for (int i = 0; i < n_tiles; ++i) {
      const int buf = i % kSBufs;
      const uint32_t sc = tmem + buf * 64;
      const bool next = st.s + i == seg_end;
      if (next) {
        go_to<kTileT, kRowsT>(a, at, st.s + i);
        const Unit u = unit_of(at, st.s + i);
        seg_end = min(u.start + at.s.n, st.e);
        begin = i;
      }
      if (warp == kQkWarpT) {
        // a new unit's Q; the score buffer: PV of the tile three back has read its P
        if (next && !wait(&sm.q_full, units++, 13)) break;
        if (i >= kSBufs && !wait(&sm.o_done[buf], i / kSBufs - 1, 14)) break;
        if (!wait(&sm.k_full[i % kKStages], i / kKStages, 15)) break;
        tc_fence_after();
        const uint64_t kd = desc128(smem_u32(sm.k[i % kKStages]), 16, 1024);
#pragma unroll
        for (int x = 0; x < D / 16; ++x)
          mma_f16_ts(leader, sc, tmem + kColQT + 8 * x, kd + (x / 4) * (BLK >> 4) + 2 * (x % 4), idesc_f16(kTileT, false), x > 0);
        commit(leader, &sm.s_full[buf]);
        commit(leader, &sm.k_empty[i % kKStages]);
      } else {
        if (!wait(&sm.v_full[i % kVStages], i / kVStages, 12) || !wait(&sm.p_full[buf], i / kSBufs, 11)) break;
        tc_fence_after();
        const uint64_t vd = desc128(smem_u32(sm.v[i % kVStages]), BLK, 1024);
        const uint32_t o = tmem + kColOT + (i & 1) * D, more = i >= begin + 2;  // the unit's first tile of a stream starts its O
#pragma unroll
        for (int x = 0; x < kTileT / 16; ++x)
          mma_f16_ts(leader, o, sc + 8 * x, vd + x * (2048 >> 4), idesc_f16(D, true), x > 0 ? 1u : more);
        commit(leader, &sm.o_done[buf]);
        commit(leader, &sm.v_empty[i % kVStages]);
      }
    }
    __syncwarp();
    uint64_t* drain = &sm.drain[warp - kQkWarpT];
    commit(leader, drain);
    wait_bounded(drain, 0, abort_flag, nullptr, 116, a.wait_limit, false);
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
  if (const int rc = launch_dependent(fn, dim3(kMaxCtas), kThreadsT, smem, s, mk, mv, a)) return rc;
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
