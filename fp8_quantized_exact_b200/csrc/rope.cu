// Rotary positions on Q and K views.
//
// Per token at position p and rotated pair (x0, x1) number j of a head:
//   a  = p * f_j,          c = m cos a,  s = m sin a   (s negated for the transpose)
//   y0 = bf16(x0 c - x1 s), y1 = bf16(x1 c + x0 s)      in FP32, one rounding.
// Pair j is (x_j, x_{j + rot/2}) in the half layout and (x_{2j}, x_{2j+1}) in
// the interleaved one; channels from rot on are copied.  The map is linear
// and orthogonal up to m, so its gradient is the same kernel with -s.
//
// The angle is taken in FP64: a position of 10^6 times a frequency of 1 needs
// 2^-24 of a turn left after 20 bits of whole turns, which FP32 does not
// have.  The product is reduced to a fraction of a turn in FP64 and only that
// goes to the FP32 sine and cosine.  Each block computes the (cos, sin) of its
// tokens once, in shared memory, for all its heads.
//
// Bound: HBM, 4 bytes per element (2 read, 2 written).
#include "cache_common.cuh"

namespace sage {
namespace {

constexpr int kRopeThreads = 256;

__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// One pair, (y0, y1) = (x0 c - x1 s, x1 c + x0 s).
__device__ __forceinline__ void rotate(float x0, float x1, float2 cs, float& y0, float& y1) {
  y0 = fmaf(x0, cs.x, -x1 * cs.y);
  y1 = fmaf(x1, cs.x, x0 * cs.y);
}

// One item of a head: item < rot_items rotates, the others copy 8 channels.
// HALF: 8 pairs (8 channels of each half).  Interleaved: 4 pairs.
template <bool HALF>
__device__ __forceinline__ void rope_item(uint4 a, uint4 b, uint16_t* y, bool turn, int d, int rot,
                                          const float2* __restrict__ cs) {
  if (!turn) {
    *reinterpret_cast<uint4*>(y + d) = a;
    return;
  }
  const uint32_t aw[4] = {a.x, a.y, a.z, a.w};
  uint32_t yw[4];
  if (HALF) {
    const uint32_t bw[4] = {b.x, b.y, b.z, b.w};
    uint32_t zw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float y0, y1, z0, z1;
      const float4 c = *reinterpret_cast<const float4*>(cs + d + 2 * i);
      rotate(lo_bf16(aw[i]), lo_bf16(bw[i]), make_float2(c.x, c.y), y0, z0);
      rotate(hi_bf16(aw[i]), hi_bf16(bw[i]), make_float2(c.z, c.w), y1, z1);
      yw[i] = pack_bf16(y0, y1);
      zw[i] = pack_bf16(z0, z1);
    }
    *reinterpret_cast<uint4*>(y + d + rot / 2) = make_uint4(zw[0], zw[1], zw[2], zw[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float y0, y1;
      rotate(lo_bf16(aw[i]), hi_bf16(aw[i]), cs[d / 2 + i], y0, y1);
      yw[i] = pack_bf16(y0, y1);
    }
  }
  *reinterpret_cast<uint4*>(y + d) = make_uint4(yw[0], yw[1], yw[2], yw[3]);
}

// The same for a rotated width that does not split into 16-byte vectors: one
// pair, or one copied channel.
template <bool HALF>
__device__ __forceinline__ void rope_item_1(const uint16_t* x, uint16_t* y, int item, int rot_items, int rot,
                                            const float2* __restrict__ cs) {
  if (item >= rot_items) {
    const int d = rot + (item - rot_items);
    y[d] = x[d];
    return;
  }
  const int d0 = HALF ? item : 2 * item, d1 = HALF ? item + rot / 2 : 2 * item + 1;
  float y0, y1;
  rotate(bf16_bits_to_f32(x[d0]), bf16_bits_to_f32(x[d1]), cs[item], y0, y1);
  y[d0] = f32_to_bf16_rn(y0);
  y[d1] = f32_to_bf16_rn(y1);
}

// Where a token's rows begin: input and output of Q and of K.
struct TokenRows {
  int64_t x[2], y[2];
};

// grid (token groups of `toks`, head groups of `heads`); the tokens are the
// B*N of the batch, the heads Q's Hq then K's.  A thread takes one item of
// ROWS rows at a time, their loads issued together: one row in the half layout,
// whose items have two loads already, four in the interleaved one (measured on
// B200 with 1, 2 and 4 rows: 343 (337 to 371 by the box), 379, 399 us for the half layout at B1 N37810
// 56+56 heads D128, 331 us at the copy rate; 141, 138, 135 us for the interleaved
// one at B4 N16384 24+24 heads D64 rot 32, 123 us at the copy rate).
template <bool HALF, bool VEC>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a, int toks, int heads, int items,
                                                            int rot_items, int item_shift) {
  constexpr int ROWS = HALF ? 1 : 4;
  extern __shared__ __align__(16) uint8_t rope_smem[];
  TokenRows* tokens = reinterpret_cast<TokenRows*>(rope_smem);       // [toks]
  float2* cs = reinterpret_cast<float2*>(rope_smem + toks * sizeof(TokenRows));  // [toks][pitch]
  const int half_rot = a.rot / 2, pitch = (half_rot + 1) & ~1;  // 16-byte reads of two
  const unsigned tok0 = blockIdx.x * (unsigned)toks;
  const int nt = (int)min((unsigned)toks, (unsigned)(a.B * a.N) - tok0);
  begin_dependent();
  for (int i = threadIdx.x; i < nt * half_rot; i += kRopeThreads) {
    const int t = i / half_rot, j = i - t * half_rot;
    const unsigned b = (tok0 + t) / (unsigned)a.N, n = (tok0 + t) - b * a.N;
    const int pos = a.positions ? a.positions[b * a.pos_stride_b + n] : (int)n;
    double turns = (double)pos * a.inv_freq[j] * 0.15915494309189533577;  // 1 / (2 pi)
    turns -= rint(turns);
    float s, c;
    sincospif(2.0f * (float)turns, &s, &c);
    cs[t * pitch + j] = make_float2(a.mscale * c, a.inverse ? -a.mscale * s : a.mscale * s);
  }
  for (int t = threadIdx.x; t < nt; t += kRopeThreads) {
    const int64_t b = (tok0 + t) / (unsigned)a.N, n = (tok0 + t) - (unsigned)b * a.N;
    tokens[t].x[0] = b * a.q.sb + n * a.q.sn;
    tokens[t].y[0] = b * a.q.yb + n * a.q.yn;
    tokens[t].x[1] = b * a.k.sb + n * a.k.sn;
    tokens[t].y[1] = b * a.k.yb + n * a.k.yn;
  }
  __syncthreads();
  const int item = threadIdx.x & ((1 << item_shift) - 1);
  if (item >= items) return;
  const int h0 = blockIdx.y * heads, nh = min(heads, a.Hq + a.Hk - h0), n_rows = nt * nh;
  const int step = kRopeThreads >> item_shift;
  const bool turn = item < rot_items;
  const int d = turn ? 8 * item : a.rot + 8 * (item - rot_items);
  auto locate = [&](int r, const uint16_t*& x, uint16_t*& y, int& t) {
    t = (unsigned)r / (unsigned)nh;
    const int h = h0 + r - t * nh, is_k = h >= a.Hq;
    const RopeSide& s = is_k ? a.k : a.q;
    const int64_t hh = is_k ? h - a.Hq : h;
    x = s.x + tokens[t].x[is_k] + hh * s.sh;
    y = s.y + tokens[t].y[is_k] + hh * s.yh;
  };
  if (VEC) {
    for (int r = threadIdx.x >> item_shift; r < n_rows; r += ROWS * step) {
      uint4 u[ROWS], v[ROWS];
      uint16_t* y[ROWS];
      int t[ROWS];
#pragma unroll
      for (int k = 0; k < ROWS; ++k) {
        if (r + k * step >= n_rows) continue;
        const uint16_t* x;
        locate(r + k * step, x, y[k], t[k]);
        u[k] = *reinterpret_cast<const uint4*>(x + d);
        if (HALF && turn) v[k] = *reinterpret_cast<const uint4*>(x + d + a.rot / 2);
      }
#pragma unroll
      for (int k = 0; k < ROWS; ++k)
        if (r + k * step < n_rows) rope_item<HALF>(u[k], v[k], y[k], turn, d, a.rot, cs + t[k] * pitch);
    }
  } else {
    for (int r = threadIdx.x >> item_shift; r < n_rows; r += step) {
      const uint16_t* x;
      uint16_t* y;
      int t;
      locate(r, x, y, t);
      rope_item_1<HALF>(x, y, item, rot_items, a.rot, cs + t * pitch);
    }
  }
}

template <bool HALF>
int run(const RopeArgs& a, cudaStream_t s) {
  const int64_t tokens = (int64_t)a.B * a.N;
  const int H = a.Hq + a.Hk;
  const bool vec = a.rot % (HALF ? 16 : 8) == 0;
  const int rot_items = vec ? (HALF ? a.rot / 16 : a.rot / 8) : a.rot / 2;
  const int items = rot_items + (a.in_place ? 0 : vec ? (a.D - a.rot) / 8 : a.D - a.rot);
  int shift = 0;
  while ((1 << shift) < items) ++shift;
  // about one (cos, sin) per thread in a block, fewer tokens where that
  // leaves SMs without a block, then fewer heads
  int toks = max(1, 2 * kRopeThreads / a.rot);
  while (toks > 1 && (tokens + toks - 1) / toks < 4 * 148) toks >>= 1;
  const int64_t groups = (tokens + toks - 1) / toks;
  int heads = H;
  while (heads > 4 && groups * ((H + heads - 1) / heads) < 2 * 148) heads = (heads + 1) / 2;
  const dim3 grid((unsigned)groups, (H + heads - 1) / heads);
  const size_t smem = (size_t)toks * (sizeof(TokenRows) + ((a.rot / 2 + 1) & ~1) * sizeof(float2));
  return launch_dependent(vec ? rope_kernel<HALF, true> : rope_kernel<HALF, false>, grid, kRopeThreads, smem, s, a, toks, heads,
                          items, rot_items, shift);
}

}  // namespace

int launch_rope(const RopeArgs& a, cudaStream_t s) {
  return a.half ? run<true>(a, s) : run<false>(a, s);
}

}  // namespace sage
