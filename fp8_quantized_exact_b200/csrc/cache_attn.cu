// Attention of new or drafted tokens over the quantised paged cache.
//
// Row (b, t, h) of Q sees slots 0 .. context[b]-1 of its sequence, and slot
// context[b] + j of the drafted tokens where bit j of its mask is set:
//   s_j = (q . k_j) * kscale_j * sm_scale,  out = sum_j softmax(s)_j v_j vscale_j,
//   lse = ln sum_j exp(s_j);  a row that sees nothing has out = 0, lse = -inf.
//
// One block per row; each warp takes every fourth key, with its own running
// maximum and sum, and the warps are joined at the end.
#include "cache_common.cuh"

namespace sage {
namespace {

constexpr int kAttnWarps = 4;

__device__ __forceinline__ float code_value(uint8_t c, int format) {
  if (format == SAGE_CACHE_INT8) return (float)(int8_t)c;
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
  float f;
  asm("{.reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.f32.f16 %0, lo;}" : "=f"(f) : "r"(h));
  return f;
}

template <int D>
__global__ void __launch_bounds__(32 * kAttnWarps) cache_attn_kernel(const CacheAttnArgs a) {
  constexpr int E = D / 32;
  __shared__ float m_s[kAttnWarps], l_s[kAttnWarps], o_s[kAttnWarps][D];
  const int hq = blockIdx.x % a.Hq, t = blockIdx.x / a.Hq, b = blockIdx.y;
  const int h = hq / a.G, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int ctx = a.context[b], count = a.count ? a.count[b] : a.T;
  if ((ctx < 0 || count < 0 || count > a.T) && threadIdx.x == 0) flag_bad(a.c.status, kWhereAttn);
  ctx = max(ctx, 0);
  count = min(count, a.T);
  if (t >= count) return;
  const uint16_t* q = a.q + b * a.qb + t * a.qn + hq * a.qh;
  float qv[E], o[E], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qv[e] = bf16_bits_to_f32(q[e * 32 + lane]);
    o[e] = 0.0f;
  }
  const int words = (a.T + 31) / 32;
  for (int64_t j = warp; j < (int64_t)ctx + count; j += kAttnWarps) {
    if (j >= ctx) {
      const int i = (int)(j - ctx);
      if (a.mask ? !((a.mask[((int64_t)b * a.T + t) * words + i / 32] >> (i % 32)) & 1u) : i > t) continue;
    }
    const int64_t row = cache_row(a.c, b, h, j);
    if (row < 0) {
      if (lane == 0) flag_bad(a.c.status, kWhereAttn);
      continue;
    }
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(qv[e], code_value(a.c.codes[0][row * D + e * 32 + lane], a.c.format[0]), s);
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    s *= a.c.scale[0][row] * a.sl2;
    const float m_new = fmaxf(m, s), r = exp2f(m - m_new), p = exp2f(s - m_new), w = p * a.c.scale[1][row];
    l = l * r + p;
#pragma unroll
    for (int e = 0; e < E; ++e)
      o[e] = fmaf(w, code_value(a.c.codes[1][row * D + e * 32 + lane], a.c.format[1]), o[e] * r);
    m = m_new;
  }
  if (lane == 0) {
    m_s[warp] = m;
    l_s[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) o_s[warp][e * 32 + lane] = o[e];
  __syncthreads();
  m = -INFINITY;
  for (int w = 0; w < kAttnWarps; ++w) m = fmaxf(m, m_s[w]);
  float f[kAttnWarps];
  l = 0.0f;
  for (int w = 0; w < kAttnWarps; ++w) {
    f[w] = l_s[w] == 0.0f ? 0.0f : exp2f(m_s[w] - m);
    l += l_s[w] * f[w];
  }
  const bool none = l == 0.0f;
  for (int d = threadIdx.x; d < D; d += 32 * kAttnWarps) {
    float v = 0.0f;
    for (int w = 0; w < kAttnWarps; ++w) v += o_s[w][d] * f[w];
    a.out[b * a.ob + t * a.on + hq * a.oh + d] = f32_to_bf16_rn(none ? 0.0f : v / l);
  }
  if (a.lse && threadIdx.x == 0)
    a.lse[((int64_t)b * a.T + t) * a.Hq + hq] = none ? -INFINITY : (m + log2f(l)) * 0.69314718f;
}

}  // namespace

size_t cache_attn_workspace_bytes() { return 0; }

int launch_cache_attn(const CacheAttnArgs& a, cudaStream_t s) {
  const dim3 grid(a.T * a.Hq, a.B);
  if (a.c.D == 128) cache_attn_kernel<128><<<grid, 32 * kAttnWarps, 0, s>>>(a);
  else cache_attn_kernel<64><<<grid, 32 * kAttnWarps, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? SAGE_OK : SAGE_ERR_CUDA;
}

}  // namespace sage
