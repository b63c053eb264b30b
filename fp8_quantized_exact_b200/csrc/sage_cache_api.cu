// C ABI of the rotary positions and of the quantised paged cache: argument
// checks and launches.  See include/sage_b200.h for the contracts.
#include <math.h>

#include "api_checks.cuh"
#include "cache_common.cuh"

using namespace sage;

namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Rows of a call's token grid: at most 2^34, so that blocks of 16 rows fit a
// grid extent.
int check_rows(int N, int H) { return (int64_t)N * H > ((int64_t)1 << 34) ? SAGE_ERR_UNSUPPORTED : SAGE_OK; }

int check_cache(const sage_cache* c, int B, int N) {
  if (!c || B < 0 || N < 0 || c->pages < 0 || c->H < 0) return SAGE_ERR_INVALID_ARG;
  const int rc = check_dims(B, N, c->H, c->D);
  if (rc) return rc;
  for (int f : {c->k_format, c->v_format})
    if (f != SAGE_CACHE_INT8 && f != SAGE_CACHE_E4M3) return SAGE_ERR_INVALID_ARG;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128) return SAGE_ERR_UNSUPPORTED;
  if ((int64_t)c->pages * c->H * c->page_size > INT32_MAX) return SAGE_ERR_UNSUPPORTED;
  return SAGE_OK;
}

// The rest of a non-empty call's common arguments.
int check_table(const sage_cache* c, const int32_t* table, int table_pages, const int32_t* a, const int32_t* b,
                void* ws, size_t ws_bytes, size_t need) {
  if (!c->k_codes || !c->v_codes || !c->k_scale || !c->v_scale || !table) return SAGE_ERR_INVALID_ARG;
  if (table_pages < 1 || c->pages < 1) return SAGE_ERR_INVALID_ARG;
  if ((int64_t)table_pages * c->page_size > (1 << 28)) return SAGE_ERR_UNSUPPORTED;
  if (!aligned16(c->k_codes) || !aligned16(c->v_codes) || !aligned16(c->k_scale) || !aligned16(c->v_scale) ||
      !aligned4(table) || !aligned4(a) || !aligned4(b))
    return SAGE_ERR_UNSUPPORTED;
  return check_ws(ws, ws_bytes, need);
}

CacheArgs cache_args(const sage_cache* c, const int32_t* table, int table_pages, void* ws) {
  CacheArgs a;
  a.codes[0] = static_cast<uint8_t*>(c->k_codes);
  a.codes[1] = static_cast<uint8_t*>(c->v_codes);
  a.scale[0] = c->k_scale;
  a.scale[1] = c->v_scale;
  a.format[0] = c->k_format;
  a.format[1] = c->v_format;
  a.pages = c->pages;
  a.page_shift = c->page_size == 16 ? 4 : c->page_size == 32 ? 5 : c->page_size == 64 ? 6 : 7;
  a.H = c->H;
  a.D = c->D;
  a.table = table;
  a.table_pages = table_pages;
  a.status = static_cast<DeviceStatus*>(ws);
  return a;
}

}  // namespace

extern "C" {

int sage_clear_device_status(void* workspace, void* stream) {
  if (!workspace) return SAGE_ERR_INVALID_ARG;
  return cudaMemsetAsync(workspace, 0, SAGE_STATUS_BYTES, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? SAGE_OK
             : SAGE_ERR_CUDA;
}

int sage_rope_freqs(const sage_rope_config* c, double* inv_freq, float* mscale) {
  if (!c || !inv_freq || !mscale) return SAGE_ERR_INVALID_ARG;
  if (c->rot_dim < 2 || c->rot_dim % 2 || c->rot_dim > 128) return SAGE_ERR_UNSUPPORTED;
  if (c->scaling < SAGE_ROPE_PLAIN || c->scaling > SAGE_ROPE_YARN) return SAGE_ERR_INVALID_ARG;
  if (!(c->base > 1.0) || !isfinite(c->base)) return SAGE_ERR_INVALID_ARG;
  const int rot = c->rot_dim;
  const double factor = c->scaling == SAGE_ROPE_PLAIN ? 1.0 : c->factor;
  if (!(factor >= 1.0) || !isfinite(factor)) return SAGE_ERR_INVALID_ARG;
  double base = c->base;
  if (c->scaling == SAGE_ROPE_NTK) {
    if (rot == 2) return SAGE_ERR_UNSUPPORTED;  // one frequency, which is 1 for every base
    base *= pow(factor, (double)rot / (rot - 2));
  }
  *mscale = 1.0f;
  for (int j = 0; j < rot / 2; ++j) inv_freq[j] = pow(base, -2.0 * j / rot);
  if (c->scaling == SAGE_ROPE_LINEAR)
    for (int j = 0; j < rot / 2; ++j) inv_freq[j] /= factor;
  if (c->scaling == SAGE_ROPE_YARN) {
    if (!(c->trained_len >= 1.0) || !isfinite(c->trained_len) || !(c->beta_fast > c->beta_slow) ||
        !(c->beta_slow > 0.0) || !isfinite(c->beta_fast))
      return SAGE_ERR_INVALID_ARG;
    // pair number that makes `turns` turns over the trained length
    auto pair = [&](double turns) { return rot * log(c->trained_len / (turns * 6.283185307179586)) / (2.0 * log(base)); };
    const double lo = fmax(0.0, floor(pair(c->beta_fast)));
    const double hi = fmin(rot - 1.0, ceil(pair(c->beta_slow)));
    const double width = fmax(hi - lo, 0.001);
    for (int j = 0; j < rot / 2; ++j) {
      const double ramp = fmin(1.0, fmax(0.0, (j - lo) / width));
      inv_freq[j] *= ramp / factor + (1.0 - ramp);
    }
    *mscale = (float)(0.1 * log(factor) + 1.0);
  }
  return SAGE_OK;
}

int sage_rope(sage_view_bf16 q, int Hq, void* q_out, int64_t q_out_stride_b, int64_t q_out_stride_n,
              int64_t q_out_stride_h, sage_view_bf16 k, int Hk, void* k_out, int64_t k_out_stride_b,
              int64_t k_out_stride_n, int64_t k_out_stride_h, const int32_t* positions, int64_t pos_stride_b,
              const double* inv_freq, float mscale, int layout, int rot_dim, int inverse, int B, int N, int D,
              void* stream) {
  int rc;
  if (Hq < 0 || Hk < 0 || pos_stride_b < 0) return SAGE_ERR_INVALID_ARG;
  if ((rc = check_dims(B, N, Hq, D)) || (rc = check_dims(B, N, Hk, D))) return rc;
  if (layout != SAGE_ROPE_HALF && layout != SAGE_ROPE_INTERLEAVED) return SAGE_ERR_INVALID_ARG;
  if (rot_dim < 2 || rot_dim % 2 || rot_dim > D) return SAGE_ERR_UNSUPPORTED;
  if ((int64_t)B * N > INT32_MAX) return SAGE_ERR_UNSUPPORTED;
  if (!isfinite(mscale)) return SAGE_ERR_INVALID_ARG;
  if (empty(B, N, Hq + Hk)) return SAGE_OK;
  if (Hq && ((rc = check_view(q)) || (rc = check_out(q_out, q_out_stride_b, q_out_stride_n, q_out_stride_h)))) return rc;
  if (Hk && ((rc = check_view(k)) || (rc = check_out(k_out, k_out_stride_b, k_out_stride_n, k_out_stride_h)))) return rc;
  if (!inv_freq) return SAGE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(inv_freq) & 7u) || !aligned4(positions)) return SAGE_ERR_UNSUPPORTED;
  RopeArgs a;
  a.q = RopeSide{static_cast<const uint16_t*>(q.data), q.stride_b, q.stride_n, q.stride_h,
                 static_cast<uint16_t*>(q_out), q_out_stride_b, q_out_stride_n, q_out_stride_h};
  a.k = RopeSide{static_cast<const uint16_t*>(k.data), k.stride_b, k.stride_n, k.stride_h,
                 static_cast<uint16_t*>(k_out), k_out_stride_b, k_out_stride_n, k_out_stride_h};
  a.positions = positions;
  a.pos_stride_b = pos_stride_b;
  a.inv_freq = inv_freq;
  a.mscale = mscale;
  a.B = B; a.N = N; a.Hq = Hq; a.Hk = Hk; a.D = D; a.rot = rot_dim;
  a.half = layout == SAGE_ROPE_HALF;
  a.inverse = inverse != 0;
  auto same = [](const RopeSide& s) { return s.x == s.y && s.sb == s.yb && s.sn == s.yn && s.sh == s.yh; };
  a.in_place = (!Hq || same(a.q)) && (!Hk || same(a.k));
  return launch_rope(a, static_cast<cudaStream_t>(stream));
}

int sage_cache_append(const sage_cache* cache, sage_view_bf16 k, sage_view_bf16 v, const int32_t* page_table,
                      int table_pages, const int32_t* start, const int32_t* count, int B, int N, void* workspace,
                      size_t workspace_bytes, void* stream) {
  int rc = check_cache(cache, B, N);
  if (rc) return rc;
  if (empty(B, N, cache->H)) return SAGE_OK;
  if ((rc = check_view(k)) || (rc = check_view(v)) || (rc = check_rows(N, cache->H))) return rc;
  if ((rc = check_table(cache, page_table, table_pages, start, count, workspace, workspace_bytes, SAGE_STATUS_BYTES)))
    return rc;
  AppendArgs a;
  a.c = cache_args(cache, page_table, table_pages, workspace);
  const sage_view_bf16* in[2] = {&k, &v};
  for (int i = 0; i < 2; ++i) {
    a.x[i] = static_cast<const uint16_t*>(in[i]->data);
    a.sb[i] = in[i]->stride_b; a.sn[i] = in[i]->stride_n; a.sh[i] = in[i]->stride_h;
  }
  a.start = start;
  a.count = count;
  a.B = B; a.N = N;
  return launch_cache_append(a, static_cast<cudaStream_t>(stream));
}

int sage_cache_read(const sage_cache* cache, const int32_t* page_table, int table_pages, const int32_t* start,
                    const int32_t* count, void* k_out, int64_t k_out_stride_b, int64_t k_out_stride_n,
                    int64_t k_out_stride_h, void* v_out, int64_t v_out_stride_b, int64_t v_out_stride_n,
                    int64_t v_out_stride_h, int B, int N, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_cache(cache, B, N);
  if (rc) return rc;
  if (empty(B, N, cache->H)) return SAGE_OK;
  if (!k_out && !v_out) return SAGE_ERR_INVALID_ARG;
  if ((k_out && (rc = check_out(k_out, k_out_stride_b, k_out_stride_n, k_out_stride_h))) ||
      (v_out && (rc = check_out(v_out, v_out_stride_b, v_out_stride_n, v_out_stride_h))) ||
      (rc = check_rows(N, cache->H)))
    return rc;
  if ((rc = check_table(cache, page_table, table_pages, start, count, workspace, workspace_bytes, SAGE_STATUS_BYTES)))
    return rc;
  ReadArgs a;
  a.c = cache_args(cache, page_table, table_pages, workspace);
  a.y[0] = static_cast<uint16_t*>(k_out);
  a.y[1] = static_cast<uint16_t*>(v_out);
  a.yb[0] = k_out_stride_b; a.yn[0] = k_out_stride_n; a.yh[0] = k_out_stride_h;
  a.yb[1] = v_out_stride_b; a.yn[1] = v_out_stride_n; a.yh[1] = v_out_stride_h;
  a.start = start;
  a.count = count;
  a.B = B; a.N = N;
  return launch_cache_read(a, static_cast<cudaStream_t>(stream));
}

int sage_cache_attn(sage_view_bf16 q, const sage_cache* cache, const int32_t* page_table, int table_pages,
                    const int32_t* context, const int32_t* count, const uint32_t* mask, void* out,
                    int64_t out_stride_b, int64_t out_stride_n, int64_t out_stride_h, float* lse, int B, int T, int Hq,
                    float sm_scale, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_cache(cache, B, T);
  if (rc) return rc;
  if ((rc = check_dims(B, T, Hq, cache->D))) return rc;
  if (empty(B, T, Hq)) return SAGE_OK;
  if (cache->H == 0 || Hq % cache->H) return SAGE_ERR_INVALID_ARG;
  if (T > SAGE_CACHE_MAX_DRAFT) return SAGE_ERR_UNSUPPORTED;
  if ((rc = check_view(q)) || (rc = check_out(out, out_stride_b, out_stride_n, out_stride_h))) return rc;
  if (!context) return SAGE_ERR_INVALID_ARG;
  if (!aligned4(mask) || !aligned4(lse)) return SAGE_ERR_UNSUPPORTED;
  if ((rc = check_table(cache, page_table, table_pages, context, count, workspace, workspace_bytes,
                        align_up(SAGE_STATUS_BYTES) + cache_attn_workspace_bytes())))
    return rc;
  CacheAttnArgs a;
  a.c = cache_args(cache, page_table, table_pages, workspace);
  a.q = static_cast<const uint16_t*>(q.data);
  a.qb = q.stride_b; a.qn = q.stride_n; a.qh = q.stride_h;
  a.context = context;
  a.count = count;
  a.mask = mask;
  a.out = static_cast<uint16_t*>(out);
  a.ob = out_stride_b; a.on = out_stride_n; a.oh = out_stride_h;
  a.lse = lse;
  a.B = B; a.T = T; a.Hq = Hq; a.G = Hq / cache->H;
  a.sl2 = log2_scale(sm_scale, cache->D);
  a.workspace = at<void>(workspace, align_up(SAGE_STATUS_BYTES));
  a.wait_limit = debug_wait_limit();
  a.stall_tile = debug_stall_tile();
  return launch_cache_attn(a, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
