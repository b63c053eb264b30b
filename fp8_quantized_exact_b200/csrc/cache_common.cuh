// Launch parameter blocks of the rotary positions and of the quantised paged
// cache, and the lookup of a token's row.
#pragma once
#include "sage_common.cuh"

namespace sage {

// The serving kernels are short and follow one another, so each is launched as a programmatic dependent of what is before
// it on its stream: its blocks become resident while that drains, prepare what needs no input, and wait in
// `begin_dependent` until it has completed and its writes are visible.  What follows is let on only behind that wait,
// so at most two of these kernels overlap, and no block of a later one is resident before the one two
// back has ended.  Inputs are read by plain loads: the read-only path is for what nobody writes during a kernel's life.
__device__ __forceinline__ void begin_dependent() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <class... P, class... A>
int launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A&&... args) {
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...) == cudaSuccess ? SAGE_OK : SAGE_ERR_CUDA;
}

// One tensor of a rotary call: input and output with element strides.
struct RopeSide {
  const uint16_t* x;
  int64_t sb, sn, sh;
  uint16_t* y;
  int64_t yb, yn, yh;
};
struct RopeArgs {
  RopeSide q, k;
  const int32_t* positions;  // [B][N] with row stride pos_stride_b, or null: 0 .. N-1
  int64_t pos_stride_b;
  const double* inv_freq;    // [rot / 2]
  float mscale;
  int B, N, Hq, Hk, D, rot;
  bool half, inverse;
  bool in_place;             // both outputs are their inputs: channels from rot on stay as they are
};
int launch_rope(const RopeArgs& a, cudaStream_t s);

// Codes [pages][H][page][D] and scales [pages][H][page] of K and V, and the
// page table [B][table_pages].
struct CacheArgs {
  uint8_t* codes[2];  // K, V
  float* scale[2];
  int format[2];
  int pages, page_shift, H, D;
  const int32_t* table;
  int table_pages;
  DeviceStatus* status;
};

// Checks that a kernel can fail on device data; `where` in the status word.
enum CacheWhere { kWhereAppend = 40, kWhereRead = 41, kWhereAttn = 42 };

__device__ __forceinline__ void flag_bad(DeviceStatus* st, int where) {
  if (atomicCAS(&st->code, 0, (int)SAGE_ERR_DEVICE) == 0) {
    st->where = where;
    st->block = (int)(blockIdx.x + gridDim.x * (blockIdx.y + gridDim.y * blockIdx.z));
  }
}

// The row (of the [pages][H][page] rows) of slot `slot` of sequence b and
// head h, or -1 where the slot is behind the table or its entry names no page.
__device__ __forceinline__ int64_t cache_row(const CacheArgs& c, int b, int h, int64_t slot) {
  if (slot < 0 || (slot >> c.page_shift) >= c.table_pages) return -1;
  const int page = c.table[(int64_t)b * c.table_pages + (int)(slot >> c.page_shift)];
  if (page < 0 || page >= c.pages) return -1;
  return (((int64_t)page * c.H + h) << c.page_shift) + (slot & ((1 << c.page_shift) - 1));
}

struct AppendArgs {
  CacheArgs c;
  const uint16_t* x[2];  // K, V: BF16 [B, N, H, D]
  int64_t sb[2], sn[2], sh[2];
  const int32_t* start;  // [B] or null: 0
  const int32_t* count;  // [B] or null: N
  int B, N;
};
int launch_cache_append(const AppendArgs& a, cudaStream_t s);

struct ReadArgs {
  CacheArgs c;
  uint16_t* y[2];  // K, V outputs; either may be null
  int64_t yb[2], yn[2], yh[2];
  const int32_t* start;
  const int32_t* count;
  int B, N;
};
int launch_cache_read(const ReadArgs& a, cudaStream_t s);

struct CacheAttnArgs {
  CacheArgs c;
  const uint16_t* q;       // BF16 [B, T, Hq, D]
  int64_t qb, qn, qh;
  const int32_t* context;  // [B]
  const int32_t* count;    // [B] or null: T
  const uint32_t* mask;    // [B][T][ceil(T/32)] or null: token i sees drafted tokens 0 .. i
  uint16_t* out;
  int64_t ob, on, oh;
  float* lse;              // [B][T][Hq] or null
  int B, T, Hq, G;         // G = Hq / H
  float sl2;               // fl32(sm_scale * log2 e)
  void* workspace;
  long long wait_limit;    // clock cycles a bounded device wait may spin
  int stall_tile;          // test hook: the producers withhold this tile of their own counting (-1: none)
};
size_t cache_attn_workspace_bytes();
int launch_cache_attn(const CacheAttnArgs& a, cudaStream_t s);
int launch_cache_attn_tc(const CacheAttnArgs& a, cudaStream_t s);  // its variant for many rows per head

}  // namespace sage
