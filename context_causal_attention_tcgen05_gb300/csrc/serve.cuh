// Shared by the key/value cache and rotary translation units: launch arguments,
// device-side lookups of ragged batches and pages, e4m3 conversions.
#pragma once

#include <atomic>

#include "common.cuh"

namespace cpa {

// The kernels of a step follow one another closely, so each may be launched while the
// one before it still runs: it sets up, waits (grid_dependency_wait, before its first
// access to memory another kernel may have written or read) until that one is complete,
// and lets the next one come (grid_launch_dependents).  Launched behind another kernel
// this is an ordinary launch.
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
// Memory that a kernel before may still be writing after this one has started is read by ordinary loads:
// the read-only path is for what nothing writes while the kernel lives, and the compiler may move such a
// load in front of the wait.
template <class T>
__device__ __forceinline__ T ld(const T* p) {
  return *p;
}
template <class... P, class... A>
cp_status launch_chained(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, const char* what,
                         const A&... args) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = grid;
  lc.blockDim = dim3((unsigned)threads);
  lc.dynamicSmemBytes = smem;
  lc.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = at;
  lc.numAttrs = 1;
  return cuda_check(cudaLaunchKernelEx(&lc, kern, args...), what);
}

// What a kernel needs once a device: its shared memory limit raised, and checks of its own.
struct KernelReady {
  std::atomic<int> sms_of[64] = {};
  template <class K, class F>
  cp_status prepare(K kern, int smem, const char* what, int* sms, F extra) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && dev >= 0 && dev < 64 && (*sms = sms_of[dev].load(std::memory_order_acquire)) > 0) return CP_OK;
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return cuda_check(e, what);
    const cp_status r = extra();
    if (r == CP_OK && dev < 64) sms_of[dev].store(*sms, std::memory_order_release);
    return r;
  }
};

constexpr int kScaleExpMin = -100;  // exponents of a block's power-of-two scale
constexpr int kScaleExpMax = 120;

// Rows of a ragged batch written to or read from the cache (cp_kv_cache_append / _read).
struct CacheRowsArgs {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  const int32_t* page_table;
  const int32_t* cu_rows;
  const int32_t* start;
  void* k_rows;  // [rows, Hkv, D], consecutive rows row_ld elements apart
  void* v_rows;
  int64_t rows, row_ld;
  int32_t n_pages, n_seqs, max_pages, Hkv, page, D;
  int32_t* err;
};

// Attention over the cache (cp_kv_cache_attention).
struct CacheAttnArgs {
  const uint8_t* k;
  const uint8_t* v;
  const float* k_scale;
  const float* v_scale;
  const int32_t* page_table;
  const int32_t* cu_q;
  const int32_t* kv_len;
  const int32_t* q_pos;  // or nullptr
  const void* q;
  void* out;
  float* lse;
  int64_t rows, q_ld;
  int64_t k_offset, k_stride;
  int32_t n_pages, n_seqs, max_pages, Hkv, page, D;
  int32_t Hq, G;  // G = Hq / Hkv
  int32_t causal, window;
  float scale_log2;  // softmax scale * log2(e)
  int32_t* err;
};

cp_status launch_kv_append(const CacheRowsArgs& a, int is_bf16, cudaStream_t st);
cp_status launch_kv_read(const CacheRowsArgs& a, int is_bf16, cudaStream_t st);
cp_status launch_kv_attention(const CacheAttnArgs& a, int is_bf16, void* ws, cudaStream_t st);
size_t kv_attention_ws(int64_t rows, int32_t Hq, int32_t Hkv, int32_t D, int32_t is_bf16, int32_t n_seqs);

struct RotaryArgs {
  const void* x[2];  // q, k
  void* y[2];
  int64_t x_ld[2], y_ld[2];
  int32_t H[2];
  int64_t S;
  int32_t D, rot, n_axes;
  int32_t axis_end[4];  // first pair after each axis's section
  const int32_t* positions;
  const float* inv_freq;
  int32_t inverse;
};
cp_status launch_rotary(const RotaryArgs& a, int is_bf16, int interleaved, cudaStream_t st);

// ---------------------------------------------------------------- device helpers

// Two fp32 to two e4m3 codes (lo in the low byte), nearest even, saturating.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e4m3 codes to two halves (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)codes));
  return r;
}
__device__ __forceinline__ float2 f16x2_to_f32(uint32_t h) {
  float2 f;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}
// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// Largest b in [0, n) with f(b) <= x, for f ascending with f(0) <= x; every lane of the
// warp takes part and gets b.  32 probes a round: two dependent loads reach 1024 entries.
template <class F>
__device__ __forceinline__ int warp_find(int n, int64_t x, F f) {
  const int lane = threadIdx.x & 31;
  int lo = 0, len = n;
  while (len > 1) {
    const int step = (len + 31) / 32;
    const int b = lo + lane * step;
    const bool le = lane * step < len && f(b) <= x;
    const int last = 31 - __clz(__ballot_sync(0xffffffffu, le) | 1u);
    lo += last * step;
    len = min(step, len - last * step);
  }
  return lo;
}

// First and number of packed rows of sequence b, clamped into [0, rows].
__device__ __forceinline__ void seq_rows(const int32_t* cu, int b, int64_t rows, int* first, int* n) {
  const int64_t r0 = min(max((int64_t)ld(cu + b), (int64_t)0), rows);
  const int64_t r1 = min(max((int64_t)ld(cu + b + 1), r0), rows);
  *first = (int)r0;
  *n = (int)(r1 - r0);
}

// The page of entry p of sequence b's table; -1 (recorded as an index error) when the
// table has no such entry or the id names no page.
__device__ __forceinline__ int page_id(const int32_t* table, int max_pages, int n_pages, int b, int64_t p,
                                       int32_t* err) {
  int id = -1;
  if (p >= 0 && p < max_pages) id = ld(table + (int64_t)b * max_pages + p);
  if (id < 0 || id >= n_pages) {
    record_device_error(err, kDevIndex);
    return -1;
  }
  return id;
}

}  // namespace cpa
