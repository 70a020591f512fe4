// Writing the quantised key/value cache and reading it back.
//
// A page holds `page` tokens of one sequence for every head as e4m3 codes
// [Hkv, page, D], with one power-of-two scale per (page, head): the least 2^e with
// amax <= 448 * 2^e.  Dividing by it and multiplying it back are exact, so a value
// is rounded once, to 4 significant bits.
#include "serve.cuh"

namespace cpa {
namespace {

// ---------------------------------------------------------------- append
// One CTA quantises one run of new rows inside one page, for one head of k or v.  Its rows come by
// asynchronous copies into shared memory (each thread reads back only what it copied itself, so
// there is no barrier on the data), are searched for their largest magnitude there and then
// rounded: each is read once and each code written once.  Bound by HBM for prompts (254 MB, 41000
// tokens of 8 heads, in 43 us; kept in registers between the two passes, which left 640 threads
// on an SM, 53 us), by latency for single tokens.
//
// Runs are found without a plan: sequence b with n_b rows touches at most
// floor((c_b + n_b) / page) - floor(c_b / page) + 2 pages (c_b its first packed row),
// so slots floor(c_b / page) + 2b onwards are its own; a slot past its last page
// returns at once.
constexpr int kAppendThreads = 128;

// The 8 values of vector v of a run in shared memory as fp32: bf16 16 bytes a vector; fp32 two
// planes of 16 bytes a vector.
template <bool kBf16>
__device__ __forceinline__ void vec_f32(float (&x)[8], const uint4* sm, uint32_t v, uint32_t plane) {
  const uint4 a = sm[v];
  if constexpr (kBf16) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    const uint4 c = sm[v + plane];
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
  }
}

__device__ __forceinline__ void cp_async16(void* smem_dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(smem_dst)),
               "l"(reinterpret_cast<uint64_t>(src))
               : "memory");
}

template <bool kBf16>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const CacheRowsArgs a) {
  extern __shared__ uint4 rows_sm[];  // a page's worth of one head's rows
  const int page = a.page;
  // heads fastest: the CTAs that run together read whole rows
  const int head = blockIdx.x % a.Hkv, rest = blockIdx.x / a.Hkv, is_v = rest & 1, slot = rest >> 1;
  grid_dependency_wait();
  grid_launch_dependents();
  int b, c0, n;
  int64_t s0;
  if (a.n_seqs <= 32) {  // one round of loads finds the sequence and brings what is needed of it
    const int lane = threadIdx.x & 31, i = min(lane, a.n_seqs - 1);
    int first, count;
    seq_rows(a.cu_rows, i, a.rows, &first, &count);
    const int start = ld(a.start + i);
    const bool le = lane < a.n_seqs && first / page + 2 * lane <= slot;
    b = 31 - __clz(__ballot_sync(0xffffffffu, le) | 1u);
    c0 = __shfl_sync(0xffffffffu, first, b);
    n = __shfl_sync(0xffffffffu, count, b);
    s0 = __shfl_sync(0xffffffffu, start, b);
  } else {
    b = warp_find(a.n_seqs, slot, [&](int i) {
      return (min(max((int64_t)ld(a.cu_rows + i), (int64_t)0), a.rows) / page) + 2 * i;
    });
    seq_rows(a.cu_rows, b, a.rows, &c0, &n);
    s0 = ld(a.start + b);
  }
  if (n == 0) return;
  if (s0 < 0) {
    record_device_error(a.err, kDevIndex);
    return;
  }
  const int64_t p = s0 / page + (slot - (c0 / page + 2 * b));  // page of the sequence
  const int64_t t0 = max(s0, p * page), t1 = min(s0 + n, (p + 1) * page);
  if (t0 >= t1) return;
  const uint32_t vpr = a.D >> 3, log_vpr = 31 - __clz(vpr);  // vectors of 8 values a row
  const uint32_t plane = (uint32_t)page << log_vpr;
  const int s_first = (int)(t0 - p * page), n_run = (int)(t1 - t0);
  constexpr int64_t es = kBf16 ? 2 : 4;
  const char* src = static_cast<const char*>(is_v ? a.v_rows : a.k_rows) +
                    ((c0 + (t0 - s0)) * a.row_ld + (int64_t)head * a.D) * es;
  const uint32_t nv = (uint32_t)n_run << log_vpr;
  for (uint32_t v = threadIdx.x; v < nv; v += kAppendThreads) {
    const char* from = src + (int64_t)(v >> log_vpr) * a.row_ld * es + (v & (vpr - 1)) * 8 * es;
    cp_async16(rows_sm + v, from);
    if (!kBf16) cp_async16(rows_sm + v + plane, from + 16);
  }
  // the page's id and scale come while the rows do
  const int id = page_id(a.page_table, a.max_pages, a.n_pages, b, p, a.err);
  const int64_t blk = (int64_t)id * a.Hkv + head;
  float* scale = (is_v ? a.v_scale : a.k_scale) + blk;
  const uint32_t old_bits = s_first > 0 && id >= 0 ? __float_as_uint(*scale) : 0u;
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (id < 0) return;
  uint8_t* codes = (is_v ? a.v : a.k) + blk * page * a.D;

  // the bits of the run's largest magnitude (NaN above infinity above every finite value)
  uint32_t mx = 0;
#pragma unroll 4
  for (uint32_t v = threadIdx.x; v < nv; v += kAppendThreads) {
    float x[8];
    vec_f32<kBf16>(x, rows_sm, v, plane);
#pragma unroll
    for (int j = 0; j < 8; ++j) mx = max(mx, __float_as_uint(x[j]) & 0x7fffffffu);
  }
  mx = __reduce_max_sync(0xffffffffu, mx);
  __shared__ uint32_t wmax[kAppendThreads / 32];
  if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = mx;
  __syncthreads();  // also: every thread has read the old scale
#pragma unroll
  for (int i = 0; i < kAppendThreads / 32; ++i) mx = max(mx, wmax[i]);

  // 448 = 1.75 * 2^8: amax = 1.f * 2^x needs e = x - 8, one more when its fraction passes .75
  int e = max((int)(mx >> 23) - 127 - 8 + ((mx & 0x7fffffu) > 0x600000u ? 1 : 0), kScaleExpMin);
  const int e_old = (int)(old_bits >> 23) - 127;
  const bool nan = mx >= 0x7f800000u || old_bits >= 0x7f800000u;
  if (s_first > 0 && !nan) e = max(e, min(max(e_old, kScaleExpMin), kScaleExpMax));
  e = min(e, kScaleExpMax);
  const float inv = nan ? 0.f : pow2i(-e);

  if (s_first > 0 && !nan && e > e_old) {  // earlier tokens move to the grown scale
    const float f = pow2i(max(e_old - e, -126));
    for (uint32_t v = threadIdx.x; v < (uint32_t)s_first << log_vpr; v += kAppendThreads) {
      uint2* c = reinterpret_cast<uint2*>(codes) + v;
      const uint2 w = *c;
      uint32_t o[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t x = k ? w.y : w.x;
        const float2 lo = f16x2_to_f32(e4m3x2_to_f16x2(x & 0xffffu)), hi = f16x2_to_f32(e4m3x2_to_f16x2(x >> 16));
        o[k] = e4m3x2(lo.x * f, lo.y * f) | (e4m3x2(hi.x * f, hi.y * f) << 16);
      }
      *c = make_uint2(o[0], o[1]);
    }
  }
  uint2* dst = reinterpret_cast<uint2*>(codes + s_first * a.D);  // the run's slots are consecutive
#pragma unroll 4
  for (uint32_t v = threadIdx.x; v < nv; v += kAppendThreads) {
    float x[8];
    vec_f32<kBf16>(x, rows_sm, v, plane);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = nan ? 0.f : x[j] * inv;
    __stcs(dst + v, make_uint2(e4m3x2(x[0], x[1]) | (e4m3x2(x[2], x[3]) << 16),
                               e4m3x2(x[4], x[5]) | (e4m3x2(x[6], x[7]) << 16)));
  }
  if (threadIdx.x == 0) *scale = nan ? __uint_as_float(0x7fc00000u) : pow2i(e);
}

// ---------------------------------------------------------------- read
// One CTA brings kReadRows consecutive packed rows of one head of k or v back.
constexpr int kReadRows = 64;
constexpr int kReadThreads = 256;
constexpr int64_t kNoPage = -1, kNoRow = -2;

template <bool kBf16>
__global__ void __launch_bounds__(kReadThreads) kv_read_kernel(const CacheRowsArgs a) {
  __shared__ int32_t at[kReadRows];     // slot of a row's token in its page
  __shared__ int64_t blk0[kReadRows];  // block of head 0 in its page, or kNoPage / kNoRow
  const int head = blockIdx.x % a.Hkv, rest = blockIdx.x / a.Hkv, is_v = rest & 1;  // heads fastest
  const int64_t r0 = (int64_t)(rest >> 1) * kReadRows;
  grid_dependency_wait();
  grid_launch_dependents();
  const int n = (int)min((int64_t)kReadRows, a.rows - r0);
  for (int i = threadIdx.x; i < n; i += kReadThreads) {
    const int64_t row = r0 + i;
    int lo = 0, hi = a.n_seqs - 1;
    while (lo < hi) {  // largest b with cu_rows[b] <= row
      const int mid = (lo + hi + 1) >> 1;
      if (ld(a.cu_rows + mid) <= row) lo = mid; else hi = mid - 1;
    }
    if (row < ld(a.cu_rows + lo) || row >= ld(a.cu_rows + lo + 1)) {  // no sequence's row: left as it is
      blk0[i] = kNoRow;
      continue;
    }
    const int64_t tok = (int64_t)ld(a.start + lo) + row - ld(a.cu_rows + lo);
    int id = -1;
    if (tok < 0) record_device_error(a.err, kDevIndex);
    else id = page_id(a.page_table, a.max_pages, a.n_pages, lo, tok / a.page, a.err);
    blk0[i] = id < 0 ? kNoPage : (int64_t)id * a.Hkv;
    at[i] = (int32_t)(tok % a.page);
  }
  __syncthreads();
  const uint8_t* codes = is_v ? a.v : a.k;
  const float* scales = is_v ? a.v_scale : a.k_scale;
  char* dst = static_cast<char*>(is_v ? a.v_rows : a.k_rows);
  const int vpr = a.D >> 3;
  for (int v = threadIdx.x; v < n * vpr; v += kReadThreads) {
    const int i = v / vpr, c = (v % vpr) * 8;
    if (blk0[i] == kNoRow) continue;
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (blk0[i] >= 0) {
      const int64_t blk = blk0[i] + head;
      const uint2 w = __ldcs(reinterpret_cast<const uint2*>(codes + (blk * a.page + at[i]) * a.D + c));
      const float s = ld(scales + blk);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t u = k ? w.y : w.x;
        const float2 lo = f16x2_to_f32(e4m3x2_to_f16x2(u & 0xffffu)), hi = f16x2_to_f32(e4m3x2_to_f16x2(u >> 16));
        x[4 * k] = lo.x * s;
        x[4 * k + 1] = lo.y * s;
        x[4 * k + 2] = hi.x * s;
        x[4 * k + 3] = hi.y * s;
      }
    }
    const int64_t e = (r0 + i) * a.row_ld + (int64_t)head * a.D + c;
    if constexpr (kBf16) {
      __nv_bfloat162 h[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) h[k] = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
      __stcs(reinterpret_cast<uint4*>(dst + e * 2), *reinterpret_cast<uint4*>(h));
    } else {
      __stcs(reinterpret_cast<float4*>(dst + e * 4), make_float4(x[0], x[1], x[2], x[3]));
      __stcs(reinterpret_cast<float4*>(dst + e * 4) + 1, make_float4(x[4], x[5], x[6], x[7]));
    }
  }
}

}  // namespace

cp_status launch_kv_append(const CacheRowsArgs& a, int is_bf16, cudaStream_t st) {
  const int64_t blocks = (a.rows / a.page + 2 * (int64_t)a.n_seqs) * a.Hkv * 2;
  if (blocks > INT32_MAX) {
    set_last_error("too many rows, sequences and heads for one launch");
    return CP_ERR_UNSUPPORTED;
  }
  const size_t smem = (size_t)a.page * a.D * (is_bf16 ? 2 : 4);  // at most 64 KiB
  if (!is_bf16) {
    static KernelReady ready;
    int sms = 0;
    const cp_status r = ready.prepare(kv_append_kernel<false>, 64 * 1024, "kv_append_kernel", &sms, [] { return CP_OK; });
    if (r != CP_OK) return r;
    return launch_chained(kv_append_kernel<false>, dim3((unsigned)blocks), kAppendThreads, smem, st,
                          "kv_append_kernel launch", a);
  }
  return launch_chained(kv_append_kernel<true>, dim3((unsigned)blocks), kAppendThreads, smem, st,
                        "kv_append_kernel launch", a);
}

cp_status launch_kv_read(const CacheRowsArgs& a, int is_bf16, cudaStream_t st) {
  const int64_t blocks = (a.rows + kReadRows - 1) / kReadRows * a.Hkv * 2;
  if (blocks > INT32_MAX) {
    set_last_error("too many rows and heads for one launch");
    return CP_ERR_UNSUPPORTED;
  }
  const dim3 grid((unsigned)blocks);
  return launch_chained(is_bf16 ? kv_read_kernel<true> : kv_read_kernel<false>, grid, kReadThreads, 0, st,
                        "kv_read_kernel launch", a);
}

}  // namespace cpa
