// Shared by the cache attention kernels: units of work, their even division over the
// CTAs, and the join of units that several CTAs worked on.
//
// A sequence's packed rows (query row * G + head of the group) are cut into tiles of RT;
// a unit is one row tile and key/value head; its work is the 128-token tiles that any of
// its rows sees.  All units' tiles form one line in the order (row tile, head, tile), cut
// into equal runs, one a CTA: no length or mask leaves an SM idle.  A unit takes some places
// of the line before its first tile, which stand for the work around its tiles (its q, its
// first maximum, its result): runs end together whether they cross few units or many (64
// sequences of 750 to 3000 tokens, one row each, 54.9 us without such places, 52.3 so; three
// prompts' chunks of 150 to 300 rows 103.8 and 96.8).  A unit inside one run
// is written by its CTA; a unit cut between runs leaves per-row (m, l, O) in the
// workspace, and kv_attn_join_kernel adds them in the runs' order, so results do not
// depend on timing.
#pragma once

#include <cuda.h>

#include "ptx.cuh"
#include "serve.cuh"

namespace cpa {

// 2-D tensor map over codes [rows, D] with boxes of box_rows x box_cols, swizzled as wide as a row
// (`swizzle`, box_cols = D) or plain.
cp_status make_codes_map(CUtensorMap* m, const void* base, int64_t rows, int D, int box_rows, int box_cols,
                         bool swizzle);

// kv_attn_rows.cu: many rows a key, bf16.
size_t kv_attention_rows_ws(int64_t rows, int32_t G, int32_t Hkv, int32_t D, int32_t n_seqs);
cp_status launch_kv_attention_rows(const CacheAttnArgs& a, void* ws, cudaStream_t st);

namespace {

constexpr int kRowsMaxPairs = 80;  // CTA pairs its workspace has partial results for
constexpr int BK = 128;  // tokens per tile
constexpr float kLn2 = 0.6931471805599453f;

// log(sum * 2^m), -inf for an empty sum.  m may lie far from the result, with the sum as much larger:
// the sum's exponent joins it first.
__device__ __forceinline__ float lse_of(float m, float sum) {
  const int e = min(max((int)(__float_as_uint(sum) >> 23) - 127, -126), 126);  // (of NaN and infinity: any)
  return sum == 0.f ? -INFINITY : (m + (float)e + log2f(sum * pow2i(-e))) * kLn2;
}

// Result record of a (row slot, head) unit for the join.
struct UnitInfo {
  int32_t row;    // first packed (query row * G + g) of the unit
  int32_t nrows;  // rows (0: the slot holds none)
  int32_t c0;     // first CTA working on it (-1: no visible token)
  int32_t c1;     // last
};

// ---------------------------------------------------------------- planning
// Row tiles of sequence b (its n_b * G packed rows in tiles of RT) take the slots from
// floor(cu[b] * G / RT) + b on; ceil(n_b * G / RT) of them fit before the next one's.
struct SlotSeq {
  int b, c0, n, len;
};
__device__ __forceinline__ int64_t slot_base(const CacheAttnArgs& a, const int32_t* cu, int b, int RT) {
  return (min(max((int64_t)cu[b], (int64_t)0), a.rows) * a.G) / RT + b;
}
__device__ __forceinline__ void slot_seq(const CacheAttnArgs& a, const int32_t* cu, const int32_t* kl, int b,
                                         SlotSeq& s) {
  const int64_t r0 = min(max((int64_t)cu[b], (int64_t)0), a.rows);
  s.b = b;
  s.c0 = (int)r0;
  s.n = (int)(min(max((int64_t)cu[b + 1], r0), a.rows) - r0);
  const int cap = a.max_pages * a.page;
  s.len = min(max(kl[b], 0), cap);
  if (s.len != kl[b]) record_device_error(a.err, kDevIndex);
}
// Planning code runs once a unit and meets a cold instruction cache, so its largest part is
// a function of its own (decoding one token over 1000: 10.9 us inlined everywhere, 10.4 us so).
// The rows kernel defines it inline: a call costs its register split.
#ifndef KV_PLAN_INLINE
#define KV_PLAN_INLINE __noinline__
#endif

// Tokens [lo, hi) that query row i of the sequence sees.
__device__ KV_PLAN_INLINE int2 row_bounds_at(int64_t d, int64_t k_stride, int window, int len) {
  // d: the row's distance from token 0.  last visible token; last token before the window
  const int64_t last = k_stride == 1 ? d : floor_div(d, k_stride);
  const int hi = (int)max(min((int64_t)len, last + 1), (int64_t)0);
  int lo = 0;
  if (window > 0) {
    const int64_t first = k_stride == 1 ? d - window : floor_div(d - window, k_stride);
    lo = (int)min(max(first + 1, (int64_t)0), (int64_t)len);
  }
  return lo >= hi ? make_int2(0, 0) : make_int2(lo, hi);
}
__device__ __forceinline__ void row_bounds(const CacheAttnArgs& a, const SlotSeq& s, int i, int& lo, int& hi) {
  lo = 0;
  hi = s.len;
  if (!a.causal) return;
  const int64_t d = a.q_pos ? (int64_t)ld(a.q_pos + s.c0 + i) - a.k_offset
                            : ((int64_t)s.len - s.n + i) * a.k_stride;
  const int2 r = row_bounds_at(d, a.k_stride, a.window, s.len);
  lo = r.x;
  hi = r.y;
}
// Tokens [lo, hi) that the rows [r0, r0 + nrows) of a sequence (packed with G) see, hi = 0 for none.
__device__ __forceinline__ void rows_tokens(const CacheAttnArgs& a, const SlotSeq& s, int r0, int nrows, int& lo,
                                            int& hi) {
  lo = INT32_MAX;
  hi = 0;
  const int i0 = r0 / a.G, i1 = (r0 + nrows - 1) / a.G;
  if (!a.q_pos) {  // both bounds ascend: the first and the last row decide
    int l0, h0;
    row_bounds(a, s, i0, l0, h0);
    row_bounds(a, s, i1, lo, hi);
    lo = h0 > l0 ? l0 : 0;  // (a first row that sees nothing leaves the start open)
  } else {
#pragma unroll 8
    for (int i = i0; i <= i1; ++i) {
      int l, h;
      row_bounds(a, s, i, l, h);
      if (h > l) {
        lo = min(lo, l);
        hi = max(hi, h);
      }
    }
  }
  if (hi == 0) lo = 0;
}

// Rows of a slot that starts at packed row r0 of a sequence's `total` (r0 < 0: rows in front of the
// first sequence, which belong to none).
template <int RT>
__device__ __forceinline__ int slot_rows(int64_t r0, int64_t total) {
  return r0 < 0 ? 0 : (int)max((int64_t)0, min((int64_t)RT, total - r0));
}

// A slot's rows: r0 .. r0 + nrows - 1 of a sequence's packed rows, which see tokens [lo, hi), in
// tiles [t0, t1).
struct SlotRows {
  SlotSeq q;
  int r0, nrows, lo, hi;
  __device__ __forceinline__ int t0() const { return lo / BK; }
  __device__ __forceinline__ int t1() const { return (hi + BK - 1) / BK; }
};

struct WsPtrs {
  UnitInfo* info;  // [slots * Hkv]
  float2* ml;      // [2 * ctas][RT] maximum (log2) and sum
  float* o;        // [2 * ctas][RT][D]
};

// Evaluates slots [s_begin, s_end) in order: f(slot, rows); slots without rows have nrows = 0.
template <int RT, class F>
__device__ __forceinline__ void for_slots(const CacheAttnArgs& a, const int32_t* cu, const int32_t* kl, int s_begin,
                                          int s_end, F f) {
  if (s_begin >= s_end) return;
  int lo = 0, hi = a.n_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (slot_base(a, cu, mid, RT) <= s_begin) lo = mid; else hi = mid - 1;
  }
  SlotSeq q;
  slot_seq(a, cu, kl, lo, q);
  int64_t base = slot_base(a, cu, lo, RT);
  for (int s = s_begin; s < s_end; ++s) {
    while (q.b + 1 < a.n_seqs && slot_base(a, cu, q.b + 1, RT) <= s) {
      slot_seq(a, cu, kl, q.b + 1, q);
      base = slot_base(a, cu, q.b, RT);
    }
    const int64_t r0 = (s - base) * RT, total = (int64_t)q.n * a.G;
    SlotRows rows = {q, (int)r0, slot_rows<RT>(r0, total), 0, 0};
    if (rows.nrows > 0) rows_tokens(a, q, rows.r0, rows.nrows, rows.lo, rows.hi);
    if (!f(s, rows)) return;
  }
}


// This CTA's run: it starts at place `off` of unit (slot, head) and holds places [f0, f1) of T;
// slot < 0: nothing to do.
struct Run {
  int64_t f0, f1;
  int64_t base, more;  // run c holds base places, one more for c < more
  int slot, head, off;
};
template <int kWarps>
struct PlanSmem {
  int64_t scan[kWarps];
  int32_t slot, head, off;
  SlotRows rows;  // of the run's first slot
};

// Divides the line of tiles (every thread of the CTA takes part).  `lens`: shared memory for
// 2 * cap_seqs + 1 integers, where a batch that fits keeps its lengths meanwhile.  Slots whose
// rows see nothing get their record for the join here.
// `cta` of `ctas`: the worker (a CTA or a pair of CTAs).
template <int RT, int kCost, int kWarps>
__device__ __forceinline__ Run plan_run(const CacheAttnArgs& a, const WsPtrs& ws, int slots, int cta, int ctas,
                                        int32_t* lens, int cap_seqs, PlanSmem<kWarps>& sm) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kThreads = kWarps * 32;
  const int32_t *cu = a.cu_q, *kl = a.kv_len;
  if (tid == 0) sm.slot = -1;
  const bool staged = a.n_seqs <= cap_seqs;
  bool bad = false;
  for (int i = tid; i <= a.n_seqs; i += kThreads) {
    const int first = ld(a.cu_q + i), next = ld(a.cu_q + min(i + 1, a.n_seqs));
    const int len = ld(a.kv_len + min(i, a.n_seqs - 1));
    bad |= next < first;
    if (staged) {
      lens[i] = first;
      lens[a.n_seqs + 1 + min(i, a.n_seqs - 1)] = len;
    }
  }
  if (staged) {
    cu = lens;
    kl = lens + a.n_seqs + 1;
  }
  if (__syncthreads_or(bad)) {  // slots would not be the sequences' own: nothing is done
    if (tid == 0) record_device_error(a.err, kDevIndex);
    for (int64_t i = cta + (int64_t)tid * ctas; i < (int64_t)slots * a.Hkv; i += (int64_t)ctas * kThreads)
      ws.info[i] = {0, 0, -1, -1};
    return {0, 0, 0, 0, -1, 0, 0};
  }
  const int per = (slots + kThreads - 1) / kThreads;
  const int s_begin = min(tid * per, slots), s_end = min(s_begin + per, slots);
  int64_t mine = 0;
  SlotRows last;  // of the thread's last slot: its only one, usually
  for_slots<RT>(a, cu, kl, s_begin, s_end, [&](int s, const SlotRows& rows) {
    last = rows;
    const int c = rows.t1() - rows.t0();
    if (c > 0) mine += c + kCost;
    if (c == 0 && s % ctas == cta) {  // nothing visible: the join writes the rows
      const UnitInfo u = {(int32_t)((int64_t)rows.q.c0 * a.G + rows.r0), rows.nrows, -1, -1};
      for (int h = 0; h < a.Hkv; ++h) ws.info[(int64_t)s * a.Hkv + h] = u;
    }
    return true;
  });
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) sm.scan[warp] = incl;
  __syncthreads();
  int64_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sm.scan[w];
    total += sm.scan[w];
  }
  const int64_t T = total * a.Hkv, base = udiv_pos(T, ctas), more = T - base * ctas;
  const int64_t f0 = cta * base + min((int64_t)cta, more), f1 = f0 + base + (cta < more ? 1 : 0);
  {
    int64_t acc = before + incl - mine;  // places before this thread's slots
    if (f0 < f1 && f0 >= acc * a.Hkv && f0 < (acc + mine) * a.Hkv) {
      auto begin = [&](int s, const SlotRows& rows) {
        const int64_t c = rows.t1() - rows.t0() + kCost, rem = f0 - acc * a.Hkv;
        sm.slot = s;
        sm.head = (int)udiv_pos(rem, c);
        sm.off = (int)(rem - sm.head * c);
        sm.rows = rows;
      };
      if (per == 1) {
        begin(s_begin, last);
      } else {
        for_slots<RT>(a, cu, kl, s_begin, s_end, [&](int s, const SlotRows& rows) {
          const int64_t c = rows.hi > 0 ? rows.t1() - rows.t0() + kCost : 0;
          if (f0 < (acc + c) * a.Hkv) {
            begin(s, rows);
            return false;
          }
          acc += c;
          return true;
        });
      }
    }
  }
  __syncthreads();
  Run r;
  r.f0 = f0;
  r.f1 = f1;
  r.base = base;
  r.more = more;
  r.slot = sm.slot;
  r.head = sm.head;
  r.off = sm.off;
  return r;
}

// Moves to the next slot that has visible tokens (there is one while the run lasts).
template <int RT>
__device__ __forceinline__ bool next_rows(const CacheAttnArgs& a, int slots, int& slot, SlotRows& s) {
  while (++slot < slots) {
    while (s.q.b + 1 < a.n_seqs && slot_base(a, a.cu_q, s.q.b + 1, RT) <= slot)
      slot_seq(a, a.cu_q, a.kv_len, s.q.b + 1, s.q);
    const int64_t r0 = (slot - slot_base(a, a.cu_q, s.q.b, RT)) * RT;
    s.r0 = (int)r0;
    s.nrows = slot_rows<RT>(r0, (int64_t)s.q.n * a.G);
    s.lo = s.hi = 0;
    if (s.nrows > 0) rows_tokens(a, s.q, s.r0, s.nrows, s.lo, s.hi);
    if (s.hi > 0) return true;
  }
  return false;
}

// What a run that reaches place `off` of a unit of n tiles, at place f of the line, holds of it:
// tiles [k0, k1) (none where only places before the first tile are its own) in `take` places.
struct Piece {
  int k0, k1;
  int64_t take;
};
template <int kCost>
__device__ __forceinline__ Piece unit_piece(const Run& r, int64_t f, int off, int n) {
  const int64_t take = min((int64_t)(n + kCost - off), r.f1 - f);
  return {max(off - kCost, 0), max((int)(off + take) - kCost, 0), take};
}
// The record of a unit of n tiles whose place `off` is place f of the line (written by the CTA that
// holds its first tile).
template <int kCost>
__device__ __forceinline__ UnitInfo unit_record(const Run& r, int cta, int row, int nrows, int64_t f, int off, int n) {
  const int64_t last = f - off + kCost + n - 1, cut = r.more * (r.base + 1);  // its last tile's CTA
  const int64_t c1 = last < cut ? udiv_pos(last, r.base + 1) : r.more + udiv_pos(last - cut, r.base);
  return {row, nrows, cta, (int32_t)c1};
}

// ---------------------------------------------------------------- join
// Adds, in the runs' order, the partial results of the units that several CTAs worked on,
// and writes the rows that see no token.  A block takes 16 rows of a unit; with fewer rows
// each has 2 .. 16 warps, which share its parts (one long sequence is cut into many) and
// add their sums in a fixed order.  Latency-bound: two dependent loads.
constexpr int kJoinWarps = 16;

template <int D, int RT, bool kBf16>
__global__ void __launch_bounds__(kJoinWarps * 32) kv_attn_join_kernel(const CacheAttnArgs a, const WsPtrs ws) {
  constexpr int EPL = D / 32, kAhead = 8;  // elements a lane; parts in flight
  __shared__ float acc_sm[kJoinWarps][D];
  __shared__ float2 ml_sm[kJoinWarps];
  grid_dependency_wait();
  grid_launch_dependents();
  const int hk = blockIdx.x % a.Hkv;
  const UnitInfo u = ws.info[blockIdx.x];
  const int rows = min(kJoinWarps, u.nrows - (int)blockIdx.y * kJoinWarps);
  if (rows <= 0 || (u.c0 == u.c1 && u.c0 >= 0)) return;  // nothing, or written by the unit's only CTA
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int wpr = rows > 8 ? 1 : (rows > 4 ? 2 : (rows > 2 ? 4 : (rows > 1 ? 8 : 16)));  // warps a row
  const int r_in = warp / wpr, sub = warp % wpr;
  const bool mine = r_in < rows;
  const int r = (int)blockIdx.y * kJoinWarps + r_in;
  float acc[EPL], sum = 0.f, mx = -INFINITY;  // of this warp's parts, relative to its mx
#pragma unroll
  for (int e = 0; e < EPL; ++e) acc[e] = 0.f;
  if (mine && u.c0 >= 0) {
    for (int c = u.c0 + sub; c <= u.c1; c += wpr * kAhead) {
      float2 ml[kAhead];
      float o[kAhead][EPL];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int ci = c + i * wpr;
        ml[i] = make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int e = 0; e < EPL; ++e) o[i][e] = 0.f;
        if (ci <= u.c1) {
          const int64_t p = (int64_t)(ci == u.c0 ? 2 * ci + 1 : 2 * ci) * RT + r;
          ml[i] = ws.ml[p];
          const float* src = ws.o + p * D + lane * EPL;
          if constexpr (EPL == 4) *reinterpret_cast<float4*>(o[i]) = *reinterpret_cast<const float4*>(src);
          else *reinterpret_cast<float2*>(o[i]) = *reinterpret_cast<const float2*>(src);
        }
      }
      float mn = mx;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) mn = fmaxf(mn, ml[i].x);
      const float base = mn == -INFINITY ? 0.f : mn, f0 = ptx::ex2_approx(mx - base);
      sum *= f0;
#pragma unroll
      for (int e = 0; e < EPL; ++e) acc[e] *= f0;
      mx = mn;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const float f = ptx::ex2_approx(ml[i].x - base);
        sum += f * ml[i].y;
#pragma unroll
        for (int e = 0; e < EPL; ++e) acc[e] += f * o[i][e];
      }
    }
  }
  if (wpr > 1) {
#pragma unroll
    for (int e = 0; e < EPL; ++e) acc_sm[warp][lane * EPL + e] = acc[e];
    if (lane == 0) ml_sm[warp] = make_float2(mx, sum);
    __syncthreads();
    if (mine && sub == 0) {
      float mn = mx;
      for (int i = 1; i < wpr; ++i) mn = fmaxf(mn, ml_sm[warp + i].x);
      const float base = mn == -INFINITY ? 0.f : mn, f0 = ptx::ex2_approx(mx - base);
      sum *= f0;
#pragma unroll
      for (int e = 0; e < EPL; ++e) acc[e] *= f0;
      mx = mn;
      for (int i = 1; i < wpr; ++i) {
        const float f = ptx::ex2_approx(ml_sm[warp + i].x - base);
        sum += f * ml_sm[warp + i].y;
#pragma unroll
        for (int e = 0; e < EPL; ++e) acc[e] += f * acc_sm[warp + i][lane * EPL + e];
      }
    }
  }
  if (!mine || sub != 0) return;
  const int row = (u.row + r) / a.G, h = hk * a.G + (u.row + r) % a.G;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int64_t at = ((int64_t)row * a.Hq + h) * D + lane * EPL;
  if constexpr (kBf16) {
    __nv_bfloat162 y[EPL / 2];
#pragma unroll
    for (int e = 0; e < EPL / 2; ++e) y[e] = __floats2bfloat162_rn(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    __nv_bfloat162* dst = reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(a.out) + at);
#pragma unroll
    for (int e = 0; e < EPL / 2; ++e) dst[e] = y[e];
  } else {
#pragma unroll
    for (int e = 0; e < EPL; ++e) static_cast<float*>(a.out)[at + e] = acc[e] * inv;
  }
  if (lane == 0) a.lse[(int64_t)h * a.rows + row] = lse_of(mx, sum);
}

template <int D, int RT, bool kBf16>
cp_status launch_join(const CacheAttnArgs& a, const WsPtrs& ws, int64_t slots, cudaStream_t st) {
  return launch_chained(kv_attn_join_kernel<D, RT, kBf16>, dim3((unsigned)(slots * a.Hkv), (RT + kJoinWarps - 1) / kJoinWarps),
                        kJoinWarps * 32, 0, st, "kv_attn_join_kernel launch", a, ws);
}

inline size_t al256(size_t x) { return (x + 255) / 256 * 256; }
inline int64_t slot_count(int64_t rows, int64_t G, int64_t n_seqs, int RT) { return rows * G / RT + n_seqs; }
// Bytes and pointers of a workspace for `slots` row tiles of RT rows and `ctas` CTAs.
inline size_t ws_layout(void* base, int64_t slots, int Hkv, int RT, int ctas, int D, WsPtrs* ws) {
  char* p = static_cast<char*>(base);
  size_t off = 0;
  if (ws) ws->info = reinterpret_cast<UnitInfo*>(p);
  off += al256((size_t)slots * Hkv * sizeof(UnitInfo));
  if (ws) ws->ml = reinterpret_cast<float2*>(p + off);
  off += al256((size_t)2 * ctas * RT * sizeof(float2));
  if (ws) ws->o = reinterpret_cast<float*>(p + off);
  return off + al256((size_t)2 * ctas * RT * D * 4);
}

}  // namespace
}  // namespace cpa
