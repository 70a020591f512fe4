// Attention over the quantised key/value cache for many query rows a key (a prompt's
// chunk), bf16 queries, sm_103a.
//
// Mathematics as in kv_attn.cu; here the products bound, 4*D flops a (row, key) pair and
// query head, so the queries are the M side and the products run in kind::f16: an e4m3
// code times a power of two down to 2^-15 is exact in fp16, so a page's scale relative to the
// unit's largest goes into its converted codes; q is scaled to [128, 256) a row (its 8 bits are
// exact down to 2^-24 of the row's largest), and the weights keep 11 bits (2^-12 of each, an eighth of
// half a step of a bf16 result; their sum is kept whole).  Codes are converted
// once per key tile and used by 256 rows.
// A unit whose seen pages differ by more than kKeySpan or kValueSpan (`wide`) is rare and
// would lose its small pages so: there the codes are converted as they are and the softmax
// applies the scales in fp32 (wide_tile), which no row's accuracy depends on another's for.
//
// Two CTAs on neighbouring SMs work as a pair (cta_group::2): a product has 256 rows, 128 in
// each CTA, and each CTA holds half of its B operand (64 of the tile's keys for S, half of the
// head's columns for O).  So a code is converted once for 512 query rows, and an SM reads and
// converts half a tile.  A chunk of 2048 rows over 32768 tokens, 32 heads: 0.828 ms, 1286 TFLOP/s
// (one CTA a tile, with twice the conversion on each SM: 1.16 ms).
//
// One CTA an SM, 16 warps:
//   warps 0..3, 4..7  softmax of this CTA's query tile 0 / 1 (128 packed rows (query row, head
//             of the group) each): thread = row = TMEM lane.  Loads and scales its q row, keeps
//             the running maximum (renewed when it grows by 2^8), writes the weights over
//             S as the next product's A operand.
//   warp 8    producer: decodes the pair's units, finds a unit's largest scales, brings this
//             CTA's halves of the 8-bit K and V tiles by TMA, and their pages' factors.
//   warp 9    MMA issuer (first CTA of the pair), order S0_j | O1 += P1 V_{j-1} | S1_j |
//             O0 += P0 V_j, so each softmax overlaps the other tile's two products; one wait
//             between two products.
// A unit of at most 256 rows has one query tile in each CTA; then the two warpgroups take its even
// and its odd key tiles (order O_w += P_w V_t | S_w = Q K_{t+2}, w = t mod 2), each with sums and an
// O of its own, and the second's go to the first through shared memory at the end: 96 rows over
// 16 sequences of 8192 tokens, 8 heads, in 166 us (221 when one warpgroup worked alone).
//   warps 10, 11 and 12, 15  converters of K and of V: 8-bit half tile -> fp16 (codes times
//             factor) in the layout the products read; tokens past the end become zeros.
// The line of tiles is divided over the pairs as kv_plan.cuh says; a run crosses units.
#include <algorithm>

#define KV_PLAN_INLINE __forceinline__
#include "kv_plan.cuh"

namespace cpa {
namespace {

constexpr int kThreads = 512;
// Converters: K warps 10, 11, V warps 12, 15.  (Warp w issues from scheduler w % 4: the MMA
// thread's is spared, and warps 13, 14 only help to plan.)
constexpr int kProducerWarp = 8, kMmaWarp = 9, kConvHalf = 64;  // threads for K, and for V
constexpr int BM = 128, RT = 4 * BM;  // rows of a query tile; of a unit (two tiles in each CTA)
constexpr int kCost = 2;  // the work around a unit's tiles, in tiles
constexpr int kStages = 3, kIn = 2;   // fp16 half tiles; 8-bit half tiles
// Register split: 256 threads at 112 and 256 at 144 are the launch's 512 x 128.
constexpr int kRegsLow = 112, kRegsHigh = 144;
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr uint64_t kDrainNs = 200000000ull;
// The reference of a row's weights 2^(x - m) is its largest score less kLog2Unit, renewed when
// a score passes m + kLog2Range: weights stay under 2^15, and fp16's smallest step is 2^-31 of
// the largest.
constexpr float kLog2Unit = 7.0f, kLog2Range = 15.0f;
// Least ratio of a unit's scales that goes into its codes: keys stay exact; values leave a row that
// sees small ones beside large ones its weights to 2^-22 of its largest product.
constexpr float kKeySpan = 0x1p-15f, kValueSpan = 0x1p-10f;
// In a wide unit a row's reference goes down to this under its largest score, so that the weights of
// values 2^-100 as large as the unit's largest still fill fp16's range (the sums stay under 2^127).
constexpr int kWideLog2 = 100;

template <int D>
struct Layout {
  static constexpr int kQTile = BM * D * 2;
  static constexpr int kHalf16 = BK * D, kHalf8 = BK * D / 2;  // bytes of half a tile of K or V
  static constexpr int kVRow = D;                               // bytes of a row of the V half (D/2 halves): its swizzle
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + 2 * kQTile;
  static constexpr int kV = kK + kStages * kHalf16;
  static constexpr int kK8 = kV + kStages * kHalf16;
  static constexpr int kV8 = kK8 + kIn * kHalf8;
  static constexpr int kMl = kV8 + kIn * kHalf8;  // (m, l) of the second warpgroup's rows
  static constexpr int kCtl = kMl + 1024;
  static constexpr int kBytes = kCtl + 1024 + 1024;
  static constexpr int kSmemRequest = kBytes > 120 * 1024 ? kBytes : 120 * 1024;  // one CTA an SM
};

constexpr int kBad = 1, kWide = 2;  // kWide: the codes are converted without their scales (k_ref is 1)
struct Unit {
  int32_t b, hk, tile0, ntiles, len, n, nrows, c0, r0, part;
  int32_t special;      // kBad: some page of the unit does not exist (its tokens are hidden); kWide
  float k_ref, v_ref;   // largest key / value scale of the unit's pages
};

struct Ctl {
  // arrived on by both CTAs, waited for by the first one's MMA thread
  uint64_t q_full[2], p_full[2], k_full[kStages], v_full[kStages];
  // arrived on in both CTAs as products complete
  uint64_t s_full[2], k_empty[kStages], v_empty[kStages], o_done;
  // this CTA's own
  uint64_t k8_full[kIn], k8_empty[kIn], v8_full[kIn], v8_empty[kIn], u_full[2], u_empty[2], drained;
  uint64_t half_full, half_free;  // the second warpgroup's sums and O in shared memory
  Unit unit[2];
  uint32_t kf[kIn][8], vf[kIn][8];  // factor of a tile's pages as a pair of halves
  PlanSmem<kThreads / 32> plan;
  uint32_t tmem;
  int abort_flag;
};
static_assert(sizeof(Ctl) <= 1024, "control block");

__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int b_mn) {
  return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// The issuing thread adds one constant to the low word of each descriptor (address >> 4) and
// nothing else between two products: what it computes there the tensor cores wait for.
constexpr uint32_t desc_hi(int row_bytes) {  // rows of 8 apart, version 1, swizzle as wide as a row
  return (uint32_t)(8 * row_bytes >> 4) | (1u << 14) | ((row_bytes == 128 ? 2u : 4u) << 29);
}
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) { return ((saddr >> 4) & 0x3FFFu) | (1u << 16); }
// Step of K slice kk (16 halves) of a K-major operand in blocks of 64 columns [rows][128 bytes].
__host__ __device__ constexpr uint32_t kmajor_step(int rows, int kk) { return ((kk >> 2) * (rows * 128) + (kk & 3) * 32) >> 4; }

// ---- pair forms of the tensor-core instructions, and barriers across the pair
__device__ __forceinline__ void tmem_alloc2(uint32_t* result, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(ptx::smem_u32(result)), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc2(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
template <uint32_t kHiA, uint32_t kHiB, uint32_t kIdesc>
__device__ __forceinline__ void mma2_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tmov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %4};\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %5, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "n"(kHiA), "n"(kHiB), "r"(kIdesc), "r"((uint32_t)acc)
      : "memory");
}
template <uint32_t kHiB, uint32_t kIdesc>
__device__ __forceinline__ void mma2_ts(uint32_t d, uint32_t a, uint32_t b_lo, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tmov.b64 db, {%2, %3};\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b_lo), "n"(kHiB), "r"(kIdesc), "r"((uint32_t)acc)
      : "memory");
}
// One arrival on `bar` in both CTAs once every product issued so far has completed.
__device__ __forceinline__ void commit2(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          ptx::smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
// One arrival of the warp on the first CTA's `bar`.  (The default forms here and in the waits: spelled
// out as .release.cluster and .acquire.cluster they took the chunk above from 1.34 to 1.40 ms.)
__device__ __forceinline__ void arrive_first(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane != 0) return;
  asm volatile(
      "{\n\t.reg .b32 ra;\n\tmapa.shared::cluster.u32 ra, %0, 0;\n\t"
      "mbarrier.arrive.shared::cluster.b64 _, [ra];\n\t}" ::"r"(ptx::smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ bool try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(ptx::smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// ptx::mbar_wait_bounded for a barrier that the other CTA arrives on too.
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort, int32_t* err) {
  if (ptx::mbar_test_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (true) {
    if (try_wait_cluster(bar, parity)) return true;
    if (*abort) return false;
    if (global_timer_ns() - t0 > kWaitNs) {
      *abort = 1;
      record_device_error(err, kDevTimeout);
      return false;
    }
  }
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A ring of kStages buffers: the next one and the parity of its use.
struct Ring {
  int st = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next() {
    if (++st == kStages) {
      st = 0;
      ph ^= 1u;
    }
  }
};
__device__ __forceinline__ int cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return (int)r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The converters' view of a half tile: codes [rows][cols] to fp16 blocks of up to 64 columns, each
// row swizzled as wide as it is (sw bytes).  Item = 16 codes, two 16-byte chunks; of the 8 items of
// a row of 128 those of the second block write their chunks in the other order, so that a quarter
// warp's stores fall on distinct banks.  The 64 threads of a step cover whole groups of 8 rows, so
// a thread's swizzle is the same in every step.
//
// One rolled loop serves K and V, whole and last tiles: the SM's warps run three programs at once,
// and their instructions have to stay cached (unrolled and specialised, the conversion slowed the
// softmax and the products of its SM by a fifth, whatever it computed).
struct ConvMap {
  uint32_t src, dst0, dst1;  // offsets of the thread's first item
  int row0, row_step, steps; // its first row; rows a step; steps of a tile
  uint32_t dst_step;
  bool flip;
};
template <int kRows, int kCols>
__device__ __forceinline__ ConvMap conv_map(int t) {
  constexpr int kPerRow = kCols / 16, kStepRows = kConvHalf / kPerRow;
  constexpr int kSw = kCols >= 64 ? 128 : kCols * 2, kChunks = kSw / 16;
  static_assert(kStepRows % 8 == 0 && kRows % kStepRows == 0, "conversion steps");
  const int r0 = t / kPerRow, c = t % kPerRow;
  const bool flip = kPerRow == 8 && (c & 4) != 0;
  auto at = [&](int chunk) {
    const uint32_t o = (uint32_t)r0 * kSw + (chunk % kChunks) * 16;
    return (uint32_t)(chunk / kChunks) * (kRows * kSw) + (o ^ (((o >> 7) & (kChunks - 1)) << 4));
  };
  return {(uint32_t)t * 16, at(2 * c + (flip ? 1 : 0)), at(2 * c + (flip ? 0 : 1)), r0, kStepRows, kRows / kStepRows,
          (uint32_t)kStepRows * kSw, flip};
}
// Addresses are 32-bit shared ones.
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 r;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(addr));
  return r;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t r;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(addr));
  return r;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// `t0`: first token of the half; tokens from `rows` on become zeros, and those of a page that was
// not loaded (factor 0).
__device__ __forceinline__ void convert_half(const ConvMap& m, uint32_t src, uint32_t dst, uint32_t factor, int page_log2,
                                             int t0, int rows) {
  int r = t0 + m.row0;
  uint32_t s = src + m.src, d0 = dst + m.dst0, d1 = dst + m.dst1;
#pragma unroll 1
  for (int i = 0; i < m.steps; ++i) {
    const uint4 w = lds128(s);
    uint32_t f = lds32(factor + ((r >> page_log2) << 2));
    if (r >= rows) f = 0u;
    uint32_t u[4] = {m.flip ? w.z : w.x, m.flip ? w.w : w.y, m.flip ? w.x : w.z, m.flip ? w.y : w.w};
    if (f == 0u) u[0] = u[1] = u[2] = u[3] = 0u;  // its bytes may be anything
    sts128(d0, hmul2(e4m3x2_to_f16x2(u[0] & 0xffffu), f), hmul2(e4m3x2_to_f16x2(u[0] >> 16), f),
           hmul2(e4m3x2_to_f16x2(u[1] & 0xffffu), f), hmul2(e4m3x2_to_f16x2(u[1] >> 16), f));
    sts128(d1, hmul2(e4m3x2_to_f16x2(u[2] & 0xffffu), f), hmul2(e4m3x2_to_f16x2(u[2] >> 16), f),
           hmul2(e4m3x2_to_f16x2(u[3] & 0xffffu), f), hmul2(e4m3x2_to_f16x2(u[3] >> 16), f));
    s += kConvHalf * 16;
    r += m.row_step;
    d0 += m.dst_step;
    d1 += m.dst_step;
  }
}

// Scores of columns ch*32 .. ch*32 + 31 that the row does not see ([ilo, ihi) of the tile) or whose
// page does not exist become -inf.
__device__ __forceinline__ void hide(uint32_t (&s)[32], int ch, int ilo, int ihi, int key0, const Unit& un,
                                     const CacheAttnArgs& a) {
  const uint32_t kInf = 0xff800000u;
#pragma unroll
  for (int i = 0; i < 32; ++i) s[i] = (ch * 32 + i >= ilo && ch * 32 + i < ihi) ? s[i] : kInf;
  if (!(un.special & kBad)) return;
#pragma unroll
  for (int i = 0; i < 32; i += 16) {  // pages are multiples of 16 tokens
    const int key = key0 + ch * 32 + i;
    if (key >= un.len) break;
    const int id = ld(a.page_table + (int64_t)un.b * a.max_pages + key / a.page);
    if (id >= 0 && id < a.n_pages) continue;
#pragma unroll
    for (int k = 0; k < 16; ++k) s[i + k] = kInf;
  }
}

// One key tile of a wide unit, its scores in the warp's lanes of TMEM from `s_addr` on; the weights
// are left there as the product wants them.  qs: factor of the row's scores without the keys' scales;
// [ilo, ihi): the tile's tokens that the row sees; o_addr: the row's O, rescaled where `rescale`.
// The reference m is chosen by the weights times their value scales (v_ref is the unit's largest), and
// renewed in every tile.  Speed does not matter here; rolled loops keep the usual path's registers and
// instruction cache.
template <int D>
__device__ __forceinline__ float2 wide_tile(const Unit& un, const CacheAttnArgs& a, uint32_t s_addr, uint32_t o_addr, float qs,
                                         int ilo, int ihi, int key0, float m, float l, bool rescale) {
  const float v_inv = 1.f / un.v_ref;
  // key and value scale of the 16 tokens from column col on (pages are multiples of 16 tokens), the
  // latter relative to v_ref; a token that some row sees has at most v_ref
  auto scales = [&](int col) {
    const int key = key0 + col;
    if (key >= un.len) return make_float2(0.f, 0.f);
    const int id = ld(a.page_table + (int64_t)un.b * a.max_pages + key / a.page);
    if (id < 0 || id >= a.n_pages) return make_float2(0.f, 0.f);
    const int64_t at = (int64_t)id * a.Hkv + un.hk;
    const float f = ld(a.k_scale + at) * qs, v = ld(a.v_scale + at);
    // (a score of 0 stays 0 where the factor alone passes fp32)
    return make_float2(f > 3e38f ? 3e38f : f, v > 0.f ? fminf(v * v_inv, 1.f) : 0.f);
  };
  float top = -INFINITY;
#pragma unroll 1
  for (int ch = 0; ch < BK / 32; ++ch) {
    uint32_t s[32];
    ptx::tmem_ld32(s_addr + ch * 32, s);
    ptx::tmem_wait_ld_regs(s);
#pragma unroll
    for (int g = 0; g < 32; g += 16) {
      const float2 f = scales(ch * 32 + g);
#pragma unroll
      for (int i = 0; i < 16; ++i) s[g + i] = __float_as_uint(__uint_as_float(s[g + i]) * f.x);
    }
    hide(s, ch, ilo, ihi, key0, un, a);
#pragma unroll
    for (int g = 0; g < 32; g += 16) {
      const int e = (int)(__float_as_uint(scales(ch * 32 + g).y) >> 23) - 127;
      float mt = -INFINITY;
#pragma unroll
      for (int i = 0; i < 16; ++i) mt = fmaxf(mt, __uint_as_float(s[g + i]));
      top = fmaxf(top, mt + (float)max(e, -kWideLog2));
    }
    ptx::tmem_st32(s_addr + ch * 32, s);
  }
  const float m_new = fmaxf(m, top - kLog2Unit), alpha = m == -INFINITY ? 0.f : ptx::ex2_approx(m - m_new);
  l *= alpha;
  if (rescale) {
#pragma unroll 1
    for (int ch = 0; ch < D / 32; ++ch) {
      uint32_t o[32];
      ptx::tmem_ld32(o_addr + ch * 32, o);
      ptx::tmem_wait_ld_regs(o);
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
      ptx::tmem_st32(o_addr + ch * 32, o);
    }
  }
  ptx::tmem_wait_st();
  const float ref = m_new == -INFINITY ? 0.f : m_new;
#pragma unroll 1
  for (int ch = 0; ch < BK / 32; ++ch) {  // the weights of 32 tokens take 16 columns, behind the scores read so far
    uint32_t s[32], p[16];
    ptx::tmem_ld32(s_addr + ch * 32, s);
    ptx::tmem_wait_ld_regs(s);
#pragma unroll
    for (int g = 0; g < 32; g += 16) {
      const float f = scales(ch * 32 + g).y;
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const float p0 = ptx::ex2_approx(__uint_as_float(s[g + i]) - ref), p1 = ptx::ex2_approx(__uint_as_float(s[g + i + 1]) - ref);
        l += p0 + p1;
        p[(g + i) / 2] = pack_f16x2(p0 * f, p1 * f);
      }
    }
    ptx::tmem_st16(s_addr + ch * 16, p);
  }
  ptx::tmem_wait_st();
  return make_float2(m_new, l);
}

template <int D>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
kv_attn_rows_kernel(const __grid_constant__ CacheAttnArgs a, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const WsPtrs ws, const int slots) {
  using L = Layout<D>;
  extern __shared__ uint8_t smem_raw[];
  // (the dynamic shared memory starts at one address in both CTAs, so the offsets agree)
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Ctl& ctl = *reinterpret_cast<Ctl*>(smem + L::kCtl);
  const uint32_t sbase = ptx::smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = cluster_rank(), pair = blockIdx.x >> 1;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&ctl.q_full[i], 2 * 4);
      ptx::mbar_init(&ctl.p_full[i], 2 * 4);
      ptx::mbar_init(&ctl.s_full[i], 1);
      ptx::mbar_init(&ctl.u_full[i], 1);
      ptx::mbar_init(&ctl.u_empty[i], 256 + 2 * kConvHalf + (rank == 0 ? 1 : 0));
    }
    for (int i = 0; i < kStages; ++i) {
      ptx::mbar_init(&ctl.k_full[i], 2 * kConvHalf / 32);
      ptx::mbar_init(&ctl.v_full[i], 2 * kConvHalf / 32);
      ptx::mbar_init(&ctl.k_empty[i], 1);
      ptx::mbar_init(&ctl.v_empty[i], 1);
    }
    for (int i = 0; i < kIn; ++i) {
      ptx::mbar_init(&ctl.k8_full[i], 1);
      ptx::mbar_init(&ctl.v8_full[i], 1);
      ptx::mbar_init(&ctl.k8_empty[i], kConvHalf);
      ptx::mbar_init(&ctl.v8_empty[i], kConvHalf);
    }
    ptx::mbar_init(&ctl.o_done, 1);
    ptx::mbar_init(&ctl.drained, 1);
    ptx::mbar_init(&ctl.half_full, 128);
    ptx::mbar_init(&ctl.half_free, 128);
    ctl.abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == kProducerWarp && lane == 0) {
    ptx::prefetch_tensormap(&tm_k);
    ptx::prefetch_tensormap(&tm_v);
  }
  if (warp == kMmaWarp) tmem_alloc2(&ctl.tmem, kTmemCols);
  grid_dependency_wait();
  // both CTAs of a pair come to the same run
  const Run run = plan_run<RT, kCost, kThreads / 32>(a, ws, slots, pair, gridDim.x >> 1,
                                              reinterpret_cast<int32_t*>(smem + L::kQ), L::kQTile / 4 - 1, ctl.plan);
  ptx::fence_proxy_async_smem();  // the staged lengths lie where the products will read
  ptx::tc_fence_before();
  __syncthreads();
  cluster_sync();  // the other CTA's barriers are there
  ptx::tc_fence_after();
  const uint32_t tmem = ctl.tmem;
  volatile int* abort_flag = &ctl.abort_flag;
  auto wait = [&](uint64_t* bar, uint32_t par) {
    return ptx::mbar_wait_bounded(bar, par & 1u, abort_flag, a.err, kWaitNs);
  };

  if (warp >= 8) {
    ptx::setmaxnreg_dec<kRegsLow>();
    if (run.slot < 0) {
      if (warp == kMmaWarp && lane == 0 && rank == 0) commit2(&ctl.drained);
    } else if (warp == kProducerWarp) {
      // ------------------------------------------------------------ units, TMA
      const int ppt = BK / a.page;
      // this CTA's keys of a tile: 64, i.e. k_pages pages from k_first on, or half of a page of 128
      const int k_rows = min(a.page, BK / 2), k_pages = a.page < BK ? BK / 2 / a.page : 1;
      const int k_first = a.page < BK ? rank * k_pages : 0, k_skip = a.page < BK ? 0 : rank * (BK / 2);
      const uint32_t k_bytes = (uint32_t)(k_rows * D), v_bytes = (uint32_t)(a.page * D / 2);
      int64_t f = run.f0;
      int slot = run.slot, head = run.head, off = run.off, u = 0, j = 0;
      bool ok = true;
      SlotRows sr = ctl.plan.rows;
      while (f < run.f1) {
        const SlotSeq& q = sr.q;
        const int b = q.b, t0 = sr.t0(), t1 = sr.t1();
        const Piece pc = unit_piece<kCost>(run, f, off, t1 - t0);
        const int n = pc.k1 - pc.k0, tile0 = t0 + pc.k0;
        // The join goes by the records, so each of the run's is written, after a wait that gave up too.
        if (n > 0 && pc.k0 == 0 && rank == 0 && lane == 0)
          ws.info[(int64_t)slot * a.Hkv + head] =
              unit_record<kCost>(run, pair, q.c0 * a.G + sr.r0, sr.nrows, f, off, t1 - t0);
        if (n > 0 && ok && u >= 2) ok = __all_sync(0xffffffffu, wait(&ctl.u_empty[u & 1], (u >> 1) - 1));
        if (n > 0 && ok) {
          const int32_t* table = a.page_table + (int64_t)b * a.max_pages;
          // pages [p_first, p_end) of its tiles hold tokens that some row sees; the others' tokens count as
          // zeros and need not exist (those before a window may have been given back)
          const int p0 = tile0 * ppt, p_first = max(p0, sr.lo / a.page);
          const int p_end = min((tile0 + n) * ppt, (sr.hi + a.page - 1) / a.page);
          float kr = 0.f, vr = 0.f, k_min = INFINITY, v_min = INFINITY;
          bool bad = false;
#pragma unroll 4
          for (int p = p_first + lane; p < p_end; p += 32) {
            const int id = ld(table + p);
            if (id < 0 || id >= a.n_pages) {
              record_device_error(a.err, kDevIndex);
              bad = true;
            } else {
              const float k = ld(a.k_scale + (int64_t)id * a.Hkv + head), v = ld(a.v_scale + (int64_t)id * a.Hkv + head);
              kr = fmaxf(kr, k);  // (NaN is none of these)
              vr = fmaxf(vr, v);
              k_min = fminf(k_min, k);
              v_min = fminf(v_min, v);
            }
          }
          kr = fmaxf(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(kr))), 1.17549435e-38f);
          vr = fmaxf(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(vr))), 1.17549435e-38f);
          bad = __any_sync(0xffffffffu, bad);
          const bool wide = __any_sync(0xffffffffu, k_min < kr * kKeySpan || v_min < vr * kValueSpan);
          if (lane == 0) {
            Unit& un = ctl.unit[u & 1];
            un.b = b;
            un.hk = head;
            un.tile0 = tile0;
            un.ntiles = n;
            un.len = q.len;
            un.n = q.n;
            un.nrows = sr.nrows;
            un.c0 = q.c0;
            un.r0 = sr.r0;
            un.part = n == t1 - t0 ? -1 : 2 * pair + (pc.k0 > 0 ? 0 : 1);
            un.special = (bad ? kBad : 0) | (wide ? kWide : 0);
            un.k_ref = wide ? 1.f : kr;
            un.v_ref = vr;
            ptx::mbar_arrive(&ctl.u_full[u & 1]);
          }
          __syncwarp();
          // tiles: 32 pages at a time, their ids and factors one batch ahead
          const float k_inv = wide ? 0.f : 1.f / kr, v_inv = wide ? 0.f : 1.f / vr, one = wide ? 1.f : 0.f;
          int id, id_n;
          uint32_t kf, vf, kf_n, vf_n;
          auto fetch = [&](int p, int& i, uint32_t& k2, uint32_t& v2) {
            i = -1;
            k2 = v2 = 0u;
            if (p + lane >= p_first && p + lane < p_end) {
              i = ld(table + p + lane);
              if (i < 0 || i >= a.n_pages) {
                i = -1;
              } else {
                const float k = ld(a.k_scale + (int64_t)i * a.Hkv + head), v = ld(a.v_scale + (int64_t)i * a.Hkv + head);
                const float kf = fmaf(k, k_inv, one), vf = fmaf(v, v_inv, one);
                k2 = v != v ? 0x7e007e00u : pack_f16x2(kf, kf);  // a NaN scale reaches the scores
                v2 = v != v ? 0u : pack_f16x2(vf, vf);
              }
            }
          };
          fetch(p0, id, kf, vf);
          fetch(p0 + 32, id_n, kf_n, vf_n);
          for (int t = 0; t < n; ++t, ++j) {
            const int at = (t * ppt) & 31;
            if (at == 0 && t > 0) {
              id = id_n;
              kf = kf_n;
              vf = vf_n;
              fetch(p0 + t * ppt + 32, id_n, kf_n, vf_n);
            }
            const int pg = lane - at, st = j % kIn;  // this lane's page of the tile
            const bool in = pg >= 0 && pg < ppt, in_k = in && pg >= k_first && pg < k_first + k_pages;
            const uint32_t have = __ballot_sync(0xffffffffu, in && id >= 0);
            const uint32_t have_k = __ballot_sync(0xffffffffu, in_k && id >= 0);
            const int row = in && id >= 0 ? (id * a.Hkv + head) * a.page : 0;
            if (j >= kIn) ok = wait(&ctl.k8_empty[st], j / kIn - 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (in_k && id >= 0)
              ptx::tma_load_2d(smem + L::kK8 + st * L::kHalf8 + (uint32_t)(pg - k_first) * k_bytes, &tm_k, &ctl.k8_full[st], 0,
                               row + k_skip);
            if (in) ctl.kf[st][pg] = kf;
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive_expect_tx(&ctl.k8_full[st], k_bytes * __popc(have_k));
            if (j >= kIn) ok = wait(&ctl.v8_empty[st], j / kIn - 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (in && id >= 0)
              ptx::tma_load_2d(smem + L::kV8 + st * L::kHalf8 + (uint32_t)pg * v_bytes, &tm_v, &ctl.v8_full[st], rank * (D / 2), row);
            if (in) ctl.vf[st][pg] = vf;
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive_expect_tx(&ctl.v8_full[st], v_bytes * __popc(have));
            __syncwarp();
          }
          if (ok) ++u;
        }
        f += pc.take;
        off = 0;
        if (++head == a.Hkv) {
          head = 0;
          if (f < run.f1 && !next_rows<RT>(a, slots, slot, sr)) break;
        }
      }
      if (ok && u >= 2) ok = wait(&ctl.u_empty[u & 1], (u >> 1) - 1);  // the end of the run
      if (lane == 0) {
        if (ok) {
          ctl.unit[u & 1].ntiles = 0;
          ptx::mbar_arrive(&ctl.u_full[u & 1]);
        } else {  // bounded wait for this CTA's copies in flight
          for (int i = max(0, j - kIn); i <= j; ++i) {
            (void)ptx::mbar_wait_bounded(&ctl.k8_full[i % kIn], (i / kIn) & 1, nullptr, nullptr, kDrainNs);
            (void)ptx::mbar_wait_bounded(&ctl.v8_full[i % kIn], (i / kIn) & 1, nullptr, nullptr, kDrainNs);
          }
        }
      }
      __syncwarp();
    } else if (warp == kMmaWarp) {
      // ------------------------------------------------------------ MMA issuer
      if (lane == 0 && rank == 0) {
        constexpr uint32_t id_qk = idesc_f16(2 * BM, BK, 0), id_pv = idesc_f16(2 * BM, D, 1);
        auto wait2 = [&](uint64_t* bar, uint32_t par) { return wait_cluster(bar, par & 1u, abort_flag, a.err); };
        const uint32_t q_lo = desc_lo(sbase + L::kQ), k_lo = desc_lo(sbase + L::kK), v_lo = desc_lo(sbase + L::kV);
        auto qk = [&](int w, int tile, int st) {
          const uint32_t qa = q_lo + tile * (L::kQTile >> 4), ka = k_lo + st * (L::kHalf16 >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma2_ss<desc_hi(128), desc_hi(128), id_qk>(tmem + w * 256, qa + kmajor_step(BM, kk), ka + kmajor_step(BK / 2, kk),
                                                       kk > 0);
          commit2(&ctl.s_full[w]);
        };
        auto pv = [&](int w, int st, bool acc, bool release) {
          const uint32_t va = v_lo + st * (L::kHalf16 >> 4);
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk)
            mma2_ts<desc_hi(L::kVRow), id_pv>(tmem + w * 256 + 128, tmem + w * 256 + kk * 8, va + kk * L::kVRow,
                                              acc || kk > 0);
          if (release) commit2(&ctl.v_empty[st]);
        };
        // next stage of the K and the V ring with its phase; S products so far by warpgroup; units
        // with a second query tile
        Ring kr, vr;
        int c[2] = {0, 0}, u1 = 0;
        bool ok = true;
        for (int u = 0; ok; ++u) {
          if (!(ok = wait(&ctl.u_full[u & 1], u >> 1))) break;
          const int n = ctl.unit[u & 1].ntiles;
          if (n == 0) break;
          const bool has1 = ctl.unit[u & 1].nrows > 2 * BM;
          ptx::mbar_arrive(&ctl.u_empty[u & 1]);
          if (!(ok = wait2(&ctl.q_full[0], u))) break;
          if (has1 && !(ok = wait2(&ctl.q_full[1], u1++))) break;
          // K and V tiles are waited for and released apart: a K tile is free after its last S,
          // three products before its V tile
          if (!(ok = wait2(&ctl.k_full[kr.st], kr.ph))) break;
          ptx::tc_fence_after();
          qk(0, 0, kr.st);
          ++c[0];
          if (has1) {
            int prev = 0;  // the V stage before
            for (int t = 0; t < n; ++t) {
              if (t >= 1) {  // O1 += P1 V_{t-1}
                if (!(ok = wait2(&ctl.p_full[1], c[1] - 1))) break;
                ptx::tc_fence_after();
                pv(1, prev, t - 1 > 0, true);
              }
              if (!(ok = wait2(&ctl.v_full[vr.st], vr.ph))) break;
              qk(1, 1, kr.st);
              commit2(&ctl.k_empty[kr.st]);
              kr.next();
              ++c[1];
              if (!(ok = wait2(&ctl.p_full[0], c[0] - 1))) break;
              ptx::tc_fence_after();
              prev = vr.st;
              vr.next();
              pv(0, prev, t > 0, false);
              if (t + 1 < n) {
                if (!(ok = wait2(&ctl.k_full[kr.st], kr.ph))) break;
                ptx::tc_fence_after();
                qk(0, 0, kr.st);
                ++c[0];
              }
            }
            if (!ok) break;
            if (!(ok = wait2(&ctl.p_full[1], c[1] - 1))) break;
            ptx::tc_fence_after();
            pv(1, prev, n > 1, true);
          } else {
            commit2(&ctl.k_empty[kr.st]);
            kr.next();
            if (n > 1) {
              if (!(ok = wait2(&ctl.k_full[kr.st], kr.ph))) break;
              ptx::tc_fence_after();
              qk(1, 0, kr.st);
              commit2(&ctl.k_empty[kr.st]);
              kr.next();
              ++c[1];
            }
            if (!(ok = wait2(&ctl.v_full[vr.st], vr.ph))) break;
            for (int t = 0; t < n; ++t) {
              const int w = t & 1;
              if (!(ok = wait2(&ctl.p_full[w], c[w] - 1))) break;
              ptx::tc_fence_after();
              pv(w, vr.st, t > 1, true);
              vr.next();
              if (t + 2 < n) {
                if (!(ok = wait2(&ctl.k_full[kr.st], kr.ph))) break;
                ptx::tc_fence_after();
                qk(w, 0, kr.st);
                commit2(&ctl.k_empty[kr.st]);
                kr.next();
                ++c[w];
              }
              if (t + 1 < n && !(ok = wait2(&ctl.v_full[vr.st], vr.ph))) break;
            }
            if (!ok) break;
          }
          commit2(&ctl.o_done);
        }
        // every product has completed before TMEM (either CTA's) is released
        commit2(&ctl.drained);
        (void)ptx::mbar_wait_bounded(&ctl.drained, 0, nullptr, a.err, kDrainNs);
      }
      __syncwarp();
    } else if (warp <= 12 || warp == 15) {
      // ------------------------------------------------------------ converters
      const bool is_v = warp >= 12;
      const int t = lane + (warp == 11 || warp == 15 ? 32 : 0);
      const int page_log2 = 31 - __clz(a.page), t0 = is_v ? 0 : rank * (BK / 2);
      const ConvMap map = is_v ? conv_map<BK, D / 2>(t) : conv_map<BK / 2, D>(t);
      const uint32_t in_base = sbase + (is_v ? L::kV8 : L::kK8), out_base = sbase + (is_v ? L::kV : L::kK);
      const uint32_t f_base = ptx::smem_u32(is_v ? ctl.vf : ctl.kf);
      uint64_t *in_full = is_v ? ctl.v8_full : ctl.k8_full, *in_empty = is_v ? ctl.v8_empty : ctl.k8_empty;
      uint64_t *out_full = is_v ? ctl.v_full : ctl.k_full, *out_empty = is_v ? ctl.v_empty : ctl.k_empty;
      int j = 0, st = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int u = 0; ok; ++u) {
        if (!(ok = wait(&ctl.u_full[u & 1], u >> 1))) break;
        const int n = ctl.unit[u & 1].ntiles, tile0 = ctl.unit[u & 1].tile0, len = ctl.unit[u & 1].len;
        if (n == 0) break;
        ptx::mbar_arrive(&ctl.u_empty[u & 1]);
        for (int i = 0; i < n; ++i, ++j) {
          const int rows = len - (tile0 + i) * BK, in = j % kIn;
          if (j >= kStages && !(ok = wait(&out_empty[st], ph ^ 1u))) break;
          if (!(ok = wait(&in_full[in], j / kIn))) break;
          convert_half(map, in_base + in * L::kHalf8, out_base + st * L::kHalf16, f_base + in * 32, page_log2, t0, rows);
          ptx::fence_proxy_async_smem();
          ptx::mbar_arrive(&in_empty[in]);
          arrive_first(&out_full[st], lane);
          if (++st == kStages) {
            st = 0;
            ph ^= 1u;
          }
        }
      }
      __syncwarp();
    }
  } else {
    ptx::setmaxnreg_inc<kRegsHigh>();
    // ------------------------------------------------------------ softmax warpgroups
    const int w = warp >> 2, quad = warp & 3, r = quad * 32 + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)(quad * 32) << 16) + w * 256;
    int c = 0, n_half = 0;  // tiles of this warpgroup and units in halves so far
    bool ok = run.slot >= 0;
    for (int u = 0; ok; ++u) {
      ok = __all_sync(0xffffffffu, wait(&ctl.u_full[u & 1], u >> 1));
      if (!ok) break;
      const Unit un = ctl.unit[u & 1];
      if (un.ntiles == 0) break;
      ptx::mbar_arrive(&ctl.u_empty[u & 1]);
      const bool halves = un.nrows <= 2 * BM;  // both warpgroups have this CTA's one query tile
      const int r_unit = ((halves ? 0 : 2 * w) + rank) * BM + r;  // the thread's row of the unit
      const bool valid = r_unit < un.nrows;
      const int rho = un.r0 + r_unit, tok = rho / a.G, h = un.hk * a.G + rho % a.G;
      float sl2 = 1.f;
      int lo = 0, hi = INT32_MAX;
      {
        // this thread's q row, scaled to [128, 256), as fp16
        uint8_t* qd = smem + L::kQ + w * L::kQTile;
        uint4 x[D / 8];
        uint32_t mx = 0;
        if (valid) {
          const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                            (int64_t)(un.c0 + tok) * a.q_ld + (int64_t)h * D);
#pragma unroll
          for (int i = 0; i < D / 8; ++i) x[i] = ld(src + i);
        } else {
#pragma unroll
          for (int i = 0; i < D / 8; ++i) x[i] = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          mx = __vmaxu2(mx, x[i].x & 0x7fff7fffu);
          mx = __vmaxu2(mx, x[i].y & 0x7fff7fffu);
          mx = __vmaxu2(mx, x[i].z & 0x7fff7fffu);
          mx = __vmaxu2(mx, x[i].w & 0x7fff7fffu);
        }
        mx = max(mx >> 16, mx & 0xffffu);  // bf16 bits of the largest magnitude
        const bool finite = mx < 0x7f80u;
        const int ex = max((int)(mx >> 7) - 127, -100);
        const float up = finite ? pow2i(7 - min(ex, 127)) : 0.f;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const uint32_t in[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
          uint32_t y[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            y[k] = finite ? pack_f16x2(__uint_as_float(in[k] << 16) * up, __uint_as_float(in[k] & 0xffff0000u) * up) : 0u;
          if (w == 0 || !halves)
            *reinterpret_cast<uint4*>(qd + (i >> 3) * 16384 + r * 128 + (((i & 7) ^ (r & 7)) << 4)) =
                make_uint4(y[0], y[1], y[2], y[3]);
        }
        ptx::fence_proxy_async_smem();
        if (valid) {
          SlotSeq sq;
          sq.b = un.b;
          sq.c0 = un.c0;
          sq.n = un.n;
          sq.len = un.len;
          row_bounds(a, sq, tok, lo, hi);
          // positive and finite, so that a hidden score stays -inf
          sl2 = fminf(fmaxf(pow2i(min(ex, 127) - 7) * un.k_ref * a.scale_log2, 1e-37f), 1e37f);
          if (!finite && hi > lo) sl2 = __int_as_float(0x7fc00000);
        }
      }
      if (w == 0 || !halves) arrive_first(&ctl.q_full[w], lane);
      const int lo_max = __reduce_max_sync(0xffffffffu, lo), hi_min = __reduce_min_sync(0xffffffffu, hi);
      const uint64_t sl2x2 = ptx::f2_pack(sl2, sl2);
      float m = -INFINITY, l = 0.f;
      const int t_first = halves ? w : 0, t_step = halves ? 2 : 1;
      for (int t = t_first; t < un.ntiles; t += t_step, ++c) {
        const int key0 = (un.tile0 + t) * BK;
        ok = __all_sync(0xffffffffu, wait(&ctl.s_full[w], c));
        if (!ok) break;
        ptx::tc_fence_after();
        if (un.special & kWide) {
          const float2 ml = wide_tile<D>(un, a, lane_addr, lane_addr + 128, sl2, lo - key0, hi - key0, key0, m, l, t > t_first);
          m = ml.x;
          l = ml.y;
          ptx::tc_fence_before();
          arrive_first(&ctl.p_full[w], lane);
          continue;
        }
        if (!(key0 >= lo_max && key0 + BK <= hi_min) || un.special) {  // hidden scores become -inf in place
#pragma unroll 1
          for (int ch = 0; ch < BK / 32; ++ch) {
            uint32_t rr[32];
            ptx::tmem_ld32(lane_addr + ch * 32, rr);
            ptx::tmem_wait_ld_regs(rr);
            hide(rr, ch, lo - key0, hi - key0, key0, un, a);
            ptx::tmem_st32(lane_addr + ch * 32, rr);
          }
          ptx::tmem_wait_st();
        }
        // One pass over the scores with the reference as it is: weights up to 2^15 fit fp16, so a
        // larger maximum is looked at after the exponentials, and only where one passes that (or
        // there is none yet) a first pass finds it.  The packed weights wait in registers: until
        // then S is still there.
        uint32_t pk[BK / 2];
        float l_new;
        bool renew = __any_sync(0xffffffffu, m == -INFINITY);
        while (true) {
          if (renew) {
            float mt = -INFINITY;
#pragma unroll 1
            for (int ch = 0; ch < BK / 32; ++ch) {
              uint32_t rr[32];
              ptx::tmem_ld32(lane_addr + ch * 32, rr);
              ptx::tmem_wait_ld_regs(rr);
#pragma unroll
              for (int i = 0; i < 32; ++i) mt = fmaxf(mt, __uint_as_float(rr[i]));
            }
            const float m_new = fmaxf(m, mt * sl2 - kLog2Unit);
            const float alpha = (m == -INFINITY) ? 0.f : ptx::ex2_approx(m - m_new);
            if (m_new != -INFINITY) m = m_new;
            l *= alpha;
            if (t > t_first) {
              // the previous product of this tile completed before this tile's S (commit order)
#pragma unroll 1
              for (int ch = 0; ch < D / 32; ++ch) {
                uint32_t rr[32];
                ptx::tmem_ld32(lane_addr + 128 + ch * 32, rr);
                ptx::tmem_wait_ld_regs(rr);
#pragma unroll
                for (int i = 0; i < 32; ++i) rr[i] = __float_as_uint(__uint_as_float(rr[i]) * alpha);
                ptx::tmem_st32(lane_addr + 128 + ch * 32, rr);
              }
            }
          }
          const float neg_m = (m == -INFINITY) ? 0.f : -m;
          const uint64_t nm2 = ptx::f2_pack(neg_m, neg_m);
          uint64_t lsum[2] = {0ull, 0ull};
          float mx[2] = {-INFINITY, -INFINITY};
          uint32_t rr[2][32];
          ptx::tmem_ld32(lane_addr, rr[0]);
#pragma unroll
          for (int ch = 0; ch < BK / 32; ++ch) {
            uint32_t(&cur)[32] = rr[ch & 1];
            ptx::tmem_wait_ld_regs(cur);
            if (ch + 1 < BK / 32) ptx::tmem_ld32(lane_addr + (ch + 1) * 32, rr[(ch + 1) & 1]);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float s0 = __uint_as_float(cur[i]), s1 = __uint_as_float(cur[i + 1]);
              mx[(i >> 1) & 1] = ptx::fmax3(mx[(i >> 1) & 1], s0, s1);
              float x0, x1;
              ptx::f2_unpack(ptx::ffma2(ptx::f2_pack(s0, s1), sl2x2, nm2), x0, x1);
              const float p0 = ptx::ex2_approx(x0), p1 = ptx::ex2_approx(x1);
              lsum[(i >> 1) & 1] = ptx::fadd2(lsum[(i >> 1) & 1], ptx::f2_pack(p0, p1));
              pk[ch * 16 + i / 2] = pack_f16x2(p0, p1);
            }
          }
          float ls0, ls1;
          ptx::f2_unpack(ptx::fadd2(lsum[0], lsum[1]), ls0, ls1);
          l_new = ls0 + ls1;
          if (renew || !__any_sync(0xffffffffu, fmaxf(mx[0], mx[1]) * sl2 > m + kLog2Range)) break;
          renew = true;
        }
        l += l_new;
        ptx::tmem_st32(lane_addr, *reinterpret_cast<uint32_t(*)[32]>(pk));
        ptx::tmem_st32(lane_addr + 32, *reinterpret_cast<uint32_t(*)[32]>(pk + 32));
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        arrive_first(&ctl.p_full[w], lane);
      }
      if (ok) ok = __all_sync(0xffffffffu, wait(&ctl.o_done, u));
      if (!ok) break;
      ptx::tc_fence_after();
      // ---- epilogue: the row's O, normalised or as this CTA's part.  In halves, the second
      // warpgroup leaves its sums and O (fp32, 16-byte chunks permuted by the row: a quarter warp
      // writes distinct banks) over Q, whose last product has completed, and the first adds them.
      float* half_o = reinterpret_cast<float*>(smem + L::kQ) + r * D;
      float2* half_ml = reinterpret_cast<float2*>(smem + L::kMl) + r;
      auto chunk = [&](int i) { return reinterpret_cast<float4*>(half_o + ((i ^ (r & (D / 4 - 1))) << 2)); };
      if (halves && w == 1) {
        const bool some = un.ntiles > 1;  // else O1 was never written
#pragma unroll 1
        for (int ch = 0; ch < D / 32; ++ch) {
          uint32_t rr[32];
          ptx::tmem_ld32(lane_addr + 128 + ch * 32, rr);
          ptx::tmem_wait_ld_regs(rr);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *chunk(ch * 8 + i) = some ? make_float4(__uint_as_float(rr[4 * i]), __uint_as_float(rr[4 * i + 1]),
                                                    __uint_as_float(rr[4 * i + 2]), __uint_as_float(rr[4 * i + 3]))
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        *half_ml = make_float2(m, l);
        ptx::tc_fence_before();
        ptx::mbar_arrive(&ctl.half_full);
        ok = __all_sync(0xffffffffu, wait(&ctl.half_free, n_half++));  // before Q is written again
        if (!ok) break;
        continue;
      }
      float a0 = 1.f, a1 = 0.f;
      if (halves) {
        ok = __all_sync(0xffffffffu, wait(&ctl.half_full, n_half++));
        if (!ok) break;
        const float2 o = *half_ml;
        const float top = fmaxf(m, o.x), base = top == -INFINITY ? 0.f : top;
        a0 = ptx::ex2_approx(m - base);
        a1 = ptx::ex2_approx(o.x - base);
        l = l * a0 + o.y * a1;
        m = top;
      }
      const float f = un.part >= 0 ? un.v_ref : (l == 0.f ? 0.f : un.v_ref / l);
      const int row = un.c0 + tok;
#pragma unroll 1
      for (int ch = 0; ch < D / 32; ++ch) {
        uint32_t rr[32];
        ptx::tmem_ld32(lane_addr + 128 + ch * 32, rr);
        ptx::tmem_wait_ld_regs(rr);
        if (halves) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 o = *chunk(ch * 8 + i);
            rr[4 * i] = __float_as_uint(__uint_as_float(rr[4 * i]) * a0 + o.x * a1);
            rr[4 * i + 1] = __float_as_uint(__uint_as_float(rr[4 * i + 1]) * a0 + o.y * a1);
            rr[4 * i + 2] = __float_as_uint(__uint_as_float(rr[4 * i + 2]) * a0 + o.z * a1);
            rr[4 * i + 3] = __float_as_uint(__uint_as_float(rr[4 * i + 3]) * a0 + o.w * a1);
          }
        }
        if (!valid) {
        } else if (un.part >= 0) {
          float4* dst = reinterpret_cast<float4*>(ws.o + ((int64_t)un.part * RT + r_unit) * D + ch * 32);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            dst[i] = make_float4(__uint_as_float(rr[4 * i]) * f, __uint_as_float(rr[4 * i + 1]) * f,
                                 __uint_as_float(rr[4 * i + 2]) * f, __uint_as_float(rr[4 * i + 3]) * f);
        } else {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + ((int64_t)row * a.Hq + h) * D + ch * 32);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            dst[i] = make_uint4(ptx::pack_bf16x2(__uint_as_float(rr[8 * i]) * f, __uint_as_float(rr[8 * i + 1]) * f),
                                ptx::pack_bf16x2(__uint_as_float(rr[8 * i + 2]) * f, __uint_as_float(rr[8 * i + 3]) * f),
                                ptx::pack_bf16x2(__uint_as_float(rr[8 * i + 4]) * f, __uint_as_float(rr[8 * i + 5]) * f),
                                ptx::pack_bf16x2(__uint_as_float(rr[8 * i + 6]) * f, __uint_as_float(rr[8 * i + 7]) * f));
        }
        __syncwarp();
      }
      if (valid) {
        if (un.part >= 0) ws.ml[un.part * RT + r_unit] = make_float2(m, l);
        else a.lse[(int64_t)h * a.rows + row] = lse_of(m, l);
      }
      if (halves) {  // nobody writes Q again before every row has been added
        ptx::mbar_arrive(&ctl.half_free);
        ok = __all_sync(0xffffffffu, wait(&ctl.half_free, n_half - 1));
        if (!ok) break;
      }
      ptx::tc_fence_before();
    }
    ptx::tc_fence_before();
  }
  grid_launch_dependents();
  __syncthreads();
  // the last products' arrivals in this CTA have come
  if (rank == 1 && tid == 0) (void)ptx::mbar_wait_bounded(&ctl.drained, 0, nullptr, a.err, kWaitNs);
  cluster_sync();  // neither CTA leaves while the other's products or arrivals may reach it
  if (warp == kMmaWarp) {
    ptx::tc_fence_after();
    tmem_dealloc2(tmem, kTmemCols);
  }
}

template <int D>
cp_status launch_typed(const CacheAttnArgs& a, void* wsp, cudaStream_t st) {
  using L = Layout<D>;
  const int64_t slots = slot_count(a.rows, a.G, a.n_seqs, RT);
  if (slots * a.Hkv > INT32_MAX) {
    set_last_error("too many rows and sequences for one launch");
    return CP_ERR_UNSUPPORTED;
  }
  auto kern = kv_attn_rows_kernel<D>;
  static KernelReady ready;
  int sms = 0;
  cp_status r = ready.prepare(kern, L::kSmemRequest, "kv_attn_rows_kernel", &sms, [&] {
    // setmaxnreg.inc waits until the registers it asks for are free in the block's
    // launch budget, so launch only if the split fits that budget.
    cudaFuncAttributes fa;
    const cudaError_t e = cudaFuncGetAttributes(&fa, kern);
    if (e != cudaSuccess) return cuda_check(e, "cudaFuncGetAttributes(kv_attn_rows)");
    if ((int64_t)fa.numRegs * kThreads < 256 * (kRegsLow + kRegsHigh)) {
      set_last_error("kv_attn_rows compiled with " + std::to_string(fa.numRegs) +
                     " registers per thread, too few for its warpgroup register split");
      return CP_ERR_UNSUPPORTED;
    }
    return CP_OK;
  });
  if (r != CP_OK) return r;
  WsPtrs ws;
  (void)ws_layout(wsp, slots, a.Hkv, RT, kRowsMaxPairs, D, &ws);
  CUtensorMap mk, mv;
  const int64_t code_rows = (int64_t)a.n_pages * a.Hkv * a.page;
  if ((r = make_codes_map(&mk, a.k, code_rows, D, std::min(a.page, BK / 2), D, false)) != CP_OK) return r;
  if ((r = make_codes_map(&mv, a.v, code_rows, D, a.page, D / 2, false)) != CP_OK) return r;
  if ((r = launch_chained(kern, dim3((unsigned)(2 * std::min(sms / 2, kRowsMaxPairs))), kThreads, L::kSmemRequest, st,
                          "kv_attn_rows_kernel launch", a, mk, mv, ws, (int)slots)) != CP_OK)
    return r;
  return launch_join<D, RT, true>(a, ws, slots, st);
}

}  // namespace

size_t kv_attention_rows_ws(int64_t rows, int32_t G, int32_t Hkv, int32_t D, int32_t n_seqs) {
  return ws_layout(nullptr, slot_count(rows, G, n_seqs, RT), Hkv, RT, kRowsMaxPairs, D, nullptr);
}

cp_status launch_kv_attention_rows(const CacheAttnArgs& a, void* ws, cudaStream_t st) {
  return a.D == 128 ? launch_typed<128>(a, ws, st) : launch_typed<64>(a, ws, st);
}

}  // namespace cpa
