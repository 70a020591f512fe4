// Attention over the quantised key/value cache for few query rows a key (decoding,
// drafted tokens), sm_103a.
//
// Mathematics.  s = scale q.k^, p = 2^(s log2 e - m), out = sum p v^ / sum p with the
// running maximum m and sum kept in fp32.  k^ and v^ are e4m3 codes times a power of
// two per (page, head), so the codes go to the tensor cores as they are and the scales
// are applied to scores and weights.  tcgen05's kind::f8f6f4 multiplies e4m3 exactly
// and adds in fp32 (measured: 1e-8 relative, as an fp32 chain), so the other operand
// is split into e4m3 parts: q = 2^e sum_i q_i 16^-i with q_i the e4m3
// rounding of 16 times what the parts before it left, 3 parts for the 8 bits of bf16,
// 6 for the 24 of fp32 (whole for elements down to 2^-17 and 2^-13 of the row's largest;
// smaller ones are off by up to 2^-25 and 2^-37 of it).  The weights of bf16 likewise, 3 parts of an 11-bit
// rounding (fp16: 2^-12 of each, an eighth of half a step of a bf16 result; their sum is
// kept whole); those of fp32 as 32-bit whole numbers in 8 parts of 4 bits: code k < 16 is k 2^-9 (subnormals
// and the first binade are one line), so a digit is its own code and no conversion is needed.
//
// Layout.  Keys are the M side: S^T [128 tokens x rows*parts] = K (A, K-major, as TMA
// brings it) Q^T (B), and O^T [D x rows*parts] = V^T (A, MN-major, the same page bytes)
// P^T (B, MN-major).  No code is converted or moved by a thread, and the few query rows
// cost little as the N side.  Thread t owns token t: its key and value scale are one
// value for all rows, the masks two comparisons a row.  A row's reference m follows its
// largest product of a weight and a value scale, whatever the scales that other rows see,
// and is renewed only when one grows to 2^3 times the largest at the last renewal (a
// warpgroup's vote), so a usual tile needs no reduction; sums stay per thread to the end.
//
// Bound by HBM: 2*D bytes a token and head.  The work, every (sequence, row tile, head)
// unit's tiles of 128 tokens in one line, is cut into equal runs, one a CTA (two CTAs an
// SM), whatever the lengths; a unit cut between CTAs leaves partial (m, l, O) in the
// workspace and kv_attn_join_kernel adds them in order, so results do not vary.
//
// Roles of a CTA: one or two warpgroups softmax and epilogue (two share the 8 rows of an fp32
// tile: 24 sequences of 1000 to 4000 tokens, 16 rows, D = 128, in 56.0 us; 57.5 with one), then a
// warp each: TMA producer (page ids and scales a batch ahead), MMA issuer (S of tile j+1 before
// PV of tile j), planner (decodes the next unit, splits its q); of 8 warps the last only helps
// to plan.
#include <algorithm>

#include "kv_plan.cuh"

namespace cpa {
namespace {

constexpr int kMaxCtas = 512;      // CTAs a workspace has partial results for
constexpr int kMaxRows = 16;       // largest row tile
constexpr int kMinRows = 4;        // smallest
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr uint64_t kDrainNs = 200000000ull;
// A row's weights are 2^(x - m) times their value scales in units of ev, the largest one seen so far.
// Its reference m puts the largest of them at 2^kLog2Unit, and is renewed when one passes 2^kLog2Range
// (e4m3 ends at 448, and a weight's whole number counts steps of 2^-23).  The last step of three parts
// is 2^-17, 2^-22 of the largest weight, that of eight 2^-28.  Where ev grows, m falls with it, so that
// a row that sees only small scales keeps its unit: by up to kLog2Fall a unit of work, and a score
// stays within kLog2Far of m, which keeps the sums under 2^117.
constexpr float kLog2Unit = 5.0f, kLog2Range = 8.0f, kLog2Far = 60.0f;
constexpr int kLog2Fall = 40;
constexpr float kNoMax = -1e30f;  // of a row that has seen nothing: finite, so that -inf less it is -inf
constexpr float kHidden = -1.0f;    // scale slot of a page that is not brought

// Row tile RT, parts of q and of a weight, softmax warpgroups.
template <int D_, int RT_, int NPQ_, int NPP_, int NG_>
struct Cfg {
  static constexpr int D = D_, RT = RT_, NPQ = NPQ_, NPP = NPP_, NG = NG_;
  static constexpr int NR = RT / NG;  // rows of a warpgroup; its columns are consecutive
  static constexpr int kSG = NR * NPQ, kOG = NR * NPP;
  static constexpr int kWarps = NG == 1 ? 8 : 11, kThreads = kWarps * 32;
  static constexpr int kProducerWarp = 4 * NG, kMmaWarp = 4 * NG + 1, kPlanWarp = 4 * NG + 2;
  static_assert(NG == 1 || kOG % 8 == 0, "columns are loaded by eights");
  static_assert(NPP == 3 || NPP == 8, "parts of a weight");
  // The work around a unit's tiles in tiles of these bytes.
  static constexpr int kCost = D == 64 ? 3 : 2;
  static constexpr int NS = (RT * NPQ + 15) / 16 * 16;  // columns of S^T
  static constexpr int NO = (RT * NPP + 15) / 16 * 16;  // columns of O^T
  // Part i of row r of q.
  static constexpr int q_row(int r, int i) { return r / NR * kSG + i * NR + r % NR; }
  // Column, within its warpgroup's, of part i of the group's row r: 3 parts (the first the largest)
  // i * NR + r; 8 digits (the first the smallest) a row's 8 bytes, the even ones before the odd ones.
  static constexpr int col(int r, int i) { return NPP == 3 ? i * NR + r : r * 8 + (i & 1) * 4 + (i >> 1); }
  static constexpr int row_of(int c) { return NPP == 3 ? c % NR : c / 8 % NR; }
  static constexpr int kPitch = NO <= 32 ? 32 : (NO <= 64 ? 64 : 128);  // bytes of a token's weights
  static constexpr int kTile = BK * D;
  // (a product of NS columns reads up to 8 rows behind its Q, of the next buffer: columns that nobody loads)
  static constexpr int kQBytes = (RT * NPQ * D + 1023) / 1024 * 1024;
  static constexpr int kPBytes = BK * kPitch;
  static constexpr int kFixed = 2 * kQBytes + 2 * kPBytes + 2048 + 1024;
  static constexpr int kBudget = 113 * 1024;  // two CTAs an SM
  static constexpr int kStagesFit = (kBudget - kFixed) / (2 * kTile);
  static constexpr int kStages = kStagesFit > 6 ? 6 : kStagesFit;
  static constexpr int kK = 0;
  static constexpr int kV = kK + kStages * kTile;
  static constexpr int kQ = kV + kStages * kTile;
  static constexpr int kP = kQ + 2 * kQBytes;
  static constexpr int kCtl = kP + 2 * kPBytes;
  static constexpr int kBytes = kCtl + 2048 + 1024;  // + alignment
  static constexpr int kCols = 2 * NS + NO <= 64 ? 64 : (2 * NS + NO <= 128 ? 128 : 256);
  static_assert(kStages >= 2 && 2 * NS + NO <= 256, "tile configuration");
  static_assert(kQBytes % 1024 == 0 && kPBytes % 1024 == 0, "swizzle atoms");
};

template <int RT>
struct Unit {
  int32_t b, hk, tile0, ntiles, len, nrows, row, part;  // part: partial slot, -1 = the whole unit
  int32_t lo_max, hi_min;  // tokens every row sees
  int32_t lo_min, hi_max;  // tokens some row sees
  int32_t lo[RT], hi[RT];
  float qs[RT];  // factor of a row's scores: q's power of two * softmax scale * log2(e)
};

template <class C>
struct Ctl {
  uint64_t kv_full[C::kStages], kv_empty[C::kStages];
  uint64_t s_full[2], p_full[2], pv_done[2], u_full[2], q_full[2], u_empty[2];
  Unit<C::RT> unit[2];
  float sc[C::kStages][8][2];  // key and value scale of a tile's pages
  int wred[C::NG][2][4][C::NR + 1];  // per warp: rows' maxima and the largest value scale; then sums
  uint64_t drained;
  PlanSmem<C::kWarps> plan;
  uint32_t tmem;
  int abort_flag;
};

template <int kSw>
__device__ __forceinline__ uint32_t swz(uint32_t off) {
  return off ^ (((off >> 7) & (kSw / 16 - 1)) << 4);
}
// Words of a shared-memory matrix descriptor for a swizzle of 32, 64 or 128 bytes.  The issuing
// thread works alone, so it adds one constant to a low word between two products and nothing else.
__host__ __device__ constexpr uint32_t desc_hi(int sw) {
  return (uint32_t)((8 * sw) >> 4) | (1u << 14) | ((sw == 128 ? 2u : (sw == 64 ? 4u : 6u)) << 29);
}
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) { return ((saddr >> 4) & 0x3FFFu) | (1u << 16); }
template <uint32_t kHiA, uint32_t kHiB, uint32_t kIdesc>
__device__ __forceinline__ void mma_f8_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tmov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %4};\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %5, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "n"(kHiA), "n"(kHiB), "r"(kIdesc), "r"((uint32_t)acc)
      : "memory");
}
// e4m3 x e4m3 -> fp32
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N, int a_mn, int b_mn) {
  return (1u << 4) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}
// 8, 16, 24 or 32 columns, loaded and waited for in one statement: the compiler must find no place
// between the two to move or spill registers that are yet to be filled.
__device__ __forceinline__ void tmem_ld_wait(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_wait(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, "
      "%8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_wait(uint32_t taddr, uint32_t (&r)[24]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, "
      "%8, %9, %10, %11, %12, %13, %14, %15}, [%24];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 "
      "{%16, %17, %18, %19, %20, %21, %22, %23}, [%25];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3]), "=&r"(r[4]), "=&r"(r[5]), "=&r"(r[6]), "=&r"(r[7]),
        "=&r"(r[8]), "=&r"(r[9]), "=&r"(r[10]), "=&r"(r[11]), "=&r"(r[12]), "=&r"(r[13]), "=&r"(r[14]), "=&r"(r[15]),
        "=&r"(r[16]), "=&r"(r[17]), "=&r"(r[18]), "=&r"(r[19]), "=&r"(r[20]), "=&r"(r[21]), "=&r"(r[22]), "=&r"(r[23])
      : "r"(taddr), "r"(taddr + 16)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_wait(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, "
      "%8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, "
      "%24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_wait(uint32_t taddr, uint32_t (&r)[48]) {
  tmem_ld_wait(taddr, *reinterpret_cast<uint32_t(*)[24]>(r));
  tmem_ld_wait(taddr + 24, *reinterpret_cast<uint32_t(*)[24]>(r + 24));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// Barriers of softmax warpgroup g.
__device__ __forceinline__ bool vote_any_128(int g, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(g + 1)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void sync_128(int g) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(g + 1) : "memory"); }

// Splits x into N e4m3 parts (part i scaled by 16^i); returns code i of the pair in out[i].
template <int N>
__device__ __forceinline__ void split_pair_f32(float x0, float x1, uint32_t (&out)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    out[i] = e4m3x2(x0, x1);
    if (i + 1 < N) {
      const float2 h = f16x2_to_f32(e4m3x2_to_f16x2(out[i]));
      x0 = (x0 - h.x) * 16.f;
      x1 = (x1 - h.y) * 16.f;
    }
  }
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// Two weights in three parts, by way of their fp16 roundings (11 bits, which three parts hold).
__device__ __forceinline__ void split_pair_f16(float x0, float x1, uint32_t (&out)[3]) {
  uint32_t h;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(x1), "f"(x0));
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c) : "r"(h));
    out[i] = c;
    if (i < 2) {  // (h - part) * 16; both steps are exact
      const uint32_t d = hfma2(e4m3x2_to_f16x2(c), 0xbc00bc00u, h);
      h = hfma2(d, 0x4c004c00u, 0u);
    }
  }
}
// O of row r from its parts' columns.
template <class C, int N>
__device__ __forceinline__ float join_parts(const uint32_t (&o)[N], int r) {
  auto part = [&](int i) { return __uint_as_float(o[C::col(r, i)]); };
  if constexpr (C::NPP == 3) return fmaf(fmaf(part(2), 0.0625f, part(1)), 0.0625f, part(0));
  float x = part(0);
#pragma unroll
  for (int i = 1; i < 8; ++i) x = fmaf(x, 0.0625f, part(i));
  return x * 16384.f;  // 2^9 a code, 16^7, 2^-23 a step
}

// 8 consecutive elements of q as fp32.
template <bool kBf16>
__device__ __forceinline__ void load8(float (&x)[8], const char* p, int at) {
  if constexpr (kBf16) {
    const uint4 w = ld(reinterpret_cast<const uint4*>(p + at * 2));
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 w = ld(reinterpret_cast<const float4*>(p + at * 4) + i);
      x[4 * i] = w.x;
      x[4 * i + 1] = w.y;
      x[4 * i + 2] = w.z;
      x[4 * i + 3] = w.w;
    }
  }
}

// ---------------------------------------------------------------- kernel
template <class C, bool kBf16>
__global__ void __launch_bounds__(C::kThreads, 2)
kv_attn_kernel(const __grid_constant__ CacheAttnArgs a, const __grid_constant__ CUtensorMap tm_k,
               const __grid_constant__ CUtensorMap tm_v, const WsPtrs ws, const int slots) {
  constexpr int D = C::D, RT = C::RT, NR = C::NR, NS = C::NS, NO = C::NO, ST = C::kStages;
  constexpr int kProducerWarp = C::kProducerWarp, kMmaWarp = C::kMmaWarp, kPlanWarp = C::kPlanWarp;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  static_assert(sizeof(Ctl<C>) <= 2048, "control block");
  Ctl<C>& ctl = *reinterpret_cast<Ctl<C>*>(smem + C::kCtl);
  const uint32_t sbase = ptx::smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      ptx::mbar_init(&ctl.kv_full[i], 1);
      ptx::mbar_init(&ctl.kv_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&ctl.s_full[i], 1);
      ptx::mbar_init(&ctl.p_full[i], 128 * C::NG);
      ptx::mbar_init(&ctl.pv_done[i], 1);
      ptx::mbar_init(&ctl.u_full[i], 1);
      ptx::mbar_init(&ctl.q_full[i], 1);
      ptx::mbar_init(&ctl.u_empty[i], 128 * C::NG + 2);
    }
    ptx::mbar_init(&ctl.drained, 1);
    ctl.abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == kProducerWarp && lane == 0) {
    ptx::prefetch_tensormap(&tm_k);
    ptx::prefetch_tensormap(&tm_v);
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(&ctl.tmem, C::kCols);
    ptx::tmem_relinquish();
  }

  // The batch's lengths are staged in the (still unused) tile buffers.
  grid_dependency_wait();
  const Run run = plan_run<RT, C::kCost, C::kWarps>(a, ws, slots, blockIdx.x, gridDim.x,
                                                    reinterpret_cast<int32_t*>(smem + C::kK), 2 * ST * C::kTile / 8 - 1,
                                                    ctl.plan);
  ptx::fence_proxy_async_smem();  // the staged lengths were written where TMA will write
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = ctl.tmem;
  volatile int* abort_flag = &ctl.abort_flag;
  auto wait = [&](uint64_t* bar, uint32_t par) {
    return ptx::mbar_wait_bounded(bar, par & 1u, abort_flag, a.err, kWaitNs);
  };

  if (run.slot >= 0) {
    if (warp == kPlanWarp) {
      // ------------------------------------------------------------ planner
      int64_t f = run.f0;
      const int64_t f1 = run.f1;
      int slot = run.slot, head = run.head, off = run.off;
      int u = 0;
      SlotRows sr = ctl.plan.rows;
      bool ok = true;
      while (f < f1) {
        const SlotSeq& q = sr.q;
        const int r0 = sr.r0, nrows = sr.nrows, t0 = sr.t0(), t1 = sr.t1();
        const Piece pc = unit_piece<C::kCost>(run, f, off, t1 - t0);
        const int n = pc.k1 - pc.k0, buf = u & 1;
        // The join goes by the records, so each of the run's is written, after a wait that gave up too.
        if (n > 0 && pc.k0 == 0 && lane == 0)
          ws.info[(int64_t)slot * a.Hkv + head] =
              unit_record<C::kCost>(run, blockIdx.x, q.c0 * a.G + r0, nrows, f, off, t1 - t0);
        if (n > 0 && ok && u >= 2) ok = __all_sync(0xffffffffu, wait(&ctl.u_empty[buf], (u >> 1) - 1));
        if (n > 0 && ok) {
          Unit<RT>& un = ctl.unit[buf];
          if (lane == 0) {
            un.b = q.b;
            un.hk = head;
            un.tile0 = t0 + pc.k0;
            un.ntiles = n;
            un.len = q.len;
            un.lo_min = sr.lo;
            un.hi_max = sr.hi;
            un.nrows = nrows;
            un.row = q.c0 * a.G + r0;
            un.part = n == t1 - t0 ? -1 : 2 * (int)blockIdx.x + (pc.k0 > 0 ? 0 : 1);
          }
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&ctl.u_full[buf]);  // the producer may start; the rest comes with q
          int lo = 0, hi = INT32_MAX;
          if (lane < RT && lane < nrows) row_bounds(a, q, (r0 + lane) / a.G, lo, hi);
          if (lane < RT) {
            un.lo[lane] = lane < nrows ? lo : 0;
            un.hi[lane] = lane < nrows ? hi : 0;
          }
          const int lo_max = __reduce_max_sync(0xffffffffu, lane < nrows && lane < RT ? lo : 0);
          const int hi_min = __reduce_min_sync(0xffffffffu, lane < nrows && lane < RT ? hi : INT32_MAX);
          if (lane == 0) {
            un.lo_max = lo_max;
            un.hi_min = hi_min;
          }
          // q of the unit's rows, split into e4m3 parts.
          // 32/RT lanes a row; rolled loops, as this code too is met cold.
          constexpr int LPR = 32 / RT, EPL = D / LPR;  // lanes a row, elements a lane
          const int r = lane / LPR, d0 = (lane % LPR) * EPL;
          const int rho = r0 + min(r, nrows - 1);
          const char* src = static_cast<const char*>(a.q) +
                            ((int64_t)(q.c0 + rho / a.G) * a.q_ld + (int64_t)(head * a.G + rho % a.G) * D + d0) * (kBf16 ? 2 : 4);
          uint32_t mx = 0;
#pragma unroll
          for (int v = 0; v < EPL / 8; ++v) {
            float x[8];
            load8<kBf16>(x, src, v * 8);
#pragma unroll
            for (int e = 0; e < 8; ++e) mx = max(mx, __float_as_uint(x[e]) & 0x7fffffffu);
          }
#pragma unroll
          for (int o = LPR / 2; o; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          const int ex = min(max((int)(mx >> 23) - 127, -100), 127);  // the row goes to [128, 256)
          const bool finite = mx < 0x7f800000u;
          const float up = finite ? pow2i(7 - ex) : 0.f;
          if (lane % LPR == 0) un.qs[r] = finite ? pow2i(ex - 7) * a.scale_log2 : __int_as_float(0x7fc00000);
          uint8_t* qdst = smem + C::kQ + buf * C::kQBytes;
#pragma unroll 1
          for (int v = 0; v < EPL / 8; ++v) {
            float x[8];
            load8<kBf16>(x, src, v * 8);
            uint32_t c[4][C::NPQ];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              split_pair_f32<C::NPQ>(finite ? x[2 * e] * up : 0.f, finite ? x[2 * e + 1] * up : 0.f, c[e]);
#pragma unroll
            for (int i = 0; i < C::NPQ; ++i)
              *reinterpret_cast<uint2*>(qdst + swz<D>((uint32_t)C::q_row(r, i) * D + d0 + v * 8)) =
                  make_uint2(c[0][i] | (c[1][i] << 16), c[2][i] | (c[3][i] << 16));
          }
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&ctl.q_full[buf]);
          ++u;
        }
        f += pc.take;
        off = 0;
        if (++head == a.Hkv) {
          head = 0;
          if (f < f1 && !next_rows<RT>(a, slots, slot, sr)) break;
        }
      }
      // the end of the run
      const int buf = u & 1;
      if (ok && u >= 2) ok = wait(&ctl.u_empty[buf], (u >> 1) - 1);
      if (lane == 0 && ok) {
        ctl.unit[buf].ntiles = 0;
        ptx::mbar_arrive(&ctl.u_full[buf]);
      }
    } else if (warp == kProducerWarp) {
      // ------------------------------------------------------------ TMA producer
      const int ppt = BK / a.page;  // pages a tile
      const uint32_t page_bytes = (uint32_t)(a.page * D);
      // With one row tile a sequence each code is read once: it should not push the partial results
      // and the next kernels' code and data out of L2.
      const uint64_t policy =
          a.rows * a.G <= (int64_t)RT * a.n_seqs ? ptx::evict_first_policy() : ptx::evict_normal_policy();
      int j = 0;
      bool ok = true;
      for (int u = 0;; ++u) {
        ok = wait(&ctl.u_full[u & 1], u >> 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const Unit<RT>& un = ctl.unit[u & 1];
        const int n = un.ntiles;
        if (n == 0) break;
        const int hk = un.hk;
        const int32_t* table = a.page_table + (int64_t)un.b * a.max_pages;
        // pages [p_first, p_end) of its tiles hold tokens that some row sees; the others are not brought and
        // need not exist (those before a window may have been given back)
        const int p0 = un.tile0 * ppt, p_first = un.lo_min / a.page;
        const int p_end = min((un.tile0 + n) * ppt, (un.hi_max + a.page - 1) / a.page);
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&ctl.u_empty[u & 1]);
        // 32 pages at a time, their ids and scales one batch ahead
        int id, id_n;
        float ks, vs, ks_n, vs_n;
        auto fetch = [&](int p, int& i, float& k, float& v) {
          i = -1;
          k = v = kHidden;
          if (p + lane >= p_first && p + lane < p_end) {
            i = ld(table + p + lane);
            if (i < 0 || i >= a.n_pages) {
              record_device_error(a.err, kDevIndex);
              i = -1;
            } else {
              k = ld(a.k_scale + (int64_t)i * a.Hkv + hk);
              v = ld(a.v_scale + (int64_t)i * a.Hkv + hk);
            }
          }
        };
        fetch(p0, id, ks, vs);
        fetch(p0 + 32, id_n, ks_n, vs_n);
        for (int t = 0; t < n; ++t, ++j) {
          const int at = (t * ppt) & 31;  // the tile's first page in the batch
          if (at == 0 && t > 0) {
            id = id_n;
            ks = ks_n;
            vs = vs_n;
            fetch(p0 + t * ppt + 32, id_n, ks_n, vs_n);
          }
          const int st = j % ST;
          if (j >= ST) ok = wait(&ctl.kv_empty[st], j / ST - 1);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const bool in = lane >= at && lane < at + ppt;
          if (in && id >= 0) {
            const int row = (id * a.Hkv + hk) * a.page;
            const uint32_t o = (uint32_t)(st * C::kTile) + (lane - at) * page_bytes;
            ptx::tma_load_2d(smem + C::kK + o, &tm_k, &ctl.kv_full[st], 0, row, policy);
            ptx::tma_load_2d(smem + C::kV + o, &tm_v, &ctl.kv_full[st], 0, row, policy);
          }
          // the copies need the ids alone; the scales (another dependent load) follow, and with
          // them the barrier's one arrival, before which its phase cannot end
          const uint32_t have = __ballot_sync(0xffffffffu, in && id >= 0);
          if (in) {
            ctl.sc[st][lane - at][0] = ks;
            ctl.sc[st][lane - at][1] = vs;
          }
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive_expect_tx(&ctl.kv_full[st], 2u * page_bytes * __popc(have));
          __syncwarp();
        }
        if (!ok) break;
      }
      if (*abort_flag && lane == 0)  // bounded wait for this CTA's copies in flight
        for (int i = max(0, j - ST); i < j; ++i)
          (void)ptx::mbar_wait_bounded(&ctl.kv_full[i % ST], (i / ST) & 1, nullptr, nullptr, kDrainNs);
      __syncwarp();
    } else if (warp == kMmaWarp) {
      // ------------------------------------------------------------ MMA issuer
      if (lane == 0) {
        constexpr uint32_t id_s = idesc_f8(BK, NS, 0, 0);
        constexpr uint32_t id_o = idesc_f8(D, NO, 1, 1);
        const uint32_t k_lo = desc_lo(sbase + C::kK), v_lo = desc_lo(sbase + C::kV), q_lo = desc_lo(sbase + C::kQ),
                       p_lo = desc_lo(sbase + C::kP);
        auto pv = [&](int j, int st, bool first) {  // O^T (+)= V_j^T P_j^T, V_j in stage st
          if (!wait(&ctl.p_full[j & 1], j >> 1)) return false;
          ptx::tc_fence_after();
          const uint32_t v = v_lo + st * (C::kTile >> 4), p = p_lo + (j & 1) * (C::kPBytes >> 4);
#pragma unroll
          for (int kk = 0; kk < BK / 32; ++kk)
            mma_f8_ss<desc_hi(D), desc_hi(C::kPitch), id_o>(tmem + 2 * NS, v + kk * 2 * D, p + kk * 2 * C::kPitch,
                                                            !first || kk > 0);
          ptx::tc_commit(&ctl.kv_empty[st]);
          ptx::tc_commit(&ctl.pv_done[j & 1]);
          return true;
        };
        int j = 0, st = 0, prev = 0;  // tile, its stage, the stage before
        uint32_t ph = 0;
        bool ok = true, pend = false, pend_first = false;
        for (int u = 0; ok; ++u) {
          if (!(ok = wait(&ctl.u_full[u & 1], u >> 1))) break;
          const int n = ctl.unit[u & 1].ntiles;
          if (n == 0) break;
          const uint32_t q = q_lo + (u & 1) * (C::kQBytes >> 4);
          if (!(ok = wait(&ctl.q_full[u & 1], u >> 1))) break;
          for (int t = 0; ok && t < n; ++t, ++j) {
            if (!(ok = wait(&ctl.kv_full[st], ph))) break;
            ptx::tc_fence_after();
            const uint32_t k = k_lo + st * (C::kTile >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk)
              mma_f8_ss<desc_hi(D), desc_hi(D), id_s>(tmem + (j & 1) * NS, k + kk * 2, q + kk * 2, kk > 0);
            ptx::tc_commit(&ctl.s_full[j & 1]);
            if (t == n - 1) ptx::tc_commit(&ctl.u_empty[u & 1]);  // the unit's Q has been read
            if (pend) ok = pv(j - 1, prev, pend_first);
            pend = true;
            pend_first = t == 0;
            prev = st;
            if (++st == ST) {
              st = 0;
              ph ^= 1u;
            }
          }
        }
        if (ok && pend) ok = pv(j - 1, prev, pend_first);
        // every product has completed before TMEM is released
        ptx::tc_commit(&ctl.drained);
        (void)ptx::mbar_wait_bounded(&ctl.drained, 0, nullptr, a.err, kDrainNs);
      }
      __syncwarp();
    } else if (warp < 4 * C::NG) {
      // ------------------------------------------------------------ softmax and epilogue
      // group g: rows row_g .. row_g + NR - 1 of the tile; wq, gt: this warp and thread of it
      const int g = C::NG == 1 ? 0 : warp >> 2, wq = warp & 3, gt = tid & 127, row_g = g * NR;
      const uint32_t lane_base = tmem + ((uint32_t)(wq * 32) << 16);
      const uint32_t s_addr = lane_base + g * C::kSG, o_addr = lane_base + 2 * NS + g * C::kOG;
      constexpr int kSL = (C::kSG + 7) / 8 * 8, kOL = (C::kOG + 7) / 8 * 8;  // columns loaded
      const int page_log2 = 31 - __clz(a.page);
      int j = 0, renewals = 0;
      bool ok = true;
      const float nan = __int_as_float(0x7fc00000);
      // A wait that gave up only clears `ok`: the four warps stay in step (they meet at named
      // barriers) and leave together at the next unit.
      for (int u = 0;; ++u) {
        ok &= wait(&ctl.u_full[u & 1], u >> 1);
        if (vote_any_128(g, !ok)) break;
        const Unit<RT>& un = ctl.unit[u & 1];
        const int n = un.ntiles;
        if (n == 0) break;
        ok &= wait(&ctl.q_full[u & 1], u >> 1);
        float m[NR], l[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          m[r] = kNoMax;
          l[r] = 0.f;
        }
        float ev = 0.f, inv_ev = INFINITY;  // largest value scale so far: the weights' unit
        int fall = kLog2Fall;               // what is left of it
        for (int t = 0; t < n; ++t, ++j) {
          const int key0 = (un.tile0 + t) * BK, key = key0 + gt, st = j % ST, buf = j & 1;
          ok &= wait(&ctl.s_full[buf], j >> 1);
          __syncwarp();
          ptx::tc_fence_after();
          const float ks = ctl.sc[st][gt >> page_log2][0], vs = ctl.sc[st][gt >> page_log2][1];
          const bool there = key < un.len && ks != kHidden;
          const float kf = vs != vs ? nan : ks;
          uint32_t sr[kSL];
          tmem_ld_wait(s_addr + buf * NS, sr);
          float x[NR];
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            float s = __uint_as_float(sr[(C::NPQ - 1) * NR + r]);
#pragma unroll
            for (int i = C::NPQ - 2; i >= 0; --i) s = fmaf(s, 0.0625f, __uint_as_float(sr[i * NR + r]));
            x[r] = s * un.qs[row_g + r] * kf;
          }
          if (!(key0 >= un.lo_max && key0 + BK <= un.hi_min) || !there) {
#pragma unroll
            for (int r = 0; r < NR; ++r)
              if (!there || key < un.lo[row_g + r] || key >= un.hi[row_g + r]) x[r] = -INFINITY;
          }
          // a weight times its value scale (in units of ev, a power of two: its exponent is its
          // logarithm) has to stay under 2^kLog2Range; larger scales alone are no reason to renew
          const float vw = there && key >= un.lo_min && key < un.hi_max && vs > 0.f ? vs : 0.f;
          float fv = vw * (vw > 0.f ? inv_ev : 0.f);
          const float room = fminf(kLog2Range + 127.f - (float)(__float_as_uint(fv) >> 23), kLog2Far);
          bool grow = fv > 8.f;
#pragma unroll
          for (int r = 0; r < NR; ++r) grow |= x[r] > m[r] + room;
          if (vote_any_128(g, grow)) {
            // new maxima, and O in their unit (an integer maximum over the warp is one instruction;
            // ordered as the floats are)
            auto ordered = [](float f) { const int i = __float_as_int(f); return i ^ ((i >> 31) & 0x7fffffff); };
            auto back = [](int i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); };
            int(*red)[NR + 1] = ctl.wred[g][renewals++ & 1];
            const int e_top = __reduce_max_sync(0xffffffffu, __float_as_int(vw));
            if (lane == 0) red[wq][NR] = e_top;
            sync_128(g);
            float e = fmaxf(__int_as_float(max(max(red[0][NR], red[1][NR]), max(red[2][NR], red[3][NR]))), ev);
            e = fmaxf(e, 1.17549435e-38f);
            const float ef = ev / e;
            const int drop = ev > 0.f ? min((__float_as_int(e) >> 23) - (__float_as_int(ev) >> 23), fall) : 0;
            fall -= drop;
            ev = e;
            inv_ev = 1.f / e;
            fv = vw * inv_ev;
            // logarithm of the value scale; smaller ones count as 2^(kLog2Unit - kLog2Far)
            const float lv = fmaxf((float)((int)(__float_as_uint(fv) >> 23) - 127), kLog2Unit - kLog2Far);
#pragma unroll
            for (int r = 0; r < NR; ++r) {
              const int top = __reduce_max_sync(0xffffffffu, ordered(x[r] == x[r] ? x[r] + lv : -INFINITY));
              if (lane == 0) red[wq][r] = top;
            }
            sync_128(g);
            float alpha[NR];
#pragma unroll
            for (int r = 0; r < NR; ++r) {
              const float mt = back(max(max(red[0][r], red[1][r]), max(red[2][r], red[3][r])));
              const float mn = fmaxf(m[r] - (float)drop, mt - kLog2Unit);
              alpha[r] = ptx::ex2_approx(m[r] - mn);
              l[r] *= alpha[r];
              m[r] = mn;
              alpha[r] *= ef;
            }
            if (t > 0) {
              ok &= wait(&ctl.pv_done[(j - 1) & 1], (j - 1) >> 1);
              __syncwarp();
              ptx::tc_fence_after();
#pragma unroll
              for (int c = 0; c < kOL; c += 8) {
                uint32_t o[8];
                tmem_ld_wait(o_addr + c, o);
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha[C::row_of(c + i)]);
                tmem_st8(o_addr + c, o);
              }
              ptx::tmem_wait_st();
            }
          }
          if (j >= 2) ok &= wait(&ctl.pv_done[buf], (j >> 1) - 1);  // the weights of tile j - 2 have been read
          uint8_t* pd = smem + C::kP + buf * C::kPBytes;
          if constexpr (C::NPP == 3) {
            uint32_t pc[3][NR / 2];
#pragma unroll
            for (int r = 0; r < NR; r += 2) {
              const float p0 = ptx::ex2_approx(x[r] - m[r]);
              const float p1 = ptx::ex2_approx(x[r + 1] - m[r + 1]);
              l[r] += p0;
              l[r + 1] += p1;
              uint32_t c[3];
              split_pair_f16(p0 * fv, p1 * fv, c);
#pragma unroll
              for (int i = 0; i < 3; ++i) pc[i][r / 2] = c[i];
            }
#pragma unroll
            for (int i = 0; i < 3; ++i)
#pragma unroll
              for (int r = 0; r < NR; r += 4)
                *reinterpret_cast<uint32_t*>(pd + swz<C::kPitch>((uint32_t)(gt * C::kPitch + g * C::kOG + C::col(r, i)))) =
                    pc[i][r / 2] | (pc[i][r / 2 + 1] << 16);
          } else {
            const float fs = fv * 8388608.f;
#pragma unroll
            for (int r = 0; r < NR; r += 2) {
              const float p0 = ptx::ex2_approx(x[r] - m[r]);
              const float p1 = ptx::ex2_approx(x[r + 1] - m[r + 1]);
              l[r] += p0;
              l[r + 1] += p1;
              const uint32_t n0 = __float2uint_rn(p0 * fs), n1 = __float2uint_rn(p1 * fs);  // (a NaN is in the sum)
              constexpr uint32_t kEven = 0x0f0f0f0fu;
              *reinterpret_cast<uint4*>(pd + swz<C::kPitch>((uint32_t)(gt * C::kPitch + g * C::kOG + r * 8))) =
                  make_uint4(n0 & kEven, (n0 >> 4) & kEven, n1 & kEven, (n1 >> 4) & kEven);
            }
          }
          if (!there && g == 0) {  // a token past the end or of a page that was not brought: its bytes may be anything
            (void)wait(&ctl.kv_full[st], j / ST);
            uint4* vz = reinterpret_cast<uint4*>(smem + C::kV + st * C::kTile + gt * D);
#pragma unroll
            for (int i = 0; i < D / 16; ++i) vz[i] = make_uint4(0, 0, 0, 0);
          }
          ptx::fence_proxy_async_smem();
          ptx::tc_fence_before();
          ptx::mbar_arrive(&ctl.p_full[buf]);
        }
        // ---- epilogue: the sums over the tokens, then O^T: thread = element d of every row
        int(*sums)[NR + 1] = ctl.wred[g][renewals++ & 1];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
#pragma unroll
          for (int o = 16; o; o >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
          if (lane == 0) sums[wq][r] = __float_as_int(l[r]);
        }
        sync_128(g);
        ok &= wait(&ctl.pv_done[(j - 1) & 1], (j - 1) >> 1);
        ok = __all_sync(0xffffffffu, ok);
        ptx::tc_fence_after();
        uint32_t orr[kOL];
        tmem_ld_wait(o_addr, orr);
        const int d = D == 128 ? gt : wq * 16 + lane;  // M = 64 keeps 16 rows in each warp's lanes
        const bool has_d = D == 128 || lane < 16;
        const int nrows = un.nrows - row_g, row0 = un.row + row_g, part = un.part, hk = un.hk;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          if (r < nrows && ok) {
            const float o = join_parts<C>(orr, r) * ev;
            const float sum = __int_as_float(sums[0][r]) + __int_as_float(sums[1][r]) + __int_as_float(sums[2][r]) +
                              __int_as_float(sums[3][r]);
            if (part >= 0) {
              if (has_d) ws.o[((int64_t)part * RT + row_g + r) * D + d] = o;
              if (gt == 0) ws.ml[part * RT + row_g + r] = make_float2(m[r], sum);
            } else {
              const int row = (row0 + r) / a.G, h = hk * a.G + (row0 + r) % a.G;
              const float y = sum == 0.f ? 0.f : o / sum;
              const int64_t at = ((int64_t)row * a.Hq + h) * D + d;
              if (has_d) {
                if constexpr (kBf16) static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(y);
                else static_cast<float*>(a.out)[at] = y;
              }
              if (gt == 0)
                a.lse[(int64_t)h * a.rows + row] = lse_of(m[r], sum);
            }
          }
        }
        ptx::tc_fence_before();
        sync_128(g);  // wred is free, every thread has read the unit
        ptx::mbar_arrive(&ctl.u_empty[u & 1]);
      }
      ptx::tc_fence_before();
    }
  }
  grid_launch_dependents();
  __syncthreads();
  if (warp == kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::kCols);
  }
}

// ---------------------------------------------------------------- host side
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn get_encode_fn() {
  static const EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<EncodeTiledFn>(p);
    return (EncodeTiledFn) nullptr;
  }();
  return fn;
}

template <class C, bool kBf16>
cp_status launch_cfg(const CacheAttnArgs& a, void* wsp, cudaStream_t st) {
  const int64_t slots = slot_count(a.rows, a.G, a.n_seqs, C::RT);
  if (slots * a.Hkv > INT32_MAX) {
    set_last_error("too many rows and sequences for one launch");
    return CP_ERR_UNSUPPORTED;
  }
  WsPtrs ws;
  (void)ws_layout(wsp, slots, a.Hkv, C::RT, kMaxCtas, C::D, &ws);
  CUtensorMap mk, mv;
  const int64_t code_rows = (int64_t)a.n_pages * a.Hkv * a.page;
  cp_status r;
  if ((r = make_codes_map(&mk, a.k, code_rows, C::D, a.page, C::D, true)) != CP_OK) return r;
  if ((r = make_codes_map(&mv, a.v, code_rows, C::D, a.page, C::D, true)) != CP_OK) return r;
  auto kern = kv_attn_kernel<C, kBf16>;
  static KernelReady ready;
  int sms = 0;
  if ((r = ready.prepare(kern, C::kBytes, "kv_attn_kernel", &sms, [] { return CP_OK; })) != CP_OK) return r;
  if ((r = launch_chained(kern, dim3((unsigned)std::min(2 * sms, kMaxCtas)), C::kThreads, C::kBytes, st,
                          "kv_attn_kernel launch", a, mk, mv, ws, (int)slots)) != CP_OK)
    return r;
  return launch_join<C::D, C::RT, kBf16>(a, ws, slots, st);
}

}  // namespace

cp_status make_codes_map(CUtensorMap* m, const void* base, int64_t rows, int D, int box_rows, int box_cols,
                         bool swizzle) {
  const EncodeTiledFn enc = get_encode_fn();
  if (!enc) {
    set_last_error("cuTensorMapEncodeTiled unavailable from the driver");
    return CP_ERR_CUDA;
  }
  cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)std::max<int64_t>(rows, 1)};
  cuuint64_t strides[1] = {(cuuint64_t)D};
  cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE,
                         !swizzle ? CU_TENSOR_MAP_SWIZZLE_NONE
                                  : (D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B),
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_last_error("cuTensorMapEncodeTiled failed (code " + std::to_string((int)r) + ")");
    return CP_ERR_CUDA;
  }
  return CP_OK;
}

namespace {

// Many rows a key: the rows kernel.  Its tile costs the same for 1 to 256 rows, this kernel's
// grows by 16 rows (16 sequences of 8192 tokens, 8 heads of 128: 156 to 161 us for 16 to 64 rows
// against 67 for 16, 124 for 32, 176 for 48, 225 for 64; D = 64: 135 to 141 us against 56, 90, 129 and
// 161).
bool many_rows(int64_t rows, int64_t G, int64_t n_seqs, bool is_bf16) { return is_bf16 && rows * G > 32 * n_seqs; }

}  // namespace

size_t kv_attention_ws(int64_t rows, int32_t Hq, int32_t Hkv, int32_t D, int32_t is_bf16, int32_t n_seqs) {
  const int32_t G = std::max(1, Hq / std::max(1, Hkv));
  if (many_rows(rows, G, n_seqs, is_bf16)) return kv_attention_rows_ws(rows, G, Hkv, D, n_seqs);
  return ws_layout(nullptr, slot_count(rows, G, n_seqs, kMinRows), Hkv, kMaxRows, kMaxCtas, D, nullptr);
}

cp_status launch_kv_attention(const CacheAttnArgs& a, int is_bf16, void* ws, cudaStream_t st) {
  if (many_rows(a.rows, a.G, a.n_seqs, is_bf16)) return launch_kv_attention_rows(a, ws, st);
  // Rows of a tile: 4 or 8 while a sequence has no more (row, head of its group) pairs on
  // average, else 16 (fp32, whose parts fill the columns with 8 rows: 8).
  const int64_t rows = a.rows * a.G, n = a.n_seqs;
  if (a.D == 128) {
    if (!is_bf16)
      return rows <= 4 * n ? launch_cfg<Cfg<128, 4, 6, 8, 1>, false>(a, ws, st) : launch_cfg<Cfg<128, 8, 6, 8, 2>, false>(a, ws, st);
    if (rows <= 4 * n) return launch_cfg<Cfg<128, 4, 3, 3, 1>, true>(a, ws, st);
    return rows <= 8 * n ? launch_cfg<Cfg<128, 8, 3, 3, 1>, true>(a, ws, st) : launch_cfg<Cfg<128, 16, 3, 3, 1>, true>(a, ws, st);
  }
  if (!is_bf16)
    return rows <= 4 * n ? launch_cfg<Cfg<64, 4, 6, 8, 1>, false>(a, ws, st) : launch_cfg<Cfg<64, 8, 6, 8, 2>, false>(a, ws, st);
  if (rows <= 4 * n) return launch_cfg<Cfg<64, 4, 3, 3, 1>, true>(a, ws, st);
  return rows <= 8 * n ? launch_cfg<Cfg<64, 8, 3, 3, 1>, true>(a, ws, st) : launch_cfg<Cfg<64, 16, 3, 3, 1>, true>(a, ws, st);
}

}  // namespace cpa
