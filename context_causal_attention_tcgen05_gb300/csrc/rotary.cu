// Rotary positions with several axes, applied to q and k in one launch.
//
// Pair i of row s turns by positions[axis(i)][s] * inv_freq[i].  Whole turns do not
// matter, so the angle is kept as a 64-bit fixed-point fraction of a turn: with
// F = inv_freq / (2 pi) * 2^64, position * F modulo 2^64 drops the whole turns by
// itself, at any position.  F is formed from the 24 bits of inv_freq and 64 bits of
// 1 / (2 pi) in integers, so it is off by at most two units and the angle of a 32-bit
// position by 2^-32 of a turn.  Quarter turns are taken off in integers, so what is rounded
// to fp32 is at most an eighth of a turn, and cos and sin are right to their own size (fp32
// results are off by 3.9e-8 of theirs in the 2-norm: a rounding each of cos, sin, a product, a sum).
#include "serve.cuh"

namespace cpa {
namespace {

constexpr int kThreads = 128;

// inv_freq / (2 pi) modulo 1, times 2^64.
__device__ __forceinline__ uint64_t turn_fraction(float inv_freq) {
  constexpr uint64_t kInv2Pi = 0xa2f9836e4e441529ull;  // floor(2^66 / (2 pi))
  const uint32_t bits = __float_as_uint(inv_freq), ex = (bits >> 23) & 0xffu;
  const uint64_t m = (bits & 0x7fffffu) | (ex ? 0x800000u : 0u);
  const int shift = 2 - ((int)(ex ? ex : 1u) - 150);  // inv_freq = m * 2^(ex - 150)
  const uint64_t lo = m * kInv2Pi, hi = __umul64hi(m, kInv2Pi);
  uint64_t f = 0;
  if (shift <= 0) f = -shift < 64 ? lo << -shift : 0;
  else if (shift < 64) f = (lo >> shift) | (hi << (64 - shift));
  else if (shift < 128) f = hi >> (shift - 64);
  return (bits >> 31) ? 0 - f : f;
}

// One work item: 16 bytes of a head (neighbouring pairs, or elements that are only copied), or 16
// bytes of each half.  Items of a tensor are numbered (row, head, place), a thread taking every
// kThreads-th; the position is carried along, which costs no division.
struct Place {
  int r, h, v;
};

// Bound by HBM: every element is read and written once.  A block takes a few rows; cos and sin of
// each of their pairs are computed once for all heads, while the first loads are on their way.
// 64 bytes a thread are loaded before any are written (q and k of 65536 rows, 40 heads of 128, bf16:
// 207 us, 6.5 TB/s; half of 64 heads of 8192 fp32 rows: 85 us, 6.3 TB/s, against 107 with 16 bytes;
// 128 bytes, which leave fewer blocks a SM, 93).
template <bool kBf16, bool kInter>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryArgs a, int rows_per_block) {
  extern __shared__ float2 cs[];  // [rows_per_block][rot / 2]
  constexpr int kV = kBf16 ? 8 : 4;  // elements in 16 bytes
  constexpr int kU = kInter ? 4 : 2;
  constexpr int64_t es = kBf16 ? 2 : 4;
  const int pairs = a.rot >> 1;
  const int64_t s0 = (int64_t)blockIdx.x * rows_per_block;
  const int n = (int)min((int64_t)rows_per_block, a.S - s0);
  const int vpp = kInter ? a.rot / kV : pairs / kV;  // rotated items of a head
  const int half = pairs * (int)es;
  grid_dependency_wait();
  grid_launch_dependents();
  bool have_cs = false;
#pragma unroll 1
  for (int w = 0; w < 2; ++w) {
    if (a.x[w] == nullptr) continue;
    const int per_head = vpp + (a.x[w] == a.y[w] ? 0 : (a.D - a.rot) / kV), H = a.H[w];
    const int dh = kThreads / per_head, dv = kThreads - dh * per_head;
    const char* src0 = static_cast<const char*>(a.x[w]) + s0 * a.x_ld[w] * es;
    char* dst0 = static_cast<char*>(a.y[w]) + s0 * a.y_ld[w] * es;
    const int64_t x_row = a.x_ld[w] * es, y_row = a.y_ld[w] * es;
    Place p;
    p.h = threadIdx.x / per_head;
    p.v = threadIdx.x - p.h * per_head;
    p.r = 0;
    auto carry = [&] {
      while (p.h >= H && p.r < n) {
        p.h -= H;
        ++p.r;
      }
    };
    carry();
    while (true) {
      Place at[kU];
      uint4 x[kU], z[kU];
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        at[i] = p;
        if (p.r < n) {
          const char* src = src0 + p.r * x_row + p.h * a.D * es;
          const bool copy = p.v >= vpp;
          x[i] = *reinterpret_cast<const uint4*>(src + (copy ? a.rot * es + (p.v - vpp) * 16 : p.v * 16));
          if (!kInter && !copy) z[i] = *reinterpret_cast<const uint4*>(src + half + p.v * 16);
          p.v += dv;
          p.h += dh;
          if (p.v >= per_head) {
            p.v -= per_head;
            ++p.h;
          }
          carry();
        }
      }
      if (!have_cs) {
        for (int t = threadIdx.x; t < n * pairs; t += kThreads) {
          const int r = t / pairs, i = t - r * pairs;
          int ax = 0;
          while (ax + 1 < a.n_axes && i >= a.axis_end[ax]) ++ax;
          const int64_t pos = ld(a.positions + (int64_t)ax * a.S + s0 + r);
          const float f = ld(a.inv_freq + i);
          const uint64_t turn = turn_fraction(f) * (uint64_t)pos;  // whole turns drop out
          const uint32_t quarter = (uint32_t)((turn + (1ull << 61)) >> 62);
          float rest = (float)(int64_t)(turn - ((uint64_t)quarter << 62)) * 0x1p-63f;  // half turns
          if (!isfinite(f)) rest = __int_as_float(0x7fc00000);
          float sn, c;
          sincospif(rest, &sn, &c);
          const float c4 = quarter & 1 ? -sn : c, s4 = quarter & 1 ? c : sn;
          c = quarter & 2 ? -c4 : c4;
          sn = quarter & 2 ? -s4 : s4;
          cs[t] = make_float2(c, a.inverse ? -sn : sn);
        }
        __syncthreads();
        have_cs = true;
      }
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        if (at[i].r >= n) break;
        char* dst = dst0 + at[i].r * y_row + at[i].h * a.D * es;
        const int v = at[i].v;
        if (v >= vpp) {  // not rotated
          *reinterpret_cast<uint4*>(dst + a.rot * es + (v - vpp) * 16) = x[i];
          continue;
        }
        const float2* row_cs = cs + at[i].r * pairs;
        const uint32_t xi[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        uint32_t yo[4];
        if constexpr (kInter) {
          if constexpr (kBf16) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 c = row_cs[v * 4 + k];
              const float e = __uint_as_float(xi[k] << 16), o = __uint_as_float(xi[k] & 0xffff0000u);
              const __nv_bfloat162 y = __floats2bfloat162_rn(e * c.x - o * c.y, o * c.x + e * c.y);
              yo[k] = *reinterpret_cast<const uint32_t*>(&y);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float2 c = row_cs[v * 2 + k];
              const float e = __uint_as_float(xi[2 * k]), o = __uint_as_float(xi[2 * k + 1]);
              yo[2 * k] = __float_as_uint(e * c.x - o * c.y);
              yo[2 * k + 1] = __float_as_uint(o * c.x + e * c.y);
            }
          }
          *reinterpret_cast<uint4*>(dst + v * 16) = make_uint4(yo[0], yo[1], yo[2], yo[3]);
        } else {
          const uint32_t zi[4] = {z[i].x, z[i].y, z[i].z, z[i].w};
          uint32_t wo[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if constexpr (kBf16) {
              const float2 c0 = row_cs[v * 8 + 2 * k], c1 = row_cs[v * 8 + 2 * k + 1];
              const float p0 = __uint_as_float(xi[k] << 16), q0 = __uint_as_float(zi[k] << 16);
              const float p1 = __uint_as_float(xi[k] & 0xffff0000u), q1 = __uint_as_float(zi[k] & 0xffff0000u);
              const __nv_bfloat162 o = __floats2bfloat162_rn(p0 * c0.x - q0 * c0.y, p1 * c1.x - q1 * c1.y);
              const __nv_bfloat162 g = __floats2bfloat162_rn(q0 * c0.x + p0 * c0.y, q1 * c1.x + p1 * c1.y);
              yo[k] = *reinterpret_cast<const uint32_t*>(&o);
              wo[k] = *reinterpret_cast<const uint32_t*>(&g);
            } else {
              const float2 c = row_cs[v * 4 + k];
              const float e = __uint_as_float(xi[k]), o = __uint_as_float(zi[k]);
              yo[k] = __float_as_uint(e * c.x - o * c.y);
              wo[k] = __float_as_uint(o * c.x + e * c.y);
            }
          }
          *reinterpret_cast<uint4*>(dst + v * 16) = make_uint4(yo[0], yo[1], yo[2], yo[3]);
          *reinterpret_cast<uint4*>(dst + half + v * 16) = make_uint4(wo[0], wo[1], wo[2], wo[3]);
        }
      }
      if (p.r >= n) break;
    }
  }
}

}  // namespace

cp_status launch_rotary(const RotaryArgs& a, int is_bf16, int interleaved, cudaStream_t st) {
  const int rpb = 4;
  const unsigned grid = (unsigned)((a.S + rpb - 1) / rpb);
  const size_t sm = (size_t)rpb * (a.rot / 2) * sizeof(float2);
  auto kern = is_bf16 ? (interleaved ? rotary_kernel<true, true> : rotary_kernel<true, false>)
                      : (interleaved ? rotary_kernel<false, true> : rotary_kernel<false, false>);
  return launch_chained(kern, dim3(grid), kThreads, sm, st, "rotary_kernel launch", a, rpb);
}

}  // namespace cpa
