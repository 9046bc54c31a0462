// norm_rope.cu -- RMS norm, rotary embedding and, for cache entries, the FP4
// quantisation into a paged cache, in one launch (csa2_qk_norm_rope).
//
//   y = x (mean(x^2) + eps)^(-1/2) w, then for channel pair i at position p
//   (u, v) <- s (u cos phi - v sin phi, v cos phi + u sin phi), phi = 2 pi frac(p t_i)
// with t_i the pair's turns per position as a 64-bit binary fraction: p * t_i
// modulo 2^64 is the exact fraction of a turn, whatever the position, where an
// fp32 angle would be off by 0.03 rad at a position of a million.
//
// One warp per head of a token (fp32, bf16 out) or per entry (fp64, so that a
// value next to a border of the E2M1 grid falls to its own side: a borderline
// flip would make the stored codes depend on the order of a sum). A lane holds
// chunks of 8 channels (lane + 32 j), read as 16-byte words, two heads at a time;
// the weights stay in its registers and the cosines and sines of a token are
// computed once per CTA, while the first heads are on their way. Rotation:
//   neighbouring channels are in one lane's chunk (the first an even one);
//   halves R/2 apart are R/16 chunks apart: one exchange between lanes, where
//   the rotary part lies within one round of 32 chunks on chunk borders;
//   anything else goes through a per-warp strip of shared memory.
// An entry's group of 16 channels is two neighbouring lanes: one exchange gives its
// maximum, the codes of a lane are one 32-bit word. Bound: HBM (a few dozen
// instructions per 16 bytes read and written); at single tokens, the launch. Measured:
// 4096 tokens of 64 heads of 512 channels (bf16) and 1024 entries, 539 MB, in 89 us of
// device time (6.0 TB/s; a plain copy: 6.5), 95 with the host's part.
#include "common.cuh"
#include "kernels.h"

namespace csa2 {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
// tables and strips: what a launch may have, without the words of far rows
constexpr size_t kTableBytes = 48 * 1024 - kWarps * sizeof(uint32_t);

// how channels rotate (kPairs: kInLane where the rotary part is not whole chunks)
enum : int { kNone = 0, kInLane = 1, kPairs = 2, kExchange = 3, kStrip = 4 };

// Two floats in one 64-bit register: half the instructions of separate ones.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

struct NormRope {
  csa2_norm_rope_args a;
  fp4_kv_pages pg;
  int shift;
  int entry_blocks, entries_per_cta;
  int rows_per_cta;  // (token, head) rows, of tokens_per_cta tokens at most
  int tokens_per_cta;
  int step_tok, step_head;   // kWarps rows as tokens and heads
  int* err;
};

__device__ __forceinline__ void load8(const void* base, bool f32, size_t at, float (&v)[8]) {
  if (f32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    const float4 a = __ldcs(p), b = __ldcs(p + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 w = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at));
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(x[k] << 16);
      v[2 * k + 1] = __uint_as_float(x[k] & 0xffff0000u);
    }
  }
}

__device__ __forceinline__ uint32_t pack_bf162(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

__device__ __forceinline__ uint4 pack_bf16x8(const float (&v)[8]) {
  return make_uint4(pack_bf162(v[0], v[1]), pack_bf162(v[2], v[3]), pack_bf162(v[4], v[5]),
                    pack_bf162(v[6], v[7]));
}

// The signed fraction of a turn, in [-1/2, 1/2), of pair t at position p.
__device__ __forceinline__ long long turn_fraction(int p, uint64_t t) {
  return (long long)((uint64_t)(long long)p * t);
}

template <typename F>
__device__ __forceinline__ F warp_sum(F x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Place of channel c in a strip: one word of 33 skipped, as the lanes are 8 channels apart.
__host__ __device__ constexpr int strip_at(int c) { return c + (c >> 5); }

// Rotates through `strip` (by channel, strip_at(D) values of the warp): the chunks that
// hold rotary channels go there, a lane takes every 32nd pair, and the chunks come back.
// (Each lane rotating its own channels from there takes 1.15 to 1.45 times as long.)
template <int J, typename F>
__device__ __forceinline__ void rotate_strip(const csa2_norm_rope_args& a, F (&y)[J][8], F* strip,
                                             const F* cs) {
  const int lane = threadIdx.x & 31;
  const int b = a.rot_begin, end = b + a.R, half = a.R / 2;
  const int next = a.interleaved ? 2 : 1, other = a.interleaved ? 1 : half;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c0 = (lane + 32 * j) * 8;
    if (c0 >= a.D || c0 + 8 <= b || c0 >= end) continue;
    F* at = strip + strip_at(c0);                      // a chunk lies within one run of 32
#pragma unroll
    for (int k = 0; k < 8; ++k) at[k] = y[j][k];
  }
  __syncwarp();
  for (int i = lane; i < half; i += 32) {
    const int c = b + i * next;
    F* pu = strip + strip_at(c);
    F* pv = strip + strip_at(c + other);
    const F u = *pu, v = *pv, co = cs[2 * i], si = cs[2 * i + 1];
    *pu = u * co - v * si;
    *pv = v * co + u * si;
  }
  __syncwarp();
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c0 = (lane + 32 * j) * 8;
    if (c0 >= a.D || c0 + 8 <= b || c0 >= end) continue;
    const F* at = strip + strip_at(c0);
#pragma unroll
    for (int k = 0; k < 8; ++k) y[j][k] = at[k];
  }
  __syncwarp();
}

// E2M1 magnitude code of |x| at scale s, by comparison with the midpoints (exact
// products); at a midpoint the even code wins.
__device__ __forceinline__ uint32_t e2m1_code64(double x, double s) {
  if (s == 0.0) return 0u;
  const double a = fabs(x);
  const uint32_t c = (a > 0.25 * s) + (a >= 0.75 * s) + (a > 1.25 * s) + (a >= 1.75 * s) +
                     (a > 2.5 * s) + (a >= 3.5 * s) + (a > 5.0 * s);
  return c | (signbit(x) ? 8u : 0u);
}

// Nearest E4M3 code of x >= 0 (ties to even, saturating at 448), exactly: the
// candidates are multiples of 2^(e - 3) in x's binade (2^-9 below 2^-6), and a
// double holds x / step without rounding. A NaN gives 0x7f.
__device__ __forceinline__ uint32_t e4m3_code64(double x) {
  if (!(x <= 448.0)) return x != x ? 0x7fu : 0x7eu;
  const int e = max(-6, (int)((__double2hiint(x) >> 20) & 0x7ff) - 1023);
  const double step_inv = __hiloint2double((1023 + 3 - e) << 20, 0);
  const int n = __double2int_rn(x * step_inv);         // 0 .. 16, ties to even
  return (uint32_t)((e + 6) * 8 + n);                  // n = 16 carries into the exponent
}

template <int J, int kPath>
__device__ void entry_row(const NormRope& p, int e, double* strip, const double* cs) {
  const csa2_norm_rope_args& a = p.a;
  const int lane = threadIdx.x & 31;
  const int D = a.D;
  double y[J][8];
  double sum = 0.0;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c0 = (lane + 32 * j) * 8;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (c0 < D) load8(a.kv, a.kv_f32 != 0, (size_t)e * a.kv_stride + c0, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      y[j][k] = (double)v[k];
      sum = fma(y[j][k], y[j][k], sum);
    }
  }
  if (a.kv_norm) {
    const double r = 1.0 / sqrt(warp_sum(sum) / D + (double)a.eps);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c0 = (lane + 32 * j) * 8;
      if (c0 >= D) continue;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        y[j][k] *= a.kv_weight ? r * (double)__ldg(a.kv_weight + c0 + k) : r;
    }
  }
  if (kPath == kInLane || kPath == kPairs) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c0 = (lane + 32 * j) * 8 - a.rot_begin;     // in the rotary part; even
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        if (c0 + k < 0 || c0 + k >= a.R) continue;
        const double u = y[j][k], v = y[j][k + 1], c = cs[c0 + k], s = cs[c0 + k + 1];
        y[j][k] = u * c - v * s;
        y[j][k + 1] = v * c + u * s;
      }
    }
  } else if (kPath != kNone) {
    rotate_strip<J>(a, y, strip, cs);
  }

  // the row in the cache: its slot's page must be this slot's alone
  const int s = __ldg(a.seq + e), at = __ldg(a.entry + e);
  uint8_t* row = nullptr;
  if (s >= 0 && s < p.pg.S && at >= 0 && at < __ldg(p.pg.len + s) &&
      (at >> p.shift) < p.pg.M) {
    const int page = __ldg(p.pg.table + (size_t)s * p.pg.M + (at >> p.shift));
    if (page >= 0 && page < p.pg.P && __ldg(p.pg.refs + page) == 1)
      row = p.pg.rows + (((size_t)page << p.shift) + (at & (p.pg.page - 1))) *
                            (size_t)(D / 2 + D / 16);
  }
  if (row == nullptr && lane == 0) record_error(p.err, CSA2_ERR_DEVICE_INDEX);
  bool bad = false;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c0 = (lane + 32 * j) * 8;
    double amax = 0.0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      bad |= !isfinite(y[j][k]);
      amax = fmax(amax, fabs(y[j][k]));
    }
    amax = fmax(amax, __shfl_xor_sync(0xffffffffu, amax, 1));   // D % 128 == 0: pairs stay whole
    if (c0 >= D) continue;
    const uint32_t sc = e4m3_code64(amax / 6.0);
    const float sf = __low2float(e4m3x2_to_half2((uint16_t)sc));
    uint32_t word = 0;
    float val[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t c = e2m1_code64(y[j][k], (double)sf);
      word |= c << (4 * k);
      // magnitudes 0, 1/2, 1, 3/2, 2, 3, 4, 6
      const uint32_t m = c & 7u;
      const float mag = m < 4u ? 0.5f * m : (m < 6u ? (float)(m - 2u) : (m == 6u ? 4.0f : 6.0f));
      val[k] = (c & 8u) ? -mag * sf : mag * sf;
    }
    if (row) {
      *reinterpret_cast<uint32_t*>(row + c0 / 2) = word;
      if (!(lane & 1)) row[D / 2 + c0 / 16] = (uint8_t)sc;
    }
    if (a.kv_out)
      *reinterpret_cast<uint4*>(a.kv_out + (size_t)e * D + c0) = pack_bf16x8(val);
  }
  if (bad) record_error(p.err, CSA2_ERR_NONFINITE);
}

// Rotates the fp32 channels of a row held as chunks of four pairs (see the top of
// the file).
template <int J, int kPath>
__device__ __forceinline__ void rotate_row(const csa2_norm_rope_args& a, uint64_t (&y)[J][4],
                                           float* strip, const float* cs) {
  const int lane = threadIdx.x & 31;
  const int b = a.rot_begin, R = a.R;
  if (kPath == kInLane) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c0 = (lane + 32 * j) * 8 - b;          // in the rotary part; whole chunks
      if (c0 < 0 || c0 >= R) continue;
      const float4 t0 = *reinterpret_cast<const float4*>(cs + c0);
      const float4 t1 = *reinterpret_cast<const float4*>(cs + c0 + 4);
      const float c[4] = {t0.x, t0.z, t1.x, t1.z}, s[4] = {t0.y, t0.w, t1.y, t1.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 v = unpack2(y[j][k]);
        y[j][k] = pack2(v.x * c[k] - v.y * s[k], v.y * c[k] + v.x * s[k]);
      }
    }
  } else if (kPath == kPairs) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c0 = (lane + 32 * j) * 8 - b;          // in the rotary part; even
      if (c0 <= -8 || c0 >= R) continue;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (c0 + 2 * k < 0 || c0 + 2 * k >= R) continue;
        const float2 t = *reinterpret_cast<const float2*>(cs + c0 + 2 * k);
        const float2 v = unpack2(y[j][k]);
        y[j][k] = pack2(v.x * t.x - v.y * t.y, v.y * t.x + v.x * t.y);
      }
    }
  } else if (kPath == kExchange) {
    const int jr = b >> 8, first = (b >> 3) & 31, half = R >> 4;   // in chunks
#pragma unroll
    for (int j = 0; j < J; ++j) {
      if (j != jr) continue;                                       // the same for every lane
      const int i = lane - first;
      const bool mine = i >= 0 && i < 2 * half, low = i < half;
      const int other = mine ? (low ? lane + half : lane - half) : lane;
      const float* t = cs + (low ? i : i - half) * 16;             // pairs 8 i .. of (cos, sin)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint64_t o2 = __shfl_sync(0xffffffffu, y[j][k], other);
        if (mine) {
          const float2 v = unpack2(y[j][k]), o = unpack2(o2);
          const float4 f = *reinterpret_cast<const float4*>(t + 4 * k);
          const float s0 = low ? -f.y : f.y, s1 = low ? -f.w : f.w;
          y[j][k] = pack2(v.x * f.x + o.x * s0, v.y * f.z + o.y * s1);
        }
      }
    }
  } else if (kPath == kStrip) {
    float x[J][8];
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 v = unpack2(y[j][k]);
        x[j][2 * k] = v.x;
        x[j][2 * k + 1] = v.y;
      }
    rotate_strip<J>(a, x, strip, cs);
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) y[j][k] = pack2(x[j][2 * k], x[j][2 * k + 1]);
  }
}

// Whether a row's mean(x^2) + eps lies where fp32 squares may have overflowed, or lost
// bits below 2^-126 that count (NaN too).
__device__ __forceinline__ bool far_mean(float mean) {
  // outside [2^-100, 2^100], as bits
  return __float_as_uint(mean) - 0x0d800000u > 0x71800000u - 0x0d800000u;
}

// Such a row from its place in memory to its output: the row (and eps) times a power of
// two that takes the largest magnitude to [1, 2), or [1, 4) at the top of the range. A
// row with a NaN or an infinity, or of zeros with eps 0, is computed as it is. (In the
// loop over ordinary rows the same costs registers: 88 -> 96 us for 4096 tokens of 64
// heads. So these rows, which that loop has not written, come after it.)
template <int J, int kPath, bool kWide>
__device__ __forceinline__ void far_row(const csa2_norm_rope_args& a, const void* src,
                                        uint16_t* dst, float* strip, const float* cs) {
  const int lane = threadIdx.x & 31;
  float x[J][8];
  uint32_t bits = __float_as_uint(sqrtf(a.eps));       // (a NaN is larger than every number)
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c0 = (lane + 32 * j) * 8;
#pragma unroll
    for (int k = 0; k < 8; ++k) x[j][k] = 0.0f;
    if (c0 < a.D) load8(src, kWide, (size_t)c0, x[j]);
#pragma unroll
    for (int k = 0; k < 8; ++k) bits = max(bits, __float_as_uint(fabsf(x[j][k])));
  }
  bits = __reduce_max_sync(0xffffffffu, bits);
  const int e = (int)(bits >> 23) - 127;               // -127: zero or subnormal
  const float up = e == 128 ? 1.0f
                            : __uint_as_float((uint32_t)(127 - max(-126, min(e, 126))) << 23);
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x[j][k] *= up;
      sum = fmaf(x[j][k], x[j][k], sum);
    }
  const float f = rsqrtf(warp_sum(sum) / a.D + a.eps * up * up);
  uint64_t y[J][4];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c0 = (lane + 32 * j) * 8;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x[j][k] *= f;
      if (a.q_weight != nullptr && c0 < a.D) x[j][k] *= __ldg(a.q_weight + c0 + k);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) y[j][k] = pack2(x[j][2 * k], x[j][2 * k + 1]);
  }
  rotate_row<J, kPath>(a, y, strip, cs);
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c0 = (lane + 32 * j) * 8;
    if (c0 >= a.D) continue;
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 v = unpack2(y[j][k]);
      o[k] = pack_bf162(v.x, v.y);
    }
    *reinterpret_cast<uint4*>(dst + c0) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// The rows of this warp with a bit in `bits`, their places found again. (For wide rows: holding
// the places through the loop over ordinary rows spills there, 794 tokens of 64 heads of
// 1024 in halves 78 us instead of 74; for narrower ones finding them again does, 92 and 89.)
template <int J, int kPath, bool kWide>
__device__ __forceinline__ void far_rows(const NormRope& p, float* table, uint32_t bits) {
  const csa2_norm_rope_args& a = p.a;
  const int warp = (int)(threadIdx.x >> 5);
  const long long r0 = (long long)(blockIdx.x - p.entry_blocks) * p.rows_per_cta;
  const int t0 = (int)(r0 / a.Hq);
  float* strip = table + (size_t)p.tokens_per_cta * a.R + (size_t)warp * strip_at(a.D);
  for (; bits != 0; bits &= bits - 1) {
    const long long row = r0 + warp + (__ffs(bits) - 1) * kWarps;
    const int t = (int)(row / a.Hq), h = (int)(row - (long long)t * a.Hq);
    const size_t at = (size_t)t * a.q_stride + (size_t)h * a.D;
    far_row<J, kPath, kWide>(a, static_cast<const char*>(a.q) + at * (kWide ? 4 : 2),
                             a.q_out + row * a.D, strip, table + (t - t0) * a.R);
  }
}

// CTAs [0, entry_blocks) take entries, one per warp (they come first, being the
// longest chains); the others rows_per_cta (token, head) rows, warp w every 8th from w.
// 64 registers a thread where they suffice (neighbouring channels of 512 in bf16 spill 8
// bytes, which costs nothing measurable): 32 warps per SM, 2 KB each in flight.
// Elsewhere 80 and 24 warps (2000 tokens of 40 heads of 512 rotated in halves: 36 us,
// with 64 registers 42; neighbouring channels in whole chunks 32 and 33).
constexpr int min_ctas(int J, int path) { return J > 2 ? 2 : path <= kInLane ? 4 : 3; }
template <int J, int kPath, bool kWide>
__global__ void __launch_bounds__(kThreads, min_ctas(J, kPath))
norm_rope_kernel(const __grid_constant__ NormRope p) {
  // queries: (cos, sin) of the R/2 pairs of each token, then (kStrip) a strip per
  // warp; entries: per warp the same as doubles
  extern __shared__ double smem[];
  pdl_wait_and_release();
  const csa2_norm_rope_args& a = p.a;
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int D = a.D;
  if ((int)blockIdx.x < p.entry_blocks) {
    const int e = blockIdx.x * p.entries_per_cta + warp;
    if (warp >= p.entries_per_cta || e >= a.E) return;
    constexpr bool kStripped = kPath == kExchange || kPath == kStrip;
    double* cs = smem + (size_t)warp * (a.R + (kStripped ? strip_at(D) : 0));
    const int pos = __ldg(a.kv_pos + e);
    if (lane == 0 && pos < 0) record_error(p.err, CSA2_ERR_DEVICE_INDEX);
    for (int i = lane; i < a.R / 2; i += 32) {
      double s, c;
      // 2 pi frac: sincospi of twice the fraction
      sincospi((double)turn_fraction(pos, a.turns[i]) * 0x1p-63, &s, &c);
      cs[2 * i] = c * (double)a.rot_scale;
      cs[2 * i + 1] = (a.inverse ? -s : s) * (double)a.rot_scale;
    }
    __syncwarp();
    entry_row<J, kPath>(p, e, cs + a.R, cs);
    return;
  }
  __shared__ uint32_t far[kWarps];                     // rows left for the end, a bit each
  far[warp] = 0;
  __syncwarp();
  const int Hq = a.Hq;
  const long long r0 = (long long)(blockIdx.x - p.entry_blocks) * p.rows_per_cta;
  const int rows = (int)min((long long)p.rows_per_cta, (long long)a.T * Hq - r0);
  const int t0 = (int)(r0 / Hq), h0 = (int)(r0 - (long long)t0 * Hq);    // the first row's
  const int tokens = (h0 + rows - 1) / Hq + 1;
  float* table = reinterpret_cast<float*>(smem);
  float* strip = table + (size_t)p.tokens_per_cta * a.R + (size_t)warp * strip_at(D);
  constexpr int kRows = kWide ? 1 : J == 1 ? 4 : 2;    // rows of a warp in flight
  constexpr int kVecs = kWide ? 2 : 1;                 // 16-byte words of a chunk
  uint4 raw[kRows][J][kVecs];
  const float inv_d = 1.0f / D;
  const int esz = kWide ? 4 : 2;
  const size_t token_bytes = (size_t)a.q_stride * esz;
  const char* src = static_cast<const char*>(a.q) + (size_t)t0 * token_bytes + lane * 8 * esz;
  uint16_t* dst = a.q_out + r0 * D + lane * 8;
  // (token, head) of this warp's next row to load and to compute, kWarps rows apart
  int load_tok = (h0 + warp) / Hq, load_h = h0 + warp - load_tok * Hq;
  int tok[kRows];                                      // of the rows in flight
  auto next = [&](int& t, int& h) {
    t += p.step_tok;
    h += p.step_head;
    if (h >= Hq) {
      h -= Hq;
      ++t;
    }
  };
  auto load = [&](uint4 (&v)[J][kVecs], int row) -> int {
    const int t = load_tok;
    const char* at = src + (size_t)load_tok * token_bytes + (size_t)(load_h * D * esz);
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int k = 0; k < kVecs; ++k)
        v[j][k] = row < rows && (lane + 32 * j) * 8 < D
                      ? __ldcs(reinterpret_cast<const uint4*>(at + (256 * j + 4 * k) * esz))
                      : make_uint4(0, 0, 0, 0);
    next(load_tok, load_h);
    return t;
  };
#pragma unroll
  for (int r = 0; r < kRows; ++r) tok[r] = load(raw[r], warp + r * kWarps);
  uint64_t w[J][4];
  const bool weighted = a.q_norm && a.q_weight != nullptr;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c0 = (lane + 32 * j) * 8;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      w[j][k] = weighted && c0 < D ? pack2(__ldg(a.q_weight + c0 + 2 * k),
                                           __ldg(a.q_weight + c0 + 2 * k + 1))
                                   : pack2(1.0f, 1.0f);
  }
  if (kPath != kNone) {
    for (int i = threadIdx.x; i < tokens * (a.R / 2); i += kThreads) {
      const int k = i / (a.R / 2), pair = i - k * (a.R / 2);
      const int pos = __ldg(a.pos + t0 + k);
      if (pair == 0 && pos < 0) record_error(p.err, CSA2_ERR_DEVICE_INDEX);
      float s, c;
      sincospif((float)turn_fraction(pos, a.turns[pair]) * 0x1p-63f, &s, &c);
      table[2 * i] = c * a.rot_scale;
      table[2 * i + 1] = (a.inverse ? -s : s) * a.rot_scale;
    }
    __syncthreads();
  }
  for (int row = warp; row < rows;) {
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (row >= rows) break;                          // the same for every lane
      uint64_t y[J][4];
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if (kWide) {
#pragma unroll
          for (int k = 0; k < kVecs; ++k) {
            const uint4 v = raw[r][j][k];
            y[j][2 * k] = pack2(__uint_as_float(v.x), __uint_as_float(v.y));
            y[j][2 * k + 1] = pack2(__uint_as_float(v.z), __uint_as_float(v.w));
          }
        } else {
          const uint4 v = raw[r][j][0];
          const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            y[j][k] = pack2(__uint_as_float(x[k] << 16), __uint_as_float(x[k] & 0xffff0000u));
        }
      }
      const int t = tok[r];
      tok[r] = load(raw[r], row + kRows * kWarps);
      bool write = true;
      if (a.q_norm) {
        uint64_t s2 = 0;
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) s2 = fma2(y[j][k], y[j][k], s2);
        const float2 s = unpack2(s2);
        // (rsqrtf is within 2 ulp; the divide and the square root cost 40 instructions a row)
        const float mean = fmaf(warp_sum(s.x + s.y), inv_d, a.eps);
        write = !far_mean(mean);
        if (!write) far[threadIdx.x >> 5] |= 1u << (row / kWarps);   // (each lane the same)
        const float f = rsqrtf(mean);
        const uint64_t f2 = pack2(f, f);
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) y[j][k] = mul2(mul2(y[j][k], f2), w[j][k]);
      }
      rotate_row<J, kPath>(a, y, strip, table + t * a.R);
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if ((lane + 32 * j) * 8 >= D || !write) continue;
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 v = unpack2(y[j][k]);
          o[k] = pack_bf162(v.x, v.y);
        }
        __stcs(reinterpret_cast<uint4*>(dst + (size_t)row * D + 256 * j),
               make_uint4(o[0], o[1], o[2], o[3]));
      }
      row += kWarps;
    }
  }
  if (!a.q_norm) return;
  __syncwarp();
  uint32_t bits = far[threadIdx.x >> 5];
  if (J > 2) {
    if (bits != 0) far_rows<J, kPath, kWide>(p, table, bits);
    return;
  }
  for (; bits != 0; bits &= bits - 1) {
    const int row = warp + (__ffs(bits) - 1) * kWarps;
    const int t = (h0 + row) / Hq, h = h0 + row - t * Hq;
    far_row<J, kPath, kWide>(a, src - lane * 8 * esz + (size_t)t * token_bytes +
                                    (size_t)(h * D * esz),
                             dst - lane * 8 + (size_t)row * D, strip, table + t * a.R);
  }
}

template <int J, bool kWide>
cudaError_t launch_j(int path, const NormRope& p, unsigned grid, size_t smem,
                     cudaStream_t stream) {
  void (*kernel)(const NormRope) = path == kNone     ? norm_rope_kernel<J, kNone, kWide>
                                   : path == kInLane ? norm_rope_kernel<J, kInLane, kWide>
                                   : path == kPairs ? norm_rope_kernel<J, kPairs, kWide>
                                   : path == kExchange ? norm_rope_kernel<J, kExchange, kWide>
                                                       : norm_rope_kernel<J, kStrip, kWide>;
  return launch_pdl(kernel, dim3(grid), dim3(kThreads), smem, stream, dim3(1), p);
}

template <bool kWide>
cudaError_t launch_wide(int path, const NormRope& p, unsigned grid, size_t smem,
                        cudaStream_t stream) {
  switch (ceil_div(p.a.D, 256)) {
    case 1: return launch_j<1, kWide>(path, p, grid, smem, stream);
    case 2: return launch_j<2, kWide>(path, p, grid, smem, stream);
    case 3: return launch_j<3, kWide>(path, p, grid, smem, stream);
    default: return launch_j<4, kWide>(path, p, grid, smem, stream);
  }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const csa2_norm_rope_args& a, const fp4_kv_pages* pages, int* err,
                                cudaStream_t stream) {
  NormRope p;
  p.a = a;
  p.pg = pages ? *pages : fp4_kv_pages{};
  p.shift = 0;
  while (pages && (1 << p.shift) < pages->page) ++p.shift;
  p.err = err;
  int sms = 148, dev = 0;
  if (cudaGetDevice(&dev) == cudaSuccess)
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  int path = kStrip;
  if (a.R == 0) path = kNone;
  else if (a.interleaved && a.rot_begin % 2 == 0)
    path = a.rot_begin % 8 == 0 && a.R % 8 == 0 ? kInLane : kPairs;
  else if (!a.interleaved && a.R % 16 == 0 && a.rot_begin % 8 == 0 &&
           a.rot_begin / 256 == (a.rot_begin + a.R - 1) / 256)
    path = kExchange;
  // rows per CTA: few rows spread over the SMs, one per warp; many share the start and
  // the cosines, up to 64 of them (64 KB of bf16) while the tables and strips fit
  // and about a wave of CTAs is left (256 tokens of 64 heads: 512 CTAs of 32 rows 9.4 us,
  // 1024 of 16 rows 11, 2048 of 8 rows 16)
  const long long all = (long long)a.T * a.Hq;
  const long long words = kTableBytes / 4 - (path == kStrip ? kWarps * strip_at(a.D) : 0);
  auto tokens_of = [&](int rows) { return a.T > 0 ? (rows - 2 + a.Hq) / a.Hq + 1 : 0; };   // touched at most
  p.rows_per_cta = kWarps;
  while (p.rows_per_cta > 1 && (long long)tokens_of(p.rows_per_cta) * a.R > words)
    p.rows_per_cta /= 2;
  const int top = a.D >= 512 || a.q_f32 ? 64 : 64 * 512 / a.D;
  while (p.rows_per_cta < top && all / (2 * p.rows_per_cta) >= 3ll * sms &&
         (long long)tokens_of(2 * p.rows_per_cta) * a.R <= words)
    p.rows_per_cta *= 2;
  p.tokens_per_cta = tokens_of(p.rows_per_cta);
  if (p.tokens_per_cta > a.T) p.tokens_per_cta = a.T;
  p.step_tok = a.T > 0 ? kWarps / a.Hq : 0;
  p.step_head = a.T > 0 ? kWarps % a.Hq : 0;
  const long long query_blocks = (all + p.rows_per_cta - 1) / p.rows_per_cta;
  // entries: as many warps as the tables and strips allow (D = R = 1024: five in the lane,
  // two through the strip)
  const size_t per_entry =
      (a.R + (path == kExchange || path == kStrip ? strip_at(a.D) : 0)) * sizeof(double);
  p.entries_per_cta = per_entry * kWarps <= kTableBytes ? kWarps : (int)(kTableBytes / per_entry);
  // few entries: a CTA each, as their chains are what a small call waits for
  if (a.E <= sms) p.entries_per_cta = 1;
  p.entry_blocks = ceil_div(a.E, p.entries_per_cta);
  const long long grid = (long long)p.entry_blocks + query_blocks;
  if (grid == 0) return cudaSuccess;
  if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
  const size_t for_entries = a.E > 0 ? p.entries_per_cta * per_entry : 0;
  const size_t for_queries = ((size_t)p.tokens_per_cta * a.R +
                              (path == kStrip ? (size_t)kWarps * strip_at(a.D) : 0)) * sizeof(float);
  const size_t smem = for_entries > for_queries ? for_entries : for_queries;
  return a.T > 0 && a.q_f32 ? launch_wide<true>(path, p, (unsigned)grid, smem, stream)
                            : launch_wide<false>(path, p, (unsigned)grid, smem, stream);
}

}  // namespace csa2
