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
// chunks of 8 channels (lane + 32 j), read as 16-byte words; the rotary part goes
// through a per-warp strip of shared memory, so that either pair layout and any
// first channel work alike; the cosines and sines of a token are computed once
// per CTA and shared by its warps' heads. An entry's group of 16 channels is two
// neighbouring lanes: one exchange gives its maximum, the codes of a lane are one
// 32-bit word. Bound: HBM (a few dozen instructions per 16 bytes read and
// written); at single tokens, the launch.
#include "common.cuh"
#include "kernels.h"

namespace csa2 {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxD = 1024;

struct NormRope {
  csa2_norm_rope_args a;
  fp4_kv_pages pg;
  int shift;
  int q_blocks;      // CTAs per token's heads
  int heads_per_cta;
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

// The channels of the rotary part that pair i joins.
__device__ __forceinline__ void pair_of(const csa2_norm_rope_args& a, int i, int* u, int* v) {
  *u = a.interleaved ? 2 * i : i;
  *v = a.interleaved ? 2 * i + 1 : i + a.R / 2;
}

template <int J, typename F>
__device__ __forceinline__ F warp_sum(F x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Moves the rotary channels of a row held as chunks through `strip`: f64 or f32.
template <int J, typename F>
__device__ __forceinline__ void rotate(const csa2_norm_rope_args& a, F (&y)[J][8], F* strip,
                                       const F* cs) {
  const int lane = threadIdx.x & 31;
  const int b = a.rot_begin, R = a.R;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c0 = (lane + 32 * j) * 8;
    if (c0 < a.D && c0 + 8 > b && c0 < b + R) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (c0 + k >= b && c0 + k < b + R) strip[c0 + k - b] = y[j][k];
    }
  }
  __syncwarp();
  for (int i = lane; i < R / 2; i += 32) {
    int u, v;
    pair_of(a, i, &u, &v);
    const F x0 = strip[u], x1 = strip[v], c = cs[2 * i], s = cs[2 * i + 1];
    strip[u] = x0 * c - x1 * s;
    strip[v] = x1 * c + x0 * s;
  }
  __syncwarp();
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c0 = (lane + 32 * j) * 8;
    if (c0 < a.D && c0 + 8 > b && c0 < b + R) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (c0 + k >= b && c0 + k < b + R) y[j][k] = strip[c0 + k - b];
    }
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

template <int J>
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
    const double r = 1.0 / sqrt(warp_sum<J>(sum) / D + (double)a.eps);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c0 = (lane + 32 * j) * 8;
      if (c0 >= D) continue;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        y[j][k] *= a.kv_weight ? r * (double)__ldg(a.kv_weight + c0 + k) : r;
    }
  }
  if (a.R) rotate<J>(a, y, strip, cs);

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

template <int J>
__device__ void query_head(const NormRope& p, int t, int h, float* strip, const float* cs) {
  const csa2_norm_rope_args& a = p.a;
  const int lane = threadIdx.x & 31;
  const int D = a.D;
  float y[J][8];
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c0 = (lane + 32 * j) * 8;
#pragma unroll
    for (int k = 0; k < 8; ++k) y[j][k] = 0.0f;
    if (c0 < D) load8(a.q, a.q_f32 != 0, (size_t)t * a.q_stride + (size_t)h * D + c0, y[j]);
#pragma unroll
    for (int k = 0; k < 8; ++k) sum = fmaf(y[j][k], y[j][k], sum);
  }
  if (a.q_norm) {
    const float r = 1.0f / sqrtf(warp_sum<J>(sum) / D + a.eps);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c0 = (lane + 32 * j) * 8;
      if (c0 >= D) continue;
#pragma unroll
      for (int k = 0; k < 8; ++k) y[j][k] *= a.q_weight ? r * __ldg(a.q_weight + c0 + k) : r;
    }
  }
  if (a.R) rotate<J>(a, y, strip, cs);
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c0 = (lane + 32 * j) * 8;
    if (c0 < D)
      __stcs(reinterpret_cast<uint4*>(a.q_out + ((size_t)t * a.Hq + h) * D + c0),
             pack_bf16x8(y[j]));
  }
}

// CTAs [0, E) take an entry each (one warp works; they come first, being the
// longest chains), the others heads_per_cta heads of a token.
template <int J>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const NormRope p) {
  // cosines and sines of the R/2 pairs, then a strip of R channels per warp; an
  // entry uses the same bytes as doubles (one warp)
  extern __shared__ double smem[];
  pdl_wait_and_release();
  const csa2_norm_rope_args& a = p.a;
  const int warp = threadIdx.x >> 5;
  if ((int)blockIdx.x < a.E) {
    const int e = blockIdx.x;
    const int pos = __ldg(a.kv_pos + e);
    if (threadIdx.x == 0 && pos < 0) record_error(p.err, CSA2_ERR_DEVICE_INDEX);
    for (int i = threadIdx.x; i < a.R / 2; i += kThreads) {
      double s, c;
      // 2 pi frac: sincospi of twice the fraction
      sincospi((double)turn_fraction(pos, a.turns[i]) * 0x1p-63, &s, &c);
      smem[2 * i] = c * (double)a.rot_scale;
      smem[2 * i + 1] = (a.inverse ? -s : s) * (double)a.rot_scale;
    }
    __syncthreads();
    if (warp == 0) entry_row<J>(p, e, smem + a.R, smem);
    return;
  }
  const int blk = blockIdx.x - a.E;
  const int t = blk / p.q_blocks, h0 = (blk % p.q_blocks) * p.heads_per_cta;
  const int pos = __ldg(a.pos + t);
  if (threadIdx.x == 0 && pos < 0) record_error(p.err, CSA2_ERR_DEVICE_INDEX);
  float* cs = reinterpret_cast<float*>(smem);
  for (int i = threadIdx.x; i < a.R / 2; i += kThreads) {
    float s, c;
    sincospif((float)turn_fraction(pos, a.turns[i]) * 0x1p-63f, &s, &c);
    cs[2 * i] = c * a.rot_scale;
    cs[2 * i + 1] = (a.inverse ? -s : s) * a.rot_scale;
  }
  __syncthreads();
  float* strip = cs + a.R + warp * a.R;
  const int h1 = min(a.Hq, h0 + p.heads_per_cta);
  for (int h = h0 + warp; h < h1; h += kWarps) query_head<J>(p, t, h, strip, cs);
}

template <int J>
cudaError_t launch_j(const NormRope& p, unsigned grid, size_t smem, cudaStream_t stream) {
  return launch_pdl(norm_rope_kernel<J>, dim3(grid), dim3(kThreads), smem, stream, dim3(1), p);
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
  // heads of a token per CTA: few tokens spread over the SMs a warp per head;
  // many tokens share the cosines of a token among all of its heads
  p.heads_per_cta = kWarps;
  if ((long long)a.T * ceil_div(a.Hq > 0 ? a.Hq : 1, 4 * kWarps) >= 4ll * sms)
    p.heads_per_cta = 4 * kWarps;
  p.q_blocks = a.T > 0 ? ceil_div(a.Hq, p.heads_per_cta) : 0;
  const long long grid = (long long)a.E + (long long)a.T * p.q_blocks;
  if (grid == 0) return cudaSuccess;
  if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
  const size_t smem = 2 * (size_t)a.R * sizeof(double) > (1 + kWarps) * (size_t)a.R * sizeof(float)
                          ? 2 * (size_t)a.R * sizeof(double)
                          : (1 + kWarps) * (size_t)a.R * sizeof(float);
  switch (ceil_div(a.D, 256)) {
    case 1: return launch_j<1>(p, (unsigned)grid, smem, stream);
    case 2: return launch_j<2>(p, (unsigned)grid, smem, stream);
    case 3: return launch_j<3>(p, (unsigned)grid, smem, stream);
    default: return launch_j<4>(p, (unsigned)grid, smem, stream);
  }
}

}  // namespace csa2
