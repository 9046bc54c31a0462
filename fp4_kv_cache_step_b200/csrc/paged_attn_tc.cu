// paged_attn_tc.cu -- attention of a few query tokens over every visible entry of
// a paged FP4 cache (csa2_paged_attn without a list), on the 5th-generation
// tensor cores.
//
// One entry is key and value; all heads share it. The query rows of a sequence
// (its Tq tokens x Hq heads, contiguous) are taken in blocks of 64, the entries
// in tiles of 96:
//   S   = Q V^T    M = 64 rows, N = 96 entries, K = 512: Q is the A operand in
//                  tensor memory, V the K-major B operand;
//   O^T += V^T P^T M = 128 channels (four blocks of them), N = 64 rows, K = 96:
//                  V is the MN-major A operand, P the K-major B operand.
// Why these shapes (cycles per instruction of K = 16, measured on a B200 with
// operands in place): M = 64 costs as much as M = 128, and no instruction takes
// under 47: 47 at N = 64, 48.5 at N = 96, 65 at N = 128, 129 at N = 256. So O as
// M = 64, N = 256 would take 16 cycles per entry, O^T takes 12; S takes 16.2 at
// N = 96 (23.5 at N = 64). Two tiles of 96 entries x 512 channels of fp16 are
// 192 KB, all that shared memory holds: one is filled while the other is used.
// Tensor memory: O^T in columns 0-255 (all lanes); the query block's channels
// 0-255 in lanes 0-15 of each quadrant and 256-511 in lanes 16-31, columns
// 256-383; the two halves' partial logits in the same lanes, columns 384-479,
// added when they are read.
//
// Work is dealt out by tiles: the tiles of all (sequence, row block) pairs stand in
// one line that is cut into as many equal pieces as there are SMs, so a ragged
// batch keeps every SM busy. A pair that lies within one piece is written out;
// one that is cut leaves fp32 partials with their (maximum, sum), which
// paged_combine_kernel joins. A sequence without entries has one empty tile.
//
// Roles: warps 0-7 load codes and scales a tile ahead into registers, dequantise
// (exact in fp16: at most 6 significant bits) and fill the tile, 12 entries each;
// they also stage the query block. Warp 8 issues the MMAs. Warps 9-12 run the
// softmax: a thread has one row's 48 entries of a tile. The reference maximum is
// lazy (raised, with O^T's columns rescaled, only by a logit more than 8 above it
// in log2 units), so P stays below 2^8 in fp16. All sums are fp32. Every wait is
// bounded.
#include "common.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace csa2 {
namespace {

using namespace sm100;

constexpr int kD = kHeadDim;               // 512
constexpr int kRows = 64;                  // query rows of a block
constexpr int kT = 80;                     // entries of a tile
constexpr int kHalfT = kT / 2;
constexpr int kAtom = kT * 128;            // 80 entries x 64 channels of fp16
constexpr int kVTile = 8 * kAtom;
constexpr int kPTile = 2 * 8192;           // 64 rows x (64 + 16) entries of fp16, 128-byte rows
constexpr int kRowBytes = kD / 2 + kD / 16;     // 288
constexpr int kRawTile = kT * kRowBytes;
constexpr int kProducerWarps = 8;
constexpr int kPerWarp = kT / kProducerWarps;   // 10 entries of a tile per producer warp
constexpr int kMmaWarp = 8;
constexpr int kLoadWarp = 13;
constexpr int kThreads = 14 * 32;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemQ = 256, kTmemS = 384;
constexpr uint32_t kHalfLanes = 16u << 16;      // lanes 16-31 of a quadrant
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleSlack = 8.0f;

struct __align__(8) Bars {
  uint64_t q_ld, q_conv, q_full, q_free, o_full, s_full, s_free;
  uint64_t raw_full[2], raw_free[2], v_full[2], v_free[2], p_full;
};

struct Smem {
  Bars bar;
  uint32_t tmem_slot;
  int abort_flag;
  long long base;                   // tiles before the first sequence of this piece
  long long total;                  // tiles in all
  int first_b;
  uint32_t valid[4][3];             // bit i of a tile's 96: entry i is there
  float2 mlf[kRows];                // (reference maximum, row sum)
  float factor[kRows];              // rescaling of each row
  float qdown[kRows];               // the power of two each row was scaled up by, inverted
};

constexpr size_t kSmemBytes = 1024 + 2 * kVTile + kPTile + 2 * kRawTile + sizeof(Smem);
static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");

struct Params {
  const uint16_t* q;
  fp4_kv_pages pg;
  int shift;
  const int32_t* seq;
  const int32_t* nvalid;
  int B, Tq, Hq, nblk;
  float softmax_scale;
  uint16_t* out;
  float* lse;
  float* ws_o;        // [slot][64][512]
  float2* ws_ml;      // [slot][64]
  int4* ws_info;      // [B][nblk]: first and last piece, the first one's slot
  int* err;
};

// ---------------------------------------------------------------- small wrappers
__device__ __forceinline__ int swz(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)((sbo >> 4) & 0x3FFFu) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// kind::f16, F16 x F16 -> F32; A K-major (0) or M-major (1); B K-major.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int a_mn) {
  return (1u << 4) | ((uint32_t)a_mn << 15) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

// One lane of the (converged) warp, always the same one.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)::"memory");
  return r != 0;
}

__device__ __forceinline__ void sts128(uint32_t a, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
  return r;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(a));
  return r;
}

// 8 E2M1 codes (low nibble first) times one scale -> 16 bytes of fp16, exact
__device__ __forceinline__ uint4 dq8(uint32_t codes, __half2 scale) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&h[k]), scale);
    h[k] = *reinterpret_cast<const uint32_t*>(&r);
  }
  return make_uint4(h[0], h[1], h[2], h[3]);
}

// The sum of 8 columns of the two partial logits of a row: threads 0-15 read
// columns taddr .. + 7, threads 16-31 columns taddr + 40 .. + 47, of lanes 0-15
// and 16-31 of the quadrant.
__device__ __forceinline__ void tmem_ld_partials(uint32_t taddr, float* y) {
  uint32_t a[8], b[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x32bx2.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%16], %18;\n\t"
      "tcgen05.ld.sync.aligned.16x32bx2.x8.b32 {%8,%9,%10,%11,%12,%13,%14,%15}, [%17], %18;\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]),
        "=r"(a[7]), "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3]), "=r"(b[4]), "=r"(b[5]),
        "=r"(b[6]), "=r"(b[7])
      : "r"(taddr), "r"(taddr + kHalfLanes), "n"(kHalfT)
      : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = __uint_as_float(a[i]) + __uint_as_float(b[i]);
}
__device__ __forceinline__ void tmem_ld_partials16(uint32_t taddr, float* y) {
  uint32_t a[16], b[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x32bx2.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32], %34;\n\t"
      "tcgen05.ld.sync.aligned.16x32bx2.x16.b32 "
      "{%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33], %34;\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]),
        "=r"(a[7]), "=r"(a[8]), "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]),
        "=r"(a[14]), "=r"(a[15]), "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3]), "=r"(b[4]),
        "=r"(b[5]), "=r"(b[6]), "=r"(b[7]), "=r"(b[8]), "=r"(b[9]), "=r"(b[10]), "=r"(b[11]),
        "=r"(b[12]), "=r"(b[13]), "=r"(b[14]), "=r"(b[15])
      : "r"(taddr), "r"(taddr + kHalfLanes), "n"(kHalfT)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) y[i] = __uint_as_float(a[i]) + __uint_as_float(b[i]);
}

// mbar_wait without its sleeps: the hardware suspends the thread in try_wait
// (up to a microsecond at a time), and wakes it with the phase
__device__ __forceinline__ bool wait_hot(uint64_t* bar, uint32_t parity, volatile int* abort) {
  uint64_t t0 = 0;
  for (uint32_t it = 0;; ++it) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (done) return true;
    if ((it & 63u) == 63u) {
      if (t0 == 0) t0 = global_ns();
      if (*abort) return false;
      if (global_ns() - t0 > kWaitLimitNs) {
        *abort = 1;
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool wait_hot_warp(uint64_t* bar, uint32_t parity, volatile int* abort) {
  const bool ok = wait_hot(bar, parity, abort);
  return __all_sync(0xffffffffu, ok) != 0;
}

// Whether any of the softmax threads says so (also a barrier among them).
__device__ __forceinline__ bool softmax_any(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void softmax_sync() {
  asm volatile("barrier.cta.sync 1, 128;" ::: "memory");
}

// ---------------------------------------------------------------- lengths, pieces
// Visible entries of query (b, t): nvalid, or the slot's length.
__device__ int visible(const Params& p, int b, int t, bool tell) {
  const int s = p.seq ? __ldg(p.seq + b) : b;
  if (s < 0 || s >= p.pg.S) {
    if (tell) record_error(p.err, CSA2_ERR_DEVICE_INDEX);
    return 0;
  }
  const int len = min(max(0, __ldg(p.pg.len + s)), p.pg.M << p.shift);
  if (p.nvalid == nullptr) return len;
  const int n = __ldg(p.nvalid + (size_t)b * p.Tq + t);
  if (tell && (n < 0 || n > len)) record_error(p.err, CSA2_ERR_DEVICE_INDEX);
  return min(max(0, n), len);
}

__device__ int visible_most(const Params& p, int b, bool tell) {
  int n = 0;
  for (int t = 0; t < (p.nvalid ? p.Tq : 1); ++t) n = max(n, visible(p, b, t, tell));
  return n;
}

__device__ __forceinline__ int tiles_of(int n) { return max(1, (n + kT - 1) / kT); }

// Piece i of `pieces` holds the tiles [piece_begin(i), piece_begin(i + 1)) of `total`.
__device__ __forceinline__ long long piece_begin(int i, int pieces, long long total) {
  return (long long)i * total / pieces;
}
__device__ __forceinline__ int piece_of(long long tile, int pieces, long long total) {
  return (int)(((tile + 1) * pieces - 1) / total);
}

__global__ void __launch_bounds__(kThreads, 1) paged_attn_tc_kernel(const Params p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* vs = base;                          // [2][8 atoms][80 entries][128 B]
  uint8_t* ps = vs + 2 * kVTile;               // [2 atoms][64 rows][128 B]
  uint8_t* raw = ps + kPTile;                  // [2][80 entries][288 B]
  Smem& sm = *reinterpret_cast<Smem*>(raw + 2 * kRawTile);
  volatile int* abort_flag = &sm.abort_flag;
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(&sm.bar.q_ld, 1);
    mbar_init(&sm.bar.q_conv, kProducerWarps);
    mbar_init(&sm.bar.q_full, kProducerWarps);
    mbar_init(&sm.bar.q_free, kProducerWarps);
    mbar_init(&sm.bar.o_full, 1);
    mbar_init(&sm.bar.s_full, 1);
    mbar_init(&sm.bar.s_free, 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.bar.v_full[i], kProducerWarps);
      mbar_init(&sm.bar.v_free[i], 1);
      mbar_init(&sm.bar.raw_full[i], 1);
      mbar_init(&sm.bar.raw_free[i], kProducerWarps);
    }
    mbar_init(&sm.bar.p_full, 4);
    sm.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_alloc(&sm.tmem_slot, kTmemCols);
  pdl_wait_and_release();

  // ---- this CTA's piece: each thread adds up the tiles of a stretch of
  // sequences; the one whose stretch holds the piece's first tile finds its sequence
  {
    long long* sums = reinterpret_cast<long long*>(vs);
    const int each = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(p.B, (int)threadIdx.x * each), b1 = min(p.B, b0 + each);
    long long mine = 0;
    for (int b = b0; b < b1; ++b)
      mine += (long long)p.nblk * tiles_of(visible_most(p, b, blockIdx.x == 0));
    sums[threadIdx.x] = mine;
    __syncthreads();
    if (threadIdx.x < 32) {
      long long run = 0;
      for (int i = lane; i < kThreads; i += 32) {
        const long long x = sums[i];
        long long incl = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        sums[i] = run + incl - x;
        run += __shfl_sync(0xffffffffu, incl, 31);
      }
      if (lane == 0) sm.total = run;
    }
    __syncthreads();
    const long long total = sm.total;
    const int pieces = (int)min((long long)gridDim.x, total);
    const long long before = sums[threadIdx.x];
    const long long begin = piece_begin(min((int)blockIdx.x, pieces - 1), pieces, total);
    if (begin >= before && begin < before + mine) {
      long long at = before;
      int b = b0;
      for (;; ++b) {
        const long long k = (long long)p.nblk * tiles_of(visible_most(p, b, false));
        if (begin < at + k) break;
        at += k;
      }
      sm.first_b = b;
      sm.base = at;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_slot;
  const long long total = sm.total;
  const int pieces = (int)min((long long)gridDim.x, total);
  const int piece = blockIdx.x;
  long long pos = piece < pieces ? piece_begin(piece, pieces, total) : 0;
  const long long end = piece < pieces ? piece_begin(piece + 1, pieces, total) : 0;
  long long seq_base = sm.base;
  int b = sm.first_b;

  const uint32_t vs_s = smem_u32(vs), ps_s = smem_u32(ps);
  const int quad = warp & 3;
  const uint32_t lanes = (uint32_t)(quad * 32) << 16;
  uint32_t g0 = 0;                  // tiles of this CTA before the current segment
  const long long piece_first = pos;

  for (uint32_t sg = 0; pos < end; ++sg) {
    // ---- the next segment: tiles [t0, t1) of (b, blk)
    const int n_most = visible_most(p, b, false);
    const int tiles = tiles_of(n_most);
    const int blk = (int)((pos - seq_base) / tiles);
    const long long pair_base = seq_base + (long long)blk * tiles;
    const int t0 = (int)(pos - pair_base);
    const int nt = (int)min((long long)(tiles - t0), end - pos);
    const bool whole = nt == tiles;
    const int slot = 2 * piece + (pos == piece_first ? 0 : 1);
    const int r0 = blk * kRows;                            // first query row of the block
    const int nr = min(kRows, p.Tq * p.Hq - r0);
    const size_t row0 = (size_t)b * p.Tq * p.Hq + r0;
    const uint32_t sph = sg & 1;                           // phase of the per-segment barriers
    const int qbuf = (int)((g0 + 1) & 1);                  // the tile that holds the query block first
    if (threadIdx.x == 0) {
      if (t0 == 0) {
        const int first = piece, last = piece_of(pair_base + tiles - 1, pieces, total);
        p.ws_info[(size_t)b * p.nblk + blk] = make_int4(first, last, slot, 0);
      }
      const uint32_t qbytes = (uint32_t)nr * kD * 2;
      mbar_arrive_expect_tx(&sm.bar.q_ld, qbytes);
      bulk_load(vs + qbuf * kVTile, p.q + row0 * kD, qbytes, &sm.bar.q_ld);
    }
    float m_ref = -INFINITY, l = 0.0f;

    if (warp < kProducerWarps) {
      // ---------------------------------------------------------- load + dequantise
      // Lane 16 j + u takes channels 16u .. + 15 and 256 + 16u .. + 15 of entries
      // 10 w + 2 r + j of a tile, r = 0 .. 4: whole lines of two rows at a time.
      const int u = lane & 15, half = lane >> 4;
      // the query block: see sparse attention's staging; rows are converted in
      // place to fp16, scaled by a power of two per row (exact), then moved to
      // tensor memory, thread (row, channel half) of two warps per quadrant
      auto stage_q = [&]() {
        const uint32_t qsm = vs_s + (uint32_t)(qbuf * kVTile);
        bool ok = mbar_wait_warp(&sm.bar.q_ld, sph, abort_flag);
        if (ok) {
#pragma unroll 1
          for (int i0 = 0; i0 < 8; i0 += 2) {
            uint4 a[2], c[2];
            uint32_t amax[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const int hh = quad * 16 + (warp >> 2) * 8 + i0 + r;
              a[r] = c[r] = make_uint4(0, 0, 0, 0);
              if (hh < nr) {
                a[r] = lds128(qsm + hh * 1024 + 16 * lane);
                c[r] = lds128(qsm + hh * 1024 + 512 + 16 * lane);
              }
              const uint32_t m = __vmaxu2(
                  __vmaxu2(__vmaxu2(a[r].x & 0x7fff7fffu, a[r].y & 0x7fff7fffu),
                           __vmaxu2(a[r].z & 0x7fff7fffu, a[r].w & 0x7fff7fffu)),
                  __vmaxu2(__vmaxu2(c[r].x & 0x7fff7fffu, c[r].y & 0x7fff7fffu),
                           __vmaxu2(c[r].z & 0x7fff7fffu, c[r].w & 0x7fff7fffu)));
              amax[r] = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
            }
            __syncwarp();
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const int hh = quad * 16 + (warp >> 2) * 8 + i0 + r;
              if (hh >= nr) continue;
              int ex2 = 0;
              const uint32_t eb = (amax[r] >> 7) & 0xffu;
              if (amax[r] != 0u && eb != 0xffu) ex2 = min(100, max(-100, 15 - ((int)eb - 126)));
              const float up = __uint_as_float((uint32_t)(127 + ex2) << 23);
              const uint32_t w[8] = {a[r].x, a[r].y, a[r].z, a[r].w,
                                     c[r].x, c[r].y, c[r].z, c[r].w};
              uint32_t f[8];
#pragma unroll
              for (int k = 0; k < 8; ++k)
                f[k] = pack_half2(__uint_as_float(w[k] << 16) * up,
                                  __uint_as_float(w[k] & 0xffff0000u) * up);
              const uint32_t qr = qsm + hh * 1024;
              sts128(qr + ((lane ^ (hh & 7)) << 4), make_uint4(f[0], f[1], f[2], f[3]));
              sts128(qr + (((32 + lane) ^ (hh & 7)) << 4), make_uint4(f[4], f[5], f[6], f[7]));
              if (lane == 0) sm.qdown[hh] = __uint_as_float((uint32_t)(127 - ex2) << 23);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.bar.q_conv);
        ok = mbar_wait_warp(&sm.bar.q_conv, sph, abort_flag) && ok;
        const int h = quad * 16 + u;
#pragma unroll 1
        for (int i = 2 * (warp >> 2); i < 2 * (warp >> 2) + 2; ++i) {
          float pk[32];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (ok && h < nr)
              v = lds128(qsm + h * 1024 + (((32 * half + 8 * i + j) ^ (h & 7)) << 4));
            pk[4 * j] = __uint_as_float(v.x);
            pk[4 * j + 1] = __uint_as_float(v.y);
            pk[4 * j + 2] = __uint_as_float(v.z);
            pk[4 * j + 3] = __uint_as_float(v.w);
          }
          // lanes 0-15: channels 64 i .. + 63; lanes 16-31: 256 further
          tmem_st_32(tmem + lanes + kTmemQ + 32u * i, pk);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sm.bar.q_full);
          mbar_arrive(&sm.bar.q_free);
        }
      };

      stage_q();
      for (int t = 0; t < nt; ++t) {
        const uint32_t g = g0 + t;
        const int buf = (int)(g & 1);
        const uint32_t ph = (g >> 1) & 1;
        if (!wait_hot_warp(&sm.bar.raw_full[buf], ph, abort_flag)) break;
        if (!wait_hot_warp(&sm.bar.v_free[buf], ph ^ 1, abort_flag)) break;
        if (t == 1 && !wait_hot_warp(&sm.bar.q_free, sph, abort_flag)) break;
        const uint32_t tile = vs_s + (uint32_t)(buf * kVTile);
        const uint32_t rows = smem_u32(raw) + (uint32_t)(buf * kRawTile);
        const uint32_t* valid = sm.valid[g & 3];
#pragma unroll
        for (int r = 0; r < kPerWarp / 2; ++r) {
          const int e = warp * kPerWarp + 2 * r + half;
          const uint32_t row = rows + (uint32_t)(e * kRowBytes);
          uint2 c0 = lds64(row + 8 * u), c1 = lds64(row + 128 + 8 * u);
          uint32_t s0 = lds8(row + 256 + u), s1 = lds8(row + 272 + u);
          if (!(valid[e >> 5] >> (e & 31) & 1u)) {      // nothing was copied there
            c0 = c1 = make_uint2(0, 0);
            s0 = s1 = 0;
          }
          const __half2 f0 = e4m3x2_to_half2((uint16_t)(s0 * 0x0101u));
          const __half2 f1 = e4m3x2_to_half2((uint16_t)(s1 * 0x0101u));
          // channels 256 hh + 16 u: atom 4 hh + u / 4, 16-byte chunks 2 (u % 4), + 1
          const uint32_t a0 = tile + (uint32_t)((u >> 2) * kAtom), a1 = a0 + 4u * kAtom;
          // lanes u and u + 4 would meet in one bank group: every other four take
          // their two chunks in the other order
          const int odd = (u >> 2) & 1, c = (u & 3) * 2 + odd;
          sts128(a0 + swz(e, c), dq8(odd ? c0.y : c0.x, f0));
          sts128(a0 + swz(e, c ^ 1), dq8(odd ? c0.x : c0.y, f0));
          sts128(a1 + swz(e, c), dq8(odd ? c1.y : c1.x, f1));
          sts128(a1 + swz(e, c ^ 1), dq8(odd ? c1.x : c1.y, f1));
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sm.bar.v_full[buf]);
          mbar_arrive(&sm.bar.raw_free[buf]);
        }
      }
    } else if (warp == kLoadWarp) {
      // ---------------------------------------------------------- bulk copies
      // Lane i copies the rows of a tile that lie in its i-th page (a tile of 80
      // entries touches at most 11 pages of 8).
      const int s = p.seq ? __ldg(p.seq + b) : b;
      const int32_t* table = p.pg.table + (size_t)(n_most > 0 ? s : 0) * p.pg.M;
      // entries [lo, hi) of the sequence in lane i's page of tile t
      auto range = [&](int t, long long* lo, long long* hi) {
        const long long e0 = (long long)(t0 + t) * kT;
        const long long pg = (e0 >> p.shift) + lane;
        *lo = max(e0, pg << p.shift);
        *hi = max(*lo, min(min(e0 + kT, (long long)n_most), (pg + 1) << p.shift));
        return pg;
      };
      auto fetch = [&](int t) -> int {
        if (t >= nt) return -1;
        long long lo, hi;
        const long long pg = range(t, &lo, &hi);
        return hi > lo ? __ldg(table + pg) : -1;
      };
      int place = fetch(0);
      for (int t = 0; t < nt; ++t) {
        const uint32_t g = g0 + t;
        const int buf = (int)(g & 1);
        long long lo, hi;
        range(t, &lo, &hi);
        const int place_next = fetch(t + 1);
        if (hi > lo && (place < 0 || place >= p.pg.P)) {
          record_error(p.err, CSA2_ERR_DEVICE_INDEX);
          hi = lo;
        }
        const int count = (int)(hi - lo);
        const int at = count ? (int)(lo - (long long)(t0 + t) * kT) : 0;   // place in the tile
        uint32_t bits[3];
#pragma unroll
        for (int w = 0; w < 3; ++w) {
          const int x0 = min(32, max(0, at - 32 * w)), x1 = min(32, max(0, at + count - 32 * w));
          const uint32_t m = (x1 >= 32 ? ~0u : (1u << x1) - 1u) & ~(x0 >= 32 ? ~0u : (1u << x0) - 1u);
          bits[w] = __reduce_or_sync(0xffffffffu, count ? m : 0u);
        }
        if (!wait_hot_warp(&sm.bar.raw_free[buf], ((g >> 1) & 1) ^ 1, abort_flag)) break;
        if (lane == 0) {
#pragma unroll
          for (int w = 0; w < 3; ++w) sm.valid[g & 3][w] = bits[w];
          mbar_arrive_expect_tx(&sm.bar.raw_full[buf],
                                (uint32_t)(__popc(bits[0]) + __popc(bits[1]) + __popc(bits[2])) *
                                    kRowBytes);
        }
        __syncwarp();
        if (count)
          bulk_load(raw + buf * kRawTile + at * kRowBytes,
                    p.pg.rows + (((size_t)place << p.shift) + (size_t)(lo & (p.pg.page - 1))) * kRowBytes,
                    (uint32_t)count * kRowBytes, &sm.bar.raw_full[buf]);
        place = place_next;
      }
    } else if (warp == kMmaWarp) {
      // ---------------------------------------------------------- MMA issuer
      // The whole warp runs this with warp-uniform values and one elected lane
      // issues: descriptors then stay in uniform registers (from one divergent
      // thread an instruction took 65 to 80 cycles to issue, more than to run).
      const uint32_t id_s = idesc_f16(64, kT, 0);
      const uint32_t id_o = idesc_f16(128, kRows, 1);
      const uint64_t vk = desc_sw128(vs_s, 16, 1024);       // V as K-major B
      const uint64_t vm = desc_sw128(vs_s, kAtom, 1024);    // V as M-major A
      const uint64_t pk = desc_sw128(ps_s, 16, 1024);       // P as K-major B
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t gu = __shfl_sync(0xffffffffu, g0, 0);
      const int ntu = __shfl_sync(0xffffffffu, nt, 0);
      bool ok = wait_hot_warp(&sm.bar.q_full, sph, abort_flag);
      tc_fence_after();
      auto issue_s = [&](uint32_t buf) {
        tc_fence_after();
        const uint64_t v = vk + (uint64_t)((buf * kVTile) >> 4);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 16; ++k)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
              mma_ts(tm + hf * kHalfLanes + kTmemS, tm + hf * kHalfLanes + kTmemQ + 8u * k,
                     v + (uint64_t)(((4 * hf + (k >> 2)) * kAtom + (k & 3) * 32) >> 4), id_s,
                     k > 0 ? 1u : 0u);
          mma_commit(&sm.bar.s_full);
        }
        __syncwarp();
      };
      auto issue_pv = [&](uint32_t buf, uint32_t acc0) {
        tc_fence_after();
        const uint64_t v = vm + (uint64_t)((buf * kVTile) >> 4);
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int ks = 0; ks < kT / 16; ++ks)
              mma_ss(tm + 64u * j, v + (uint64_t)((2 * j * kAtom + ks * 2048) >> 4),
                     pk + (uint64_t)(((ks >> 2) * 8192 + (ks & 3) * 32) >> 4), id_o,
                     ks > 0 ? 1u : acc0);
          mma_commit(&sm.bar.v_free[buf]);
        }
        __syncwarp();
      };
      auto done = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_test_wait(bar, parity)) != 0;
      };
      // whichever is ready first: S of a tile (filled, and the logits before it
      // read) or O^T += of a tile (its P published)
      int next_s = 0, next_pv = 0;
      uint64_t t_last = 0;
      uint32_t spins = 0;
      while (ok && next_pv < ntu) {
        bool did = false;
        const uint32_t gs = gu + next_s, gp = gu + next_pv;
        if (next_s < ntu && done(&sm.bar.s_free, (gs & 1) ^ 1) &&
            done(&sm.bar.v_full[gs & 1], (gs >> 1) & 1)) {
          issue_s(gs & 1);
          ++next_s;
          did = true;
        }
        if (next_pv < next_s && done(&sm.bar.p_full, gp & 1)) {
          issue_pv(gp & 1, next_pv > 0 ? 1u : 0u);
          ++next_pv;
          did = true;
        }
        if (did) {
          spins = 0;
        } else {
          __nanosleep(20);
          if ((++spins & 63u) == 0u) {
            const uint64_t now = global_ns();
            if (spins == 64u) t_last = now;
            if (__any_sync(0xffffffffu, *abort_flag != 0 || now - t_last > kWaitLimitNs)) {
              *abort_flag = 1;
              ok = false;
            }
          }
        }
      }
      if (elect_one()) mma_commit(&sm.bar.o_full);
      __syncwarp();
      // nothing may be in flight when tensor memory is reused or released
      wait_hot_warp(&sm.bar.o_full, sph, abort_flag);
    } else {
      // ---------------------------------------------------------- softmax (warps 9-12)
      const int hl = lane & 15, ch = lane >> 4;
      const int h = quad * 16 + hl;
      bool ok = mbar_wait_warp(&sm.bar.q_full, sph, abort_flag);
      const bool real = h < nr;
      const float hs = ok && real ? p.softmax_scale * kLog2e * sm.qdown[h] : 0.0f;
      // entries that this row sees
      const int n_row = real ? (p.nvalid ? visible(p, b, (r0 + h) / p.Hq, false) : n_most) : n_most;
      for (int t = 0; t < nt; ++t) {
        const uint32_t g = g0 + t;
        const int buf = (int)(g & 1);
        ok = ok && wait_hot_warp(&sm.bar.v_full[buf], (g >> 1) & 1, abort_flag) &&
             wait_hot_warp(&sm.bar.s_full, g & 1, abort_flag);
        // every softmax warp takes part in the barriers below, or none does
        if (softmax_any(!ok)) break;
        tc_fence_after();
        // this thread's entries: 40 ch .. + 39 of the tile, masks of 32 and 8
        const int left = n_row - (t0 + t) * kT - kHalfT * ch;
        uint32_t m0, m1;
        {
          const uint32_t* v = sm.valid[g & 3];
          m0 = ch ? (v[1] >> 8) | (v[2] << 24) : v[0];
          m1 = (ch ? v[2] >> 8 : v[1]) & 0xffu;
          if (left < kHalfT) {
            m0 &= left <= 0 ? 0u : left >= 32 ? ~0u : (1u << left) - 1u;
            m1 &= left <= 32 ? 0u : (1u << (left - 32)) - 1u;
          }
        }
        const bool all = __all_sync(0xffffffffu, m0 == ~0u && m1 == 0xffu);
        float y[kHalfT];
        tmem_ld_partials16(tmem + lanes + kTmemS, y);
        tmem_ld_partials16(tmem + lanes + kTmemS + 16u, y + 16);
        tmem_ld_partials(tmem + lanes + kTmemS + 32u, y + 32);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.bar.s_free);
        float xmax = -INFINITY;
        if (all) {
#pragma unroll
          for (int j = 0; j < kHalfT; ++j) {
            y[j] *= hs;
            xmax = fmaxf(xmax, y[j]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < kHalfT; ++j) {
            const bool there = ((j < 32 ? m0 >> j : m1 >> (j - 32)) & 1u) != 0u;
            y[j] = there ? y[j] * hs : -INFINITY;
            xmax = fmaxf(xmax, y[j]);
          }
        }
        xmax = fmaxf(xmax, __shfl_xor_sync(0xffffffffu, xmax, 16));
        const bool raise = xmax > m_ref + kRescaleSlack;
        const bool had = m_ref != -INFINITY;
        float alpha = 1.0f;
        if (raise) {
          alpha = had ? fast_exp2(m_ref - xmax) : 1.0f;
          m_ref = xmax;
          l *= alpha;
        }
        // O^T's columns are rows of the query block, its lanes channels: a warp
        // rescales its lanes for all rows
        if (softmax_any(raise && had)) {
          if (ch == 0) sm.factor[h] = alpha;
          softmax_sync();
          ok = wait_hot_warp(&sm.bar.v_free[(g - 1) & 1], ((g - 1) >> 1) & 1, abort_flag);
          if (ok) {
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              float o[32];
              tmem_ld_32(tmem + lanes + 32u * c, o);
              const float* f = sm.factor + 32 * (c & 1);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] *= f[i];
              tmem_st_32(tmem + lanes + 32u * c, o);
            }
          }
        }
        const float mm = m_ref == -INFINITY ? 0.0f : m_ref;   // nothing seen yet: 2^-inf = 0
        uint32_t w[kHalfT / 2];
#pragma unroll
        for (int i = 0; i < kHalfT / 2; ++i) {
          const float p0 = fast_exp2(y[2 * i] - mm), p1 = fast_exp2(y[2 * i + 1] - mm);
          l += p0 + p1;
          w[i] = pack_half2(p0, p1);
        }
        // P is free once O^T += of the tile before is complete
        if (t > 0) ok = wait_hot_warp(&sm.bar.v_free[(g - 1) & 1], ((g - 1) >> 1) & 1, abort_flag);
#pragma unroll
        for (int k = 0; k < kHalfT / 8; ++k) {
          const int c = (kHalfT / 8) * ch + k;      // 16-byte chunk: entries 8 c .. + 7
          sts128(ps_s + (uint32_t)((c >> 3) * 8192 + swz(h, c & 7)),
                 make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]));
        }
        fence_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.bar.p_full);
      }
      const float l_tot = l + __shfl_xor_sync(0xffffffffu, l, 16);
      if (ch == 0) sm.mlf[h] = make_float2(l_tot > 0.0f ? m_ref : -INFINITY, l_tot);
    }

    // -------------------------------------------------------------- output
    bool have_o = false;
    if (warp != kMmaWarp && warp != kLoadWarp) have_o = mbar_wait_warp(&sm.bar.o_full, sph, abort_flag);
    tc_fence_before();
    __syncthreads();                  // O^T is final, the (maximum, sum) pairs are in place
    tc_fence_after();
    if (have_o) {
      // chunks of 32 columns (32 rows of one block of 128 channels): the
      // quadrant's softmax warp takes two, its producer warps three each
      const int cb = warp > kMmaWarp ? 0 : warp < 4 ? 2 : 5;
      const int ce = warp > kMmaWarp ? 2 : warp < 4 ? 5 : 8;
#pragma unroll 1
      for (int c = cb; c < ce; ++c) {
        float o[32];
        tmem_ld_32(tmem + lanes + 32u * c, o);
        const int d = 128 * (c >> 1) + quad * 32 + lane, h0 = 32 * (c & 1);
        if (whole) {
          uint16_t* dst = p.out + (row0 + h0) * kD + d;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            if (h0 + i >= nr) break;
            const float lt = sm.mlf[h0 + i].y;
            const __nv_bfloat16 x = __float2bfloat16_rn(lt > 0.0f ? o[i] / lt : 0.0f);
            dst[(size_t)i * kD] = *reinterpret_cast<const uint16_t*>(&x);
          }
        } else {
          float* dst = p.ws_o + ((size_t)slot * kRows + h0) * kD + d;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            if (h0 + i >= nr) break;
            dst[(size_t)i * kD] = sm.mlf[h0 + i].y > 0.0f ? o[i] : 0.0f;
          }
        }
      }
      if (warp > kMmaWarp && lane < 16) {
        const int h = quad * 16 + lane;
        const float2 ml = sm.mlf[h];
        if (h < nr) {
          if (!whole)
            p.ws_ml[(size_t)slot * kRows + h] = ml;
          else if (p.lse)
            p.lse[row0 + h] = ml.y > 0.0f ? (ml.x + log2f(ml.y)) * kLn2 : -INFINITY;
        }
      }
    }
    tc_fence_before();
    const bool stop = __syncthreads_or(*abort_flag) != 0;
    tc_fence_after();
    if (stop) break;
    g0 += (uint32_t)nt;
    pos += nt;
    if (pos == seq_base + (long long)p.nblk * tiles) {
      seq_base = pos;
      ++b;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (threadIdx.x == 0 && *abort_flag) record_error(p.err, CSA2_ERR_TIMEOUT);
}

// Joins the pieces of one query row: out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i.
__global__ void __launch_bounds__(128) paged_combine_kernel(const Params p) {
  pdl_wait_and_release();
  const int per_seq = p.Tq * p.Hq;
  const int r = blockIdx.x;                            // row of the sequence
  const size_t b = blockIdx.y;
  const int4 info = p.ws_info[b * p.nblk + r / kRows];
  const int first = info.x, last = info.y;
  if (first == last) return;
  const int h = r % kRows;
  auto slot_of = [&](int i) { return (size_t)(i == first ? info.z : 2 * i) * kRows + h; };
  float M = -INFINITY;
  for (int i = first; i <= last; ++i) M = fmaxf(M, p.ws_ml[slot_of(i)].x);
  float L = 0.0f;
  float4 acc = make_float4(0, 0, 0, 0);
  const int d = threadIdx.x * 4;
  if (M != -INFINITY) {
#pragma unroll 4
    for (int i = first; i <= last; ++i) {
      const float2 ml = p.ws_ml[slot_of(i)];
      const float4 v = *reinterpret_cast<const float4*>(p.ws_o + slot_of(i) * kD + d);
      const float w = exp2f(ml.x - M);                 // 0 for a piece that saw nothing
      L = fmaf(w, ml.y, L);
      acc.x = fmaf(w, v.x, acc.x);
      acc.y = fmaf(w, v.y, acc.y);
      acc.z = fmaf(w, v.z, acc.z);
      acc.w = fmaf(w, v.w, acc.w);
    }
  }
  const float inv = L > 0.0f ? 1.0f / L : 0.0f;
  const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
  const __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
  const size_t row = b * per_seq + r;
  *reinterpret_cast<uint2*>(p.out + row * kD + d) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  if (p.lse && threadIdx.x == 0) p.lse[row] = L > 0.0f ? (M + log2f(L)) * kLn2 : -INFINITY;
}

int sm_count_of_device() {
  int dev = 0, n = 148;
  if (cudaGetDevice(&dev) == cudaSuccess)
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n;
}

// Pieces of the line of tiles: one per SM, never more than there can be tiles.
int most_pieces(const fp4_kv_pages& pg, int B, int nblk) {
  const long long tiles = ((long long)pg.M * pg.page + kT - 1) / kT;
  const long long all = tiles * B * nblk;
  const int sms = sm_count_of_device();
  return (int)(all < sms ? all : sms);
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

size_t paged_attn_dense_workspace_bytes(const fp4_kv_pages& pg, int B, int Tq, int Hq) {
  const int nblk = ceil_div(Tq * Hq, kRows);
  const size_t slots = 2 * (size_t)most_pieces(pg, B, nblk);
  return up256((size_t)B * nblk * sizeof(int4)) + up256(slots * kRows * sizeof(float2)) +
         slots * kRows * kD * sizeof(float);
}

cudaError_t launch_paged_attn_dense(const uint16_t* q, const fp4_kv_pages& pg, const int32_t* seq,
                                    const int32_t* nvalid, int B, int Tq, int Hq,
                                    float softmax_scale, uint16_t* out, float* lse,
                                    void* workspace, int* err, cudaStream_t stream) {
  Params p;
  p.q = q;
  p.pg = pg;
  p.shift = 0;
  while ((1 << p.shift) < pg.page) ++p.shift;
  p.seq = seq;
  p.nvalid = nvalid;
  p.B = B;
  p.Tq = Tq;
  p.Hq = Hq;
  p.nblk = ceil_div(Tq * Hq, kRows);
  p.softmax_scale = softmax_scale;
  p.out = out;
  p.lse = lse;
  const int pieces = most_pieces(pg, B, p.nblk);
  unsigned char* w = static_cast<unsigned char*>(workspace);
  p.ws_info = reinterpret_cast<int4*>(w);
  w += up256((size_t)B * p.nblk * sizeof(int4));
  p.ws_ml = reinterpret_cast<float2*>(w);
  w += up256(2 * (size_t)pieces * kRows * sizeof(float2));
  p.ws_o = reinterpret_cast<float*>(w);
  p.err = err;
  cudaError_t e = cudaFuncSetAttribute(paged_attn_tc_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)kSmemBytes);
  if (e != cudaSuccess) return e;
  e = launch_pdl(paged_attn_tc_kernel, dim3(pieces), dim3(kThreads), kSmemBytes, stream, dim3(1),
                 p);
  if (e != cudaSuccess) return e;
  return launch_pdl(paged_combine_kernel, dim3(Tq * Hq, B), dim3(128), 0, stream, dim3(1), p);
}

}  // namespace csa2
