// paged_attn_tc.cu -- attention of a few query tokens over a paged FP4 cache
// (csa2_paged_attn), every visible entry or a list of them, on the 5th-generation
// tensor cores.
//
// One entry is key and value; all heads share it. The query rows of a sequence
// (its Tq tokens x Hq heads, contiguous) are taken in blocks of 64, the entries
// in tiles of 80:
//   S  = Q V^T   M = 64 rows, N = 80 entries, K = 512: Q is the A operand in
//                tensor memory, V the K-major B operand;
//   O += P V     M = 64 rows, N = 256 channels twice, K = 80: P is the K-major A
//                operand, V the N-major B operand.
// Tensor memory: lanes 0-15 of each quadrant hold two S buffers (columns 0-159)
// and the query block (256-511), lanes 16-31 hold O (512 columns).
//
// Work is dealt out by tiles: the tiles of all (sequence, row block) pairs stand in
// one line that is cut into as many equal pieces as there are SMs, so a ragged
// batch keeps every SM busy. (Before each pair's tiles the line has kSetup units of
// nothing, what a further pair costs a piece: its query block and its output take
// as long as four tiles. Without them, pieces with two pairs ended 10 us after
// the others, of 24 us.) Where the pairs are short, the pieces are whole pairs. A
// pair that lies within one piece is written out; one that is cut leaves fp16
// partials with their (maximum, sum), which paged_combine_kernel joins. A sequence
// without entries has one empty tile.
//
// What a piece has of a pair is taken in segments of kMostTiles tiles at most, whose
// sums are joined in fp32 (the carry). A sum in tensor memory loses about a last place
// (2^-23) at every step of 16 entries, always towards zero, measured: beside a few
// entries far above a long tail that was 0.5 % of the output at 2^20 entries, and is
// 2^-11 at most with 64000. (148 row blocks over 2^20 entries: 20.3 ms with and without.)
//
// With lists each query token is a sequence of its own here, its list the entries
// (a place without an id takes its turn as an entry that is not there).
//
// Roles. Warp 15 copies rows (288 bytes each, contiguous within a page) to shared
// memory, two tiles ahead: bulk copies of a page's part of a tile, or with lists
// 16-byte copies, 18 to a row (a bulk copy of one row costs about 58 cycles to
// issue, 80 of them more than a tile's products). Warps 0-9 dequantise them (exact
// in fp16: at most 6 significant bits) into the tile, channels 0-255 first; 0-7 also
// stage the query block. Warp 14 issues the MMAs, two tiles at a time: S S PV PV, so
// that the softmax of one tile runs beside S of the next, and a tile is filled again
// while the other is multiplied. Warps 10-13 run the softmax, a thread having half
// of one row's entries. The reference maximum is lazy (raised, with O rescaled, only
// by a logit more than 8 above it in log2 units). P is 2^7 times the exponential, to use
// fp16's whole range: below 2^15, with 2^-24 (its least step) 2^-31 of the reference.
// What rounds to 0 of a segment's entries is then at most 2^-16 of the row sum (without
// the factor 2^-9). All sums are fp32.
// Warps hand work to each other through named barriers, which cost tens of cycles
// where a waiting mbarrier's wake-up beside this shared-memory load cost 500 to
// 800; what the tensor core or the copy engine signals are mbarriers, every wait
// on one of which is bounded. Named barriers need no bound: each role passes every
// one of them for every tile, whether or not a wait before it ran out.
//
// What bounds it: the tensor core. An instruction of M = 64, K = 16 takes 47 cycles
// at N = 80 (and at any N up to 96: the least there is) and 129 at N = 256, so a tile
// costs 32 x 47 + 10 x 129 = 2794 cycles; measured 2865 (ncu: the tensor pipe active
// 72 to 79 % of the kernel on 32 sequences of 16384 to 32768 entries, 64 heads, 138 to
// 140 us).
// M = 64 leaves half of the array idle; 128 rows of O would be all of tensor memory.
// Larger tiles would cost less per entry (96 entries: 32.3 cycles instead of 35), but
// two of them leave no room for the rows to come. Shared memory is the next bound:
// about 32 cycles per entry for filling a tile, reading it twice and staging rows.
// Before and after its tiles a CTA spends about 10 us (plan 2.7, query block and
// first tile 3.5, output 2.3).
#include <mutex>

#include "common.cuh"
#include "kernels.h"
#include "paged_join.h"
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
constexpr int kP0 = 64 * 128;              // P, entries 0-63: rows of 128 bytes
constexpr int kP1 = 64 * 32;               // P, entries 64-79: rows of 32 bytes
constexpr int kRowBytes = kD / 2 + kD / 16;     // 288
constexpr int kRawTile = kT * kRowBytes;
constexpr int kProducerWarps = 10;         // 8 entries of a tile each
constexpr int kMmaWarp = 14;
constexpr int kLoadWarp = 15;
constexpr int kThreads = 16 * 32;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemQ = 256;
constexpr uint32_t kHalfLanes = 16u << 16;      // lanes 16-31 of a quadrant
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleSlack = 8.0f;
constexpr float kLift = 7.0f;              // log2 of the factor in P
constexpr int kMostTiles = 800;            // tiles of a segment at most

// Named barriers (0 is __syncthreads): who arrives -> who waits; all but the first
// two once per tile, each role passing all of its own in order, so that none is
// passed twice before its other side came by.
enum : int {
  kBarQ = 1,          // producers -> MMA, softmax: the query block is in tensor memory
  kBarProducers = 2,  // among the producers
  kBarP = 3,          // + buffer: softmax -> MMA: P is there
  kBarL = 5,          // + buffer: loader -> producers: the copies are issued
  kBarV = 7,          // + 2 buffer + half: producers -> MMA (and, second half, loader): filled
  kBarS = 11,         // + buffer: MMA -> softmax: S of the tile is issued
};
constexpr int kProducers = kProducerWarps * 32, kSoftmax = 4 * 32;
constexpr int kNumQ = kProducers + 32 + kSoftmax, kNumP = kSoftmax + 32, kNumL = kProducers + 32;
constexpr int kNumV0 = kProducers + 32, kNumV1 = kProducers + 64;
constexpr int kNumS = kSoftmax + 32;
constexpr int kSetup = 4;           // units of the line of tiles before each pair

struct __align__(8) Bars {
  uint64_t q_ld, o_full, s_full[2], raw_full[2], v_free[2][2];   // v_free: [tile][half]
};

// A segment of a CTA's piece: tiles [t0, t0 + nt) of row block blk of sequence b.
// (In shared memory, so that no role holds it in registers through its loop.)
struct Segment {
  int b, blk, t0, nt;        // nt 0: there is none
  int carry, more;           // sums of the pair's tiles before are in the carry; tiles are left
  int n_most;                // entries that the sequence's queries see at most
  int tiles;
  int slot;                  // where its partial goes, -1: it is whole
  uint32_t g0, used0, used1; // tiles of this CTA before it, in all and by buffer
};

struct __align__(16) Smem {
  Bars bar;
  Segment seg[2];
  uint32_t tmem_slot;
  int abort_flag;
  long long total;                  // units of the line
  long long pos, end;               // this piece's units not yet in a segment
  long long end_pair;               // pairs from this one on are not this piece's
  long long base;                   // units before the sequence that pos lies in
  int most[kThreads / 32];          // units of the longest pair, by warp
  int whole;                        // pairs are dealt out whole
  uint4 valid[4];                   // bit i of a tile's 128: entry i is there
  float2 mlf[kRows];                // (reference maximum, row sum)
  float qdown[kRows];               // the power of two each row was scaled up by, inverted
};

constexpr size_t kSmemBytes = 2 * kVTile + 2 * (kP0 + kP1) + 2 * kRawTile + sizeof(Smem);
static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");

struct Params {
  const uint16_t* q;
  fp4_kv_pages pg;
  int shift;
  long long share;     // pairs that a piece has at most if they are dealt out whole
  const int32_t* seq;
  const int32_t* nvalid;
  const int32_t* ids;  // [B][K], or null for every entry
  int K;
  int B, Tq, Hq, nblk; // with lists B counts query tokens, and Tq is 1
  int per_slot;        // query tokens to an entry of seq (with lists; else 1)
  float softmax_scale;
  uint16_t* out;
  float* lse;
  __half* ws_o;       // [slot][64][512]: partial outputs, each over its own row sum
  float2* ws_ml;      // [slot][64]
  int4* ws_info;      // [B][nblk]: first and last piece, the first one's slot
  float* ws_carry;    // [piece][64][512]: sums of the segments before, null where none has more
  float2* ws_carry_ml;      // [piece][64]: their reference and row sum
  int pieces;         // of the line of tiles: ws_o and ws_ml have two slots each
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

// the same for rows of 32 bytes with the 32-byte swizzle (16-byte chunk c of row r
// at chunk c ^ (r >> 2 & 1)), 8-row groups of 256 bytes
__device__ __forceinline__ uint64_t desc_sw32(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)1 << 16 | (uint64_t)(256 >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)6 << 61;
}

// kind::f16, F16 x F16 -> F32; A K-major; B K-major (0) or N-major (1).
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int b_mn) {
  return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) |
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

__device__ __forceinline__ uint32_t pack_bf162(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t r;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(a));
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

// 40 columns of a row: threads 0-15 read columns taddr .. + 39 of lanes 0-15,
// threads 16-31 columns taddr + 40 .. + 79.
__device__ __forceinline__ void tmem_ld_logits(uint32_t taddr, float (&y)[kHalfT]) {
  uint32_t a[kHalfT];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x32bx2.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%40], 40;\n\t"
      "tcgen05.ld.sync.aligned.16x32bx2.x8.b32 {%32,%33,%34,%35,%36,%37,%38,%39}, [%41], 40;\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]),
        "=r"(a[7]), "=r"(a[8]), "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]),
        "=r"(a[14]), "=r"(a[15]), "=r"(a[16]), "=r"(a[17]), "=r"(a[18]), "=r"(a[19]),
        "=r"(a[20]), "=r"(a[21]), "=r"(a[22]), "=r"(a[23]), "=r"(a[24]), "=r"(a[25]),
        "=r"(a[26]), "=r"(a[27]), "=r"(a[28]), "=r"(a[29]), "=r"(a[30]), "=r"(a[31]),
        "=r"(a[32]), "=r"(a[33]), "=r"(a[34]), "=r"(a[35]), "=r"(a[36]), "=r"(a[37]),
        "=r"(a[38]), "=r"(a[39])
      : "r"(taddr), "r"(taddr + 32u)
      : "memory");
#pragma unroll
  for (int i = 0; i < kHalfT; ++i) y[i] = __uint_as_float(a[i]);
}
static_assert(kHalfT == 40, "the loads above");

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

__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void bar_arrive(int id, int threads) {
  asm volatile("barrier.cta.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// ((a - m) s + kLift, (b - m) s + kLift), two values to an instruction
__device__ __forceinline__ float2 lifted_difference(float a, float b, float m, float s) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%2, %3};\n\t"
      "mov.b64 y, {%4, %4};\n\t"
      "add.rn.f32x2 x, x, y;\n\t"
      "mov.b64 y, {%5, %5};\n\t"
      "mov.b64 z, {%6, %6};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\t"
      "mov.b64 {%0, %1}, x;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a), "f"(b), "f"(-m), "f"(s), "f"(kLift));
  return r;
}

// ---------------------------------------------------------------- lengths, pieces
__device__ __forceinline__ int slot_of(const Params& p, int b) {
  return p.seq ? __ldg(p.seq + b / p.per_slot) : b / p.per_slot;
}

// Entries that b's slot holds (0 for a bad slot).
__device__ __forceinline__ int slot_len(const Params& p, int b, bool tell) {
  const int s = slot_of(p, b);
  if (s < 0 || s >= p.pg.S) {
    if (tell) record_error(p.err, CSA2_ERR_DEVICE_INDEX);
    return 0;
  }
  return min(max(0, __ldg(p.pg.len + s)), p.pg.M << p.shift);
}

// Entries that query (b, t) sees: nvalid within [0, len], or len.
__device__ int visible(const Params& p, int b, int t) {
  const int len = slot_len(p, b, false);
  return p.nvalid ? min(max(0, __ldg(p.nvalid + (size_t)b * p.Tq + t)), len) : len;
}

// ... that b's queries see at most.
__device__ int visible_most(const Params& p, int b, bool tell) {
  int lo = 0, hi = 0;
  if (p.nvalid) {
    const int32_t* n = p.nvalid + (size_t)b * p.Tq;
    lo = hi = __ldg(n);
#pragma unroll 4
    for (int t = 1; t < p.Tq; ++t) {
      const int x = __ldg(n + t);
      lo = min(lo, x);
      hi = max(hi, x);
    }
  }
  const int len = slot_len(p, b, tell);
  if (!p.nvalid) return len;
  if (tell && (lo < 0 || hi > len)) record_error(p.err, CSA2_ERR_DEVICE_INDEX);
  return min(max(0, hi), len);
}

// Entries to go through for b: those its queries see at most, or its list's places.
template <bool kListed>
__device__ __forceinline__ int entries_of(const Params& p, int b, bool tell) {
  return kListed ? p.K : visible_most(p, b, tell);
}

__device__ __forceinline__ int tiles_of(int n) { return max(1, (n + kT - 1) / kT); }

// a / b for a >= 0, b > 0 (the 32-bit division is several times shorter)
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}
// Units of a sequence's (row block) pairs, and of one of them.
__device__ __forceinline__ int pair_units(int n) { return kSetup + tiles_of(n); }
// Piece i of `pieces` holds the units [piece_begin(i), piece_begin(i + 1)) of `total`.
__device__ __forceinline__ long long piece_begin(int i, int pieces, long long total) {
  return quotient((long long)i * total, pieces);
}
__device__ __forceinline__ int piece_of(long long unit, int pieces, long long total) {
  return (int)quotient((unit + 1) * pieces - 1, total);
}

// Cuts the next segment off the piece: sm.seg[at] from its predecessor
// sm.seg[at ^ 1] (whose b, or the one after it, is the sequence at sm.pos). One
// thread. n_most: the sequence's visible entries where they are known, else -1.
template <bool kListed>
__device__ __noinline__ void next_segment(const Params& p, Smem& sm, int at, int n_most) {
  const Segment& prev = sm.seg[at ^ 1];
  Segment s;
  s.g0 = prev.g0 + (uint32_t)prev.nt;
  s.used0 = prev.used0 + (uint32_t)(prev.nt + 1) / 2;
  s.used1 = prev.used1 + (uint32_t)prev.nt / 2;
  s.b = prev.b;
  s.nt = 0;
  s.blk = s.t0 = s.n_most = s.tiles = s.slot = s.more = 0;
  s.carry = prev.nt > 0 && prev.more;                    // the same pair goes on
  long long pos = sm.pos;
  const long long last_pair = sm.end_pair - 1;
  if (pos < sm.end) {
    if (prev.nt > 0 && pos == sm.base + (long long)p.nblk * (kSetup + prev.tiles)) {
      sm.base = pos;
      ++s.b;
    }
    if ((long long)s.b * p.nblk > last_pair) {           // whole pairs, and they are done
      sm.pos = sm.end;
      sm.seg[at] = s;
      return;
    }
    const int pieces = (int)min((long long)gridDim.x, sm.total), piece = (int)blockIdx.x;
    s.n_most = s.carry ? prev.n_most : n_most >= 0 ? n_most : entries_of<kListed>(p, s.b, false);
    s.tiles = tiles_of(s.n_most);
    const int units = kSetup + s.tiles;
    s.blk = (int)quotient(pos - sm.base, units);
    const long long first = sm.base + (long long)s.blk * units + kSetup;   // the pair's first tile
    pos = max(pos, first);
    s.t0 = (int)(pos - first);
    // the piece's tiles of the pair from here on
    const int part = (long long)s.b * p.nblk + s.blk > last_pair
                         ? 0 : (int)max(0ll, min((long long)(s.tiles - s.t0), sm.end - pos));
    s.nt = p.ws_carry ? min(part, kMostTiles) : part;
    s.more = part > s.nt;
    if (s.carry) {
      s.slot = prev.slot;
    } else if (s.nt > 0) {
      const int slot = 2 * piece + (prev.nt > 0 ? 1 : 0);
      s.slot = part == s.tiles ? -1 : slot;
      if (s.t0 == 0)
        p.ws_info[(size_t)s.b * p.nblk + s.blk] =
            make_int4(piece, part == s.tiles ? piece : piece_of(first + s.tiles - 1, pieces, sm.total),
                      slot, 0);
    }
    sm.pos = s.nt > 0 ? pos + s.nt : sm.end;
  }
  sm.seg[at] = s;
}

template <bool kListed>
__global__ void __launch_bounds__(kThreads, 1) paged_attn_tc_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(1024) uint8_t vs[];   // [2][8 atoms][80 entries][128 B]
  uint8_t* ps = vs + 2 * kVTile;               // [2][64 rows][128 B], [2][64 rows][32 B]
  uint8_t* raw = ps + 2 * (kP0 + kP1);         // [2][80 entries][288 B]
  Smem& sm = *reinterpret_cast<Smem*>(raw + 2 * kRawTile);
  volatile int* abort_flag = &sm.abort_flag;
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(&sm.bar.q_ld, 1);
    mbar_init(&sm.bar.o_full, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.bar.s_full[i], 1);
      mbar_init(&sm.bar.raw_full[i], kListed ? 32 : 1);
      mbar_init(&sm.bar.v_free[i][0], 1);
      mbar_init(&sm.bar.v_free[i][1], 1);
    }
    sm.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_alloc(&sm.tmem_slot, kTmemCols);
  pdl_wait_and_release();

  // ---- this CTA's piece: each thread adds up the units of a stretch of
  // sequences; the one whose stretch holds the piece's first unit finds its sequence
  {
    long long* sums = reinterpret_cast<long long*>(vs);
    const int each = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(p.B, (int)threadIdx.x * each), b1 = min(p.B, b0 + each);
    long long mine = 0;
    int n_last = 0, most = 0;                            // units of the longest pair
    for (int b = b0; b < b1; ++b) {
      n_last = entries_of<kListed>(p, b, blockIdx.x == 0);
      mine += (long long)p.nblk * pair_units(n_last);
      most = max(most, pair_units(n_last));
    }
    sums[threadIdx.x] = mine;
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) sm.most[warp] = most;
    __syncthreads();
    if (threadIdx.x < 32) {
      long long run = 0;
      for (int i = lane; i - lane < (p.B + each - 1) / each; i += 32) {
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
      // Short pairs are better dealt out whole than cut: the longest such share against
      // an even piece, one of whose pairs is cut (its query block is read again).
      // 36 sequences of 3 to 169 entries with 256 rows: 21 us whole, 28 cut.
      most = __reduce_max_sync(0xffffffffu, lane < kThreads / 32 ? sm.most[lane] : 0);
      if (lane == 0) {
        sm.total = run;
        const long long pieces = min((long long)gridDim.x, run);
        sm.whole = p.share * most * pieces <= run + kSetup * pieces;
      }
    }
    __syncthreads();
    const long long total = sm.total;
    const int pieces = (int)min((long long)gridDim.x, total);
    const long long before = sums[threadIdx.x];
    const long long pairs = (long long)p.B * p.nblk;
    if (sm.whole) {
      const long long j0 = quotient(blockIdx.x * pairs, gridDim.x);
      const int b = (int)quotient(j0, p.nblk);
      if (b >= b0 && b < b1) {
        long long at = before;
        for (int k = b0; k < b; ++k)
          at += (long long)p.nblk * pair_units(entries_of<kListed>(p, k, false));
        const int n = each == 1 ? n_last : entries_of<kListed>(p, b, false);
        sm.seg[1].b = b;
        sm.base = at;
        sm.seg[1].nt = 0;
        sm.seg[1].g0 = sm.seg[1].used0 = sm.seg[1].used1 = 0;
        sm.pos = at + (j0 - (long long)b * p.nblk) * pair_units(n);
        sm.end = total;
        sm.end_pair = quotient((blockIdx.x + 1) * pairs, gridDim.x);
        next_segment<kListed>(p, sm, 0, n);
      }
    } else {
      const long long begin = piece_begin(min((int)blockIdx.x, pieces - 1), pieces, total);
      if (begin >= before && begin < before + mine) {
        long long at = before;
        int b = b0;
        for (; b + 1 < b1; ++b) {
          const long long k = (long long)p.nblk * pair_units(entries_of<kListed>(p, b, false));
          if (begin < at + k) break;
          at += k;
        }
        sm.seg[1].b = b;
        sm.base = at;
        sm.seg[1].nt = 0;
        sm.seg[1].g0 = sm.seg[1].used0 = sm.seg[1].used1 = 0;
        sm.pos = begin;
        sm.end_pair = pairs;
        sm.end = (int)blockIdx.x < pieces ? piece_begin((int)blockIdx.x + 1, pieces, total) : begin;
        next_segment<kListed>(p, sm, 0, each == 1 ? n_last : -1);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_slot;
  const uint32_t vs_s = smem_u32(vs), ps_s = smem_u32(ps);
  const int quad = warp & 3;
  const uint32_t lanes = (uint32_t)(quad * 32) << 16;

  for (uint32_t sg = 0; sm.seg[sg & 1].nt > 0; ++sg) {
    const Segment& S = sm.seg[sg & 1];
    const uint32_t sph = sg & 1;                           // phase of the per-segment barriers
    const int nt = S.nt;
    if (threadIdx.x == 0) {
      // the query block, for now in the second tile
      const int r0 = S.blk * kRows;
      const uint32_t qbytes = (uint32_t)min(kRows, p.Tq * p.Hq - r0) * kD * 2;
      mbar_arrive_expect_tx(&sm.bar.q_ld, qbytes);
      bulk_load(vs + kVTile, p.q + ((size_t)S.b * p.Tq * p.Hq + r0) * kD, qbytes, &sm.bar.q_ld);
    }

    if (warp < kProducerWarps) {
      // ---------------------------------------------------------- load + dequantise
      // Eight lanes take one half (256 channels) of a row: the lane with (i, j) the
      // 32 channels 256 hh + 32 j .. of entry 8 w + 4 k + i of a tile, k = 0, 1.
      // Eight neighbouring lanes have four rows and two neighbouring j: rows lie
      // 288 bytes apart in the copy (32 more than a multiple of 128) and at other
      // swizzle phases in the tile, so their 16-byte accesses meet no bank twice.
      // The query block goes to tensor memory as fp16, scaled per row by a power of
      // two (which loses no bit of a bf16 value within 2^-24 of the row's largest).
      // Warps w and w + 4 convert quadrant w's 16 rows in place, 16-byte chunk c of
      // row h stored at c ^ (h & 7), and then move them, a thread 128 channels of one.
      auto stage_q = [&]() {
        const uint32_t qsm = vs_s + (uint32_t)kVTile;
        const bool ok = wait_hot_warp(&sm.bar.q_ld, sph, abort_flag);
        const int nr = min(kRows, p.Tq * p.Hq - S.blk * kRows);
        if (ok && warp < 8) {
#pragma unroll 1
          for (int i0 = 0; i0 < 8; i0 += 4) {
            uint4 a[4], c[4];
            uint32_t amax[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int hh = quad * 16 + (warp >> 2) * 8 + i0 + r;
              a[r] = c[r] = make_uint4(0, 0, 0, 0);
              if (hh < nr) {
                a[r] = lds128(qsm + hh * 1024 + 16 * lane);
                c[r] = lds128(qsm + hh * 1024 + 512 + 16 * lane);
              }
            }
            // (magnitudes of bf16 values order like their bits)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const uint32_t m = __vmaxu2(
                  __vmaxu2(__vmaxu2(a[r].x & 0x7fff7fffu, a[r].y & 0x7fff7fffu),
                           __vmaxu2(a[r].z & 0x7fff7fffu, a[r].w & 0x7fff7fffu)),
                  __vmaxu2(__vmaxu2(c[r].x & 0x7fff7fffu, c[r].y & 0x7fff7fffu),
                           __vmaxu2(c[r].z & 0x7fff7fffu, c[r].w & 0x7fff7fffu)));
              amax[r] = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
            }
            __syncwarp();                            // read before it is rewritten
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int hh = quad * 16 + (warp >> 2) * 8 + i0 + r;
              if (hh >= nr) continue;
              // 2^ex2 takes the largest magnitude to [2^14, 2^15); a row with a NaN or an
              // infinity is staged as zeros and marked by a negative factor
              int ex2 = 0;
              const uint32_t eb = (amax[r] >> 7) & 0xffu;
              const bool bad = eb == 0xffu;
              if (amax[r] != 0u && !bad) ex2 = min(126, 15 - ((int)eb - 126));
              const float up =
                  copysignf(__uint_as_float((uint32_t)(127 + ex2) << 23), p.softmax_scale);
              const uint32_t w[8] = {a[r].x, a[r].y, a[r].z, a[r].w,
                                     c[r].x, c[r].y, c[r].z, c[r].w};
              uint32_t f[8];
#pragma unroll
              for (int k = 0; k < 8; ++k)
                f[k] = bad ? 0u : pack_half2(__uint_as_float(w[k] << 16) * up,
                                             __uint_as_float(w[k] & 0xffff0000u) * up);
              const uint32_t qr = qsm + hh * 1024;
              sts128(qr + ((lane ^ (hh & 7)) << 4), make_uint4(f[0], f[1], f[2], f[3]));
              sts128(qr + (((32 + lane) ^ (hh & 7)) << 4), make_uint4(f[4], f[5], f[6], f[7]));
              if (lane == 0)
                sm.qdown[hh] = bad ? -1.0f : __uint_as_float((uint32_t)(127 - ex2) << 23);
            }
          }
        }
        bar_sync(kBarProducers, kProducers);
        if (warp < 8) {
          const int ch = lane >> 4, h = quad * 16 + (lane & 15);
#pragma unroll 1
          for (int i = 2 * (warp >> 2); i < 2 * (warp >> 2) + 2; ++i) {
            uint32_t w[32];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              uint4 v = make_uint4(0, 0, 0, 0);
              if (ok && h < nr)
                v = lds128(qsm + h * 1024 + (((32 * ch + 8 * i + j) ^ (h & 7)) << 4));
              w[4 * j] = v.x;
              w[4 * j + 1] = v.y;
              w[4 * j + 2] = v.z;
              w[4 * j + 3] = v.w;
            }
            // threads 0-15: channels 64 i .. + 63; threads 16-31: 256 further
            tmem_st16x2_32<128>(tmem + lanes + kTmemQ + 32u * i, w);
          }
          tc_fence_before();
        }
        bar_sync(kBarProducers, kProducers);     // the block is read: its tile can be filled
        bar_arrive(kBarQ, kNumQ);
        return ok;
      };

      const int i4 = (lane >> 1) & 3, j8 = (lane >> 3) * 2 + (lane & 1);
      // where the lane's 16-byte pieces go in a tile: chunk 4 (j % 2) + x of atom j / 2
      uint32_t at[2][4];
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          at[k][x] = vs_s + (uint32_t)((j8 >> 1) * kAtom + swz(8 * warp + 4 * k + i4, 4 * (j8 & 1) + x));
      const uint32_t row = smem_u32(raw) + (uint32_t)((8 * warp + i4) * kRowBytes + 16 * j8);
      const uint32_t srow = smem_u32(raw) + (uint32_t)((8 * warp + i4) * kRowBytes + 256 + 2 * j8);
      bool ok = stage_q();
      const uint32_t g0 = S.g0, used0 = S.used0, used1 = S.used1;
      // one tile of buffer `buf` (a constant after inlining)
      auto tile = [&](int t, int buf) {
        const uint32_t ph = ((buf ? used1 : used0) + (uint32_t)(t >> 1)) & 1;
        uint4 code[2][2];            // [half][k]: 32 channels
        uint32_t scale[2][2];        // their two scales
        bar_sync(kBarL + buf, kNumL);
        ok = ok && wait_hot_warp(&sm.bar.raw_full[buf], ph, abort_flag);
        if (ok) {
          const uint32_t o = (uint32_t)(buf * kRawTile);
#pragma unroll
          for (int hh = 0; hh < 2; ++hh)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              code[hh][k] = lds128(row + o + 4 * k * kRowBytes + 128 * hh);
              scale[hh][k] = lds16(srow + o + 4 * k * kRowBytes + 16 * hh);
            }
          const uint4 v = sm.valid[(g0 + t) & 3];
          if (!((v.x & v.y) == ~0u && (v.z & 0xffffu) == 0xffffu)) {
            const uint32_t w = warp < 4 ? v.x : warp < 8 ? v.y : v.z;
#pragma unroll
            for (int k = 0; k < 2; ++k)
              if (!(w >> ((8 * warp + 4 * k + i4) & 31) & 1u)) {   // nothing was copied there
                code[0][k] = code[1][k] = make_uint4(0, 0, 0, 0);
                scale[0][k] = scale[1][k] = 0;
              }
          }
        }
        // channels 0-255, then 256-511: each half is freed, filled and multiplied
        // on its own, so that S starts when half a tile is there
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          ok = ok && wait_hot_warp(&sm.bar.v_free[buf][hh], ph ^ 1, abort_flag);
          if (ok) {
            const uint32_t o = (uint32_t)(buf * kVTile + hh * 4 * kAtom);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint4 c = code[hh][k];
              // byte 0 twice, byte 1 twice
              const __half2 lo = e4m3x2_to_half2((uint16_t)__byte_perm(scale[hh][k], 0, 0x0000));
              const __half2 hi = e4m3x2_to_half2((uint16_t)__byte_perm(scale[hh][k], 0, 0x1111));
              sts128(at[k][0] + o, dq8(c.x, lo));
              sts128(at[k][1] + o, dq8(c.y, lo));
              sts128(at[k][2] + o, dq8(c.z, hi));
              sts128(at[k][3] + o, dq8(c.w, hi));
            }
          }
          fence_async_smem();
          bar_arrive(kBarV + 2 * buf + hh, hh ? kNumV1 : kNumV0);
        }
      };
#pragma unroll 1
      for (int t = 0; t < nt; t += 2) {
        tile(t, 0);
        if (t + 1 < nt) tile(t + 1, 1);
      }
    } else if (warp == kLoadWarp && kListed) {
      // ---------------------------------------------------------- copies of listed rows
      // Lane i has places i, i + 32 and i + 64 of a tile: their ids are loaded two
      // tiles ahead, the table places of the ids one.
      constexpr int kIds = 3;
      const int t0 = S.t0;
      const uint32_t g0 = S.g0;
      const int s = slot_of(p, S.b);
      const int n = visible_most(p, S.b, true);            // ids lie below
      const int32_t* ids = p.ids + (size_t)S.b * p.K;
      const int32_t* table = p.pg.table + (size_t)(n > 0 ? s : 0) * p.pg.M;
      auto fetch_id = [&](int t, int k) -> int {
        const int i = lane + 32 * k;
        const long long e = (long long)(t0 + t) * kT + i;
        if (t >= nt || i >= kT || e >= p.K) return -1;
        return __ldg(ids + e);
      };
      auto check_id = [&](int id) -> int {
        if (id >= -1 && id < n) return id;
        record_error(p.err, CSA2_ERR_DEVICE_INDEX);
        return -1;
      };
      auto fetch_place = [&](int id) { return id >= 0 ? __ldg(table + (id >> p.shift)) : 0; };
      int id[kIds], place[kIds], id_next[kIds];
#pragma unroll
      for (int k = 0; k < kIds; ++k) {
        id[k] = check_id(fetch_id(0, k));
        place[k] = fetch_place(id[k]);
        id_next[k] = fetch_id(1, k);
      }
      for (int t = 0; t < nt; ++t) {
        const int buf = t & 1;
        int row[kIds];
        uint32_t bits[kIds];
#pragma unroll
        for (int k = 0; k < kIds; ++k) {
          row[k] = -1;
          if (id[k] >= 0) {
            if (place[k] < 0 || place[k] >= p.pg.P)
              record_error(p.err, CSA2_ERR_DEVICE_INDEX);
            else
              row[k] = (place[k] << p.shift) + (id[k] & (p.pg.page - 1));
          }
          bits[k] = __ballot_sync(0xffffffffu, row[k] >= 0);
          id[k] = check_id(id_next[k]);
          place[k] = fetch_place(id[k]);
          id_next[k] = fetch_id(t + 2, k);
        }
        if (t >= 2) bar_sync(kBarV + 2 * buf + 1, kNumV1);     // the rows before are read
        if (lane == 0) sm.valid[(g0 + t) & 3] = make_uint4(bits[0], bits[1], bits[2], 0);
        const uint32_t dst = smem_u32(raw) + (uint32_t)(buf * kRawTile) + 16u * lane;
#pragma unroll
        for (int k = 0; k < kIds; ++k) {
          // rows 32 k .. : 18 16-byte pieces each, dealt to the lanes in order
          constexpr int kPieces = kRowBytes / 16;
          const int rounds = k < 2 ? kPieces : (kT - 64) * kPieces / 32;
#pragma unroll 6
          for (int j = 0; j < rounds; ++j) {
            const int x = 32 * j + lane, r = x / kPieces;
            const int at = __shfl_sync(0xffffffffu, row[k], r);
            if (at >= 0)
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                               dst + (uint32_t)(32 * k * kRowBytes + 512 * j)),
                           "l"(p.pg.rows + (size_t)at * kRowBytes + (x - r * kPieces) * 16)
                           : "memory");
          }
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                         smem_u32(&sm.bar.raw_full[buf]))
                     : "memory");
        __syncwarp();
        bar_arrive(kBarL + buf, kNumL);
      }
      for (int t = max(0, nt - 2); t < nt; ++t)
        bar_sync(kBarV + 2 * (t & 1) + 1, kNumV1);
      if (lane == 0) next_segment<kListed>(p, sm, (int)(sph ^ 1), -1);
    } else if (warp == kLoadWarp) {
      // ---------------------------------------------------------- bulk copies
      // Lane i copies the rows of a tile that lie in its i-th page (a tile of 80
      // entries touches at most 11 pages of 8).
      const int n_most = S.n_most, t0 = S.t0;
      const uint32_t g0 = S.g0;
      const int s = n_most > 0 ? slot_of(p, S.b) : 0;
      const int32_t* table = p.pg.table + (size_t)s * p.pg.M;
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
        const int buf = t & 1;
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
        if (t >= 2) bar_sync(kBarV + 2 * buf + 1, kNumV1);     // the rows before are read
        if (lane == 0) {
          sm.valid[(g0 + t) & 3] = make_uint4(bits[0], bits[1], bits[2], 0);
          mbar_arrive_expect_tx(&sm.bar.raw_full[buf],
                                (uint32_t)(__popc(bits[0]) + __popc(bits[1]) + __popc(bits[2])) *
                                    kRowBytes);
        }
        __syncwarp();
        if (count)
          bulk_load(raw + buf * kRawTile + at * kRowBytes,
                    p.pg.rows + (((size_t)place << p.shift) + (size_t)(lo & (p.pg.page - 1))) * kRowBytes,
                    (uint32_t)count * kRowBytes, &sm.bar.raw_full[buf]);
        bar_arrive(kBarL + buf, kNumL);
        place = place_next;
      }
      for (int t = max(0, nt - 2); t < nt; ++t)
        bar_sync(kBarV + 2 * (t & 1) + 1, kNumV1);
      if (lane == 0) next_segment<kListed>(p, sm, (int)(sph ^ 1), -1);
    } else if (warp == kMmaWarp) {
      // ---------------------------------------------------------- MMA issuer
      // The whole warp runs this with warp-uniform values and one elected lane
      // issues: descriptors then stay in uniform registers (from one divergent
      // thread an instruction took 65 to 80 cycles to issue, more than to run).
      const uint32_t id_s = idesc_f16(64, kT, 0);
      const uint32_t id_o = idesc_f16(64, 256, 1);
      const uint64_t vk = desc_sw128(vs_s, 16, 1024);       // V as K-major B
      const uint64_t vn = desc_sw128(vs_s, kAtom, 1024);    // V as N-major B
      const uint64_t p0 = desc_sw128(ps_s, 16, 1024);       // P as K-major A
      const uint64_t p1 = desc_sw32(ps_s + 2 * kP0);
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const int ntu = __shfl_sync(0xffffffffu, nt, 0);
      bar_sync(kBarQ, kNumQ);
      auto issue_s = [&](uint32_t buf, int hh) {
        tc_fence_after();
        const uint64_t v = vk + (uint64_t)((buf * kVTile + hh * 4 * kAtom) >> 4);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 16; ++k)
            mma_ts(tm + (uint32_t)kT * buf, tm + kTmemQ + 128u * hh + 8u * k,
                   v + (uint64_t)(((k >> 2) * kAtom + (k & 3) * 32) >> 4), id_s,
                   k > 0 || hh > 0 ? 1u : 0u);
          if (hh == 1) mma_commit(&sm.bar.s_full[buf]);
        }
        __syncwarp();
      };
      auto issue_pv = [&](uint32_t buf, uint32_t acc0) {
        tc_fence_after();
        const uint64_t v = vn + (uint64_t)((buf * kVTile) >> 4);
        const uint64_t a0 = p0 + (uint64_t)((buf * kP0) >> 4);
        const uint64_t a1 = p1 + (uint64_t)((buf * kP1) >> 4);
        if (elect_one()) {
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
#pragma unroll
            for (int ks = 0; ks < kT / 16; ++ks)
              mma_ss(tm + kHalfLanes + 256u * hh, ks < 4 ? a0 + (uint64_t)(ks * 32 >> 4) : a1,
                     v + (uint64_t)((4 * hh * kAtom + ks * 2048) >> 4), id_o, ks > 0 ? 1u : acc0);
            mma_commit(&sm.bar.v_free[buf][hh]);
          }
        }
        __syncwarp();
      };
      bool go = true;
      for (int t = 0; t < ntu; t += 2) {
        const int more = min(2, ntu - t);
#pragma unroll 1
        for (int i = 0; i < more; ++i) {
          const uint32_t buf = (uint32_t)i;      // t is even
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            bar_sync(kBarV + 2 * buf + hh, hh ? kNumV1 : kNumV0);
            if (go) issue_s(buf, hh);
          }
          bar_arrive(kBarS + buf, kNumS);
        }
        go = !__any_sync(0xffffffffu, *abort_flag != 0);
#pragma unroll 1
        for (int i = 0; i < more; ++i) {
          const uint32_t buf = (uint32_t)i;      // t is even
          bar_sync(kBarP + buf, kNumP);
          if (go) issue_pv(buf, t + i > 0 ? 1u : 0u);
        }
      }
      if (elect_one()) mma_commit(&sm.bar.o_full);
      __syncwarp();
      // nothing may be in flight when tensor memory is reused or released
      wait_hot_warp(&sm.bar.o_full, sph, abort_flag);
    } else {
      // ---------------------------------------------------------- softmax
      const int hl = lane & 15, ch = lane >> 4;
      const int h = quad * 16 + hl;
      bar_sync(kBarQ, kNumQ);
      const int r0 = S.blk * kRows;
      const bool real = r0 + h < p.Tq * p.Hq;
      const float hs = real ? fabsf(p.softmax_scale) * kLog2e * fabsf(sm.qdown[h]) : 0.0f;
      // entries that this row sees from the segment's first on
      const int n_row = (!kListed && real && p.nvalid ? visible(p, S.b, (r0 + h) / p.Hq) : S.n_most) -
                        S.t0 * kT;
      const uint32_t g0 = S.g0, used0 = S.used0, used1 = S.used1;
      // (the reference is kept as S has it, and logits are the differences times hs: a
      // product rounded before the difference is off by its own size 2^-24, which is
      // more than one for logits of 2^24 and above)
      float m_ref = -INFINITY, l = 0.0f;
      bool ok = true;
      for (int t = 0; t < nt; ++t) {
        const int buf = t & 1;
        bar_sync(kBarS + buf, kNumS);
        ok = ok && wait_hot_warp(&sm.bar.s_full[buf], ((buf ? used1 : used0) + (uint32_t)(t >> 1)) & 1, abort_flag);
        if (ok) {
          tc_fence_after();
          // this thread's entries: 40 ch .. + 39 of the tile, masks of 32 and 8
          const int left = n_row - t * kT - kHalfT * ch;
          uint32_t m0, m1;
          {
            const uint4 v = sm.valid[(g0 + t) & 3];
            m0 = ch ? (v.y >> 8) | (v.z << 24) : v.x;
            m1 = (ch ? v.z >> 8 : v.y) & 0xffu;
            if (left < kHalfT) {
              m0 &= left <= 0 ? 0u : left >= 32 ? ~0u : (1u << left) - 1u;
              m1 &= left <= 32 ? 0u : (1u << (left - 32)) - 1u;
            }
          }
          float y[kHalfT];
          tmem_ld_logits(tmem + lanes + (uint32_t)kT * buf, y);
          // (the scale is not negative: its sign went into the query block)
          float xm[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          const bool all = __all_sync(0xffffffffu, m0 == ~0u && m1 == 0xffu) != 0;
          if (all) {
#pragma unroll
            for (int j = 0; j < kHalfT; ++j) xm[j & 3] = fmaxf(xm[j & 3], y[j]);
          } else {
#pragma unroll
            for (int j = 0; j < kHalfT; ++j)
              if ((j < 32 ? m0 >> j : m1 >> (j - 32)) & 1u) xm[j & 3] = fmaxf(xm[j & 3], y[j]);
          }
          float xmax = fmaxf(fmaxf(xm[0], xm[1]), fmaxf(xm[2], xm[3]));
          xmax = fmaxf(xmax, __shfl_xor_sync(0xffffffffu, xmax, 16));
          const bool raise = m_ref == -INFINITY ? xmax != -INFINITY
                                                : (xmax - m_ref) * hs > kRescaleSlack;
          if (__any_sync(0xffffffffu, raise)) {
            float alpha = 1.0f;
            if (raise) {
              if (m_ref != -INFINITY) alpha = fast_exp2((m_ref - xmax) * hs);
              m_ref = xmax;
              l *= alpha;
            }
            // O holds the tiles before: rescaled once they are complete (O += of
            // this one waits for its P)
            if (t > 0 && __any_sync(0xffffffffu, alpha != 1.0f)) {
              const int pb = buf ^ 1;
              ok = wait_hot_warp(&sm.bar.v_free[pb][1], ((pb ? used1 : used0) + (uint32_t)((t - 1) >> 1)) & 1,
                                 abort_flag);
              if (ok) {
                tc_fence_after();
#pragma unroll 1
                for (int c0 = 0; c0 < kD / 2; c0 += 32) {
                  float o[32];
                  tmem_ld16x2_32<256>(tmem + lanes + kHalfLanes + c0, o);
                  uint32_t ow[32];
#pragma unroll
                  for (int c = 0; c < 32; ++c) ow[c] = __float_as_uint(o[c] * alpha);
                  tmem_st16x2_32<256>(tmem + lanes + kHalfLanes + c0, ow);
                }
              }
            }
          }
          const float mm = m_ref == -INFINITY ? 0.0f : m_ref;   // nothing seen yet: 2^-inf = 0
          float ls[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int k = 0; k < kHalfT / 8; ++k) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int j = 8 * k + 2 * i;
              const float2 z = lifted_difference(y[j], y[j + 1], mm, hs);
              float x0 = fast_exp2(z.x), x1 = fast_exp2(z.y);
              if (!all) {
                if (!((j < 32 ? m0 >> j : m1 >> (j - 32)) & 1u)) x0 = 0.0f;
                if (!((j + 1 < 32 ? m0 >> (j + 1) : m1 >> (j + 1 - 32)) & 1u)) x1 = 0.0f;
              }
              ls[i] += x0 + x1;
              w[i] = pack_half2(x0, x1);
            }
            const int c = (kHalfT / 8) * ch + k;      // 16-byte chunk: entries 8 c .. + 7
            const uint32_t at =
                c < 8 ? ps_s + (uint32_t)(buf * kP0 + swz(h, c))
                      : ps_s + (uint32_t)(2 * kP0 + buf * kP1 + h * 32 +
                                          (((c - 8) ^ (h >> 2 & 1)) << 4));
            sts128(at, make_uint4(w[0], w[1], w[2], w[3]));
          }
          l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
          fence_async_smem();
          tc_fence_before();
        }
        bar_arrive(kBarP + buf, kNumP);
      }
      float l_tot = l + __shfl_xor_sync(0xffffffffu, l, 16);
      if (ch == 0) {
        if (real && sm.qdown[h] < 0.0f && l_tot > 0.0f) l_tot = NAN;     // and it saw something
        sm.mlf[h] = make_float2(l_tot == 0.0f ? -INFINITY : m_ref * hs - kLift, l_tot);
      }
    }

    // -------------------------------------------------------------- output
    // O through shared memory (the idle tiles), so that rows are written whole:
    // [64 rows][2 KB], 16-byte chunk c of row h at c ^ (h & 7).
    const bool softmaxer = warp >= kProducerWarps && warp < kMmaWarp;
    if (warp < 8 || softmaxer) {
      const bool have_o = wait_hot_warp(&sm.bar.o_full, sph, abort_flag);
      tc_fence_after();
      if (have_o) {
        const int h = quad * 16 + (lane & 15), ch = lane >> 4;
        // chunks of 32 columns (and the same 256 further): the quadrant's softmax
        // warp takes 0-2, its producer warps 3-5 and 6-7
        const int cb = softmaxer ? 0 : warp < 4 ? 3 : 6;
        const int ce = softmaxer ? 3 : warp < 4 ? 6 : 8;
#pragma unroll 1
        for (int c = cb; c < ce; ++c) {
          float o[32];
          tmem_ld16x2_32<256>(tmem + lanes + kHalfLanes + 32u * c, o);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            sts128(vs_s + (uint32_t)(h * 2048 + (((64 * ch + 8 * c + k) ^ (h & 7)) << 4)),
                   make_uint4(__float_as_uint(o[4 * k]), __float_as_uint(o[4 * k + 1]),
                              __float_as_uint(o[4 * k + 2]), __float_as_uint(o[4 * k + 3])));
        }
      }
    }
    tc_fence_before();
    const bool stop = __syncthreads_or(*abort_flag) != 0;
    tc_fence_after();
    if (stop) {
      // a wait ran out: what was copied may still be on its way (waited for again,
      // for a limited time)
      if (threadIdx.x == 0) {
        int none = 0;
        mbar_wait(&sm.bar.q_ld, sph, &none);
        for (int i = 0; i < 2 && i < nt; ++i) {
          none = 0;
          const uint32_t last = (i ? S.used1 : S.used0) + (uint32_t)((nt - 1 - i) >> 1);
          mbar_wait(&sm.bar.raw_full[i], last & 1, &none);
        }
      }
      break;
    }
    {
      const int r0 = S.blk * kRows, slot = S.slot;
      const int nr = min(kRows, p.Tq * p.Hq - r0);
      const size_t row0 = (size_t)S.b * p.Tq * p.Hq + r0;
      const bool more = S.more != 0;
      if (S.carry || more) {
        // O and (maximum, sum) with the carry's: into the carry again, or where the
        // rows are written from. (A thread meets its own values of each row only.)
#pragma unroll 1
        for (int h = warp; h < nr; h += kThreads / 32) {
          const size_t at = (size_t)blockIdx.x * kRows + h;
          float2 ml = sm.mlf[h];
          float w = 1.0f, wc = 0.0f;
          if (S.carry) {
            const float2 c = p.ws_carry_ml[at];
            const float m = fmaxf(ml.x, c.x);
            w = ml.x == m ? 1.0f : exp2f(ml.x - m);
            wc = c.x == m ? 1.0f : exp2f(c.x - m);
            ml = make_float2(m, fmaf(ml.y, w, c.y * wc));
          }
          __syncwarp();                              // read by every lane
          if (lane == 0) {
            if (more) p.ws_carry_ml[at] = ml;
            else sm.mlf[h] = ml;
          }
          const uint32_t row = vs_s + (uint32_t)(h * 2048);
#pragma unroll
          for (int k = 0; k < kD / 128; ++k) {
            const int c = 32 * k + lane;
            const uint32_t src = row + ((c ^ (h & 7)) << 4);
            float4* sum = reinterpret_cast<float4*>(p.ws_carry + at * kD) + c;
            const uint4 o = lds128(src);
            float4 v = make_float4(__uint_as_float(o.x), __uint_as_float(o.y),
                                   __uint_as_float(o.z), __uint_as_float(o.w));
            if (S.carry) {
              const float4 u = *sum;
              v = make_float4(fmaf(v.x, w, u.x * wc), fmaf(v.y, w, u.y * wc),
                              fmaf(v.z, w, u.z * wc), fmaf(v.w, w, u.w * wc));
            }
            if (more)
              *sum = v;
            else
              sts128(src, make_uint4(__float_as_uint(v.x), __float_as_uint(v.y),
                                     __float_as_uint(v.z), __float_as_uint(v.w)));
          }
          __syncwarp();
        }
      }
#pragma unroll 2
      for (int h = more ? nr : warp; h < nr; h += kThreads / 32) {
        const float2 ml = sm.mlf[h];
        const uint32_t row = vs_s + (uint32_t)(h * 2048);
        // over the row sum (a row that saw nothing has sum 0 and zeros in O): the
        // output in bf16, or a partial, a mean of values and so below 2^12, in fp16 (half a
        // step is 2^-11 of it, an eighth of the output's 2^-8, for half of fp32's bytes)
        const float f = ml.y == 0.0f ? 0.0f : 1.0f / ml.y;
        uint4* dst = reinterpret_cast<uint4*>(
            slot < 0 ? reinterpret_cast<uint16_t*>(p.out) + (row0 + h) * kD
                     : reinterpret_cast<uint16_t*>(p.ws_o) + ((size_t)slot * kRows + h) * kD);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int c = 64 * k + 2 * lane;
          const uint4 a = lds128(row + ((c ^ (h & 7)) << 4));
          const uint4 d = lds128(row + (((c + 1) ^ (h & 7)) << 4));
          const float v[8] = {__uint_as_float(a.x) * f, __uint_as_float(a.y) * f,
                              __uint_as_float(a.z) * f, __uint_as_float(a.w) * f,
                              __uint_as_float(d.x) * f, __uint_as_float(d.y) * f,
                              __uint_as_float(d.z) * f, __uint_as_float(d.w) * f};
          dst[32 * k + lane] =
              slot < 0 ? make_uint4(pack_bf162(v[0], v[1]), pack_bf162(v[2], v[3]),
                                    pack_bf162(v[4], v[5]), pack_bf162(v[6], v[7]))
                       : make_uint4(pack_half2(v[0], v[1]), pack_half2(v[2], v[3]),
                                    pack_half2(v[4], v[5]), pack_half2(v[6], v[7]));
        }
        if (lane == 0) {
          if (slot >= 0)
            p.ws_ml[(size_t)slot * kRows + h] = ml;
          else if (p.lse)
            p.lse[row0 + h] = ml.y == 0.0f ? -INFINITY : (ml.x + log2f(ml.y)) * kLn2;
        }
      }
    }
    fence_async_smem();               // the tiles are next written by a bulk copy
    __syncthreads();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (threadIdx.x == 0 && *abort_flag) record_error(p.err, CSA2_ERR_TIMEOUT);
}

// Joins the pieces of one query row: out = sum_i w_i o_i / sum_i w_i, w_i = 2^(m_i - M) l_i,
// in one pass with the running M. A thread holds 8 channels (a 16-byte load per piece),
// kLanes threads 8 kLanes of the 512, and kGroups such groups share out the pieces,
// four pieces of each on their way at a time. Bound: the latency of those loads, so
// few rows, which come from many pieces, take many groups and CTAs. Measured (whole call):
// 64 rows of 148 pieces, 16 groups on 4 CTAs: 38 us of the call's, 4 groups on one 45;
// 512 rows of 19, 4 groups: 41 us, 16 groups 45; 960 rows of 10, one group: 30 us (16: 37).
template <int kLanes, int kGroups>
__global__ void __launch_bounds__(256) paged_combine_kernel(const Params p, int b0) {
  constexpr int kRowsPerCta = 256 / (kLanes * kGroups), kParts = 64 / kLanes;
  constexpr int kBatch = 4, kChannels = 8 * kLanes;
  static_assert(kGroups == 1 || kRowsPerCta == 1, "the groups of a row are the CTA");
  __shared__ __align__(16) float part[kGroups][kGroups > 1 ? kChannels : 4];
  __shared__ float2 part_ml[kGroups];
  pdl_wait_and_release();
  const int per_seq = p.Tq * p.Hq;
  const int grp = threadIdx.x / kLanes % kGroups;
  const int r = blockIdx.x / kParts * kRowsPerCta + threadIdx.x / (kLanes * kGroups);
  if (r >= per_seq) return;
  const size_t b = (size_t)b0 + blockIdx.y;
  const int4 info = p.ws_info[b * p.nblk + r / kRows];
  const int first = info.x, last = info.y;
  // (nothing is joined of a pair whose CTA gave up before it wrote its record)
  if (first == last || !join_record_holds(first, last, info.z, p.pieces)) return;
  const int h = r % kRows;
  const int c = blockIdx.x % kParts * kLanes + threadIdx.x % kLanes;   // of 64, 8 channels each
  float M = -INFINITY, L = 0.0f;
  float acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  for (int i0 = first + grp; i0 <= last; i0 += kGroups * kBatch) {
    float2 ml[kBatch];
    uint4 u[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * kGroups;
      ml[k] = make_float2(-INFINITY, 0.0f);
      u[k] = make_uint4(0, 0, 0, 0);
      if (i <= last) {
        const size_t at = (size_t)join_slot(i, first, info.z) * kRows + h;
        ml[k] = p.ws_ml[at];
        u[k] = *reinterpret_cast<const uint4*>(p.ws_o + at * kD + 8 * c);
      }
    }
    float m = M;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) m = fmaxf(m, ml[k].x);
    if (m == -INFINITY) continue;                      // pieces that saw nothing
    const float f = exp2f(M - m);
    M = m;
    L *= f;
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] *= f;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const float w = exp2f(ml[k].x - M) * ml[k].y;    // 0 for a piece that saw nothing
      const uint32_t v[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
      L += w;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 o = __half22float2(*reinterpret_cast<const __half2*>(&v[q]));
        acc[2 * q] = fmaf(w, o.x, acc[2 * q]);
        acc[2 * q + 1] = fmaf(w, o.y, acc[2 * q + 1]);
      }
    }
  }
  const size_t row = b * per_seq + r;
  if (kGroups == 1) {
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    reinterpret_cast<uint4*>(p.out + row * kD)[c] =
        make_uint4(pack_bf162(acc[0] * inv, acc[1] * inv), pack_bf162(acc[2] * inv, acc[3] * inv),
                   pack_bf162(acc[4] * inv, acc[5] * inv), pack_bf162(acc[6] * inv, acc[7] * inv));
    if (p.lse && c == 0) p.lse[row] = L == 0.0f ? -INFINITY : (M + log2f(L)) * kLn2;
    return;
  }
  const int lane = threadIdx.x % kLanes;
  *reinterpret_cast<float4*>(&part[grp][8 * lane]) = make_float4(acc[0], acc[1], acc[2], acc[3]);
  *reinterpret_cast<float4*>(&part[grp][8 * lane + 4]) =
      make_float4(acc[4], acc[5], acc[6], acc[7]);
  if (lane == 0) part_ml[grp] = make_float2(M, L);
  __syncthreads();
  if (threadIdx.x >= kChannels / 2) return;            // two channels each
  M = -INFINITY;
#pragma unroll
  for (int g = 0; g < kGroups; ++g) M = fmaxf(M, part_ml[g].x);
  float2 o = make_float2(0.0f, 0.0f);
  L = 0.0f;
  if (M != -INFINITY) {
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const float2 ml = part_ml[g];
      const float f = exp2f(ml.x - M);
      const float2 v = *reinterpret_cast<const float2*>(&part[g][2 * threadIdx.x]);
      L = fmaf(f, ml.y, L);
      o.x = fmaf(f, v.x, o.x);
      o.y = fmaf(f, v.y, o.y);
    }
  }
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
  reinterpret_cast<uint32_t*>(p.out + row * kD)[blockIdx.x % kParts * (kChannels / 2) + threadIdx.x] =
      pack_bf162(o.x * inv, o.y * inv);
  if (p.lse && blockIdx.x % kParts == 0 && threadIdx.x == 0)
    p.lse[row] = L == 0.0f ? -INFINITY : (M + log2f(L)) * kLn2;
}

int sm_count_of_device() {
  int dev = 0, n = 148;
  if (cudaGetDevice(&dev) == cudaSuccess)
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n;
}

// The kernels' shared memory, allowed once per device.
cudaError_t allow_shared_memory() {
  static std::mutex mu;
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (done[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(paged_attn_tc_kernel<false>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(paged_attn_tc_kernel<true>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
  done[dev] = e == cudaSuccess;
  return e;
}

// What a call goes through: pairs of a sequence (with lists: a query token) and a
// block of 64 of its rows, of at most `most` entries each.
struct Shape {
  int B, rows, nblk;
  long long most;
  Shape(const fp4_kv_pages& pg, int B_, int Tq, int Hq, int K)
      : B(K ? B_ * Tq : B_), rows(K ? Hq : Tq * Hq), nblk(ceil_div(rows, kRows)),
        most(K ? K : (long long)pg.M * pg.page) {}
  // pieces of the line of tiles: one per SM, never more than there can be units
  long long units() const { return (kSetup + (most + kT - 1) / kT) * B * nblk; }
  int pieces() const {
    const long long all = units();
    const int sms = sm_count_of_device();
    return (int)(all < sms ? all : sms);
  }
  // whether a piece can have more tiles of a pair than a segment (even pieces have
  // units() / pieces() at most, and pairs are dealt out whole where they are shorter)
  bool carries() const { return units() / pieces() + 1 > kMostTiles; }
};

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

size_t paged_attn_workspace_bytes(const fp4_kv_pages& pg, int B, int Tq, int Hq, int K) {
  const Shape sh(pg, B, Tq, Hq, K);
  const size_t slots = 2 * (size_t)sh.pieces();
  const size_t carry = sh.carries() ? slots / 2 * kRows : 0;     // rows
  return up256((size_t)sh.B * sh.nblk * sizeof(int4)) + up256(slots * kRows * sizeof(float2)) +
         up256(slots * kRows * kD * sizeof(__half)) + up256(carry * sizeof(float2)) +
         carry * kD * sizeof(float);
}

cudaError_t launch_paged_attn(const uint16_t* q, const fp4_kv_pages& pg, const int32_t* seq,
                              const int32_t* nvalid, const int32_t* topk_idx, int B, int Tq,
                              int Hq, int K, float softmax_scale, uint16_t* out, float* lse,
                              void* workspace, int* err, cudaStream_t stream) {
  if (topk_idx == nullptr) K = 0;
  const Shape sh(pg, B, Tq, Hq, K);
  Params p;
  p.q = q;
  p.pg = pg;
  p.shift = 0;
  while ((1 << p.shift) < pg.page) ++p.shift;
  p.seq = seq;
  p.nvalid = nvalid;
  p.ids = topk_idx;
  p.K = K;
  p.B = sh.B;
  p.Tq = K ? 1 : Tq;
  p.Hq = Hq;
  p.nblk = sh.nblk;
  p.per_slot = K ? Tq : 1;
  p.softmax_scale = softmax_scale;
  p.out = out;
  p.lse = lse;
  const int pieces = sh.pieces();
  p.pieces = pieces;
  p.share = ((long long)sh.B * sh.nblk + pieces - 1) / pieces;
  unsigned char* w = static_cast<unsigned char*>(workspace);
  p.ws_info = reinterpret_cast<int4*>(w);
  w += up256((size_t)sh.B * sh.nblk * sizeof(int4));
  p.ws_ml = reinterpret_cast<float2*>(w);
  w += up256(2 * (size_t)pieces * kRows * sizeof(float2));
  p.ws_o = reinterpret_cast<__half*>(w);
  w += up256(2 * (size_t)pieces * kRows * kD * sizeof(__half));
  p.ws_carry_ml = sh.carries() ? reinterpret_cast<float2*>(w) : nullptr;
  w += up256((size_t)pieces * kRows * sizeof(float2));
  p.ws_carry = sh.carries() ? reinterpret_cast<float*>(w) : nullptr;
  p.err = err;
  cudaError_t e = allow_shared_memory();
  if (e != cudaSuccess) return e;
  e = launch_pdl(K ? paged_attn_tc_kernel<true> : paged_attn_tc_kernel<false>, dim3(pieces),
                 dim3(kThreads), kSmemBytes, stream, dim3(1), p);
  if (e != cudaSuccess) return e;
  // rows in x, sequences in y (at most 65535 of each: y would not hold more)
  const int rows = sh.rows;
  for (int b0 = 0; b0 < sh.B; b0 += 65535) {
    const unsigned nb = (unsigned)(sh.B - b0 < 65535 ? sh.B - b0 : 65535);
    const long long all = (long long)sh.B * rows;
    const int sms = sm_count_of_device();
    if (all <= 2 * sms)
      e = launch_pdl(paged_combine_kernel<16, 16>, dim3(4 * rows, nb), dim3(256), 0, stream, dim3(1),
                     p, b0);
    else if (all <= 8 * sms)
      e = launch_pdl(paged_combine_kernel<64, 4>, dim3(rows, nb), dim3(256), 0, stream, dim3(1), p,
                     b0);
    else
      e = launch_pdl(paged_combine_kernel<64, 1>, dim3(ceil_div(rows, 4), nb), dim3(256), 0, stream,
                     dim3(1), p, b0);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace csa2
