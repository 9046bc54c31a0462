// pages.cu -- upkeep of the paged FP4 cache (fp4_kv_pages_*): lengths, sharing
// and compaction, all on the device, with the lowest free pages taken first so
// that the result does not depend on the order in which threads run.
//
// State: table [S][M], len [S], refs [P]; a page is free when refs is 0. Every
// call plans (reading the state, writing the workspace) and then carries the plan
// out: in one launch of one cluster where there is little to do (a launch costs
// about as much as the work, 3 us), else in a second launch over the whole GPU.
// The planner is one cluster of 8 CTAs: each of its 256 warps walks one stretch of
// refs, the counts are summed over the cluster through distributed shared memory,
// and the warps whose stretch holds a wanted page walk it again to write the pages
// out. What bounds the calls: launch and L2 latency for the plans, HBM for the
// copied pages.
#include <cooperative_groups.h>
#include <limits.h>

#include <mutex>

#include "common.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace csa2 {
namespace {

namespace cg = cooperative_groups;

constexpr int kPlanCtas = 8;
constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanCtas * kPlanThreads / 32;
constexpr int kThreads = 256;

__device__ __forceinline__ int pages_for(int n, int page_shift) {
  return (int)(((long long)n + (1 << page_shift) - 1) >> page_shift);
}

// Counts of each warp of the cluster -> the sum over the warps before this one
// (exclusive) and over all. Called by every thread; v is the warp's count.
__device__ long long cluster_exclusive(cg::cluster_group& cl, int v, long long* total) {
  __shared__ int warp_sum[kPlanThreads / 32];
  __shared__ int cta_sum[kPlanCtas];      // written by every CTA of the cluster
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __syncthreads();                        // the last call's values have been read
  cl.sync();
  if (lane == 0) warp_sum[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int s = warp_sum[lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane < kPlanCtas) *cl.map_shared_rank(&cta_sum[cl.block_rank()], lane) = s;
  }
  cl.sync();
  long long before = 0, all = 0;
  for (int c = 0; c < kPlanCtas; ++c) {
    if (c < (int)cl.block_rank()) before += cta_sum[c];
    all += cta_sum[c];
  }
  for (int w = 0; w < warp; ++w) before += warp_sum[w];
  *total = all;
  return before;
}

// The stretch of pages [lo, hi) of this warp: whole groups of 128 pages.
__device__ __forceinline__ void warp_stretch(int rank, int P, int* lo, int* hi) {
  const int w = rank * (kPlanThreads / 32) + (threadIdx.x >> 5);
  const int groups = (P + 127) / 128;
  const int each = (groups + kPlanWarps - 1) / kPlanWarps;
  *lo = (int)min((long long)P, (long long)w * each * 128);
  *hi = (int)min((long long)P, (long long)(w + 1) * each * 128);
}

// Four refs of the lane at pages p .. p + 3 (past the end: -1).
__device__ __forceinline__ int4 load_refs(const int32_t* refs, int p, int P) {
  if (p + 4 <= P) return *reinterpret_cast<const int4*>(refs + p);
  int4 v = make_int4(-1, -1, -1, -1);
  if (p < P) v.x = refs[p];
  if (p + 1 < P) v.y = refs[p + 1];
  if (p + 2 < P) v.z = refs[p + 2];
  return v;
}

// Counts, over [lo, hi), the pages for which sel(page, refs) holds.
template <typename Sel>
__device__ int count_pages(const int32_t* refs, int lo, int hi, int P, Sel sel) {
  const int lane = threadIdx.x & 31;
  int n = 0;
#pragma unroll 4
  for (int p0 = lo; p0 < hi; p0 += 128) {
    const int p = p0 + 4 * lane;
    const int4 r = load_refs(refs, p, P);
    n += sel(p, r.x) + sel(p + 1, r.y) + sel(p + 2, r.z) + sel(p + 3, r.w);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  return n;
}

// Calls put(rank, page) for the selected pages of [lo, hi) in ascending order,
// ranks from `at` on, while they are below `limit`.
template <typename Sel, typename Put>
__device__ void emit_pages(const int32_t* refs, int lo, int hi, int P, long long at,
                           long long limit, Sel sel, Put put) {
  const int lane = threadIdx.x & 31;
  int4 next = lo < hi ? load_refs(refs, lo + 4 * lane, P) : make_int4(-1, -1, -1, -1);
  for (int p0 = lo; p0 < hi && at < limit; p0 += 128) {
    const int p = p0 + 4 * lane;
    const int4 r = next;
    if (p0 + 128 < hi) next = load_refs(refs, p + 128, P);   // on its way during this round
    const int rr[4] = {r.x, r.y, r.z, r.w};
    int mine = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) mine += sel(p + k, rr[k]);
    int pre = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, pre, o);
      if (lane >= o) pre += x;
    }
    const int all = __shfl_sync(0xffffffffu, pre, 31);
    long long k_at = at + pre - mine;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (sel(p + k, rr[k])) {
        if (k_at < limit) put(k_at, p + k);
        ++k_at;
      }
    at += all;
  }
}

// A slot listed more than once: `seen` and `twice` are bitmaps over the slots in
// shared memory (zeroed here); one CTA marks all n slots.
__device__ void mark_twice(const int32_t* slot, int n, int S, uint32_t* seen, uint32_t* twice) {
  for (int i = threadIdx.x; i < (S + 31) / 32; i += blockDim.x) seen[i] = twice[i] = 0u;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int s = slot[i];
    if (s < 0 || s >= S) continue;
    const uint32_t bit = 1u << (s & 31);
    if (atomicOr(&seen[s >> 5], bit) & bit) atomicOr(&twice[s >> 5], bit);
  }
  __syncthreads();
}

// ---------------------------------------------------------------- resize
// Workspace: start [n] (the first of a request's places in free_pages, -1: the
// request is not carried out), copied [n] (the page whose filled rows are
// copied, -1: none), old_len [n], free_pages [min(P, n (M + 1))].
struct ResizePlan {
  int32_t* start;
  int32_t* copied;
  int32_t* old_len;
  int32_t* free_pages;
};

struct Request {
  bool ok;
  int cur, need, tail;   // the present length, pages to take, the page to copy or -1
};

__device__ __forceinline__ Request read_request(const fp4_kv_pages& pg, int shift,
                                                const int32_t* seq, const int32_t* new_len, int i,
                                                const uint32_t* twice) {
  Request r = {false, 0, 0, -1};
  const int s = seq[i];
  if (s < 0 || s >= pg.S || (twice[s >> 5] >> (s & 31) & 1u)) return r;
  const int want_len = new_len[i], cur = pg.len[s];
  const long long most = (long long)pg.M << shift;
  if (want_len < 0 || want_len > most || cur < 0 || cur > most) return r;
  const int have = pages_for(cur, shift);
  r.ok = true;
  r.cur = cur;
  r.need = max(0, pages_for(want_len, shift) - have);
  if (want_len > cur && (cur & (pg.page - 1)) != 0) {
    const int t = pg.table[(size_t)s * pg.M + have - 1];
    if (t < 0 || t >= pg.P) {
      r.ok = false;
      r.need = 0;
    } else if (pg.refs[t] > 1) {
      r.tail = t;
      ++r.need;
    }
  }
  return r;
}

// Carries out request i: its table places and the copied rows, shared out over
// `threads` threads of which this is number tid.
__device__ void resize_apply(const fp4_kv_pages& pg, int shift, int row_bytes, const int32_t* seq,
                             const int32_t* new_len, const ResizePlan& plan, int i, int tid,
                             int threads) {
  const int start = plan.start[i];
  if (start < 0) return;
  const int s = seq[i], want_len = new_len[i], tail = plan.copied[i], cur = plan.old_len[i];
  const int have = pages_for(cur, shift), want = pages_for(want_len, shift);
  const int first = have - (tail >= 0 ? 1 : 0);        // the copied page's place comes first
  int32_t* row = pg.table + (size_t)s * pg.M;
  for (int j = first + tid; j < want; j += threads) {
    const int p = plan.free_pages[start + j - first];
    pg.refs[p] = 1;
    row[j] = p;
  }
  for (int j = want + tid; j < have; j += threads) {
    const int p = row[j];
    if (p >= 0 && p < pg.P) atomicSub(&pg.refs[p], 1);
    row[j] = -1;
  }
  if (tail >= 0) {
    const int to = plan.free_pages[start];
    const size_t page_bytes = (size_t)row_bytes << shift;
    const uint8_t* src = pg.rows + (size_t)tail * page_bytes;
    uint8_t* dst = pg.rows + (size_t)to * page_bytes;
    const size_t filled = (size_t)(cur & (pg.page - 1)) * row_bytes;   // a multiple of 8
    for (size_t o = 16 * (size_t)tid; o + 16 <= filled; o += 16 * (size_t)threads)
      *reinterpret_cast<uint4*>(dst + o) = *reinterpret_cast<const uint4*>(src + o);
    if (tid == 0 && (filled & 8))
      *reinterpret_cast<uint2*>(dst + filled - 8) = *reinterpret_cast<const uint2*>(src + filled - 8);
    if (tid == 0) atomicSub(&pg.refs[tail], 1);
  }
  if (tid == 0) pg.len[s] = want_len;
}

__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads)
resize_plan_kernel(const fp4_kv_pages pg, int shift, const int32_t* __restrict__ seq,
                   const int32_t* __restrict__ new_len, int n, ResizePlan plan, int* err,
                   int apply_row_bytes) {
  extern __shared__ uint32_t bits[];      // 2 x (S + 31) / 32 words
  __shared__ long long base_need;
  __shared__ long long warp_incl[kPlanThreads / 32];
  pdl_wait_and_release();
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t* seen = bits;
  uint32_t* twice = bits + (pg.S + 31) / 32;
  int lo, hi;
  warp_stretch(rank, pg.P, &lo, &hi);
  const auto is_free = [](int, int r) { return r == 0 ? 1 : 0; };
  const int mine = count_pages(pg.refs, lo, hi, pg.P, is_free);
  long long nfree;
  const long long before = cluster_exclusive(cl, mine, &nfree);

  // every CTA adds up the requests' needs (it must know how many pages are
  // wanted); the first one writes the plan
  mark_twice(seq, n, pg.S, seen, twice);
  if (threadIdx.x == 0) base_need = 0;
  for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    Request r = {false, 0, 0, -1};
    if (i < n) r = read_request(pg, shift, seq, new_len, i, twice);
    // an inclusive sum over the CTA: needs are at most M + 1 each, in 64 bits
    long long incl = r.need;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    __syncthreads();
    if (lane == 31) warp_incl[warp] = incl;
    __syncthreads();
    long long at = base_need;
    for (int w = 0; w < warp; ++w) at += warp_incl[w];
    const long long end = at + incl;
    if (rank == 0 && i < n) {
      const bool fits = r.need == 0 || end <= nfree;
      if (!r.ok) record_error(err, CSA2_ERR_DEVICE_INDEX);
      if (r.ok && !fits) record_error(err, CSA2_ERR_NO_PAGES);
      plan.start[i] = r.ok && fits ? (int)min(end - r.need, (long long)INT_MAX) : -1;
      plan.copied[i] = r.tail;
      plan.old_len[i] = r.cur;
    }
    __syncthreads();
    if (threadIdx.x == kPlanThreads - 1) base_need = end;
  }
  __syncthreads();
  const long long wanted = min(base_need, nfree);
  emit_pages(pg.refs, lo, hi, pg.P, before, wanted, is_free,
             [&](long long k, int p) { plan.free_pages[k] = p; });
  if (apply_row_bytes == 0) return;                    // a launch of its own does the rest
  cl.sync();
  // a warp takes every 256th request's share: four warps to a request
  const int w = rank * (kPlanThreads / 32) + warp;
  for (int i = w >> 2; i < n; i += kPlanWarps / 4)
    resize_apply(pg, shift, apply_row_bytes, seq, new_len, plan, i, (w & 3) * 32 + lane, 128);
}

// One request per blockIdx.x, shared out over gridDim.y CTAs.
__global__ void __launch_bounds__(kThreads)
resize_apply_kernel(const fp4_kv_pages pg, int shift, int row_bytes,
                    const int32_t* __restrict__ seq, const int32_t* __restrict__ new_len,
                    const ResizePlan plan) {
  pdl_wait_and_release();
  resize_apply(pg, shift, row_bytes, seq, new_len, plan, blockIdx.x,
               blockIdx.y * kThreads + threadIdx.x, gridDim.y * kThreads);
}

// ---------------------------------------------------------------- fork
// Workspace: new_len [n] (the source's length, -1: the pair is skipped),
// old_len [n] (the destination's), staged [n][M] (the source's pages).
struct ForkPlan {
  int32_t* new_len;
  int32_t* old_len;
  int32_t* staged;
};

// Whether dst[i] is listed again, as seen by `threads` threads of which this is
// number tid (each answers for its part of the list).
__device__ __forceinline__ bool listed_again(const int32_t* dst, int n, int i, int tid,
                                             int threads) {
  const int d = dst[i];
  bool hit = false;
  for (int k = tid; k < n; k += threads) hit |= k != i && dst[k] == d;
  return hit;
}

// Whether pair i can be carried out, apart from its destination being listed
// again; its lengths.
__device__ __forceinline__ bool read_pair(const fp4_kv_pages& pg, int shift, int a, int b,
                                          int* len, int* old_len) {
  *len = *old_len = 0;
  if (a < 0 || a >= pg.S || b < 0 || b >= pg.S) return false;
  *len = pg.len[a];
  *old_len = pg.len[b];
  const long long most = (long long)pg.M << shift;
  return *len >= 0 && *len <= most && *old_len >= 0 && *old_len <= most;
}

// Reads pair i's source as it is before the call and takes the new references
// (before any is given back, so that no page is free in between). A place of the
// destination that holds the source's page already keeps its reference: branches of
// one prompt, forked again from each other, share most of theirs.
__device__ void fork_stage(const fp4_kv_pages& pg, int shift, int a, int b, bool ok, int len,
                           int old_len, const ForkPlan& plan, int i, int tid, int threads,
                           int* err) {
  if (tid == 0) {
    if (!ok) record_error(err, CSA2_ERR_DEVICE_INDEX);
    plan.new_len[i] = ok ? len : -1;
    plan.old_len[i] = old_len;
  }
  if (!ok) return;
  const int np = pages_for(len, shift), old = pages_for(old_len, shift);
  const int32_t* row = pg.table + (size_t)a * pg.M;
  const int32_t* had = pg.table + (size_t)b * pg.M;
  int32_t* to = plan.staged + (size_t)i * pg.M;
#pragma unroll 4
  for (int j = tid; j < np; j += threads) {
    int p = row[j];
    const int o = j < old ? had[j] : -1;
    if (p < 0 || p >= pg.P) {
      record_error(err, CSA2_ERR_DEVICE_INDEX);
      p = -1;
    } else if (p != o) {
      atomicAdd(&pg.refs[p], 1);
    }
    to[j] = p;
  }
}

__device__ void fork_apply(const fp4_kv_pages& pg, int shift, int b, const ForkPlan& plan, int i,
                           int tid, int threads) {
  const int len = plan.new_len[i];
  if (len < 0) return;
  const int np = pages_for(len, shift), old = pages_for(plan.old_len[i], shift);
  int32_t* row = pg.table + (size_t)b * pg.M;
  const int32_t* from = plan.staged + (size_t)i * pg.M;
#pragma unroll 4
  for (int j = tid; j < max(np, old); j += threads) {
    const int p = j < old ? row[j] : -1, to = j < np ? from[j] : -1;
    if (j < old && p == to) continue;
    if (p >= 0 && p < pg.P) atomicSub(&pg.refs[p], 1);
    row[j] = to;
  }
  if (tid == 0) pg.len[b] = len;
}

// One pair per blockIdx.x, shared out over gridDim.y CTAs.
__global__ void __launch_bounds__(kThreads)
fork_stage_kernel(const fp4_kv_pages pg, int shift, const int32_t* __restrict__ src,
                  const int32_t* __restrict__ dst, int n, const ForkPlan plan, int* err) {
  pdl_wait_and_release();
  const int i = blockIdx.x, a = src[i], b = dst[i];
  int len, old_len;
  bool ok = read_pair(pg, shift, a, b, &len, &old_len);
  ok = __syncthreads_or(listed_again(dst, n, i, threadIdx.x, kThreads)) == 0 && ok;
  fork_stage(pg, shift, a, b, ok, len, old_len, plan, i, blockIdx.y * kThreads + threadIdx.x,
             gridDim.y * kThreads, err);
}

__global__ void __launch_bounds__(kThreads)
fork_apply_kernel(const fp4_kv_pages pg, int shift, const int32_t* __restrict__ dst,
                  const ForkPlan plan) {
  pdl_wait_and_release();
  fork_apply(pg, shift, dst[blockIdx.x], plan, blockIdx.x, blockIdx.y * kThreads + threadIdx.x,
             gridDim.y * kThreads);
}

// Both by one cluster, a warp per pair.
__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads)
fork_small_kernel(const fp4_kv_pages pg, int shift, const int32_t* __restrict__ src,
                  const int32_t* __restrict__ dst, int n, const ForkPlan plan, int* err) {
  pdl_wait_and_release();
  cg::cluster_group cl = cg::this_cluster();
  const int lane = threadIdx.x & 31;
  // (warps in turn over the CTAs, so that few pairs use all of them)
  const int w = (threadIdx.x >> 5) * kPlanCtas + (int)cl.block_rank();
  for (int i = w; i < n; i += kPlanWarps) {
    const int a = src[i], b = dst[i];
    int len, old_len;
    bool ok = read_pair(pg, shift, a, b, &len, &old_len);
    ok = !__any_sync(0xffffffffu, listed_again(dst, n, i, lane, 32)) && ok;
    fork_stage(pg, shift, a, b, ok, len, old_len, plan, i, lane, 32, err);
  }
  cl.sync();
  for (int i = w; i < n; i += kPlanWarps) fork_apply(pg, shift, dst[i], plan, i, lane, 32);
}

// ---------------------------------------------------------------- compact
// Workspace: head [4] (U, moves), move_src [P / 2 + 1], move_dst [P / 2 + 1],
// place [P] (the new place of each used page at U or above, else -1).
struct CompactPlan {
  int32_t* head;
  int32_t* move_src;
  int32_t* move_dst;
  int32_t* place;
};

// U used pages in all. Of the places below U as many are free ("holes") as used
// pages lie at U or above, at most min(U, P - U) <= P / 2: the k-th hole takes the
// k-th of those. One count of used pages per warp's stretch gives all offsets: with
// `before` used pages in front of a stretch that starts at lo, there are lo - before
// holes in front of it if lo <= U, and before - below used pages from U to it if
// lo >= U, below being the used pages under U (the warp whose stretch holds U tells).
__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads)
compact_plan_kernel(const fp4_kv_pages pg, CompactPlan plan, int32_t* used) {
  __shared__ int below_shared;                         // written by one warp of the cluster
  pdl_wait_and_release();
  cg::cluster_group cl = cg::this_cluster();
  const int lane = threadIdx.x & 31;
  int lo, hi;
  warp_stretch((int)cl.block_rank(), pg.P, &lo, &hi);
  const auto in_use = [](int, int r) { return r > 0 ? 1 : 0; };
  long long total;
  const long long before =
      cluster_exclusive(cl, count_pages(pg.refs, lo, hi, pg.P, in_use), &total);
  const int U = (int)total;
  const auto is_hole = [U](int p, int r) { return p < U && r <= 0 ? 1 : 0; };
  const auto is_moved = [U](int p, int r) { return p >= U && r > 0 ? 1 : 0; };
  // (U itself lies in one stretch, or behind the last page when all are used)
  if (lo <= U && U < hi) {
    const auto is_below = [U](int p, int r) { return p < U && r > 0 ? 1 : 0; };
    const int below = (int)before + count_pages(pg.refs, lo, hi, pg.P, is_below);
    if (lane < kPlanCtas) *cl.map_shared_rank(&below_shared, lane) = below;
  }
  cl.sync();
  const int below = U < pg.P ? below_shared : U;
  const int m = U - below;                             // holes, and pages to move
  if (hi > U)
    for (int p = max(lo, U) + lane; p < hi; p += 32) plan.place[p] = -1;
  __syncwarp();
  if (lo < U)
    emit_pages(pg.refs, lo, hi, pg.P, lo - before, m, is_hole,
               [&](long long k, int p) { plan.move_dst[k] = p; });
  if (hi > U)
    emit_pages(pg.refs, lo, hi, pg.P, lo >= U ? before - below : 0, m, is_moved,
               [&](long long k, int p) { plan.move_src[k] = p; });
  // the source and the destination of a move were listed by different warps
  cl.sync();
  for (int k = cl.block_rank() * kPlanThreads + threadIdx.x; k < m;
       k += kPlanCtas * kPlanThreads) {
    const int a = plan.move_src[k], b = plan.move_dst[k];
    plan.place[a] = b;
    pg.refs[b] = pg.refs[a];
    pg.refs[a] = 0;
  }
  if (cl.block_rank() == 0 && threadIdx.x == 0) {
    plan.head[0] = U;
    plan.head[1] = m;
    if (used) *used = U;
  }
}

// Warp 0 of each CTA copies pages, in pieces of at most 16 KB, by bulk copies
// through a ring of shared memory (no page is both read and written: sources lie
// at U or above, destinations below); the other warps rewrite the tables.
// Measured on 16384 pages of 18 KB: 5.7 to 5.9 TB/s read and written (104 us with the
// tables); copies through registers 5.0.
constexpr int kPieceMax = 16384, kStages = 4;
constexpr size_t kCopySmem = (size_t)kStages * kPieceMax;

__global__ void __launch_bounds__(128)
compact_apply_kernel(const fp4_kv_pages pg, long long page_bytes, int pieces, int piece_bytes,
                     const CompactPlan plan, int* err) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[kStages];
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) sm100::mbar_init(&full[i], 1);
    abort_flag = 0;
    sm100::fence_mbar_init();
  }
  pdl_wait_and_release();
  __syncthreads();
  const int U = plan.head[0], m = plan.head[1];
  if (threadIdx.x >= 32) {
    const size_t places = (size_t)pg.S * pg.M;
    const int threads = 96;
    for (size_t k = blockIdx.x * (size_t)threads + threadIdx.x - 32; k < places;
         k += (size_t)gridDim.x * threads) {
      const int p = pg.table[k];
      if (p < U) continue;
      const int to = p < pg.P ? plan.place[p] : -1;
      if (to < 0) record_error(err, CSA2_ERR_DEVICE_INDEX);
      pg.table[k] = to;
    }
    return;
  }
  if (threadIdx.x > 0) return;
  // one thread: piece c of this CTA is number blockIdx.x + c gridDim.x of all
  const long long all = (long long)m * pieces;
  const long long mine = blockIdx.x < all ? (all - blockIdx.x + gridDim.x - 1) / gridDim.x : 0;
  auto where = [&](long long c, size_t* src, size_t* dst) -> uint32_t {
    const long long w = blockIdx.x + c * gridDim.x;
    const long long k = w / pieces, o = (w - k * pieces) * piece_bytes;
    *src = (size_t)plan.move_src[k] * page_bytes + o;
    *dst = (size_t)plan.move_dst[k] * page_bytes + o;
    return (uint32_t)min((long long)piece_bytes, page_bytes - o);
  };
  size_t dst[kStages];
  uint32_t bytes[kStages];
  // a stage is loaded again once the store out of it, kStages - 1 stores back at
  // most, has been read
  auto load = [&](long long c) {
    const int st = (int)(c % kStages);
    size_t src;
    bytes[st] = where(c, &src, &dst[st]);
    sm100::mbar_arrive_expect_tx(&full[st], bytes[st]);
    sm100::bulk_load(ring + st * kPieceMax, pg.rows + src, bytes[st], &full[st]);
  };
  for (long long c = 0; c < mine && c < kStages - 1; ++c) load(c);
  for (long long c = 0; c < mine; ++c) {
    const int st = (int)(c % kStages);
    if (!sm100::mbar_wait(&full[st], (uint32_t)(c / kStages) & 1, &abort_flag)) {
      record_error(err, CSA2_ERR_TIMEOUT);
      // the copies still on their way, for a limited time again
      for (long long d = c; d < mine && d < c + kStages - 1; ++d) {
        abort_flag = 0;
        sm100::mbar_wait(&full[d % kStages], (uint32_t)(d / kStages) & 1, &abort_flag);
      }
      break;
    }
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n\t"
                 "cp.async.bulk.commit_group;" ::"l"(pg.rows + dst[st]),
                 "r"(smem_u32(ring + st * kPieceMax)), "r"(bytes[st])
                 : "memory");
    if (c + kStages - 1 < mine) {
      // the stage that comes free is the one stored before this
      asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
      load(c + kStages - 1);
    }
  }
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

int page_shift(int page) {
  int s = 0;
  while ((1 << s) < page) ++s;
  return s;
}

size_t up4(size_t n) { return (n + 3) / 4 * 4; }   // ints, to 16-byte steps

ResizePlan resize_plan(void* ws, int n) {
  int32_t* w = static_cast<int32_t*>(ws);
  const size_t n4 = up4((size_t)n);
  return {w, w + n4, w + 2 * n4, w + 3 * n4};
}

ForkPlan fork_plan(void* ws, int n) {
  int32_t* w = static_cast<int32_t*>(ws);
  const size_t n4 = up4((size_t)n);
  return {w, w + n4, w + 2 * n4};
}

CompactPlan compact_plan(void* ws, int P) {
  int32_t* w = static_cast<int32_t*>(ws);
  const size_t half = up4((size_t)P / 2 + 1);
  return {w, w + 4, w + 4 + half, w + 4 + 2 * half};
}

int sm_count_of_device() {
  int dev = 0, n = 148;
  if (cudaGetDevice(&dev) == cudaSuccess)
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n;
}

// The copy kernel's shared memory, allowed once per device.
cudaError_t allow_copy_ring() {
  static std::mutex mu;
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (done[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(compact_apply_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)kCopySmem);
  done[dev] = e == cudaSuccess;
  return e;
}

}  // namespace

size_t pages_resize_workspace_bytes(const fp4_kv_pages& pg, int n) {
  const size_t most = (size_t)n * ((size_t)pg.M + 1);
  return 4 * (3 * up4((size_t)n) + (most < (size_t)pg.P ? most : (size_t)pg.P));
}

size_t pages_fork_workspace_bytes(const fp4_kv_pages& pg, int n) {
  return 4 * (2 * up4((size_t)n) + (size_t)n * pg.M);
}

size_t pages_compact_workspace_bytes(const fp4_kv_pages& pg) {
  return 4 * (4 + 2 * up4((size_t)pg.P / 2 + 1) + (size_t)pg.P);
}

cudaError_t launch_pages_resize(const fp4_kv_pages& pg, const int32_t* seq, const int32_t* new_len,
                                int n, void* workspace, int* err, cudaStream_t stream) {
  if (n == 0) return cudaSuccess;
  const int shift = page_shift(pg.page), row_bytes = pg.D / 2 + pg.D / 16;
  const ResizePlan plan = resize_plan(workspace, n);
  const size_t smem = 2 * (size_t)((pg.S + 31) / 32) * 4;
  const size_t page_bytes = (size_t)row_bytes << shift;
  // little to do at most: the planning cluster does it
  const bool small = (size_t)n * (page_bytes + 8 * (size_t)pg.M) <= (1 << 20);
  cudaError_t e = launch_pdl(resize_plan_kernel, dim3(kPlanCtas), dim3(kPlanThreads), smem, stream,
                             dim3(1), pg, shift, seq, new_len, n, plan, err,
                             small ? row_bytes : 0);
  if (e != cudaSuccess || small) return e;
  // a copied page of more than 16 KB is shared out, as far as the GPU has room
  int parts = (int)((page_bytes + 16383) / 16384);
  parts = max(1, min(parts, 8 * sm_count_of_device() / n));
  return launch_pdl(resize_apply_kernel, dim3(n, parts), dim3(kThreads), 0, stream, dim3(1), pg,
                    shift, row_bytes, seq, new_len, plan);
}

cudaError_t launch_pages_fork(const fp4_kv_pages& pg, const int32_t* src, const int32_t* dst,
                              int n, void* workspace, int* err, cudaStream_t stream) {
  if (n == 0) return cudaSuccess;
  const int shift = page_shift(pg.page);
  const ForkPlan plan = fork_plan(workspace, n);
  // little to do at most: one cluster does both steps
  if ((size_t)n * pg.M <= 16384)
    return launch_pdl(fork_small_kernel, dim3(kPlanCtas), dim3(kPlanThreads), 0, stream, dim3(1),
                      pg, shift, src, dst, n, plan, err);
  int parts = ceil_div(pg.M, 4 * kThreads);
  parts = max(1, min(parts, 8 * sm_count_of_device() / n));
  cudaError_t e = launch_pdl(fork_stage_kernel, dim3(n, parts), dim3(kThreads), 0, stream, dim3(1),
                             pg, shift, src, dst, n, plan, err);
  if (e != cudaSuccess) return e;
  return launch_pdl(fork_apply_kernel, dim3(n, parts), dim3(kThreads), 0, stream, dim3(1), pg,
                    shift, dst, plan);
}

cudaError_t launch_pages_compact(const fp4_kv_pages& pg, int32_t* used, void* workspace, int* err,
                                 cudaStream_t stream) {
  const CompactPlan plan = compact_plan(workspace, pg.P);
  const long long page_bytes = (long long)pg.page * (pg.D / 2 + pg.D / 16);
  cudaError_t e = launch_pdl(compact_plan_kernel, dim3(kPlanCtas), dim3(kPlanThreads), 0, stream,
                             dim3(1), pg, plan, used);
  if (e != cudaSuccess) return e;
  e = allow_copy_ring();
  if (e != cudaSuccess) return e;
  // pieces of a page: equal ones, of whole 16-byte words
  const int pieces = (int)((page_bytes + kPieceMax - 1) / kPieceMax);
  const int piece_bytes = (int)((page_bytes / 16 + pieces - 1) / pieces) * 16;
  return launch_pdl(compact_apply_kernel, dim3(3 * sm_count_of_device()), dim3(128), kCopySmem,
                    stream, dim3(1), pg, page_bytes, pieces, piece_bytes, plan, err);
}

}  // namespace csa2
