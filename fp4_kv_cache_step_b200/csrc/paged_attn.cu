// paged_attn.cu -- attention over the paged FP4 cache (csa2_paged_attn). Without
// a list the kernel of paged_attn_tc.cu walks the pages. With one, the listed
// entries become rows of the whole pool (page from the table * page size +
// offset), and the attention over the 16-channel layout runs over that list with
// the pool as one sequence.
#include "common.cuh"
#include "kernels.h"

namespace csa2 {
namespace {

constexpr int kThreads = 256;

// Visible entries of query (b, t) of slot s: nvalid, or the slot's length.
__device__ __forceinline__ int visible(const fp4_kv_pages& pg, int s, const int32_t* nvalid,
                                       size_t row, int* err) {
  if (s < 0 || s >= pg.S) {
    record_error(err, CSA2_ERR_DEVICE_INDEX);
    return 0;
  }
  const int len = min(max(0, pg.len[s]), pg.M * pg.page);
  if (nvalid == nullptr) return len;
  const int n = nvalid[row];
  if (n < 0 || n > len) record_error(err, CSA2_ERR_DEVICE_INDEX);
  return min(max(0, n), len);
}

// list[row][i] = the pool row of entry ids[row][i], or -1.
__global__ void __launch_bounds__(kThreads)
list_rows_kernel(const fp4_kv_pages pg, int shift, const int32_t* __restrict__ seq,
                 const int32_t* __restrict__ nvalid, const int32_t* __restrict__ ids, int Tq, int K,
                 int32_t* __restrict__ list, int* err) {
  pdl_wait_and_release();
  const size_t row = blockIdx.x;
  const int b = (int)(row / Tq);
  const int s = seq ? seq[b] : b;
  const int n = visible(pg, s, nvalid, row, err);
  for (int i = blockIdx.y * kThreads + threadIdx.x; i < K; i += gridDim.y * kThreads) {
    const int e = ids[row * K + i];
    int at = -1;
    if (e < -1 || e >= n) {
      record_error(err, CSA2_ERR_DEVICE_INDEX);
    } else if (e >= 0) {
      const int p = pg.table[(size_t)s * pg.M + (e >> shift)];
      if (p < 0 || p >= pg.P)
        record_error(err, CSA2_ERR_DEVICE_INDEX);
      else
        at = (p << shift) + (e & (pg.page - 1));
    }
    list[row * K + i] = at;
  }
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

size_t paged_attn_workspace_bytes(const fp4_kv_pages& pg, int B, int Tq, int Hq, int K) {
  if (K == 0) return paged_attn_dense_workspace_bytes(pg, B, Tq, Hq);
  return up256((size_t)B * Tq * K * 4) + sparse_attn_workspace_bytes(1, B * Tq, Hq, K);
}

cudaError_t launch_paged_attn(const uint16_t* q, const fp4_kv_pages& pg, const int32_t* seq,
                              const int32_t* nvalid, const int32_t* topk_idx, int B, int Tq,
                              int Hq, int K, float softmax_scale, uint16_t* out, float* lse,
                              void* workspace, int* err, cudaStream_t stream) {
  if (B == 0 || Tq == 0) return cudaSuccess;
  if (topk_idx == nullptr)
    return launch_paged_attn_dense(q, pg, seq, nvalid, B, Tq, Hq, softmax_scale, out, lse,
                                   workspace, err, stream);
  int shift = 0;
  while ((1 << shift) < pg.page) ++shift;
  int32_t* list = static_cast<int32_t*>(workspace);
  const int parts = max(1, min(ceil_div(K, 4 * kThreads), 65535));
  cudaError_t e = launch_pdl(list_rows_kernel, dim3(B * Tq, parts), dim3(kThreads), 0, stream,
                             dim3(1), pg, shift, seq, nvalid, topk_idx, Tq, K, list, err);
  if (e != cudaSuccess) return e;
  unsigned char* rest = static_cast<unsigned char*>(workspace) + up256((size_t)B * Tq * K * 4);
  return launch_sparse_attn(q, pg.rows, nullptr, list, 1, B * Tq, Hq, pg.P * pg.page, K,
                            softmax_scale, out, lse, rest, err, stream);
}

}  // namespace csa2
