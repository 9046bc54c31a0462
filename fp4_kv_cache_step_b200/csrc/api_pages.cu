// api_pages.cu -- the exported calls of the paged FP4 cache (include/csa2.h):
// argument checks, and the host-side rotation frequencies.
#include <cmath>
#include <cstdio>

#include "common.cuh"
#include "kernels.h"

namespace {

bool aligned(const void* p, size_t n) {
  return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

#define CHECK_ARG(cond, ...)                                  \
  do {                                                        \
    if (!(cond)) {                                            \
      char buf[256];                                          \
      std::snprintf(buf, sizeof buf, __VA_ARGS__);            \
      return csa2::api_fail(CSA2_ERR_INVALID_ARG, buf);       \
    }                                                         \
  } while (0)

#define CHECK_PTR(p) \
  CHECK_ARG(aligned((p), 16), "%s must be a non-null 16-byte aligned device pointer", #p)
#define CHECK_PTR4(p) \
  CHECK_ARG(aligned((p), 4), "%s must be a non-null 4-byte aligned device pointer", #p)

csa2_status check_pages(const fp4_kv_pages* pages) {
  CHECK_ARG(pages != nullptr, "pages must be non-null");
  CHECK_PTR(pages->rows);
  CHECK_PTR(pages->table);
  CHECK_PTR(pages->len);
  CHECK_PTR(pages->refs);
  CHECK_ARG(pages->page >= 8 && pages->page <= 65536 && (pages->page & (pages->page - 1)) == 0,
            "page=%d must be a power of two in [8, 65536]", pages->page);
  CHECK_ARG(pages->D > 0 && pages->D % 128 == 0 && pages->D <= 1024,
            "D=%d must be a multiple of 128 in [128, 1024]", pages->D);
  CHECK_ARG(pages->S >= 1 && pages->S <= 65536, "S=%d must be in [1, 65536]", pages->S);
  CHECK_ARG(pages->M >= 1 && (long long)pages->M * pages->page < (1ll << 31),
            "M=%d must be >= 1 and M * page below 2^31", pages->M);
  CHECK_ARG(pages->P >= 1 && (long long)pages->P * pages->page < (1ll << 31),
            "P=%d must be >= 1 and P * page below 2^31", pages->P);
  return CSA2_OK;
}

csa2_status check_workspace(const void* ws, size_t got, size_t need, const char* what) {
  if (need > 0 && (!aligned(ws, 16) || got < need)) {
    char buf[160];
    std::snprintf(buf, sizeof buf, "%s needs %zu workspace bytes (got %zu)", what, need, got);
    return csa2::api_fail(CSA2_ERR_WORKSPACE, buf);
  }
  return CSA2_OK;
}

size_t round_up(size_t x) { return (x + 255) / 256 * 256; }

// Enters the stream's device and runs `launch(error word)`.
template <typename Launch>
csa2_status run(csa2_stream_t stream, const char* what, Launch launch) {
  cudaError_t e;
  csa2::DeviceScope scope;
  int* err = csa2::api_error_word((cudaStream_t)stream, scope, &e);
  if (!err) return csa2::api_cuda_fail(e, what);
  e = launch(err);
  if (e != cudaSuccess) return csa2::api_cuda_fail(e, what);
  return csa2::api_ok();
}

}  // namespace

extern "C" {

size_t fp4_kv_pages_resize_workspace_bytes(const fp4_kv_pages* pages, int n) {
  if (!pages || n <= 0) return 0;
  return round_up(csa2::pages_resize_workspace_bytes(*pages, n));
}

csa2_status fp4_kv_pages_resize(const fp4_kv_pages* pages, const int32_t* seq,
                                const int32_t* new_len, int n, void* workspace,
                                size_t workspace_bytes, csa2_stream_t stream) {
  csa2_status s = check_pages(pages);
  if (s != CSA2_OK) return s;
  CHECK_ARG(n >= 0 && n <= 65536, "n=%d must be in [0, 65536]", n);
  if (n == 0) return csa2::api_ok();
  CHECK_PTR4(seq);
  CHECK_PTR4(new_len);
  s = check_workspace(workspace, workspace_bytes, fp4_kv_pages_resize_workspace_bytes(pages, n),
                      "fp4_kv_pages_resize");
  if (s != CSA2_OK) return s;
  return run(stream, "fp4_kv_pages_resize", [&](int* err) {
    return csa2::launch_pages_resize(*pages, seq, new_len, n, workspace, err,
                                     (cudaStream_t)stream);
  });
}

size_t fp4_kv_pages_fork_workspace_bytes(const fp4_kv_pages* pages, int n) {
  if (!pages || n <= 0) return 0;
  return round_up(csa2::pages_fork_workspace_bytes(*pages, n));
}

csa2_status fp4_kv_pages_fork(const fp4_kv_pages* pages, const int32_t* src, const int32_t* dst,
                              int n, void* workspace, size_t workspace_bytes,
                              csa2_stream_t stream) {
  csa2_status s = check_pages(pages);
  if (s != CSA2_OK) return s;
  CHECK_ARG(n >= 0 && n <= 65536, "n=%d must be in [0, 65536]", n);
  if (n == 0) return csa2::api_ok();
  CHECK_PTR4(src);
  CHECK_PTR4(dst);
  s = check_workspace(workspace, workspace_bytes, fp4_kv_pages_fork_workspace_bytes(pages, n),
                      "fp4_kv_pages_fork");
  if (s != CSA2_OK) return s;
  return run(stream, "fp4_kv_pages_fork", [&](int* err) {
    return csa2::launch_pages_fork(*pages, src, dst, n, workspace, err, (cudaStream_t)stream);
  });
}

size_t fp4_kv_pages_compact_workspace_bytes(const fp4_kv_pages* pages) {
  if (!pages || pages->P <= 0) return 0;
  return round_up(csa2::pages_compact_workspace_bytes(*pages));
}

csa2_status fp4_kv_pages_compact(const fp4_kv_pages* pages, int32_t* used, void* workspace,
                                 size_t workspace_bytes, csa2_stream_t stream) {
  csa2_status s = check_pages(pages);
  if (s != CSA2_OK) return s;
  if (used) CHECK_PTR4(used);
  s = check_workspace(workspace, workspace_bytes, fp4_kv_pages_compact_workspace_bytes(pages),
                      "fp4_kv_pages_compact");
  if (s != CSA2_OK) return s;
  return run(stream, "fp4_kv_pages_compact", [&](int* err) {
    return csa2::launch_pages_compact(*pages, used, workspace, err, (cudaStream_t)stream);
  });
}

csa2_status csa2_rope_turns(int R, double base, csa2_rope_scaling scaling, double factor,
                            double context, double fast, double slow, uint64_t* turns) {
  CHECK_ARG(R >= 0 && R <= 1024 && R % 2 == 0, "R=%d must be even, in [0, 1024]", R);
  CHECK_ARG(std::isfinite(base) && base > 1.0, "base=%g must be > 1", base);
  CHECK_ARG(scaling >= CSA2_ROPE_PLAIN && scaling <= CSA2_ROPE_YARN, "unknown scaling %d",
            (int)scaling);
  CHECK_ARG(std::isfinite(factor) && factor >= 1.0, "factor=%g must be >= 1", factor);
  CHECK_ARG(scaling != CSA2_ROPE_NTK || R == 0 || R > 2, "NTK scaling needs R=%d above 2", R);
  CHECK_ARG(scaling != CSA2_ROPE_YARN ||
                (std::isfinite(context) && context > 0.0 && std::isfinite(fast) &&
                 std::isfinite(slow) && fast > slow),
            "YARN scaling needs context=%g > 0 and fast=%g > slow=%g", context, fast, slow);
  CHECK_ARG(R == 0 || turns != nullptr, "turns must be a non-null host pointer");
  const double two_pi = 6.283185307179586476925286766559;
  const double b = scaling == CSA2_ROPE_NTK && R > 2 ? base * std::pow(factor, R / (R - 2.0)) : base;
  for (int i = 0; i < R / 2; ++i) {
    double theta = std::pow(b, -2.0 * i / R);
    if (scaling == CSA2_ROPE_LINEAR) theta /= factor;
    if (scaling == CSA2_ROPE_YARN) {
      const double r = context * theta / two_pi;
      double g = (r - slow) / (fast - slow);
      g = g < 0.0 ? 0.0 : g > 1.0 ? 1.0 : g;
      theta = (1.0 - g) * theta / factor + g * theta;
    }
    // theta <= 1, so the fraction is below 0.16
    turns[i] = (uint64_t)std::nearbyint(std::ldexp(theta / two_pi, 64));
  }
  return csa2::api_ok();
}

csa2_status csa2_qk_norm_rope(const csa2_norm_rope_args* args, const fp4_kv_pages* pages,
                              csa2_stream_t stream) {
  CHECK_ARG(args != nullptr, "args must be non-null");
  const csa2_norm_rope_args& a = *args;
  CHECK_ARG(a.D > 0 && a.D % 128 == 0 && a.D <= 1024,
            "D=%d must be a multiple of 128 in [128, 1024]", a.D);
  CHECK_ARG(a.R >= 0 && a.R % 2 == 0 && a.rot_begin >= 0 && a.rot_begin <= a.D - a.R,
            "R=%d must be even and the rotary part [%d, %d + R) inside [0, D)", a.R, a.rot_begin,
            a.rot_begin);
  CHECK_ARG(a.R == 0 || aligned(a.turns, 8),
            "turns must be a non-null 8-byte aligned device pointer");
  CHECK_ARG(a.T >= 0 && a.E >= 0, "T=%d and E=%d must be >= 0", a.T, a.E);
  CHECK_ARG(a.eps >= 0.0f, "eps must be >= 0");
  if (a.T > 0) {
    CHECK_ARG(a.Hq >= 1 && a.Hq <= 65535, "Hq=%d must be in [1, 65535]", a.Hq);
    CHECK_PTR(a.q);
    CHECK_PTR(a.q_out);
    CHECK_PTR4(a.pos);
    if (a.q_norm && a.q_weight) CHECK_PTR4(a.q_weight);
    const long long width = (long long)a.Hq * a.D;
    CHECK_ARG(a.q_stride >= width && a.q_stride % (a.q_f32 ? 4 : 8) == 0,
              "q_stride=%lld must be >= Hq * D and a multiple of 16 bytes", a.q_stride);
    // in place, or apart: a head is read whole before it is written
    const char* in = static_cast<const char*>(a.q);
    const char* out = reinterpret_cast<const char*>(a.q_out);
    const long long in_bytes = ((a.T - 1) * a.q_stride + width) * (a.q_f32 ? 4 : 2);
    const bool in_place = in == out && !a.q_f32 && a.q_stride == width;
    CHECK_ARG(in_place || in + in_bytes <= out || out + a.T * width * 2 <= in,
              "q_out must be q itself (bf16, contiguous) or lie apart from it");
  }
  if (a.E > 0) {
    csa2_status s = check_pages(pages);
    if (s != CSA2_OK) return s;
    CHECK_ARG(pages->D == a.D, "pages->D=%d must be D=%d", pages->D, a.D);
    CHECK_PTR(a.kv);
    CHECK_PTR4(a.kv_pos);
    CHECK_PTR4(a.seq);
    CHECK_PTR4(a.entry);
    if (a.kv_norm && a.kv_weight) CHECK_PTR4(a.kv_weight);
    if (a.kv_out) CHECK_PTR(a.kv_out);
    CHECK_ARG(a.kv_stride >= a.D && a.kv_stride % (a.kv_f32 ? 4 : 8) == 0,
              "kv_stride=%lld must be >= D and a multiple of 16 bytes", a.kv_stride);
  }
  CHECK_ARG((long long)a.E + (a.T > 0 ? (long long)a.T * ((a.Hq + 7) / 8) : 0) <= 0x7fffffffll,
            "too many rows for one call");
  return run(stream, "csa2_qk_norm_rope", [&](int* err) {
    return csa2::launch_qk_norm_rope(a, a.E > 0 ? pages : nullptr, err, (cudaStream_t)stream);
  });
}

size_t csa2_paged_attn_workspace_bytes(const fp4_kv_pages* pages, int B, int Tq, int Hq, int K) {
  if (!pages || B <= 0 || Tq <= 0 || Hq <= 0 || K < 0) return 0;
  return round_up(csa2::paged_attn_workspace_bytes(*pages, B, Tq, Hq, K));
}

csa2_status csa2_paged_attn(const uint16_t* q, const fp4_kv_pages* pages, const int32_t* seq,
                            const int32_t* nvalid, const int32_t* topk_idx, int B, int Tq, int Hq,
                            int K, float softmax_scale, uint16_t* out, float* lse, void* workspace,
                            size_t workspace_bytes, csa2_stream_t stream) {
  csa2_status s = check_pages(pages);
  if (s != CSA2_OK) return s;
  if (pages->D != csa2::kHeadDim)
    return csa2::api_fail(CSA2_ERR_UNSUPPORTED, "attention is built for D=512 only");
  CHECK_ARG(B >= 0 && B <= 65535 && Tq >= 0, "B=%d must be in [0, 65535] and Tq=%d >= 0", B, Tq);
  CHECK_ARG(Hq >= 1 && (long long)Tq * Hq <= 65535, "Hq=%d must be >= 1 and Tq * Hq <= 65535", Hq);
  CHECK_ARG((long long)B * Tq < (1ll << 31), "B * Tq must be below 2^31");
  if (B == 0 || Tq == 0) return csa2::api_ok();
  CHECK_PTR(q);
  CHECK_PTR(out);
  CHECK_ARG(seq != nullptr || B <= pages->S, "B=%d rows need as many slots (S=%d)", B, pages->S);
  if (seq) CHECK_PTR4(seq);
  if (nvalid) CHECK_PTR4(nvalid);
  if (lse) CHECK_PTR4(lse);
  if (topk_idx) {
    CHECK_PTR4(topk_idx);
    CHECK_ARG(K >= 1 && K <= (1 << 30), "K=%d must be in [1, 2^30]", K);
  } else {
    K = 0;
  }
  // sized on the stream's device, as the launch plans it
  csa2::DeviceScope scope;
  const cudaError_t se = scope.enter((cudaStream_t)stream);
  s = check_workspace(workspace, workspace_bytes,
                      csa2_paged_attn_workspace_bytes(pages, B, Tq, Hq, K), "csa2_paged_attn");
  if (s != CSA2_OK) return s;
  if (se != cudaSuccess) return csa2::api_cuda_fail(se, "csa2_paged_attn device");
  return run(stream, "csa2_paged_attn", [&](int* err) {
    return csa2::launch_paged_attn(q, *pages, seq, nvalid, topk_idx, B, Tq, Hq, K, softmax_scale,
                                   out, lse, workspace, err, (cudaStream_t)stream);
  });
}

}  // extern "C"
