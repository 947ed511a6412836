// C ABI of the rotation of Q and K, and of their norm with the rotation (declared in include/sageattn.h): argument
// validation and kernel launches.  No allocation happens here.
#include <cmath>

#include "../../include/sageattn.h"
#include "api_checks.h"
#include "api_overlap.h"
#include "kernels.h"

using namespace sa::api;

namespace {

// Element strides of [B, S, H, N] rows; 0 (the same row again) only where a tensor is read.
attn_status rope_rows(const char* name, const void* ptr, int type, const int64_t* in, int B, int S, int H, bool read,
                      long long out[3]) {
  if (ptr == nullptr) return fail(ATTN_ERR_INVALID_ARG, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(ptr) % (type == ATTN_F32 ? 4 : 2) != 0)
    return fail(ATTN_ERR_ALIGNMENT, "%s is not aligned to its type", name);
  if (in == nullptr) return fail(ATTN_ERR_INVALID_ARG, "%s strides are NULL", name);
  const int ext[3] = {B, S, H};
  for (int i = 0; i < 3; ++i) {
    const long long s = ext[i] == 1 ? 0 : in[i];
    if (s < 0 || (s == 0 && ext[i] > 1 && !read) || s >= (1ll << 38))
      return fail(ATTN_ERR_INVALID_ARG, "%s stride %lld of dimension %d is out of range", name, (long long)in[i], i);
    out[i] = s;
  }
  return ATTN_OK;
}

// Sizes, positions and frequencies; *empty where there are no rows.
attn_status rope_sizes(int B, int S, int Hq, int Hk, int N, const int32_t* pos, const int64_t* pos_str, int axes,
                       const uint64_t* freq, int rope_dim, int interleaved, float magnitude, int dtype, sa::RopeArgs& a,
                       bool* empty) {
  *empty = false;
  if (dtype < ATTN_BF16 || dtype > ATTN_F32) return fail(ATTN_ERR_INVALID_ARG, "dtype=%d is none of attn_dtype", dtype);
  if (B < 0 || S < 0 || Hq < 0 || Hk < 0)
    return fail(ATTN_ERR_INVALID_ARG, "B=%d S=%d Hq=%d Hk=%d must be >= 0", B, S, Hq, Hk);
  if (N < 1 || N > 512) return fail(ATTN_ERR_INVALID_ARG, "N=%d must be in [1, 512]", N);
  if (rope_dim < 0 || rope_dim > N || rope_dim % 2 != 0)
    return fail(ATTN_ERR_INVALID_ARG, "rope_dim=%d must be even and in [0, N=%d]", rope_dim, N);
  if (interleaved != 0 && interleaved != 1) return fail(ATTN_ERR_INVALID_ARG, "interleaved=%d must be 0 or 1", interleaved);
  if (!std::isfinite(magnitude)) return fail(ATTN_ERR_INVALID_ARG, "magnitude is not finite");
  const long long bs = (long long)B * S, heads = (long long)Hq + Hk;
  if (bs > (1ll << 30) || heads > (1ll << 30) || bs * heads > (1ll << 30))
    return fail(ATTN_ERR_INVALID_ARG, "B*S*(Hq+Hk) must be at most 2^30 rows");
  a.B = B;
  a.S = S;
  a.N = N;
  a.R = rope_dim;
  a.type = dtype;
  a.interleaved = interleaved;
  a.magnitude = magnitude;
  a.inverse = 0;
  a.eps = 0.0f;
  a.w_type = dtype;
  for (auto& s : a.side) s = {};
  a.side[0].H = Hq;
  a.side[1].H = Hk;
  if (bs * heads == 0) {
    *empty = true;
    return ATTN_OK;
  }
  a.freq = reinterpret_cast<const unsigned long long*>(freq);
  a.pos = pos;
  a.axes = pos != nullptr ? axes : 1;
  for (int i = 0; i < 3; ++i) a.pos_str[i] = 0;
  if (rope_dim == 0) return ATTN_OK;
  if (freq == nullptr) return fail(ATTN_ERR_INVALID_ARG, "freq is NULL");
  if (reinterpret_cast<uintptr_t>(freq) % 8 != 0) return fail(ATTN_ERR_ALIGNMENT, "freq is not 8-byte aligned");
  if (pos == nullptr) return ATTN_OK;
  if (reinterpret_cast<uintptr_t>(pos) % 4 != 0) return fail(ATTN_ERR_ALIGNMENT, "pos is not 4-byte aligned");
  if (axes < 1 || axes > 4) return fail(ATTN_ERR_INVALID_ARG, "axes=%d must be in [1, 4]", axes);
  if (pos_str == nullptr) return fail(ATTN_ERR_INVALID_ARG, "pos strides are NULL");
  const int ext[3] = {B, S, axes};
  for (int i = 0; i < 3; ++i) {
    if (ext[i] > 1 && (pos_str[i] < 0 || pos_str[i] >= (1ll << 38)))
      return fail(ATTN_ERR_INVALID_ARG, "pos stride %lld of dimension %d is out of range", (long long)pos_str[i], i);
    a.pos_str[i] = ext[i] > 1 ? pos_str[i] : 0;
  }
  return ATTN_OK;
}

// One side's tensors: y may be x or dy itself, and overlaps no other tensor.
attn_status rope_side(sa::RopeArgs& a, int i, const char* const names[3], const void* x, const int64_t* x_str,
                      const void* dy, const int64_t* dy_str, void* y, const int64_t* y_str, bool backward) {
  sa::RopeArgs::Side& s = a.side[i];
  if (s.H == 0) return ATTN_OK;
  TRY(rope_rows(names[0], x, a.type, x_str, a.B, a.S, s.H, true, s.x_str));
  if (backward) TRY(rope_rows(names[1], dy, a.type, dy_str, a.B, a.S, s.H, true, s.dy_str));
  TRY(rope_rows(names[2], y, a.type, y_str, a.B, a.S, s.H, false, s.y_str));
  s.x = x;
  s.dy = backward ? dy : nullptr;
  s.y = y;
  return ATTN_OK;
}
attn_status rope_overlap(const char* who, const sa::RopeArgs& a) {
  const int size = a.type == ATTN_F32 ? 4 : 2;
  auto rows = [&](int i, const void* ptr, const long long* str) { return rows_of(ptr, a.B, a.S, a.side[i].H, a.N, size, str); };
  for (int i = 0; i < 2; ++i) {
    if (a.side[i].H == 0) continue;
    const Rows y = rows(i, a.side[i].y, a.side[i].y_str);
    for (int j = 0; j < 2; ++j) {
      const sa::RopeArgs::Side& s = a.side[j];
      if (s.H == 0) continue;
      const Rows x = rows(j, s.x, s.x_str);
      bool bad = share_memory(y, x) && !(i == j && same(y, x));
      if (s.dy != nullptr) {
        const Rows dy = rows(j, s.dy, s.dy_str);
        bad = bad || (share_memory(y, dy) && !(i == j && same(y, dy)));
      }
      if (j > i) bad = bad || share_memory(y, rows(j, s.y, s.y_str));
      if (bad)
        return fail(ATTN_ERR_INVALID_ARG, "%s: an output must be its own input itself or overlap no tensor", who);
    }
  }
  return ATTN_OK;
}

attn_status rope_weights(sa::RopeArgs& a, const void* qw, const void* kw, float eps, int w_dtype) {
  if (!(eps >= 0.0f && std::isfinite(eps))) return fail(ATTN_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (w_dtype != a.type && w_dtype != ATTN_F32)
    return fail(ATTN_ERR_INVALID_ARG, "w_dtype=%d must be the rows' type or ATTN_F32", w_dtype);
  const uintptr_t align = w_dtype == ATTN_F32 ? 4 : 2;
  const void* const w[2] = {qw, kw};
  for (int i = 0; i < 2; ++i) {
    if (a.side[i].H == 0) continue;   // (nothing of that side is looked at)
    if (reinterpret_cast<uintptr_t>(w[i]) % align != 0)
      return fail(ATTN_ERR_ALIGNMENT, "a weight is not aligned to its type");
    a.side[i].w = w[i];
  }
  a.eps = eps;
  a.w_type = w_dtype;
  return ATTN_OK;
}

attn_status rope_either(const char* who, int inverse, const void* q, const void* k, void* q_out, void* k_out, int B,
                        int S, int Hq, int Hk, int N, const int64_t* q_str, const int64_t* k_str, const int64_t* qo_str,
                        const int64_t* ko_str, const int32_t* pos, const int64_t* pos_str, int axes,
                        const uint64_t* freq, int rope_dim, int interleaved, float magnitude, int dtype,
                        attn_stream_t stream) {
  static const char* const names[2][3] = {{"q", "", "q_out"}, {"k", "", "k_out"}};
  bool empty = false;
  sa::RopeArgs a;
  TRY(rope_sizes(B, S, Hq, Hk, N, pos, pos_str, axes, freq, rope_dim, interleaved, magnitude, dtype, a, &empty));
  if (empty) return ATTN_OK;
  a.inverse = inverse;
  TRY(rope_side(a, 0, names[0], q, q_str, nullptr, nullptr, q_out, qo_str, false));
  TRY(rope_side(a, 1, names[1], k, k_str, nullptr, nullptr, k_out, ko_str, false));
  TRY(rope_overlap(who, a));
  TRY(check_device());
  const cudaError_t e = sa::launch_rope_fwd(a, false, (cudaStream_t)stream);
  if (e != cudaSuccess) return fail_cuda(e, who);
  return ATTN_OK;
}

}  // namespace

extern "C" {

attn_status rope_fwd(const void* q, const void* k, void* q_out, void* k_out, int B, int S, int Hq, int Hk, int N,
                     const int64_t q_str[3], const int64_t k_str[3], const int64_t qo_str[3], const int64_t ko_str[3],
                     const int32_t* pos, const int64_t pos_str[3], int axes, const uint64_t* freq, int rope_dim,
                     int interleaved, float magnitude, int dtype, attn_stream_t stream) {
  return rope_either("rope_fwd", 0, q, k, q_out, k_out, B, S, Hq, Hk, N, q_str, k_str, qo_str, ko_str, pos, pos_str, axes,
                     freq, rope_dim, interleaved, magnitude, dtype, stream);
}

attn_status rope_bwd(const void* dq_out, const void* dk_out, void* dq, void* dk, int B, int S, int Hq, int Hk, int N,
                     const int64_t dqo_str[3], const int64_t dko_str[3], const int64_t dq_str[3], const int64_t dk_str[3],
                     const int32_t* pos, const int64_t pos_str[3], int axes, const uint64_t* freq, int rope_dim,
                     int interleaved, float magnitude, int dtype, attn_stream_t stream) {
  return rope_either("rope_bwd", 1, dq_out, dk_out, dq, dk, B, S, Hq, Hk, N, dqo_str, dko_str, dq_str, dk_str, pos,
                     pos_str, axes, freq, rope_dim, interleaved, magnitude, dtype, stream);
}

attn_status qk_norm_rope_fwd(const void* q, const void* k, const void* q_weight, const void* k_weight, void* q_out,
                             void* k_out, int B, int S, int Hq, int Hk, int N, const int64_t q_str[3],
                             const int64_t k_str[3], const int64_t qo_str[3], const int64_t ko_str[3], float eps,
                             const int32_t* pos, const int64_t pos_str[3], int axes, const uint64_t* freq, int rope_dim,
                             int interleaved, float magnitude, int dtype, int w_dtype, attn_stream_t stream) {
  static const char* const names[2][3] = {{"q", "", "q_out"}, {"k", "", "k_out"}};
  bool empty = false;
  sa::RopeArgs a;
  TRY(rope_sizes(B, S, Hq, Hk, N, pos, pos_str, axes, freq, rope_dim, interleaved, magnitude, dtype, a, &empty));
  TRY(rope_weights(a, q_weight, k_weight, eps, w_dtype));
  if (empty) return ATTN_OK;
  TRY(rope_side(a, 0, names[0], q, q_str, nullptr, nullptr, q_out, qo_str, false));
  TRY(rope_side(a, 1, names[1], k, k_str, nullptr, nullptr, k_out, ko_str, false));
  TRY(rope_overlap("qk_norm_rope_fwd", a));
  TRY(check_device());
  const cudaError_t e = sa::launch_rope_fwd(a, true, (cudaStream_t)stream);
  if (e != cudaSuccess) return fail_cuda(e, "qk_norm_rope_fwd");
  return ATTN_OK;
}

size_t qk_norm_rope_bwd_workspace_size(int B, int S, int Hq, int Hk, int N) {
  if (B < 1 || S < 1 || Hq < 0 || Hk < 0 || N < 1 || N > 512) return 0;
  const long long bs = (long long)B * S, heads = (long long)Hq + Hk;
  if (heads == 0 || bs > (1ll << 30) || heads > (1ll << 30) || bs * heads > (1ll << 30)) return 0;
  return (size_t)2 * sa::rope_bwd_ctas(B, S, Hq, Hk) * N * sizeof(float);
}

attn_status qk_norm_rope_bwd(const void* dq_out, const void* dk_out, const void* q, const void* k, const void* q_weight,
                             const void* k_weight, void* dq, void* dk, void* dq_weight, void* dk_weight, int B, int S,
                             int Hq, int Hk, int N, const int64_t dqo_str[3], const int64_t dko_str[3],
                             const int64_t q_str[3], const int64_t k_str[3], const int64_t dq_str[3],
                             const int64_t dk_str[3], float eps, const int32_t* pos, const int64_t pos_str[3], int axes,
                             const uint64_t* freq, int rope_dim, int interleaved, float magnitude, int dtype, int w_dtype,
                             void* workspace, size_t workspace_bytes, attn_stream_t stream) {
  static const char* const names[2][3] = {{"q", "dq_out", "dq"}, {"k", "dk_out", "dk"}};
  bool empty = false;
  sa::RopeArgs a;
  TRY(rope_sizes(B, S, Hq, Hk, N, pos, pos_str, axes, freq, rope_dim, interleaved, magnitude, dtype, a, &empty));
  TRY(rope_weights(a, q_weight, k_weight, eps, w_dtype));
  const size_t w_size = w_dtype == ATTN_F32 ? 4 : 2;
  void* const dw[2] = {dq_weight, dk_weight};
  for (int i = 0; i < 2; ++i) {
    if (reinterpret_cast<uintptr_t>(dw[i]) % w_size != 0)
      return fail(ATTN_ERR_ALIGNMENT, "a weight's gradient is not aligned to its type");
    a.side[i].dw = dw[i];
  }
  // sums over no rows (after the last check: a refused call writes nothing)
  auto zeros = [&]() -> attn_status {
    for (int i = 0; i < 2; ++i) {
      if (dw[i] == nullptr || !(empty || a.side[i].H == 0)) continue;
      TRY(check_device());
      const cudaError_t e = cudaMemsetAsync(dw[i], 0, w_size * N, (cudaStream_t)stream);
      if (e != cudaSuccess) return fail_cuda(e, "qk_norm_rope_bwd");
    }
    return ATTN_OK;
  };
  if (empty) return zeros();
  a.inverse = 1;
  TRY(rope_side(a, 0, names[0], q, q_str, dq_out, dqo_str, dq, dq_str, true));
  TRY(rope_side(a, 1, names[1], k, k_str, dk_out, dko_str, dk, dk_str, true));
  TRY(rope_overlap("qk_norm_rope_bwd", a));
  if ((dw[0] != nullptr && Hq > 0) || (dw[1] != nullptr && Hk > 0)) {
    if (workspace == nullptr) return fail(ATTN_ERR_INVALID_ARG, "workspace is NULL");
    if (!aligned16(workspace)) return fail(ATTN_ERR_ALIGNMENT, "workspace is not 16-byte aligned");
    const size_t need = qk_norm_rope_bwd_workspace_size(B, S, Hq, Hk, N);
    if (workspace_bytes < need)
      return fail(ATTN_ERR_INVALID_ARG, "qk_norm_rope_bwd: workspace_bytes=%zu < %zu required", workspace_bytes, need);
  }
  TRY(check_device());
  TRY(zeros());
  const cudaError_t e = sa::launch_qk_norm_rope_bwd(a, reinterpret_cast<float*>(workspace), (cudaStream_t)stream);
  if (e != cudaSuccess) return fail_cuda(e, "qk_norm_rope_bwd");
  return ATTN_OK;
}

}  // extern "C"
