// C ABI of the training operators (declared in include/sageattn.h): argument validation, TMA tensor
// maps and kernel launches.  No allocation happens here.
#include <algorithm>
#include <cmath>

#include "../../include/sageattn.h"
#include "api_checks.h"
#include "kernels.h"

using namespace sa::api;

// ------------------------------------------------------------------ tensors that share memory
namespace {

// Rows of `row` bytes from ptr on, ext[i] of them str[i] bytes apart in dimension i.
struct Rows {
  uintptr_t ptr;
  long long ext[3], str[3], row, span;   // span: bytes from the first row's start to the last one's end, or 0
};
Rows rows_of(const void* ptr, int B, int S, int H, int n, int size, const long long str[3]) {
  Rows r = {reinterpret_cast<uintptr_t>(ptr), {B, S, H}, {}, (long long)n * size, 0};
  double span = 0;
  for (int i = 0; i < 3; ++i) {
    r.str[i] = r.ext[i] > 1 ? str[i] * size : 0;
    span += (double)(r.ext[i] - 1) * (double)r.str[i];
  }
  // (larger than any memory: nothing to compare, and nothing below overflows)
  if (span < 0x1p56) r.span = (r.ext[0] - 1) * r.str[0] + (r.ext[1] - 1) * r.str[1] + (r.ext[2] - 1) * r.str[2] + r.row;
  return r;
}
bool same(const Rows& a, const Rows& b) {
  return a.ptr == b.ptr && std::equal(a.str, a.str + 3, b.str) && std::equal(a.ext, a.ext + 3, b.ext) && a.row == b.row;
}

// Whether `at` plus a sum of multiples of steps[0..n), largest step first, each multiple in its range, can come to between
// -room and room.  steps_left bounds the search: slices of one buffer, whose steps lie within one another, take
// two or three tries a step.  (Undecided is taken for no.)
struct Step {
  long long by, lo, hi;
};
bool meets(const Step* steps, int n, long long at, long long room, int& steps_left) {
  if (n == 0) return -room < at && at < room;
  long long lo = 0, hi = 0;   // what the steps after this one can add
  for (int i = 1; i < n; ++i) {
    lo += steps[i].by * steps[i].lo;
    hi += steps[i].by * steps[i].hi;
  }
  auto down = [](long long a, long long b) { return a / b - (a % b < 0 ? 1 : 0); };
  const long long first = std::max(steps->lo, -down(at + hi + room - 1, steps->by));
  const long long last = std::min(steps->hi, down(room - 1 - at - lo, steps->by));
  for (long long x = first; x <= last; ++x) {
    if (--steps_left < 0) return false;
    if (meets(steps + 1, n - 1, at + x * steps->by, room, steps_left)) return true;
  }
  return false;
}

// Whether a row of a and a row of b (of one length) have a byte in common.
bool share_memory(const Rows& a, const Rows& b) {
  if (a.span == 0 || b.span == 0 || a.ptr + a.span <= b.ptr || b.ptr + b.span <= a.ptr) return false;
  Step steps[6];
  int n = 0;
  auto add = [&](long long by, long long lo, long long hi) {
    if (by == 0) return;
    int i = 0;
    while (i < n && steps[i].by != by) ++i;
    if (i == n) steps[n++] = {by, 0, 0};
    steps[i].lo += lo;
    steps[i].hi += hi;
  };
  for (int i = 0; i < 3; ++i) {
    add(a.str[i], 1 - a.ext[i], 0);
    add(b.str[i], 0, b.ext[i] - 1);
  }
  std::sort(steps, steps + n, [](const Step& x, const Step& y) { return x.by > y.by; });
  int steps_left = 10000;
  return meets(steps, n, (long long)(b.ptr - a.ptr), a.row, steps_left);
}

}  // namespace

extern "C" {

// ------------------------------------------------------------------ attention
// Shapes and mask of the training calls: *empty is set for B = 0 or no heads.
static attn_status check_train(int B, int Sq, int Sk, int Hq, int Hkv, int D, int causal, const int32_t* kv_len,
                               float softmax_scale, sa::TrainArgs& a, bool* empty) {
  *empty = false;
  if (D != 128) return fail(ATTN_ERR_UNSUPPORTED, "head dimension D=%d; only D=128 is supported", D);
  if (B < 0 || Hq < 0 || Hkv < 0) return fail(ATTN_ERR_INVALID_ARG, "B=%d Hq=%d Hkv=%d must be >= 0", B, Hq, Hkv);
  if (Sq < 1 || Sk < 1 || Sq > (1 << 30) || Sk > (1 << 30))
    return fail(ATTN_ERR_INVALID_ARG, "Sq=%d Sk=%d must be in [1, 2^30]", Sq, Sk);
  if ((Hq == 0) != (Hkv == 0) || (Hkv > 0 && Hq % Hkv != 0))
    return fail(ATTN_ERR_INVALID_ARG, "Hq=%d must be a multiple of Hkv=%d", Hq, Hkv);
  if (causal != 0 && causal != 1) return fail(ATTN_ERR_INVALID_ARG, "causal=%d must be 0 or 1", causal);
  if (!(softmax_scale >= 0.0f && std::isfinite(softmax_scale)))
    return fail(ATTN_ERR_INVALID_ARG, "softmax_scale must be finite and >= 0");
  if (reinterpret_cast<uintptr_t>(kv_len) % 4 != 0) return fail(ATTN_ERR_ALIGNMENT, "kv_len is not 4-byte aligned");
  if (B == 0 || Hq == 0) {
    *empty = true;
    return ATTN_OK;
  }
  TRY(check_grid(B, Hq, ((long long)Sq + 127) / 128 * 128));
  TRY(check_grid(B, Hkv, ((long long)Sk + 127) / 128 * 128));
  a.B = B;
  a.Sq = Sq;
  a.Sk = Sk;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.scale = softmax_scale;
  a.c_log2 = (float)((double)softmax_scale * kLog2e);
  a.causal = causal;
  a.kv_len = kv_len;
  return ATTN_OK;
}

static attn_status check_buffer(const char* name, const void* ptr) {
  if (ptr == nullptr) return fail(ATTN_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned16(ptr)) return fail(ATTN_ERR_ALIGNMENT, "%s is not 16-byte aligned", name);
  return ATTN_OK;
}

attn_status attn_fwd_bf16_lse(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Sq, int Sk,
                              int Hq, int Hkv, int D, const int64_t q_str[3], const int64_t k_str[3],
                              const int64_t v_str[3], const int64_t o_str[3], float softmax_scale, int causal,
                              const int32_t* kv_len, attn_stream_t stream) {
  bool empty = false;
  sa::TrainArgs a;
  TRY(check_train(B, Sq, Sk, Hq, Hkv, D, causal, kv_len, softmax_scale, a, &empty));
  if (empty) return ATTN_OK;
  long long qs[3], ks[3], vs[3], os[3];
  TRY(check_strides("q", q, q_str, B, Sq, Hq, qs));
  TRY(check_strides("k", k, k_str, B, Sk, Hkv, ks));
  TRY(check_strides("v", v, v_str, B, Sk, Hkv, vs));
  TRY(check_strides("o", o, o_str, B, Sq, Hq, os));
  TRY(check_buffer("lse", lse));
  const Rows o_rows = rows_of(o, B, Sq, Hq, D, 2, os);
  if (share_memory(o_rows, rows_of(q, B, Sq, Hq, D, 2, qs)) || share_memory(o_rows, rows_of(k, B, Sk, Hkv, D, 2, ks)) ||
      share_memory(o_rows, rows_of(v, B, Sk, Hkv, D, 2, vs)))
    return fail(ATTN_ERR_INVALID_ARG, "attn_fwd_bf16_lse: o must overlap no input");
  TRY(check_device());
  TRY(get_encoder());
  CUtensorMap tq, tk, tv, to;
  TRY(tmap_bhsd_bf16(&tq, q, B, Sq, Hq, qs));
  TRY(tmap_bhsd_bf16(&tk, k, B, Sk, Hkv, ks));
  TRY(tmap_bhsd_bf16(&tv, v, B, Sk, Hkv, vs));
  TRY(tmap_bhsd_bf16(&to, o, B, Sq, Hq, os, 32));
  cudaError_t e = sa::launch_attn_fwd_bf16_lse(tq, tk, tv, to, a, lse, (cudaStream_t)stream);
  if (e != cudaSuccess) return fail_cuda(e, "attn_fwd_bf16_lse launch");
  return ATTN_OK;
}

size_t attn_bwd_bf16_workspace_size(int B, int Sq, int Sk, int Hq, int Hkv) {
  bool empty = false;
  sa::TrainArgs a;
  if (check_train(B, Sq, Sk, Hq, Hkv, 128, 0, nullptr, 0.0f, a, &empty) != ATTN_OK || empty) return 0;
  return sa::attn_bwd_workspace(a);
}

attn_status attn_bwd_bf16(const void* dout, const void* q, const void* k, const void* v, const void* o,
                          const float* lse, void* dq, void* dk, void* dv, int B, int Sq, int Sk, int Hq, int Hkv,
                          int D, const int64_t dout_str[3], const int64_t q_str[3], const int64_t k_str[3],
                          const int64_t v_str[3], const int64_t o_str[3], const int64_t dq_str[3],
                          const int64_t dk_str[3], const int64_t dv_str[3], float softmax_scale, int causal,
                          const int32_t* kv_len, void* workspace, size_t workspace_bytes, attn_stream_t stream) {
  bool empty = false;
  sa::TrainArgs a;
  TRY(check_train(B, Sq, Sk, Hq, Hkv, D, causal, kv_len, softmax_scale, a, &empty));
  if (empty) return ATTN_OK;
  long long qs[3], ks[3], vs[3], ds[3], os[3];
  sa::BwdTensors t;
  TRY(check_strides("dout", dout, dout_str, B, Sq, Hq, ds));
  TRY(check_strides("q", q, q_str, B, Sq, Hq, qs));
  TRY(check_strides("k", k, k_str, B, Sk, Hkv, ks));
  TRY(check_strides("v", v, v_str, B, Sk, Hkv, vs));
  TRY(check_strides("o", o, o_str, B, Sq, Hq, os));
  TRY(check_strides("dq", dq, dq_str, B, Sq, Hq, t.dq_str));
  TRY(check_strides("dk", dk, dk_str, B, Sk, Hkv, t.dk_str));
  TRY(check_strides("dv", dv, dv_str, B, Sk, Hkv, t.dv_str));
  TRY(check_buffer("lse", lse));
  TRY(check_buffer("workspace", workspace));
  // dK and dV are formed from the inputs after dQ has been written
  const Rows out[3] = {rows_of(dq, B, Sq, Hq, D, 2, t.dq_str), rows_of(dk, B, Sk, Hkv, D, 2, t.dk_str),
                       rows_of(dv, B, Sk, Hkv, D, 2, t.dv_str)};
  const Rows in[5] = {rows_of(dout, B, Sq, Hq, D, 2, ds), rows_of(q, B, Sq, Hq, D, 2, qs),
                      rows_of(k, B, Sk, Hkv, D, 2, ks), rows_of(v, B, Sk, Hkv, D, 2, vs),
                      rows_of(o, B, Sq, Hq, D, 2, os)};
  bool shared = share_memory(out[0], out[1]) || share_memory(out[0], out[2]) || share_memory(out[1], out[2]);
  for (const Rows& x : out)
    for (const Rows& y : in) shared = shared || share_memory(x, y);
  if (shared)
    return fail(ATTN_ERR_INVALID_ARG, "attn_bwd_bf16: dq, dk and dv must overlap neither the inputs nor one another");
  const size_t need = sa::attn_bwd_workspace(a);
  if (workspace_bytes < need)
    return fail(ATTN_ERR_INVALID_ARG, "attn_bwd_bf16: workspace_bytes=%zu < %zu required", workspace_bytes, need);
  TRY(check_device());
  TRY(get_encoder());
  CUtensorMap tq, tk, tv, td, to;
  TRY(tmap_bhsd_bf16(&tq, q, B, Sq, Hq, qs));
  TRY(tmap_bhsd_bf16(&tk, k, B, Sk, Hkv, ks));
  TRY(tmap_bhsd_bf16(&tv, v, B, Sk, Hkv, vs));
  TRY(tmap_bhsd_bf16(&td, dout, B, Sq, Hq, ds));
  TRY(tmap_bhsd_bf16(&to, o, B, Sq, Hq, os));
  t.k = k;
  for (int i = 0; i < 3; ++i) t.k_str[i] = ks[i];
  t.lse = lse;
  t.dq = dq;
  t.dk = dk;
  t.dv = dv;
  cudaError_t e = sa::launch_attn_bwd_bf16(tq, tk, tv, td, to, a, t, reinterpret_cast<float*>(workspace),
                                           (cudaStream_t)stream);
  if (e != cudaSuccess) return fail_cuda(e, "attn_bwd_bf16 launch");
  return ATTN_OK;
}

// ------------------------------------------------------------------ layer norm
// Strides of [B, S, H, N] rows in whole elements; 0 (the same row again) only where a tensor is read.
static attn_status check_rows(const char* name, const void* ptr, int type, const int64_t* in, const sa::LayerNormArgs& a,
                              bool read, long long out[3]) {
  if (ptr == nullptr) return fail(ATTN_ERR_INVALID_ARG, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(ptr) % (type == ATTN_F32 ? 4 : 2) != 0)
    return fail(ATTN_ERR_ALIGNMENT, "%s is not aligned to its type", name);
  if (in == nullptr) return fail(ATTN_ERR_INVALID_ARG, "%s strides are NULL", name);
  const int ext[3] = {a.B, a.S, a.H};
  for (int i = 0; i < 3; ++i) {
    const long long s = ext[i] == 1 ? 0 : in[i];
    if (s < 0 || (s == 0 && ext[i] > 1 && !read) || s >= (1ll << 38))
      return fail(ATTN_ERR_INVALID_ARG, "%s stride %lld of dimension %d is out of range", name, (long long)in[i], i);
    out[i] = s;
  }
  return ATTN_OK;
}

static attn_status check_norm(const void* x, const void* w, const void* b, float* mean, float* rstd, int B, int S,
                              int H, int N, const int64_t* x_str, int type, int w_type, sa::LayerNormArgs& a,
                              bool* empty) {
  *empty = false;
  if (type < ATTN_BF16 || type > ATTN_F32) return fail(ATTN_ERR_INVALID_ARG, "dtype=%d is none of attn_dtype", type);
  if (w_type != type && w_type != ATTN_F32)
    return fail(ATTN_ERR_INVALID_ARG, "w_dtype=%d must be the rows' type or ATTN_F32", w_type);
  if (B < 0 || S < 0 || H < 0) return fail(ATTN_ERR_INVALID_ARG, "B=%d S=%d H=%d must be >= 0", B, S, H);
  if (N < 1 || N > 16384) return fail(ATTN_ERR_INVALID_ARG, "N=%d must be in [1, 16384]", N);
  // (no overflow: a factor that makes it too large ends the product)
  const long long bs = (long long)B * S;
  if (bs > (1ll << 30) || bs * H > (1ll << 30)) return fail(ATTN_ERR_INVALID_ARG, "B*S*H must be at most 2^30 rows");
  a.B = B;
  a.S = S;
  a.H = H;
  a.N = N;
  a.type = type;
  a.w_type = w_type;
  a.x = x;
  a.w = w;
  a.b = b;
  a.mean = mean;
  a.rstd = rstd;
  if (B == 0 || S == 0 || H == 0) {
    *empty = true;
    return ATTN_OK;
  }
  TRY(check_rows("x", x, type, x_str, a, true, a.x_str));
  const uintptr_t w_align = w_type == ATTN_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(w) % w_align != 0 || reinterpret_cast<uintptr_t>(b) % w_align != 0)
    return fail(ATTN_ERR_ALIGNMENT, "weight or bias is not aligned to its type");
  if (mean == nullptr || rstd == nullptr) return fail(ATTN_ERR_INVALID_ARG, "mean or rstd is NULL");
  if (reinterpret_cast<uintptr_t>(mean) % 4 != 0 || reinterpret_cast<uintptr_t>(rstd) % 4 != 0)
    return fail(ATTN_ERR_ALIGNMENT, "mean or rstd is not 4-byte aligned");
  return ATTN_OK;
}

attn_status layer_norm_fwd(const void* x, const void* weight, const void* bias, void* y, float* mean, float* rstd,
                           int B, int S, int H, int N, const int64_t x_str[3], const int64_t y_str[3], float eps,
                           int dtype, int w_dtype, attn_stream_t stream) {
  bool empty = false;
  sa::LayerNormArgs a;
  if (!(eps >= 0.0f && std::isfinite(eps))) return fail(ATTN_ERR_INVALID_ARG, "eps must be finite and >= 0");
  TRY(check_norm(x, weight, bias, mean, rstd, B, S, H, N, x_str, dtype, w_dtype, a, &empty));
  if (empty) return ATTN_OK;
  a.eps = eps;
  long long ys[3];
  TRY(check_rows("y", y, dtype, y_str, a, false, ys));
  const int size = dtype == ATTN_F32 ? 4 : 2;
  const Rows x_rows = rows_of(x, B, S, H, N, size, a.x_str), y_rows = rows_of(y, B, S, H, N, size, ys);
  if (!same(x_rows, y_rows) && share_memory(x_rows, y_rows))
    return fail(ATTN_ERR_INVALID_ARG, "layer_norm_fwd: y must be x itself or overlap it nowhere");
  TRY(check_device());
  cudaError_t e = sa::launch_layer_norm_fwd(a, y, ys, (cudaStream_t)stream);
  if (e != cudaSuccess) return fail_cuda(e, "layer_norm_fwd launch");
  return ATTN_OK;
}

size_t layer_norm_bwd_workspace_size(int B, int S, int H, int N) {
  if (B < 1 || S < 1 || H < 1 || N < 1 || N > 16384) return 0;
  const long long bs = (long long)B * S;
  if (bs > (1ll << 30) || bs * H > (1ll << 30)) return 0;
  return sa::layer_norm_bwd_workspace((int)(bs * H), N);
}

attn_status layer_norm_bwd(const void* dy, const void* x, const void* weight, const float* mean, const float* rstd,
                           void* dx, void* dweight, void* dbias, int B, int S, int H, int N, const int64_t dy_str[3],
                           const int64_t x_str[3], const int64_t dx_str[3], int dtype, int w_dtype, void* workspace,
                           size_t workspace_bytes, attn_stream_t stream) {
  bool empty = false;
  sa::LayerNormArgs a;
  TRY(check_norm(x, weight, nullptr, const_cast<float*>(mean), const_cast<float*>(rstd), B, S, H, N, x_str, dtype,
                 w_dtype, a, &empty));
  a.eps = 0.0f;
  if ((dweight == nullptr) != (dbias == nullptr))
    return fail(ATTN_ERR_INVALID_ARG, "dweight and dbias must both be given or both be NULL");
  const uintptr_t w_size = w_dtype == ATTN_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(dweight) % w_size != 0 || reinterpret_cast<uintptr_t>(dbias) % w_size != 0)
    return fail(ATTN_ERR_ALIGNMENT, "dweight or dbias is not aligned to its type");
  if (empty) {   // sums over no rows
    if (dweight == nullptr) return ATTN_OK;
    TRY(check_device());
    cudaError_t e = cudaMemsetAsync(dweight, 0, w_size * N, (cudaStream_t)stream);
    if (e == cudaSuccess) e = cudaMemsetAsync(dbias, 0, w_size * N, (cudaStream_t)stream);
    if (e != cudaSuccess) return fail_cuda(e, "layer_norm_bwd");
    return ATTN_OK;
  }
  long long ds[3], xs[3];
  TRY(check_rows("dy", dy, dtype, dy_str, a, true, ds));
  TRY(check_rows("dx", dx, dtype, dx_str, a, false, xs));
  if (dweight != nullptr) {
    TRY(check_buffer("workspace", workspace));
    const size_t need = layer_norm_bwd_workspace_size(B, S, H, N);
    if (workspace_bytes < need)
      return fail(ATTN_ERR_INVALID_ARG, "layer_norm_bwd: workspace_bytes=%zu < %zu required", workspace_bytes, need);
  }
  const int size = dtype == ATTN_F32 ? 4 : 2;
  const Rows dx_rows = rows_of(dx, B, S, H, N, size, xs);
  for (const Rows& in : {rows_of(dy, B, S, H, N, size, ds), rows_of(x, B, S, H, N, size, a.x_str)})
    if (!same(dx_rows, in) && share_memory(dx_rows, in))
      return fail(ATTN_ERR_INVALID_ARG, "layer_norm_bwd: dx must be dy or x itself or overlap them nowhere");
  TRY(check_device());
  cudaError_t e = sa::launch_layer_norm_bwd(a, dy, ds, dx, xs, dweight, dbias, reinterpret_cast<float*>(workspace),
                                            (cudaStream_t)stream);
  if (e != cudaSuccess) return fail_cuda(e, "layer_norm_bwd launch");
  return ATTN_OK;
}

}  // extern "C"
