// C ABI of the K/V cache in 4 bits and the attention over it (declared in include/sageattn.h): argument validation and
// kernel launches.  No allocation happens here.
#include <cmath>

#include "../../include/sageattn.h"
#include "api_checks.h"
#include "api_overlap.h"
#include "kernels.h"

using namespace sa::api;

namespace {

attn_status check_cache(const void* cache, int num_pages, int page_size, const int32_t* table, int64_t table_str,
                        int max_pages, int B, int S, int Hkv, int D, sa::Kv4Args& a, bool* empty) {
  *empty = false;
  if (D != 128) return fail(ATTN_ERR_UNSUPPORTED, "head dimension D=%d; only D=128 is supported", D);
  if (B < 0 || S < 0 || Hkv < 0 || num_pages < 0 || max_pages < 0)
    return fail(ATTN_ERR_INVALID_ARG, "B=%d S=%d Hkv=%d num_pages=%d max_pages=%d must be >= 0", B, S, Hkv, num_pages,
                max_pages);
  if (page_size < 16 || page_size % 16 != 0)
    return fail(ATTN_ERR_INVALID_ARG, "page_size=%d must be a positive multiple of 16", page_size);
  if ((long long)max_pages * page_size > (1ll << 30))
    return fail(ATTN_ERR_INVALID_ARG, "max_pages * page_size must be at most 2^30 tokens");
  const long long bh = (long long)B * Hkv;
  if (bh > (1ll << 30) || bh * sa::kv4_tiles(S) > (1ll << 30))
    return fail(ATTN_ERR_INVALID_ARG, "B * Hkv * S is too large");
  if (bh == 0 || S == 0) {
    *empty = true;
    return ATTN_OK;
  }
  if (num_pages > 0 && cache == nullptr) return fail(ATTN_ERR_INVALID_ARG, "cache is NULL");
  if (!aligned16(cache)) return fail(ATTN_ERR_ALIGNMENT, "cache is not 16-byte aligned");
  if (max_pages > 0 && table == nullptr) return fail(ATTN_ERR_INVALID_ARG, "page_table is NULL");
  if (reinterpret_cast<uintptr_t>(table) % 4 != 0) return fail(ATTN_ERR_ALIGNMENT, "page_table is not 4-byte aligned");
  if (B > 1 && (table_str < 0 || table_str >= (1ll << 38)))
    return fail(ATTN_ERR_INVALID_ARG, "page_table's row stride %lld is out of range", (long long)table_str);
  a.cache = const_cast<void*>(cache);
  a.table = table;
  a.table_str = B > 1 ? table_str : 0;
  a.num_pages = num_pages;
  a.max_pages = max_pages;
  a.page_size = page_size;
  a.B = B;
  a.S = S;
  a.Hkv = Hkv;
  return ATTN_OK;
}

attn_status check_ints(const char* name, const int32_t* p, bool needed) {
  if (needed && p == nullptr) return fail(ATTN_ERR_INVALID_ARG, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) % 4 != 0) return fail(ATTN_ERR_ALIGNMENT, "%s is not 4-byte aligned", name);
  return ATTN_OK;
}

}  // namespace

extern "C" {

size_t kv4_cache_size(int num_pages, int Hkv, int page_size) {
  if (num_pages < 1 || Hkv < 1 || page_size < 16 || page_size % 16 != 0) return 0;
  return (size_t)num_pages * Hkv * (page_size / 16) * 2304;
}

attn_status kv4_write(const void* k, const void* v, void* cache, int num_pages, int page_size, const int32_t* page_table,
                      int64_t table_str, int max_pages, const int32_t* start, const int32_t* count, int B, int S, int Hkv,
                      int D, const int64_t k_str[3], const int64_t v_str[3], attn_stream_t stream) {
  bool empty = false;
  sa::Kv4Args a;
  TRY(check_cache(cache, num_pages, page_size, page_table, table_str, max_pages, B, S, Hkv, D, a, &empty));
  if (empty) return ATTN_OK;
  TRY(check_strides("k", k, k_str, B, S, Hkv, a.k_str));
  TRY(check_strides("v", v, v_str, B, S, Hkv, a.v_str));
  TRY(check_ints("start", start, true));
  TRY(check_ints("count", count, false));
  if (num_pages == 0 || max_pages == 0) return ATTN_OK;   // no place for any token
  a.k = k;
  a.v = v;
  a.start = start;
  a.count = count;
  TRY(check_device());
  const cudaError_t e = sa::launch_kv4_write(a, (cudaStream_t)stream);
  if (e != cudaSuccess) return fail_cuda(e, "kv4_write launch");
  return ATTN_OK;
}

attn_status kv4_read(const void* cache, int num_pages, int page_size, const int32_t* page_table, int64_t table_str,
                     int max_pages, const int32_t* start, const int32_t* count, void* k, void* v, int B, int S, int Hkv,
                     int D, const int64_t k_str[3], const int64_t v_str[3], attn_stream_t stream) {
  bool empty = false;
  sa::Kv4Args a;
  TRY(check_cache(cache, num_pages, page_size, page_table, table_str, max_pages, B, S, Hkv, D, a, &empty));
  if (empty) return ATTN_OK;
  TRY(check_strides("k", k, k_str, B, S, Hkv, a.k_str));
  TRY(check_strides("v", v, v_str, B, S, Hkv, a.v_str));
  TRY(check_ints("start", start, true));
  TRY(check_ints("count", count, false));
  if (share_memory(rows_of(k, B, S, Hkv, D, 2, a.k_str), rows_of(v, B, S, Hkv, D, 2, a.v_str)))
    return fail(ATTN_ERR_INVALID_ARG, "kv4_read: k and v must not overlap");
  a.k_out = k;
  a.v_out = v;
  a.start = start;
  a.count = count;
  TRY(check_device());
  const cudaError_t e = sa::launch_kv4_read(a, (cudaStream_t)stream);
  if (e != cudaSuccess) return fail_cuda(e, "kv4_read launch");
  return ATTN_OK;
}

static attn_status check_heads(int B, int Sq, int Hq, int Hkv) {
  if (Hq < 0 || (Hq == 0) != (Hkv == 0) || (Hkv > 0 && Hq % Hkv != 0))
    return fail(ATTN_ERR_INVALID_ARG, "Hq=%d must be a multiple of Hkv=%d", Hq, Hkv);
  const long long bs = (long long)B * Sq;
  if (bs > (1ll << 30) || bs * Hq > (1ll << 30)) return fail(ATTN_ERR_INVALID_ARG, "B*Sq*Hq must be at most 2^30 rows");
  return ATTN_OK;
}

size_t attn_fwd_kv4_workspace_size(int B, int Sq, int Hq, int Hkv, int max_pages, int page_size) {
  bool empty = false;
  sa::Kv4Args a;
  static const int32_t none = 0;   // (any address: nothing is read)
  alignas(16) static const char place[16] = {};
  if (check_cache(place, 1, page_size, &none, 0, max_pages, B, Sq, Hkv, 128, a, &empty) != ATTN_OK || empty ||
      check_heads(B, Sq, Hq, Hkv) != ATTN_OK)
    return 0;
  return sa::attn_kv4_workspace(B, Sq, Hq, Hkv, max_pages, page_size);
}

attn_status attn_fwd_kv4(const void* q, const void* cache, int num_pages, int page_size, const int32_t* page_table,
                         int64_t table_str, int max_pages, const int32_t* kv_len, void* o, float* lse, int B, int Sq,
                         int Hq, int Hkv, int D, const int64_t q_str[3], const int64_t o_str[3], float softmax_scale,
                         int causal, void* workspace, size_t workspace_bytes, attn_stream_t stream) {
  bool empty = false;
  sa::Kv4Args a;
  TRY(check_cache(cache, num_pages, page_size, page_table, table_str, max_pages, B, Sq, Hkv, D, a, &empty));
  TRY(check_heads(B, Sq, Hq, Hkv));
  if (causal != 0 && causal != 1) return fail(ATTN_ERR_INVALID_ARG, "causal=%d must be 0 or 1", causal);
  if (!(softmax_scale >= 0.0f && std::isfinite(softmax_scale)))
    return fail(ATTN_ERR_INVALID_ARG, "softmax_scale must be finite and >= 0");
  if (empty) return ATTN_OK;
  TRY(check_strides("q", q, q_str, B, Sq, Hq, a.q_str));
  TRY(check_strides("o", o, o_str, B, Sq, Hq, a.o_str));
  TRY(check_ints("kv_len", kv_len, true));
  if (lse == nullptr) return fail(ATTN_ERR_INVALID_ARG, "lse is NULL");
  if (reinterpret_cast<uintptr_t>(lse) % 4 != 0) return fail(ATTN_ERR_ALIGNMENT, "lse is not 4-byte aligned");
  if (share_memory(rows_of(o, B, Sq, Hq, D, 2, a.o_str), rows_of(q, B, Sq, Hq, D, 2, a.q_str)))
    return fail(ATTN_ERR_INVALID_ARG, "attn_fwd_kv4: o must not overlap q");
  if (workspace == nullptr) return fail(ATTN_ERR_INVALID_ARG, "workspace is NULL");
  if (!aligned16(workspace)) return fail(ATTN_ERR_ALIGNMENT, "workspace is not 16-byte aligned");
  const size_t need = sa::attn_kv4_workspace(B, Sq, Hq, Hkv, max_pages, page_size);
  if (workspace_bytes < need)
    return fail(ATTN_ERR_INVALID_ARG, "attn_fwd_kv4: workspace_bytes=%zu < %zu required", workspace_bytes, need);
  a.q = q;
  a.o = o;
  a.lse = lse;
  a.kv_len = kv_len;
  a.Hq = Hq;
  a.causal = causal;
  a.c_log2 = (float)((double)softmax_scale * kLog2e);
  TRY(check_device());
  const cudaError_t e = sa::launch_attn_kv4(a, workspace, (cudaStream_t)stream);
  if (e != cudaSuccess) return fail_cuda(e, "attn_fwd_kv4 launch");
  return ATTN_OK;
}

}  // extern "C"
