// Host-side launchers of the device kernels (internal to the library).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <atomic>
#include <cstddef>
#include <cstdint>
#include <mutex>

namespace sa {

// The unique id (cuCtxGetId) of the CUDA context current on the calling thread; when none
// is current yet, the current device's primary context is made current first, as the
// runtime's next call would.  Ids are never reused within a process.
cudaError_t current_context_id(unsigned long long* id);

// A value made once per CUDA context and cached, thread-safe.  Keyed by the context id,
// so a device that was reset, or a second context on the same device, makes its own
// value; the cache keeps the last 64 contexts (an older one simply makes it again).
template <class T>
class PerContext {
 public:
  // make: cudaError_t(T*), called with the context current; its value is cached on success
  template <class F>
  cudaError_t get(F&& make, T* out) {
    unsigned long long id = 0;
    cudaError_t e = current_context_id(&id);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lk(mu_);
    for (int i = 0; i < kSlots && i < n_; ++i)
      if (ids_[i] == id) {
        *out = vals_[i];
        return cudaSuccess;
      }
    T v{};
    e = make(&v);
    if (e != cudaSuccess) return e;
    ids_[n_ % kSlots] = id;
    vals_[n_ % kSlots] = v;
    ++n_;
    *out = v;
    return cudaSuccess;
  }

 private:
  static constexpr int kSlots = 64;
  std::mutex mu_;
  unsigned long long ids_[kSlots] = {};
  T vals_[kSlots] = {};
  int n_ = 0;
};

// A set-up step run once per CUDA context (e.g. a kernel attribute).
class ContextOnce {
 public:
  template <class F>
  cudaError_t run(F&& step) {
    char done = 0;
    return cache_.get([&](char* v) {
      cudaError_t e = step();
      *v = 1;
      return e;
    }, &done);
  }

 private:
  PerContext<char> cache_;
};

// Number of SMs of the current device (cached per context).
int device_sm_count();

// The attention forward kernel, three modes (attn_fwd.cu).  BF16 flash attention:
// Q, K, V through [B, S, H, 128] BF16 tensor maps.
// withhold_loads: the failure-path self-test (the producer loads nothing).
cudaError_t launch_attn_fwd_bf16(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v, void* o,
                                 long long o_sb, long long o_ss, long long o_sh, int B, int S, int H, float c_log2,
                                 cudaStream_t stream, bool withhold_loads = false);
// Timing instrumentation: per-SM {clock64, globaltimer} into out[n_slots][2] (cleared first).
cudaError_t launch_sm_clock_probe(unsigned long long* out, int n_slots, int num_sms, cudaStream_t stream);
// The device error word all three modes record bounded-wait timeouts in.
cudaError_t read_and_clear_err_attn(uint32_t* out);
// Other translation units with bounded waits add the reader of their error word when the library is loaded.
using ErrReader = cudaError_t (*)(uint32_t* out);
bool add_err_reader(ErrReader read);
// Reads such a word, and clears it if it is set.  launched: a kernel that may set it has been launched; until then there is
// nothing to read, and reading it would load the unit's kernels (the first status call 58 us, with three more
// units' words read 1770; later ones 18 and 56).
template <class Word>
cudaError_t read_and_clear_err(Word& word, const std::atomic<bool>& launched, uint32_t* out) {
  *out = 0;
  if (!launched.load(std::memory_order_relaxed)) return cudaSuccess;
  cudaError_t e = cudaMemcpyFromSymbol(out, word, sizeof(uint32_t));
  if (e != cudaSuccess || *out == 0) return e;
  const uint32_t zero = 0;
  return cudaMemcpyToSymbol(word, &zero, sizeof(uint32_t));
}

// Sage prepare (sage_prepare.cu)
struct PrepareArgs {
  const void* x[3];          // q, k, v (BF16)
  long long str[3][3];       // element strides (b, s, h)
  int B, S, H;
  long long S_pad;
  const void* q_norm_w;
  const void* k_norm_w;
  float rms_eps;
  const void* rope_cos;
  const void* rope_sin;
  int rope_dim;
  int8_t* q_i8;
  int8_t* k_i8;
  uint8_t* v_fp8;
  float* q_scale;
  float* k_scale;
  float* v_scale;
  float c_log2;
  uint32_t* vmax;            // workspace: B*H*128 words
  float* k_mean = nullptr;   // K smoothing: output [B*H*128] (nullptr: no smoothing)
  float* k_partial = nullptr;  // K smoothing workspace: [B*H, S_pad/32, 128] block sums
  void* q16 = nullptr;       // when set: Q/K codes written as FP16 [B*H, S_pad, 128] here, not as INT8
  void* k16 = nullptr;
  bool skip_v = false;       // V not prepared (the 16-bit P V mode reads the BF16 input)
  bool skip_q = false;       // Q not prepared (the forward quantises Q as it loads it)
  bool skip_k = false;       // K not prepared either (the forward codes K as well; needs skip_q)
  void* q_mean16 = nullptr;  // Q smoothing: output, binary16 [B*H, S_pad/32, 128] block means in step units
                             // (nullptr: no Q smoothing); the FP16 codes (q16) are then f16(code + mean)
};
cudaError_t launch_sage_prepare(const PrepareArgs& a, cudaStream_t stream);
// Q's score operand with Q smoothing, f16(code + mean), from the INT8 codes and the block means.
cudaError_t launch_widen_q_mean(const int8_t* q8, const void* qmean16, void* q16, long long n_codes, int num_sms,
                               cudaStream_t stream);
// e4m3 codes of n binary32 values through the prepare's and the attention's packing.
cudaError_t launch_e4m3_encode(const float* x, uint8_t* y, long long n, int num_sms, cudaStream_t stream);

// Device address, in the current context, of the static scratch used by the
// allocation-free prepare entry point; it holds kNoAllocMaxHeads * 128 words.
// Looked up on the first call in each context and cached.
constexpr int kNoAllocMaxHeads = 2048;
cudaError_t noalloc_prepare_scratch(uint32_t** out);

// Sage attention on prepared tensors (attn_fwd.cu)
size_t sage_attn_smem_bytes();
cudaError_t launch_sage_widen(const int8_t* q8, const int8_t* k8, void* q16, void* k16, long long n_codes,
                              int num_sms, cudaStream_t stream);
cudaError_t launch_sage_attn(const CUtensorMap& tm_q16, const CUtensorMap& tm_k16, const CUtensorMap& tm_v8,
                             const float* q_scale, const float* k_scale, const float* v_scale, void* o,
                             long long o_sb, long long o_ss, long long o_sh, int B, int S, int H, long long S_pad,
                             cudaStream_t stream);
// The 16-bit P V mode: V is the BF16 input through a [B, S, H, 128] tensor map.
cudaError_t launch_sage_attn_pv16(const CUtensorMap& tm_q16, const CUtensorMap& tm_k16,
                                  const CUtensorMap& tm_v_bf16, const float* q_scale, const float* k_scale, void* o,
                                  long long o_sb, long long o_ss, long long o_sh, int B, int S, int H,
                                  long long S_pad, cudaStream_t stream);

// Quantise-on-load of Q: the forward reads BF16 Q through a [B, S, H, 128] tensor
// map and each softmax thread turns its own row into the codes and the scale the
// prepare would have written (optional RMSNorm + RoPE first, the same arithmetic).
struct QLoadArgs {
  const void* q_norm_w = nullptr;   // BF16 [128], or nullptr: no RMSNorm
  const void* k_norm_w = nullptr;   // the same for K (K coded on load)
  float rms_eps = 0.0f;
  const void* rope_cos = nullptr;   // BF16 [S, rope_dim], or nullptr: no RoPE
  const void* rope_sin = nullptr;
  int rope_dim = 0;
  float c_log2 = 0.0f;              // fl32(softmax_scale * log2 e), folded into Q's scales
};
cudaError_t launch_sage_attn_qload(const CUtensorMap& tm_q_bf16, const CUtensorMap& tm_k16,
                                   const CUtensorMap& tm_v8, const QLoadArgs& qa, const float* k_scale,
                                   const float* v_scale, void* o, long long o_sb, long long o_ss, long long o_sh,
                                   int B, int S, int H, long long S_pad, cudaStream_t stream);
// K coded on load as well: K through a BF16 [B, S, H, 128] tensor map, coded per tile by the
// softmax warpgroups (the prepare's arithmetic); the block scales never leave shared memory.
cudaError_t launch_sage_attn_qkload(const CUtensorMap& tm_q_bf16, const CUtensorMap& tm_k_bf16,
                                    const CUtensorMap& tm_v8, const QLoadArgs& qa, const float* v_scale, void* o,
                                    long long o_sb, long long o_ss, long long o_sh, int B, int S, int H,
                                    long long S_pad, cudaStream_t stream);
cudaError_t launch_sage_attn_pv16_qkload(const CUtensorMap& tm_q_bf16, const CUtensorMap& tm_k_bf16,
                                         const CUtensorMap& tm_v_bf16, const QLoadArgs& qa, void* o, long long o_sb,
                                         long long o_ss, long long o_sh, int B, int S, int H, long long S_pad,
                                         cudaStream_t stream);
cudaError_t launch_sage_attn_pv16_qload(const CUtensorMap& tm_q_bf16, const CUtensorMap& tm_k16,
                                        const CUtensorMap& tm_v_bf16, const QLoadArgs& qa, const float* k_scale,
                                        void* o, long long o_sb, long long o_ss, long long o_sh, int B, int S, int H,
                                        long long S_pad, cudaStream_t stream);

// n / d for n < 2^31 by a product (Granlund and Montgomery, "Division by invariant integers using
// multiplication", 1994): d <= 2^shift, mul = floor(2^32 (2^shift - d) / d) + 1.
struct Div {
  uint32_t d, mul, shift;
};
inline Div make_div(int d) {
  Div r = {(uint32_t)d, 0, 0};
  while ((1ll << r.shift) < d) ++r.shift;
  r.mul = (uint32_t)(((1ull << 32) * ((1ull << r.shift) - (uint64_t)d)) / (uint64_t)d + 1);
  return r;
}
#ifdef __CUDACC__
__device__ __forceinline__ int div_by(int n, const Div& d) {
  return (int)((__umulhi((uint32_t)n, d.mul) + (uint32_t)n) >> d.shift);
}
#endif

// ------------------------------------------------------------------ training
// What the forward with row statistics and the backward share (attn_lse.cu, attn_bwd.cu).
struct TrainArgs {
  int B, Sq, Sk, Hq, Hkv;
  float scale;            // softmax_scale >= 0
  float c_log2;           // softmax_scale * log2 e
  int causal;             // query i sees the keys j <= i + Sk - Sq
  const int* kv_len;      // device [B], or nullptr: Sk keys
};
// Q [B, Sq, Hq, 128], K and V [B, Sk, Hkv, 128] through BF16 tensor maps; lse [B, Hq, Sq].
// tm_o: boxes of 32 rows.
cudaError_t launch_attn_fwd_bf16_lse(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                     const CUtensorMap& tm_o, const TrainArgs& a, float* lse, cudaStream_t stream);

struct BwdTensors {
  const void* k;
  long long k_str[3];
  const float* lse;
  void *dq, *dk, *dv;
  long long dq_str[3], dk_str[3], dv_str[3];
};
// Bytes of workspace for these shapes, whatever the mask.
size_t attn_bwd_workspace(TrainArgs a);
cudaError_t launch_attn_bwd_bf16(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                 const CUtensorMap& tm_d, const CUtensorMap& tm_o, const TrainArgs& a,
                                 const BwdTensors& t, float* workspace, cudaStream_t stream);

// Layer norm (layer_norm.cu).  Types of x, dy and the results, and of the weights.
enum : int { kBF16 = 0, kF16 = 1, kF32 = 2 };
struct LayerNormArgs {
  const void *x, *w, *b;      // w, b: or nullptr
  float *mean, *rstd;
  int B, S, H, N;
  long long x_str[3];         // element strides (b, s, h)
  int type, w_type;
  float eps;
};
size_t layer_norm_bwd_workspace(int rows, int N);
cudaError_t launch_layer_norm_fwd(const LayerNormArgs& a, void* y, const long long y_str[3], cudaStream_t stream);
// dw, db: both or neither.
cudaError_t launch_layer_norm_bwd(const LayerNormArgs& a, const void* dy, const long long dy_str[3], void* dx,
                                  const long long dx_str[3], void* dw, void* db, float* workspace,
                                  cudaStream_t stream);

// The order of a grid's items (tile, head): `group` heads go together, tile by tile.  One head after another
// (group = 1) keeps few heads' tiles in L2.  Where a causal mask makes the first tiles of a head the longest
// items, several heads' long ones come before their short ones, so that the grid ends with short
// ones: four items per SM go together.
struct Order {
  int tiles, heads, group, items;
  Div by_group, by_heads, by_rest;   // a group's items; its heads; the heads of a last, smaller group
};
inline Order make_order(int tiles, int heads, bool causal) {
  Order o;
  const int want = (4 * 152 + tiles - 1) / tiles;
  o.tiles = tiles;
  o.heads = heads;
  o.group = !causal ? 1 : want < heads ? want : heads;
  o.items = tiles * heads;
  o.by_group = make_div(o.group * tiles);
  o.by_heads = make_div(o.group);
  o.by_rest = make_div(heads % o.group ? heads % o.group : o.group);
  return o;
}

// A launch as a programmatic dependent of the previous kernel in the stream: the kernel may set
// up while that one finishes, and waits (griddep_wait) before it reads or writes what others do.
// (The training kernels do not let their dependents start before they end: CTAs that wait for the last items held SMs,
// and 20 captured steps of 512 x 512 tokens took 36.2 us each in place of 31.5.)
template <class... P, class... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                             const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace sa
