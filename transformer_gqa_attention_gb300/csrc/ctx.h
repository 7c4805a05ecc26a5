// ctx.h — the library's context (packed weights, status word, workspaces) and the host
// helpers every entry point shares: argument and device checks, tensor maps, workspace growth
// and the per-launch profiling bracket.  Internal; the public interface is gqa_attn.h.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>
#include <vector>

#include <nvtx3/nvToolsExt.h>

#include "gqa_attn.h"
#include "launch.h"
#include "params.h"

namespace gqa {

// Grow-only device memory of a context.
struct DeviceBuffer {
  uint8_t* p = nullptr;
  size_t bytes = 0;
  bool captured = false;  // a call recorded into a CUDA graph uses it
};

}  // namespace gqa

struct gqa_ctx {
  int device = -1;
  int num_sms = 0;
  int pair_clusters = 0;  // co-resident 2-CTA clusters of the pair GEMM
  // kv groups of this context: 8 for the whole block, G < 8 for a head shard (4 G query
  // heads); q_cols = 512 G query features, kv_cols = 128 G key (and value) features
  int n_kv = 8;
  int q_cols() const { return 512 * n_kv; }
  int kv_cols() const { return 128 * n_kv; }
  int qkv_rows() const { return 768 * n_kv; }
  // weights, k-block-major: W_t[kb][row][64]
  __nv_bfloat16* w_qkv = nullptr;  // qkv_rows x 4096: W_Q rows 0..q_cols-1, then W_K, then W_V
  __nv_bfloat16* w_o = nullptr;    // 4096 rows x q_cols (the columns of W_O that belong to its heads)
  // residual form: W_QKV * diag(attention_norm weight), same layout (attn_set_norm)
  __nv_bfloat16* w_qkv_norm = nullptr;
  float norm_eps = 0.f;
  int* status = nullptr;           // device status word (kDevErr* bits)
  int* old_len = nullptr;          // [kDecodeMaxBatch] lengths before an eviction (behind the status word)
  int* zeros = nullptr;            // [kDecodeMaxBatch] zeros (behind old_len)
  int* counters = nullptr;         // arrival counters (kCounterInts, then kGroupCounterInts)
  gqa::DeviceBuffer ws;            // workspace of the block forms
  gqa::DeviceBuffer cache_ws;      // scratch of the attention over caches of per-sequence length
  std::vector<void*> retired;      // outgrown buffers that a captured graph may still use
  const void* last_q = nullptr;
  const void* last_h = nullptr;
  // per-kernel device timing
  bool profiling = false;
  std::vector<cudaEvent_t> ev;        // 2 per recorded launch
  std::vector<int> ev_kind;           // kind of each recorded launch
  size_t ev_used = 0;                 // launches recorded so far
  int fault_kind = -1;                // test hook armed by attn_debug_inject_timeout
};


namespace gqa {

inline gqa_status cuda_fail(cudaError_t e) {
  set_last_cuda_error(e);
  return GQA_ERR_CUDA;
}

#define GQA_CUDA(call)                          \
  do {                                          \
    cudaError_t e_ = (call);                    \
    if (e_ != cudaSuccess) return cuda_fail(e_); \
  } while (0)

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr long long kMaxTokens = 262144;
constexpr long long kMaxSMax = 1048576;
constexpr int kDecodeMaxBatch = 1024;
// Arrival counters: one per (sequence, kv group, position group), and behind them those of groups of pieces of the
// attention over pages, two per CTA.
constexpr int kCounterInts = kDecodeMaxBatch * 8;
constexpr int kGroupCounterInts = 2048;

// ------------------------------------------------------------------ tensor maps
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                   CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                   CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// Tensor map (bf16 unless `type` says otherwise) with 128-byte swizzle; dims[0] innermost; strides in
// bytes for dims 1..; `fetch`: bytes of a row that a miss brings to L2 together.
inline bool make_map(CUtensorMap* m, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
              const uint32_t* box, CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
              CUtensorMapL2promotion fetch = CU_TENSOR_MAP_L2_PROMOTION_L2_256B) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t d[5], s[4];
  cuuint32_t b[5], e[5];
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i];
    b[i] = box[i];
    e[i] = 1;
  }
  for (int i = 0; i < rank - 1; ++i) s[i] = strides[i];
  return fn(m, type, rank, const_cast<void*>(base), d, s, b, e,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, fetch,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// KV cache [B, S_max, n_kv, 128] bf16 seen as (d, g, s < kv_len, b); box 64 d x key_rows.
inline bool map_cache(CUtensorMap* m, const void* base, int B, int S_max, int n_kv, int kv_len, uint32_t key_rows) {
  const uint64_t dims[4] = {128, static_cast<uint64_t>(n_kv), static_cast<uint64_t>(kv_len), static_cast<uint64_t>(B)};
  const uint64_t strides[3] = {128 * 2, static_cast<uint64_t>(n_kv) * 128 * 2,
                               static_cast<uint64_t>(S_max) * n_kv * 128 * 2};
  const uint32_t box[4] = {64, 1, key_rows, 1};
  return make_map(m, base, 4, dims, strides, box);
}

inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

// Make `buf` hold at least `bytes` (enqueued work on `s` may still use the old memory, so growing
// synchronises `s` and a call that has to grow cannot be captured).  Memory that a captured call
// uses is kept until the context is destroyed, not freed, when the buffer outgrows it: the graph
// holds its address.
inline gqa_status ensure_buffer(gqa_ctx* c, DeviceBuffer& buf, size_t bytes, cudaStream_t s) {
  if (bytes <= buf.bytes && buf.captured) return GQA_OK;
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(s, &cs) != cudaSuccess) {  // the legacy stream beside another capture
    cudaGetLastError();
    cs = cudaStreamCaptureStatusNone;
  }
  const bool capturing = cs != cudaStreamCaptureStatusNone;
  if (bytes <= buf.bytes) {
    buf.captured |= capturing;
    return GQA_OK;
  }
  if (capturing) return cuda_fail(cudaErrorStreamCaptureUnsupported);
  GQA_CUDA(cudaStreamSynchronize(s));
  if (buf.p) {
    if (buf.captured) {
      try {
        c->retired.push_back(buf.p);
      } catch (...) {
        return GQA_ERR_OOM;
      }
    } else {
      GQA_CUDA(cudaFree(buf.p));
    }
  }
  buf = DeviceBuffer{};
  const size_t want = round_up(bytes, 1 << 20);
  if (cudaMalloc(&buf.p, want) != cudaSuccess) {
    cudaGetLastError();
    buf.p = nullptr;
    return GQA_ERR_OOM;
  }
  buf.bytes = want;
  return GQA_OK;
}

inline gqa_status check_device(gqa_ctx* c) {
  int dev = -1;
  GQA_CUDA(cudaGetDevice(&dev));
  if (dev != c->device) return GQA_ERR_DEVICE;
  return GQA_OK;
}

// One-shot test hook: 1 if the next launch of `kind` should skip its first unit's loads.
inline int take_fault(gqa_ctx* c, int kind) {
  if (c->fault_kind != kind) return 0;
  c->fault_kind = -1;
  return 1;
}

constexpr size_t kMaxProfiledLaunches = 65536;

// RAII bracket of one kernel launch with two events when profiling is on.
// NVTX range names of the kernel kinds (host-side ranges around each launch; without a tool
// attached an NVTX call returns at once).
inline const char* const kKindNames[GQA_KERNEL_KINDS] = {"gqa.qkv_gemm", "gqa.qkv_splitk", "gqa.flash_prefill",
                                                  "gqa.decode_attn", "gqa.out_gemm", "gqa.out_splitk",
                                                  "gqa.rms_norm", "gqa.cache_attn", "gqa.cache_merge", "gqa.cache_weights", "gqa.cache_commit", "gqa.evict_select",
                                                         "gqa.evict_move", "gqa.paged_attn", "gqa.paged_append", "gqa.rope"};

// RAII NVTX range around one entry point's host work (its launches nest inside it).
struct CallRange {
  explicit CallRange(const char* name) { nvtxRangePushA(name); }
  ~CallRange() { nvtxRangePop(); }
};

struct ProfScope {
  gqa_ctx* c;
  cudaStream_t s;
  bool on;
  ProfScope(gqa_ctx* c_, int kind, cudaStream_t s_) : c(c_), s(s_), on(false) {
    nvtxRangePushA(kind >= 0 && kind < GQA_KERNEL_KINDS ? kKindNames[kind] : "gqa.kernel");
    if (c->profiling && c->ev_used < kMaxProfiledLaunches) {
      if (c->ev.size() < 2 * (c->ev_used + 1)) {
        cudaEvent_t a, b;
        if (cudaEventCreate(&a) != cudaSuccess) return;
        if (cudaEventCreate(&b) != cudaSuccess) { cudaEventDestroy(a); return; }
        try {
          c->ev.reserve(c->ev.size() + 2);
          c->ev_kind.push_back(kind);
        } catch (...) {  // this launch goes unrecorded
          cudaEventDestroy(a);
          cudaEventDestroy(b);
          return;
        }
        c->ev.push_back(a);
        c->ev.push_back(b);
      }
      c->ev_kind[c->ev_used] = kind;
      on = cudaEventRecord(c->ev[2 * c->ev_used], s) == cudaSuccess;
    }
  }
  ~ProfScope() {
    if (on) {
      cudaEventRecord(c->ev[2 * c->ev_used + 1], s);
      ++c->ev_used;
    }
    nvtxRangePop();
  }
};

inline const float kScaleLog2 = static_cast<float>(1.4426950408889634 / std::sqrt(128.0));

}  // namespace gqa
