// What the host sources of the library share: the error text, the per-device
// state, launch profiling and the tensor-map encoder.  Defined in muonclip.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <map>
#include <mutex>
#include <set>
#include <string>
#include <vector>

#include "muonclip.h"

#define MC_API extern "C" __attribute__((visibility("default")))

#define MC_CUDA(expr)                                                                      \
  do {                                                                                     \
    cudaError_t e_ = (expr);                                                               \
    if (e_ != cudaSuccess) return fail(MC_ERR_CUDA, std::string(#expr) + ": " + cudaGetErrorString(e_)); \
  } while (0)

namespace mc {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Largest dynamic shared memory a CTA may opt into on sm_100.
constexpr int kSmemOptIn = 232448;

struct DeviceState {
  bool init = false;
  bool act_init = false;  // the activation operators' kernel attributes are set
  std::set<const void*> wide_smem;  // kernels allowed more than 48 KiB of shared memory on first use
  int sms = 0;
  int pair_clusters = 0;  // CTA pairs of the GEMM kernel that fit on the device at once
  int cc_major = 0, cc_minor = 0;
  int* err_ptr = nullptr;
  void* own_ws = nullptr;
  size_t own_ws_bytes = 0;
  // mc_muon_step_host_grads: a non-blocking stream for the gradient copies and
  // events that order each chunk's compute after its copies
  cudaStream_t copy_stream = nullptr;
  std::vector<cudaEvent_t> chunk_ev;
};

extern std::mutex g_mu;

// Set the calling thread's error text; returns `code`.
int fail(int code, const std::string& msg);
// State of the current device, set up on first use.  Caller holds g_mu.
int device_state(DeviceState** out);
// The library's own workspace of the device, grown to `bytes`.  Caller holds g_mu.
int own_workspace(DeviceState& st, size_t bytes, void** ws);
// bf16 tensor map unless `type` says otherwise (128-byte swizzle unless
// given), zero fill out of bounds.  Strides in bytes, outermost excluded.
int make_map(CUtensorMap* map, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
             const uint32_t* box, CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B,
             CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16);
// Programmatic stream serialisation as a launch attribute.
void set_pdl(cudaLaunchAttribute& a, bool on);

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline int64_t round8(int64_t x) { return (x + 7) / 8 * 8; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// ----------------------------------------------------------- profiling
enum Kind : int { K_MOMENTUM, K_FINALIZE, K_GRAM, K_POLY, K_APPLY_MIXED, K_APPLY, K_APPLY_FINAL, K_QK_PROJ,
                  K_QK_CMAX, K_QK_KEYS, K_QK_CLIP, K_MLA_PROJ, K_MLA_CMAX, K_QK_CLIP_SLICES, K_NORM_ROWS,
                  K_NORM_APPLY, K_TABLE_UPLOAD, K_NS_THIN, K_ACT_PACK, K_ACT_UNPACK, K_RMS_NORM, K_RMS_NORM_BWD,
                  K_RMS_NORM_DW, K_WGRAD_PREP, K_WGRAD, K_WGRAD_JOIN, K_EXPERT_SORT, K_EXPERT_GATHER,
                  K_EXPERT_COMBINE, K_EXPERT_COMBINE_BWD, K_COUNT };
struct ProfRec {
  int kind;
  cudaEvent_t b, e;
  double flops, flops_exec, flops_dense, bytes;
};
extern thread_local bool t_prof;
extern thread_local std::vector<ProfRec> t_recs;

// Brackets one launch with CUDA events on its stream while profiling is on.
struct ProfScope {
  bool on = false;
  ProfRec r{};
  cudaStream_t s;
  ProfScope(int kind, cudaStream_t st, double flops = 0, double flops_exec = 0, double bytes = 0,
            double flops_dense = -1) : s(st) {
    if (!t_prof || kind < 0) return;
    r.kind = kind;
    r.flops = flops;
    r.flops_exec = flops_exec;
    r.flops_dense = flops_dense < 0 ? flops : flops_dense;
    r.bytes = bytes;
    if (cudaEventCreate(&r.b) != cudaSuccess) return;
    if (cudaEventCreate(&r.e) != cudaSuccess) {
      cudaEventDestroy(r.b);
      return;
    }
    on = cudaEventRecord(r.b, s) == cudaSuccess;
  }
  ~ProfScope() {
    if (!on) return;
    cudaEventRecord(r.e, s);
    t_recs.push_back(r);
  }
};

}  // namespace mc
