// Host-side helpers shared by the C-ABI entry points: workspace carving, alignment checks, status
// of a CUDA error, the groups' table.
#pragma once

#include "lora_kernels.h"

namespace lora {

constexpr size_t kWsAlign = 256;

struct Carve {
  char* base;
  size_t off = 0;
  explicit Carve(void* b) : base(static_cast<char*>(b)) {}
  template <typename T>
  T* take(size_t count) {
    off = (off + kWsAlign - 1) / kWsAlign * kWsAlign;
    T* p = base ? reinterpret_cast<T*>(base + off) : nullptr;
    off += count * sizeof(T);
    return p;
  }
};

inline bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Errors left behind by other code in this thread (cudaGetLastError reports the most recent
// error of any runtime call) are cleared before our launches, so that a LORA_ERR_CUDA is ours.
inline void clear_stale() { (void)cudaGetLastError(); }

// LORA_OK or LORA_ERR_CUDA, the latter kept for lora_last_cuda_error (api.cu).
int cuda_status(cudaError_t e);

// The groups of a prepare / update call, checked (api.cu).
int build_groups(int32_t n_groups, const lora_group* groups, GroupTab& g, const lora_adamw_hp* hp);

}  // namespace lora

#define LORA_TRY(expr)                                       \
  do {                                                       \
    cudaError_t _e = (expr);                                 \
    if (_e != cudaSuccess) return ::lora::cuda_status(_e);   \
  } while (0)
