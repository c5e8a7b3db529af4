// What the entry points' host code shares (internal to the library): the status word, launch tracing,
// tensor maps and the argument helpers. Defined in api.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "sparsesam.h"

namespace ss {

// Device address of the current device's status word (null: the lookup failed).
int* status_word();
// SMs of the current device.
int sm_count();

// The GEMM and attention work splits are planned for the B200's 148 SMs, so workspace sizes do
// not depend on the device a call runs on; launches use min(units, the device's SMs) CTAs.
constexpr int kPlanSMs = 148;

// bf16 tensor of `mats` matrices [rows, inner] with rows `row_bytes` apart; box [box_rows, box_inner].
// `rank` must match the dimensionality of the kernel's TMA instruction (2: one matrix, 3: a stack).
bool encode_bf16(CUtensorMap* m, cuuint32_t rank, const void* base, uint64_t inner, uint64_t rows,
                 uint64_t mats, uint64_t row_bytes, uint32_t box_inner, uint32_t box_rows,
                 CUtensorMapSwizzle sw);

// Tracing of one launch: trace_open records its first event and returns its record (-1: not
// tracing), trace_close the second; count_launch counts it.
int trace_open(const char* name, cudaStream_t st);
void trace_close(int rec, cudaStream_t st);
void count_launch();

template <class F>
cudaError_t traced(const char* name, cudaStream_t st, F&& f) {
  const int rec = trace_open(name, st);
  const cudaError_t e = f();
  if (rec >= 0) trace_close(rec, st);
  count_launch();
  return e;
}

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline int cuda_err(cudaError_t e) { return e == cudaSuccess ? SS_OK : SS_ECUDA; }

}  // namespace ss
