// experts.hpp -- what the expert products (experts.cu) and the 8-bit codes
// (quantize.cu) share: argument checks, element access, programmatic launches.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "himuon.h"

namespace himuon {

int device_usable();         // api.cu: HIMUON_OK or HIMUON_ERR_NO_DEVICE for the current device
int *device_status_word();   // api.cu: the current device's status word
// HIMUON_OK, or why the current device cannot be used.  The first call on a
// device loads every kernel of the expert entry points, so that a call captured
// into a graph later loads nothing.
int expert_device();         // experts.cu
bool load_quantize();        // quantize.cu: its part of that
int sm_count();              // experts.cu: SMs of the current device

// Matrices in the parameters of one launch (longer lists run as several).
constexpr int kMaxList = 64;

// ---------------------------------------------------------------- argument checks
inline size_t size_of(int32_t dt) { return dt == HIMUON_FP32 ? 4 : dt == HIMUON_I8 ? 1 : 2; }
inline bool is16(int32_t dt) { return dt == HIMUON_BF16 || dt == HIMUON_FP16; }
inline bool is_float(int32_t dt) { return dt >= HIMUON_BF16 && dt <= HIMUON_FP32; }

// Longest side of an operand: a sum of that length still ends well inside the
// kernels' bounded waits (two seconds).
constexpr int64_t kMaxSide = (int64_t)1 << 27;
constexpr int32_t kMaxGroups = 1 << 16;

// A matrix operand: shape, pointer and 16-byte alignment of its rows.
// `min_rows` 0: a row operand, which may be empty (its pointer is not used).
inline int check_operand(const himuon_mat &m, int64_t min_rows) {
  if (m.rows < min_rows || m.cols < 1 || m.ld < m.cols || (m.rows > 0 && !m.data)) return HIMUON_ERR_INVALID;
  if (m.dtype < HIMUON_BF16 || m.dtype > HIMUON_I8) return HIMUON_ERR_UNSUPPORTED;
  if (m.rows > kMaxSide || m.cols > kMaxSide || m.ld > (int64_t)1 << 36) return HIMUON_ERR_UNSUPPORTED;
  if (m.rows > 0 && reinterpret_cast<uintptr_t>(m.data) % 16 != 0) return HIMUON_ERR_ALIGNMENT;
  // (the pitch of a single row is never used)
  if (m.rows > 1 && (m.ld * static_cast<int64_t>(size_of(m.dtype))) % 16 != 0) return HIMUON_ERR_ALIGNMENT;
  return HIMUON_OK;
}

// n matrices that differ in `data` alone.
inline int check_list(const himuon_mat *m, int32_t n) {
  for (int32_t e = 0; e < n; ++e) {
    const int rc = check_operand(m[e], 1);
    if (rc) return rc;
    if (m[e].rows != m[0].rows || m[e].cols != m[0].cols || m[e].ld != m[0].ld || m[e].dtype != m[0].dtype)
      return HIMUON_ERR_INVALID;
  }
  return HIMUON_OK;
}

// Scales: fp32, `rows` x `cols`, natural alignment.
inline int check_scale(const himuon_mat *m, int64_t rows, int64_t cols) {
  if (!m || m->rows != rows || m->cols != cols || m->ld < m->cols) return HIMUON_ERR_INVALID;
  if (m->dtype != HIMUON_FP32) return HIMUON_ERR_UNSUPPORTED;
  if (cols > 0 && rows > 0 && !m->data) return HIMUON_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(m->data) % 4 != 0) return HIMUON_ERR_ALIGNMENT;
  return HIMUON_OK;
}

__device__ __forceinline__ float ld_any(const void *p, int32_t dtype, int64_t i) {
  if (dtype == HIMUON_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
  if (dtype == HIMUON_FP16) return __half2float(static_cast<const __half *>(p)[i]);
  return static_cast<const float *>(p)[i];
}

// The expert entry points' launches follow one another without a gap: a kernel
// lets the next one start as soon as its CTAs have (its first part, which touches no memory of
// the stream's, runs under this one's end), and waits for everything before it
// in the stream to have completed ahead of its first access.
__device__ __forceinline__ void grid_start_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace himuon
