// api_checks.h -- argument checks that the C ABI's translation units of the microscaled
// and mixture-of-experts operators share.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "common.cuh"
#include "mmact.h"
#include "mxfp4.cuh"

namespace mmact {
namespace {

constexpr int MAX_DEVICES = 64;
constexpr int64_t MAX_DIM = (int64_t(1) << 31) - 1;

[[maybe_unused]] bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
[[maybe_unused]] bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
[[maybe_unused]] int out_kind(mmact_dtype d) { return d == MMACT_BF16 ? OUT_BF16 : (d == MMACT_F16 ? OUT_F16 : OUT_F32); }
[[maybe_unused]] int elem_bytes(mmact_dtype d) { return d == MMACT_F32 ? 4 : 2; }
[[maybe_unused]] bool valid_16(mmact_dtype d) { return d == MMACT_F16 || d == MMACT_BF16; }
[[maybe_unused]] bool valid_float(mmact_dtype d) { return valid_16(d) || d == MMACT_F32; }
[[maybe_unused]] bool valid_act(mmact_act a) { return a >= MMACT_ACT_NONE && a <= MMACT_ACT_SILU; }
[[maybe_unused]] int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }
[[maybe_unused]] bool mx_dims(int64_t rows, int64_t K) { return rows >= 0 && K >= 0 && rows <= MAX_DIM && K <= MAX_DIM; }
[[maybe_unused]] mmact_status enqueued(cudaError_t e) { return e == cudaSuccess ? MMACT_OK : MMACT_ERR_CUDA; }

}  // namespace
}  // namespace mmact
