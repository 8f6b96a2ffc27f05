// Host helpers of the calls that take no handle.
#pragma once

#include <cstdint>
#include <string>

#include <cuda_runtime.h>

#include "zero_gb300.h"
#include "zero_internal.h"

namespace zg {
namespace {

inline int refuse(int code, const std::string& msg) {
    set_global_error(msg.c_str());
    return code;
}
inline int cuda_refuse(cudaError_t e, const char* what) {
    cudaGetLastError();
    return refuse(ZERO_ECUDA, std::string(what) + ": " + cudaGetErrorString(e));
}
inline bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
inline uint64_t up(uint64_t x, uint64_t to) { return (x + to - 1) / to * to; }

}  // namespace

// The ring stage whose barrier block 0 of the next matrix kernel is to wait for
// in vain, counted from 1, or 0; takes it (zero_debug_hold_matrix).
uint32_t take_matrix_hold();

}  // namespace zg
