// abi.h -- small helpers of the C ABI's host side, shared by its translation units.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "mla.h"

namespace mla {

constexpr size_t HDR = MLA_WS_HEADER_BYTES;

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline cudaStream_t S(mla_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }
inline uint32_t *err_word(void *ws) { return reinterpret_cast<uint32_t *>(ws); }
inline mla_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA; }
inline bool heads_ok(int H) { return H == 16 || H == 32 || H == 64 || H == 128; }

}  // namespace mla
