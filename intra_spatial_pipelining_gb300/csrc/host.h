// What the C entry points outside runtime.cu share with it (all defined there).
#pragma once

#include "serving.h"
#include "sgp.h"

namespace sgp {

// Record the text of sgp_last_error and return the status code.
int host_fail_arg(const char* what);
int host_fail_cuda(cudaError_t e, const char* what);

// Launches on a stream, shared-memory limits included (cudaError_t as int).
int host_launch(cudaStream_t s, const void* func, dim3 grid, dim3 block, size_t smem, void** args,
                bool overlap_ok);

// bf16 tensor maps over two buffers of [rows][inner], box {box_inner, box_rows}, 128-byte swizzle.
int host_tmap_pair(CUtensorMap* a, CUtensorMap* b, const void* base_a, const void* base_b,
                   uint64_t inner, uint64_t rows, uint32_t box_inner, uint32_t box_rows);

bool host_driver_ready();               // tensor maps can be encoded
int host_sms();                         // SMs of the current device
KCtx host_ctx(void* status, uint32_t op);
constexpr int kHostMaxTokens = 512;     // sequences per call

}  // namespace sgp
