// capi_internal.h - what the translation units of the C ABI share (hidden
// symbols; defined in blasst_capi.cu).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdint>

namespace blasst {
namespace capi {

constexpr uint64_t kTimeoutNs = 2000000000ull;  // 2 s per bounded wait

// The address of the two device error words (waits that gave up, index errors)
// on the current device, or null.
int* error_word();
// A tiled tensor map with zero fill outside; false if it cannot be had. Works on
// host threads without a current context.
bool encode_tiled(CUtensorMap* map, CUtensorMapDataType dt, int rank, void* base, const cuuint64_t* dims,
                  const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swizzle);
// BLASST_OK or BLASST_ECUDA, with the error's text kept for
// blasst_last_cuda_error().
int cuda_status(cudaError_t e);

}  // namespace capi
}  // namespace blasst
