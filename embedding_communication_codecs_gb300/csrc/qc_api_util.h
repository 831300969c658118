// qc_api_util.h -- what the C ABI's translation units share: error reporting and
// the checks of addresses.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/qcodec.h"

namespace qc {
namespace api {

// Stores the message that qc_last_error() returns, and returns `st`.
qc_status fail(qc_status st, const char *fmt, ...);
// QC_OK, with the message cleared.
qc_status ok();
qc_status from_cuda(cudaError_t e, const char *what);
// The status word that launches from this thread report failures into, or null.
uint32_t *status_word();

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// [a, a+na) and [b, b+nb) (bytes) share a byte.
inline bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
    if (!a || !b || na == 0 || nb == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

}  // namespace api
}  // namespace qc
