// Host-side helpers that the library's translation units share (definitions in gdn_api.cu).
#pragma once

#include <atomic>
#include <cstdint>

#include "gdn.h"

namespace gdn {

// Bit of the device error word: a block-table entry or a sequence length outside the paged cache.
constexpr unsigned kErrPages = 4u;

// Records a printf-style message as the calling thread's last error and returns `st`.
gdn_status fail(gdn_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

// Forgets the calling thread's last error (every entry point does so first).
void clear_error();

// Device address of the current device's error word; nullptr with *st set when the look-up fails.
unsigned* err_word_ptr(gdn_status* st);

// Whether the device time-out diagnostic is on (gdn_debug_stall).
bool debug_stall();

// Allows `Kern` up to `bytes` of dynamic shared memory on the current device, once per device and process.
template <auto Kern>
cudaError_t allow_shared(int bytes) {
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace gdn
