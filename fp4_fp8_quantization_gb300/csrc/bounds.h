// The condition of the debug builds' store guard, for the host too.
#pragma once

#include <stdint.h>

namespace moeq {

#ifdef __CUDACC__
#define MOEQ_HOST_DEVICE __host__ __device__
#else
#define MOEQ_HOST_DEVICE
#endif

// Whether the bytes [at, at + bytes) lie in the buffer [buf, buf + size).
MOEQ_HOST_DEVICE inline bool range_inside(const void *at, int64_t bytes, const void *buf,
                                          int64_t size) {
    const int64_t off = (int64_t)((uintptr_t)at - (uintptr_t)buf);
    return off >= 0 && bytes >= 0 && bytes <= size && off <= size - bytes;
}

}  // namespace moeq
