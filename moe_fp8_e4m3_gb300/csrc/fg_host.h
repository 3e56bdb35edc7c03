// fg_host.h - what the entry points outside fg_api.cu need of the library's per-device state
// and of its TMA map encoder.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace fg {

struct HostState {
    int sms;                         // SMs the kernels may use
    int* status;                     // device status word
    unsigned long long timeout_ns;   // bound of every wait
    int pdl, debug_stall;
};

// The current device's state: FG_OK, or FG_ERR_CUDA when there is no usable device.
int host_state(HostState* out);

// Row-major tiled tensor map of `rank` dimensions (innermost first; pitches in bytes of
// dimensions 1..rank-1); elements outside the array read as zero.
bool encode_tiled(CUtensorMap* map, CUtensorMapDataType type, int rank, const void* base, const uint64_t* dims,
                  const uint64_t* pitches, const uint32_t* box, CUtensorMapSwizzle swizzle);

bool print_configs_enabled();

// p is a multiple of n, a power of two.
inline bool al(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline int align4(int x) { return (x + 3) / 4 * 4; }
inline long long up256(long long x) { return (x + 255) / 256 * 256; }

}  // namespace fg
