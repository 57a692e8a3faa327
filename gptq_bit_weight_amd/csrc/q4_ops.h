// Internal declarations of the operators around the quantized product:
// rotary positions, the paged cache and attention over it, adapters.
#pragma once

#include <hip/hip_runtime.h>

#include "q4_internal.h"

struct q4_rotary {
    uint64_t* turns = nullptr;   // [rot / 2] on the device: turns a position, times 2^64
    float magnitude = 1.f;
    int dim = 0, rot = 0;
    bool interleaved = false;
    int device = -1;
};

namespace q4 {

// The current device, checked to be gfx950, and its CUs (looked up once a
// device).
q4_status device_info(int* dev, int* num_cu);
// Shape and pointers of a cache description.
q4_status check_cache(const q4_cache* c, const char* who);

}  // namespace q4
