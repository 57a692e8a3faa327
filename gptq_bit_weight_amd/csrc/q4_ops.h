// Internal declarations of the operators around the quantized product:
// rotary positions, the paged cache and attention over it, adapters.
#pragma once

#include <hip/hip_runtime.h>

#include "q4_internal.h"
#include "q4_meet.h"

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
// A rotary handle and its positions: widths, and that it was made on the current device.
q4_status check_rotary(const q4_rotary* r, const void* positions, int position_bits, const char* who);

// (of one token, or one head, the stride does not count)
inline bool same_view(const uint16_t* a, int64_t at, int64_t ah, const uint16_t* b, int64_t bt, int64_t bh, int tokens, int heads)
{
    return a == b && (at == bt || tokens == 1) && (ah == bh || heads == 1);
}

// 16-bit values of `tokens` tokens and `heads` heads; the keys or values of a cache.
inline View head_view(const void* at, int64_t token, int64_t head, int tokens, int heads, int dim)
{
    return View{at, (int64_t)dim * 2, {{tokens, token * 2}, {heads, head * 2}, {1, 0}}};
}
inline View cache_view(const q4_cache* c, bool values)
{
    const int64_t* s = values ? c->v_stride : c->k_stride;
    return View{values ? c->v : c->k, (int64_t)c->dim * 2,
                {{c->pages, s[0] * 2}, {c->kv_heads, s[1] * 2}, {c->page_size, s[2] * 2}}};
}
inline View flat_view(const void* at, int64_t bytes) { return View{at, bytes, {{1, 0}, {1, 0}, {1, 0}}}; }

}  // namespace q4
