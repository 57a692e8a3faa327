// Host side of the cache held in 4 bits: its checks and the memory it takes.
#pragma once

#include "q4_ops.h"

namespace q4 {

// Shape, pointers, alignment and strides of a cache held in 4 bits.
q4_status check_cache4(const q4_cache4* c, const char* who);

inline View cache4_view(const q4_cache4* c, bool values, bool scales)
{
    const int64_t* s = scales ? (values ? c->v_scale_stride : c->k_scale_stride) : values ? c->v_stride : c->k_stride;
    return View{scales ? (values ? c->v_scale : c->k_scale) : values ? c->v : c->k,
                scales ? (int64_t)c->dim / c->group * 4 : (int64_t)c->dim / 2,
                {{c->pages, s[0]}, {c->kv_heads, s[1]}, {c->page_size, s[2]}}};
}

inline bool meets_cache4(const View& v, const q4_cache4* c)
{
    return meet(v, cache4_view(c, false, false)) || meet(v, cache4_view(c, true, false)) || meet(v, cache4_view(c, false, true)) ||
           meet(v, cache4_view(c, true, true));
}

}  // namespace q4
