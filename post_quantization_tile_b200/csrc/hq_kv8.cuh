// hq_kv8.cuh -- the e4m3 KV cache as its kernels see it: pages [page][head][token][dim] of codes for
// keys and for values, one scale per page and head.
#pragma once
#include "hq_fp8.cuh"
#include "hq_launch.h"

namespace hq {

// argument checks common to the entry points on a cache
inline bool kv8_cache_ok(const hq_kv8_t* c)
{
    if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale || c->pages < 1 || c->pages > ((int64_t)1 << 31) - 1 ||
        c->heads < 1 || c->heads > 65535)
        return false;
    const uintptr_t al = reinterpret_cast<uintptr_t>(c->k) | reinterpret_cast<uintptr_t>(c->v);
    const uintptr_t a4 = reinterpret_cast<uintptr_t>(c->k_scale) | reinterpret_cast<uintptr_t>(c->v_scale);
    return !(al & 15u) && !(a4 & 3u);
}
inline bool kv8_shape_supported(const hq_kv8_t* c)
{
    return (c->dim == 64 || c->dim == 128) && (c->page == 16 || c->page == 32 || c->page == 64 || c->page == 128);
}

// whether rows of an output share memory: a dimension longer than one without a stride
template <int N>
inline bool expanded(const int64_t (&stride)[N], const int64_t (&length)[N])
{
    for (int i = 0; i < N; ++i)
        if (stride[i] == 0 && length[i] > 1) return true;
    return false;
}

inline int page_shift_of(int page) { return page == 16 ? 4 : (page == 32 ? 5 : (page == 64 ? 6 : 7)); }

}  // namespace hq
