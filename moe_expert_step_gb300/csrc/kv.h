// Host-side checks and device addressing shared by the paged key-value cache calls.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "moestep.h"

namespace moestep {

inline bool kv_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline int kv_act_bytes(int dtype) { return dtype == MOESTEP_F32 ? 4 : 2; }

inline int check_kv_dims(const moestep_kv_dims* d) {
    if (d == nullptr) return MOESTEP_EINVAL;
    if (d->Hq <= 0 || d->Hkv <= 0 || d->D <= 0 || d->page <= 0 || d->n_pages <= 0 || d->max_pages <= 0)
        return MOESTEP_EINVAL;
    if (d->dtype != MOESTEP_BF16 && d->dtype != MOESTEP_F32 && d->dtype != MOESTEP_FP8) return MOESTEP_EINVAL;
    if (d->Hq % d->Hkv || d->Hq > 1024) return MOESTEP_EUNSUPPORTED;
    if (d->D != 64 && d->D != 128) return MOESTEP_EUNSUPPORTED;
    if (d->page != 16 && d->page != 32 && d->page != 64 && d->page != 128) return MOESTEP_EUNSUPPORTED;
    const long long lim = (1ll << 31) - 1;
    if (1ll * d->max_pages * d->page > lim - 255) return MOESTEP_EUNSUPPORTED;
    if (1ll * d->n_pages * d->Hkv > lim / d->page) return MOESTEP_EUNSUPPORTED;
    return MOESTEP_OK;
}

inline int check_kv_cache(const moestep_kv_dims* d, const moestep_kv_cache* c) {
    if (c == nullptr || !c->k || !c->v || !c->table) return MOESTEP_EINVAL;
    if (d->dtype == MOESTEP_FP8 && (!c->k_exp || !c->v_exp)) return MOESTEP_EINVAL;
    if (!kv_aligned16(c->k) || !kv_aligned16(c->v) || !kv_aligned16(c->table)) return MOESTEP_EALIGN;
    if (d->dtype == MOESTEP_FP8 && (!kv_aligned16(c->k_exp) || !kv_aligned16(c->v_exp))) return MOESTEP_EALIGN;
    return MOESTEP_OK;
}

// rows `ld` elements apart that hold `width` elements each
inline int check_kv_rows(const void* p, long long ld, long long width, int dtype) {
    if (!p || ld < width) return MOESTEP_EINVAL;
    if (!kv_aligned16(p) || (ld * kv_act_bytes(dtype)) % 16) return MOESTEP_EALIGN;
    return MOESTEP_OK;
}

constexpr size_t kKvHeader = 512;  // error word and timeout record, as in every workspace

inline int check_kv_ws(const void* ws, size_t have, size_t need) {
    if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255u) || have < need) return MOESTEP_EWORKSPACE;
    return MOESTEP_OK;
}

}  // namespace moestep
