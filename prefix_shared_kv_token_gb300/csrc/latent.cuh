// The latent pool: one row a token, its latent (keys and values of every head come from it) and
// behind it the rotary key that all heads share.
#pragma once

#include "../../include/pkv.h"
#include "common.cuh"
#include "launch.h"

namespace pkv {

constexpr int kLatentRope = 64;  // elements of the rotary key

inline int64_t latent_stride(const pkv_latent_pool *p) {
    return p->slot_stride != 0 ? p->slot_stride : (int64_t)p->latent_dim + p->rope_dim;
}

inline int validate_latent_pool(const pkv_latent_pool *p) {
    if (!p || !p->rows || p->num_slots <= 0) return PKV_E_INVALID;
    if ((p->latent_dim != 256 && p->latent_dim != 512) || p->rope_dim != kLatentRope) return PKV_E_UNSUPPORTED;
    if (p->num_slots >= ((int64_t)1 << 31)) return PKV_E_UNSUPPORTED;
    if (reinterpret_cast<uintptr_t>(p->rows) & 15) return PKV_E_INVALID;
    if (p->slot_stride != 0 && (p->slot_stride < p->latent_dim + p->rope_dim || (p->slot_stride & 7))) return PKV_E_INVALID;
    if (latent_stride(p) > ((int64_t)1 << 32)) return PKV_E_UNSUPPORTED;
    return PKV_OK;
}

}  // namespace pkv
