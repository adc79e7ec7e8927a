// The block-scaled 8-bit KV cache: e4m3 codes in pages of P tokens, one exponent byte per
// (page, KV head) for K and one for V.  A code c under byte b stands for c * 2^(b - 127).
//
// Scales are powers of two.  Dividing a bf16 value by one is exact, so a stored code is a single
// rounding of its value; a page whose exponent has to grow is rescaled exactly but for e4m3's
// subnormals; and every value is a bf16 value, so the tensor-core path reads it unrounded.  A
// floating-point code keeps its relative precision under a scale up to twice as coarse as
// amax / 448.
#pragma once

#include <cuda_fp16.h>

#include "../../include/pkv.h"
#include "common.cuh"
#include "launch.h"

namespace pkv {

// Exponent bytes a page may have: 2^-117 keeps the smallest code (2^-9) a normal bf16 value,
// 2^118 keeps the largest (448) finite in bf16.
constexpr int kExpMin = 10, kExpMax = 245;

PKV_DEV int clamp_exp(int b) { return min(max(b, kExpMin), kExpMax); }
// 2^(b - 127) for b in [1, 254]
PKV_DEV float exp_value(int b) { return __uint_as_float((uint32_t)b << 23); }

// Two e4m3 codes (low byte first) -> f16x2, exactly (every e4m3 value is an f16 value).
PKV_DEV uint32_t e4m3x2_to_f16x2(uint32_t v) {
    uint32_t h;
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(h) : "r"(v));
    return h;
}
PKV_DEV uint32_t e4m3x2_hi_to_f16x2(uint32_t v) {
    uint32_t h;
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, u;\n\t}" : "=r"(h) : "r"(v));
    return h;
}

inline int validate_block_pool(const pkv_block_pool *p) {
    if (!p || !p->k || !p->v || !p->k_exp || !p->v_exp) return PKV_E_INVALID;
    if (p->num_pages <= 0 || p->num_kv_heads <= 0) return PKV_E_INVALID;
    if (p->head_dim != 64 && p->head_dim != 128) return PKV_E_UNSUPPORTED;
    if (p->page_size < 16 || p->page_size > 256 || (p->page_size & (p->page_size - 1))) return PKV_E_UNSUPPORTED;
    if (p->num_pages >= ((int64_t)1 << 31) ||
        p->num_pages * p->page_size >= ((int64_t)1 << 31) / p->num_kv_heads)
        return PKV_E_UNSUPPORTED;
    if ((reinterpret_cast<uintptr_t>(p->k) | reinterpret_cast<uintptr_t>(p->v)) & 15) return PKV_E_INVALID;
    if (p->slot_stride != 0 &&
        (p->slot_stride < (int64_t)p->num_kv_heads * p->head_dim || (p->slot_stride & 15)))
        return PKV_E_INVALID;
    return PKV_OK;
}

inline int64_t block_slot_bytes(const pkv_block_pool *p) {
    return p->slot_stride != 0 ? p->slot_stride : (int64_t)p->num_kv_heads * p->head_dim;
}

inline int log2_of(int x) {
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

}  // namespace pkv
