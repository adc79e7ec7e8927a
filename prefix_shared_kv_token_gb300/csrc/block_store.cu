// kv_store_block: new K/V rows quantised into the pages of a block-scaled pool.
//
// Tokens come as kv_store takes them; tokens of one page stand next to each other in the call,
// at consecutive offsets (a *run*).  For each run, KV head and tensor:
//     e_new = the smallest exponent with max |x| over the run's finite values <= 448 * 2^e_new;
//     e = e_new when the run starts its page (offset 0: what the page held before is dead),
//         else max(e_old, e_new), and where that is above e_old the page's earlier rows are
//         rescaled: code' = e4m3(code * 2^(e_old - e));
//     code = e4m3(x * 2^-e), round to nearest even, saturating; NaN is stored as NaN.
//
// Bound: HBM (bf16 rows in, codes out).  One warp owns a run of one (KV head, tensor), since the
// exponent needs the whole run before its first code: 16 rows at a time sit in registers (16-byte
// loads, all in flight), so a run of at most 16 rows is read once; longer runs read their rows
// again from L2 for the second pass.

#include <algorithm>

#include "block.cuh"

namespace pkv {

struct BlockStoreParams {
    const uint16_t *k_new, *v_new;
    uint8_t *k, *v, *k_exp, *v_exp;
    const int32_t *loc;
    int64_t n, num_slots, slot_bytes;
    int32_t hkv, shift, window;
    int32_t *err;
};

// |x| bits of the larger finite bf16 half of w
PKV_DEV uint32_t finite_amax(uint32_t w, uint32_t m) {
    const uint32_t a = w & 0x7FFFu, b = (w >> 16) & 0x7FFFu;
    if (a < 0x7F80u) m = max(m, a);
    if (b < 0x7F80u) m = max(m, b);
    return m;
}

template <int D>
__global__ void __launch_bounds__(256) block_store_kernel(const BlockStoreParams p) {
    constexpr int kLanes = D / 8;          // lanes of 16 bytes for one row
    constexpr int kRows = 32 / kLanes;     // rows a warp-wide load covers
    constexpr int kChunk = 16, kLoads = kChunk / kRows;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int unit = blockIdx.y * 8 + (threadIdx.x >> 5);
    if (unit >= 2 * p.hkv) return;
    const int tensor = unit >= p.hkv, head = unit - tensor * p.hkv;
    const int mask = (1 << p.shift) - 1;
    const int row_in = lane / kLanes, col = (lane % kLanes) * 8;
    const uint16_t *src = (tensor ? p.v_new : p.k_new) + (int64_t)head * D + col;
    const int64_t src_row = (int64_t)p.hkv * D;
    uint8_t *codes = (tensor ? p.v : p.k) + (int64_t)head * D;
    uint8_t *exps = (tensor ? p.v_exp : p.k_exp) + head;

    const int64_t w0 = (int64_t)blockIdx.x * p.window, w1 = min(w0 + p.window, p.n);
    for (int64_t i = w0; i < w1; ++i) {
        const int32_t slot = __ldg(p.loc + i);
        if (slot < 0 || (int64_t)slot >= p.num_slots) {
            if (slot != -1 && lane == 0) set_error(p.err, DERR_SLOT_RANGE);  // -1 is padding
            continue;
        }
        const int off = slot & mask;
        if (i > 0 && off > 0 && __ldg(p.loc + i - 1) == slot - 1) continue;  // inside a run
        // the run's length: consecutive slots up to the page's end
        const int most = (int)min((int64_t)(mask + 1 - off), p.n - i);
        int len = 1;
        while (len < most) {
            const int j = len + lane;
            const bool on = j < most && __ldg(p.loc + i + j) == slot + j;
            const uint32_t stop = ~__ballot_sync(0xffffffffu, on);
            len += stop ? __ffs(stop) - 1 : 32;
            if (stop) break;
        }
        uint4 x[kLoads];
        uint32_t amax = 0;
        for (int c = 0; c < len; c += kChunk) {
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
                const int j = c + k * kRows + row_in;
                x[k] = make_uint4(0u, 0u, 0u, 0u);
                if (j < len) x[k] = __ldg(reinterpret_cast<const uint4 *>(src + (i + j) * src_row));
            }
#pragma unroll
            for (int k = 0; k < kLoads; ++k)
                amax = finite_amax(x[k].w, finite_amax(x[k].z, finite_amax(x[k].y, finite_amax(x[k].x, amax))));
        }
        amax = __reduce_max_sync(0xffffffffu, amax);
        // bf16 bits: exponent field + 1 where the mantissa is above 1.75, less 8 (448 = 1.75 * 2^8)
        int e = clamp_exp((int)((amax + 0x1Fu) >> 7) - 8);
        uint8_t *page_exp = exps + (int64_t)(slot >> p.shift) * p.hkv;
        if (off > 0) {
            const int old = clamp_exp(*page_exp);
            if (e > old) {
                const float f = exp_value(max(old - e + 127, 1));
                uint8_t *first = codes + (int64_t)(slot - off) * p.slot_bytes;
                for (int b = lane; b < off * (D / 4); b += 32) {
                    uint32_t *at = reinterpret_cast<uint32_t *>(first + (int64_t)(b / (D / 4)) * p.slot_bytes) + b % (D / 4);
                    const uint32_t w = *at, lo = e4m3x2_to_f16x2(w), hi = e4m3x2_hi_to_f16x2(w);
                    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
                    const float2 z = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
                    *at = (uint32_t)f32x2_to_e4m3x2(a.x * f, a.y * f) | ((uint32_t)f32x2_to_e4m3x2(z.x * f, z.y * f) << 16);
                }
            } else {
                e = old;
            }
        }
        if (lane == 0) *page_exp = (uint8_t)e;
        const float f = exp_value(254 - e);  // 2^-(e - 127)
        for (int c = 0; c < len; c += kChunk) {
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
                const int j = c + k * kRows + row_in;
                if (j >= len) continue;
                if (len > kChunk) x[k] = __ldg(reinterpret_cast<const uint4 *>(src + (i + j) * src_row));
                const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
                uint32_t y[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) y[u] = f32x2_to_e4m3x2(bf16_lo(w[u]) * f, bf16_hi(w[u]) * f);
                *reinterpret_cast<uint2 *>(codes + (int64_t)(slot + j) * p.slot_bytes + col) =
                    make_uint2(y[0] | (y[1] << 16), y[2] | (y[3] << 16));
            }
        }
    }
}

}  // namespace pkv

extern "C" int pkv_kv_store_block(const pkv_block_pool *pool, const void *k_new, const void *v_new,
                                  const int32_t *out_cache_loc, int64_t n, void *workspace, void *stream) {
    using namespace pkv;
    const int rc = validate_block_pool(pool);
    if (rc) return rc;
    if (n < 0 || n >= ((int64_t)1 << 31)) return PKV_E_INVALID;
    if (n == 0) return PKV_OK;
    if (!k_new || !v_new || !out_cache_loc) return PKV_E_INVALID;
    if ((reinterpret_cast<uintptr_t>(k_new) | reinterpret_cast<uintptr_t>(v_new)) & 15) return PKV_E_INVALID;
    BlockStoreParams p;
    p.k_new = static_cast<const uint16_t *>(k_new);
    p.v_new = static_cast<const uint16_t *>(v_new);
    p.k = static_cast<uint8_t *>(pool->k);
    p.v = static_cast<uint8_t *>(pool->v);
    p.k_exp = pool->k_exp;
    p.v_exp = pool->v_exp;
    p.loc = out_cache_loc;
    p.n = n;
    p.num_slots = pool->num_pages * pool->page_size;
    p.slot_bytes = block_slot_bytes(pool);
    p.hkv = pool->num_kv_heads;
    p.shift = log2_of(pool->page_size);
    p.err = static_cast<int32_t *>(workspace);
    // tokens a CTA looks through: one while that leaves the GPU with less than a wave, else 16
    p.window = n >= 16 * (int64_t)num_sms() ? 16 : 1;
    const dim3 grid((unsigned)((n + p.window - 1) / p.window), (unsigned)((2 * p.hkv + 7) / 8));
    const cudaError_t e = launch_pdl(pool->head_dim == 128 ? block_store_kernel<128> : block_store_kernel<64>, grid,
                                     dim3(256), 0, reinterpret_cast<cudaStream_t>(stream), true, p);
    return e == cudaSuccess ? PKV_OK : PKV_E_CUDA;
}
