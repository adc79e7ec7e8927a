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
// Bound: HBM (bf16 rows in, codes out).  The exponent needs the whole run before its first code, so a
// run's rows wait in registers, 16 rows (4 KB at d = 128) a warp with all their loads in flight: 1, 2, 4
// or 8 warps share a run of one (KV head, tensor) by its length, and the rows are read once.  131,072
// tokens of 8 heads x 128 in pages of 64: 145 us, 5.5 TB/s (one warp a run, reading runs of more than
// 16 rows twice: 217 us).  The quantisation itself is 5 us of it.

#include <algorithm>

#include "block.cuh"

namespace pkv {

constexpr int kWindow = 64;  // tokens a CTA looks through, at most

struct BlockStoreParams {
    const uint16_t *k_new, *v_new;
    uint8_t *k, *v, *k_exp, *v_exp;
    const int32_t *loc;
    int64_t n, num_slots, slot_bytes;
    int32_t hkv, shift, window;
    int32_t *err;
};

// |x| bits of the bf16 halves of w, maximised half by half into m.
PKV_DEV uint32_t max_abs2(uint32_t w, uint32_t m) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(w & 0x7FFF7FFFu), "r"(m));
    return r;
}
PKV_DEV uint32_t larger_half(uint32_t m) { return max(m & 0xFFFFu, m >> 16); }
// w with its infinities and NaN as zeros.
PKV_DEV uint32_t finite2(uint32_t w) {
    return ((w & 0x7FFFu) < 0x7F80u ? w & 0xFFFFu : 0u) | (((w >> 16) & 0x7FFFu) < 0x7F80u ? w & 0xFFFF0000u : 0u);
}
// The codes of two bf16 values times the power of two f: the product is exact in fp32 (-0 as the
// addend keeps a zero's sign), so the conversion rounds once.
PKV_DEV uint32_t quantise2(uint32_t w, uint16_t f) {
    uint16_t y;
    asm("{\n\t.reg .b16 l, h;\n\t.reg .f32 a, b;\n\tmov.b32 {l, h}, %1;\n\tfma.rn.f32.bf16 a, l, %2, 0f80000000;\n\t"
        "fma.rn.f32.bf16 b, h, %2, 0f80000000;\n\tcvt.rn.satfinite.e4m3x2.f32 %0, b, a;\n\t}"
        : "=h"(y)
        : "r"(w), "h"(f));
    return y;
}

PKV_DEV bool is_slot(const BlockStoreParams &p, int32_t s) { return s >= 0 && (int64_t)s < p.num_slots; }

// Whether token i, in a slot of the pool, begins a run: its page's first row, or not behind its
// neighbour (over skipped tokens).
PKV_DEV bool begins_run(const BlockStoreParams &p, int64_t i, int32_t slot) {
    const int off = slot & ((1 << p.shift) - 1);
    for (int d = 1; d <= off && d <= i; ++d) {
        const int32_t s = ld(p.loc + i - d);
        if (is_slot(p, s)) return s != slot - d;
    }
    return true;
}

// Tokens from i on in consecutive slots of one page (a warp's lanes look together).  A skipped token
// leaves its row out of the run: holes.
PKV_DEV int run_length(const BlockStoreParams &p, int64_t i, int32_t slot, bool &holes) {
    const int mask = (1 << p.shift) - 1, lane = threadIdx.x & 31;
    const int most = (int)min((int64_t)(mask + 1 - (slot & mask)), p.n - i);
    int len = 1;
    holes = false;
    while (len < most) {
        const int j = len + lane;
        const int32_t s = j < most ? ld(p.loc + i + j) : -1;
        const bool here = s == slot + j, out = j < most && !is_slot(p, s);
        const uint32_t stop = ~__ballot_sync(0xffffffffu, here || out), skip = __ballot_sync(0xffffffffu, out);
        const int more = stop ? __ffs(stop) - 1 : 32;
        holes |= (more == 32 ? skip : skip & ((1u << more) - 1)) != 0;
        len += more;
        if (stop) break;
    }
    return len;
}

template <int D>
__global__ void __launch_bounds__(256) block_store_kernel(const BlockStoreParams p) {
    constexpr int kLanes = D / 8;          // lanes of 16 bytes for one row
    constexpr int kRows = 32 / kLanes;     // rows a warp-wide load covers
    constexpr int kChunk = 16, kLoads = kChunk / kRows;
    __shared__ int32_t num_runs;
    __shared__ int32_t runs[kWindow], slots[kWindow], lens[kWindow];  // the window's runs: first token, slot, length (< 0: holes)
    __shared__ uint32_t part[8];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int mask = (1 << p.shift) - 1;
    const int64_t w0 = (int64_t)blockIdx.x * p.window;
    if (warp == 0) {
        int count = 0;
        for (int t = 0; t < p.window; t += 32) {
            const int64_t i = w0 + t + lane;
            bool begins = false;
            if (t + lane < p.window && i < p.n) {
                const int32_t slot = ld(p.loc + i);
                begins = is_slot(p, slot) && begins_run(p, i, slot);
                if (slot != -1 && !is_slot(p, slot) && blockIdx.y == 0) set_error(p.err, DERR_SLOT_RANGE);
            }
            const uint32_t who = __ballot_sync(0xffffffffu, begins);
            if (begins) {
                const int k = count + __popc(who & ((1u << lane) - 1));
                runs[k] = t + lane;
                slots[k] = ld(p.loc + i);
            }
            count += __popc(who);
        }
        if (lane == 0) num_runs = count;
    }
    __syncthreads();
    const int count = num_runs;
    if (count == 0) return;
    for (int k = warp; k < count; k += 8) {
        bool holes;
        const int len = run_length(p, w0 + runs[k], slots[k], holes);
        if (lane == 0) lens[k] = holes ? -len : len;
    }
    __syncthreads();
    // warps that share a run, by the first one's length (any number is right for any run)
    int share = 1;
    while (share < 8 && share * kChunk < abs(lens[0])) share *= 2;
    const int group = warp / share, sub = warp % share, groups = 8 / share;
    const int units = min(8, 2 * p.hkv - (int)blockIdx.y * 8);
    const int row_in = lane / kLanes, col = (lane % kLanes) * 8;
    const int64_t src_row = (int64_t)p.hkv * D;

    for (int k = group; k < count * units; k += groups) {  // pairs of run and unit, dealt in turn
        const int run = units == 8 ? k >> 3 : k / units, unit = blockIdx.y * 8 + (k - run * units);
        const int tensor = unit >= p.hkv, head = unit - tensor * p.hkv;
        const int64_t i = w0 + runs[run];
        const int32_t slot = slots[run];
        const uint16_t *src = (tensor ? p.v_new : p.k_new) + i * src_row + (int64_t)head * D + col;
        uint8_t *codes = (tensor ? p.v : p.k) + (int64_t)head * D;
        uint8_t *page_exp = (tensor ? p.v_exp : p.k_exp) + (int64_t)(slot >> p.shift) * p.hkv + head;
        const int off = slot & mask;
        const int len = abs(lens[run]);
        const bool holes = lens[run] < 0;
        auto stored = [&](int j) { return j < len && (!holes || ld(p.loc + i + j) == slot + j); };
        const int old = off > 0 ? clamp_exp(*page_exp) : 0;
        const bool held = len <= share * kChunk;  // the group's registers hold the run
        uint4 x[kLoads];
        uint32_t amax = 0, good = 0;
        for (int c = sub * kChunk; c < len; c += share * kChunk) {
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                const int j = c + u * kRows + row_in;
                x[u] = make_uint4(0u, 0u, 0u, 0u);
                if (stored(j)) x[u] = __ldcs(reinterpret_cast<const uint4 *>(src + j * src_row));
            }
#pragma unroll
            for (int u = 0; u < kLoads; ++u)
                amax = max_abs2(x[u].w, max_abs2(x[u].z, max_abs2(x[u].y, max_abs2(x[u].x, amax))));
            if (larger_half(amax) >= 0x7F80u) {  // an infinity or NaN: again, without them
                amax = good;
#pragma unroll
                for (int u = 0; u < kLoads; ++u)
                    amax = max_abs2(finite2(x[u].w), max_abs2(finite2(x[u].z), max_abs2(finite2(x[u].y), max_abs2(finite2(x[u].x), amax))));
            }
            good = amax;
        }
        amax = __reduce_max_sync(0xffffffffu, larger_half(amax));
        if (share > 1) {
            if (lane == 0) part[warp] = amax;
            named_bar_sync(1 + group, share * 32);
            amax = __reduce_max_sync(0xffffffffu, lane < share ? part[group * share + lane] : 0u);
            named_bar_sync(1 + group, share * 32);  // part is free again, and every warp has read `old`
        } else {
            __syncwarp();
        }
        // bf16 bits: exponent field + 1 where the mantissa is above 1.75, less 8 (448 = 1.75 * 2^8)
        int e = clamp_exp((int)((amax + 0x1Fu) >> 7) - 8);
        if (off > 0) {
            if (e > old) {
                const float f = exp_value(max(old - e + 127, 1));
                uint8_t *first = codes + (int64_t)(slot - off) * p.slot_bytes;
                for (int b = sub * 32 + lane; b < off * (D / 4); b += share * 32) {
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
        if (sub == 0 && lane == 0) *page_exp = (uint8_t)e;
        const uint16_t f = (uint16_t)((254 - e) << 7);  // 2^-(e - 127) in bf16
        for (int c = sub * kChunk; c < len; c += share * kChunk) {
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                const int j = c + u * kRows + row_in;
                if (!stored(j)) continue;
                if (!held) x[u] = ld(reinterpret_cast<const uint4 *>(src + j * src_row));
                *reinterpret_cast<uint2 *>(codes + (int64_t)(slot + j) * p.slot_bytes + col) =
                    make_uint2(__byte_perm(quantise2(x[u].x, f), quantise2(x[u].y, f), 0x5410),
                               __byte_perm(quantise2(x[u].z, f), quantise2(x[u].w, f), 0x5410));
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
    if (reinterpret_cast<uintptr_t>(workspace) & 3) return PKV_E_INVALID;  // (its error word is changed atomically)
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
    // tokens a CTA looks through: as many as leave the GPU four CTAs an SM, up to a page
    const int64_t y = (2 * p.hkv + 7) / 8, want = 4 * (int64_t)num_sms();
    p.window = 1;
    while (p.window < std::min<int>(kWindow, pool->page_size) && (n + 2 * p.window - 1) / (2 * p.window) * y >= want)
        p.window *= 2;
    const dim3 grid((unsigned)((n + p.window - 1) / p.window), (unsigned)y);
    const cudaError_t e = launch_pdl(pool->head_dim == 128 ? block_store_kernel<128> : block_store_kernel<64>, grid,
                                     dim3(256), 0, reinterpret_cast<cudaStream_t>(stream), true, p);
    return e == cudaSuccess ? PKV_OK : PKV_E_CUDA;
}
