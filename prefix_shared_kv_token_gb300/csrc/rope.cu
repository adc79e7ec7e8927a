// Rotary positions: rope (any heads, in place or not), rope_store (q and k rotated, k and v stored
// into pool slots in the same pass) and latent_store (a latent normalised, its rotary key rotated,
// both written as one row of a latent pool).
//
// A pair (x1, x2) at frequency f and position p turns by the angle p f:
//     y1 = m (x1 cos - x2 sin),  y2 = m (x2 cos + x1 sin).
// f is held as the 64-bit fraction of a turn that one position adds, so the product with p wraps
// modulo a whole turn by itself: the reduction of the angle is exact, and its error is that of the
// fraction: p * 2^-65 turns for its last bit, and |p f| 2^-52 radians at most for f and its division by
// 2 pi in 64-bit floats.  The top 32 bits are the angle.  (A float product p f is off by
// 2^-24 of itself, 0.06 radians at position 10^6; a table of cosines would have to be read.)
//
// All three are bandwidth kernels: every element read once and written once, 16 bytes a load.  A
// warp takes a token, or a part of its heads while there are too few tokens to fill the GPU; a lane
// keeps one unit of 8 pairs (two 16-byte vectors) and walks the heads with it, so its 8 sines and
// cosines are computed once for all of them.

#include <algorithm>
#include <cmath>

#include "../../include/pkv.h"
#include "common.cuh"
#include "latent.cuh"
#include "launch.h"

namespace pkv {

// A lane's 8 cosines and sines.
struct Turn {
    float c[8], s[8];
};

// Sine and cosine of h * 2^-32 turns.  To the nearest quarter turn in integers; what remains, an angle of at most
// pi / 4, by the Taylor series up to the 9th and 8th power (the next terms are below 2e-9 and 3e-8).
PKV_DEV void sincos_of(int32_t h, float &sine, float &cosine) {
    const int32_t quarter = (int32_t)(((uint32_t)h + 0x20000000u) >> 30);
    const float x = (float)(int32_t)((uint32_t)h - ((uint32_t)quarter << 30)) * 1.4629180792671596e-9f;  // 2 pi / 2^32
    const float z = x * x;
    const float s = fmaf(x * z, fmaf(z, fmaf(z, fmaf(z, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6), x);
    const float c = fmaf(z, fmaf(z, fmaf(z, fmaf(z, 1.f / 40320, -1.f / 720), 1.f / 24), -0.5f), 1.f);
    sine = quarter & 1 ? c : s;
    cosine = quarter & 1 ? s : c;
    if (quarter & 2) sine = -sine;
    if ((quarter + 1) & 2) cosine = -cosine;
}

// Of pairs a .. a + 3 and b .. b + 3.
PKV_DEV Turn turn_of(const uint64_t *phases, int a, int b, int32_t pos, float magnitude) {
    Turn t;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint64_t turns = (uint64_t)(int64_t)pos * ld(phases + (i < 4 ? a + i : b + i - 4));  // modulo 2^64: modulo a turn
        float s, c;
        sincos_of((int32_t)(turns >> 32), s, c);
        t.c[i] = c * magnitude;
        t.s[i] = s * magnitude;
    }
    return t;
}

PKV_DEV void unpack8(const uint4 &v, float *x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
    }
}
PKV_DEV uint4 pack8(const float *x) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

// The 8 pairs of two vectors: (a[i], b[i]) in the half layout; in the interleaved one four in a and four in b.
template <bool INTER>
PKV_DEV void rotate16(float *a, float *b, const Turn &t) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float &x1 = INTER ? (i < 4 ? a[2 * i] : b[2 * i - 8]) : a[i];
        float &x2 = INTER ? (i < 4 ? a[2 * i + 1] : b[2 * i - 7]) : b[i];
        const float y1 = fmaf(x1, t.c[i], -x2 * t.s[i]), y2 = fmaf(x2, t.c[i], x1 * t.s[i]);
        x1 = y1;
        x2 = y2;
    }
}

struct RopeParams {
    const uint64_t *phases;
    float magnitude;
    int32_t rot_units, units;  // units of a head: rotated, in all
    int32_t last_vecs;         // vectors of the last unit (1 where dim - rot is an odd number of vectors)
    int32_t half;              // rot / 2
    int32_t lane_shift;        // lanes a head: 1 << lane_shift >= units
    int32_t rot;
    const uint16_t *q;
    uint16_t *q_out;
    int64_t q_tok, q_head, o_tok, o_head;  // strides in elements
    int32_t hq, hkv, d;
    const uint16_t *k, *v;
    int64_t k_tok, v_tok;
    uint8_t *k_pool, *v_pool;
    int64_t slot_bytes, num_slots;
    float k_scale, v_scale;
    const int32_t *positions, *loc;
    int64_t n;
    int32_t head_shift;        // heads a warp takes at a time: 1 << head_shift; tokens: what lanes are left
    int32_t parts;             // warps a token
    int32_t *err;
};

// (Written to be the first to leave L2, as they are read once: 65,536 tokens into an e4m3 pool 234 us, else 244.)
// What did not turn keeps its bits, a NaN's payload too: its upper halves are what was read.
PKV_DEV void store8(uint16_t *dst, const float *x, bool turned) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = turned ? pack_bf16x2(x[2 * i], x[2 * i + 1]) : __byte_perm(__float_as_uint(x[2 * i]), __float_as_uint(x[2 * i + 1]), 0x7632);
    __stcs(reinterpret_cast<uint4 *>(dst), make_uint4(w[0], w[1], w[2], w[3]));
}
PKV_DEV void store8_e4m3(uint8_t *dst, const float *x, float scale) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        w[i] = (uint32_t)f32x2_to_e4m3x2(__fdiv_rn(x[4 * i], scale), __fdiv_rn(x[4 * i + 1], scale)) |
               (uint32_t)f32x2_to_e4m3x2(__fdiv_rn(x[4 * i + 2], scale), __fdiv_rn(x[4 * i + 3], scale)) << 16;
    __stcs(reinterpret_cast<uint2 *>(dst), make_uint2(w[0], w[1]));
}

// STORE 0: rotate q only; 1, 2: k and v into a bf16 or an e4m3 pool too.
// Three CTAs an SM leave 80 registers, of which each form spills 20 to 120 bytes; with two and no spills 65,536 tokens take
// 257 us into an e4m3 pool, not 234, 236 into a bf16 one, not 240, and rope of 262,144 tokens of one head 24, not 21.
template <bool INTER, int STORE>
__global__ void __launch_bounds__(256, 3) rope_kernel(const RopeParams p) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, per = 1 << p.head_shift, tokens = 32 >> (p.lane_shift + p.head_shift);
    const int u = lane & ((1 << p.lane_shift) - 1), h0 = (lane >> p.lane_shift) & (per - 1), sub = lane >> (p.lane_shift + p.head_shift);
    const bool on = u < p.units, turned = u < p.rot_units;
    // Offsets of the unit's two vectors in its head: neighbouring lanes have neighbouring vectors, the rotated part's
    // first half and its second, then the rest's.  (Two neighbours a lane: 65,536 tokens into an e4m3 pool 288 us, not 256.)
    const int off_a = turned ? 8 * u : p.rot + 8 * (u - p.rot_units);
    const int off_b = off_a + (turned ? p.half : 8 * (p.units - p.rot_units));
    const int pair_a = INTER ? 4 * u : 8 * u, pair_b = INTER ? 4 * (u + p.rot_units) : 8 * u + 4;
    const bool two = u != p.units - 1 || p.last_vecs == 2;
    const int heads = p.hq + (STORE ? 2 * p.hkv : 0);
    // The warps go through the tokens once; where a token has several, each has only its part of that one.  A
    // token's slot and position are loaded while the one before is worked on.
    const uint32_t w = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int part = (int)(w % p.parts);
    const int64_t step = (int64_t)((gridDim.x * blockDim.x) >> 5) * tokens;
    int32_t next_slot = 0, next_pos = 0;
    auto look = [&](int64_t tok) {
        if (tok >= p.n) return;
        next_pos = ld(p.positions + tok);
        if constexpr (STORE != 0) next_slot = ld(p.loc + tok);
    };
    int64_t tok = (int64_t)(w / p.parts) * tokens + sub;
    look(tok);
    for (; tok < p.n; tok += step) {
        const int32_t slot = next_slot, pos = next_pos;
        look(tok + step);
        if (!on) continue;
        bool stored = true;
        if constexpr (STORE != 0) {
            if (slot == -1) continue;  // a padded token
            stored = slot >= 0 && slot < p.num_slots;
            if (!stored && part == 0 && u == 0 && h0 == 0) set_error(p.err, DERR_SLOT_RANGE);
        }
        Turn t;
        bool have = false;
        constexpr int kInFlight = 4;
        for (int h = part * per + h0; h < heads; h += kInFlight * per * p.parts) {
            uint4 a[kInFlight], b[kInFlight];
#pragma unroll
            for (int i = 0; i < kInFlight; ++i) {
                const int hd = h + i * per * p.parts;
                a[i] = b[i] = make_uint4(0u, 0u, 0u, 0u);
                if (hd >= heads || (STORE && hd >= p.hq && !stored)) continue;
                const uint16_t *src;
                if (!STORE || hd < p.hq) src = p.q + tok * p.q_tok + hd * p.q_head;
                else if (hd < p.hq + p.hkv) src = p.k + tok * p.k_tok + (hd - p.hq) * p.d;
                else src = p.v + tok * p.v_tok + (hd - p.hq - p.hkv) * p.d;
                a[i] = __ldcs(reinterpret_cast<const uint4 *>(src + off_a));
                if (two) b[i] = __ldcs(reinterpret_cast<const uint4 *>(src + off_b));
            }
            if (!have) {  // behind the first loads
                if (turned) t = turn_of(p.phases, pair_a, pair_b, pos, p.magnitude);
                have = true;
            }
#pragma unroll
            for (int i = 0; i < kInFlight; ++i) {
                const int hd = h + i * per * p.parts;
                if (hd >= heads) continue;
                const bool is_q = !STORE || hd < p.hq, is_v = STORE && hd >= p.hq + p.hkv;
                if (!is_q && !stored) continue;
                float x[8], y[8];
                unpack8(a[i], x);
                unpack8(b[i], y);
                if (turned && !is_v) rotate16<INTER>(x, y, t);
                if (is_q) {
                    uint16_t *dst = p.q_out + tok * p.o_tok + hd * p.o_head;
                    store8(dst + off_a, x, turned);
                    if (two) store8(dst + off_b, y, turned);
                } else if constexpr (STORE != 0) {
                    const int g = is_v ? hd - p.hq - p.hkv : hd - p.hq;
                    uint8_t *dst = (is_v ? p.v_pool : p.k_pool) + (int64_t)slot * p.slot_bytes;
                    if constexpr (STORE == 1) {
                        uint16_t *row = reinterpret_cast<uint16_t *>(dst) + g * p.d;
                        store8(row + off_a, x, turned && !is_v);
                        if (two) store8(row + off_b, y, turned && !is_v);
                    } else {
                        const float scale = is_v ? p.v_scale : p.k_scale;
                        store8_e4m3(dst + g * p.d + off_a, x, scale);
                        if (two) store8_e4m3(dst + g * p.d + off_b, y, scale);
                    }
                }
            }
        }
    }
}

// Rows of padded tokens, heads of d elements, to zeros: a lane looks at a token's slot, a warp writes a row.
__global__ void __launch_bounds__(256) zero_padded_kernel(uint16_t *out, int64_t tok_stride, int64_t head_stride, int32_t heads,
                                                          int32_t vecs, const int32_t *loc, int64_t n) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t first = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) & ~(int64_t)31; first < n; first += step) {
        uint32_t padded = __ballot_sync(0xffffffffu, first + lane < n && ld(loc + first + lane) == -1);
        for (; padded; padded &= padded - 1) {
            uint16_t *row = out + (first + __ffs(padded) - 1) * tok_stride;
            for (int v = lane; v < heads * vecs; v += 32)
                *reinterpret_cast<uint4 *>(row + v / vecs * head_stride + v % vecs * 8) = make_uint4(0u, 0u, 0u, 0u);
        }
    }
}

static int check_spec(const pkv_rope_spec *r) {
    if (!r || !r->phases || reinterpret_cast<uintptr_t>(r->phases) & 7) return PKV_E_INVALID;
    if (r->rotary_dim <= 0 || r->rotary_dim % 16) return PKV_E_UNSUPPORTED;
    if (r->interleaved != 0 && r->interleaved != 1) return PKV_E_INVALID;
    if (!std::isfinite(r->magnitude)) return PKV_E_INVALID;
    return PKV_OK;
}

// Rows of bf16 heads: 16-byte vectors, strides that keep them so.
static bool rows_ok(const void *x, int64_t tok, int64_t head) {
    return x && !(reinterpret_cast<uintptr_t>(x) & 15) && tok % 8 == 0 && head % 8 == 0;
}
// The same to write to: no two heads or tokens in one place.
static bool out_ok(const void *x, int64_t tok, int64_t head, int64_t n, int32_t heads) {
    return rows_ok(x, tok, head) && (tok != 0 || n == 1) && (head != 0 || heads == 1);
}

static int launch_rope(RopeParams p, const pkv_rope_spec *r, int store, cudaStream_t s) {
    p.phases = r->phases;
    p.magnitude = r->magnitude;
    p.rot = r->rotary_dim;
    p.half = r->rotary_dim / 2;
    p.rot_units = r->rotary_dim / 16;
    const int rest = (p.d - p.rot) / 8;  // vectors behind the rotated part
    p.units = p.rot_units + (rest + 1) / 2;
    p.last_vecs = rest & 1 ? 1 : 2;
    p.lane_shift = 0;
    while ((1 << p.lane_shift) < p.units) ++p.lane_shift;
    // Heads side by side in a warp, as many as there are; where that leaves lanes, several tokens (262,144 tokens of one
    // head of 64: 152 us by a token a warp, 22 by eight).
    const int heads = p.hq + (store ? 2 * p.hkv : 0);
    p.head_shift = 0;
    while ((1 << p.head_shift) < heads && p.head_shift < 5 - p.lane_shift) ++p.head_shift;
    const int per = 1 << p.head_shift, tokens = 32 >> (p.lane_shift + p.head_shift);
    // Warps a token: all of a token's heads in one warp's steps of four once that fills the GPU
    // (16 warps an SM), else as many as its heads give work, for then the time is a chain of loads.
    // 256 tokens of 128 heads: 5.3 us by 9 warps a token, 8.9 by one.
    const int64_t steps = (heads + per - 1) / per, full = (int64_t)num_sms() * 16;
    p.parts = (int32_t)std::min<int64_t>(steps, std::max<int64_t>(1, full / p.n));
    const int64_t warps = (p.n + tokens - 1) / tokens * p.parts;
    const int64_t blocks = std::min<int64_t>((warps + 7) / 8, (int64_t)num_sms() * 32);
    auto kern = r->interleaved ? (store == 0 ? rope_kernel<true, 0> : store == 1 ? rope_kernel<true, 1> : rope_kernel<true, 2>)
                               : (store == 0 ? rope_kernel<false, 0> : store == 1 ? rope_kernel<false, 1> : rope_kernel<false, 2>);
    return launch_pdl(kern, dim3((unsigned)blocks), dim3(256), 0, s, true, p) == cudaSuccess ? PKV_OK : PKV_E_CUDA;
}

// ------------------------------------------------------------------------------------------
// latent_store

struct LatentStoreParams {
    const uint16_t *c, *pe, *w;
    int64_t c_tok, pe_tok;
    float eps;
    const uint64_t *phases;
    float magnitude;
    uint16_t *rows;
    int64_t stride, num_slots;
    const int32_t *positions, *loc;
    int64_t n;
    int32_t *err;
};

// A warp T tokens at a time, two by two: R / 256 vectors of a latent a lane, the sums of squares over the warp.  The
// T tokens' rotary keys, four units each, go to four lanes a token: with T = 8 to all lanes at once, where with two the sines
// and cosines of 8 lanes took half of the kernel's instructions (131,072 tokens 60 us, with 8 56, and 53 with loads past L1).  A
// token's loads are issued before its slot is known.
template <int R, bool INTER, int T>
__global__ void __launch_bounds__(256) latent_store_kernel(const LatentStoreParams p) {
    constexpr int V = R / 256;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, u = lane & 3, mine = lane >> 2;  // (with T = 2, lanes 8 and up have no unit)
    const int off_a = 8 * u, off_b = off_a + kLatentRope / 2;
    uint4 w[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (p.w) w[i] = ld(reinterpret_cast<const uint4 *>(p.w) + 32 * i + lane);
    const int64_t warps = ((int64_t)gridDim.x * blockDim.x) >> 5;
    for (int64_t first = (((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5) * T; first < p.n; first += T * warps) {
        const bool turns = mine < T && first + mine < p.n;
        uint4 a, b;
        int32_t own_slot = -1, pos = 0;
        if (turns) {
            own_slot = ld(p.loc + first + mine);
            pos = ld(p.positions + first + mine);
            a = __ldcg(reinterpret_cast<const uint4 *>(p.pe + (first + mine) * p.pe_tok + off_a));
            b = __ldcg(reinterpret_cast<const uint4 *>(p.pe + (first + mine) * p.pe_tok + off_b));
        }
#pragma unroll 1
        for (int pair = 0; pair < T; pair += 2) {
            const int64_t tok = first + pair;
            if (tok >= p.n) break;
            uint4 x[2][V];
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (tok + k < p.n) x[k][i] = __ldcg(reinterpret_cast<const uint4 *>(p.c + (tok + k) * p.c_tok) + 32 * i + lane);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int32_t slot = __shfl_sync(0xffffffffu, own_slot, 4 * (pair + k));
                if (slot < 0 || slot >= p.num_slots) {
                    if (slot != -1 && lane == 0) set_error(p.err, DERR_SLOT_RANGE);
                    continue;  // padding (or past the end), or not there
                }
                if (p.w) {
                    float y[8 * V], z[8], sum = 0.f;
#pragma unroll
                    for (int i = 0; i < V; ++i) unpack8(x[k][i], y + 8 * i);
#pragma unroll
                    for (int i = 0; i < 8 * V; ++i) sum = fmaf(y[i], y[i], sum);
#pragma unroll
                    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                    const float inv = rsqrtf(sum * (1.f / R) + p.eps);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        unpack8(w[i], z);
#pragma unroll
                        for (int j = 0; j < 8; ++j) z[j] *= y[8 * i + j] * inv;
                        x[k][i] = pack8(z);
                    }
                }
                uint4 *row = reinterpret_cast<uint4 *>(p.rows + (int64_t)slot * p.stride);
#pragma unroll
                for (int i = 0; i < V; ++i) row[32 * i + lane] = x[k][i];
            }
        }
        if (own_slot >= 0 && own_slot < p.num_slots) {
            const Turn t = turn_of(p.phases, INTER ? 4 * u : 8 * u, INTER ? 4 * (u + 4) : 8 * u + 4, pos, p.magnitude);
            float ya[8], yb[8];
            unpack8(a, ya);
            unpack8(b, yb);
            rotate16<INTER>(ya, yb, t);
            uint16_t *row = p.rows + (int64_t)own_slot * p.stride + R;
            store8(row + off_a, ya, true);
            store8(row + off_b, yb, true);
        }
    }
}

}  // namespace pkv

extern "C" int pkv_rope_phases(const double *inv_freq, int32_t n, uint64_t *phases) {
    if (!inv_freq || !phases || n < 0) return PKV_E_INVALID;
    for (int32_t i = 0; i < n; ++i)
        if (!std::isfinite(inv_freq[i])) return PKV_E_INVALID;
    for (int32_t i = 0; i < n; ++i) {
        double t = std::fabs(inv_freq[i]) / 6.283185307179586476925;  // turns a position
        t -= std::floor(t);  // whole ones do not show (exact; of a negative t it would round to the bits of 1 - |t|)
        const uint64_t turns = (uint64_t)std::rint(std::ldexp(t, 64));
        phases[i] = inv_freq[i] < 0 ? 0 - turns : turns;
    }
    return PKV_OK;
}

extern "C" int pkv_rope(const pkv_rope_spec *rope, const void *x, int64_t x_token_stride, int64_t x_head_stride, void *out,
                        int64_t out_token_stride, int64_t out_head_stride, int32_t num_heads, int32_t dim,
                        const int32_t *positions, int64_t n, void *stream) {
    using namespace pkv;
    const int rc = check_spec(rope);
    if (rc) return rc;
    if (n < 0 || num_heads < 0) return PKV_E_INVALID;
    if (dim < rope->rotary_dim) return PKV_E_INVALID;
    if (dim % 8 || dim > 512 || n >= ((int64_t)1 << 40) || num_heads > 65536) return PKV_E_UNSUPPORTED;
    if (n == 0 || num_heads == 0) return PKV_OK;
    if (!rows_ok(x, x_token_stride, x_head_stride) || !out_ok(out, out_token_stride, out_head_stride, n, num_heads) || !positions)
        return PKV_E_INVALID;
    RopeParams p{};
    p.q = static_cast<const uint16_t *>(x);
    p.q_tok = x_token_stride;
    p.q_head = x_head_stride;
    p.q_out = static_cast<uint16_t *>(out);
    p.o_tok = out_token_stride;
    p.o_head = out_head_stride;
    p.hq = num_heads;
    p.d = dim;
    p.positions = positions;
    p.n = n;
    return launch_rope(p, rope, 0, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int pkv_rope_store(const pkv_pool *pool, const pkv_rope_spec *rope, const void *q, int64_t q_token_stride,
                              int64_t q_head_stride, void *q_out, int64_t q_out_token_stride, int64_t q_out_head_stride,
                              int32_t num_q_heads, const void *k_new, int64_t k_token_stride, const void *v_new,
                              int64_t v_token_stride, const int32_t *positions, const int32_t *out_cache_loc, int64_t n,
                              void *workspace, void *stream) {
    using namespace pkv;
    int rc = validate_pool(pool);
    if (!rc) rc = check_spec(rope);
    if (rc) return rc;
    if (n < 0 || num_q_heads < 0) return PKV_E_INVALID;
    if (pool->head_dim < rope->rotary_dim) return PKV_E_INVALID;
    if (n >= ((int64_t)1 << 40) || num_q_heads > 65536 || pool->num_kv_heads > 65536) return PKV_E_UNSUPPORTED;
    if (n == 0) return PKV_OK;
    if (num_q_heads > 0 && (!rows_ok(q, q_token_stride, q_head_stride) || !out_ok(q_out, q_out_token_stride, q_out_head_stride, n, num_q_heads)))
        return PKV_E_INVALID;
    if (!rows_ok(k_new, k_token_stride, 0) || !rows_ok(v_new, v_token_stride, 0) || !positions || !out_cache_loc)
        return PKV_E_INVALID;
    if (reinterpret_cast<uintptr_t>(workspace) & 3) return PKV_E_INVALID;
    RopeParams p{};
    p.q = static_cast<const uint16_t *>(q);
    p.q_tok = q_token_stride;
    p.q_head = q_head_stride;
    p.q_out = static_cast<uint16_t *>(q_out);
    p.o_tok = q_out_token_stride;
    p.o_head = q_out_head_stride;
    p.hq = num_q_heads;
    p.hkv = pool->num_kv_heads;
    p.d = pool->head_dim;
    p.k = static_cast<const uint16_t *>(k_new);
    p.v = static_cast<const uint16_t *>(v_new);
    p.k_tok = k_token_stride;
    p.v_tok = v_token_stride;
    p.k_pool = static_cast<uint8_t *>(pool->k);
    p.v_pool = static_cast<uint8_t *>(pool->v);
    p.slot_bytes = slot_bytes(pool);
    p.num_slots = pool->num_slots;
    p.k_scale = pool->k_scale;
    p.v_scale = pool->v_scale;
    p.positions = positions;
    p.loc = out_cache_loc;
    p.n = n;
    p.err = static_cast<int32_t *>(workspace);
    return launch_rope(p, rope, pool->dtype == PKV_BF16 ? 1 : 2, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int pkv_zero_padded(void *out, int64_t token_stride, int64_t head_stride, int32_t num_heads, int32_t dim,
                               const int32_t *out_cache_loc, int64_t n, void *stream) {
    using namespace pkv;
    if (n < 0 || num_heads < 0 || dim <= 0) return PKV_E_INVALID;
    if (dim % 8 || dim > 512 || n >= ((int64_t)1 << 40) || num_heads > 65536) return PKV_E_UNSUPPORTED;
    if (n == 0 || num_heads == 0) return PKV_OK;
    if (!out_ok(out, token_stride, head_stride, n, num_heads) || !out_cache_loc) return PKV_E_INVALID;
    const int64_t blocks = std::min<int64_t>((n + 255) / 256, (int64_t)num_sms() * 8);
    return launch_pdl(zero_padded_kernel, dim3((unsigned)blocks), dim3(256), 0, reinterpret_cast<cudaStream_t>(stream), true,
                      static_cast<uint16_t *>(out), token_stride, head_stride, num_heads, dim / 8, out_cache_loc, n) == cudaSuccess
               ? PKV_OK
               : PKV_E_CUDA;
}

extern "C" int pkv_latent_store(const pkv_latent_pool *pool, const pkv_rope_spec *rope, const void *c_new, int64_t c_token_stride,
                                const void *pe_new, int64_t pe_token_stride, const void *norm_weight, float eps,
                                const int32_t *positions, const int32_t *out_cache_loc, int64_t n, void *workspace, void *stream) {
    using namespace pkv;
    int rc = validate_latent_pool(pool);
    if (!rc) rc = check_spec(rope);
    if (rc) return rc;
    if (rope->rotary_dim != pool->rope_dim) return PKV_E_INVALID;
    if (n < 0) return PKV_E_INVALID;
    if (n >= ((int64_t)1 << 40)) return PKV_E_UNSUPPORTED;
    if (n == 0) return PKV_OK;
    if (!rows_ok(c_new, c_token_stride, 0) || !rows_ok(pe_new, pe_token_stride, 0) || !positions || !out_cache_loc)
        return PKV_E_INVALID;
    if (reinterpret_cast<uintptr_t>(workspace) & 3) return PKV_E_INVALID;
    if (norm_weight && ((reinterpret_cast<uintptr_t>(norm_weight) & 15) || !(eps >= 0.f) || !std::isfinite(eps))) return PKV_E_INVALID;
    LatentStoreParams p{};
    p.c = static_cast<const uint16_t *>(c_new);
    p.pe = static_cast<const uint16_t *>(pe_new);
    p.w = static_cast<const uint16_t *>(norm_weight);
    p.c_tok = c_token_stride;
    p.pe_tok = pe_token_stride;
    p.eps = eps;
    p.phases = rope->phases;
    p.magnitude = rope->magnitude;
    p.rows = static_cast<uint16_t *>(pool->rows);
    p.stride = latent_stride(pool);
    p.num_slots = pool->num_slots;
    p.positions = positions;
    p.loc = out_cache_loc;
    p.n = n;
    p.err = static_cast<int32_t *>(workspace);
    // Eight tokens a warp once that leaves every SM 16 warps (256 tokens: 5.1 us with two, 8.4 with eight).
    const bool many = n >= (int64_t)num_sms() * 16 * 8;
    const int64_t per_block = 8 * (many ? 8 : 2), blocks = std::min<int64_t>((n + per_block - 1) / per_block, (int64_t)num_sms() * 12);
    void (*kern)(const LatentStoreParams);
    if (pool->latent_dim == 512)
        kern = rope->interleaved ? (many ? latent_store_kernel<512, true, 8> : latent_store_kernel<512, true, 2>)
                                 : (many ? latent_store_kernel<512, false, 8> : latent_store_kernel<512, false, 2>);
    else
        kern = rope->interleaved ? (many ? latent_store_kernel<256, true, 8> : latent_store_kernel<256, true, 2>)
                                 : (many ? latent_store_kernel<256, false, 8> : latent_store_kernel<256, false, 2>);
    return launch_pdl(kern, dim3((unsigned)blocks), dim3(256), 0, reinterpret_cast<cudaStream_t>(stream), true, p) == cudaSuccess
               ? PKV_OK
               : PKV_E_CUDA;
}
