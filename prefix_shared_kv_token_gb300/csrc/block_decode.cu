// attn_decode_block: one query token per request over its whole context in a block-scaled 8-bit
// pool (block.cuh), read through a page table, with lengths that only the device knows.
//
// What is computed: for request r of length L and query head h of KV head g = h / G,
//     o[r, h] = sum_{j < L} softmax_j(sm_scale * q[r, h] . K_j) V_j,
//     K_j = 2^(ek - 127) * code,  V_j = 2^(ev - 127) * code  (exponent bytes of j's page and g).
// With s_j the logits in log2 units, R = max_j (s_j + ev_j) and w_j = 2^(s_j + ev_j - R), the sum
// is  sum w_j code_j / sum 2^(s_j - R):  V's exponents move into the weights, so the codes enter
// the product as they are, and a weight is at most 1 however far the pages' exponents differ.  The
// sum below is kept as l = sum 2^(s_j - R + ea), ea = ev of the key that set R, so that it too is of
// size 1 whatever the pages' exponents; the result is acc / l * 2^ea.
//
// Design.  The work is a stream of codes, so what counts is bytes in flight:
//   * 16-key tiles of all requests, laid end to end, are cut into equal contiguous ranges, one
//     per warp and KV head (each CTA scans the lengths itself: no host plan, no set-up kernel,
//     ragged batches balance to a tile, and a captured graph follows the lengths).  A request
//     inside one range is written directly; one that crosses ranges leaves a record (R, l, acc)
//     in each, joined by a second kernel.
//   * A warp loads its codes straight into registers in fragment order: K rows are the A operand
//     (16 keys) of S^T = K Q^T, V^T the A operand of O^T = V^T P^T, and the query heads are the 8
//     columns of B.  So a group of up to 8 heads shares one MMA, the accumulators are d x 8, no
//     shared memory is used and 16 warps an SM keep 64 KB in flight.
//   * mma.sync m16n8k16 in f16: an e4m3 code is an f16 value, and so is a query element over a
//     power of two that brings its row's largest to [2^14, 2^15) (elements below 2^-31 of it
//     round, far under the fp32 sum's own rounding).  Weights are f16 times 2^15: 11 bits down to
//     2^-29 of the largest, against bf16's 8.

#include <algorithm>

#include "block.cuh"

namespace pkv {

constexpr int kTile = 16;         // keys
constexpr int kMinTiles = 4;      // per range, while there are few
constexpr int kWarps = 8;
constexpr float kBias = 15.f;     // weights carry 2^15
constexpr float kUnbias = 1.f / (1 << 15);
constexpr float kLog2eB = 1.4426950408889634f;

struct BlockDecodeParams {
    const uint8_t *k, *v, *k_exp, *v_exp;
    int64_t num_pages, slot_bytes;
    int32_t shift, hkv, hg, groups;  // hg KV heads read side by side, `groups` times
    const int32_t *table;
    int64_t stride;
    int32_t num_rows, batch;
    const int32_t *rows, *lens;
    const uint16_t *q;
    uint16_t *o;
    float scale_log2;
    int32_t ranges;  // at most
    float *rec;      // [range][2][hg][G][D], then (R, l, ea, -) [range][2][hg][G][4]
    float *rec_ml;
    int32_t *err;
};

// A request's length as the kernels use it: 0 where its row or length is out of range.
PKV_DEV int32_t checked_len(const BlockDecodeParams &p, int r, bool report) {
    const int32_t len = __ldg(p.lens + r), row = __ldg(p.rows + r);
    if (len == 0) return 0;
    if (len < 0 || row < 0 || row >= p.num_rows || (int64_t)len > (p.stride << p.shift)) {
        if (report) set_error(p.err, DERR_POSITION);
        return 0;
    }
    return len;
}
PKV_DEV int32_t tiles_of(int32_t len) { return (int32_t)(((int64_t)len + kTile - 1) / kTile); }

// The cut of `total` tiles into n ranges whose sizes differ by at most one.
struct Cut {
    int64_t size, extra;
    int32_t n;
    PKV_DEV Cut(int64_t total, int32_t most) {
        n = (int32_t)min((int64_t)most, max((int64_t)1, total / kMinTiles));
        size = total / n;
        extra = total - size * n;
    }
    PKV_DEV int64_t start(int32_t i) const { return size * i + min((int64_t)i, extra); }
    PKV_DEV int32_t range_of(int64_t t) const {
        const int64_t big = extra * (size + 1);
        return (int32_t)(t < big ? t / (size + 1) : extra + (t - big) / size);
    }
};

PKV_DEV void mma_f16_16816(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
PKV_DEV uint32_t transpose_8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
PKV_DEV uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
    return r;
}
PKV_DEV int64_t block_sum(int64_t x, int64_t *warp_sums) {  // kWarps warps; every thread gets it
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    if ((threadIdx.x & 31) == 0) warp_sums[threadIdx.x >> 5] = x;
    __syncthreads();
    x = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) x += warp_sums[w];
    return x;
}

// Query rows of the group as B fragments, in the d order that K's 16-byte pieces have: k-step
// (half, j) holds d = 64 half + 16 c + 4 j + {0, 1 | 2, 3} of head g.  Returns the power of two
// taken out of head g's row.
template <int D, int G>
PKV_DEV int load_query(const BlockDecodeParams &p, int r, int kv_head, uint32_t (&qb)[D / 16][2]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    uint32_t w[D / 8];
    const uint16_t *row = p.q + ((int64_t)r * p.hkv * G + kv_head * G + (g < G ? g : 0)) * D + 16 * c;
    uint32_t amax = 0;
#pragma unroll
    for (int h = 0; h < D / 64; ++h)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint4 x = __ldg(reinterpret_cast<const uint4 *>(row + 64 * h) + u);
            w[8 * h + 4 * u] = x.x;
            w[8 * h + 4 * u + 1] = x.y;
            w[8 * h + 4 * u + 2] = x.z;
            w[8 * h + 4 * u + 3] = x.w;
        }
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
        if (g >= G) w[i] = 0u;
        const uint32_t a = w[i] & 0x7FFFu, b = (w[i] >> 16) & 0x7FFFu;
        if (a < 0x7F80u) amax = max(amax, a);
        if (b < 0x7F80u) amax = max(amax, b);
    }
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const int e = amax == 0 ? 0 : (int)(amax >> 7) - 127 - 14;  // largest element to [2^14, 2^15)
    // 2^-e in two steps: -e alone may leave fp32's exponents
    const float f0 = exp_value(127 - e / 2), f1 = exp_value(127 - (e - e / 2));
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint32_t x = w[2 * ks + u];
            qb[ks][u] = pack_f16x2(bf16_lo(x) * f0 * f1, bf16_hi(x) * f0 * f1);
        }
    return e;
}

// One tile's codes: K rows g and g + 8, V rows 2c, 2c + 1, 2c + 8, 2c + 9.
template <int D>
struct TileRegs {
    uint4 k[2][D / 64];
    uint32_t v[4][D / 32];
    int ek, ev;
};

template <int D>
PKV_DEV void load_k(const BlockDecodeParams &p, TileRegs<D> &x, int64_t slot, bool ok, int head) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint8_t *row = p.k + (slot + g + 8 * h) * p.slot_bytes + (int64_t)head * D + 16 * c;
#pragma unroll
        for (int u = 0; u < D / 64; ++u)
            x.k[h][u] = ok ? __ldg(reinterpret_cast<const uint4 *>(row + 64 * u)) : make_uint4(0u, 0u, 0u, 0u);
    }
    x.ek = ok ? clamp_exp(__ldg(p.k_exp + (slot >> p.shift) * p.hkv + head)) : 127;
}

// Rows at or past `valid` read as zeros: a weight of 0 does not undo a NaN or an infinity.
template <int D>
PKV_DEV void load_v(const BlockDecodeParams &p, TileRegs<D> &x, int64_t slot, bool ok, int head, int valid) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int key = 2 * c + (i & 1) + 8 * (i >> 1);
        const uint8_t *at = p.v + (slot + key) * p.slot_bytes + (int64_t)head * D + g * (D / 8);
        const bool on = ok && key < valid;
        if constexpr (D == 128) {
            const uint4 y = on ? __ldg(reinterpret_cast<const uint4 *>(at)) : make_uint4(0u, 0u, 0u, 0u);
            x.v[i][0] = y.x;
            x.v[i][1] = y.y;
            x.v[i][2] = y.z;
            x.v[i][3] = y.w;
        } else {
            const uint2 y = on ? __ldg(reinterpret_cast<const uint2 *>(at)) : make_uint2(0u, 0u);
            x.v[i][0] = y.x;
            x.v[i][1] = y.y;
        }
    }
    x.ev = ok ? clamp_exp(__ldg(p.v_exp + (slot >> p.shift) * p.hkv + head)) : 127;
}

// Running state of one warp: columns 2c and 2c + 1 (query heads) of this lane.
template <int D>
struct DecodeState {
    float acc[D / 16][4];  // MMA i: d = (D/8) g + 2i + {0, 0, 1, 1}, heads 2c + {0, 1, 0, 1}
    float m[2], l[2], ea[2];
};

// The result of a row from its sums.
PKV_DEV float row_scale(float l, float ea) { return l == 0.f ? 0.f : kUnbias / l * exp_value((int)ea + 127); }

template <int D>
PKV_DEV void attend_tile(DecodeState<D> &st, const uint32_t (&qb)[D / 16][2], const TileRegs<D> &x, const float (&cs)[2],
                         int valid) {
    const int lane = threadIdx.x & 31, g = lane >> 2;
    float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};  // two chains of MMAs
#pragma unroll
    for (int u = 0; u < D / 64; ++u) {
        const uint32_t a[4] = {x.k[0][u].x, x.k[0][u].y, x.k[0][u].z, x.k[0][u].w};
        const uint32_t b[4] = {x.k[1][u].x, x.k[1][u].y, x.k[1][u].z, x.k[1][u].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            mma_f16_16816(s[j & 1], e4m3x2_to_f16x2(a[j]), e4m3x2_to_f16x2(b[j]), e4m3x2_hi_to_f16x2(a[j]),
                          e4m3x2_hi_to_f16x2(b[j]), qb[4 * u + j][0], qb[4 * u + j][1]);
    }
    const float kf = exp_value(x.ek), ev = (float)(x.ev - 127);
    float t[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        t[e] = (s[0][e] + s[1][e]) * (cs[e & 1] * kf) + ev;
        if (g + 8 * (e >> 1) >= valid) t[e] = -INFINITY;
    }
    float mn[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float y = fmaxf(t[h], t[2 + h]);
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, d));
        mn[h] = fmaxf(st.m[h], y);
    }
    if (__any_sync(0xffffffffu, mn[0] > st.m[0] || mn[1] > st.m[1])) {
        float al[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            al[h] = 1.f;
            if (mn[h] > st.m[h]) {
                al[h] = ex2(st.m[h] - mn[h]);
                st.l[h] *= ex2(st.m[h] - mn[h] + (ev - st.ea[h]));
                st.m[h] = mn[h];
                st.ea[h] = ev;
            }
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) st.acc[i][e] *= al[e & 1];
    }
    float w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float rel = t[e] - (mn[e & 1] == -INFINITY ? 0.f : mn[e & 1]);
        w[e] = ex2(rel + kBias);
        st.l[e & 1] += ex2(rel - (ev - st.ea[e & 1]));
    }
    const uint32_t b0 = transpose_8x8(pack_f16x2(w[0], w[1])), b1 = transpose_8x8(pack_f16x2(w[2], w[3]));
#pragma unroll
    for (int j = 0; j < D / 32; ++j)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            // bytes (key, key + 1) of d and d + 1 next to each other
            const uint32_t lo = __byte_perm(x.v[0][j], x.v[1][j], u ? 0x7362 : 0x5140);
            const uint32_t hi = __byte_perm(x.v[2][j], x.v[3][j], u ? 0x7362 : 0x5140);
            mma_f16_16816(st.acc[2 * j + u], e4m3x2_to_f16x2(lo), e4m3x2_hi_to_f16x2(lo), e4m3x2_to_f16x2(hi),
                          e4m3x2_hi_to_f16x2(hi), b0, b1);
        }
}

template <int D, int G>
PKV_DEV void write_segment(const BlockDecodeParams &p, DecodeState<D> &st, int r, int kv_head, int32_t rec, int hl) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) st.l[h] += __shfl_xor_sync(0xffffffffu, st.l[h], d);
        const int head = 2 * c + h;
        if (head >= G) continue;
        if (rec < 0) {
            const float inv = row_scale(st.l[h], st.ea[h]);
            uint32_t *dst = reinterpret_cast<uint32_t *>(p.o + ((int64_t)r * p.hkv * G + kv_head * G + head) * D + g * (D / 8));
#pragma unroll
            for (int i = 0; i < D / 16; ++i) dst[i] = pack_bf16x2(st.acc[i][h] * inv, st.acc[i][2 + h] * inv);
        } else {
            const int64_t at = ((int64_t)rec * p.hg + hl) * G + head;
            float2 *dst = reinterpret_cast<float2 *>(p.rec + at * D + g * (D / 8));
#pragma unroll
            for (int i = 0; i < D / 16; ++i) dst[i] = make_float2(st.acc[i][h], st.acc[i][2 + h]);
            if (g == 0) *reinterpret_cast<float4 *>(p.rec_ml + at * 4) = make_float4(st.m[h], st.l[h], st.ea[h], 0.f);
        }
    }
}

template <int D, int G>
__global__ void __launch_bounds__(32 * kWarps, 2) block_decode_kernel(const BlockDecodeParams p) {
    __shared__ int64_t warp_sums[kWarps];
    __shared__ int64_t base[32 * kWarps + 1];  // tiles before each thread's chunk of requests
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, warp = tid >> 5;
    const int chunk = (p.batch + 32 * kWarps - 1) / (32 * kWarps);
    int64_t mine = 0;
    for (int r = tid * chunk; r < min((tid + 1) * chunk, p.batch); ++r)
        mine += tiles_of(checked_len(p, r, blockIdx.x == 0));
    int64_t scan = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, scan, d);
        if ((tid & 31) >= d) scan += y;
    }
    if ((tid & 31) == 31) warp_sums[warp] = scan;
    __syncthreads();
    int64_t before = 0, n = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w == warp) before = n;
        n += warp_sums[w];
    }
    base[tid] = before + scan - mine;
    if (tid == 0) base[32 * kWarps] = n;
    __syncthreads();
    if (n == 0) return;

    const Cut cut(n * p.groups, p.ranges);
    const int hl = warp % p.hg;
    const int32_t range = blockIdx.x * (kWarps / p.hg) + warp / p.hg;
    if (range >= cut.n) return;
    int64_t at = cut.start(range);
    const int64_t end = cut.start(range + 1);
    const int64_t begin = at;

    while (at < end) {
        const int grp = (int)(at / n);
        const int head = grp * p.hg + hl;
        const int64_t off = (int64_t)grp * n;
        // the chunk of requests that holds tile at - off, then the request
        int lo = 0, hi = 32 * kWarps;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (base[mid] <= at - off) lo = mid; else hi = mid;
        }
        int r = lo * chunk;
        int64_t first = off + base[lo];  // request r's first tile
        const int64_t stop = min(end, off + n);
        for (; at < stop; ++r) {
            if (r >= p.batch) return;  // the lengths changed under the call
            const int32_t len = checked_len(p, r, false);
            const int32_t tiles = tiles_of(len);
            if (first + tiles <= at) {
                first += tiles;
                continue;
            }
            const int32_t j0 = (int32_t)(at - first), j1 = (int32_t)min((int64_t)tiles, stop - first);
            const int32_t *row = p.table + (int64_t)__ldg(p.rows + r) * p.stride;
            uint32_t qb[D / 16][2];
            const int e = load_query<D, G>(p, r, head, qb);
            // this lane's columns are heads 2c and 2c + 1, whose exponents lanes 8c and 8c + 4 hold
            float cs[2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
                cs[h] = ldexpf(p.scale_log2, __shfl_sync(0xffffffffu, e, 8 * (tid & 3) + 4 * h));
            DecodeState<D> st;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) st.acc[i][0] = st.acc[i][1] = st.acc[i][2] = st.acc[i][3] = 0.f;
            st.m[0] = st.m[1] = -INFINITY;
            st.l[0] = st.l[1] = st.ea[0] = st.ea[1] = 0.f;
            for (int j = j0; j < j1; ++j) {
                const int32_t key = j * kTile;
                const int32_t page = __ldg(row + (key >> p.shift));
                const bool ok = page >= 0 && (int64_t)page < p.num_pages;
                if (!ok && (tid & 31) == 0) set_error(p.err, DERR_SLOT_RANGE);
                const int64_t slot = ((int64_t)(ok ? page : 0) << p.shift) + (key & ((1 << p.shift) - 1));
                TileRegs<D> x;
                load_k<D>(p, x, slot, ok, head);
                load_v<D>(p, x, slot, ok, head, len - key);
                attend_tile<D>(st, qb, x, cs, len - key);
            }
            const bool whole = j0 == 0 && j1 == tiles;
            write_segment<D, G>(p, st, r, head, whole ? -1 : 2 * range + (first < begin ? 0 : 1), hl);
            at = first + j1;
            first += tiles;
        }
    }
}

// Joins the records of the requests that cross ranges and clears the rows of empty ones.  A CTA
// takes one (request, KV head): its warps share each query head's records and combine through
// shared memory.
template <int D, int G>
__global__ void __launch_bounds__(32 * kWarps) block_merge_kernel(const BlockDecodeParams p) {
    __shared__ int64_t warp_sums[kWarps];
    __shared__ float s_acc[kWarps][D];
    __shared__ float4 s_ml[kWarps];
    const int r = blockIdx.x, head = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int32_t tiles = tiles_of(checked_len(p, r, false));
    int64_t mine = 0, all = 0;
    for (int i = tid; i < p.batch; i += 32 * kWarps) {
        const int32_t t = tiles_of(checked_len(p, i, false));
        all += t;
        if (i < r) mine += t;
    }
    const int64_t before = block_sum(mine, warp_sums);
    __syncthreads();
    const int64_t n = block_sum(all, warp_sums);
    pdl_wait();  // the records
    pdl_trigger();
    uint16_t *out = p.o + ((int64_t)r * p.hkv + head) * G * D;
    if (tiles == 0) {
        for (int i = tid; i < G * D / 8; i += 32 * kWarps) reinterpret_cast<uint4 *>(out)[i] = make_uint4(0u, 0u, 0u, 0u);
        return;
    }
    const Cut cut(n * p.groups, p.ranges);
    const int64_t first = (int64_t)(head / p.hg) * n + before;
    const int32_t i0 = cut.range_of(first), i1 = cut.range_of(first + tiles - 1);
    if (i0 == i1) return;
    constexpr int V = D / 32;            // elements a lane holds
    constexpr int kShare = kWarps / G;   // warps of one query head
    const int q = warp / kShare, sub = warp % kShare;
    float M = -INFINITY, L = 0.f, E = 0.f, O[V];
#pragma unroll
    for (int v = 0; v < V; ++v) O[v] = 0.f;
    // folds in a record (or another warp's sums): its acc scaled by the returned factor
    auto join = [&](const float4 &x, const float *a) {
        if (x.x > M) {
            const float f = ex2(M - x.x);
            L *= ex2(M - x.x + (x.z - E));
#pragma unroll
            for (int v = 0; v < V; ++v) O[v] *= f;
            M = x.x;
            E = x.z;
        }
        if (x.x == -INFINITY) return;
        const float w = ex2(x.x - M);
        L += x.y * ex2(x.x - M - (x.z - E));
#pragma unroll
        for (int v = 0; v < V; ++v) O[v] += a[v] * w;
    };
    for (int32_t i = i0 + sub; i <= i1; i += kShare) {
        const int64_t rec = (((int64_t)i * 2 + (first < cut.start(i) ? 0 : 1)) * p.hg + head % p.hg) * G + q;
        float a[V];
#pragma unroll
        for (int v = 0; v < V; ++v) a[v] = p.rec[rec * D + lane * V + v];
        join(*reinterpret_cast<const float4 *>(p.rec_ml + rec * 4), a);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) s_acc[warp][lane * V + v] = O[v];
    if (lane == 0) s_ml[warp] = make_float4(M, L, E, 0.f);
    __syncthreads();
    if (sub != 0) return;
    for (int w = 1; w < kShare; ++w) {
        float a[V];
#pragma unroll
        for (int v = 0; v < V; ++v) a[v] = s_acc[warp + w][lane * V + v];
        join(s_ml[warp + w], a);
    }
    const float inv = row_scale(L, E);
#pragma unroll
    for (int v = 0; v < V; v += 2)
        reinterpret_cast<uint32_t *>(out + q * D + lane * V)[v / 2] = pack_bf16x2(O[v] * inv, O[v + 1] * inv);
}

static int head_group(int32_t hkv) {
    int hg = kWarps;
    while (hkv % hg) hg /= 2;
    return hg;
}
static int decode_ctas() { return 2 * num_sms(); }

static size_t decode_workspace(int32_t hkv, int32_t G, int32_t d) {
    const int hg = head_group(hkv);
    const size_t ranges = (size_t)decode_ctas() * (kWarps / hg);
    return kWorkspaceHeader + ranges * 2 * hg * G * (d + 4) * sizeof(float);
}

template <int D, int G>
static int launch(const BlockDecodeParams &p, cudaStream_t s) {
    if (launch_pdl(block_decode_kernel<D, G>, dim3(decode_ctas()), dim3(32 * kWarps), 0, s, true, p) != cudaSuccess)
        return PKV_E_CUDA;
    return launch_pdl(block_merge_kernel<D, G>, dim3(p.batch, p.hkv), dim3(32 * kWarps), 0, s, true, p) == cudaSuccess
               ? PKV_OK
               : PKV_E_CUDA;
}

template <int D>
static int launch_group(int G, const BlockDecodeParams &p, cudaStream_t s) {
    switch (G) {
        case 1: return launch<D, 1>(p, s);
        case 2: return launch<D, 2>(p, s);
        case 4: return launch<D, 4>(p, s);
        default: return launch<D, 8>(p, s);
    }
}

static int check_group(const pkv_block_pool *pool, int32_t num_q_heads) {
    if (num_q_heads <= 0 || num_q_heads % pool->num_kv_heads) return PKV_E_INVALID;
    const int32_t G = num_q_heads / pool->num_kv_heads;
    return G == 1 || G == 2 || G == 4 || G == 8 ? PKV_OK : PKV_E_UNSUPPORTED;
}

}  // namespace pkv

extern "C" int pkv_decode_block_workspace(const pkv_block_pool *pool, int32_t num_q_heads, size_t *bytes) {
    using namespace pkv;
    int rc = validate_block_pool(pool);
    if (!rc) rc = check_group(pool, num_q_heads);
    if (rc) return rc;
    if (!bytes) return PKV_E_INVALID;
    *bytes = decode_workspace(pool->num_kv_heads, num_q_heads / pool->num_kv_heads, pool->head_dim);
    return PKV_OK;
}

extern "C" int pkv_attn_decode_block(const pkv_block_pool *pool, const pkv_batch *batch, const void *q, void *o,
                                     int32_t num_q_heads, float sm_scale, void *workspace, size_t ws_bytes,
                                     void *stream) {
    using namespace pkv;
    int rc = validate_block_pool(pool);
    if (!rc) rc = check_group(pool, num_q_heads);
    if (rc) return rc;
    if (!batch || batch->batch < 0) return PKV_E_INVALID;
    if (batch->batch == 0) return PKV_OK;
    if (!batch->req_to_token || !batch->req_pool_indices || !batch->seq_lens || !q || !o || !workspace)
        return PKV_E_INVALID;
    if (batch->page_size != pool->page_size || batch->stride < 0 || batch->stride >= ((int64_t)1 << 31) ||
        batch->num_rows < 0)
        return PKV_E_INVALID;
    if (pool->num_kv_heads > 65535) return PKV_E_UNSUPPORTED;
    if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(o)) & 15) return PKV_E_INVALID;
    if (reinterpret_cast<uintptr_t>(workspace) & 255) return PKV_E_INVALID;
    const int32_t hkv = pool->num_kv_heads, G = num_q_heads / hkv, D = pool->head_dim;
    if (ws_bytes < decode_workspace(hkv, G, D)) return PKV_E_WORKSPACE;
    BlockDecodeParams p;
    p.k = static_cast<const uint8_t *>(pool->k);
    p.v = static_cast<const uint8_t *>(pool->v);
    p.k_exp = pool->k_exp;
    p.v_exp = pool->v_exp;
    p.num_pages = pool->num_pages;
    p.slot_bytes = block_slot_bytes(pool);
    p.shift = log2_of(pool->page_size);
    p.hkv = hkv;
    p.hg = head_group(hkv);
    p.groups = hkv / p.hg;
    p.table = batch->req_to_token;
    p.stride = batch->stride;
    p.num_rows = batch->num_rows;
    p.batch = batch->batch;
    p.rows = batch->req_pool_indices;
    p.lens = batch->seq_lens;
    p.q = static_cast<const uint16_t *>(q);
    p.o = static_cast<uint16_t *>(o);
    p.scale_log2 = sm_scale * kLog2eB;
    p.ranges = decode_ctas() * (kWarps / p.hg);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.err = reinterpret_cast<int32_t *>(ws);
    p.rec = reinterpret_cast<float *>(ws + kWorkspaceHeader);
    p.rec_ml = p.rec + (size_t)p.ranges * 2 * p.hg * G * D;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return D == 128 ? launch_group<128>(G, p, s) : launch_group<64>(G, p, s);
}
