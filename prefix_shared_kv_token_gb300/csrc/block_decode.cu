// attn_decode_block: one query token per request over its whole context in a block-scaled 8-bit
// pool (block.cuh), read through a page table, with lengths that only the device knows.
//
// What is computed: for request r of length L and query head h of KV head g = h / G,
//     o[r, h] = sum_{j < L} softmax_j(sm_scale * q[r, h] . K_j) V_j,
//     K_j = 2^(ek - 127) * code,  V_j = 2^(ev - 127) * code  (exponent bytes of j's page and g).
// With s_j the logits in log2 units, R = max_j (s_j + ev_j) and w_j = 2^(s_j + ev_j - R), the sum
// is  sum w_j code_j / sum 2^(s_j - R):  V's exponents move into the weights, so the codes enter
// the product as they are, and a weight is at most 1 however far the pages' exponents differ.  The
// sum below is kept as l = sum 2^(s_j - R + ea), ea = ev of the key that set R, and the result is
// acc / l * 2^ea: that key counts 1 in l whatever its page's exponent.  A key of a far smaller ev may stand far
// above it in s_j alone and pass fp32's range in l (ev 127 or more below, s_j as much above).  Where l
// passes 2^100 the piece is attended once more with l's own reference R - ea moved up with max s_j; the
// joining kernel always takes the largest of its records' R - ea.
//
// Design.  The work is a stream of codes, so what counts is bytes in flight:
//   * 16-key tiles of all requests, laid end to end, are cut into equal contiguous ranges (each CTA
//     scans the lengths itself: no host plan, no set-up kernel, ragged batches balance to a tile,
//     and a captured graph follows the lengths).  A request inside one range is written directly;
//     one that crosses ranges leaves a record (R, l, acc, ea) in each, joined by a second kernel.
//   * A CTA has a warp for each of 8 KV heads (fewer heads: several ranges side by side).  Each warp
//     keeps a ring of its own full, asking for tiles 3 (d = 64: 6) ahead over the ends of requests:
//     one 16-row TMA box, swizzled, for K and one for V; two CTAs an SM, 192 KB of ring.
//   * K rows are the A operand (16 keys) of S^T = K Q^T, V^T the A operand of O^T = V^T P^T, and the
//     query rows are the 8 columns of B: a group of up to 8 heads shares one MMA and the accumulators
//     are d x 8.  V's bytes are paired by key with byte permutes on their way to f16.
//   * mma.sync m16n8k16 in f16: an e4m3 code is an f16 value, and so is a query element over a
//     power of two that brings its row's largest to [2^14, 2^15) (elements below 2^-31 of it
//     round, far under the fp32 sum's own rounding).  Weights are f16 times 2^6: 11 bits down to
//     2^-20 of the largest and a step of 2^-30 of it below, against bf16's 8 bits.
// A request may also have several query tokens (the last ext[r] positions of its context): each
// block of 8 / G of them is a *stream* of its own over the same keys, which only the first finds in
// HBM.

#include <algorithm>
#include <atomic>

#include "block.cuh"
#include "block_plan.h"

namespace pkv {

constexpr int kTile = 16;         // keys
constexpr int kMinTiles = 2;      // per range, while there are few (a lone tile takes 0.8 us)
constexpr int kWarps = 8;
constexpr int kRingBytes = 96 * 1024;
constexpr int kThreads = 32 * kWarps;
constexpr int kBatch = 4;         // records a merging warp has in flight
constexpr float kBias = 6.f;      // weights carry 2^6 over their reference, which may lag the
constexpr float kSlack = 8.f;     // largest by 2^8: they stay below 2^15 in f16
constexpr float kNoKey = -3.402823466e38f;  // the reference of a column that has seen no key: the least finite,
                                            // so that a logit of -inf less it is -inf
constexpr float kUnbias = 1.f / (1 << 6);
constexpr float kFarSum = 1.2676506e30f;  // 2^100: see careful
constexpr float kLog2eB = 1.4426950408889634f;

struct BlockDecodeParams {
    const uint8_t *k_exp, *v_exp;
    int64_t num_pages;
    int32_t shift, hkv, hg, groups;  // hg (a power of two) KV heads read side by side, `groups` times
    int32_t hg_shift;
    const int32_t *table;
    int64_t stride;
    int32_t num_rows, batch;
    const int32_t *rows, *lens;
    const int32_t *indptr;  // NULL: one query token a request; else request r's are rows
                            // [indptr[r], indptr[r + 1]) of q, its last positions
    const uint16_t *q;
    uint16_t *o;
    float scale_log2;
    int32_t ranges;  // at most
    int32_t *before;  // tiles before each unit, written by the first kernel for the second where there are
                      // too many units to add them up again; NULL: none
    const int32_t *share;  // decode: tiles that the requests of a stream have in common, NULL: none
    float *rec;      // [range][2][hg][8 columns][D] (d in the order that merge_head says), then
                     // (R, l, ea, -) [range][2][hg][8][4]
    float *rec_ml;
    int32_t *err;
    WaitPolicy wait;
};

// A request's length as the kernels use it: 0 where its row or length is out of range.
PKV_DEV int32_t checked_len(const BlockDecodeParams &p, int r, bool report) {
    const int32_t len = ld(p.lens + r), row = ld(p.rows + r);
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
    int32_t size, extra, n;
    PKV_DEV Cut(int32_t total, int32_t most) {
        n = min(most, max(1, total / kMinTiles));
        size = (int32_t)((uint32_t)total / (uint32_t)n);
        extra = total - size * n;
    }
    PKV_DEV int32_t start(int32_t i) const { return size * i + min(i, extra); }
    PKV_DEV int32_t range_of(int32_t t) const {
        const int32_t big = extra * (size + 1);
        return t < big ? (int32_t)((uint32_t)t / (uint32_t)(size + 1)) : extra + (int32_t)((uint32_t)(t - big) / (uint32_t)size);
    }
};
// The line's length for one group of heads as the kernels use it: 0 for one past 2^31 tiles in all
// (34 billion keys).
PKV_DEV int32_t line_length(const BlockDecodeParams &p, int64_t n, bool report) {
    if (n * p.groups <= 0x7FFFFFFF) return (int32_t)n;
    if (report) set_error(p.err, DERR_POSITION);
    return 0;
}

PKV_DEV void mma_f16_16816(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
PKV_DEV uint32_t transpose_8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
PKV_DEV uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
    return r;
}
// Query tokens of request r: (first row of q, how many), and of them the streams.
PKV_DEV int2 query_rows(const BlockDecodeParams &p, int r, int32_t len) {
    if (!p.indptr) return make_int2(r, 1);
    const int32_t a = ld(p.indptr + r), n = ld(p.indptr + r + 1) - a;
    return make_int2(a, min(n, len));
}
// Keys that the last token of stream s of a request sees (streams of M = 8 / G tokens).
PKV_DEV int32_t stream_len(int32_t len, int32_t ext, int32_t s, int32_t M) { return len - ext + min(ext, (s + 1) * M); }

// Decode: stream i is requests i M .. i M + M - 1, whose first shared_tiles are the same pages.  Its
// tiles: those, seen by every column, then each request's others, seen by its own.
PKV_DEV int32_t shared_tiles(const BlockDecodeParams &p, int i) { return p.share ? p.share[i] : 0; }

template <int32_t M>
PKV_DEV int64_t stream_tiles(const BlockDecodeParams &p, int i, bool report) {
    const int32_t share = shared_tiles(p, i);
    int64_t n = share;
#pragma unroll
    for (int m = 0; m < M; ++m)
        if (i * M + m < p.batch) n += tiles_of(checked_len(p, i * M + m, report)) - share;
    return n;
}
// Member i's own tiles of a decode stream that begins at tile `from` and shares `share`: where they
// begin and end.
template <int32_t M>
PKV_DEV int2 own_tiles(const BlockDecodeParams &p, int32_t r, int i, int32_t from, int32_t share) {
    int32_t a = from + share, b = a;
#pragma unroll
    for (int m = 0; m < M; ++m)
        if (m <= i && r + m < p.batch) {
            a = b;
            b += tiles_of(checked_len(p, r + m, false)) - share;
        }
    return make_int2(a, b);
}
// Whether a request's columns get results and records by its own tiles and not by its stream's: a request that
// shares no pages with the others of its stream then has no more records than it has ranges.  With 8 or 4
// requests a stream that is worth its bookkeeping (237 requests of up to 93 keys, 16 heads x 64, G = 1: 34 to
// 26 us), with 2 it is not (64 of up to 40 keys, 8 heads x 128, G = 4: 13.3 to 14.4).
template <int32_t M>
constexpr bool kApart = M >= 4;

// What a chunk of the line is counted in: streams (decode), or requests with all their streams.
template <int32_t M>
PKV_DEV int32_t num_units(const BlockDecodeParams &p) { return p.indptr ? p.batch : (p.batch + M - 1) / M; }
template <int32_t M>
PKV_DEV int64_t unit_tiles(const BlockDecodeParams &p, int i, bool report) {
    if (!p.indptr) return stream_tiles<M>(p, i, report);
    const int32_t len = checked_len(p, i, report), ext = query_rows(p, i, len).y;
    int64_t n = 0;
    for (int32_t s = 0; s * M < ext; ++s) n += tiles_of(stream_len(len, ext, s, M));
    return n;
}

// Query rows as B fragments, in the d order that K's 16-byte pieces have: k-step (half, j) holds
// d = 64 half + 16 c + 4 j + {0, 1 | 2, 3} of column g.  Returns the power of two taken out of
// column g.  `row`: column g's row of q (of num_q_heads * D elements at its head), NULL for none.
template <int D>
PKV_DEV int load_query(const uint16_t *row, uint32_t (&qb)[D / 16][2]) {
    const int c = threadIdx.x & 3;
    uint32_t w[D / 8];
    uint32_t amax = 0;
#pragma unroll
    for (int h = 0; h < D / 64; ++h)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint4 x = row ? ld(reinterpret_cast<const uint4 *>(row + 64 * h + 16 * c) + u) : make_uint4(0u, 0u, 0u, 0u);
            w[8 * h + 4 * u] = x.x;
            w[8 * h + 4 * u + 1] = x.y;
            w[8 * h + 4 * u + 2] = x.z;
            w[8 * h + 4 * u + 3] = x.w;
        }
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
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

// One (head, tensor) tile in shared memory: 16 rows of D bytes, 16-byte pieces swizzled by TMA (128
// bytes: piece ^ row mod 8; 64 bytes: piece ^ (row / 2) mod 4).  MMA row r holds key_of(r), an order
// under which the 8 lanes of a 16-byte access hit 8 different pieces (d = 128).
template <int D>
PKV_DEV int key_of(int r) {
    if constexpr (D == 128) return (int)((0x37156240u >> (4 * (r & 7))) & 7u) + (r & 8);
    return r;
}
template <int D>
PKV_DEV int piece_at(int key, int piece) {
    return D == 128 ? key * 128 + ((piece ^ (key & 7)) << 4) : key * 64 + ((piece ^ ((key >> 1) & 3)) << 4);
}

// Running state of one warp: columns 2c and 2c + 1 (query heads) of this lane.
template <int D>
struct DecodeState {
    float acc[D / 16][4];  // MMA i: d = (D/8) g + 2i + {0, 0, 1, 1}, heads 2c + {0, 1, 0, 1}
    float m[2], l[2], ea[2];
};

// The result of a row from its sums: acc times the first factor, then times the second.  (Their product may
// lie below fp32's normal numbers where the result does not: 2^-117 over the weights of a million keys.)
PKV_DEV float2 row_scale(float l, float ea) { return make_float2(l == 0.f ? 0.f : kUnbias / l, l == 0.f ? 0.f : ex2(ea)); }
PKV_DEV uint32_t pack_result(float a, float b, float2 f) { return pack_bf16x2(a * f.x * f.y, b * f.x * f.y); }

// Logits of a tile's 16 keys: this lane's MMA rows g and g + 8 of columns 2c and 2c + 1.  The rows
// g + 8 are 8 D bytes behind the rows g, under the same swizzle.
template <int D>
PKV_DEV void tile_scores(float (&t)[4], const uint32_t (&qb)[D / 16][2], const uint8_t *k, int off) {
    float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};  // two chains of MMAs
#pragma unroll
    for (int u = 0; u < D / 64; ++u) {
        // (piece 4 + c is piece c with that bit changed, under the swizzle too)
        const uint8_t *at = k + (off ^ 64 * u);
        const uint4 x = *reinterpret_cast<const uint4 *>(at), y = *reinterpret_cast<const uint4 *>(at + 8 * D);
        const uint32_t a[4] = {x.x, x.y, x.z, x.w}, b[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            mma_f16_16816(s[j & 1], e4m3x2_to_f16x2(a[j]), e4m3x2_to_f16x2(b[j]), e4m3x2_hi_to_f16x2(a[j]),
                          e4m3x2_hi_to_f16x2(b[j]), qb[4 * u + j][0], qb[4 * u + j][1]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) t[e] = s[0][e] + s[1][e];
}

// V rows of MMA k 2c, 2c + 1, 2c + 8, 2c + 9: D / 8 bytes each.  Rows at or past `valid` read as
// zeros: a weight of 0 does not undo a NaN or an infinity.
template <int D>
PKV_DEV void read_v(uint32_t (&v)[4][D / 32], const uint8_t *at, int off, bool ragged, int valid) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // (the key of MMA row 2c + 1 is that of 2c with one bit changed: 4 at d = 128, 1 at d = 64)
        const uint8_t *row = at + (i & 1 ? off ^ (D == 128 ? 4 * 128 | 4 << 4 : 64) : off) + (i >> 1) * 8 * D;
        if constexpr (D == 128) {
            const uint4 y = *reinterpret_cast<const uint4 *>(row);
            v[i][0] = y.x;
            v[i][1] = y.y;
            v[i][2] = y.z;
            v[i][3] = y.w;
        } else {
            const uint2 y = *reinterpret_cast<const uint2 *>(row);
            v[i][0] = y.x;
            v[i][1] = y.y;
        }
    }
    if (ragged) {
        const int c = threadIdx.x & 3;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (key_of<D>(2 * c + (i & 1) + 8 * (i >> 1)) >= valid)
#pragma unroll
                for (int j = 0; j < D / 32; ++j) v[i][j] = 0u;
    }
}

// Folds the tile's weights (as B fragments b0, b1) and its maximum into the running state.  ek, ev_byte:
// the tile's exponent bytes.  Columns are G heads each of the stream's requests or tokens: only the
// `only`-th sees the tile (-1: all do); ragged: the i-th sees of it the keys before sees + i step.
// (A logit that is not seen may be NaN: it is replaced.)
// The reference moves, and the state is rescaled, only when a key is more than 2^8 above it: then
// the lanes agree on the column's maximum.  careful: with every tile, and l's reference moves to the largest s
// too (a key's s is at most R - ea).
template <int D, int G>
PKV_DEV void tile_weights(DecodeState<D> &st, float (&t)[4], const float (&cs)[2], int ek, int ev_byte,
                          int only, bool ragged, int sees, int step, bool careful, uint32_t &b0, uint32_t &b1) {
    const float kf = exp_value(ek);
    // (a whole number below 2^23 as a float: its bits under those of 2^23)
    const float ev = __uint_as_float(0x4B000000u | (uint32_t)ev_byte) - (8388608.f + 127.f);
#pragma unroll
    for (int e = 0; e < 4; ++e) t[e] = t[e] * (cs[e & 1] * kf) + ev;
    const int col = 2 * (threadIdx.x & 3);
    if (only >= 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if ((col + (e & 1)) / G != only) t[e] = -INFINITY;
    }
    if (ragged) {
        const int row = key_of<D>((threadIdx.x & 31) >> 2);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (row + 8 * (e >> 1) >= sees + (col + (e & 1)) / G * step) t[e] = -INFINITY;
    }
    if (careful || __any_sync(0xffffffffu, fmaxf(t[0], t[2]) > st.m[0] + kSlack || fmaxf(t[1], t[3]) > st.m[1] + kSlack)) {
        float al[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float y = fmaxf(t[h], t[2 + h]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, d));
            al[h] = 1.f;
            if (y > st.m[h] || careful) {
                const float top = fmaxf(y, st.m[h]), ea = careful ? fminf(st.ea[h] + (top - st.m[h]), ev + (top - y)) : ev;
                al[h] = ex2(st.m[h] - top);
                st.l[h] *= ex2(st.m[h] - top + (ea - st.ea[h]));
                st.m[h] = top;
                st.ea[h] = ea;
            }
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) st.acc[i][e] *= al[e & 1];
    }
    float w[4], rw[2], rl[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        rw[h] = st.m[h] - kBias;
        rl[h] = st.m[h] + (ev - st.ea[h]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        w[e] = ex2(t[e] - rw[e & 1]);
        st.l[e & 1] += ex2(t[e] - rl[e & 1]);
    }
    b0 = transpose_8x8(pack_f16x2(w[0], w[1]));
    b1 = transpose_8x8(pack_f16x2(w[2], w[3]));
}

// O^T += V^T P^T.
template <int D>
PKV_DEV void tile_product(DecodeState<D> &st, const uint32_t (&v)[4][D / 32], uint32_t b0, uint32_t b1) {
#pragma unroll
    for (int j = 0; j < D / 32; ++j)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            // bytes (key, key + 1) of d and d + 1 next to each other
            const uint32_t lo = __byte_perm(v[0][j], v[1][j], u ? 0x7362 : 0x5140);
            const uint32_t hi = __byte_perm(v[2][j], v[3][j], u ? 0x7362 : 0x5140);
            mma_f16_16816(st.acc[2 * j + u], e4m3x2_to_f16x2(lo), e4m3x2_hi_to_f16x2(lo), e4m3x2_to_f16x2(hi),
                          e4m3x2_hi_to_f16x2(hi), b0, b1);
        }
}

// A weight of 0 does not undo a NaN in a V row that a column does not see.  Where there may be one
// (a segment of one of several requests; a tile that tokens see in part), the columns that did not
// see it get back what they had.
template <int D>
struct Kept {
    volatile float acc[D / 4];
    PKV_DEV void take(const DecodeState<D> &st) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[4 * i + e] = st.acc[i][e];
    }
    PKV_DEV void give_back(DecodeState<D> &st, const bool (&mine)[2]) const {
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (!mine[e & 1]) st.acc[i][e] = acc[4 * i + e];
    }
};
// Whether a column outside `mine` has become NaN (or infinite).
template <int D>
PKV_DEV bool poisoned(const DecodeState<D> &st, const bool (&mine)[2]) {
    float x[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e & 1] += st.acc[i][e] * 0.f;
    return (!mine[0] && x[0] != 0.f) || (!mine[1] && x[1] != 0.f);
}

// The results and records of a stream's piece.  Column 2c + h of this lane belongs to query row `row[h]`:
// a result where rec[h] < 0, that record elsewhere (row < 0: neither).
template <int D, int G>
PKV_DEV void write_piece(const BlockDecodeParams &p, DecodeState<D> &st, int kv_head, const int32_t (&row)[2], const int32_t (&rec)[2], int hl) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) st.l[h] += __shfl_xor_sync(0xffffffffu, st.l[h], d);
        const int col = 2 * c + h;
        if (row[h] < 0) continue;
        if (rec[h] < 0) {
            const float2 f = row_scale(st.l[h], st.ea[h]);
            uint4 *dst = reinterpret_cast<uint4 *>(p.o + ((int64_t)row[h] * p.hkv * G + kv_head * G + col % G) * D + g * (D / 8));
#pragma unroll
            for (int i = 0; i < D / 16; i += 4)
                dst[i / 4] = make_uint4(pack_result(st.acc[i][h], st.acc[i][2 + h], f),
                                        pack_result(st.acc[i + 1][h], st.acc[i + 1][2 + h], f),
                                        pack_result(st.acc[i + 2][h], st.acc[i + 2][2 + h], f),
                                        pack_result(st.acc[i + 3][h], st.acc[i + 3][2 + h], f));
        } else {
            const int64_t at = ((int64_t)rec[h] * p.hg + hl) * 8 + col;
            // piece i / 2 of lane g's run of d next to its neighbours' (see merge_head)
            float4 *dst = reinterpret_cast<float4 *>(p.rec + at * D) + g;
#pragma unroll
            for (int i = 0; i < D / 16; i += 2)
                dst[4 * i] = make_float4(st.acc[i][h], st.acc[i][2 + h], st.acc[i + 1][h], st.acc[i + 1][2 + h]);
            if (g == 0) *reinterpret_cast<float4 *>(p.rec_ml + at * 4) = make_float4(st.m[h], st.l[h], st.ea[h], 0.f);
        }
    }
}

// A place on the line: segment s of a stream, whose first tile is tile `first` of the line, for one
// group of heads.  A segment is a run of tiles of one request that the same columns see.
template <int G>
struct Walk {
    static constexpr int32_t M = 8 / G;
    int32_t grp, r, s;             // r: the stream's (first) request
    int32_t len, ext, q0;          // of the segment's request: length; query tokens and first row (decode: of r)
    int32_t first, tiles, key0;    // the segment's tiles; its first tile's number in the request
    int32_t from, all;             // the stream's first tile on the line and its tiles
    int32_t share;                 // decode: tiles that the stream's requests have in common

    // The request whose pages the segment reads, and the one member whose columns see it (-1: all).
    PKV_DEV int32_t member(const BlockDecodeParams &p) const { return p.indptr || s == 0 ? -1 : s - 1; }
    PKV_DEV int32_t request(const BlockDecodeParams &p) const { return r + max(member(p), 0); }

    // The stream that begins at tile `from`.
    PKV_DEV void load(const BlockDecodeParams &p) {
        first = from;
        if (p.indptr) {
            len = checked_len(p, r, false);
            const int2 qr = query_rows(p, r, len);
            q0 = qr.x;
            ext = qr.y;
            share = 0;
            all = tiles = s * M < ext ? tiles_of(stream_len(len, ext, s, M)) : 0;
            key0 = 0;
        } else {
            q0 = r;
            ext = min(M, p.batch - r);
            share = shared_tiles(p, r / M);
            all = (int32_t)stream_tiles<M>(p, r / M, false);
            s = 0;
            len = share * kTile;
            tiles = share;
            key0 = 0;
        }
    }
    // To the segment that holds tile `at` of the line, from one at or before it.  False when there is
    // none (the lengths changed under the call).
    PKV_DEV bool seek(const BlockDecodeParams &p, int32_t at) {
        while (at - first >= tiles) {
            first += tiles;
            if (!p.indptr && s < ext) {  // the next member's own tiles
                ++s;
                len = checked_len(p, r + s - 1, false);
                tiles = tiles_of(len) - share;
                key0 = share;
                continue;
            }
            from = first;
            if (p.indptr && (s + 1) * M < ext) {
                ++s;
            } else {
                s = 0;
                r += p.indptr ? 1 : M;
                if (r >= p.batch) {
                    r = 0;
                    if (++grp >= p.groups) return false;
                }
            }
            load(p);
        }
        return true;
    }
    // base: tiles before each of the 256 chunks of requests (decode: of streams); n tiles in a group
    // of heads
    PKV_DEV bool start(const BlockDecodeParams &p, const int32_t *base, int chunk, int32_t n, int32_t at) {
        grp = p.groups == 1 ? 0 : at / n;
        // the last chunk that begins at or before the tile: first of every 8, then of the 8
        const int lane = threadIdx.x & 31;
        const int32_t x = at - grp * n;
        int lo = 8 * (31 - __clz(__ballot_sync(0xffffffffu, base[8 * lane] <= x)));
        lo += 31 - __clz(__ballot_sync(0xffffffffu, lane < 8 && base[lo + lane] <= x));
        r = lo * chunk * (p.indptr ? 1 : M);
        s = 0;
        from = grp * n + base[lo];
        load(p);
        return seek(p, at);
    }
};

// Tiles that the M requests of each decode stream have in common: whole pages, counted from the
// front while every request's table names the same one.  A CTA a stream.
template <int M>
__global__ void __launch_bounds__(kThreads) block_share_kernel(const BlockDecodeParams p, int32_t *share) {
    __shared__ int32_t s_first;
    pdl_wait();
    pdl_trigger();
    const int r0 = blockIdx.x * M, members = min(M, p.batch - r0);
    const int32_t *rows[M];
    int32_t pages = 0x7FFFFFFF;
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const int r = r0 + min(m, members - 1);
        const int32_t len = checked_len(p, r, false);
        pages = min(pages, len >> p.shift);
        rows[m] = p.table + (int64_t)(len > 0 ? ld(p.rows + r) : 0) * p.stride;
    }
    if (members < M) pages = 0;  // the last stream, when it is not full
    if (threadIdx.x == 0) s_first = pages;
    __syncthreads();
    for (int32_t j0 = 0; j0 < pages; j0 += 2 * kThreads) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int32_t j = j0 + u * kThreads + threadIdx.x;
            if (j >= pages) continue;
            bool same = true;
            const int32_t first = ld(rows[0] + j);
#pragma unroll
            for (int m = 1; m < M; ++m) same &= ld(rows[m] + j) == first;
            if (!same) atomicMin(&s_first, j);
        }
        __syncthreads();
        if (s_first < j0 + 2 * kThreads) break;
        __syncthreads();
    }
    if (threadIdx.x == 0) share[blockIdx.x] = s_first << (p.shift - 4);
}

// A batch of tiles to ask for: up to tile `lim` of the line, of one KV head.
struct Ahead {
    int32_t lim, head;
};

// Touches a stream's query rows for one KV head, so that they are in L1 when the stream begins.
template <int D, int G>
PKV_DEV void warm_query(const BlockDecodeParams &p, const Walk<G> &w, int hl) {
    constexpr int32_t M = 8 / G, kLines = G * D * 2 / 128;  // 128-byte lines of a query row's group
    const int lane = threadIdx.x & 31, t = (p.indptr ? w.s * M : 0) + lane / kLines;
    if (lane < M * kLines && t < w.ext) {
        const uint16_t *at = p.q + ((int64_t)(w.q0 + t) * p.hkv * G + (w.grp * p.hg + hl) * G) * D + lane % kLines * 64;
        uint32_t x;
        asm volatile("ld.global.b32 %0, [%1];" : "=r"(x) : "l"(at));
    }
}

// A bounded wait for a tile (see WaitPolicy).
PKV_DEV bool tile_wait(uint64_t *bar, uint32_t parity, const BlockDecodeParams &p) {
    if (p.wait.quick ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t it = 1;; ++it) {
        if (p.wait.quick ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity)) return true;
        if ((it & p.wait.check_mask) == 0 && global_timer_ns() - t0 > p.wait.limit_ns) {
            set_error(p.err, DERR_TIMEOUT | 0x41);
            return false;
        }
    }
}

template <int D>
struct Ring {
    static constexpr int kBox = kTile * D;                            // a head's K or V tile
    static constexpr int kStages = kRingBytes / (kWarps * 2 * kBox);  // of one warp: 3 (d = 128), 6 (d = 64)
    static constexpr int kSmem = kRingBytes + 1024;                   // + alignment
};

template <int D, int G>
__global__ void __launch_bounds__(kThreads, 2)
    block_decode_kernel(const BlockDecodeParams p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
    using R = Ring<D>;
    extern __shared__ uint8_t dyn[];
    __shared__ int64_t warp_sums[kWarps];
    __shared__ int32_t base[kThreads + 1];  // tiles before each thread's chunk
    __shared__ uint64_t full[kWarps][R::kStages];
    __shared__ uint32_t exps[kWarps][R::kStages];  // of each tile in the ring: K's exponent byte, V's above it
    __shared__ Ahead ahead[kWarps][2];
    // where each warp asks and where it attends: read and written at a segment's end only
    __shared__ Walk<G> walks[kWarps], curs[kWarps];
    constexpr int32_t M = 8 / G;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < kWarps * R::kStages; ++i) mbar_init(&full[0][0] + i, 1);
        fence_mbar_init();
        prefetch_tmap(&kmap);
        prefetch_tmap(&vmap);
    }
    pdl_wait();
    pdl_trigger();
    const int32_t units = num_units<M>(p);
    const int chunk = (units + kThreads - 1) / kThreads;
    int64_t mine = 0;
    for (int i = tid * chunk; i < min((tid + 1) * chunk, units); ++i) mine += unit_tiles<M>(p, i, blockIdx.x == 0);
    int64_t scan = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, scan, d);
        if (lane >= d) scan += y;
    }
    if (lane == 31) warp_sums[warp] = scan;
    __syncthreads();
    int64_t before = 0, all = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w == warp) before = all;
        all += warp_sums[w];
    }
    const int32_t n = line_length(p, all, blockIdx.x == 0 && tid == 0);
    base[tid] = (int32_t)(before + scan - mine);
    if (tid == 0) base[kThreads] = n;
    if (p.before && blockIdx.x == 0) {
        int32_t at = base[tid];
        for (int i = tid * chunk; i < min((tid + 1) * chunk, units); ++i) {
            p.before[i] = at;
            at += (int32_t)unit_tiles<M>(p, i, false);
        }
        if (tid == 0) p.before[units] = n;
    }
    __syncthreads();
    if (n == 0) return;

    const Cut cut(n * p.groups, p.ranges);
    const int tpp = p.shift - 4;  // log2 of the tiles in a page
    const int hl = warp & (p.hg - 1);
    const int32_t range = blockIdx.x * (kWarps >> p.hg_shift) + (warp >> p.hg_shift);
    if (range >= cut.n) return;
    const int32_t begin = cut.start(range);
    int32_t end = cut.start(range + 1);
    const int g = lane >> 2, c = lane & 3;
    // this lane's first K piece and V bytes in a tile (see tile_scores and read_v for the others)
    const int k_off = piece_at<D>(key_of<D>(g), c);
    const int v_off = D == 128 ? piece_at<D>(key_of<D>(2 * c), g) : piece_at<D>(key_of<D>(2 * c), g >> 1) + 8 * (g & 1);
    uint8_t *ring = dyn + ((1024 - (smem_u32(dyn) & 1023)) & 1023) + warp * R::kStages * 2 * R::kBox;
    uint64_t *bars = full[warp];

    // The asking side runs up to kStages tiles ahead, over the ends of streams, in batches of up to 32
    // tiles of a segment: the lanes hold the first slots and exponents of the batch that is asked for
    // (tiles ask_b on, up to ask_lim), the same of the next, whose exponents are on their way, and the
    // slots of the one after, on their way too.  So no load is waited for where batches follow.
    const int32_t num_slots = (int32_t)(p.num_pages << p.shift);
    bool bad = false;
    // The batch that begins at tile `from` of the line; `warm`: its stream's queries have not been seen.
    auto take_batch = [&](int32_t from, Ahead &to, bool warm) {
        int32_t slot = num_slots;
        Ahead x = {from, 0};
        if (from < end) {
            Walk<G> w = walks[warp];
            if (w.seek(p, from)) {
                __syncwarp();
                if (lane == 0) walks[warp] = w;
                if (from == w.from || warm) warm_query<D, G>(p, w, hl);
                x.lim = min(min(w.first + w.tiles, from + 32), end);
                x.head = w.grp * p.hg + hl;
                const int32_t j = w.key0 + min(from + lane, x.lim - 1) - w.first;
                const int32_t page = ld(p.table + (int64_t)ld(p.rows + w.request(p)) * p.stride + (j >> tpp));
                // a page outside the pool: rows past the maps' last, which read as zeros
                const bool in = (uint32_t)page < (uint64_t)p.num_pages;
                bad |= !in;
                if (in) slot = (page << p.shift) + ((j * kTile) & ((1 << p.shift) - 1));
            } else {
                end = from;  // no such tile: what was taken is all there is
            }
        }
        __syncwarp();
        if (lane == 0) to = x;
        __syncwarp();
        return slot;
    };
    auto exps_of = [&](int32_t slot, int32_t head) {
        const int64_t at = (int64_t)(slot < num_slots ? slot >> p.shift : 0) * p.hkv + head;
        return (uint32_t)clamp_exp(ld(p.k_exp + at)) | (uint32_t)clamp_exp(ld(p.v_exp + at)) << 8;
    };
    int32_t slot_c, slot_n, slot_m, ask_at, ask_b, ask_lim, ask_head;
    uint32_t exps_c, exps_n, turn = 0;  // ahead[warp][turn] is the next batch, the other the one after it
    auto ask_tile = [&](uint32_t st) {
        if (ask_at >= ask_lim) return;
        const int32_t slot = __shfl_sync(0xffffffffu, slot_c, ask_at - ask_b);
        const uint32_t e = __shfl_sync(0xffffffffu, exps_c, ask_at - ask_b);
        if (lane == 0) {
            exps[warp][st] = e;
            mbar_arrive_expect_tx(&bars[st], 2 * R::kBox);
            const uint32_t dst = smem_u32(ring + st * 2 * R::kBox);
            tma_load_3d(dst, &kmap, 0, ask_head, slot, &bars[st]);
            tma_load_3d(dst + R::kBox, &vmap, 0, ask_head, slot, &bars[st]);
        }
        if (++ask_at == ask_lim) {
            const Ahead next = ahead[warp][turn], after = ahead[warp][turn ^ 1];
            ask_b = ask_at;
            ask_lim = next.lim;
            ask_head = next.head;
            slot_c = slot_n;
            exps_c = exps_n;
            slot_n = slot_m;
            exps_n = exps_of(slot_n, after.head);
            slot_m = take_batch(after.lim, ahead[warp][turn], false);
            turn ^= 1;
        }
    };
    uint32_t sg = 0, phase = 0;
    int32_t at = begin, piece = begin;  // the tile to attend next; the first tile of its piece
    // A piece is attended once more where a NaN was met (see poisoned; then columns are kept apart segment by
    // segment, which costs 8 % where it is not needed) or l passed 2^100 (its reference then moves with every tile).
    bool careful = false;
again:
    // from the piece's first tile, with nothing asked for
    at = ask_at = ask_b = piece;
    {
        Walk<G> w;
        if (!w.start(p, base, chunk, n, at)) return;
        if (lane == 0) walks[warp] = curs[warp] = w;
        __syncwarp();
    }
    slot_c = take_batch(at, ahead[warp][0], true);
    ask_lim = ahead[warp][0].lim;
    ask_head = ahead[warp][0].head;
    __syncwarp();
    slot_n = take_batch(ask_lim, ahead[warp][0], false);
    slot_m = take_batch(ahead[warp][0].lim, ahead[warp][1], false);
    turn = 0;
    exps_c = exps_of(slot_c, ask_head);
    exps_n = exps_of(slot_n, ahead[warp][0].head);
#pragma unroll 1
    for (uint32_t i = 0; i < R::kStages; ++i) ask_tile(sg + i < R::kStages ? sg + i : sg + i - R::kStages);

    bool ok = true, fresh = true, nan = false;  // fresh: a piece begins
    uint32_t qb[D / 16][2];
    float cs[2];
    DecodeState<D> st;
    while (at < end) {
        // last, all_see: keys of the segment's request that some column and every column see; only: the
        // one request or token whose columns do, -1: all
        int32_t last, all_see, only = -1, shift, j, j1;
        {
            Walk<G> w = curs[warp];
            if (!w.seek(p, at)) break;
            __syncwarp();
            if (lane == 0) curs[warp] = w;
            __syncwarp();
            if (fresh) {
                // columns: query row col / G of the stream's M, head col % G of the group
                const int32_t row = (p.indptr ? w.s * M : 0) + g / G, kv_head = w.grp * p.hg + hl;
                const int e = load_query<D>(
                    g / G < M && row < w.ext ? p.q + ((int64_t)(w.q0 + row) * p.hkv * G + kv_head * G + g % G) * D : nullptr, qb);
#pragma unroll
                for (int h = 0; h < 2; ++h) cs[h] = ldexpf(p.scale_log2, __shfl_sync(0xffffffffu, e, 8 * c + 4 * h));
#pragma unroll
                for (int i = 0; i < D / 16; ++i) st.acc[i][0] = st.acc[i][1] = st.acc[i][2] = st.acc[i][3] = 0.f;
                st.m[0] = st.m[1] = kNoKey;
                st.l[0] = st.l[1] = st.ea[0] = st.ea[1] = 0.f;
                fresh = false;
            }
            last = all_see = w.len;
            if (p.indptr) {
                last = stream_len(w.len, w.ext, w.s, M);
                all_see = w.len - w.ext + w.s * M + 1;
            } else if (M > 1 && w.ext > 1) {
                only = w.member(p);
            }
            shift = w.first - w.key0;
            j = at - shift;
            j1 = min(w.first + w.tiles, end) - shift;
        }
        Kept<D> had;
        const bool mine[2] = {2 * c / G == only, (2 * c + 1) / G == only};
        if (M > 1 && only >= 0 && careful) had.take(st);
#pragma unroll 1
        for (; j < j1; ++j) {
            ok = __all_sync(0xffffffffu, tile_wait(&bars[sg], phase, p));
            if (!ok) break;
            const uint8_t *tile = ring + sg * 2 * R::kBox;
            const uint32_t e = exps[warp][sg];
            float w[4];
            tile_scores<D>(w, qb, tile, k_off);
            uint32_t v[4][D / 32];
            const bool ragged = (j + 1) * kTile > all_see;
            read_v<D>(v, tile + R::kBox, v_off, ragged, last - j * kTile);
            __syncwarp();  // every lane has read the stage: ask for the tile kStages ahead
            ask_tile(sg);
            if (++sg == R::kStages) {
                sg = 0;
                phase ^= 1;
            }
            uint32_t b0, b1;
            tile_weights<D, G>(st, w, cs, e & 0xFF, e >> 8, M > 1 ? only : -1, ragged, all_see - j * kTile, M > 1 && p.indptr ? 1 : 0,
                               careful, b0, b1);
            // where tokens see different keys of the tile, one token at a time, from the one that sees
            // most: V's rows past each one's last key become zeros
            int t = M > 1 && ragged && p.indptr ? M - 1 : -1;
            do {
                if (M > 1 && t >= 0) {
                    had.take(st);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (j * kTile + key_of<D>(2 * c + (i & 1) + 8 * (i >> 1)) >= all_see + t)
#pragma unroll
                            for (int k = 0; k < D / 32; ++k) v[i][k] = 0u;
                }
                tile_product<D>(st, v, b0, b1);
                if (M > 1 && t >= 0) {
                    const bool its[2] = {2 * c / G == t, (2 * c + 1) / G == t};
                    had.give_back(st, its);
                }
            } while (M > 1 && --t >= 0);
        }
        at = shift + j;
        if (!ok) break;
        if (M > 1 && only >= 0) {
            if (careful) had.give_back(st, mine);
            else nan = nan || __any_sync(0xffffffffu, poisoned(st, mine));
        }
        const Walk<G> w = curs[warp];
        if (at == end || at == w.from + w.all) {
            bool far = false;  // (a column without a query row may see what nobody does)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                far |= (p.indptr ? w.s * M : 0) + (2 * c + h) / G < w.ext && !(st.l[h] <= kFarSum);
            nan = nan || (!careful && __any_sync(0xffffffffu, far));
            if (nan) break;
            // this lane's columns: a result where the range holds every tile that they see, a record
            // where it holds some
            const bool whole = w.from >= begin && at == w.from + w.all;
            int32_t out[2], rec[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int32_t i = (2 * c + h) / G, row = (p.indptr ? w.s * M : 0) + i;
                out[h] = i < M && row < w.ext ? w.q0 + row : -1;
                rec[h] = whole ? -1 : 2 * range + (w.from < begin ? 0 : 1);
                if (kApart<M> && !p.indptr && !whole && w.ext > 1) {
                    const int2 own = own_tiles<M>(p, w.r, i, w.from, w.share);
                    const int32_t first = w.share == 0 ? own.x : w.from, past = own.y > own.x ? own.y : w.from + w.share;
                    if (first >= begin && past <= at) rec[h] = -1;
                    if (piece >= w.from + w.share && max(own.x, piece) >= min(own.y, at)) out[h] = -1;
                }
            }
            write_piece<D, G>(p, st, w.grp * p.hg + hl, out, rec, hl);
            fresh = true;
            piece = at;
        }
    }
    // what was asked for and not attended lands before the warp goes on or ends (a wait gave up, or NaN)
    for (int32_t left = ask_at - at; left > 0; --left) {
        mbar_wait(&bars[sg], phase);
        if (++sg == R::kStages) {
            sg = 0;
            phase ^= 1;
        }
    }
    if (nan && ok) {
        careful = true;
        goto again;
    }
    if (bad) set_error(p.err, DERR_SLOT_RANGE);
}

// A query row's records: those of n1 ranges from i0 on and of the others, up to n, from j0 on.  They are
// the second ones in the range in which their stream begins.
struct Records {
    int32_t i0, n1, j0, n, stream;
};

// One query head's records into its row; `on`: there are any for this warp's head.  E is R - (l's reference):
// the least of ea_k + (R - R_k), so that no record's l counts more than once in L.
template <int D, int W, int S, bool kTwo, class Where>
PKV_DEV void merge_head(const BlockDecodeParams &p, uint16_t *out, bool on, const Where &from, int hl, int col,
                         float (&s_acc)[W][D], float4 (&s_ml)[W]) {
    constexpr int V = D / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp % S;
    // the records one after the other (kTwo), or the ranges themselves
    const int32_t i0 = kTwo ? 0 : from.i0, past = on ? i0 + from.n : i0;
    float top = -INFINITY, L = 0.f, E = INFINITY, O[V];
#pragma unroll
    for (int v = 0; v < V; ++v) O[v] = 0.f;
    for (int32_t i = i0 + sub; i < past; i += S * kBatch) {
        float4 ml[kBatch];
        float a[kBatch][V];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int32_t at = i + b * S, k = !kTwo ? at : at < from.n1 ? from.i0 + at : from.j0 + at - from.n1;
            ml[b] = make_float4(-INFINITY, 0.f, 0.f, 0.f);
#pragma unroll
            for (int v = 0; v < V; ++v) a[b][v] = 0.f;
            if (at >= past) continue;
            const int64_t rec = (((int64_t)k * 2 + (k == (kTwo ? from.stream : i0))) * p.hg + hl) * 8 + col;
            ml[b] = *reinterpret_cast<const float4 *>(p.rec_ml + rec * 4);
            if constexpr (V == 4) {
                const float4 y = *reinterpret_cast<const float4 *>(p.rec + rec * D + lane * V);
                a[b][0] = y.x;
                a[b][1] = y.y;
                a[b][2] = y.z;
                a[b][3] = y.w;
            } else {
                const float2 y = *reinterpret_cast<const float2 *>(p.rec + rec * D + lane * V);
                a[b][0] = y.x;
                a[b][1] = y.y;
            }
        }
        // the batch's reference first, so that its terms add independently
        const float was = top, was_e = E;
#pragma unroll
        for (int b = 0; b < kBatch; ++b) top = fmaxf(top, ml[b].x);
        if (top == -INFINITY) continue;
        E += top - was;
#pragma unroll
        for (int b = 0; b < kBatch; ++b) E = fminf(E, ml[b].z + (top - ml[b].x));
        const float f = ex2(was - top);
        L *= ex2(was - top + (E - was_e));
#pragma unroll
        for (int v = 0; v < V; ++v) O[v] *= f;
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const float w = ex2(ml[b].x - top);
            L += ml[b].y * ex2(ml[b].x - top + (E - ml[b].z));
#pragma unroll
            for (int v = 0; v < V; ++v) O[v] += a[b][v] * w;
        }
    }
    if constexpr (S > 1) {
        __syncthreads();  // the combining warp of the head before has read
#pragma unroll
        for (int v = 0; v < V; ++v) s_acc[warp][lane * V + v] = O[v];
        if (lane == 0) s_ml[warp] = make_float4(top, L, E, 0.f);
        __syncthreads();
        if (sub != 0) return;
        // the warps' sums the same way: lane w takes warp w's reference, sum and factor
        const float4 x = lane < S ? s_ml[warp + lane] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
        top = x.x;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float m = top == -INFINITY ? 0.f : top;
        E = x.z + (m - x.x);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) E = fminf(E, __shfl_xor_sync(0xffffffffu, E, d));
        const float f = ex2(x.x - m);
        L = x.x == -INFINITY ? 0.f : x.y * ex2(x.x - m + (E - x.z));
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) L += __shfl_xor_sync(0xffffffffu, L, d);
#pragma unroll
        for (int v = 0; v < V; ++v) O[v] = 0.f;
#pragma unroll 4
        for (int w = 0; w < S; ++w) {
            const float fw = __shfl_sync(0xffffffffu, f, w);
#pragma unroll
            for (int v = 0; v < V; ++v) O[v] += s_acc[warp + w][lane * V + v] * fw;
        }
    }
    if (!on) return;
    const float2 f = row_scale(L, E);
    // a record's 16-byte piece 8 i + g is d = (D / 8) g + 4 i + {0 .. 3}
    const int piece = lane * V / 4, d = D / 8 * (piece % 8) + 4 * (piece / 8) + lane * V % 4;
#pragma unroll
    for (int v = 0; v < V; v += 2)
        reinterpret_cast<uint32_t *>(out + d)[v / 2] = pack_result(O[v], O[v + 1], f);
}

// Joins the records of the streams that cross ranges and clears the rows of empty requests.  A CTA
// takes a query row and every gridDim.y-th (W / S) query heads, S warps a head: they share the
// head's records, four in flight a warp, and combine through shared memory.  S grows with the
// records of a stream: 1 for a few, 32 for a request alone in the batch, which may have one of every
// range (100,001 keys: 24 us with 8 warps a head, 6 with 32).  Lengths, rows and shared tiles are read
// before the wait: the decode kernel lets this one start only after its own wait for what wrote them.
template <int D, int G, int W, int S>
__global__ void __launch_bounds__(32 * W, 32 / W) block_merge_kernel(const BlockDecodeParams p) {
    __shared__ int64_t warp_sums[2 * W];
    __shared__ float s_acc[W][D];
    __shared__ float4 s_ml[W];
    __shared__ int32_t s_req;
    __shared__ Records s_from[kApart<8 / G> ? W : 1];  // (registers are short)
    constexpr int32_t M = 8 / G;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int32_t r = blockIdx.x / M, tok = blockIdx.x % M;  // decode: the stream and the row's place in it
    if (p.indptr) {  // the request of this query row, the row's place in it
        if (warp == 0) {
            // the last request that begins at or before the row, each step among 32 times fewer
            int lo = 0;
            for (int left = p.batch; left > 1;) {
                const int step = (left + 31) / 32, at = lo + lane * step;
                const bool on = lane * step < left && ld(p.indptr + at) <= (int32_t)blockIdx.x;
                const int skip = step * (31 - __clz(__ballot_sync(0xffffffffu, on) | 1u));
                lo += skip;
                left = min(step, left - skip);
            }
            if (lane == 0) s_req = (int32_t)blockIdx.x < ld(p.indptr + lo + 1) ? lo : -1;
        }
        __syncthreads();
        r = s_req;
        tok = r < 0 ? 0 : blockIdx.x - ld(p.indptr + r);
    }
    int64_t before = 0, all = 0;
    if (p.before) {
        pdl_wait();
        before = p.before[max(r, 0)];
        all = p.before[num_units<M>(p)];
    } else {
        for (int i = tid; i < num_units<M>(p); i += 32 * W) {
            const int64_t t = unit_tiles<M>(p, i, false);
            all += t;
            if (i < r) before += t;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            all += __shfl_xor_sync(0xffffffffu, all, d);
            before += __shfl_xor_sync(0xffffffffu, before, d);
        }
        if (lane == 0) {
            warp_sums[warp] = all;
            warp_sums[W + warp] = before;
        }
        __syncthreads();
        all = before = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            all += warp_sums[w];
            before += warp_sums[W + w];
        }
    }
    const int32_t n = line_length(p, all, false);
    // the row's tiles on the line of a group of heads: `share` from `before` on and own.x .. own.y (or the
    // stream's); tiles: how many (0: the row sees no key)
    int32_t tiles = 0, share = 0;
    int2 own = make_int2(0, 0);
    if (n > 0 && !p.indptr) {
        if (kApart<M>) {
            share = shared_tiles(p, r);
            own = own_tiles<M>(p, r * M, tok, (int32_t)before, share);
        } else {
            tiles = (int32_t)stream_tiles<M>(p, r, false);
        }
        if (checked_len(p, blockIdx.x, false) == 0) tiles = 0;
        else if (kApart<M>) tiles = share + own.y - own.x;
    } else if (n > 0 && r >= 0) {
        const int32_t len = checked_len(p, r, false), ext = query_rows(p, r, len).y, s = tok / M;
        for (int32_t i = 0; i < s; ++i) before += tiles_of(stream_len(len, ext, i, M));
        if (tok < ext) tiles = tiles_of(stream_len(len, ext, s, M));
        own = make_int2((int32_t)before, (int32_t)before + tiles);
    }
    constexpr int V = D / 32;  // elements a lane holds
    const int sub = warp % S;
    const Cut cut(max(n * p.groups, 1), p.ranges);
    const int hq = p.hkv * G, step = W / S * gridDim.y;
    int32_t grp = -1;
    Records from{};
    // where the records of a group of heads are, for this warp
    auto locate = [&](int32_t of) {
        grp = of;
        const int32_t first = grp * n + (int32_t)before;
        if constexpr (kApart<M>) {
            const int32_t base = grp * n;
            const bool shares = share > 0;
            Records x{};
            x.stream = cut.range_of(first);
            x.i0 = shares ? x.stream : cut.range_of(base + own.x);
            x.n = x.n1 = cut.range_of((shares ? first + share : base + own.y) - 1) - x.i0 + 1;
            if (shares && own.y > own.x) {  // (a range that holds tiles of both has one record)
                x.j0 = max(cut.range_of(base + own.x), x.i0 + x.n1);
                x.n += max(cut.range_of(base + own.y - 1) - x.j0 + 1, 0);
            }
            __syncwarp();
            if (lane == 0) s_from[warp] = x;
            __syncwarp();
        } else {
            from.i0 = cut.range_of(first);
            from.n = cut.range_of(first + tiles - 1) - from.i0 + 1;
        }
    };
    if (kApart<M> && tiles > 0) locate(min(W / S * (int)blockIdx.y + warp / S, hq - 1) / G / p.hg);
    pdl_wait();  // the records
    pdl_trigger();
    for (int h0 = W / S * blockIdx.y; h0 < hq; h0 += step) {
        const int qh = h0 + warp / S;
        const bool on = qh < hq;
        const int head = on ? qh / G : 0, q = qh % G;
        uint16_t *out = p.o + ((int64_t)blockIdx.x * hq + qh) * D;
        if (tiles == 0) {
            if (on && sub == 0)
                for (int d = lane; d < D / 2; d += 32) reinterpret_cast<uint32_t *>(out)[d] = 0u;
            continue;
        }
        if (head / p.hg != grp) locate(head / p.hg);
        if constexpr (kApart<M>) {
            const volatile Records &where = s_from[warp];
            merge_head<D, W, S, true>(p, out, on && where.n > 1, where, head % p.hg, tok % M * G + q, s_acc, s_ml);
        } else {
            merge_head<D, W, S, false>(p, out, on && from.n > 1, from, head % p.hg, tok % M * G + q, s_acc, s_ml);
        }
    }
}

static int head_group(int32_t hkv) {
    int hg = kWarps;
    while (hkv % hg) hg /= 2;
    return hg;
}
static int decode_ctas() { return 2 * num_sms(); }

// Bytes of a range's two records.
static size_t range_bytes(int hg, int32_t d) { return 2 * (size_t)hg * 8 * (d + 4) * sizeof(float); }

// Requests of rows shorter than this are not looked through: the look costs about 2 us.
constexpr int64_t kMinShared = 1024;
constexpr int kMaxListed = 65536;  // streams that have a place in the lists: share, and before with its end
constexpr size_t kListBytes = 2 * kMaxListed * sizeof(int32_t) + 256;

static size_t decode_workspace(int32_t hkv, int32_t d) {
    const int hg = head_group(hkv);
    return kWorkspaceHeader + kListBytes + (size_t)decode_ctas() * (kWarps / hg) * range_bytes(hg, d);
}

template <int D, int G>
static int launch(BlockDecodeParams p, int32_t *share, const CUtensorMap &kmap, const CUtensorMap &vmap, int64_t q_rows, cudaStream_t s) {
    constexpr int smem = Ring<D>::kSmem;
    static std::atomic<uint64_t> allowed{0};  // devices on which the kernel may use that much
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return PKV_E_CUDA;
    if (dev >= 64 || !((allowed.load(std::memory_order_relaxed) >> dev) & 1)) {
        if (cudaFuncSetAttribute(block_decode_kernel<D, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
            return PKV_E_CUDA;
        if (dev < 64) allowed.fetch_or((uint64_t)1 << dev, std::memory_order_relaxed);
    }
    const int per_cta = kWarps / p.hg;
    constexpr int M = 8 / G;
    if constexpr (M > 1) {
        const int64_t streams = (p.batch + M - 1) / M;
        if (share && p.batch > 1 && streams <= kMaxListed && (p.stride << p.shift) >= kMinShared) {
            if (launch_pdl(block_share_kernel<M>, dim3((unsigned)streams), dim3(kThreads), 0, s, true, p, share) != cudaSuccess)
                return PKV_E_CUDA;
            p.share = share;
        }
    }
    if (launch_pdl(block_decode_kernel<D, G>, dim3((p.ranges + per_cta - 1) / per_cta), dim3(kThreads), smem, s, true, p, kmap,
                   vmap) != cudaSuccess)
        return PKV_E_CUDA;
    // records of a row, at most, in a batch like this one (a request that shares no pages has those of its own
    // tiles)
    const int64_t parts = p.indptr || p.share || !kApart<M> ? (q_rows + M - 1) / M : q_rows;
    const int64_t each = p.ranges / std::max<int64_t>(parts * p.groups, 1), hq = p.hkv * G;
    auto merge = each > 64 ? block_merge_kernel<D, G, 32, 32> : each > 4 ? block_merge_kernel<D, G, kWarps, kWarps>
                                                                         : block_merge_kernel<D, G, kWarps, 1>;
    const int64_t heads = each > 4 ? 1 : kWarps;  // a CTA's at a time
    const int64_t y = std::min<int64_t>((hq + heads - 1) / heads, std::max<int64_t>(1, 8 * (int64_t)num_sms() / q_rows));
    return launch_pdl(merge, dim3((unsigned)q_rows, (unsigned)y), dim3(each > 64 ? 1024 : 32 * kWarps), 0, s, true, p) ==
                   cudaSuccess
               ? PKV_OK
               : PKV_E_CUDA;
}

template <int D>
static int launch_group(int G, const BlockDecodeParams &p, int32_t *share, const CUtensorMap &kmap, const CUtensorMap &vmap, int64_t q_rows,
                        cudaStream_t s) {
    switch (G) {
        case 1: return launch<D, 1>(p, share, kmap, vmap, q_rows, s);
        case 2: return launch<D, 2>(p, share, kmap, vmap, q_rows, s);
        case 4: return launch<D, 4>(p, share, kmap, vmap, q_rows, s);
        default: return launch<D, 8>(p, share, kmap, vmap, q_rows, s);
    }
}

static int check_group(const pkv_block_pool *pool, int32_t num_q_heads) {
    if (num_q_heads <= 0 || num_q_heads % pool->num_kv_heads) return PKV_E_INVALID;
    const int32_t G = num_q_heads / pool->num_kv_heads;
    return G == 1 || G == 2 || G == 4 || G == 8 ? PKV_OK : PKV_E_UNSUPPORTED;
}

// [slot][head][d] codes as 16-slot boxes of one head.
static int code_map(CUtensorMap *m, const pkv_block_pool *pool, void *codes) {
    const cuuint64_t dims[3] = {(cuuint64_t)pool->head_dim, (cuuint64_t)pool->num_kv_heads,
                                (cuuint64_t)(pool->num_pages * pool->page_size)};
    const cuuint64_t strides[2] = {(cuuint64_t)pool->head_dim, (cuuint64_t)block_slot_bytes(pool)};
    const cuuint32_t box[3] = {(cuuint32_t)pool->head_dim, 1, kTile};
    return encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, codes, dims, strides, box,
                        pool->head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B) == CUDA_SUCCESS
               ? PKV_OK
               : PKV_E_CUDA;
}

// Few query tokens a request (indptr NULL: one), over as many ranges as the workspace has records for.
int block_attend_few(const pkv_block_pool *pool, const pkv_batch *batch, const int32_t *indptr, int64_t q_rows, const void *q,
                     void *o, int32_t num_q_heads, float sm_scale, void *workspace, size_t ws_bytes, cudaStream_t s) {
    const int32_t hkv = pool->num_kv_heads, G = num_q_heads / hkv, D = pool->head_dim;
    BlockDecodeParams p;
    p.k_exp = pool->k_exp;
    p.v_exp = pool->v_exp;
    p.num_pages = pool->num_pages;
    p.shift = log2_of(pool->page_size);
    p.hkv = hkv;
    p.hg = head_group(hkv);
    p.groups = hkv / p.hg;
    p.hg_shift = log2_of(p.hg);
    p.table = batch->req_to_token;
    p.stride = batch->stride;
    p.num_rows = batch->num_rows;
    p.batch = batch->batch;
    p.rows = batch->req_pool_indices;
    p.lens = batch->seq_lens;
    p.indptr = indptr;
    p.q = static_cast<const uint16_t *>(q);
    p.o = static_cast<uint16_t *>(o);
    p.scale_log2 = sm_scale * kLog2eB;
    // workspace: header | decode: tiles shared by each stream, tiles before each; else, of many requests, tiles
    // before each | records
    const size_t list = block_list_bytes(batch->batch), head = kWorkspaceHeader + (indptr ? list : kListBytes);
    const size_t room = ws_bytes < head ? 0 : (ws_bytes - head) / range_bytes(p.hg, D);
    // no more ranges than the tables have room for tiles of
    const int64_t M = 8 / G, tiles = (std::min<int64_t>(batch->stride, ((int64_t)1 << 31) >> p.shift) << p.shift) / kTile;
    const int64_t line = (indptr ? (q_rows + M - 1) / M + batch->batch : batch->batch) * tiles * p.groups;
    p.ranges = (int32_t)std::min<int64_t>({(int64_t)decode_ctas() * (kWarps / p.hg), (int64_t)room,
                                           std::max<int64_t>(1, line / kMinTiles)});
    if (p.ranges < 1) return PKV_E_WORKSPACE;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.err = reinterpret_cast<int32_t *>(ws);
    int32_t *share = indptr ? nullptr : reinterpret_cast<int32_t *>(ws + kWorkspaceHeader);
    p.share = nullptr;
    const int64_t streams = (batch->batch + M - 1) / M;
    if (indptr) p.before = list ? reinterpret_cast<int32_t *>(ws + kWorkspaceHeader) : nullptr;
    else p.before = streams > kManyUnits && streams <= kMaxListed ? share + kMaxListed : nullptr;
    p.rec = reinterpret_cast<float *>(ws + head);
    p.rec_ml = p.rec + (size_t)p.ranges * 2 * p.hg * 8 * D;
    p.wait = wait_policy(wait_limit_ns());
    CUtensorMap kmap, vmap;
    int rc = code_map(&kmap, pool, pool->k);
    if (!rc) rc = code_map(&vmap, pool, pool->v);
    if (rc) return rc;
    return D == 128 ? launch_group<128>(G, p, share, kmap, vmap, q_rows, s) : launch_group<64>(G, p, share, kmap, vmap, q_rows, s);
}

}  // namespace pkv

extern "C" int pkv_decode_block_workspace(const pkv_block_pool *pool, int32_t num_q_heads, size_t *bytes) {
    using namespace pkv;
    int rc = validate_block_pool(pool);
    if (!rc) rc = check_group(pool, num_q_heads);
    if (rc) return rc;
    if (!bytes) return PKV_E_INVALID;
    *bytes = decode_workspace(pool->num_kv_heads, pool->head_dim);
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
    if (num_q_heads > 65535) return PKV_E_UNSUPPORTED;
    if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(o)) & 15) return PKV_E_INVALID;
    if (reinterpret_cast<uintptr_t>(workspace) & 255) return PKV_E_INVALID;
    if (ws_bytes < decode_workspace(pool->num_kv_heads, pool->head_dim)) return PKV_E_WORKSPACE;
    return block_attend_few(pool, batch, nullptr, batch->batch, q, o, num_q_heads, sm_scale, workspace, ws_bytes,
                            reinterpret_cast<cudaStream_t>(stream));
}
