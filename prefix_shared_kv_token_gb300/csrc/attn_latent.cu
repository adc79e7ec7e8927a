// attn_latent: attention of each request's newest tokens over a latent pool (the absorbed form).
// A pool row is a token's latent c (R elements) and its rotary key (64); every head's key is the
// whole row, every head's value the latent:
//     o[t, h] = sum_{j <= position of t} softmax_j(sm_scale * q[t, h] . row_j) * c_j.
//
// One row of 2 (R + 64) bytes serves all heads, so the product is far denser than attention over
// K/V heads: 2 (2 R + 64) flops a head and key.  With 16 heads the row's bytes bound the call, with
// 128 the tensor cores do as much.
//
// Both products run transposed, keys and latent elements in the M rows of tcgen05.mma and query
// rows (token x head) in its N columns:
//     S^T [64 keys x N] = rows Q^T           (A: the tile as it lies in shared memory, K-major)
//     O^T [R x N]      += c^T P^T            (A: the same tile, MN-major, R / 128 products of M 128)
// So one copy of a tile feeds both; the accumulator takes R / 128 * N columns of tensor memory,
// where O itself would take all 512 for any M and leave no room for S; and N may be as small as the
// rows there are (16, 32 or 64), with M still full.  A tile of 64 keys is 72 KB at R = 512: two of
// them and Q fill the 227 KB; P takes the place of its tile's rotary keys, which are done with once S is.
//
// A CTA of 12 warps:
//   warps 0, 1  issue the products, S and P V
//   warps 2, 3  copy the tile's rows, 16 bytes a cp.async, straight into the 128-byte swizzle; Q by TMA
//   warps 4-11  softmax: S^T from tensor memory (16x32bx2: the 16 lanes that an M of 64 fills, columns split
//               between the half-warps), a thread one key and N / 4 columns; P back through shared memory
// The softmax needs a column's maximum, which lies across lanes.  A running reference stands in for it: weights
// are 2^(s - ref), and only where a logit passes ref by more than 8 (a vote a tile) is the tile's maximum
// reduced, ref raised and O^T rescaled: once at a unit's start, seldom after.  Weights stay below 2^8, in
// bf16 (their own sum is what they are divided by).  Sums are fp32.
//
// Where a row sees fewer than kPreciseKeys keys, each with a large share of the output, a rounded weight would cost as much as
// the output's own rounding leaves: such a unit's first tile is gone through a second time, with what the first time's
// rounding left of those rows' weights.  (There is no room for both parts of P at once.)  At 2, 8 and 31 keys the relative
// error is then that of the output's rounding, 0.00166; with one part it is 0.00175, 0.00190 and 0.00202, and stays near
// that (0.0020 to 0.0022 from 32 keys on).  64 requests of 1 to 31 keys and 16 heads take 12.8 us, 11.7 with one part; 8
// prompts of 128 tokens and 128 heads 106 and 85.
//
// What bounds it (R = 512).  64 ragged requests of 32 heads, 648 MB: 115 us, 5.6 TB/s, 83 % of a copy's rate: DRAM.
// With 128 heads the products, 1,920 cycles a tile and 64 rows (S 36 of 32 cycles, half of a full M's rate; P V 16 of 48, for a
// product of N 64 is bound by reading A), are busy half of the time: 256 requests 207 us, 733 TFLOP/s, 38 % of cuBLAS's
// rate.  A tile lives for some 6,000 cycles in its stage (2,700 to be copied, 1,900 in S beside the other tile's P V, 1,200 in
// the softmax, 200 in its own P V's first 16 keys), there is room for two, and so one is done every 3,000.
//
// Work is divided on the device, from seq_lens: tiles of all requests in a line, an equal range of them a
// CTA (or pair, below), so a captured graph follows the lengths.  A request's rows beyond N are further units of the
// line; with more than 64 rows two CTAs take the same range, 64 rows each, so that the second one's tiles
// come from L2.  A range's first and last unit may be shared with its neighbours: their partial sums go to records
// in the workspace, which latent_merge_kernel joins.

#include <algorithm>
#include <atomic>
#include <cmath>

#include "../../include/pkv.h"
#include "common.cuh"
#include "latent.cuh"
#include "launch.h"

namespace pkv {

constexpr int kLTile = 64;              // keys a tile
constexpr int kLThreads = 384;
constexpr int kLSoftmax = 256;          // threads of the softmax warps
constexpr int kLBarHalf = 1;            // named barriers of the softmax warps' halves: 1 and 2
constexpr float kLUnset = -3.4028234e38f;  // a reference before any key was seen: no finite logit is below it
constexpr int kLCached = 64;            // requests of a range that are kept in shared memory
constexpr int kLMaxCtas = 160;          // the lists of latent_merge_kernel
constexpr int32_t kLLongest = 0x7FFFFF00;  // keys of a request: tiles' ends stay within 32 bits
// What a unit counts in the line beside its tiles, for its start and its output: 32 requests of 500 to 1,500 keys and 32 heads
// take 21.2 us with 0, 18.8 with 2 and 19.6 with 3; 64 of 1 to 200 keys 19.0, 15.0 and 15.4; 256 of 1,200 to 3,000 keys and 128
// heads 214, 211 and 213.
constexpr int kLUnitTiles = 2;
constexpr int kLMinTiles = 2;           // a range's tiles at least
constexpr float kLog2eL = 1.4426950408889634f;
constexpr float kLagL = 8.0f;           // log2 units by which a logit may pass its reference

struct LatentParams {
    const int32_t *table;
    int64_t stride;
    int32_t num_rows, shift;
    const int32_t *rows, *lens, *indptr;  // indptr NULL: one token a request
    int32_t batch, heads;
    int64_t total_q, num_slots;
    const uint16_t *pool;
    int64_t pool_stride;                  // elements
    uint16_t *o;
    float scale_log2;
    int32_t gs, ranges;                   // CTAs that share a range; ranges
    float *rec;                           // [range][2][gs][N][R]
    float *rec_ml;                        // [range][2][gs][N][2]
    int32_t *units;                       // [range][8]: first unit (request, set, ends there), last unit (request, set);
                                          // words 3 and 7: whether the range's first CTA gave up, and its second
    int32_t *err;
    WaitPolicy wait;
};

template <int R, int N>
struct LCfg {
    static constexpr int kBlocks = R / 64 + 1;                   // 64-column blocks of a row
    static constexpr int kBlk = kLTile * 128;
    static constexpr int kStage = kBlocks * kBlk;
    static constexpr int kStages = R == 512 ? 2 : 4;
    static constexpr int kQBlk = N * 128;
    static constexpr int kQOff = kStages * kStage;
    static constexpr int kMiscOff = kQOff + kBlocks * kQBlk;
    static constexpr int kSmem = kMiscOff + 4096;
    static constexpr int kCols = N / 4;                          // columns a softmax thread
    static constexpr uint32_t kColO = 128;                       // O^T block b at kColO + b * N
};

struct LMisc {
    uint64_t full[4], empty[16];  // [stage], [stage][16 keys]
    uint64_t qfull, qempty, sfull[2], pfull[2], pvdone[2], ofull, drain[2];
    uint32_t tmem_base;
    int32_t abort_flag;
    int32_t start_r;      // the range's first request, and the tiles of it that earlier ranges have
    int32_t pad;
    int64_t start_off, left;
    int64_t scan[12];
    int4 req[kLCached];   // the range's first requests
    float4 col[64];       // the quarters' column maxima; sums at the end
    float ref[64];        // columns' references
    float alpha[64];      // factors of a rescaling; 1 / sum at the end
    int32_t lim[64];      // keys that each row sees
    int32_t zeroed[2][kLTile];  // [tile mod 2]: the last tile, from 1, in which a key's latent was not finite
};
static_assert(sizeof(LMisc) <= 4096, "LMisc");

// ------------------------------------------------------------------------------------------
// the line of tiles

// A request as it is read, (length, row, first query token, new tokens), with what is out of range set to 0.
PKV_DEV int4 read_req(const LatentParams &p, int r, bool report) {
    int4 q = make_int4(ld(p.lens + r), ld(p.rows + r), r, 1);
    if (p.indptr) {
        q.z = ld(p.indptr + r);
        q.w = ld(p.indptr + r + 1) - q.z;
    }
    bool bad = false;
    if (q.z < 0 || q.w < 0 || (int64_t)q.z + q.w > p.total_q) {
        bad = true;
        q.z = q.w = 0;
    }
    if (q.y < 0 || q.y >= p.num_rows || q.x < 0 || q.x > kLLongest || (int64_t)q.x > (p.stride << p.shift)) {
        bad = true;
        q.x = 0;
    }
    if (bad && report) set_error(p.err, DERR_POSITION);
    return q;
}
// Its units, and what each counts in the line.
template <int N>
PKV_DEV int32_t sets_of(const LatentParams &p, const int4 &q) {
    const int rps = N * p.gs;
    return (int32_t)(((uint32_t)q.w * (uint32_t)p.heads + rps - 1) / rps);
}
PKV_DEV int32_t tiles_of(const int4 &q) { return max(1, (q.x + kLTile - 1) / kLTile) + kLUnitTiles; }

// A piece of one unit: this CTA's rows against tiles [t0, t1).
struct LSeg {
    int32_t r, set, row, vis;     // vis: keys that the unit's last row sees
    int32_t t0, t1, nrows;        // nrows: this CTA's rows of the unit (0: none)
    int32_t q_row0;               // first of them, in rows of q
    int32_t vis0;                 // keys that the request's first new token sees (0 or less: none)
    int32_t row_lo;               // first of them, in rows of the request
    bool whole, first, ends;      // all of the unit is in this range; the range begins inside it; it ends in this range
    int32_t twice;                // 1: tile 0 is gone through twice (see kPreciseKeys).  Steps i are start() .. t1 - 1, their
                                  // tiles max(i, 0)
    PKV_DEV int32_t start() const { return t0 - twice; }
};

struct LCursor {
    int32_t r, j, t;              // request; its unit and tile
    int64_t left;
    int4 q;                       // the request
    int32_t sets, tiles;          // 0 sets: not read yet
};

template <int N>
PKV_DEV void load_cursor(const LatentParams &p, const LMisc *m, LCursor &c) {
    const int at = c.r - m->start_r;
    c.q = at < kLCached ? m->req[at] : read_req(p, c.r, false);
    c.sets = sets_of<N>(p, c.q);
    c.tiles = tiles_of(c.q);
}

template <int N>
PKV_DEV LCursor cursor_at(const LatentParams &p, const LMisc *m) {
    LCursor c{m->start_r, 0, 0, m->left, make_int4(0, 0, 0, 0), 0, 0};
    if (c.left > 0) {
        load_cursor<N>(p, m, c);
        c.j = (int32_t)(m->start_off / c.tiles);
        c.t = (int32_t)(m->start_off - (int64_t)c.j * c.tiles);
    }
    return c;
}

template <int N>
PKV_DEV bool next_seg(const LatentParams &p, const LMisc *m, LCursor &c, LSeg &s, int g) {
    const int rps = N * p.gs;
    if (c.left <= 0) return false;
    while (c.sets == 0) {
        if (c.r >= p.batch) return false;
        load_cursor<N>(p, m, c);
        c.j = c.t = 0;
        if (c.sets == 0) ++c.r;
    }
    // A request's units in the order first, last, second, last but one, ..: the earlier ones see fewer keys of the
    // new tokens than they count for, and so any stretch of the line has about its share of the work.
    s.set = c.j & 1 ? c.sets - 1 - (c.j >> 1) : c.j >> 1;
    s.r = c.r;
    s.row = c.q.y;
    const int32_t n = (int32_t)min((int64_t)(c.tiles - c.t), c.left);
    const uint32_t all = (uint32_t)c.q.w * (uint32_t)p.heads;  // (below 2^31, as all rows of q are)
    const uint32_t lo = (uint32_t)s.set * rps + g * N, set_end = min((uint32_t)(s.set + 1) * rps, all);
    s.row_lo = (int32_t)lo;
    s.nrows = lo < all ? (int32_t)min((uint32_t)N, all - lo) : 0;
    s.q_row0 = (int32_t)((uint32_t)c.q.z * (uint32_t)p.heads + lo);
    s.vis0 = c.q.x - c.q.w + 1;
    s.vis = max(0, s.vis0 + (int32_t)((set_end - 1) / (uint32_t)p.heads));
    s.t0 = c.t;
    s.t1 = max(c.t, min(c.t + n, (s.vis + kLTile - 1) / kLTile));
    s.first = c.t > 0;
    s.ends = c.t + n == c.tiles;
    s.whole = !s.first && s.ends;
    // keys that this CTA's first row sees, and its last one: some row from 2 to kPreciseKeys - 1?
    const int32_t fewest = s.vis0 + (int32_t)(lo / (uint32_t)p.heads), most = s.vis0 + (int32_t)((lo + s.nrows - 1) / (uint32_t)p.heads);
    s.twice = s.t0 == 0 && s.t1 > 0 && s.nrows > 0 && fewest < kPreciseKeys && most > 1;
    c.left -= n;
    c.t += n;
    if (c.t == c.tiles) {
        c.t = 0;
        if (++c.j == c.sets) {
            c.sets = 0;
            ++c.r;
        }
    }
    return true;
}

// The next piece with rows and tiles; the producer and the issuer see no others.
template <int N>
PKV_DEV bool next_work(const LatentParams &p, const LMisc *m, LCursor &c, LSeg &s, int g) {
    while (next_seg<N>(p, m, c, s, g))
        if (s.nrows > 0 && s.t1 > s.t0) return true;
    return false;
}

// ------------------------------------------------------------------------------------------

// A wait that gave up: unlike what else may stand in the word, it leaves outputs unwritten, and so takes that one's place.
PKV_DEV void set_timeout(int32_t *err, int32_t code) {
    const int32_t had = atomicCAS(err, 0, code);
    if (had != 0 && !(had & DERR_TIMEOUT)) atomicCAS(err, had, code);
}

// (The timer is read from the 256th retry on.)
PKV_DEV bool lwait(uint64_t *bar, uint32_t parity, LMisc *m, const LatentParams &p, int where) {
    uint64_t t0 = 0;
    for (uint32_t it = 0;; ++it) {
        if (p.wait.quick ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity)) return true;
        if ((it & p.wait.check_mask) != p.wait.check_mask) continue;
        if (*reinterpret_cast<volatile int32_t *>(&m->abort_flag)) return false;
        const uint64_t now = global_timer_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > p.wait.limit_ns) {
            set_timeout(p.err, DERR_TIMEOUT | where);
            *reinterpret_cast<volatile int32_t *>(&m->abort_flag) = 1;
            return false;
        }
    }
}

// Lanes 0-15 of a warp's quarter: columns [col, col + n) to threads 0-15, [col + n, col + 2 n) to threads 16-31.
template <int NC>
PKV_DEV void tmem_ld_split(uint32_t taddr, uint32_t *r) {
    if constexpr (NC == 16) {
        asm volatile(
            "tcgen05.ld.sync.aligned.16x32bx2.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
            "[%16], 16;"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
              "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
            : "r"(taddr));
    } else if constexpr (NC == 8) {
        asm volatile("tcgen05.ld.sync.aligned.16x32bx2.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8], 8;"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(taddr));
    } else {
        asm volatile("tcgen05.ld.sync.aligned.16x32bx2.x4.b32 {%0, %1, %2, %3}, [%4], 4;"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(taddr));
    }
}
PKV_DEV void tmem_ld8(uint32_t taddr, uint32_t *r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
PKV_DEV void tmem_ld16(uint32_t taddr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
template <int n>
PKV_DEV void tmem_ldn(uint32_t taddr, uint32_t *r) {
    if constexpr (n == 16) tmem_ld16(taddr, r);
    else tmem_ld8(taddr, r);
}
PKV_DEV void tmem_st8(uint32_t taddr, const uint32_t *r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
PKV_DEV void tma_load_2d(uint32_t dst, const CUtensorMap *map, int32_t c0, int32_t c1, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_u32(bar))
        : "memory");
}

// Arrives on bar when this thread's copies so far have landed (the barrier counts on the arrival).
PKV_DEV void cp_async_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// One lane of a converged warp.  (A branch on this issues a product every 24 cycles, one on lane == 0 every 47 and
// a predicate from it every 70, for the compiler knows only of this one that the lanes agree.)
PKV_DEV bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

PKV_DEV bool finite(uint32_t bits) { return (bits & 0x7F800000u) != 0x7F800000u; }
// whether one of eight bf16 values is an infinity or a NaN
PKV_DEV bool nonfinite8(const uint4 &v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) bad |= (w[i] & 0x7F80u) == 0x7F80u || (w[i] & 0x7F800000u) == 0x7F800000u;
    return bad;
}

// The sum, or the maximum, of each of a thread's NC values over its half-warp's 16 lanes: lane i of them gets that of
// column i mod NC.  Lanes halve what they hold at each step (15 shuffles for 16 values; 64 with every sum in every lane).
template <int NC, bool MAX>
PKV_DEV float reduce_keys(float (&v)[NC], int lane) {
    auto join = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
    int w = NC;
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) {
        if (w == 2 * d) {
#pragma unroll
            for (int i = 0; i < NC / 2; ++i) {
                if (i >= d) break;
                const float mine = lane & d ? v[i + d] : v[i], other = lane & d ? v[i] : v[i + d];
                v[i] = join(mine, __shfl_xor_sync(0xffffffffu, other, d));
            }
            w = d;
        } else {
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                if (i >= w) break;
                v[i] = join(v[i], __shfl_xor_sync(0xffffffffu, v[i], d));
            }
        }
    }
    return v[0];
}

// Where the range begins: its first request, how many of that request's tiles come before it, and
// its tiles.  Each thread takes a stretch of the batch (one request, up to 384); a scan over the threads' sums.
template <int N>
PKV_DEV void find_range(const LatentParams &p, LMisc *m, int range) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (p.batch + kLThreads - 1) / kLThreads;
    const int r0 = min(p.batch, (int)threadIdx.x * per), r1 = min(p.batch, r0 + per);
    auto cost = [&](const int4 &q) { return (int64_t)sets_of<N>(p, q) * tiles_of(q); };
    int4 q = make_int4(0, 0, 0, 0);
    int64_t own = 0;
    for (int r = r0; r < r1; ++r) {
        q = read_req(p, r, blockIdx.x == 0);
        own += cost(q);
    }
    int64_t incl = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += x;
    }
    if (lane == 31) m->scan[warp] = incl;
    if (threadIdx.x == 0) m->start_r = p.batch;
    __syncthreads();
    int64_t before = incl - own, total = 0;
#pragma unroll
    for (int w = 0; w < kLThreads / 32; ++w) {
        if (w < warp) before += m->scan[w];
        total += m->scan[w];
    }
    const int64_t each = max((int64_t)kLMinTiles, (total + p.ranges - 1) / p.ranges), t0 = (int64_t)range * each;
    if (threadIdx.x == 0) m->left = max((int64_t)0, min(each, total - t0));
    if (t0 >= before && t0 < before + own) {  // one thread, where there is work
        int64_t at = before;
        int r = r0;
        if (per > 1)
            for (; r < r1 - 1; ++r) {
                const int64_t c = cost(read_req(p, r, false));
                if (t0 < at + c) break;
                at += c;
            }
        m->start_r = r;
        m->start_off = t0 - at;
    }
    __syncthreads();
    if (per == 1) {
        const int at = (int)threadIdx.x - m->start_r;
        if (r0 < r1 && at >= 0 && at < kLCached) m->req[at] = q;
    } else if (threadIdx.x < kLCached && m->start_r + (int)threadIdx.x < p.batch) {
        m->req[threadIdx.x] = read_req(p, m->start_r + threadIdx.x, false);
    }
    __syncthreads();
}

template <int R, int N>
__global__ void __launch_bounds__(kLThreads, 1)
    latent_kernel(const LatentParams p, const __grid_constant__ CUtensorMap qmap) {
    using C = LCfg<R, N>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    LMisc *m = reinterpret_cast<LMisc *>(smem + C::kMiscOff);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = blockIdx.x % p.gs, range = blockIdx.x / p.gs;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) mbar_init(&m->full[s], 64);
        for (int s = 0; s < C::kStages * 4; ++s) mbar_init(&m->empty[s], 1);
        mbar_init(&m->qfull, 1);
        mbar_init(&m->qempty, 1);
        mbar_init(&m->sfull[0], 1);
        mbar_init(&m->sfull[1], 1);
        mbar_init(&m->pfull[0], kLSoftmax / 32);  // (two: a warp may be done with a tile before another is with the one before)
        mbar_init(&m->pfull[1], kLSoftmax / 32);
        mbar_init(&m->pvdone[0], 1);
        mbar_init(&m->pvdone[1], 1);
        mbar_init(&m->ofull, 1);
        mbar_init(&m->drain[0], 1);
        mbar_init(&m->drain[1], 1);
        m->abort_flag = 0;
        fence_mbar_init();
    }
    if (threadIdx.x < 2 * kLTile) m->zeroed[threadIdx.x / kLTile][threadIdx.x % kLTile] = 0;
    if (warp == 1) {
        tmem_alloc(&m->tmem_base, 512);
        tmem_relinquish();
    }
    if (warp == 0 && lane == 0) prefetch_tmap(&qmap);
    tc_fence_before();
    pdl_wait();
    pdl_trigger();
    find_range<N>(p, m, range);  // (its barriers cover the set-up above)
    tc_fence_after();
    const uint32_t tmem = m->tmem_base;
    LCursor cur = cursor_at<N>(p, m);
    LSeg s;

    if (warp < 2) {
        // ================= issuers: warp 0 of S, warp 1 of P V =================
        // A warp each, for neither's products may wait for the other's operands.  The whole warp runs the loop, one lane
        // issues.
        const bool leader = elect_one();
        bool ok = true;
        int n = 0, nq = 0;  // tiles; Q loads consumed
        if (warp == 0) {
            constexpr uint32_t idesc = idesc_bf16_f32(kLTile, N, 0, 0);
            const uint64_t rows = sdesc_sw128(sbase, 16, 1024), q = sdesc_sw128(sbase + C::kQOff, 16, 1024);
            while (ok && next_work<N>(p, m, cur, s, g)) {
                ok = __all_sync(0xffffffffu, lwait(&m->qfull, nq & 1, m, p, 1));
                for (int i = s.start(); ok && i < s.t1; ++i, ++n) {
                    // S's place is free: the P V of two tiles ago is done.  (Not merely its P written: the issuer of P V
                    // has then seen that, before the same barrier can pass its next phase.)
                    if (n >= 2) ok = __all_sync(0xffffffffu, lwait(&m->pvdone[n & 1], ((n >> 1) - 1) & 1, m, p, 2));
                    const int st = __shfl_sync(0xffffffffu, n % C::kStages, 0);
                    ok = __all_sync(0xffffffffu, ok && lwait(&m->full[st], (n / C::kStages) & 1, m, p, 3));
                    if (!ok) break;
                    fence_proxy_async_smem();  // the rows were written by ordinary copies
                    tc_fence_after();
                    const uint64_t k = rows + (uint32_t)(st * (C::kStage >> 4));
                    const uint32_t d = tmem + __shfl_sync(0xffffffffu, n & 1, 0) * 64;
                    if (leader) {
#pragma unroll
                        for (int ks = 0; ks < (R + 64) / 16; ++ks)
                            mma_ss(d, k + (((ks >> 2) * C::kBlk + (ks & 3) * 32) >> 4), q + (((ks >> 2) * C::kQBlk + (ks & 3) * 32) >> 4),
                                   idesc, ks > 0 ? 1u : 0u);
                        tc_commit(&m->sfull[n & 1]);
                        if (i + 1 == s.t1) tc_commit(&m->qempty);
                    }
                    __syncwarp();
                }
                ++nq;
            }
        } else {
            constexpr uint32_t idesc = idesc_bf16_f32(128, N, 1, 1);
            const uint64_t rows = sdesc_sw128(sbase, C::kBlk, 1024);
            while (ok && next_work<N>(p, m, cur, s, g)) {
                for (int i = s.start(); ok && i < s.t1; ++i, ++n) {
                    ok = __all_sync(0xffffffffu, lwait(&m->pfull[n & 1], (n >> 1) & 1, m, p, 4));
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t v = rows + (uint32_t)(__shfl_sync(0xffffffffu, n % C::kStages, 0) * (C::kStage >> 4));
                    const int st = __shfl_sync(0xffffffffu, n % C::kStages, 0);
                    const uint32_t more = __shfl_sync(0xffffffffu, i > s.start(), 0);
                    if (leader) {
                        // by 16 keys, whose rows are given back as they are done with
#pragma unroll
                        for (int kk = 0; kk < kLTile / 16; ++kk) {
#pragma unroll
                            for (int mb = 0; mb < R / 128; ++mb)
                                mma_ss(tmem + C::kColO + mb * N, v + ((2 * mb * C::kBlk + kk * 2048) >> 4),
                                       v + (((C::kBlocks - 1) * C::kBlk + kk * 2048) >> 4), idesc, kk > 0 ? 1u : more);
                            tc_commit(&m->empty[st * 4 + kk]);
                        }
                        tc_commit(&m->pvdone[n & 1]);
                        if (i + 1 == s.t1) tc_commit(&m->ofull);
                    }
                    __syncwarp();
                }
            }
        }
        if (leader) tc_commit(&m->drain[warp]);  // every product issued completes before tensor memory is freed
        mbar_wait(&m->drain[warp], 0);
        __syncwarp();
    } else if (warp < 4) {
        // ================= Q and rows =================
        // Each of the two warps has 32 keys of a tile, 16 by 16 as the product gives them back.  Four rows a copy, eight
        // lanes a 128-byte block of each, all blocks of a row after one another: asked for by groups of columns, so that an
        // S could start with the first, rows came out of DRAM in pieces of 256 bytes (64 ragged requests: 200 us instead of
        // 128).  TMA is no better here: boxes of 16 rows of a page 138 us, gathers of four rows 180 us.
        const int half = warp - 2, sub = lane >> 3;
        int tp = 0, nq = 0;
        bool ok = true;
        while (ok && next_work<N>(p, m, cur, s, g)) {
            if (half == 0) {
                if (nq > 0) ok = __all_sync(0xffffffffu, lwait(&m->qempty, (nq - 1) & 1, m, p, 5));
                if (!ok) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&m->qfull, C::kBlocks * C::kQBlk);
                    for (int b = 0; b < C::kBlocks; ++b)
                        tma_load_2d(sbase + C::kQOff + b * C::kQBlk, &qmap, b * 64, s.q_row0, &m->qfull);
                }
                ++nq;
            }
            const int32_t *row = p.table + (int64_t)s.row * p.stride;
            // the slot of this lane's key; beyond the keys that are seen, and for a slot outside the pool, -1: zeros
            auto slot_of = [&](int t) -> int32_t {
                const int k = t * kLTile + half * 32 + lane;
                if (t >= s.t1 || k >= s.vis) return -1;
                const int32_t x = table_slot(row, k, p.shift, p.num_slots);
                if (x >= 0 && x < p.num_slots) return x;
                set_error(p.err, DERR_SLOT_RANGE);
                return -1;
            };
            int32_t next = slot_of(s.t0);
            for (int i = s.start(); ok && i < s.t1; ++i, ++tp) {
                const int32_t mine = next;
                next = slot_of(i + 1);
                const int st = __shfl_sync(0xffffffffu, tp % C::kStages, 0);
                const uint16_t *src[8];
                uint32_t there = 0;  // bit j: row 4 j + sub has a slot
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int32_t at = __shfl_sync(0xffffffffu, mine, 4 * j + sub);
                    src[j] = p.pool + (int64_t)max(at, 0) * p.pool_stride + (lane & 7) * 8;
                    there |= at < 0 ? 0u : 1u << j;
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int quarter = half * 2 + i;
                    if (tp >= C::kStages)
                        ok = __all_sync(0xffffffffu, ok && lwait(&m->empty[st * 4 + quarter], (tp / C::kStages - 1) & 1, m, p, 6));
                    if (!ok) break;
#pragma unroll
                    for (int j = 4 * i; j < 4 * i + 4; ++j) {
                        const int r = 4 * j + sub;  // of the warp's 32; its chunks lie at chunk ^ r mod 8
                        const uint32_t dst = sbase + st * C::kStage + (half * 32 + r) * 128 + (((lane & 7) ^ (r & 7)) << 4);
#pragma unroll
                        for (int b = 0; b < C::kBlocks; ++b) cp_async_16(dst + b * C::kBlk, src[j] + b * 64, there >> j & 1u ? 16u : 0u);
                    }
                }
                if (!ok) break;
                cp_async_arrive(&m->full[st]);
            }
        }
        cp_async_commit();
        cp_async_wait<0>();  // every copy issued lands before the CTA leaves
        if (nq > 0) mbar_wait(&m->qfull, (nq - 1) & 1);
    } else if (warp >= 4) {
        // ================= softmax and output =================
        // Four warps, a quarter of tensor memory each, have half of the columns from S to the output: the two halves share
        // nothing but P's barrier.
        constexpr int NC = C::kCols, NH = N / 2;                   // columns of a thread, of a half
        const int wq = warp & 3, hf = (warp - 4) >> 2;
        const int k_in = wq * 16 + (lane & 15);                    // this thread's key in a tile
        const int c0 = hf * NH + (lane >> 4) * NC;                 // and its first column
        const uint32_t quarter = (uint32_t)(wq * 32) << 16;
        const int in_half = wq * 32 + lane, bar = kLBarHalf + hf;
        int n = 0, nseg = 0;                                       // tiles and pieces before this one
        bool ok = true;
        int32_t *units = p.units + range * 8;
        if (g == 0 && warp == 4 && lane == 0) units[0] = units[4] = -1;
        while (next_seg<N>(p, m, cur, s, g)) {
            const int slot_rec = s.first ? 0 : 1;
            if (g == 0 && warp == 4 && lane == 0 && !s.whole) {
                units[slot_rec * 4 + 1] = s.set;
                units[slot_rec * 4 + 2] = s.ends;
                units[slot_rec * 4] = s.r;
            }
            if (s.nrows <= 0) continue;
            // keys that each column sees; columns without a row see what the last row does
            if (in_half < NH) m->lim[hf * NH + in_half] = s.vis0 + (int32_t)((uint32_t)(s.row_lo + min(hf * NH + in_half, s.nrows - 1)) / (uint32_t)p.heads);
            const int lim_min = s.vis0 + (int32_t)((uint32_t)s.row_lo / (uint32_t)p.heads);
            if (in_half < NH) m->ref[hf * NH + in_half] = kLUnset;
            float ref[NC], l[NC];
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                ref[c] = kLUnset;
                l[c] = 0.f;
            }
            named_bar_sync(bar, kLSoftmax / 2);
            for (int i = s.start(); i < s.t1; ++i, ++n) {
                const int t = max(i, 0);
                const bool split = i < s.twice;  // weights in two parts: the first at i = -1, the second at 0
                ok = __all_sync(0xffffffffu, ok && lwait(&m->sfull[n & 1], (n >> 1) & 1, m, p, 7));
                uint32_t sv[NC];
                float x[NC];  // logits above their references
                uint32_t hidden = 0;
                bool odd_row = false;
                float most = -INFINITY;  // the largest logit above its reference
                if (ok) {
                    tc_fence_after();
                    tmem_ld_split<NC>(tmem + quarter + (n & 1) * 64 + hf * NH, sv);
                    tmem_ld_wait();
                    if ((t + 1) * kLTile > lim_min) {
#pragma unroll
                        for (int c = 0; c < NC; ++c) {
                            odd_row |= !finite(sv[c]);
                            if (t * kLTile + k_in >= m->lim[c0 + c]) {
                                hidden |= 1u << c;
                                sv[c] = __float_as_uint(-INFINITY);
                            }
                        }
                    }
                    // (not one fma: a reference is a rounded product, and among logits past 2^31 the difference from an
                    // unrounded one is more than a weight has room for)
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        sv[c] = __float_as_uint(__fmul_rn(__uint_as_float(sv[c]), p.scale_log2));
                        x[c] = __uint_as_float(sv[c]) - ref[c];
                        most = fmaxf(most, x[c]);
                    }
                }
                if (!named_bar_and(bar, kLSoftmax / 2, ok && !split && !(most > kLagL))) {
                    if (!named_bar_and(bar, kLSoftmax / 2, ok)) {
                        ok = false;
                        break;
                    }
                    if (!split || i < 0) {
                        // Raise to the tile's maxima the references that those pass.  Maxima over a warp's keys, a column
                        // a lane at the end; a thread a column joins the quarters; all read what concerns them.
#pragma unroll
                        for (int c = 0; c < NC; ++c) x[c] = __uint_as_float(sv[c]);
                        const float most_of = reduce_keys<NC, true>(x, lane);
                        if ((lane & 15) < NC) reinterpret_cast<float *>(&m->col[c0 + (lane & (NC - 1))])[wq] = most_of;
                        named_bar_sync(bar, kLSoftmax / 2);
                        if (in_half < NH) {
                            const int c = hf * NH + in_half;
                            const float4 y = m->col[c];
                            const float top = fmaxf(fmaxf(y.x, y.y), fmaxf(y.z, y.w)), had = m->ref[c];
                            const bool up = top > had + kLagL;  // (a column's references follow its own logits alone)
                            m->alpha[c] = up ? ex2(had - top) : 1.f;  // (0 where there was no reference, and l is)
                            if (up) m->ref[c] = top;
                        }
                        if (n > 0) ok = __all_sync(0xffffffffu, lwait(&m->pvdone[(n - 1) & 1], ((n - 1) >> 1) & 1, m, p, 8));
                        named_bar_sync(bar, kLSoftmax / 2);
#pragma unroll
                        for (int c = 0; c < NC; c += 4) {
                            const float4 f = *reinterpret_cast<const float4 *>(&m->alpha[c0 + c]), y = *reinterpret_cast<const float4 *>(&m->ref[c0 + c]);
                            const float fs[4] = {f.x, f.y, f.z, f.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                l[c + i] *= fs[i];
                                ref[c + i] = ys[i];
                                x[c + i] = __uint_as_float(sv[c + i]) - ys[i];
                            }
                        }
                        if (i > s.start() && ok) {
                            tc_fence_after();
#pragma unroll 1
                            for (int i = 0; i < R / 128 * (NH / 8); ++i) {
                                const int cc = hf * NH + i % (NH / 8) * 8;
                                const uint32_t at = tmem + quarter + C::kColO + i / (NH / 8) * N + cc;
                                uint32_t ov[8];
                                tmem_ld8(at, ov);
                                tmem_ld_wait();
#pragma unroll
                                for (int c = 0; c < 8; ++c) ov[c] = __float_as_uint(__uint_as_float(ov[c]) * m->alpha[cc + c]);
                                tmem_st8(at, ov);
                            }
                            tmem_st_wait();
                        }
                    }
                    if (split) {
                        // The part of a weight that its first 8 bits hold, or what is left (no less than 0): their logarithms,
                        // as exponents of what follows, which rounds the first back to itself.  (In this branch, so that the
                        // usual tile pays one predicate: 256 requests 207 us, 211 with a choice behind the exponential.)
#pragma unroll
                        for (int c = 0; c < NC; ++c) {
                            const float w = ex2(x[c]), first = __uint_as_float(__float_as_uint(w) & 0xFFFF0000u);
                            const bool few = m->lim[c0 + c] < kPreciseKeys;
                            if (few) x[c] = __log2f(i < 0 ? first : w - first);
                            else if (i == 0) x[c] = -INFINITY;
                        }
                    }
                }
                // weights, rounded to bf16 for the product; what they are divided by sums the rounded ones
                uint32_t pk[NC / 2];
#pragma unroll
                for (int c = 0; c < NC; c += 2)
                    pk[c / 2] = pack_bf16x2(ex2(x[c]), ex2(x[c + 1]));
                const int st = n % C::kStages;
                if (odd_row) {
                    // A latent with an infinity or a NaN that some columns may not see: a weight of 0 would not keep it
                    // from them.  It becomes zeros; the columns that see it get a weight of NaN.  (One under a logit of -inf and
                    // a finite latent, by an infinity in the rotary key, keeps its 0, as in a tile without hidden keys.)
                    lwait(&m->full[st], (n / C::kStages) & 1, m, p, 9);  // (long complete: the copies, seen by this thread)
                    uint8_t *at = smem + st * C::kStage + k_in * 128;
                    bool bad = false;
                    for (int b = 0; b < R / 64; ++b)
                        for (int j = 0; j < 8; ++j) bad |= nonfinite8(*reinterpret_cast<const uint4 *>(at + b * C::kBlk + j * 16));
                    // Four threads have a key.  One that finds zeros where another was first finds that one's mark behind them.
                    // (The halves are a tile apart at most: S of n + 2 waits for P V of n, and that for both.)
                    volatile int32_t *mark = &m->zeroed[n & 1][k_in];
                    __threadfence_block();
                    bad |= *mark == n + 1;
                    if (bad) {
                        *mark = n + 1;
                        __threadfence_block();
                        for (int b = 0; b < R / 64; ++b)
                            for (int j = 0; j < 8; ++j) *reinterpret_cast<uint4 *>(at + b * C::kBlk + j * 16) = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                        for (int c = 0; c < NC; ++c)
                            if (!((hidden >> c) & 1u)) pk[c / 2] |= 0x7FFFu << (16 * (c & 1));
                    }
                }
                {
                    uint8_t *row = smem + st * C::kStage + (C::kBlocks - 1) * C::kBlk + k_in * 128;
                    if constexpr (NC == 16) {
                        const int j = c0 / 8;
                        *reinterpret_cast<uint4 *>(row + ((j ^ (k_in & 7)) << 4)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                        *reinterpret_cast<uint4 *>(row + (((j + 1) ^ (k_in & 7)) << 4)) = make_uint4(pk[4], pk[5], pk[6], pk[7]);
                    } else if constexpr (NC == 8) {
                        *reinterpret_cast<uint4 *>(row + (((c0 / 8) ^ (k_in & 7)) << 4)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                    } else {
                        *reinterpret_cast<uint2 *>(row + (((c0 / 8) ^ (k_in & 7)) << 4) + (c0 & 4) * 2) = make_uint2(pk[0], pk[1]);
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&m->pfull[n & 1]);
#pragma unroll
                for (int c = 0; c < NC; c += 2) add_bf16x2_f32(pk[c / 2], l[c], l[c + 1]);
            }
            // the columns' sums, over a warp's keys and then the quarters (col and alpha may still be in use)
            const float part = reduce_keys<NC, false>(l, lane);
            named_bar_sync(bar, kLSoftmax / 2);
            if ((lane & 15) < NC) reinterpret_cast<float *>(&m->col[c0 + (lane & (NC - 1))])[wq] = part;
            const bool any = s.t1 > s.t0;
            if (any) ok = __all_sync(0xffffffffu, ok && lwait(&m->ofull, nseg & 1, m, p, 10));
            if (!named_bar_and(bar, kLSoftmax / 2, ok)) {
                ok = false;
                break;
            }
            if (any) ++nseg;
            tc_fence_after();
            const int64_t rec = ((int64_t)range * 2 + slot_rec) * p.gs + g;
            if (in_half < NH) {
                const int c = hf * NH + in_half;
                const float4 y = m->col[c];
                const float sum = (y.x + y.y) + (y.z + y.w);
                // (A sum of 0 over keys that were seen, all logits -inf, divides to NaN.)
                m->alpha[c] = !s.whole ? 1.f : m->lim[c] <= 0 ? 0.f : 1.f / sum;
                // a reference of -inf: no key of this piece was seen
                if (!s.whole)
                    reinterpret_cast<float2 *>(p.rec_ml)[rec * N + c] = make_float2(m->lim[c] <= s.t0 * kLTile ? -INFINITY : m->ref[c], sum);
            }
            named_bar_sync(bar, kLSoftmax / 2);
            if (!s.whole && !any) continue;  // its (-inf, 0) says that there is nothing to add
            constexpr int CH = NH < 16 ? NH : 16;  // columns at a time
            const int chunks = (min(s.nrows - hf * NH, NH) + CH - 1) / CH;
            const uint32_t trade = lane & 1 ? 0x3276u : 0x5410u;
            // (Few instructions: this code is run once a piece, and their fetch is what it costs.)
#pragma unroll 1
            for (int i = 0; i < chunks * (R / 128); ++i) {
                const int cc = hf * NH + i / (R / 128) * CH, mb = i % (R / 128);
                const int col = mb * 128 + wq * 32 + lane;  // this thread's latent element
                uint32_t ov[CH];
                if (any) {
                    tmem_ldn<CH>(tmem + quarter + C::kColO + mb * N + cc, ov);
                    tmem_ld_wait();
                } else {
#pragma unroll
                    for (int c = 0; c < CH; ++c) ov[c] = 0u;
                }
                const bool all = cc + CH <= s.nrows;
                if (!s.whole) {  // (the workspace has room for rows that are not there)
                    float *out = p.rec + (rec * N + cc) * R + col;
#pragma unroll
                    for (int c = 0; c < CH; ++c) out[c * R] = __uint_as_float(ov[c]);
                    continue;
                }
                uint32_t *out = reinterpret_cast<uint32_t *>(p.o + (int64_t)(s.q_row0 + cc + (lane & 1)) * R) + (col >> 1);
                const int rows = s.nrows - cc - (lane & 1);
#pragma unroll
                for (int c = 0; c < CH; c += 4) {
                    const float4 inv = *reinterpret_cast<const float4 *>(&m->alpha[cc + c]);
                    const uint32_t w[2] = {pack_bf16x2(__uint_as_float(ov[c]) * inv.x, __uint_as_float(ov[c + 1]) * inv.y),
                                           pack_bf16x2(__uint_as_float(ov[c + 2]) * inv.z, __uint_as_float(ov[c + 3]) * inv.w)};
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        // neighbouring lanes trade a value: even lanes write column c, odd ones c + 1, two elements each
                        const uint32_t y = __byte_perm(w[k], __shfl_xor_sync(0xffffffffu, w[k], 1), trade);
                        if (all || c + 2 * k < rows) out[(c + 2 * k) * (R / 2)] = y;
                    }
                }
            }
            tc_fence_before();
            // col, ref, alpha and lim are read before the next piece writes them
            named_bar_sync(bar, kLSoftmax / 2);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
    if (threadIdx.x == 0) p.units[range * 8 + 3 + 4 * g] = m->abort_flag;
}

// ------------------------------------------------------------------------------------------
// Joins the records of units that several ranges share.  A unit's pieces are range c's last record and the
// first records of the ranges behind it, up to the one in which it ends.  A row of a unit with up to 8 records is a
// warp's task; of one with more, 64 elements of a row are a CTA's.  A unit that reaches into a range that gave up is left
// out: records of it may be missing, or another call's.

struct LatentMerge {
    const float *rec, *rec_ml;
    const int32_t *units, *indptr;
    int32_t ranges, gs, heads, N;
    uint16_t *o;
};

// A record's factor under the common maximum; 0 where it saw nothing.  (Where it saw keys and none had a logit to raise the
// reference, only NaN and -inf, that is kLUnset still, below all others.)
PKV_DEV float weight_of(float2 ml, float M) { return ml.x == -INFINITY ? 0.f : ex2(ml.x - M); }

template <int R>
__global__ void __launch_bounds__(256, 4) latent_merge_kernel(const LatentMerge p) {
    constexpr int V = R / 128;  // float4s a lane
    constexpr int kFew = 8;
    __shared__ int4 s_first[kLMaxCtas], s_last[kLMaxCtas];    // the ranges' units, as they were written
    __shared__ int32_t s_unit[2][kLMaxCtas];                  // units of few records from one end, of many: range | records << 16
    __shared__ int32_t s_warp[2][8];
    __shared__ uint32_t s_ends[8];
    __shared__ float4 s_acc[16][16];
    __shared__ float s_w[kLMaxCtas], s_m[8], s_l[8];
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto gave_up = [&](int c) { return s_first[c].w != 0 || (p.gs == 2 && s_last[c].w != 0); };
    if ((int)threadIdx.x < p.ranges) {
        s_first[threadIdx.x] = ld(reinterpret_cast<const int4 *>(p.units) + threadIdx.x * 2);
        s_last[threadIdx.x] = ld(reinterpret_cast<const int4 *>(p.units) + threadIdx.x * 2 + 1);
    }
    const bool any_gave_up = __syncthreads_or((int)threadIdx.x < p.ranges && gave_up(threadIdx.x));
    // Two lists in the ranges' order: every CTA has the same.  A unit ends with the first range behind its own whose first
    // piece ends there.
    const uint32_t ends = __ballot_sync(0xffffffffu, (int)threadIdx.x < p.ranges && s_first[threadIdx.x].x >= 0 && s_first[threadIdx.x].z);
    if (lane == 0) s_ends[warp] = ends;
    __syncthreads();
    int n = 0;
    if ((int)threadIdx.x < p.ranges && s_last[threadIdx.x].x >= 0) {
        n = 1;
        const int from = threadIdx.x + 1;
        for (int w = from >> 5; w < 8 && n == 1; ++w) {
            const uint32_t bits = s_ends[w] & (w == from >> 5 ? 0xffffffffu << (from & 31) : 0xffffffffu);
            if (bits) n = w * 32 + __ffs(bits) - (int)threadIdx.x;
        }
        if (any_gave_up)
            for (int c = threadIdx.x, to = n == 1 ? p.ranges : c + n; c < to; ++c)
                if (gave_up(c)) n = 0;
    }
    const uint32_t few = __ballot_sync(0xffffffffu, n > 0 && n <= kFew), many = __ballot_sync(0xffffffffu, n > kFew);
    if (lane == 0) {
        s_warp[0][warp] = __popc(few);
        s_warp[1][warp] = __popc(many);
    }
    __syncthreads();
    int count[2] = {0, 0}, at_list = __popc((n > kFew ? many : few) & ((1u << lane) - 1));
    for (int w = 0; w < 8; ++w) {
        if (w < warp) at_list += s_warp[n > kFew][w];
        count[0] += s_warp[0][w];
        count[1] += s_warp[1][w];
    }
    if (n > 0) s_unit[n > kFew][at_list] = threadIdx.x | n << 16;
    __syncthreads();
    const int rows = p.N * p.gs;
    const float2 *ml = reinterpret_cast<const float2 *>(p.rec_ml);
    // where row `row` of a unit goes (-1: nowhere, the unit is shorter)
    auto out_of = [&](int c, int row) -> int64_t {
        const int32_t r = s_last[c].x, set = s_last[c].y;
        const int64_t q0 = p.indptr ? ld(p.indptr + r) : r, e = p.indptr ? ld(p.indptr + r + 1) - q0 : 1;
        const int64_t at = (int64_t)set * rows + row;
        return at < e * p.heads ? q0 * p.heads + at : -1;
    };

    for (int i = blockIdx.x * 8 + warp; i < count[0] * rows; i += gridDim.x * 8) {
        const int unit = i / rows, row = i - unit * rows, c = s_unit[0][unit] & 0xFFFF, cnt = s_unit[0][unit] >> 16;
        const int64_t out_row = out_of(c, row);
        if (out_row < 0) continue;
        const int gi = row / p.N, k = row - gi * p.N;
        auto rec_of = [&](int j) { return ((((int64_t)c + j) * 2 + (j == 0)) * p.gs + gi) * p.N + k; };
        const float2 mine = lane < cnt ? ld(ml + rec_of(lane)) : make_float2(-INFINITY, 0.f);
        float M = mine.x;
#pragma unroll
        for (int d = kFew / 2; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
        M = __shfl_sync(0xffffffffu, M, 0);
        const float weight = weight_of(mine, M);
        float4 acc[V];
        float L = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
        for (int j = 0; j < cnt; ++j) {
            const float w = __shfl_sync(0xffffffffu, weight, j);
            L = fmaf(w, __shfl_sync(0xffffffffu, mine.y, j), L);
            // Nothing was seen there, and nothing written.  (Not by a weight of 0: a NaN stays one.)
            if (__shfl_sync(0xffffffffu, mine.x, j) == -INFINITY) continue;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float4 y = ld(reinterpret_cast<const float4 *>(p.rec + rec_of(j) * R) + v * 32 + lane);
                acc[v] = make_float4(fmaf(w, y.x, acc[v].x), fmaf(w, y.y, acc[v].y), fmaf(w, y.z, acc[v].z), fmaf(w, y.w, acc[v].w));
            }
        }
        const float inv = M == -INFINITY ? 0.f : 1.f / L;  // zeros where no record saw a key
        uint2 *out = reinterpret_cast<uint2 *>(p.o + out_row * R);
#pragma unroll
        for (int v = 0; v < V; ++v)
            out[v * 32 + lane] = make_uint2(pack_bf16x2(acc[v].x * inv, acc[v].y * inv), pack_bf16x2(acc[v].z * inv, acc[v].w * inv));
    }

    // 64 elements of a row: 16 threads a record, the CTA's 16 records at a time
    constexpr int kChunks = R / 64;
    for (int i = blockIdx.x; i < count[1] * rows * kChunks; i += gridDim.x) {
        const int chunk = i % kChunks, task = i / kChunks, unit = task / rows, row = task - unit * rows;
        const int c = s_unit[1][unit] & 0xFFFF, cnt = s_unit[1][unit] >> 16;
        const int64_t out_row = out_of(c, row);
        if (out_row < 0) continue;  // (the same for the CTA)
        const int gi = row / p.N, k = row - gi * p.N;
        auto rec_of = [&](int j) { return ((((int64_t)c + j) * 2 + (j == 0)) * p.gs + gi) * p.N + k; };
        const float2 mine = (int)threadIdx.x < cnt ? ld(ml + rec_of(threadIdx.x)) : make_float2(-INFINITY, 0.f);
        float M = mine.x;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
        if (lane == 0) s_m[warp] = M;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < 8; ++w) M = fmaxf(M, s_m[w]);
        const float w = weight_of(mine, M);
        if ((int)threadIdx.x < cnt) s_w[threadIdx.x] = mine.x == -INFINITY ? -1.f : w;  // -1: nothing seen, nothing written
        float L = w * mine.y;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) L += __shfl_xor_sync(0xffffffffu, L, d);
        if (lane == 0) s_l[warp] = L;
        __syncthreads();
        const int part = threadIdx.x >> 4, at = threadIdx.x & 15;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        constexpr int kInFlight = 5;
        for (int j0 = part; j0 < cnt; j0 += 16 * kInFlight) {
            float4 y[kInFlight];
            float f[kInFlight];
#pragma unroll
            for (int u = 0; u < kInFlight; ++u) {
                const int j = j0 + 16 * u;
                f[u] = j < cnt ? s_w[j] : -1.f;
                y[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (!(f[u] < 0.f)) y[u] = ld(reinterpret_cast<const float4 *>(p.rec + rec_of(j) * R) + chunk * 16 + at);
            }
#pragma unroll
            for (int u = 0; u < kInFlight; ++u)
                acc = make_float4(fmaf(f[u], y[u].x, acc.x), fmaf(f[u], y[u].y, acc.y), fmaf(f[u], y[u].z, acc.z),
                                  fmaf(f[u], y[u].w, acc.w));
        }
        s_acc[part][at] = acc;
        __syncthreads();
        if (threadIdx.x < 16) {
            float sum = 0.f;
            acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                const float4 y = s_acc[v][threadIdx.x];
                acc = make_float4(acc.x + y.x, acc.y + y.y, acc.z + y.z, acc.w + y.w);
            }
#pragma unroll
            for (int v = 0; v < 8; ++v) sum += s_l[v];
            const float inv = M == -INFINITY ? 0.f : 1.f / sum;
            reinterpret_cast<uint2 *>(p.o + out_row * R)[chunk * 16 + threadIdx.x] =
                make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------------------------------

static int latent_ctas() { return std::min(num_sms(), kLMaxCtas) & ~1; }

// The workspace: header | the ranges' units | (m, l) of the records | records, two a CTA of 64 rows.
static size_t latent_bytes(int32_t r) {
    const size_t ctas = (size_t)latent_ctas();
    return kWorkspaceHeader + ctas * 32 + ctas * 2 * 64 * 8 + ctas * 2 * 64 * (size_t)r * 4;
}

template <int R, int N>
static int launch_latent(LatentParams p, const CUtensorMap &qmap, cudaStream_t s) {
    using C = LCfg<R, N>;
    static_assert(C::kSmem <= 232448, "shared memory");
    static std::atomic<uint64_t> allowed{0};  // devices on which the kernel may use that much
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return PKV_E_CUDA;
    if (dev >= 64 || !((allowed.load(std::memory_order_relaxed) >> dev) & 1)) {
        if (cudaFuncSetAttribute(latent_kernel<R, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess)
            return PKV_E_CUDA;
        if (dev < 64) allowed.fetch_or((uint64_t)1 << dev, std::memory_order_relaxed);
    }
    if (launch_pdl(latent_kernel<R, N>, dim3((unsigned)(p.ranges * p.gs)), dim3(kLThreads), C::kSmem, s, true, p, qmap) != cudaSuccess)
        return PKV_E_CUDA;
    LatentMerge mp{p.rec, p.rec_ml, p.units, p.indptr, p.ranges, p.gs, p.heads, N, p.o};
    return launch_pdl(latent_merge_kernel<R>, dim3((unsigned)(4 * num_sms())), dim3(256), 0, s, true, mp) == cudaSuccess ? PKV_OK
                                                                                                                        : PKV_E_CUDA;
}

}  // namespace pkv

extern "C" int pkv_latent_workspace(const pkv_latent_pool *pool, int32_t num_heads, size_t *bytes) {
    using namespace pkv;
    const int rc = validate_latent_pool(pool);
    if (rc) return rc;
    if (num_heads <= 0 || !bytes) return PKV_E_INVALID;
    if (num_heads > 1024) return PKV_E_UNSUPPORTED;
    *bytes = latent_bytes(pool->latent_dim);
    return PKV_OK;
}

extern "C" int pkv_attn_latent(const pkv_latent_pool *pool, const pkv_batch *batch, const void *q, void *o, int64_t total_q,
                               const int32_t *qo_indptr, int32_t num_heads, float sm_scale, void *workspace, size_t ws_bytes,
                               void *stream) {
    using namespace pkv;
    const int rc = validate_latent_pool(pool);
    if (rc) return rc;
    if (!batch || batch->batch < 0 || num_heads <= 0 || total_q < 0) return PKV_E_INVALID;
    if (num_heads > 1024 || total_q * num_heads >= ((int64_t)1 << 31)) return PKV_E_UNSUPPORTED;
    if (!(sm_scale > 0.f) || !std::isfinite(sm_scale)) return PKV_E_INVALID;
    if (!qo_indptr && total_q != batch->batch) return PKV_E_INVALID;
    if (batch->batch == 0 || total_q == 0) return PKV_OK;
    if (!batch->req_to_token || !batch->req_pool_indices || !batch->seq_lens || !q || !o || !workspace) return PKV_E_INVALID;
    const int shift = page_shift_of(batch);
    if (shift < 0 || batch->stride < 0 || batch->stride >= ((int64_t)1 << 31) || batch->num_rows < 0) return PKV_E_INVALID;
    if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(o)) & 15) return PKV_E_INVALID;
    if (reinterpret_cast<uintptr_t>(workspace) & 255) return PKV_E_INVALID;
    if (ws_bytes < latent_bytes(pool->latent_dim)) return PKV_E_WORKSPACE;

    // Rows a CTA: the smallest N that holds an average request's, for a tile's products take the longer the wider
    // they are: one request of 100,001 latents and 16 rows takes 34.3 us at N = 16, 35.7 at 32 and 36.6 at 64, 64
    // ragged ones of 32 rows 113.9 at 32 and 120.3 at 64.  Past 64 rows two CTAs share a range, so that the second
    // finds it in L2: 32 requests of 7,000..8,000 latents and 256 rows take 183 us, 210 with a range to each.  (Any N and
    // either grouping is right for any batch.)
    const int64_t rows = (total_q + batch->batch - 1) / batch->batch * num_heads;
    const int N = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
    LatentParams p{};
    p.table = batch->req_to_token;
    p.stride = batch->stride;
    p.num_rows = batch->num_rows;
    p.shift = shift;
    p.rows = batch->req_pool_indices;
    p.lens = batch->seq_lens;
    p.indptr = qo_indptr;
    p.batch = batch->batch;
    p.heads = num_heads;
    p.total_q = total_q;
    p.num_slots = pool->num_slots;
    p.pool = static_cast<const uint16_t *>(pool->rows);
    p.pool_stride = latent_stride(pool);
    p.o = static_cast<uint16_t *>(o);
    p.scale_log2 = sm_scale * kLog2eL;
    p.gs = rows > 64 ? 2 : 1;
    p.ranges = latent_ctas() / p.gs;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.err = reinterpret_cast<int32_t *>(ws);
    p.units = reinterpret_cast<int32_t *>(ws + kWorkspaceHeader);
    p.rec_ml = reinterpret_cast<float *>(ws + kWorkspaceHeader + (size_t)latent_ctas() * 32);
    p.rec = p.rec_ml + (size_t)latent_ctas() * 2 * 64 * 2;
    p.wait = wait_policy(wait_limit_ns());

    const int32_t R = pool->latent_dim, row = R + pool->rope_dim;
    CUtensorMap qmap;
    const cuuint64_t dims[2] = {(cuuint64_t)row, (cuuint64_t)(total_q * num_heads)}, strides[1] = {(cuuint64_t)row * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)N};
    if (encode_tiled(&qmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(q), dims, strides, box,
                     CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
        return PKV_E_CUDA;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (R == 512)
        return N == 16 ? launch_latent<512, 16>(p, qmap, s)
                       : N == 32 ? launch_latent<512, 32>(p, qmap, s) : launch_latent<512, 64>(p, qmap, s);
    return N == 16 ? launch_latent<256, 16>(p, qmap, s)
                   : N == 32 ? launch_latent<256, 32>(p, qmap, s) : launch_latent<256, 64>(p, qmap, s);
}
