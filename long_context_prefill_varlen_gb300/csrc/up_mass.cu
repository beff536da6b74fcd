// up_kv_mass: the attention weight that every cached row has had, added up step by step: what a cache that takes rows out by
// their weight goes by (up_kv_evict).  The cache is the one that Eqs. 16-17 of "UniPrefill: Universal Long-Context Prefill
// Acceleration via Block-wise Dynamic Sparsification" (arXiv 2605.06221) give slots and lengths to; the records are
// this library's own.
//
// After up_paged_decode has found a step's lse, a row's weight needs no other row:
//   mass_i <- decay mass_i + sum_h exp(q_h . K_i sm_scale - lse_h),
// so the keys are read once more and nothing is joined: 2 dk (dk + 1) bytes a row in bf16 (e4m3) and 8 of records,
// which HBM bounds.  A warp takes its equal share of all requests' tiles of 16 rows, one after another, through a ring of its
// own in shared memory (copies that need no registers and no other warp).  Lane 4g + t copies, and reads back, 16-byte pieces
// t, t + 4, ... of rows g and g + 8: they are the products' first operand as they come if the queries' columns are taken in
// the same order (a sum over columns does not care), in m16n8k16 with keys in the 16 rows and query heads in the 8 columns.
// Beyond 8 query heads a key head the share is a CTA's, whose warps take a tile each and have the queries in common.
//
// Measured (one GB300, 6.79 TB/s measured copy): 16 requests of 4K-128K, 8 heads of 128 in bf16, 225 us, 6.4 TB/s; 64 of 0-8K, 8
// heads of 128 in e4m3, 58 us, 5.3 TB/s; 32 of up to 16K, 8 heads of 256 in bf16 112 us (6.2), in e4m3 63 us (5.6); 32 of up to
// 32K, 32 query heads on one of 128 in bf16, 22 us (3.9 TB/s; DRAM 44% and issue slots 47% busy, 16 warps an SM: the chain of a tile of
// 8 heads, its queries from shared memory, products, exponentials, and only then the next tile).  One request of 4K takes 4.6 us in a
// replayed graph (11 called from Python), a chain of latencies (its length, its pages, the copies).
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "up_kv.cuh"

namespace up {
namespace mass {

using kv::Cache;
using kv::FastDiv;

constexpr int kWarps = 4, kThreads = 32 * kWarps;

struct Args {
    const uint8_t* q;
    int64_t q_stride;          // bytes
    Cache c;
    const int32_t* table;
    const int32_t* seqused;
    const int32_t* counted;
    const int32_t* total;
    const float* lse;
    const float* mass;
    float* out;
    int32_t* born;
    int64_t records;
    int R, max_blocks, Hq, group;
    float scale_hi, scale_lo;  // sm_scale * log2 e, in two parts of one sign
    float decay;
    FastDiv by_b;
    int32_t* status;
};

constexpr int kRows = 16;      // of a tile

template <int DK, bool E4M3, bool MANY>
struct Shape {
    static constexpr int kRowBytes = DK * (E4M3 ? 1 : 2);
    static constexpr int kPieces = kRowBytes / 64;                     // 16-byte pieces of a row that a lane copies
    static constexpr int kKeys = kRows * kRowBytes;
    static constexpr int kStage = kKeys + 128 * (E4M3 ? 3 : 1);        // and a word a lane: its record's mass, its rows' scales
    // Two tiles in flight a warp and five CTAs an SM (20 warps of 96 registers) against three tiles: 64 requests of 0-8K in
    // e4m3 58 / 59 us, 32 of up to 16K on heads of 256 63 / 77; against six CTAs (80 registers, spills): 58 / 62.
    static constexpr int kStages = 2;
    static constexpr int kBlock = 4;                                   // tiles of 8 query heads that a CTA keeps in shared memory
    static constexpr int kTile = (DK / 8 + 8) * 128;                   // bytes of such a tile: the lanes' operands and factors
    static constexpr int kRings = kWarps * kStages * kStage;
    static constexpr int kSmem = kRings + (MANY ? kBlock * kTile : 0);
    static constexpr int kFit = 224 * 1024 / (kSmem + 1024);
    static constexpr int kMost = DK == 256 ? 4 : 5;
    static constexpr int kCtas = kFit < kMost ? kFit : kMost;
};

template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float low_of(uint32_t bf2) { return __uint_as_float(bf2 << 16); }
__device__ __forceinline__ float high_of(uint32_t bf2) { return __uint_as_float(bf2 & 0xffff0000u); }

// The queries of a tile of 8 heads as a lane's second operands, and what turns its sums into log2 weights.
template <int DK, bool E4M3>
struct Queries {
    static constexpr int KS = DK / 16, V = (2 * KS + 8) / 4;
    uint32_t b[KS][2];         // head g of the tile, the columns of the lane's pieces
    float hi[2], lo[2];        // factors of heads 2t, 2t + 1 (in two parts)
    float ref_hi[2], ref_lo[2];        // and their lse in log2; infinite: nothing to add

    __device__ __forceinline__ void load(const Args& a, int r, int head, int h0) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, heads = a.group - h0;
        const uint8_t* row = a.q + r * a.q_stride + (int64_t)(head * a.group + h0 + g) * DK * 2;
        // piece p: 8 numbers from column 32p + 8t (bf16), 16 from 64p + 16t (e4m3)
#pragma unroll
        for (int i = 0; i < KS / 2; ++i) {
            const int col = E4M3 ? 64 * (i / 2) + 16 * t + 8 * (i & 1) : 32 * i + 8 * t;
            const uint4 x = g < heads ? *reinterpret_cast<const uint4*>(row + 2 * col) : make_uint4(0, 0, 0, 0);
            b[2 * i][0] = x.x, b[2 * i][1] = x.y, b[2 * i + 1][0] = x.z, b[2 * i + 1][1] = x.w;
        }
        float back[2] = {1.f, 1.f};
        if constexpr (E4M3) {
            // e4m3 codes are exact in f16, and so are the queries once their largest is in [2^14, 2^15) (numbers 2^-29
            // and less of it lose bits far below an fp32 sum's)
            uint32_t m = 0;
#pragma unroll
            for (int k = 0; k < KS; ++k) m = __vmaxu2(m, __vmaxu2(b[k][0] & 0x7fff7fffu, b[k][1] & 0x7fff7fffu));
            m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
            const int e = static_cast<int>(max(m & 0xffffu, m >> 16) >> 7), up = min(268 - e, 253);
            const float f = __uint_as_float(static_cast<uint32_t>(up) << 23), inv = __uint_as_float(static_cast<uint32_t>(254 - up) << 23);
            back[0] = __shfl_sync(0xffffffffu, inv, 8 * t);
            back[1] = __shfl_sync(0xffffffffu, inv, 8 * t + 4);
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int j = 0; j < 2; ++j) b[k][j] = f16x2(low_of(b[k][j]) * f, high_of(b[k][j]) * f);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int h = 2 * t + x;
            const float l = h < heads ? a.lse[(int64_t)r * a.Hq + head * a.group + h0 + h] : INFINITY;
            // lse * log2 e to about 48 bits: fp32 alone would leave 2^-24 |lse| of a weight's exponent
            ref_hi[x] = fabsf(l) < INFINITY ? l * 1.44269502f : fabsf(l);
            ref_lo[x] = fabsf(l) < INFINITY ? fmaf(l, 1.44269502f, -ref_hi[x]) + l * 1.92596303e-8f : 0.f;
            hi[x] = a.scale_hi * back[x];
            lo[x] = a.scale_lo * back[x];
        }
    }
    // to and from a place in shared memory
    __device__ __forceinline__ void put(uint8_t* at) const {
        uint32_t w[4 * V];
#pragma unroll
        for (int k = 0; k < KS; ++k) w[2 * k] = b[k][0], w[2 * k + 1] = b[k][1];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            w[2 * KS + x] = __float_as_uint(hi[x]), w[2 * KS + 2 + x] = __float_as_uint(lo[x]);
            w[2 * KS + 4 + x] = __float_as_uint(ref_hi[x]), w[2 * KS + 6 + x] = __float_as_uint(ref_lo[x]);
        }
#pragma unroll
        for (int v = 0; v < V; ++v)
            reinterpret_cast<uint4*>(at)[v * 32 + (threadIdx.x & 31)] = make_uint4(w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
    }
    __device__ __forceinline__ void get(const uint8_t* at) {
        uint32_t w[4 * V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const uint4 x = reinterpret_cast<const uint4*>(at)[v * 32 + (threadIdx.x & 31)];
            w[4 * v] = x.x, w[4 * v + 1] = x.y, w[4 * v + 2] = x.z, w[4 * v + 3] = x.w;
        }
#pragma unroll
        for (int k = 0; k < KS; ++k) b[k][0] = w[2 * k], b[k][1] = w[2 * k + 1];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            hi[x] = __uint_as_float(w[2 * KS + x]), lo[x] = __uint_as_float(w[2 * KS + 2 + x]);
            ref_hi[x] = __uint_as_float(w[2 * KS + 4 + x]), ref_lo[x] = __uint_as_float(w[2 * KS + 6 + x]);
        }
    }
};

// A run of units: of all requests' units in the order request, head, rows, an equal share.  A unit is a tile of rows and the run
// a warp's, or with many query heads a tile for every warp of a CTA, which share the queries.
template <int UNIT>
struct Walk {
    int r, head, unit, units;      // units: of the request's head
    int len, from;                 // rows of the request; the first new one
    int left;                      // units of the run still to come

    __device__ __forceinline__ int units_of(const Args& a, int n) const {
        return n < 0 || n > (int64_t)a.max_blocks * static_cast<int64_t>(a.by_b.d) ? 0 : (n + UNIT - 1) / UNIT;
    }
    // the units of request r, its length reported if it is none
    __device__ __forceinline__ int look(const Args& a, int r, int* n) const {
        *n = r < a.R && UP_IN(r, a.R, a.status) ? a.seqused[r] : 0;
        const int u = units_of(a, *n);
        if (u == 0 && *n != 0) set_status(a.status, UP_DEV_BAD_LENGTH);
        return u;
    }
    // x and those of the lanes before
    template <typename T>
    static __device__ __forceinline__ T upto(T x) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const T y = __shfl_up_sync(0xffffffffu, x, o);
            if ((threadIdx.x & 31) >= o) x += y;
        }
        return x;
    }
    __device__ __forceinline__ void seek(const Args& a, int64_t run, int64_t runs) {
        const int lane = threadIdx.x & 31, per = (a.R + 31) / 32;      // requests of a lane, side by side
        left = 0;
        int n = 0;
        int64_t mine = 0;
#pragma unroll 4
        for (int i = 0; i < per; ++i) mine += look(a, lane * per + i, &n);
        const int64_t sum = upto(mine), all = __shfl_sync(0xffffffffu, sum, 31) * a.c.Hkv;
        if (all == 0) return;
        int64_t first;
        if (all <= runs) {                             // few units: one each, to runs that lie evenly over the grid
            const int64_t apart = runs / all;
            first = run % apart == 0 && run / apart < all ? run / apart : all;
            left = first < all ? 1 : 0;
        } else {
            first = all * run / runs;
            left = static_cast<int>(all * (run + 1) / runs - first);
        }
        if (left == 0) return;
        // the lane whose requests the run starts in, and of those the one
        const int l = __ffs(__ballot_sync(0xffffffffu, sum * a.c.Hkv > first)) - 1;
        int64_t before = __shfl_sync(0xffffffffu, sum - mine, l);
        r = l * per;
        if (per == 1) {
            len = __shfl_sync(0xffffffffu, n, l);
            units = __shfl_sync(0xffffffffu, static_cast<int>(mine), l);
        } else {
            for (int i0 = 0;; i0 += 32) {              // (some request of the lane's is the one)
                const int u = i0 + lane < per ? look(a, l * per + i0 + lane, &n) : 0, to = upto(u);
                const uint32_t hit = __ballot_sync(0xffffffffu, (before + to) * a.c.Hkv > first);
                const int at = hit ? __ffs(hit) - 1 : 31;
                before += __shfl_sync(0xffffffffu, hit ? to - u : to, at);
                len = __shfl_sync(0xffffffffu, n, at);
                units = __shfl_sync(0xffffffffu, u, at);
                r = l * per + i0 + at;
                if (hit || i0 + 32 >= per) break;
            }
        }
        const int64_t at = first - before * a.c.Hkv;
        head = static_cast<int>(at / units);
        unit = static_cast<int>(at - (int64_t)head * units);
        from = a.counted ? a.counted[r] : len;
    }
    // n units on, no further than to the end of the request's head; true where that is another head's
    __device__ __forceinline__ bool skip(const Args& a, int n) {
        left -= n;
        unit += n;
        if (left == 0 || unit < units) return false;
        unit = 0;
        if (++head < a.c.Hkv) return true;
        head = 0;
        do {
            ++r;
            len = UP_IN(r, a.R, a.status) ? a.seqused[r] : 0;
            units = units_of(a, len);
        } while (units == 0);                          // a unit is left, so a request with one follows
        from = a.counted ? a.counted[r] : len;
        return true;
    }
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void end_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_groups() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Where a warp's tiles ahead lie, found by the lanes side by side: a tile of 16 rows lies in one page (WHOLE, pages of a
// multiple of 16), and a lane finds a tile's; or each row has its own, and a lane finds a row's.  The table's entries are
// read a batch ahead.
template <int UNIT, bool WHOLE>
struct Batch {
    static constexpr int kTiles = WHOLE ? 32 : 2;
    int sub;                   // the warp's first row in a unit
    Walk<UNIT> next;           // the batch after this one
    int next_n, page;
    int n, i, p0;              // tiles of this one, those used, and its first row
    int len, from;             // rows of its request, and those whose mass counts
    int64_t row, rec, sc;      // of the lane's tile (row): bytes, record, scale byte
    uint32_t valid;            // bit i: lane i's tile (row) has a record

    static __device__ __forceinline__ int offset() {
        const int lane = threadIdx.x & 31;
        return WHOLE ? lane * UNIT : lane / kRows * UNIT + lane % kRows;
    }
    __device__ __forceinline__ void look(const Args& a) {
        const int lane = threadIdx.x & 31;
        next_n = next.left > 0 ? min(kTiles, min(next.units - next.unit, next.left)) : 0;
        const int pos = next.unit * UNIT + sub + offset();
        const int64_t e = (int64_t)next.r * a.max_blocks + div_of(pos, a.by_b);
        const bool wanted = (WHOLE ? lane < next_n : lane < kRows * next_n) && pos < next.len;
        page = wanted && UP_IN(e, (int64_t)a.R * a.max_blocks, a.status) ? a.table[e] : -1;
    }
    __device__ __forceinline__ void turn(const Args& a) {
        const int lane = threadIdx.x & 31;
        n = next_n;
        i = 0;
        p0 = next.unit * UNIT + sub, len = next.len, from = a.decay != 0.f ? next.from : 0;
        if (n == 0) return;
        const int pos = p0 + offset();
        const int tok = pos - static_cast<int>(div_of(pos, a.by_b) * a.by_b.d);
        const bool wanted = (WHOLE ? lane < n : lane < kRows * n) && pos < len, in = page >= 0 && page < a.c.num_blocks;
        if (wanted && !in) set_status(a.status, UP_DEV_BAD_PAGE);
        // what is nowhere copies rows that are there, and leaves no record
        const int64_t pg = wanted && in ? page : 0, ph = pg * a.c.Hkv + next.head;
        row = pg * a.c.sb + next.head * a.c.sh + tok * a.c.st;
        rec = ph * a.by_b.d + tok;
        sc = ph * a.c.Bp + tok;
        valid = __ballot_sync(0xffffffffu, wanted && in);
        next.skip(a, n);
        look(a);
    }
};

template <int DK, bool E4M3, bool MANY, bool WHOLE>
__global__ void __launch_bounds__(kThreads, (Shape<DK, E4M3, MANY>::kCtas)) mass_kernel(const __grid_constant__ Args a) {
    using S = Shape<DK, E4M3, MANY>;
    constexpr int NP = S::kPieces, NS = S::kStages, NB = S::kBlock, UNIT = MANY ? kWarps * kRows : kRows;
    extern __shared__ __align__(16) uint8_t smem[];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, warp = threadIdx.x >> 5;
    uint8_t* const ring = smem + warp * (NS * S::kStage);
    uint8_t* const tiles = smem + S::kRings;               // MANY: a block of tiles of queries
    const uint32_t dst = smem_u32(ring) + 16 * lane, dst4 = smem_u32(ring) + S::kKeys + 4 * lane;

    Batch<UNIT, WHOLE> ahead{};
    ahead.sub = MANY ? warp * kRows : 0;
    ahead.next.seek(a, MANY ? blockIdx.x : (int64_t)blockIdx.x * kWarps + warp, MANY ? gridDim.x : (int64_t)gridDim.x * kWarps);
    if (ahead.next.left == 0) return;
    Walk<UNIT> w = ahead.next;
    ahead.look(a);
    // What a lane keeps of a tile while its keys are on their way: the record that it writes, of row g (t = 0) or g + 8
    // (t = 1), -1 for none, and where its rows' scale bytes lie in their words.  Nothing that is loaded stays in registers: a
    // wait for an older tile's would be one for the newer tiles' as well (64 requests of 0-8K in e4m3: 86 -> 67 us).
    int64_t record[NS];
    uint32_t byte[NS][2];
    const int64_t own = 16 * t + (WHOLE ? g * a.c.st : 0);
    const uint8_t* const keys = a.c.k + own;
    const int64_t half = 8 * a.c.st;
    const auto copy = [&](int stage) {
        if (ahead.i == ahead.n) ahead.turn(a);
        if (ahead.i < ahead.n) {
            int64_t row[2], rec[2], sc[2];
            bool valid[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (WHOLE && j) {
                    row[j] = row[0] + half, rec[j] = rec[0] + 8, sc[j] = sc[0] + 8, valid[j] = valid[0];
                } else {
                    const int from = WHOLE ? ahead.i : ahead.i * kRows + 8 * j + g;
                    row[j] = __shfl_sync(0xffffffffu, ahead.row, from);
                    rec[j] = __shfl_sync(0xffffffffu, ahead.rec, from) + (WHOLE ? g : 0);
                    // pages of a multiple of 16 have as many scale bytes
                    sc[j] = WHOLE ? rec[j] : E4M3 ? __shfl_sync(0xffffffffu, ahead.sc, from) : 0;
                    valid[j] = ahead.valid >> from & 1;
                }
#pragma unroll
                for (int p = 0; p < NP; ++p)
                    if (UP_IN(own + row[j] + 64 * p, a.c.row_limit, a.status))
                        copy16(dst + stage * S::kStage + (j * NP + p) * 512, keys + row[j] + 64 * p);
                if constexpr (E4M3) {
                    byte[stage][j] = (WHOLE ? g : static_cast<uint32_t>(sc[j])) & 3;
                    if (UP_IN(sc[j], a.c.scale_limit, a.status))
                        copy4(dst4 + stage * S::kStage + 128 * (1 + j), a.c.ks + (sc[j] & ~int64_t{3}));
                }
            }
            const int pos = ahead.p0 + ahead.i * UNIT + 8 * t + g;
            const bool mine = t < 2 && (t ? valid[1] : valid[0]) && pos < ahead.len;
            const int64_t at = t ? rec[1] : rec[0];
            record[stage] = mine ? at : -1;
            const uint32_t word = dst4 + stage * S::kStage;
            if (mine && pos < ahead.from && UP_IN(at, a.records, a.status))
                copy4(word, a.mass + at);
            else
                asm volatile("st.shared.u32 [%0], %1;" ::"r"(word), "r"(0) : "memory");
            ++ahead.i;
        }
        end_group();
    };
#pragma unroll
    for (int i = 0; i < NS - 1; ++i) copy(i);
    Queries<DK, E4M3> q;
    const int blocks = (a.group + 8 * NB - 1) / (8 * NB);
    bool fresh = true;
    for (;;) {
#pragma unroll
        for (int stage = 0; stage < NS; ++stage) {         // unrolled: a stage's rows are registers
            if (w.left == 0) return;
            copy((stage + NS - 1) % NS);
            if (!MANY && fresh) q.load(a, w.r, w.head, 0);
            wait_groups<NS - 1>();
            const uint32_t* const words = reinterpret_cast<const uint32_t*>(ring + stage * S::kStage + S::kKeys) + lane;
            float scale[2] = {1.f, 1.f};
            if constexpr (E4M3)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t b = words[32 * (1 + j)] >> (8 * byte[stage][j]) & 0xffu;
                    scale[j] = __uint_as_float(max(b << 23, 0x00400000u));         // 2^(b - 127)
                }
            float sum[2] = {0.f, 0.f};
            for (int b = 0; b < (MANY ? blocks : 1); ++b) {
                const int here = MANY ? min(NB, (a.group - 8 * NB * b + 7) / 8) : 1;
                if (MANY && (fresh || blocks > 1)) {       // the warps have the same run, and meet here together
                    __syncthreads();
                    for (int i = warp; i < here; i += kWarps) {
                        q.load(a, w.r, w.head, 8 * (NB * b + i));
                        q.put(tiles + i * S::kTile);
                    }
                    __syncthreads();
                }
                for (int i = 0; i < here; ++i) {
                    if (MANY) q.get(tiles + i * S::kTile);
                    float d[2][4] = {};                    // in two parts, so that a product need not wait for the one before
#pragma unroll
                    for (int p = 0; p < NP; ++p) {
                        const uint4 y = *reinterpret_cast<const uint4*>(ring + stage * S::kStage + p * 512 + 16 * lane);
                        const uint4 z = *reinterpret_cast<const uint4*>(ring + stage * S::kStage + (NP + p) * 512 + 16 * lane);
                        const uint32_t u[4] = {y.x, y.y, y.z, y.w}, v[4] = {z.x, z.y, z.z, z.w};
                        if constexpr (E4M3) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                uint32_t a0, a1, a2, a3;
                                kv::e4m3x4_to_f16x4(u[k], a0, a2);
                                kv::e4m3x4_to_f16x4(v[k], a1, a3);
                                mma<true>(d[k & 1], a0, a1, a2, a3, q.b[4 * p + k][0], q.b[4 * p + k][1]);
                            }
                        } else {
#pragma unroll
                            for (int k = 0; k < 2; ++k)
                                mma<false>(d[k & 1], u[2 * k], v[2 * k], u[2 * k + 1], v[2 * k + 1], q.b[2 * p + k][0], q.b[2 * p + k][1]);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float y[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            // (the row's scale, a power of two, to the factors: a sum times it may pass the largest number)
                            const float z = d[0][2 * j + k] + d[1][2 * j + k], f = E4M3 ? scale[j] : 1.f;
                            const float e = fmaf(z, f * q.hi[k], -q.ref_hi[k]) + fmaf(z, f * q.lo[k], -q.ref_lo[k]);
                            y[k] = q.ref_hi[k] == INFINITY ? 0.f : ex2(e);
                        }
                        sum[j] += y[0] + y[1];
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 1);
                sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 2);
            }
            const int64_t at = record[stage];
            if (at >= 0 && UP_IN(at, a.records, a.status)) {
                const int pos = w.unit * UNIT + ahead.sub + 8 * t + g;
                a.out[at] = fmaf(a.decay, __uint_as_float(words[0]), t ? sum[1] : sum[0]);
                if (pos >= w.from) a.born[at] = (a.total ? a.total[w.r] : w.len) - w.len + pos;
            }
            fresh = w.skip(a, 1);
        }
    }
}

template <int DK, bool E4M3, bool MANY, bool WHOLE>
static cudaError_t launch_one(const Args& a, cudaStream_t st) {
    using S = Shape<DK, E4M3, MANY>;
    static DeviceSet done{0};
    const cudaError_t e = once_per_device(done, [] {
        return cudaFuncSetAttribute(mass_kernel<DK, E4M3, MANY, WHOLE>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    });
    if (e != cudaSuccess) return e;
    const int64_t units = (int64_t)a.R * a.c.Hkv * cdiv((int64_t)a.max_blocks * a.c.B, (MANY ? kWarps : 1) * kRows);
    const int64_t ctas = std::min<int64_t>(units, (int64_t)S::kCtas * num_sms());
    return launch_pdl(mass_kernel<DK, E4M3, MANY, WHOLE>, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), S::kSmem, st, a);
}

template <int DK, bool E4M3, bool MANY>
static cudaError_t launch(const Args& a, cudaStream_t st) {
    return a.c.B % kRows == 0 ? launch_one<DK, E4M3, MANY, true>(a, st) : launch_one<DK, E4M3, MANY, false>(a, st);
}

template <int DK>
static cudaError_t launch_dk(const Args& a, bool e4m3, cudaStream_t st) {
    if (a.group <= 8) return e4m3 ? launch<DK, true, false>(a, st) : launch<DK, false, false>(a, st);
    return e4m3 ? launch<DK, true, true>(a, st) : launch<DK, false, true>(a, st);
}

}  // namespace mass
}  // namespace up

using namespace up;

extern "C" up_status up_kv_mass(const uint16_t* q, int64_t q_stride, const up_kv_cache* cache, const int32_t* block_table,
                                const int32_t* seqused, const float* lse, int R, int max_blocks, int Hq, float sm_scale,
                                const int32_t* counted, const int32_t* total, float decay, const float* mass,
                                float* mass_out, int32_t* born, int32_t* dev_status, void* stream) {
    mass::Args a{};
    if (!q || !block_table || !seqused || !lse || !mass || !mass_out || !born || !dev_status) return UP_ERR_ARG;
    const up_status s = kv::check(cache, &a.c);
    if (s != UP_OK) return s;
    if (R <= 0 || max_blocks <= 0 || Hq <= 0 || !(sm_scale > -INFINITY && sm_scale < INFINITY)) return UP_ERR_ARG;
    if (!(decay >= 0.f && decay <= 1.f)) return UP_ERR_ARG;
    if (Hq % cache->Hkv || (int64_t)R * Hq > 0x7fffffff || (int64_t)max_blocks * cache->B > 0x7fffffff - 128) return UP_ERR_SHAPE;
    if (!aligned16(q) || q_stride % 8 || (R > 1 && q_stride < (int64_t)Hq * cache->dk)) return UP_ERR_SHAPE;
    a.q = reinterpret_cast<const uint8_t*>(q);
    a.q_stride = q_stride * 2;
    a.table = block_table;
    a.seqused = seqused;
    a.counted = counted;
    a.total = total;
    a.lse = lse;
    a.mass = mass;
    a.out = mass_out;
    a.born = born;
    a.records = cache->num_blocks * cache->Hkv * cache->B;
    a.R = R;
    a.max_blocks = max_blocks;
    a.Hq = Hq;
    a.group = Hq / cache->Hkv;
    // both parts of one sign, the second never zero: a score of -inf would be NaN with parts that pull apart
    const double scale = sm_scale * 1.4426950408889634;
    a.scale_hi = static_cast<float>(scale);
    if (fabs(static_cast<double>(a.scale_hi)) >= fabs(scale)) a.scale_hi = nextafterf(a.scale_hi, 0.f);
    a.scale_lo = static_cast<float>(scale - a.scale_hi);
    a.decay = decay;
    a.by_b = kv::fast_div(cache->B);
    a.status = dev_status;
    const bool e4m3 = cache->format == UP_KV_E4M3;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = cache->dk == 64    ? mass::launch_dk<64>(a, e4m3, st)
                          : cache->dk == 128 ? mass::launch_dk<128>(a, e4m3, st)
                                             : mass::launch_dk<256>(a, e4m3, st);
    if (e != cudaSuccess) return failed_launch();
    count_launch();
    return check_launch();
}
