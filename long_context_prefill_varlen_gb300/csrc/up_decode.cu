// up_paged_decode: attention of one new token per request over its pages of the key-value cache, with the
// lengths that the drop history leaves each layer (up_seqused, section 3.5, Eq. 17 of "UniPrefill:
// Universal Long-Context Prefill Acceleration via Block-wise Dynamic Sparsification", arXiv 2605.06221).
//
// The positions [lo, len) of a request are cut into tiles of up to kTile rows (whole pages, or equal parts of
// pages) and the tiles into chunks, by the request's own length alone.  Each (request, KV head, chunk)
// gives for each query head of the group
//   lse2 = log2 sum_i 2^(s_i)   and   o = sum_i 2^(s_i - lse2) v_i,   s_i = q . k_i * sm_scale * log2 e
// and the join adds the chunks in order: out = sum_c 2^(lse2_c - L) o_c, L = log2 sum_c 2^(lse2_c).
//
// A cached number is used once per query head of its group, so HBM bounds the call from the first
// thousand positions on: 2 dk (dk + 1) bytes a row in bf16 (e4m3).  split_kernel keeps enough copies in flight
// and the rest out of their way:
//  * persistent CTAs take runs of (request, head, chunk) items of equal length in tiles, found from seqused on the
//    device: the host never waits for a length;
//  * a producer warp walks the run, tells the consumers of each item and fills a ring of stages (the K and V
//    tile of one head) by TMA, a box or two per page, swizzled so that ldmatrix reads it without bank conflicts; the
//    ring runs across items, so a new item's first tiles are there when the last one's sums are written;
//  * four consumer warps take 16 keys of a tile each and need no barrier between tiles: each has its own
//    running maximum and sums, joined through the last stage when the item ends;
//  * a call in which every chunk that its tables have room for can have a CTA at once is one launch: the chunks of a
//    row are a cluster and join through its shared memory (one 4K request in a table of 4K: 9.9 -> 8.4 us, and one launch
//    less for the host).  The host knows no lengths, so the tables' width decides, not the requests' lengths.
// The products are m16n8k16 with the long side of each in the 16 rows: scores = keys x queries (16 keys, 8
// heads), outputs = values transposed x weights transposed (16 columns, 8 heads), so that a group of up to 8
// heads, and a second tile of 8 above that, leaves little of them empty.  The scores' own layout, transposed
// in the registers, is the weights' operand.  With up to 8 heads a group the copies bound the call and the products fill
// 12 to 16% of the tensor pipe, so a larger matrix unit has nothing to win.  Beyond 8 heads issue slots and not copies
// bound it (44% of what HBM would allow with 32 heads on one of 128 in bf16, 21% in e4m3): there keys and value columns
// as the 64 or 128 rows of a tcgen05 product, the heads its columns, could win; not built.
//
// Measured (one GB300, 6.69 TB/s measured copy): 64 requests of 32K, 8 heads of 256 in bf16, 2.44 ms, 7.0 TB/s;
// 16 of 4K-128K, 8 heads of 128 in bf16, 426 us, 6.6 TB/s; 4 of 128K, 2 heads of 256 in e4m3, 97 us, 5.6 TB/s;
// 64 of 0-8K, 8 heads of 128 in e4m3, 109 us, 5.3 TB/s.  With e4m3 half the bytes come with the same work per
// number: there the starts and ends of items and the join weigh 5 to 20%.  One request of 4K in a table of 4K takes
// 8.8 us, a chain of latencies (its length, its pages, the copies, four tiles, the join); its bytes would take 2.5 us.
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "up_kv.cuh"

namespace up {
namespace decode {

using kv::Cache;
using kv::FastDiv;

constexpr int kTile = 64;            // rows of a tile
constexpr int kWarps = 4;            // consumer warps, 16 rows of a tile each
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kMinTiles = 4;         // a chunk holds at least this many tiles, if the request has them, and twice
constexpr int kFewSplits = 16;       // as many beyond this many chunks
constexpr int kMaxTiles = 16;        // about as many tiles as a chunk holds, up to kMaxSplits chunks
constexpr int kMaxSplits = 640;
constexpr int kItems = 4;            // items that the producer may be ahead
constexpr int kScaleBytes = 512;     // room of a tile's scale bytes (keys or values) in a stage
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.f;        // a running maximum moves once a score passes it by this much (log2)
// The weights of e4m3 values go to the second product in f16: an eighth of the output's own rounding (two f16 parts cost 2
// to 8% of a call).  Their reference lies kLift below the largest, so that they reach 2^kLift, and
// 2^(kLift + kSlack) before it moves, of f16's 2^16: a weight keeps its 11 bits down to 2^(-14 - kLift) of the
// largest and has an error of 2^(-25 - kLift) below.
constexpr float kLift = 7.f, kTop = 32768.f;

// How the positions of a request fall into segments (a page, or seg rows of one), tiles of spt segments, and chunks
// of tiles.
struct Cut {
    int B, seg, segp, spp, spt;      // page; rows of a segment, and of its place in a tile; segments of a
                                     // page, of a tile.  Where spp > 1, segp = seg.
    int sc;                          // bytes of a copy of scale bytes: 16, or 8 where segments have 8 rows of a longer page
    int window, s0, most;            // s0: chunks that spread one request's heads evenly over the grid; at most
                                     // `most` times as many
    int max_splits;
    FastDiv by_b, by_spt, by_spp, by_segp, by_wave;    // by_wave: s0 * kMaxTiles
};

struct Range {
    int len, lo;                     // positions [lo, len)
    int seg0, seg1, tiles, splits;   // first and last segment; tiles from the first; chunks
};

// floor(x / f.d) on either side
__host__ __device__ __forceinline__ int divided(int x, const FastDiv& f) {
#ifdef __CUDA_ARCH__
    return static_cast<int>(div_of(static_cast<uint32_t>(x), f));
#else
    return x / static_cast<int>(f.d);
#endif
}

__host__ __device__ __forceinline__ int splits_of(int tiles, const Cut& c) {
    const int few = (tiles + kMinTiles - 1) / kMinTiles, fine = (tiles + 2 * kMinTiles - 1) / (2 * kMinTiles);
    const int want = few <= kFewSplits ? few : fine > kFewSplits ? fine : kFewSplits;
    if (want <= c.s0) return want;
    const int waves = divided(tiles + c.s0 * kMaxTiles - 1, c.by_wave);
    return c.s0 * (waves < c.most ? waves : c.most);
}

__device__ __forceinline__ Range range_of(const Cut& c, int len, int64_t cap) {
    Range r;
    r.len = len < 0 || len > cap ? 0 : len;
    r.lo = c.window > 0 && r.len > c.window ? r.len - c.window : 0;
    const int last = r.len > 0 ? r.len - 1 : 0;
    const int p0 = r.lo ? divided(r.lo, c.by_b) : 0, p1 = divided(last, c.by_b);
    r.seg0 = p0 * c.spp + divided(r.lo - p0 * c.B, c.by_segp);
    r.seg1 = p1 * c.spp + divided(last - p1 * c.B, c.by_segp);
    r.tiles = r.len > 0 ? divided(r.seg1 - r.seg0, c.by_spt) + 1 : 0;
    r.splits = 0;
    return r;
}

__device__ __forceinline__ int splits_of(const Cut& c, int len, int64_t cap) { return splits_of(range_of(c, len, cap).tiles, c); }

// 2^(x - m), and 0 for x = -inf whatever m is (m is the largest of a set that x belongs to; NaN stays)
__device__ __forceinline__ float weight(float x, float m) { return x == -INFINITY ? 0.f : ex2(x - m); }

struct Args {
    const uint8_t* q;
    int64_t q_stride;          // bytes
    Cache c;
    const int32_t* table;
    const int32_t* seqused;
    int R, max_blocks, Hq, group, head_tiles;
    FastDiv by_hq;
    int both;                  // one copy brings keys and values: see make_maps
    int pitch;                 // bytes from a segment's place in a stage to the next one's
    int k_at, v_at;            // and from it to its keys, its values: multiples of 1024
    float scale2;              // sm_scale * log2 e
    Cut cut;
    float* part_lse;           // [R, Hq, max_splits]
    float* part_o;             // [R, Hq, max_splits, dk]
    int64_t parts;             // R * Hq * max_splits
    uint16_t* out;
    float* lse;
    int32_t* status;
};

// The two forms of a call give the same bits, so where a product meets a sum the code says whether they round
// together: left to the compiler, each kernel could differ.

// ln of the sum 2^m l
__device__ __forceinline__ float natural(float m, float l) {
    return l == 0.f ? -INFINITY : __fmul_rn(__fadd_rn(m, log2f(l)), kLn2);
}

__device__ __forceinline__ int length_of(const Args& a, int r) { return UP_IN(r, a.R, a.status) ? a.seqused[r] : 0; }

// x / y of numbers that mostly fit 32 bits (a 64-bit division takes a third of a microsecond, here in the way of
// the first copy)
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {
    return (x | y) >> 32 ? x / y : static_cast<int64_t>(static_cast<uint32_t>(x) / static_cast<uint32_t>(y));
}

// ------------------------------------------------------------------------------------------------
// the walk over a CTA's run of items.  Item order: request, KV head, chunk, head tile (the tiles of queries that read
// the same keys follow one another: the second finds them in L2).

struct Walk {
    int r, head, ch, ht;       // request, KV head, chunk, head tile
    Range g;
    int q, rem, err;           // tiles = q * splits + rem: chunk ch starts at tile ch q + floor(ch rem / splits);
                               // err = ch rem mod splits
    int t0, n;                 // the item's first tile of the request, and its tiles
    int64_t start, end;        // tiles before the item, and where the run ends
    int next_len;

    // an item belongs to the run that its middle falls into
    __device__ __forceinline__ bool live(const Args& a) const { return r < a.R && 2 * start + n < 2 * end; }

    // chunk i, its rem i / splits and remainder given
    __device__ __forceinline__ void chunk(int i, int whole, int left) {
        ch = i;
        t0 = i * q + whole;
        err = left;
        n = q + (err + rem >= g.splits ? 1 : 0);
    }
    __device__ __forceinline__ void enter(const Args& a, int len) {
        g = range_of(a.cut, len, (int64_t)a.max_blocks * a.cut.B);
        g.splits = splits_of(g.tiles, a.cut);
        q = g.splits ? static_cast<int>(quotient(g.tiles, g.splits)) : 0;
        rem = g.tiles - q * g.splits;
        head = ht = 0;
        chunk(0, 0, 0);
        next_len = r + 1 < a.R ? length_of(a, r + 1) : 0;
    }
    __device__ __forceinline__ void next(const Args& a) {
        start += n;
        if (++ht < a.head_tiles) return;
        ht = 0;
        if (++ch < g.splits) {
            t0 += n;
            err += rem;
            if (err >= g.splits) err -= g.splits;
            n = q + (err + rem >= g.splits ? 1 : 0);
            return;
        }
        chunk(0, 0, 0);
        if (++head < a.c.Hkv) return;
        do {
            if (++r >= a.R) return;
            enter(a, next_len);
        } while (g.splits == 0);
    }
};

// the first item whose middle lies at or after `want` tiles: in request r, which starts at `before` of them
__device__ __forceinline__ void seek(const Args& a, Walk& w, int64_t want, int64_t end, int r, int64_t before, int len) {
    w.r = r;
    w.end = end;
    w.enter(a, len);
    const int64_t per_head = (int64_t)w.g.tiles * a.head_tiles;
    const int64_t local = want - before;
    w.head = static_cast<int>(quotient(local, per_head));
    const int i = max(0, static_cast<int>(quotient((local - w.head * per_head) * w.g.splits, per_head)) - 1);
    const int whole = static_cast<int>(quotient(i * w.rem, w.g.splits));
    w.chunk(i, whole, i * w.rem - whole * w.g.splits);
    w.start = before + w.head * per_head + (int64_t)w.t0 * a.head_tiles;
    while (w.r < a.R && 2 * w.start + w.n < 2 * want) w.next(a);
}

// The CTA's run, found by its producer: the tiles of all requests, then the items whose middles lie in the CTA's
// share.  Items stay whole, so a run is off by at most one, and equal items as many as CTAs (or a multiple) fall
// one (or that many) to each.  CTAs move equal tiles in unequal time (64 requests of 0-8K in e4m3: the slowest 25%
// above the mean), but what is left at the end has the memory to itself: handing out shorter runs by a ticket
// measured 1 to 13% slower.
__device__ __forceinline__ void find_run(const Args& a, Walk& w) {
    const int lane = threadIdx.x & 31;
    const int64_t cap = (int64_t)a.max_blocks * a.cut.B;
    const int units = a.c.Hkv * a.head_tiles;
    // 32 requests at a time: a lane's length, its tiles and the tiles up to it.  Up to 32 requests are read once.
    int len = 0, mine = 0, upto = 0;
    auto scan = [&](int r0) {
        len = r0 + lane < a.R ? length_of(a, r0 + lane) : 0;
        upto = mine = range_of(a.cut, len, cap).tiles;         // at most 2^26 a request
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
    };
    int64_t total = 0;
    for (int r0 = 0; r0 < a.R; r0 += 32) {
        scan(r0);
        total += __shfl_sync(0xffffffffu, upto, 31);
        if ((len < 0 || len > cap) && blockIdx.x == 0) set_status(a.status, UP_DEV_BAD_LENGTH);
    }
    total *= units;
    // neighbours in the order of runs are half a grid apart: a short list of items leaves no SM with two
    // before every SM has one
    const int n = gridDim.x, half = (n + 1) / 2, b = blockIdx.x;
    const int64_t at = b < half ? 2 * b : 2 * (b - half) + 1;
    const int64_t end = quotient(total * (at + 1), n), want = quotient(total * at, n);
    w.r = a.R;
    w.start = w.end = 0;
    if (want >= end) return;
    int64_t before = 0;        // tiles of the requests before
    for (int r0 = 0; r0 < a.R; r0 += 32) {
        if (a.R > 32) scan(r0);
        const uint32_t hit = __ballot_sync(0xffffffffu, before + (int64_t)upto * units > want);
        if (hit) {
            const int l = __ffs(hit) - 1;
            before += (int64_t)__shfl_sync(0xffffffffu, upto - mine, l) * units;
            seek(a, w, want, end, r0 + l, before, __shfl_sync(0xffffffffu, len, l));
            return;
        }
        before += (int64_t)__shfl_sync(0xffffffffu, upto, 31) * units;
    }
}

// A cluster's CTA has one item: chunk blockIdx.x of (head, head tile) blockIdx.y of request blockIdx.z, if the
// request has as many.
__device__ __forceinline__ void own_chunk(const Args& a, Walk& w) {
    const int64_t cap = (int64_t)a.max_blocks * a.cut.B;
    const int len = length_of(a, blockIdx.z), ch = blockIdx.x;
    if ((len < 0 || len > cap) && blockIdx.x == 0 && blockIdx.y == 0) set_status(a.status, UP_DEV_BAD_LENGTH);
    w.r = blockIdx.z;
    w.enter(a, len);
    w.start = 0;
    w.end = 0;
    if (ch >= w.g.splits) return;
    w.head = static_cast<int>(blockIdx.y) / a.head_tiles;
    w.ht = static_cast<int>(blockIdx.y) - w.head * a.head_tiles;
    const int whole = static_cast<int>(static_cast<unsigned>(ch * w.rem) / static_cast<unsigned>(w.g.splits));
    w.chunk(ch, whole, ch * w.rem - whole * w.g.splits);
    w.end = w.n;               // live once: next() moves the start to the end
}

// ------------------------------------------------------------------------------------------------
// tiles in shared memory

template <int DK, bool E4M3, int HT>
struct Shape {
    static constexpr int kRowBytes = DK * (E4M3 ? 1 : 2);
    static constexpr int kPanelBytes = kRowBytes < 128 ? kRowBytes : 128;      // a segment is panels of rows
    static constexpr int kPanels = kRowBytes / kPanelBytes;
    static constexpr int kTileBytes = kTile * kRowBytes;
    static constexpr int kStage = 2 * kTileBytes + (E4M3 ? 2 * kScaleBytes : 0);
    // As many CTAs on an SM as leave each a few stages (228 KB of shared memory, 1 KB of it per CTA reserved) and the
    // registers that its sums need: 16 warps have 128 a thread, 12 have 168, 8 have 255.
    static constexpr int kLdq = DK + (HT == 16 ? 8 : 0);               // numbers of a query's row
    static constexpr int kControl = 4 * HT * kLdq + 1536 + 1024;       // queries; items, barriers and the join's; alignment
    static constexpr int kWarpsFit = DK == 256 && (HT == 16 || !E4M3) ? 8 : DK == 256 || HT == 16 || (DK == 128 && !E4M3) ? 12 : 16;
    static constexpr int fit(int ctas) { return (228 * 1024 / ctas - 1024 - kControl) / kStage; }
    static constexpr int ctas(int c) { return c == 1 || (c * (kWarps + 1) <= kWarpsFit && fit(c) >= 3) ? c : ctas(c - 1); }
    static constexpr int kCtas = ctas(6);
    static constexpr int kStages = fit(kCtas) < 8 ? fit(kCtas) : 8;
};

// Byte offset of 16-byte column c of a panel's row that starts at byte `row` of a stage (1024-byte aligned):
// the TMA swizzle takes the address bits above the row into the column.
template <int PANEL>
__device__ __forceinline__ uint32_t swizzled(uint32_t row, int c) {
    if constexpr (PANEL == 128)
        return row + (((c & 7) ^ ((row >> 7) & 7)) << 4);
    else
        return row + ((c ^ ((row >> 7) & 3)) << 4);
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// d += a b: a 16 x 16, b 16 x 8, bf16 or f16 in, fp32 sums
template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
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
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float low_of(uint32_t bf2) { return __uint_as_float(bf2 << 16); }
__device__ __forceinline__ float high_of(uint32_t bf2) { return __uint_as_float(bf2 & 0xffff0000u); }
// 16 or 8 bytes to shared memory, and one arrival of this thread at `bar` once its copies so far have landed
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
// eight scale bytes of 1
__device__ __forceinline__ void ones8(uint32_t dst) {
    asm volatile("st.shared.v2.u32 [%0], {%1, %1};" ::"r"(dst), "r"(0x7f7f7f7fu) : "memory");
}
__device__ __forceinline__ void arrive_after_copies(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
// an 8 x 8 matrix of halves, a row per four lanes, transposed
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// ------------------------------------------------------------------------------------------------
// shared memory of a CTA: the stages, then this

// what the consumers are told of an item; n = 0: no more
struct Item {
    int r, head, ch, h0;                       // h0: first query head of its tile, in the group
    int t0, n, tiles, seg0;                    // its tiles, and the request's
    int lo, len, fresh, unused;                // fresh: its queries are not the last item's
};

template <int LDQ, int HT, int NS>
struct Control {
    alignas(16) uint16_t q[2][HT * LDQ];       // queries, double-buffered
    Item item[kItems];
    float m[kWarps][16], f[kWarps][16], l[kWarps][16];
    float lse[16];                             // of a cluster's chunk; its sums take the queries' place
    uint64_t full[NS], empty[NS], qfull[2], qempty[2], ifull[kItems], iempty[kItems], joined;
    int64_t tiles, queries;                    // copies that the producer issued: to the ring, to the two query slots
    int abort;
};

template <int DK>
constexpr int kLd = DK + 4;      // floats of a row in the join of the warps: heads 2t, 2t + 1 of four lanes fall 8 banks apart

template <int DK, bool E4M3, int HT>
struct Sizes {
    using S = Shape<DK, E4M3, HT>;
    static constexpr int kSmem = S::kStages * S::kStage + static_cast<int>(sizeof(Control<S::kLdq, HT, S::kStages>)) + 1024;
    static_assert(sizeof(Control<S::kLdq, HT, S::kStages>) + 1024 <= S::kControl, "room of the control block");
};

// ------------------------------------------------------------------------------------------------

// mbar_wait for a converged warp: one answer for all of its lanes.  Where one lane's time ran out no lane goes on, so that
// the warp's shuffles and votes stay whole.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    return __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity, abort_flag));
}

// A role whose wait runs out reports it, raises the CTA's flag and leaves at once, without another arrival: what it has
// not read must not be overwritten, and no barrier is armed twice.  The others follow at their next wait.
__device__ __forceinline__ void give_up(const Args& a) {
    if ((threadIdx.x & 31) == 0) set_status(a.status, UP_DEV_WAIT_TIMEOUT);
}

// Before the CTA of an aborted run goes: the copies in flight write its shared memory, so wait for them (again with a limit).
template <int LDQ, int HT, int NS>
__device__ __noinline__ void drain(Control<LDQ, HT, NS>& sh) {
    const uint64_t t0 = globaltimer_ns();
    const int64_t tiles = sh.tiles, queries = sh.queries;
    for (int64_t k = tiles < NS ? 0 : tiles - NS; k < tiles; ++k)
        while (!mbar_try_wait(smem_u32(&sh.full[k % NS]), (k / NS) & 1))
            if (globaltimer_ns() - t0 > kDrainLimitNs) return;
    for (int64_t k = queries < 2 ? 0 : queries - 2; k < queries; ++k)
        while (!mbar_try_wait(smem_u32(&sh.qfull[k % 2]), (k / 2) & 1))
            if (globaltimer_ns() - t0 > kDrainLimitNs) return;
}

template <int DK, bool E4M3, int HT, bool TEAM>
__device__ void produce(const Args& a, const CUtensorMap* kmap, const CUtensorMap* vmap, uint32_t ring,
                        Control<Shape<DK, E4M3, HT>::kLdq, HT, Shape<DK, E4M3, HT>::kStages>& sh) {
    using S = Shape<DK, E4M3, HT>;
    const int lane = threadIdx.x & 31;
    const Cut& c = a.cut;
    int slot = 0, qslot = 0, islot = 0;
    uint32_t phase = 0, qphase = 0, iphase = 0;
    int64_t tiles = 0, queries = 0;
    auto leave = [&](bool in_order) {
        if (!in_order) give_up(a);
        if (lane == 0) sh.tiles = tiles, sh.queries = queries;
    };
    const int per = (32 / c.spt) * c.spt, tiles_per = 32 / c.spt;      // table entries and tiles of a batch
    // the scale bytes that this lane copies: of which segment of the tile, and from which byte of its part of a page
    const int per_seg = (c.seg + 15) / 16, sc_seg = lane / per_seg, sc_part = (lane - sc_seg * per_seg) * 16;
    auto part_of = [&](int s) { return c.spp == 1 ? 0 : s - div_of(s, c.by_spp) * c.spp; };      // of its page

    Walk w;
    if constexpr (TEAM) own_chunk(a, w); else find_run(a, w);
    // the table entries of an item's segments, 32 (or the most that make whole tiles) at a time, one batch ahead
    auto fetch = [&](const Walk& x, int tile) {
        const int s = x.g.seg0 + (x.t0 + tile) * c.spt + lane;
        int page = -1;
        if (x.live(a) && tile < x.n && lane < per && s <= x.g.seg1) {
            const int64_t e = (int64_t)x.r * a.max_blocks + div_of(s, c.by_spp);
            page = UP_IN(e, (int64_t)a.R * a.max_blocks, a.status) ? a.table[e] : -1;
        }
        return page;
    };
    int first_pages = fetch(w, 0);
    int q_r = -1, q_head = -1, q_ht = -1;                               // whose queries were sent last
    while (w.live(a)) {
        const int head = w.head, h0 = w.ht * HT;
        const bool fresh_q = w.r != q_r || head != q_head || w.ht != q_ht;
        if (fresh_q) {
            q_r = w.r, q_head = head, q_ht = w.ht;
            const int heads = min(HT, a.group - h0);
            if (!warp_wait(&sh.qempty[qslot], qphase ^ 1, &sh.abort)) return leave(false);
            ++queries;
            const uint32_t bar = smem_u32(&sh.qfull[qslot]), dst = smem_u32(sh.q[qslot]);
            const uint8_t* src = a.q + w.r * a.q_stride + (int64_t)(head * a.group + h0) * DK * 2;
            if (lane == 0) mbar_arrive_expect_tx(bar, heads * DK * 2);
            // up to 8 rows by one copy, where eight would hold up the first tile's; more at a distance that spreads the
            // banks (32 requests of 0-32K with 32 heads on one of 128 in bf16: 106 -> 99 us)
            if (S::kLdq == DK) {
                if (lane == 0) bulk_load(dst, src, heads * DK * 2, bar);
            } else {
                __syncwarp();
                if (lane < heads) bulk_load(dst + lane * S::kLdq * 2, src + lane * DK * 2, DK * 2, bar);
            }
            if (++qslot == 2) qslot = 0, qphase ^= 1;
        }
        if (!warp_wait(&sh.iempty[islot], iphase ^ 1, &sh.abort)) return leave(false);
        if (lane == 0) {
            sh.item[islot] = Item{w.r, head, w.ch, h0, w.t0, w.n, w.g.tiles, w.g.seg0, w.g.lo, w.g.len, fresh_q, 0};
            mbar_arrive(smem_u32(&sh.ifull[islot]));
        }
        if (++islot == kItems) islot = 0, iphase ^= 1;
        const int n = w.n, t0 = w.t0, seg0 = w.g.seg0, seg1 = w.g.seg1;
        int pages = first_pages, pages_next = -1;
        for (int i = 0, j = 0; i < n; ++i, ++j) {
            if (j == tiles_per) {                                       // a new batch
                j = 0;
                pages = pages_next;
            }
            if (!warp_wait(&sh.empty[slot], phase ^ 1, &sh.abort)) return leave(false);
            // segments s0 .. s0 + ns - 1 of the request
            const int s0 = seg0 + (t0 + i) * c.spt, ns = min(c.spt, seg1 - s0 + 1);
            const uint32_t stage = ring + slot * S::kStage, bar = smem_u32(&sh.full[slot]);
            const uint32_t sc = stage + 2 * S::kTileBytes + c.sc * lane;
            int sc_page = -1, sc_from = 0;
            bool sc_mine = false;
            if constexpr (E4M3) {
                sc_page = __shfl_sync(0xffffffffu, pages, (j * c.spt + sc_seg) & 31);
                sc_from = part_of(s0 + sc_seg) * c.seg + sc_part;
                sc_mine = sc_seg < ns && sc_from < a.c.Bp;
                if (sc_mine && (sc_page < 0 || sc_page >= a.c.num_blocks)) {       // codes of zero, scale 1
                    for (int x = 0; x < c.sc; x += 8) {
                        ones8(sc + x);
                        ones8(sc + kScaleBytes + x);
                    }
                    sc_mine = false;
                }
                __syncwarp();
            }
            if (lane == 0) mbar_arrive_expect_tx(bar, 2 * ns * c.seg * S::kRowBytes);
            __syncwarp();
            // a lane a segment: side by side they issue in 85 cycles each, one after another from one lane in 120
            int at = __shfl_sync(0xffffffffu, pages, (j * c.spt + lane) & 31);
            if (lane < ns) {
                if (at < 0 || at >= a.c.num_blocks) {
                    set_status(a.status, UP_DEV_BAD_PAGE);
                    at = static_cast<int>(a.c.num_blocks);              // out of the map's bounds: zeros
                }
                const uint32_t dst = stage + lane * a.pitch;
                const int from = part_of(s0 + lane) * c.seg;
                if (a.both) {
                    tma_load_5d(dst, kmap, bar, 0, from, 0, 0, at * a.c.Hkv + head);
                } else {
                    tma_load_5d(dst + a.k_at, kmap, bar, 0, from, 0, head, at);
                    tma_load_5d(dst + a.v_at, vmap, bar, 0, from, 0, head, at);
                }
            }
            __syncwarp();
            if constexpr (E4M3) {
                const int64_t src = ((int64_t)sc_page * a.c.Hkv + head) * a.c.Bp + sc_from;
                if (sc_mine && UP_IN(src, a.c.scale_limit - c.sc + 1, a.status)) {
                    if (c.sc == 16) {
                        copy16(sc, a.c.ks + src);
                        copy16(sc + kScaleBytes, a.c.vs + src);
                    } else {
                        copy8(sc, a.c.ks + src);
                        copy8(sc + kScaleBytes, a.c.vs + src);
                    }
                }
                arrive_after_copies(bar);
            }
            ++tiles;
            if (++slot == S::kStages) slot = 0, phase ^= 1;
            if (j == 0) pages_next = fetch(w, i + tiles_per);           // the batch after this one
        }
        // the next item, while this one's tiles are on their way
        w.next(a);
        first_pages = fetch(w, 0);
    }
    if (!warp_wait(&sh.iempty[islot], iphase ^ 1, &sh.abort)) return leave(false);
    if (lane == 0) {
        sh.item[islot].n = 0;
        mbar_arrive(smem_u32(&sh.ifull[islot]));
    }
    leave(true);
}

// bit i: row i of a warp's 16 value rows has a code other than +0 and -0.  Lanes i and i + 16 read half of row i, which
// starts at byte `row` (a lane's own), panels `panel` bytes apart.  The order of a row's columns does not matter here, so
// eight neighbouring lanes take eight different ones.  Not inline: the loop around it keeps its registers (32 query heads
// on one key head of 128: 105.8 us inline, 103.2 so).
template <int DK, int PB>
__device__ __noinline__ uint32_t nonzero_rows(uint32_t row, uint32_t panel) {
    constexpr int N = PB / 16, HALF = DK / 32;         // 16-byte columns of a panel, and of half a row
    const int lane = threadIdx.x & 31, half = lane >> 4;
    const int first = (N == 8 ? lane : lane >> 1) + (DK > PB ? 0 : half * HALF);
    const uint32_t at = row + (DK > PB ? half * panel : 0);
    uint32_t any = 0;
#pragma unroll 4
    for (int i = 0; i < HALF; ++i) {
        uint32_t x, y, z, w;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(x), "=r"(y), "=r"(z), "=r"(w)
                     : "r"(at + 16 * ((first + i) & (N - 1)))
                     : "memory");
        any |= x | y | z | w;
    }
    any &= 0x7f7f7f7fu;
    any |= __shfl_xor_sync(0xffffffffu, any, 16);
    return __ballot_sync(0xffffffffu, any != 0);
}

template <int DK, bool E4M3, int HT, bool TEAM>
__device__ void consume(const Args& a, uint32_t ring, uint8_t* ring_ptr, Control<Shape<DK, E4M3, HT>::kLdq, HT, Shape<DK, E4M3, HT>::kStages>& sh) {
    using S = Shape<DK, E4M3, HT>;
    constexpr int KS = DK / 16, NH = HT / 8;           // steps of 16 columns; tiles of 8 query heads
    constexpr int PB = S::kPanelBytes;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const Cut& c = a.cut;
    int slot = 0, qslot = 0;
    uint32_t phase = 0, qphase = 0;

    // tile row 16 warp + (lane & 15): its segment of the tile and its token there
    const int my_row = 16 * warp + (lane & 15);
    const int my_seg = div_of(my_row, c.by_segp), my_off = my_row - my_seg * c.segp;
    // where the rows that this lane addresses for ldmatrix start: a segment's place holds all panels of its rows, one
    // after another.  Keys and values are a multiple of 1024 bytes apart, so that they share the swizzled addresses.
    auto row_at = [&](int row) {
        const int j = div_of(row, c.by_segp);
        return static_cast<uint32_t>(j * a.pitch + (row - j * c.segp) * PB);
    };
    const uint32_t krow = row_at(my_row), vrow = E4M3 ? krow : row_at(16 * warp + (lane & 7) + ((lane >> 4) << 3));
    const uint32_t panel = c.seg * PB;
    const bool whole = c.spt * c.segp == kTile && c.segp == c.seg && (c.spp == 1 || c.B % c.seg == 0);
    const int scs = (c.seg + c.sc - 1) & -c.sc;
    // scale bytes of the keys g and g + 8 of the warp
    uint32_t sc_at[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int row = 16 * warp + g + 8 * j, s = div_of(row, c.by_segp);
        sc_at[j] = min(s * scs + row - s * c.segp, kScaleBytes - 1);
    }

    uint32_t qb[NH][KS][2];
    float qf[NH][2];                                   // factors of the scores of heads 2t, 2t + 1
    // queries to registers, as the products' second operand: head g (of each tile of 8), columns
    // 16k + {2t, 2t+1, 2t+8, 2t+9}; for e4m3 16k + 4t .. 4t+3, the order that the key bytes come in
    auto load_queries = [&](int heads) {
        if (!warp_wait(&sh.qfull[qslot], qphase, &sh.abort)) return false;
        const uint32_t* qs = reinterpret_cast<const uint32_t*>(sh.q[qslot]);
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            const uint32_t* row = qs + (g + 8 * h) * (S::kLdq / 2);
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                qb[h][k][0] = E4M3 ? row[8 * k + 2 * t] : row[8 * k + t];
                qb[h][k][1] = E4M3 ? row[8 * k + 2 * t + 1] : row[8 * k + t + 4];
                // a row that no query fills holds another item's, whose scores would move the warp's references
                if (g + 8 * h >= heads) qb[h][k][0] = qb[h][k][1] = 0;
            }
            qf[h][0] = qf[h][1] = a.scale2;
            if constexpr (E4M3) {
                // e4m3 codes are exact in f16, and so are the queries once their largest is in [2^14, 2^15) (numbers
                // 2^-29 and less of it lose bits far below an fp32 sum's)
                uint32_t m = 0;
#pragma unroll
                for (int k = 0; k < KS; ++k) m = __vmaxu2(m, __vmaxu2(qb[h][k][0] & 0x7fff7fffu, qb[h][k][1] & 0x7fff7fffu));
                m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
                const int e = static_cast<int>(max(m & 0xffffu, m >> 16) >> 7);      // exponent field of the head's largest
                const int up = min(268 - e, 253);                                    // 2^(up - 127) scales it
                const float f = __uint_as_float(static_cast<uint32_t>(up) << 23);
                const float back = __uint_as_float(static_cast<uint32_t>(254 - up) << 23);
                qf[h][0] *= __shfl_sync(0xffffffffu, back, 8 * t);
                qf[h][1] *= __shfl_sync(0xffffffffu, back, 8 * t + 4);
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    qb[h][k][0] = f16x2(low_of(qb[h][k][0]) * f, high_of(qb[h][k][0]) * f);
                    qb[h][k][1] = f16x2(low_of(qb[h][k][1]) * f, high_of(qb[h][k][1]) * f);
                }
            }
        }
        // The reads may still be in flight here (rows of 2 dk bytes fall into the same banks), and the copy that the arrival
        // allows is another proxy's: without the fence it overtook them.
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.qempty[qslot]));
        if (++qslot == 2) qslot = 0, qphase ^= 1;
        return true;
    };

    // the consumer warps meet: a bounded wait like the others (a warp that has given up has left)
    uint32_t jphase = 0;
    auto meet = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.joined));
        const bool all = warp_wait(&sh.joined, jphase, &sh.abort);
        jphase ^= 1;
        return all;
    };

    int islot = 0;
    uint32_t iphase = 0;
    for (;;) {
        if (!warp_wait(&sh.ifull[islot], iphase, &sh.abort)) return give_up(a);
        const Item it = sh.item[islot];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.iempty[islot]));
        if (++islot == kItems) islot = 0, iphase ^= 1;
        if (it.n == 0) return;
        const int heads = min(HT, a.group - it.h0);
        if (it.fresh && !load_queries(heads)) return give_up(a);

        // sums of the warp's keys, heads 2t and 2t + 1 (of each tile of 8).  o[h][k]: columns 16k + g (0, 1) and
        // 16k + g + 8 (2, 3); for e4m3 16k + 2g and 16k + 2g + 1.
        float o[NH][KS][4];
        // References: rs near the running maximum of the scores (of the sums l) and, with scaled values, rt near that of
        // score + the value's exponent over the rows that are not all zeros (of the sums o): a token may have nearly all the
        // weight and values 2^-100 of another's, or none.  -inf before the first score.  rf = 2^(rs - rt).
        float rs[NH][2], rt[NH][2], rf[NH][2], l[NH][2];
#pragma unroll
        for (int h = 0; h < NH; ++h) {
#pragma unroll
            for (int k = 0; k < KS; ++k) o[h][k][0] = o[h][k][1] = o[h][k][2] = o[h][k][3] = 0.f;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                rs[h][x] = rt[h][x] = -INFINITY;
                rf[h][x] = 1.f;
                l[h][x] = 0.f;
            }
        }

        const int n = it.n, t0 = it.t0;
        int last_slot = 0;
        for (int i = 0; i < n; ++i) {
            if (!warp_wait(&sh.full[slot], phase, &sh.abort)) return give_up(a);
            last_slot = slot;
            const uint32_t st = ring + slot * S::kStage, sk = st + a.k_at, sv = st + a.v_at, sb = st + 2 * S::kTileBytes;
            // bit i: the warp's i-th key counts
            uint32_t counts = 0xffffu;
            if (!whole || t0 + i == 0 || t0 + i == it.tiles - 1) {
                const int s = it.seg0 + (t0 + i) * c.spt + my_seg;
                const int page = div_of(s, c.by_spp), tok = (s - page * c.spp) * c.seg + my_off;
                const int64_t pos = (int64_t)page * c.B + tok;
                counts = __ballot_sync(0xffffffffu, my_seg < c.spt && my_off < c.seg && tok < c.B && pos >= it.lo &&
                                                        pos < it.len);
            }
            const bool masked = counts != 0xffffu;
            if (counts != 0) {                     // else nothing for this warp (rows that odd pages leave unused)
            // scores, keys in the rows: s[h] = (key g: heads 2t, 2t + 1; key g + 8: the same), in two parts so
            // that a product need not wait for the one before
            float s[NH][2][4];
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
                for (int x = 0; x < 4; ++x) s[h][0][x] = s[h][1][x] = 0.f;
            if constexpr (E4M3) {
#pragma unroll
                for (int k = 0; k < KS; k += 2) {
                    uint32_t b[4];                 // (keys 0-7, 8-15) of 16 bytes, then of the next 16
                    ldsm4(b, sk + swizzled<PB>(krow + (k >> 3) * panel, k + (lane >> 4)));
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        uint32_t a0, a1, a2, a3;
                        kv::e4m3x4_to_f16x4(b[2 * x], a0, a2);
                        kv::e4m3x4_to_f16x4(b[2 * x + 1], a1, a3);
#pragma unroll
                        for (int h = 0; h < NH; ++h) mma<true>(s[h][x], a0, a1, a2, a3, qb[h][k + x][0], qb[h][k + x][1]);
                    }
                }
            } else {
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    uint32_t b[4];                 // (keys 0-7, 8-15) of 8 columns, then of the next 8
                    ldsm4(b, sk + swizzled<PB>(krow + (k >> 2) * panel, 2 * k + (lane >> 4)));
#pragma unroll
                    for (int h = 0; h < NH; ++h) mma<false>(s[h][k & 1], b[0], b[1], b[2], b[3], qb[h][k][0], qb[h][k][1]);
                }
            }
            float kf[2] = {1.f, 1.f}, vf[2] = {1.f, 1.f};      // scales of the keys' and values' rows g, g + 8
            if constexpr (E4M3) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    kf[j] = __uint_as_float(max(lds_u8(sb + sc_at[j]) << 23, 0x00400000u));    // 2^(b - 127)
                    vf[j] = __uint_as_float(max(lds_u8(sb + kScaleBytes + sc_at[j]) << 23, 0x00400000u));
                }
            }
            const bool ok[2] = {((counts >> g) & 1) != 0, ((counts >> (g + 8)) & 1) != 0};
            if (E4M3 && masked) {                  // bytes that nobody wrote may stand for infinity
                vf[0] = ok[0] ? vf[0] : 0.f;
                vf[1] = ok[1] ? vf[1] : 0.f;
            }
            // Of key g + 8j and head 2t + x: y[h][j][x] = 2^(score - rs), and pw the same times the value's scale over
            // 2^(rt - rs).  The references stay while no weight passes 2^kSlack: a weight that does, or is NaN (also
            // before the first score), has all the warp's moved.
            float y[NH][2][2], pw[NH][2][2];
            auto weigh = [&]() {
                bool good = true;
#pragma unroll
                for (int h = 0; h < NH; ++h)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const float f = E4M3 ? kf[j] * qf[h][x] : qf[h][x];
                            float d = __fmaf_rn(s[h][0][2 * j + x] + s[h][1][2 * j + x], f, -rs[h][x]);
                            if (masked && !ok[j]) d = -INFINITY;
                            good &= d <= kSlack;
                            y[h][j][x] = ex2(d);
                            pw[h][j][x] = y[h][j][x];
                            if constexpr (E4M3) {
                                pw[h][j][x] = y[h][j][x] * vf[j] * rf[h][x];
                                good &= pw[h][j][x] <= kTop;
                            }
                        }
                return good;
            };
            if (!__all_sync(0xffffffffu, weigh())) {
                if constexpr (E4M3) {
                    // A row of zeros adds nothing whatever its weight and scale, so it must not raise the outputs'
                    // reference: the other rows' weights would lose their bits, or all of them, in f16.
                    const uint32_t live = nonzero_rows<DK, PB>(sv + vrow, panel);
                    vf[0] = (live >> g) & 1 ? vf[0] : 0.f;
                    vf[1] = (live >> (g + 8)) & 1 ? vf[1] : 0.f;
                }
#pragma unroll
                for (int h = 0; h < NH; ++h)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float p[2], top = -INFINITY, topv = -INFINITY;
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const float f = E4M3 ? kf[j] * qf[h][x] : qf[h][x];
                            p[j] = masked && !ok[j] ? -INFINITY : __fmul_rn(s[h][0][2 * j + x] + s[h][1][2 * j + x], f);
                            top = fmaxf(top, p[j]);
                            if (E4M3 && vf[j] != 0.f) topv = fmaxf(topv, p[j] + static_cast<float>(static_cast<int>(__float_as_uint(vf[j]) >> 23) - 127));
                        }
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                        const float ns = fmaxf(rs[h][x], top);
                        float f = weight(rs[h][x], ns);
                        l[h][x] *= f;
                        rs[h][x] = ns;
                        const float us = ns == -INFINITY ? 0.f : ns;       // 0 stands in for a reference of -inf
                        float ut = 0.f;
                        if constexpr (E4M3) {
#pragma unroll
                            for (int d = 4; d < 32; d <<= 1) topv = fmaxf(topv, __shfl_xor_sync(0xffffffffu, topv, d));
                            // 126 below the scores' at least, which 2^-126 and its inverse reach: a row that could
                            // need more has no weight left in 32 bits
                            const float nt = fmaxf(fmaxf(rt[h][x], topv - kLift), ns - 126.f);
                            f = weight(rt[h][x], nt);
                            rt[h][x] = nt;
                            ut = nt == -INFINITY ? 0.f : nt;
                            rf[h][x] = ex2(us - ut);
                        }
#pragma unroll
                        for (int k = 0; k < KS; ++k) {
                            o[h][k][x] *= f;
                            o[h][k][2 + x] *= f;
                        }
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            y[h][j][x] = ex2(__fsub_rn(p[j], us));
                            pw[h][j][x] = E4M3 ? y[h][j][x] * vf[j] * rf[h][x] : y[h][j][x];
                        }
                    }
            }
            // weights, transposed to the second operand (keys 2t, 2t + 1 and 2t + 8, 2t + 9 of head g)
            uint32_t pb[NH][2], lo[NH][2];
#pragma unroll
            for (int h = 0; h < NH; ++h) {
#pragma unroll
                for (int x = 0; x < 2; ++x) l[h][x] += y[h][0][x] + y[h][1][x];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if constexpr (E4M3) {
                        pb[h][j] = transposed(f16x2(pw[h][j][0], pw[h][j][1]));        // a weight's one rounding: see kLift
                    } else {
                        // bf16 values want bf16 weights: high and low part, 16 bits together
                        const uint32_t hi = bf16x2(pw[h][j][0], pw[h][j][1]);
                        pb[h][j] = transposed(hi);
                        lo[h][j] = transposed(bf16x2(pw[h][j][0] - low_of(hi), pw[h][j][1] - high_of(hi)));
                    }
                }
            }
            // values, columns in the rows; a key that does not count is zero, whatever its row holds
            const uint32_t c0 = counts >> (2 * t), c1 = counts >> (2 * t + 8);
            const uint32_t z0 = (c0 & 1 ? 0xffffu : 0u) | (c0 & 2 ? 0xffff0000u : 0u);
            const uint32_t z1 = (c1 & 1 ? 0xffffu : 0u) | (c1 & 2 ? 0xffff0000u : 0u);
            auto values = [&](auto with_mask) {
                constexpr bool M = decltype(with_mask)::value;
                if constexpr (E4M3) {
#pragma unroll
                    for (int k = 0; k < KS; k += 2) {
                        uint32_t b[4];             // (keys 0-7, 8-15) of 16 bytes, then of the next 16
                        ldsm4t(b, sv + swizzled<PB>(vrow + (k >> 3) * panel, k + (lane >> 4)));
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            // bytes (key, column): (2t, 2g) (2t, 2g+1) (2t+1, 2g) (2t+1, 2g+1)
                            const uint32_t b0 = __byte_perm(b[2 * x], 0, 0x3120), b1 = __byte_perm(b[2 * x + 1], 0, 0x3120);
                            uint32_t e0, e1, d0, d1;
                            kv::e4m3x4_to_f16x4(b0, e0, d0);
                            kv::e4m3x4_to_f16x4(b1, e1, d1);
                            if constexpr (M) e0 &= z0, d0 &= z0, e1 &= z1, d1 &= z1;
#pragma unroll
                            for (int h = 0; h < NH; ++h) mma<true>(o[h][k + x], e0, d0, e1, d1, pb[h][0], pb[h][1]);
                        }
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        uint32_t b[4];             // keys 0-7 of 8 columns and the next 8, then keys 8-15
                        ldsm4t(b, sv + swizzled<PB>(vrow + (k >> 2) * panel, 2 * k + ((lane >> 3) & 1)));
                        if constexpr (M) b[0] &= z0, b[1] &= z0, b[2] &= z1, b[3] &= z1;
#pragma unroll
                        for (int h = 0; h < NH; ++h) {
                            mma<false>(o[h][k], b[0], b[1], b[2], b[3], pb[h][0], pb[h][1]);
                            mma<false>(o[h][k], b[0], b[1], b[2], b[3], lo[h][0], lo[h][1]);
                        }
                    }
                }
            };
            if (masked) values(std::true_type{}); else values(std::false_type{});
            }
            if (i + 1 < n) {                           // the last stage is kept for the join of the warps
                fence_proxy_async_smem();              // its next content comes by the async proxy
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh.empty[slot]));
            }
            if (++slot == S::kStages) slot = 0, phase ^= 1;
        }

        // join the warps: references and sums, then the outputs through the stage
        float* scratch = reinterpret_cast<float*>(ring_ptr + last_slot * S::kStage);
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[h][x] += __shfl_xor_sync(0xffffffffu, l[h][x], d);
        if (!meet()) return give_up(a);                // every warp is done with the stage, and with sh.m of the last item
        if (g == 0) {
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    sh.m[warp][8 * h + 2 * t + x] = rs[h][x];
                    sh.f[warp][8 * h + 2 * t + x] = E4M3 ? rt[h][x] : rs[h][x];
                    sh.l[warp][8 * h + 2 * t + x] = l[h][x];
                }
        }
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            if (h && !meet()) return give_up(a);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float* row = scratch + (warp * 8 + 2 * t + x) * kLd<DK>;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    if constexpr (E4M3) {
                        *reinterpret_cast<float2*>(row + 16 * k + 2 * g) = make_float2(o[h][k][x], o[h][k][2 + x]);
                    } else {
                        row[16 * k + g] = o[h][k][x];
                        row[16 * k + g + 8] = o[h][k][2 + x];
                    }
                }
            }
            if (!meet()) return give_up(a);
            constexpr int TPH = 4 * kWarps;            // threads of a head
            const int hh = threadIdx.x / TPH, x = threadIdx.x % TPH, hr = 8 * h + hh;
            float M = sh.m[0][hr];
#pragma unroll
            for (int i = 1; i < kWarps; ++i) M = fmaxf(M, sh.m[i][hr]);
            float L = 0.f, f[kWarps];
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                L = __fmaf_rn(sh.l[i][hr], weight(sh.m[i][hr], M), L);
                f[i] = weight(sh.f[i][hr], M);
            }
            float4 s[DK / (4 * TPH)];
#pragma unroll
            for (int k = 0; k < DK / (4 * TPH); ++k) {
                s[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int i = 0; i < kWarps; ++i) {
                    const float4 y = *reinterpret_cast<const float4*>(scratch + (i * 8 + hh) * kLd<DK> + 4 * (x + k * TPH));
                    s[k].x = __fmaf_rn(f[i], y.x, s[k].x), s[k].y = __fmaf_rn(f[i], y.y, s[k].y);
                    s[k].z = __fmaf_rn(f[i], y.z, s[k].z), s[k].w = __fmaf_rn(f[i], y.w, s[k].w);
                }
            }
            if (h == NH - 1) {                         // the stage goes back before the sums leave
                fence_proxy_async_smem();              // its next content comes by the async proxy
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh.empty[last_slot]));
            }
            const int64_t part = ((int64_t)it.r * a.Hq + it.head * a.group + it.h0 + hr) * c.max_splits + it.ch;
            if (hr < heads && (TEAM || UP_IN(part, a.parts, a.status))) {
                float* sums = TEAM ? reinterpret_cast<float*>(sh.q) + hr * DK : a.part_o + part * DK;
                // L = 0: no score above -inf.  NaN goes through.
                const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
                for (int k = 0; k < DK / (4 * TPH); ++k)
                    *reinterpret_cast<float4*>(sums + 4 * (x + k * TPH)) =
                        make_float4(s[k].x * inv, s[k].y * inv, s[k].z * inv, s[k].w * inv);
                if (x == 0) *(TEAM ? sh.lse + hr : a.part_lse + part) = L == 0.f ? -INFINITY : __fadd_rn(M, log2f(L));
            }
        }
    }
}

// ------------------------------------------------------------------------------------------------
// the join of a cluster's chunks, through its CTAs' shared memory.  Same arithmetic, in the same order, as
// join_kernel's for up to 16 chunks.

constexpr int kTeam = 16;

__device__ __forceinline__ void cluster_meet() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t of_rank(uint32_t addr, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

template <int DK, int LDQ, int HT, int NS>
__device__ void join_team(const Args& a, Control<LDQ, HT, NS>& sh) {
    const int64_t cap = (int64_t)a.max_blocks * a.cut.B;
    const int r = blockIdx.z, n = splits_of(a.cut, length_of(a, r), cap);
    const int head = static_cast<int>(blockIdx.y) / a.head_tiles, h0 = (static_cast<int>(blockIdx.y) - head * a.head_tiles) * HT;
    const int pairs = min(HT, a.group - h0) * (DK / 2);
    const uint32_t sums = smem_u32(sh.q), lses = smem_u32(sh.lse);
    for (int i = blockIdx.x * 32 * kWarps + threadIdx.x; i < pairs; i += gridDim.x * 32 * kWarps) {
        const int h = i / (DK / 2), d = i - h * (DK / 2);
        float v[kTeam], x[kTeam], y[kTeam], m = -INFINITY;
#pragma unroll
        for (int c = 0; c < kTeam; ++c) {
            v[c] = -INFINITY;
            x[c] = y[c] = 0.f;
            if (c < n) {
                v[c] = ld_cluster(of_rank(lses + 4 * h, c));
                x[c] = ld_cluster(of_rank(sums + 4 * (h * DK + 2 * d), c));
                y[c] = ld_cluster(of_rank(sums + 4 * (h * DK + 2 * d + 1), c));
            }
        }
#pragma unroll
        for (int c = 0; c < kTeam; ++c) m = fmaxf(m, v[c]);
        float l[kTeam], ox = 0.f, oy = 0.f;
#pragma unroll
        for (int c = 0; c < kTeam; ++c) {
            l[c] = c < n ? weight(v[c], m) : 0.f;
            if (c < n) {
                ox = __fadd_rn(ox, __fmul_rn(l[c], x[c]));
                oy = __fadd_rn(oy, __fmul_rn(l[c], y[c]));
            }
        }
#pragma unroll
        for (int o = kTeam / 2; o > 0; o >>= 1)
#pragma unroll
            for (int c = 0; c < o; ++c) l[c] += l[c + o];
        const float inv = l[0] == 0.f ? 0.f : 1.f / l[0];
        const int64_t row = (int64_t)r * a.Hq + head * a.group + h0 + h;
        reinterpret_cast<uint32_t*>(a.out)[row * (DK / 2) + d] = bf16x2(ox * inv, oy * inv);
        if (a.lse && d == 0) a.lse[row] = natural(m, l[0]);
    }
}

// TEAM: a call whose tables are narrow enough for every chunk to have a CTA at once (one request in a table of up to 8K
// tokens on 8 key heads); the chunks of a row are a cluster and join there, without a second launch.
template <int DK, bool E4M3, int HT, bool TEAM>
__global__ void __launch_bounds__(kThreads, (Shape<DK, E4M3, HT>::kCtas))
split_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
             const __grid_constant__ Args a) {
    using S = Shape<DK, E4M3, HT>;
    using C = Control<S::kLdq, HT, S::kStages>;
    extern __shared__ uint8_t raw[];
    uint8_t* base = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    C& sh = *reinterpret_cast<C*>(base + S::kStages * S::kStage);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(smem_u32(&sh.full[i]), E4M3 ? 33 : 1);       // the bulk copies; each lane's scale bytes
            mbar_init(smem_u32(&sh.empty[i]), kWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh.qfull[i]), 1);
            mbar_init(smem_u32(&sh.qempty[i]), kWarps);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(smem_u32(&sh.ifull[i]), 1);
            mbar_init(smem_u32(&sh.iempty[i]), kWarps);
        }
        mbar_init(smem_u32(&sh.joined), kWarps);
        sh.abort = 0;
        fence_mbar_init();
        prefetch_tmap(&kmap);
        prefetch_tmap(&vmap);
    }
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    if (warp == kWarps)
        produce<DK, E4M3, HT, TEAM>(a, &kmap, &vmap, smem_u32(base), sh);
    else
        consume<DK, E4M3, HT, TEAM>(a, smem_u32(base), base, sh);
    if constexpr (TEAM) {
        __syncwarp();
        cluster_meet();
        if (warp < kWarps) join_team<DK>(a, sh);
        __syncwarp();
        cluster_meet();        // no CTA leaves while another reads its sums
    } else {
        __syncthreads();
    }
    if (warp == kWarps && sh.abort) drain(sh);
}

// ------------------------------------------------------------------------------------------------
// The largest lse2 m of a row and the sum l of its chunks' weights, by every warp for itself; then the chunks
// i = g mod 16 are group g's, whose sums are added in the order of g.  A row has W warps: 16, a group each and
// eight chunks in flight, where rows are few (4 requests of 128K: 152 chunks a row); 4, with four groups each,
// where they are many; 1 where no row can have more than 8 chunks (256 requests of 1K: 128 -> 112 us for the
// whole call).  The order of the additions, and so the result, is the same.

constexpr int kJoinGroups = 16, kJoinAlone = 8;
static_assert(kJoinAlone <= kJoinGroups, "a group's sum is one chunk's where a warp adds them one after another");

template <int DK>
struct Row {
    static constexpr int E = DK / 32, VE = E < 4 ? E : 4, V = E / VE;      // a lane's columns: V vectors of VE floats
    using Vec = typename std::conditional<VE == 2, float2, float4>::type;
    float x[E];
    __device__ __forceinline__ void load(const float* row, int lane) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const Vec y = *reinterpret_cast<const Vec*>(row + v * 32 * VE + lane * VE);
#pragma unroll
            for (int e = 0; e < VE; ++e) x[v * VE + e] = reinterpret_cast<const float*>(&y)[e];
        }
    }
    __device__ __forceinline__ void store(float* row, int lane) const {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            Vec y;
#pragma unroll
            for (int e = 0; e < VE; ++e) reinterpret_cast<float*>(&y)[e] = x[v * VE + e];
            *reinterpret_cast<Vec*>(row + v * 32 * VE + lane * VE) = y;
        }
    }
    // the result row; l = 0: no score above -inf.  NaN goes through.
    __device__ __forceinline__ void put(const Args& a, int64_t row, int lane, float m, float l) const {
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            uint32_t* out = reinterpret_cast<uint32_t*>(a.out) + (row * DK + v * 32 * VE + lane * VE) / 2;
#pragma unroll
            for (int e = 0; e < VE; e += 2) out[e / 2] = bf16x2(x[v * VE + e] * inv, x[v * VE + e + 1] * inv);
        }
        if (a.lse && lane == 0) a.lse[row] = natural(m, l);
    }
};

template <int DK, int W>
__global__ void __launch_bounds__(W == 16 ? 512 : 128) join_kernel(const __grid_constant__ Args a) {
    constexpr int GPW = W > 1 ? kJoinGroups / W : 1;                   // groups of a warp
    constexpr int U = (W == 16 ? 8 : W == 4 ? 2 : 8) / (DK == 256 ? 2 : 1);
    __shared__ alignas(16) float sums[W > 1 ? kJoinGroups : 1][DK];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = W > 1 ? threadIdx.x >> 5 : 0;
    const int64_t row = W > 1 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= (int64_t)a.R * a.Hq || !UP_IN((row + 1) * a.cut.max_splits - 1, a.parts, a.status)) return;
    const int n = splits_of(a.cut, length_of(a, divided(static_cast<int>(row), a.by_hq)), (int64_t)a.max_blocks * a.cut.B);
    const float* pl = a.part_lse + row * a.cut.max_splits;
    const float* po = a.part_o + row * a.cut.max_splits * DK;
    float m = -INFINITY, l = 0.f;
    Row<DK> s[GPW];
#pragma unroll
    for (int i = 0; i < GPW; ++i)
#pragma unroll
        for (int e = 0; e < Row<DK>::E; ++e) s[i].x[e] = 0.f;
    constexpr int STEP = W > 1 ? kJoinGroups : 1;
    for (int i0 = 0; i0 < n; i0 += STEP * U) {
        Row<DK> x[GPW][U];                             // on their way while the weights are found
#pragma unroll
        for (int i = 0; i < GPW; ++i)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int at = i0 + u * STEP + warp + i * W;
                if (at < n) x[i][u].load(po + (int64_t)at * DK, lane);
            }
        if (i0 == 0) {
            for (int i = lane; i < n; i += 32) m = fmaxf(m, pl[i]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            for (int i = lane; i < n; i += 32) l += weight(pl[i], m);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        }
#pragma unroll
        for (int i = 0; i < GPW; ++i)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int at = i0 + u * STEP + warp + i * W;
                if (at < n) {
                    const float f = weight(pl[at], m);
#pragma unroll
                    for (int e = 0; e < Row<DK>::E; ++e)       // alone: a group's sum is one product, added as the others are
                        s[i].x[e] = W > 1 ? __fmaf_rn(f, x[i][u].x[e], s[i].x[e]) : __fadd_rn(s[i].x[e], __fmul_rn(f, x[i][u].x[e]));
                }
            }
    }
    if constexpr (W > 1) {
#pragma unroll
        for (int i = 0; i < GPW; ++i) s[i].store(sums[warp + i * W], lane);
        __syncthreads();
        if (warp != 0) return;
        Row<DK> y;
#pragma unroll
        for (int e = 0; e < Row<DK>::E; ++e) s[0].x[e] = 0.f;
        for (int g = 0; g < min(kJoinGroups, n); ++g) {
            y.load(sums[g], lane);
#pragma unroll
            for (int e = 0; e < Row<DK>::E; ++e) s[0].x[e] = __fadd_rn(s[0].x[e], y.x[e]);
        }
    }
    s[0].put(a, row, lane, m, l);
}

// ------------------------------------------------------------------------------------------------
// host side

template <int DK>
static int ctas_of(bool e4m3, int group) {
    if (group <= 8) return e4m3 ? Shape<DK, true, 8>::kCtas : Shape<DK, false, 8>::kCtas;
    return e4m3 ? Shape<DK, true, 16>::kCtas : Shape<DK, false, 16>::kCtas;
}

// Whole pages, or kTile rows of longer ones, leave part of a tile empty where one is no multiple of the other, and an
// e4m3 call takes its time by the tile.  There a page goes by its largest part of 8, 16 or 32 rows: it takes more
// copies, and every tile is full (32 requests of 0-16K, 8 heads of 128, pages of 24, 40 and 200: e4m3 112 -> 92,
// 131 -> 89 and 103 -> 85 us, bf16 142 -> 140, 148 -> 139 and 141 -> 138 us).
static int segment_of(int B) {
    if (kTile % B == 0 || B % kTile == 0 || B % 8) return B < kTile ? B : kTile;
    return B % 32 == 0 ? 32 : B % 16 == 0 ? 16 : 8;
}

// 0 for arguments that the call refuses
static int make_cut(int R, int Hq, int Hkv, int dk, int B, int max_blocks, int window, bool e4m3, Cut* c) {
    if (R <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || B <= 0 || B > (1 << 20)) return 0;
    if ((int64_t)R * Hq > 0x7fffffff || max_blocks <= 0 || window < 0) return 0;
    if (dk != 64 && dk != 128 && dk != 256) return 0;
    if ((int64_t)max_blocks * B > 0x7fffffff - 2 * kTile) return 0;
    c->B = B;
    c->seg = segment_of(B);
    c->segp = (c->seg + 1) & ~1;               // 64-byte rows: a segment starts on a 128-byte boundary
    c->spp = static_cast<int>(cdiv(B, c->seg));
    c->spt = kTile / c->segp;
    c->sc = c->seg == 8 && B > 8 ? 8 : 16;
    c->window = window;
    c->by_b = kv::fast_div(B);
    c->by_spt = kv::fast_div(c->spt);
    c->by_spp = kv::fast_div(c->spp);
    c->by_segp = kv::fast_div(c->segp);
    // the least number of chunks that makes one request's items a multiple of the grid
    const int group = Hq / Hkv, units = Hkv * (group <= 8 ? 1 : static_cast<int>(cdiv(group, 16)));
    const int grid = num_sms() * (dk == 64 ? ctas_of<64>(e4m3, group) : dk == 128 ? ctas_of<128>(e4m3, group) : ctas_of<256>(e4m3, group));
    int x = grid, y = units;
    while (y) {
        const int z = x % y;
        x = y;
        y = z;
    }
    c->s0 = std::min(grid / x, kMaxSplits);
    c->most = kMaxSplits / c->s0;
    c->by_wave = kv::fast_div(c->s0 * kMaxTiles);
    int64_t segs = (int64_t)max_blocks * c->spp;
    if (window > 0) segs = std::min<int64_t>(segs, (cdiv(window, B) + 1) * (int64_t)c->spp);
    const int tiles = static_cast<int>(cdiv(segs, c->spt));
    c->max_splits = splits_of(tiles, *c);      // splits_of never falls as the tiles grow
    return 1;
}

// Maps of (columns of a panel, tokens, panels, heads, pages): a box is every panel of a segment's rows.  Where a
// page's heads follow one another at the same stride as pages do, heads and pages can be one axis, and the axis that
// frees holds keys and values, |v - k| bytes apart: one box brings both, and the producer, which issues one in 85 cycles,
// needs half as many.  That counts where a tile is many segments (32 requests of 0-16K in e4m3: pages of 8 tokens, 8
// heads of 128, 101 -> 92 us; pages of 16, heads of 64, 68 -> 59 us; one request of 4K, 9.2 -> 8.8 us); of two in a
// tile, or one, nothing is left of it.
static bool make_maps(CUtensorMap* km, CUtensorMap* vm, Args* a, int dk, bool e4m3) {
    EncodeTiledFn fn = encode_tiled_fn();
    if (!fn) return false;
    const Cache& c = a->c;
    const Cut& cut = a->cut;
    const int e = e4m3 ? 1 : 2, inner = std::min(dk, 128 / e), panels = dk / inner, row = dk * e;
    const CUtensorMapDataType type = e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const CUtensorMapSwizzle swizzle = inner * e == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    const cuuint32_t es[5] = {1, 1, 1, 1, 1};
    auto encode = [&](CUtensorMap* m, const uint8_t* ptr, const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box) {
        return fn(m, type, 5, const_cast<uint8_t*>(ptr), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    const bool keys_first = c.k < c.v;
    const uint64_t apart = keys_first ? c.v - c.k : c.k - c.v;
    const bool one_axis = c.num_blocks == 1 || c.Hkv == 1 || c.sb == c.Hkv * c.sh;
    a->both = cut.spt >= 4 && cut.seg * row % 1024 == 0 && apart != 0 && one_axis && (c.num_blocks + 1) * c.Hkv < 0x7fffffff;
    if (a->both) {
        const cuuint64_t dims[5] = {(cuuint64_t)inner, (cuuint64_t)c.B, (cuuint64_t)panels, 2, (cuuint64_t)(c.num_blocks * c.Hkv)};
        const cuuint64_t strides[4] = {(cuuint64_t)c.st, (cuuint64_t)(inner * e), apart, (cuuint64_t)(c.Hkv == 1 ? c.sb : c.sh)};
        const cuuint32_t box[5] = {(cuuint32_t)inner, (cuuint32_t)cut.seg, (cuuint32_t)panels, 2, 1};
        a->both = encode(km, keys_first ? c.k : c.v, dims, strides, box);      // not where they lie too far apart
        a->pitch = 2 * cut.seg * row;
        a->k_at = keys_first ? 0 : cut.seg * row;
        a->v_at = keys_first ? cut.seg * row : 0;
        *vm = *km;
    }
    if (a->both) return true;
    const cuuint64_t dims[5] = {(cuuint64_t)inner, (cuuint64_t)c.B, (cuuint64_t)panels, (cuuint64_t)c.Hkv, (cuuint64_t)c.num_blocks};
    const cuuint64_t strides[4] = {(cuuint64_t)c.st, (cuuint64_t)(inner * e), (cuuint64_t)c.sh, (cuuint64_t)c.sb};
    const cuuint32_t box[5] = {(cuuint32_t)inner, (cuuint32_t)cut.seg, (cuuint32_t)panels, 1, 1};
    a->pitch = cut.segp * row;             // a copy starts on a 128-byte boundary
    a->k_at = 0;
    a->v_at = kTile * row;
    return encode(km, c.k, dims, strides, box) && encode(vm, c.v, dims, strides, box);
}

// the cluster that would hold a row's chunks, 0 where they do not all run at once
template <int DK, bool E4M3, int HT>
static int team_of(const Args& a) {
    int team = 1;
    while (team < a.cut.max_splits) team *= 2;
    const int64_t units = (int64_t)a.c.Hkv * a.head_tiles;
    return team <= kTeam && units <= 65535 && a.R <= 65535 && team * units * a.R <= (int64_t)Shape<DK, E4M3, HT>::kCtas * num_sms() ? team : 0;
}

template <int DK, bool E4M3, int HT, bool TEAM>
static cudaError_t prepare_split() {
    constexpr int smem = Sizes<DK, E4M3, HT>::kSmem;
    static_assert(smem <= 227 * 1024, "shared memory of a CTA");
    static_assert(Shape<DK, E4M3, HT>::kStage >= 8 * kWarps * kLd<DK> * 4, "the join of the warps fits a stage");
    static DeviceSet done{0};
    return once_per_device(done, [] {
        const cudaError_t e = cudaFuncSetAttribute(split_kernel<DK, E4M3, HT, TEAM>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        return TEAM && e == cudaSuccess
                   ? cudaFuncSetAttribute(split_kernel<DK, E4M3, HT, TEAM>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)
                   : e;
    });
}

// a launch in clusters of `team` CTAs
struct TeamLaunch {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    TeamLaunch(int team, const Args& a, int smem, cudaStream_t st) : cfg{} {
        cfg.gridDim = dim3(team, a.c.Hkv * a.head_tiles, a.R);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = st;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = team;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
    }
    TeamLaunch(const TeamLaunch&) = delete;
};

// Whether the current device has room for a cluster of `team` CTAs (a partition with small processing clusters may not
// have it for 16): asked once on each device and for each size.
template <int DK, bool E4M3, int HT>
static bool placed(int team, const Args& a) {
    static std::atomic<uint64_t> yes[5], no[5];        // bit d: device d; sizes 1, 2, 4, 8, 16
    int dev = 0, i = 0;
    while ((1 << i) < team) ++i;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = dev >= 0 && dev < 64 ? uint64_t{1} << dev : 0;
    if (yes[i].load(std::memory_order_relaxed) & bit) return true;
    if (no[i].load(std::memory_order_relaxed) & bit) return false;
    const TeamLaunch l(team, a, Sizes<DK, E4M3, HT>::kSmem, nullptr);
    int n = 0;
    const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, split_kernel<DK, E4M3, HT, true>, &l.cfg);
    if (e != cudaSuccess) cudaGetLastError();          // an answer, too: the next call's check must not find it
    const bool fits = e == cudaSuccess && n > 0;
    (fits ? yes : no)[i].fetch_or(bit, std::memory_order_relaxed);
    return fits;
}

template <int DK, bool E4M3, int HT>
static cudaError_t launch_split(const CUtensorMap& k, const CUtensorMap& v, const Args& a, int* team, cudaStream_t st) {
    constexpr int smem = Sizes<DK, E4M3, HT>::kSmem;
    if (*team != 0) {
        const cudaError_t e = prepare_split<DK, E4M3, HT, true>();
        if (e != cudaSuccess) return e;
        if (placed<DK, E4M3, HT>(*team, a)) {
            const TeamLaunch l(*team, a, smem, st);
            return cudaLaunchKernelEx(&l.cfg, split_kernel<DK, E4M3, HT, true>, k, v, a);
        }
        *team = 0;                                     // the same bits by two launches
    }
    const cudaError_t e = prepare_split<DK, E4M3, HT, false>();
    if (e != cudaSuccess) return e;
    return launch_pdl(split_kernel<DK, E4M3, HT, false>, dim3(Shape<DK, E4M3, HT>::kCtas * num_sms()), dim3(kThreads), smem, st, k, v, a);
}

// The join asks for the split's division of an SM's memory (nearly all of it shared): with the default one an SM
// would have to run empty between the two.
template <int DK, int W>
static cudaError_t launch_join(const Args& a, int64_t ctas, cudaStream_t st) {
    static DeviceSet done{0};
    const cudaError_t e = once_per_device(done, [] {
        return cudaFuncSetAttribute(join_kernel<DK, W>, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    });
    if (e != cudaSuccess) return e;
    return launch_pdl(join_kernel<DK, W>, dim3(static_cast<unsigned>(ctas)), dim3(W == 16 ? 512 : 128), 0, st, a);
}

template <int DK, bool E4M3, int HT>
static cudaError_t launch(const CUtensorMap& k, const CUtensorMap& v, const Args& a, cudaStream_t st) {
    int team = team_of<DK, E4M3, HT>(a);
    const cudaError_t e = launch_split<DK, E4M3, HT>(k, v, a, &team, st);
    count_launch(team ? 1 : 2);
    if (e != cudaSuccess || team) return e;
    const int64_t rows = (int64_t)a.Hq * a.R;
    if (rows <= 4 * num_sms()) return launch_join<DK, 16>(a, rows, st);
    return a.cut.max_splits > kJoinAlone ? launch_join<DK, 4>(a, rows, st) : launch_join<DK, 1>(a, cdiv(rows, 4), st);
}

template <int DK>
static cudaError_t launch_dk(const CUtensorMap& k, const CUtensorMap& v, const Args& a, bool e4m3, cudaStream_t st) {
    if (a.group <= 8) return e4m3 ? launch<DK, true, 8>(k, v, a, st) : launch<DK, false, 8>(k, v, a, st);
    return e4m3 ? launch<DK, true, 16>(k, v, a, st) : launch<DK, false, 16>(k, v, a, st);
}

}  // namespace decode
}  // namespace up

using namespace up;

extern "C" size_t up_paged_decode_workspace_bytes(int R, int Hq, int Hkv, int dk, int B, int max_blocks, int window) {
    decode::Cut c{}, d{};          // of a bf16 and an e4m3 cache
    if (!decode::make_cut(R, Hq, Hkv, dk, B, max_blocks, window, false, &c) ||
        !decode::make_cut(R, Hq, Hkv, dk, B, max_blocks, window, true, &d))
        return 0;
    const size_t parts = static_cast<size_t>(R) * Hq * std::max(c.max_splits, d.max_splits);
    return align_up(parts * sizeof(float), 256) + parts * dk * sizeof(float);
}

extern "C" up_status up_paged_decode(const uint16_t* q, int64_t q_stride, const up_kv_cache* cache,
                                     const int32_t* block_table, const int32_t* seqused, int R, int max_blocks,
                                     int Hq, float sm_scale, int window, uint16_t* out, float* lse, void* ws,
                                     size_t ws_bytes, int32_t* dev_status, void* stream) {
    using namespace up::decode;
    Args a{};
    if (!q || !block_table || !seqused || !out || !ws || !dev_status) return UP_ERR_ARG;
    const up_status s = kv::check(cache, &a.c);
    if (s != UP_OK) return s;
    if (R <= 0 || max_blocks <= 0 || Hq <= 0 || window < 0 || !(sm_scale > -INFINITY && sm_scale < INFINITY)) return UP_ERR_ARG;
    const bool e4m3 = cache->format == UP_KV_E4M3;
    if (!make_cut(R, Hq, cache->Hkv, cache->dk, cache->B, max_blocks, window, e4m3, &a.cut)) return UP_ERR_SHAPE;
    if (!aligned16(q) || !aligned16(out) || q_stride % 8 || (R > 1 && q_stride < (int64_t)Hq * cache->dk)) return UP_ERR_SHAPE;
    const size_t parts = static_cast<size_t>(R) * Hq * a.cut.max_splits;
    const size_t lse_bytes = align_up(parts * sizeof(float), 256);
    if (ws_bytes < lse_bytes + parts * cache->dk * sizeof(float) || !aligned16(ws)) return UP_ERR_WORKSPACE;
    a.q = reinterpret_cast<const uint8_t*>(q);
    a.q_stride = q_stride * 2;
    a.table = block_table;
    a.seqused = seqused;
    a.R = R;
    a.max_blocks = max_blocks;
    a.Hq = Hq;
    a.by_hq = kv::fast_div(Hq);
    a.group = Hq / cache->Hkv;
    a.head_tiles = a.group <= 8 ? 1 : static_cast<int>(cdiv(a.group, 16));
    a.scale2 = sm_scale * kLog2e;
    a.part_lse = static_cast<float*>(ws);
    a.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + lse_bytes);
    a.parts = static_cast<int64_t>(parts);
    a.out = out;
    a.lse = lse;
    a.status = dev_status;
    CUtensorMap km, vm;
    if (!encode_tiled_fn()) return UP_ERR_CUDA;
    if (!make_maps(&km, &vm, &a, cache->dk, e4m3)) return UP_ERR_SHAPE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = cache->dk == 64    ? launch_dk<64>(km, vm, a, e4m3, st)
                          : cache->dk == 128 ? launch_dk<128>(km, vm, a, e4m3, st)
                                             : launch_dk<256>(km, vm, a, e4m3, st);
    if (e != cudaSuccess) return failed_launch();
    return check_launch();
}
