// up_kv_evict and up_kv_move: which rows of the cache stay, by the weight that up_kv_mass has added up, and the moves
// that make the rows that stay the first of their request again.  (The drop of "UniPrefill: Universal Long-Context
// Prefill Acceleration via Block-wise Dynamic Sparsification", arXiv 2605.06221, chooses among the prompt's tokens
// before they are cached; this chooses among the cached ones, for every key head by itself.)
//
// Attention does not care for the order of its rows, so nothing is compacted: of the len rows k stay, and those of them
// at or beyond k, as many as there are holes below, move into the holes.  That is the least that can move, and since no
// row is both a source and a destination the moves need no order among themselves.
//
// evict_kernel finds the k-th largest of a list of 32-bit keys, a cluster of CTAs to a (request, head): the keys are read
// once into shared memory and the digits of the k-th largest found from the top, a histogram of a digit's values a pass,
// which the cluster's CTAs add up through distributed shared memory.  Then every position's rank among the rows
// that stay is the number of larger keys before it plus the number of equal ones before it, as far as they stay.
#include <stdint.h>

#include <algorithm>

#include "up_kv.cuh"

namespace up {
namespace evict {

using kv::FastDiv;

constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kDigit = 8, kBins = 1 << kDigit, kPasses = 32 / kDigit;
constexpr int kMaxCluster = 8;
constexpr int kMostKeys = 48 * 1024;         // keys of a CTA in shared memory; a longer part is read again by every pass

struct Args {
    const float* mass;
    const int32_t* born;
    const int32_t* table;
    const int32_t* seqused;
    const int32_t* budget;
    const int32_t* total;
    int32_t* moves;
    int32_t* num_moves;
    int32_t* new_len;
    int64_t num_blocks, records, max_moves;
    int R, Hkv, max_blocks, sinks, recent;
    int room;                // keys that the CTA's shared memory holds
    FastDiv by_b, by_heads;
    int32_t* status;
};

__device__ __forceinline__ int cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return static_cast<int>(r);
}
__device__ __forceinline__ int cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return static_cast<int>(r);
}
__device__ __forceinline__ void cluster_meet() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t ld_rank(const void* p, int rank) {
    uint32_t at, v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

// 32-bit keys in the order of the ranking: numbers by size, -0 as 0, every NaN above them, protected rows above all
constexpr uint32_t kNan = 0xff800001u, kProtected = 0xffffffffu;
__device__ __forceinline__ uint32_t key_of(float x) {
    if (x != x) return kNan;
    const uint32_t b = __float_as_uint(x + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

struct Shared {
    uint32_t hist[2][kBins];         // of a digit, every other pass
    uint32_t scan[kWarps + 1];
    uint32_t guarded, bad;           // protected rows and bad table entries of the CTA's part
    uint32_t above[2], equal[2];     // of the CTA's part: larger and equal keys below k, and in all
    uint32_t warp_above[kWarps], warp_equal[kWarps];
    uint32_t found[2];               // a pass's digit and what remains of k
};

// A list: (request, head) and what its rows are ranked by.
struct List {
    const Args& a;
    int r, head, len, k;
    int recent_from;                 // rows born there or later are protected
    bool few;                        // the protected rows do not all fit: only they are candidates

    // the row's record, -1 for a bad table entry
    __device__ __forceinline__ int64_t at(int pos) const {
        const int col = div_of(pos, a.by_b);
        const int64_t e = (int64_t)r * a.max_blocks + col;
        const int page = UP_IN(e, (int64_t)a.R * a.max_blocks, a.status) ? a.table[e] : 0;
        if (page < 0 || page >= a.num_blocks) return -1;
        return ((int64_t)page * a.Hkv + head) * a.by_b.d + (pos - col * static_cast<int>(a.by_b.d));
    }
    __device__ __forceinline__ uint32_t key(int pos, bool* guarded, bool* bad) const {
        const int64_t i = at(pos);
        *bad = i < 0;
        *guarded = false;
        if (i < 0 || !UP_IN(i, a.records, a.status)) return 0;
        const int born = a.born[i];
        *guarded = born < a.sinks || born >= recent_from;
        const uint32_t key = key_of(a.mass[i]);
        return few ? (*guarded ? key : 0u) : *guarded ? kProtected : key;
    }
};

__global__ void __launch_bounds__(kThreads) evict_kernel(const __grid_constant__ Args a) {
    extern __shared__ uint32_t keys[];
    __shared__ Shared sh;
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = cluster_rank(), ctas = cluster_size();
    const int list = static_cast<int>(blockIdx.x) / ctas;
    const int r = div_of(list, a.by_heads), head = list - r * a.Hkv;
    const bool first = rank == 0 && tid == 0;
    List l{a, r, head, 0, 0, 0, false};
    // what the list's CTAs all see alike, and leave together for
    const int64_t cap = (int64_t)a.max_blocks * a.by_b.d;
    l.len = UP_IN(r, a.R, a.status) ? a.seqused[r] : 0;
    if (l.len < 0 || l.len > cap) {
        if (first) set_status(a.status, UP_DEV_BAD_LENGTH);
        l.len = 0;
    }
    const int budget = a.budget[r];
    l.k = min(budget, l.len);
    l.recent_from = static_cast<int>(max((int64_t)(a.total ? a.total[r] : l.len) - a.recent, (int64_t)INT32_MIN));
    const auto leave = [&](int len) {
        if (first) a.num_moves[list] = 0;
        if (first && head == 0) a.new_len[r] = len;
    };
    if (budget < 0) {
        if (first) set_status(a.status, UP_DEV_BAD_BUDGET);
        return leave(l.len);
    }
    if (min(l.k, l.len - l.k) > a.max_moves) {
        if (first) set_status(a.status, UP_DEV_TOO_MANY_MOVES);
        return leave(l.len);
    }
    if (l.k == l.len || l.k == 0) return leave(l.k);       // all rows stay, or none
    // the CTA's part of the positions and the warp's part of that
    const int per_warp = static_cast<int>((l.len + (int64_t)ctas * kThreads - 1) / (ctas * kThreads)) * 32, per = per_warp * kWarps;
    const int start = rank * per, from = min(start + warp * per_warp, l.len), to = min(from + per_warp, l.len);
    const bool held = per <= a.room;
    for (int i = tid; i < 2 * kBins; i += kThreads) (&sh.hist[0][0])[i] = 0;
    if (tid == 0) sh.guarded = sh.bad = 0;
    __syncthreads();

    uint32_t prefix = 0;             // the digits found so far
    const auto key_at = [&](int pos) {
        if (held) return keys[pos - start];
        bool guarded, bad;
        return l.key(pos, &guarded, &bad);
    };
    // the keys, and the histogram of their first digit
    const auto load = [&]() {
        uint32_t guards = 0, bads = 0;
        for (int p = from + lane; p < to; p += 32) {
            bool guarded, bad;
            const uint32_t key = l.key(p, &guarded, &bad);
            guards += guarded;
            bads += bad;
            if (held) keys[p - start] = key;
            atomicAdd(&sh.hist[0][key >> (32 - kDigit)], 1u);
        }
        guards = __reduce_add_sync(0xffffffffu, guards);
        bads = __reduce_add_sync(0xffffffffu, bads);
        if (lane == 0 && guards) atomicAdd(&sh.guarded, guards);
        if (lane == 0 && bads) atomicAdd(&sh.bad, bads);
    };
    load();
    cluster_meet();
    uint32_t guards = 0, bads = 0;
    for (int c = 0; c < ctas; ++c) {
        guards += ld_rank(&sh.guarded, c);
        bads += ld_rank(&sh.bad, c);
    }
    if (bads) {
        if (first) set_status(a.status, UP_DEV_BAD_PAGE);
        cluster_meet();                            // no CTA leaves while another reads its sums
        return leave(l.len);
    }
    if (guards > static_cast<uint32_t>(l.k)) {
        l.few = true;
        cluster_meet();                            // nobody reads the first keys' histogram
        for (int i = tid; i < kBins; i += kThreads) sh.hist[0][i] = 0;
        __syncthreads();
        load();
        cluster_meet();
    }
    uint32_t need = l.k;                           // how many of the keys with this prefix stay
    for (int pass = 0; pass < kPasses; ++pass) {
        const int shift = 32 - kDigit * (pass + 1);
        uint32_t* const hist = sh.hist[pass & 1];
        if (pass) {
            for (int p = from + lane; p < to; p += 32) {
                const uint32_t key = key_at(p);
                if ((key ^ prefix) >> (shift + kDigit) == 0) atomicAdd(&hist[(key >> shift) & (kBins - 1)], 1u);
            }
            cluster_meet();
        }
        // the digit whose keys, and all larger ones, are the first to reach `need`; thread i has digit kBins - 1 - i
        uint32_t n = 0, upto;
        if (tid < kBins)
            for (int c = 0; c < ctas; ++c) n += ld_rank(&hist[kBins - 1 - tid], c);
        upto = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        if (lane == 31) sh.scan[warp] = upto;
        __syncthreads();
        uint32_t before = upto - n;
        for (int w = 0; w < warp && w < kBins / 32; ++w) before += sh.scan[w];
        if (tid < kBins && before < need && before + n >= need) {
            sh.found[0] = kBins - 1 - tid;
            sh.found[1] = need - before;
        }
        // the other histogram was read before this pass's meeting
        for (int i = tid; i < kBins; i += kThreads) sh.hist[(pass + 1) & 1][i] = 0;
        __syncthreads();
        prefix |= sh.found[0] << shift;
        need = sh.found[1];
    }
    // prefix is the k-th largest key: rows with larger ones stay, and the first `need` with equal ones
    uint32_t above = 0, equal = 0, above_low = 0, equal_low = 0;
    for (int p = from + lane; p < to; p += 32) {
        const uint32_t key = key_at(p);
        above += key > prefix;
        equal += key == prefix;
        above_low += key > prefix && p < l.k;
        equal_low += key == prefix && p < l.k;
    }
    above = __reduce_add_sync(0xffffffffu, above);
    equal = __reduce_add_sync(0xffffffffu, equal);
    above_low = __reduce_add_sync(0xffffffffu, above_low);
    equal_low = __reduce_add_sync(0xffffffffu, equal_low);
    if (tid < 2) sh.above[tid] = sh.equal[tid] = 0;
    if (lane == 0) sh.warp_above[warp] = above, sh.warp_equal[warp] = equal;
    __syncthreads();
    if (lane == 0) {
        atomicAdd(&sh.above[0], above_low);
        atomicAdd(&sh.equal[0], equal_low);
        atomicAdd(&sh.above[1], above);
        atomicAdd(&sh.equal[1], equal);
    }
    cluster_meet();
    above = equal = above_low = equal_low = 0;     // now: before the warp's part, and below k in the whole list
    for (int c = 0; c < ctas; ++c) {
        above_low += ld_rank(&sh.above[0], c);
        equal_low += ld_rank(&sh.equal[0], c);
        if (c < rank) {
            above += ld_rank(&sh.above[1], c);
            equal += ld_rank(&sh.equal[1], c);
        }
    }
    cluster_meet();                                // as above
    for (int w = 0; w < warp; ++w) {
        above += sh.warp_above[w];
        equal += sh.warp_equal[w];
    }
    const uint32_t stay_low = above_low + min(equal_low, need);
    if (first) {
        a.num_moves[list] = l.k - static_cast<int>(stay_low);
        if (head == 0) a.new_len[r] = l.k;
    }
    int32_t* const moves = a.moves + (int64_t)list * a.max_moves * 2;
    const uint32_t under = (1u << lane) - 1;
    for (int p0 = from; p0 < to; p0 += 32) {
        const int p = p0 + lane;
        const uint32_t key = p < to ? key_at(p) : 0;
        const uint32_t gt = __ballot_sync(0xffffffffu, p < to && key > prefix), eq = __ballot_sync(0xffffffffu, p < to && key == prefix);
        const uint32_t eq_before = equal + __popc(eq & under);
        const uint32_t stay_before = above + __popc(gt & under) + min(eq_before, need);
        const bool stays = key > prefix || (key == prefix && eq_before < need);
        if (p < to && (p < l.k) != stays) {
            const int64_t i = p < l.k ? p - stay_before : stay_before - stay_low;
            if (UP_IN(i, a.max_moves, a.status)) moves[2 * i + (p < l.k ? 1 : 0)] = p;
        }
        above += __popc(gt);
        equal += __popc(eq);
    }
}

// ------------------------------------------------------------------------------------------------
// the moves

constexpr int kMoveThreads = 128, kChunk = 16, kMoveUnroll = 8;

struct MoveArgs {
    kv::Cache c;
    uint8_t* k;
    uint8_t* v;
    uint8_t* ks;
    uint8_t* vs;
    float* mass;
    int32_t* born;
    const int32_t* table;
    const int32_t* moves;
    const int32_t* num_moves;
    int64_t max_moves, lists, records;
    int R, max_blocks;
    FastDiv by_b, by_heads;
    int32_t* status;
};

// where a row lies: bytes of its keys (values), its record's index and its scale bytes'; row < 0: nowhere
struct Place {
    int64_t row, record, scale;
};

__device__ __forceinline__ Place place_of(const MoveArgs& a, int r, int head, int pos) {
    Place p{-1, -1, -1};
    if (pos < 0 || pos >= (int64_t)a.max_blocks * a.by_b.d) {
        set_status(a.status, UP_DEV_BAD_SLOT);
        return p;
    }
    const int col = div_of(pos, a.by_b), tok = pos - col * static_cast<int>(a.by_b.d);
    const int64_t e = (int64_t)r * a.max_blocks + col;
    const int page = UP_IN(e, (int64_t)a.R * a.max_blocks, a.status) ? a.table[e] : 0;
    if (page < 0 || page >= a.c.num_blocks) {
        set_status(a.status, UP_DEV_BAD_PAGE);
        return p;
    }
    p.row = page * a.c.sb + head * a.c.sh + tok * a.c.st;
    p.record = ((int64_t)page * a.c.Hkv + head) * a.by_b.d + tok;
    p.scale = ((int64_t)page * a.c.Hkv + head) * a.c.Bp + tok;
    return p;
}

// A warp takes kChunk moves of a list at a time: a lane finds where a move's rows lie, and LPR lanes carry a row.
template <int LPR, bool SCALED>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const __grid_constant__ MoveArgs a) {
    constexpr int RPI = 32 / LPR, IT = kChunk / RPI, U = IT < kMoveUnroll ? IT : kMoveUnroll;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, sub = lane % LPR, grp = lane / LPR;
    for (int64_t list = blockIdx.y; list < a.lists; list += gridDim.y) {
        const int r = div_of(static_cast<uint32_t>(list), a.by_heads), head = static_cast<int>(list) - r * a.c.Hkv;
        const int n = a.num_moves[list];
        if (n < 0 || n > a.max_moves) {
            if (blockIdx.x == 0 && threadIdx.x == 0) set_status(a.status, UP_DEV_TOO_MANY_MOVES);
            continue;
        }
        const int2* const moves = reinterpret_cast<const int2*>(a.moves) + list * a.max_moves;
        for (int64_t i0 = ((int64_t)blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5)) * kChunk; i0 < n;
             i0 += (int64_t)gridDim.x * (kMoveThreads / 32) * kChunk) {
            Place src{-1, -1, -1}, dst{-1, -1, -1};
            if (lane < kChunk && i0 + lane < n) {
                const int2 m = moves[i0 + lane];
                src = place_of(a, r, head, m.x);
                dst = place_of(a, r, head, m.y);
                if (src.row < 0 || dst.row < 0) src.row = dst.row = -1;
            }
            const bool mine = src.row >= 0;
            uint8_t sk = 0, sv = 0;
            float mass = 0.f;
            int born = 0;
            if (SCALED && mine && UP_IN(src.scale, a.c.scale_limit, a.status)) sk = a.ks[src.scale], sv = a.vs[src.scale];
            if (a.mass && mine && UP_IN(src.record, a.records, a.status)) mass = a.mass[src.record];
            if (a.born && mine && UP_IN(src.record, a.records, a.status)) born = a.born[src.record];
#pragma unroll
            for (int side = 0; side < 2; ++side) {
                uint8_t* const base = side ? a.v : a.k;
#pragma unroll
                for (int j0 = 0; j0 < IT; j0 += U) {
                    uint4 x[U];
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int64_t row = __shfl_sync(0xffffffffu, src.row, (j0 + u) * RPI + grp);
                        x[u] = make_uint4(0, 0, 0, 0);
                        if (row >= 0 && UP_IN(row + 16 * sub, a.c.row_limit, a.status)) x[u] = *reinterpret_cast<const uint4*>(base + row + 16 * sub);
                    }
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int64_t row = __shfl_sync(0xffffffffu, dst.row, (j0 + u) * RPI + grp);
                        if (row >= 0 && UP_IN(row + 16 * sub, a.c.row_limit, a.status)) *reinterpret_cast<uint4*>(base + row + 16 * sub) = x[u];
                    }
                }
            }
            if (SCALED && mine && UP_IN(dst.scale, a.c.scale_limit, a.status)) a.ks[dst.scale] = sk, a.vs[dst.scale] = sv;
            if (a.mass && mine && UP_IN(dst.record, a.records, a.status)) a.mass[dst.record] = mass;
            if (a.born && mine && UP_IN(dst.record, a.records, a.status)) a.born[dst.record] = born;
        }
    }
}

template <int LPR, bool SCALED>
static cudaError_t launch_move(const MoveArgs& a, cudaStream_t st) {
    const int64_t y = std::min<int64_t>(a.lists, 65535);
    const int64_t x = std::min<int64_t>(cdiv(a.max_moves, kChunk * (kMoveThreads / 32)), std::max<int64_t>(1, cdiv(32 * (int64_t)num_sms(), y)));
    return launch_pdl(move_kernel<LPR, SCALED>, dim3(static_cast<unsigned>(x), static_cast<unsigned>(y)), dim3(kMoveThreads), 0, st, a);
}

// lists of requests and heads, positions of a request
static bool fits(int R, int Hkv, int max_blocks, int B) {
    return (int64_t)R * Hkv <= (1 << 24) && (int64_t)max_blocks * B <= (1 << 30);
}

}  // namespace evict
}  // namespace up

using namespace up;

extern "C" up_status up_kv_evict(const float* mass, const int32_t* born, int64_t num_blocks, int Hkv, int B,
                                 const int32_t* block_table, const int32_t* seqused, const int32_t* budget, int R,
                                 int max_blocks, const int32_t* total, int sinks, int recent, int32_t* moves,
                                 int64_t max_moves, int32_t* num_moves, int32_t* new_len, int32_t* dev_status, void* stream) {
    using namespace up::evict;
    if (!mass || !born || !block_table || !seqused || !budget || !moves || !num_moves || !new_len || !dev_status) return UP_ERR_ARG;
    if (R <= 0 || Hkv <= 0 || max_blocks <= 0 || B <= 0 || B > (1 << 20) || num_blocks <= 0 || num_blocks > 0x7fffffff) return UP_ERR_ARG;
    if (sinks < 0 || recent < 0 || max_moves < 0) return UP_ERR_ARG;
    if (new_len == seqused || new_len == budget || new_len == total) return UP_ERR_ARG;      // other heads' CTAs still read those
    if (!fits(R, Hkv, max_blocks, B) || reinterpret_cast<uintptr_t>(moves) % 8) return UP_ERR_SHAPE;
    Args a{};
    a.mass = mass;
    a.born = born;
    a.table = block_table;
    a.seqused = seqused;
    a.budget = budget;
    a.total = total;
    a.moves = moves;
    a.num_moves = num_moves;
    a.new_len = new_len;
    a.num_blocks = num_blocks;
    a.records = num_blocks * Hkv * B;
    a.max_moves = max_moves;
    a.R = R;
    a.Hkv = Hkv;
    a.max_blocks = max_blocks;
    a.sinks = sinks;
    a.recent = recent;
    a.by_b = kv::fast_div(B);
    a.by_heads = kv::fast_div(Hkv);
    a.status = dev_status;
    const int64_t lists = (int64_t)R * Hkv, cap = (int64_t)max_blocks * B;
    int cluster = 1;
    while (cluster < kMaxCluster && lists * cluster * 2 <= 2 * num_sms() && cap > (int64_t)cluster * 2 * kThreads) cluster *= 2;
    const int64_t part = cdiv(cap, (int64_t)cluster * kThreads) * kThreads;
    a.room = static_cast<int>(std::min<int64_t>(part, kMostKeys));
    static DeviceSet done{0};
    cudaError_t e = once_per_device(done, [] {
        return cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostKeys * 4);
    });
    if (e != cudaSuccess) return failed_launch();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(lists * cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(a.room) * 4;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, evict_kernel, a);
    if (e != cudaSuccess) return failed_launch();
    count_launch();
    return check_launch();
}

extern "C" up_status up_kv_move(const up_kv_cache* cache, const int32_t* block_table, int R, int max_blocks,
                                const int32_t* moves, int64_t max_moves, const int32_t* num_moves, float* mass,
                                int32_t* born, int32_t* dev_status, void* stream) {
    using namespace up::evict;
    MoveArgs a{};
    if (!block_table || !moves || !num_moves || !dev_status) return UP_ERR_ARG;
    const up_status s = kv::check(cache, &a.c);
    if (s != UP_OK) return s;
    if (R <= 0 || max_blocks <= 0 || max_moves < 0) return UP_ERR_ARG;
    if (!fits(R, cache->Hkv, max_blocks, cache->B) || reinterpret_cast<uintptr_t>(moves) % 8) return UP_ERR_SHAPE;
    if (max_moves == 0) return UP_OK;
    a.k = static_cast<uint8_t*>(cache->k);
    a.v = static_cast<uint8_t*>(cache->v);
    a.ks = cache->k_scale;
    a.vs = cache->v_scale;
    a.mass = mass;
    a.born = born;
    a.table = block_table;
    a.moves = moves;
    a.num_moves = num_moves;
    a.max_moves = max_moves;
    a.lists = (int64_t)R * cache->Hkv;
    a.records = cache->num_blocks * cache->Hkv * cache->B;
    a.R = R;
    a.max_blocks = max_blocks;
    a.by_b = kv::fast_div(cache->B);
    a.by_heads = kv::fast_div(cache->Hkv);
    a.status = dev_status;
    const bool e4m3 = cache->format == UP_KV_E4M3;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int lanes = cache->dk / (e4m3 ? 16 : 8);
    cudaError_t e;
    if (e4m3)
        e = lanes == 4 ? launch_move<4, true>(a, st) : lanes == 8 ? launch_move<8, true>(a, st) : launch_move<16, true>(a, st);
    else
        e = lanes == 8 ? launch_move<8, false>(a, st) : lanes == 16 ? launch_move<16, false>(a, st) : launch_move<32, false>(a, st);
    if (e != cudaSuccess) return failed_launch();
    count_launch();
    return check_launch();
}
