// up_kv_evict and up_kv_move: which rows of the cache stay, by the weight that up_kv_mass has added up, and the moves
// that make the rows that stay the first of their request again.  (The drop of "UniPrefill: Universal Long-Context
// Prefill Acceleration via Block-wise Dynamic Sparsification", arXiv 2605.06221, chooses among the prompt's tokens
// before they are cached; this chooses among the cached ones, for every key head by itself.)
//
// Attention does not care for the order of its rows, so nothing is compacted: of the len rows k stay, and those of them
// at or beyond k, as many as there are holes below, move into the holes.  That is the least that can move, and since no
// row is both a source and a destination the moves need no order among themselves.
//
// evict_kernel finds the k-th largest of a list of 32-bit keys, a CTA or a cluster of CTAs to a (request, head): the keys are
// read once into shared memory and the digits of the k-th largest (11, 11 and 10 bits) found from the top, a histogram of a
// digit's values a pass, which the cluster's CTAs add up through distributed shared memory.  Then every position's rank
// among the rows that stay is the number of larger keys before it plus the number of equal ones before it, as far as they
// stay.  A lane takes four neighbouring positions at a time: one table entry and two 16-byte loads, where pages allow it.
// Measured (one GB300): one request of 4,097 positions on 8 heads 6.7 us in a replayed graph (9.5 called from Python), 64 of 0-8K on 8
// heads 27 us, 4 of 128K on 2 heads 25 us.  Bytes are not what bounds it (the keys come from L2 in 1 to 3 us).  A single list is a chain
// of latencies: some 4 us of launch, length, table and records, and six meetings of the CTA or cluster.  A ragged batch goes over its
// keys five times where the border needs more than a digit (load, count and gathering of the candidates, comparison, moves; about 450
// instructions for a warp's 128 positions), and its lists lie on the SMs by their number and not by their length: an SM is active for 27 to
// 60 thousand cycles, 44 in the mean.  Few long lists leave SMs idle: 64 CTAs work for 4 of 128K on 2 heads.
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "up_kv.cuh"

namespace up {
namespace evict {

using kv::FastDiv;

constexpr int kShift0 = 21, kShift1 = 10;    // where a key's first and second digit start
constexpr int kBins = 2048, kCoarse = kBins / 32;
constexpr int kMostKeys = 32 * 1024;         // keys of a CTA in shared memory; a longer part is read again by every pass

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
    int alone, part;         // keys that one CTA takes; keys that make another CTA of the cluster worth while
    int more, most;          // the launch's lists: of more than `more` and at most `most` positions
    bool quads;              // four neighbouring records lie side by side, 16-byte aligned
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

__device__ __forceinline__ uint32_t add_at_rank(const void* p, int rank, uint32_t x) {
    uint32_t at, v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(v) : "r"(at), "r"(x) : "memory");
    return v;
}
__device__ __forceinline__ void st_rank(const void* p, int rank, uint32_t x) {
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(x) : "memory");
}

// 32-bit keys in the order of the ranking: numbers by size, -0 as 0, every NaN above them, protected rows above all
constexpr uint32_t kZero = 0x80000000u, kNan = 0xff800001u, kProtected = 0xffffffffu;
__device__ __forceinline__ uint32_t key_of(float x) {
    if (x != x) return kNan;
    const uint32_t b = __float_as_uint(x + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

template <int W>
struct Shared {
    alignas(16) uint32_t hist[2][kBins];     // of a digit, every other pass; the second also for candidates
    uint32_t coarse[2][kCoarse];             // and of 32 neighbouring values together
    uint32_t guarded, bad, zeros;    // protected rows, bad table entries and zeros of the CTA's part
    uint32_t candidates;             // of the list, where this CTA collects them
    uint32_t above[2], equal[2];     // of the CTA's part: larger and equal keys below k, and in all
    uint32_t warp_above[W], warp_equal[W], warp_above_low[W], warp_equal_low[W];
    uint32_t list[3];                // protected rows, bad entries and zeros of the list
    uint32_t found[3];               // a pass's digit, what remains of k, and keys with that digit
    uint32_t sums[4];                // `above` and `equal` of the list below k, and of the CTAs before
};

// A list: (request, head) and what its rows are ranked by.
struct List {
    const Args& a;
    int r, head, len, k;
    int recent_from;                 // rows born there or later are protected
    bool few;                        // the protected rows do not all fit: only they are candidates

    // the record of a position, -1 for a bad table entry
    __device__ __forceinline__ int64_t at(int pos) const {
        const int col = div_of(pos, a.by_b);
        const int64_t e = (int64_t)r * a.max_blocks + col;
        const int page = UP_IN(e, (int64_t)a.R * a.max_blocks, a.status) ? a.table[e] : 0;
        if (page < 0 || page >= a.num_blocks) return -1;
        return ((int64_t)page * a.Hkv + head) * a.by_b.d + (pos - col * static_cast<int>(a.by_b.d));
    }
    __device__ __forceinline__ uint32_t key(float mass, int born, uint32_t* guards) const {
        const bool guarded = born < a.sinks || born >= recent_from;
        *guards += guarded;
        const uint32_t key = key_of(mass);
        return few ? (guarded ? key : 0u) : guarded ? kProtected : key;
    }
    // Four neighbouring records from pos on (a multiple of 4): where they are, then what they hold.
    struct Quad {
        int64_t at[4];               // the first one's where they lie side by side
        float m[4];
        int b[4];
    };
    // false for a bad table entry
    __device__ __forceinline__ bool locate(int pos, Quad& q) const {
        if (a.quads) {
            q.at[0] = pos < len ? at(pos) : -1;
            return pos >= len || q.at[0] >= 0;
        }
        bool good = true;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            q.at[j] = pos + j < len ? at(pos + j) : -1;
            good &= pos + j >= len || q.at[j] >= 0;
        }
        return good;
    }
    __device__ __forceinline__ void fetch(Quad& q) const {
        if (a.quads) {
            if (q.at[0] >= 0 && UP_IN(q.at[0] + 3, a.records, a.status)) {
                *reinterpret_cast<float4*>(q.m) = *reinterpret_cast<const float4*>(a.mass + q.at[0]);
                *reinterpret_cast<int4*>(q.b) = *reinterpret_cast<const int4*>(a.born + q.at[0]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (q.at[j] >= 0 && UP_IN(q.at[j], a.records, a.status)) q.m[j] = a.mass[q.at[j]], q.b[j] = a.born[q.at[j]];
        }
    }
    // their keys, 0 (below every key) for those that the list does not have
    __device__ __forceinline__ uint4 keys(int pos, const Quad& q, uint32_t* guards) const {
        uint32_t x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = pos + j < len ? key(q.m[j], q.b[j], guards) : 0u;
        return make_uint4(x[0], x[1], x[2], x[3]);
    }
};

// where the other CTAs' sums are: their own shared memory, or this CTA's alone
template <bool TEAM>
__device__ __forceinline__ void meet() {
    if constexpr (TEAM) cluster_meet(); else __syncthreads();
}
template <bool TEAM>
__device__ __forceinline__ uint32_t of_cta(const uint32_t* p, int rank) {
    if constexpr (TEAM) return ld_rank(p, rank); else return *p;
}
// the sum of a word over the list's CTAs, all on their way at once
template <int C>
__device__ __forceinline__ uint32_t over_ctas(const uint32_t* p, int ctas) {
    if constexpr (C == 1) return *p;
    uint32_t v[C], n = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) v[c] = c < ctas ? ld_rank(p, c) : 0u;
#pragma unroll
    for (int c = 0; c < C; ++c) n += v[c];
    return n;
}

// C: the most CTAs of a cluster, 1 without clusters
template <int W, int C>
__global__ void __launch_bounds__(32 * W, 1024 / (32 * W)) evict_kernel(const __grid_constant__ Args a) {
    constexpr int kThreads = 32 * W;
    constexpr bool TEAM = C > 1;
    extern __shared__ __align__(16) uint4 keys[];
    __shared__ Shared<W> sh;
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int size = TEAM ? cluster_size() : 1, rank = TEAM ? cluster_rank() : 0;
    const int list = TEAM ? static_cast<int>(blockIdx.x) / size : blockIdx.x;
    const int r = div_of(list, a.by_heads), head = list - r * a.Hkv;
    const bool first = rank == 0 && tid == 0;
    List l{a, r, head, 0, 0, 0, false};
    // what the list's CTAs all see alike, and leave together for
    const int64_t cap = (int64_t)a.max_blocks * a.by_b.d;
    l.len = UP_IN(r, a.R, a.status) ? a.seqused[r] : 0;
    const int budget = a.budget[r], total = a.total ? a.total[r] : 0;
    if (l.len < 0 || l.len > cap) {
        if (first) set_status(a.status, UP_DEV_BAD_LENGTH);
        l.len = 0;
    }
    if (l.len <= a.more || l.len > a.most) return;         // another launch's
    l.k = min(budget, l.len);
    l.recent_from = static_cast<int>(max((int64_t)(a.total ? total : l.len) - a.recent, (int64_t)INT32_MIN));
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
    // As many CTAs as the list is worth; the others leave at once (a cluster's barriers wait for those that stay).  A CTA
    // has a part of the positions, a warp a part of that, in steps of 128.
    const int ctas = TEAM && l.len > a.alone ? min(size, (l.len + a.part - 1) / a.part) : 1;
    if (rank >= ctas) return;
    const int steps = (l.len + ctas * (128 * W) - 1) / (ctas * (128 * W)), per = steps * 128 * W;
    const int from = rank * per + warp * steps * 128 + 4 * lane;      // the lane's first position
    const bool held = per <= a.room;
    uint4* const mine = keys + (warp * steps * 32 + lane);
    const auto clear = [&](uint32_t* hist) {
        for (int i = tid; i < kBins / 4; i += kThreads) reinterpret_cast<uint4*>(hist)[i] = make_uint4(0, 0, 0, 0);
    };
    clear(sh.hist[0]);
    clear(sh.hist[1]);
    if (tid == 0) sh.guarded = sh.bad = sh.zeros = sh.candidates = 0;
    __syncthreads();

    const auto load = [&]() {            // the keys, and the histogram of their first digit
        uint32_t guards = 0, bads = 0, zeros = 0;
        typename List::Quad q[2], next[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) bads += !l.locate(u < steps ? from + 128 * u : l.len, q[u]);
        for (int i0 = 0; i0 < steps; i0 += 2) {
#pragma unroll
            for (int u = 0; u < 2; ++u) l.fetch(q[u]);
#pragma unroll
            for (int u = 0; u < 2; ++u)                // the next step's places while this one's records are on their way
                bads += !l.locate(i0 + 2 + u < steps ? from + 128 * (i0 + 2 + u) : l.len, next[u]);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int p = from + 128 * (i0 + u);
                if (i0 + u < steps && p < l.len) {
                    const uint4 y = l.keys(p, q[u], &guards);
                    if (held) mine[32 * (i0 + u)] = y;
                    const uint32_t x[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {      // zeros and protected rows are many, and counted apart
                        zeros += x[j] == kZero;
                        if (x[j] != kZero && x[j] != kProtected && x[j] != 0) atomicAdd(&sh.hist[0][x[j] >> kShift0], 1u);
                    }
                }
                q[u] = next[u];
            }
        }
        if (held)                        // positions behind the list
            for (int i = 0; i < steps; ++i)
                if (from + 128 * i >= l.len) mine[32 * i] = make_uint4(0, 0, 0, 0);
        guards = __reduce_add_sync(0xffffffffu, guards);
        bads = __reduce_add_sync(0xffffffffu, bads);
        zeros = __reduce_add_sync(0xffffffffu, zeros);
        if (lane == 0) {
            if (guards) atomicAdd(&sh.guarded, guards);
            if (bads) atomicAdd(&sh.bad, bads);
            if (zeros) {
                atomicAdd(&sh.zeros, zeros);
                atomicAdd(&sh.hist[0][kZero >> kShift0], zeros);
            }
            if (guards && !l.few) atomicAdd(&sh.hist[0][kProtected >> kShift0], guards);
        }
    };
    // step i's keys again
    const auto again = [&](int i) {
        if (held) return mine[32 * i];
        typename List::Quad q;
        uint32_t guards = 0;
        l.locate(from + 128 * i, q);
        l.fetch(q);
        return l.keys(from + 128 * i, q, &guards);
    };
    // sums of 32 neighbouring values of a histogram, a warp some
    const auto coarsen = [&](int which) {
        __syncthreads();
#pragma unroll
        for (int i = warp; i < kCoarse; i += W) {
            const uint32_t n = __reduce_add_sync(0xffffffffu, sh.hist[which][32 * i + lane]);
            if (lane == 0) sh.coarse[which][i] = n;
        }
    };
    // protected rows, bad entries and zeros of the list
    const auto gather = [&]() {
        if (warp == 0) {
            const uint32_t x[3] = {over_ctas<C>(&sh.guarded, ctas), over_ctas<C>(&sh.bad, ctas), over_ctas<C>(&sh.zeros, ctas)};
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (lane == i) sh.list[i] = x[i];
        }
        __syncthreads();
    };
    load();
    coarsen(0);
    meet<TEAM>();
    gather();
    if (sh.list[1]) {
        if (first) set_status(a.status, UP_DEV_BAD_PAGE);
        meet<TEAM>();                              // no CTA leaves while another reads its sums
        return leave(l.len);
    }
    if (sh.list[0] > static_cast<uint32_t>(l.k)) {
        l.few = true;
        meet<TEAM>();                              // all have read the counts
        clear(sh.hist[0]);
        if (tid == 0) sh.zeros = 0;
        __syncthreads();
        load();
        coarsen(0);
        meet<TEAM>();
        gather();
    }
    uint32_t prefix = 0, need = l.k;               // the digits found so far, and how many of the keys with them stay
    // The digit whose keys, and all larger ones, are the first to reach `need`: first of 32 values together, then of one.
    // TOGETHER: over the histograms of all the list's CTAs, or this one's alone.
    const auto find = [&](int which, int shift, auto together) {
        constexpr bool TOGETHER = TEAM && decltype(together)::value;
        if (warp == 0) {
            uint32_t before = 0, count = 0;
            int bin = 0;
#pragma unroll
            for (int level = 0; level < 2; ++level) {
                constexpr int kEach[2] = {kCoarse / 32, 1};        // words of a lane; lane 0 has the largest
                uint32_t n[2] = {}, all = 0;
#pragma unroll
                for (int j = 0; j < kEach[level]; ++j) {
                    const int at = level ? 32 * bin + 31 - lane : kCoarse - 1 - (kEach[0] * lane + j);
                    n[j] = over_ctas<(TOGETHER ? C : 1)>(level ? &sh.hist[which][at] : &sh.coarse[which][at], ctas);
                    all += n[j];
                }
                uint32_t upto = all;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += y;
                }
                // the first lane that reaches it, and of its words the first
                const int l0 = __ffs(__ballot_sync(0xffffffffu, before + upto >= need)) - 1;
                uint32_t sum = before + upto - all;
                int j = 0;
                if (kEach[level] == 2 && sum + n[0] < need) sum += n[0], j = 1;
                const int at = level ? 32 * bin + 31 - lane : kCoarse - 1 - (kEach[0] * lane + j);
                before = __shfl_sync(0xffffffffu, sum, l0);
                bin = __shfl_sync(0xffffffffu, at, l0);
                count = __shfl_sync(0xffffffffu, n[0], l0);
            }
            if (lane == 0) sh.found[0] = bin, sh.found[1] = need - before, sh.found[2] = count;
        }
        __syncthreads();
        prefix |= sh.found[0] << shift;
        need = sh.found[1];
    };
    find(0, kShift0, std::true_type{});
    const uint32_t digit = prefix >> kShift0, rest = sh.found[2];
    if (digit == kProtected >> kShift0) {
        prefix = kProtected;                       // that digit's one key
    } else if (digit == kZero >> kShift0 && rest == sh.list[2]) {
        prefix = kZero;                            // nothing but zeros
    } else if (rest <= kBins) {
        // The keys with that digit, few by now, go to the first CTA, which finds the other digits alone.
        uint32_t n = 0;
        for (int i = 0; i < steps; ++i) {
            const uint4 y = again(i);
            n += (y.x >> kShift0 == digit) + (y.y >> kShift0 == digit) + (y.z >> kShift0 == digit) + (y.w >> kShift0 == digit);
        }
        uint32_t upto = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        const uint32_t all = __shfl_sync(0xffffffffu, upto, 31);
        if (all) {
            uint32_t at = 0;
            if (lane == 0) at = TEAM ? add_at_rank(&sh.candidates, 0, all) : atomicAdd(&sh.candidates, all);
            at = __shfl_sync(0xffffffffu, at, 0) + upto - n;
            for (int i = 0; i < steps && n; ++i) {
                const uint4 y = again(i);
                const uint32_t x[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (x[j] >> kShift0 == digit && (held || at < kBins)) {        // (all are, unless records change under the call)
                        if (TEAM) st_rank(&sh.hist[1][at], 0, x[j]); else sh.hist[1][at] = x[j];
                        ++at;
                        --n;
                    }
            }
        }
        meet<TEAM>();                              // all have read the first histograms, too
        if (rank == 0) {
#pragma unroll
            for (int pass = 1; pass < 3; ++pass) {
                const int known = pass == 1 ? kShift0 : kShift1, shift = pass == 1 ? kShift1 : 0;
                clear(sh.hist[0]);
                __syncthreads();
                for (uint32_t i = tid; i < rest; i += kThreads) {
                    const uint32_t x = sh.hist[1][i];
                    if ((x ^ prefix) >> known == 0) atomicAdd(&sh.hist[0][x >> shift & ((1u << (known - shift)) - 1)], 1u);
                }
                coarsen(0);
                __syncthreads();
                find(0, shift, std::false_type{});
            }
            __syncthreads();
            if (tid == 0) sh.found[0] = prefix;
        }
        if (TEAM) {
            meet<TEAM>();
            prefix = of_cta<TEAM>(&sh.found[0], 0);
            need = of_cta<TEAM>(&sh.found[1], 0);
        }
    } else {
#pragma unroll
        for (int pass = 1; pass < 3; ++pass) {
            const int known = pass == 1 ? kShift0 : kShift1, shift = pass == 1 ? kShift1 : 0;
            for (int i = 0; i < steps; ++i) {
                const uint4 y = again(i);
                const uint32_t x[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if ((x[j] ^ prefix) >> known == 0) atomicAdd(&sh.hist[pass & 1][x[j] >> shift & ((1u << (known - shift)) - 1)], 1u);
            }
            coarsen(pass & 1);
            meet<TEAM>();
            if (pass == 1) clear(sh.hist[0]);      // read before this pass's meeting
            find(pass & 1, shift, std::true_type{});
        }
    }
    // prefix is the k-th largest key: rows with larger ones stay, and the first `need` with equal ones.  Counts of either: the
    // lower and the upper half of a sum where it is of one step's 128 keys.
    const auto compare = [&](uint32_t x) { return x > prefix ? 1u : x == prefix ? 0x10000u : 0u; };
    uint32_t above = 0, equal = 0, above_low = 0, equal_low = 0;
    for (int i = 0; i < steps; ++i) {
        const int p = from + 128 * i;
        const uint4 y = again(i);
        const uint32_t c[4] = {compare(y.x), compare(y.y), compare(y.z), compare(y.w)};
        uint32_t all = 0, low = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            all += c[j];
            low += p + j < l.k ? c[j] : 0u;
        }
        above += all & 0xffffu, equal += all >> 16;
        above_low += low & 0xffffu, equal_low += low >> 16;
    }
    above = __reduce_add_sync(0xffffffffu, above);
    equal = __reduce_add_sync(0xffffffffu, equal);
    above_low = __reduce_add_sync(0xffffffffu, above_low);
    equal_low = __reduce_add_sync(0xffffffffu, equal_low);
    if (lane == 0) {
        sh.warp_above[warp] = above, sh.warp_equal[warp] = equal;
        sh.warp_above_low[warp] = above_low, sh.warp_equal_low[warp] = equal_low;
    }
    __syncthreads();
    // of the CTA below k, and of its warps before this one
    const auto over_warps = [&](const uint32_t* x, int warps) { return __reduce_add_sync(0xffffffffu, lane < warps ? x[lane] : 0u); };
    above_low = over_warps(sh.warp_above_low, W), equal_low = over_warps(sh.warp_equal_low, W);
    above = over_warps(sh.warp_above, warp), equal = over_warps(sh.warp_equal, warp);
    if (TEAM) {
        if (warp == 0) {
            const uint32_t x = over_warps(sh.warp_above, W), y = over_warps(sh.warp_equal, W);
            if (lane == 0) sh.above[0] = above_low, sh.equal[0] = equal_low, sh.above[1] = x, sh.equal[1] = y;
        }
        meet<TEAM>();
        if (warp == 0) {
            const uint32_t x[4] = {over_ctas<C>(&sh.above[0], ctas), over_ctas<C>(&sh.equal[0], ctas),
                                   over_ctas<C>(&sh.above[1], rank), over_ctas<C>(&sh.equal[1], rank)};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (lane == i) sh.sums[i] = x[i];
        }
        meet<TEAM>();                              // and no CTA leaves while another reads its sums
        above_low = sh.sums[0], equal_low = sh.sums[1];
        above += sh.sums[2], equal += sh.sums[3];
    }
    const uint32_t stay_low = above_low + min(equal_low, need);
    if (first) {
        a.num_moves[list] = l.k - static_cast<int>(stay_low);
        if (head == 0) a.new_len[r] = l.k;
    }
    int32_t* const moves = a.moves + (int64_t)list * a.max_moves * 2;
    const uint32_t most = static_cast<uint32_t>(min(a.max_moves, (int64_t)INT32_MAX));
    for (int i = 0; i < steps; ++i) {
        const int p = from + 128 * i, p0 = p - 4 * lane;
        const uint4 y = again(i);
        const uint32_t c[4] = {compare(y.x), compare(y.y), compare(y.z), compare(y.w)};
        const uint32_t own = c[0] + c[1] + c[2] + c[3], all = __reduce_add_sync(0xffffffffu, own);
        const uint32_t here = (all & 0xffffu) + min(equal + (all >> 16), need) - min(equal, need);     // rows of the step that stay
        // nothing moves where all of a step's rows below k stay, or none of those beyond
        if (!(p0 + 128 <= l.k && here == 128) && !(p0 >= l.k && here == 0)) {
            uint32_t upto = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t z = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += z;
            }
            uint32_t gt = above + ((upto - own) & 0xffffu), eq = equal + ((upto - own) >> 16);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t stay_before = gt + min(eq, need);
                const bool stays = c[j] == 1u || (c[j] != 0u && eq < need), low = p + j < l.k;
                if (p + j < l.len && low != stays) {
                    const uint32_t m = low ? p + j - stay_before : stay_before - stay_low;
                    // (m is below most, unless records change under the call)
                    if (m < most && UP_IN(m, a.max_moves, a.status)) moves[2 * (size_t)m + low] = p + j;
                }
                gt += c[j] & 1u;
                eq += c[j] >> 16;
            }
        }
        above += all & 0xffffu;
        equal += all >> 16;
    }
}

// a launch of evict_kernel, in clusters
struct ClusterLaunch {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    ClusterLaunch(int64_t lists, int cluster, int threads, size_t smem, cudaStream_t st) : cfg{} {
        cfg.gridDim = dim3(static_cast<unsigned>(lists * cluster));
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = st;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = cluster;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
    }
    ClusterLaunch(const ClusterLaunch&) = delete;
};

template <int W, int C>
static cudaError_t prepare_evict() {
    static DeviceSet done{0};
    return once_per_device(done, [] {
        const cudaError_t e = cudaFuncSetAttribute(evict_kernel<W, C>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostKeys * 4);
        return C > 8 && e == cudaSuccess ? cudaFuncSetAttribute(evict_kernel<W, C>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) : e;
    });
}

// The most CTAs of a cluster, `cluster` or fewer, that the current device has room for (a partition with small processing
// clusters may not have it for 8): asked once on each device and for each size, with all the memory that a call may want.
template <int W, int C>
static int placed(int cluster) {
    static std::atomic<uint64_t> yes[5], no[5];        // bit d: device d; sizes 1, 2, 4, 8, 16
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 1;
    const uint64_t bit = dev >= 0 && dev < 64 ? uint64_t{1} << dev : 0;
    for (; cluster > 1; cluster /= 2) {
        int i = 0, n = 0;
        while ((1 << i) < cluster) ++i;
        if (yes[i].load(std::memory_order_relaxed) & bit) return cluster;
        if (no[i].load(std::memory_order_relaxed) & bit) continue;
        const ClusterLaunch l(1, cluster, 32 * W, kMostKeys * 4, nullptr);
        const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, evict_kernel<W, C>, &l.cfg);
        if (e != cudaSuccess) cudaGetLastError();      // an answer, too: the next call's check must not find it
        const bool fits = e == cudaSuccess && n > 0;
        (fits ? yes : no)[i].fetch_or(bit, std::memory_order_relaxed);
        if (fits) return cluster;
    }
    return 1;
}

// the most keys that a CTA of `cluster` gets, of the longest list or of one that is not worth more CTAs, as far as it holds them
template <int W>
static int room_of(const Args& a, int cluster) {
    const int64_t cap = std::min<int64_t>((int64_t)a.max_blocks * a.by_b.d, a.most);
    const int64_t most = std::max<int64_t>(cdiv(cap, cluster), std::min<int64_t>(cap, a.alone));
    return static_cast<int>(std::min<int64_t>(cdiv(most, 128 * W) * 128 * W, kMostKeys));
}

template <int W>
static cudaError_t launch_alone(Args& a, int64_t lists, cudaStream_t st) {
    const cudaError_t e = prepare_evict<W, 1>();
    if (e != cudaSuccess) return e;
    a.room = room_of<W>(a, 1);
    return launch_pdl(evict_kernel<W, 1>, dim3(static_cast<unsigned>(lists)), dim3(32 * W), (size_t)a.room * 4, st, a);
}

template <int W, int C>
static cudaError_t launch_team(Args& a, int cluster, int64_t lists, cudaStream_t st) {
    const cudaError_t e = prepare_evict<W, C>();
    if (e != cudaSuccess) return e;
    cluster = placed<W, C>(cluster);
    if (cluster == 1) return launch_alone<W>(a, lists, st);
    a.room = room_of<W>(a, cluster);
    const ClusterLaunch l(lists, cluster, 32 * W, (size_t)a.room * 4, st);
    return cudaLaunchKernelEx(&l.cfg, evict_kernel<W, C>, a);
}

// ------------------------------------------------------------------------------------------------
// the moves

// Two rows' keys and values in flight a lane, and the registers for eight CTAs an SM, against eight rows of one side: 16
// requests of 4K-128K in bf16, half of the rows, 268 -> 230 us (6.2 TB/s); four of 128K in e4m3 to 16K 26.8 -> 26.2 (24.7 with
// sixteen, which takes a fifth longer on rows of 64 numbers).  Half as many CTAs: 243 us.
constexpr int kMoveThreads = 128, kChunk = 16, kMoveUnroll = 2, kMovePerSm = 64;

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
            for (int j0 = 0; j0 < IT; j0 += U) {
                uint4 x[U], y[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t row = __shfl_sync(0xffffffffu, src.row, (j0 + u) * RPI + grp);
                    x[u] = y[u] = make_uint4(0, 0, 0, 0);
                    if (row >= 0 && UP_IN(row + 16 * sub, a.c.row_limit, a.status)) {
                        x[u] = *reinterpret_cast<const uint4*>(a.k + row + 16 * sub);
                        y[u] = *reinterpret_cast<const uint4*>(a.v + row + 16 * sub);
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t row = __shfl_sync(0xffffffffu, dst.row, (j0 + u) * RPI + grp);
                    if (row >= 0 && UP_IN(row + 16 * sub, a.c.row_limit, a.status)) {
                        *reinterpret_cast<uint4*>(a.k + row + 16 * sub) = x[u];
                        *reinterpret_cast<uint4*>(a.v + row + 16 * sub) = y[u];
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
    const int64_t x = std::min<int64_t>(cdiv(a.max_moves, kChunk * (kMoveThreads / 32)),
                                        std::max<int64_t>(1, cdiv(kMovePerSm * (int64_t)num_sms(), y)));
    return launch_pdl(move_kernel<LPR, SCALED>, dim3(static_cast<unsigned>(x), static_cast<unsigned>(y)), dim3(kMoveThreads), 0, st, a);
}

// whether n numbers at p and m at q have one in common
static bool overlap(const int32_t* p, int64_t n, const int32_t* q, int64_t m) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return a < b ? b - a < static_cast<uint64_t>(n) * 4 : a - b < static_cast<uint64_t>(m) * 4;
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
    if (!mass || !born || !block_table || !seqused || !budget || !num_moves || !new_len || !dev_status) return UP_ERR_ARG;
    if (R <= 0 || Hkv <= 0 || max_blocks <= 0 || B <= 0 || B > (1 << 20) || num_blocks <= 0 || num_blocks > 0x7fffffff) return UP_ERR_ARG;
    if (sinks < 0 || recent < 0 || max_moves < 0 || (max_moves > 0 && !moves)) return UP_ERR_ARG;
    if (!fits(R, Hkv, max_blocks, B) || reinterpret_cast<uintptr_t>(moves) % 8) return UP_ERR_SHAPE;
    // a finished list's outputs must not be what the other lists, or CTAs of a cluster, still read their length and budget from
    const int64_t list_words = (int64_t)R * Hkv * std::min<int64_t>(max_moves, int64_t{1} << 35) * 2;
    for (const int32_t* in : {seqused, budget, total})
        if (in && (overlap(new_len, R, in, R) || overlap(num_moves, (int64_t)R * Hkv, in, R) ||
                   (moves && overlap(moves, list_words, in, R))))
            return UP_ERR_ARG;
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
    a.quads = B % 4 == 0 && aligned16(mass) && aligned16(born);
    // A list's CTAs: one where lists are many or short (up to 6K: one of 4K on 8 heads 7.6 us in a cluster, 6.8 alone; of 8K 10.9
    // and 12); a cluster where they leave SMs idle, or are longer than a CTA holds at two or three on an SM; one of 16, which
    // may not fit every device and meets more slowly, where 8 do not hold the keys (half a million on one head 93 -> 35 us).
    const bool many = lists > num_sms(), huge = cap > 8 * (int64_t)kMostKeys && lists * 16 <= num_sms();
    a.alone = many ? kMostKeys / 2 : 6144;
    a.part = many ? kMostKeys / 2 : 1024;
    a.more = -1;
    a.most = INT32_MAX;
    int cluster = 1;
    if (cap > a.alone)
        while (cluster < (huge ? 16 : 8) && cap > (int64_t)cluster * a.part &&
               (many || lists * cluster * 2 <= num_sms() || cap > (int64_t)cluster * kMostKeys))
            cluster *= 2;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // Many lists under wide tables may all be short: those go first, a CTA each, and then the clusters of the others, which leave at
    // once where they find nothing to do (64 of 0-8K on 8 heads in tables of 128K 84 -> 36 us, in such of 8K 27).
    const bool apart = many && cluster > 2;
    if (apart) {
        a.most = kMostKeys / 4;
        if (launch_alone<8>(a, lists, st) != cudaSuccess) return failed_launch();
        a.more = a.most;
        a.most = INT32_MAX;
    }
    // Many short lists go by CTAs of 8 warps, more of which an SM has at once: 128 of 1K on 8 heads 25.9 -> 15.5 us, 64 of 0-8K
    // 28.1 -> 27.3; fewer or longer ones want the threads: 16 of 4K 11.0 -> 8.9, 32 of 32K 84 -> 70.  Few lists with much for
    // each CTA of a cluster take all that an SM has: 4 of 128K on 2 heads 26.1 -> 25.0, one of a million on one 229 -> 169 (and by 16 97).
    const cudaError_t e = cluster > 8                                              ? launch_team<32, 16>(a, cluster, lists, st)
                          : cluster > 1 && !many && cap > (int64_t)cluster * 8192 ? launch_team<32, 8>(a, cluster, lists, st)
                          : cluster > 1                                            ? launch_team<16, 8>(a, cluster, lists, st)
                          : many && cap <= a.part                                  ? launch_alone<8>(a, lists, st)
                                                                                   : launch_alone<16>(a, lists, st);
    if (e != cudaSuccess) return failed_launch();
    count_launch(apart ? 2 : 1);
    return check_launch();
}

extern "C" up_status up_kv_move(const up_kv_cache* cache, const int32_t* block_table, int R, int max_blocks,
                                const int32_t* moves, int64_t max_moves, const int32_t* num_moves, float* mass,
                                int32_t* born, int32_t* dev_status, void* stream) {
    using namespace up::evict;
    MoveArgs a{};
    if (!block_table || !num_moves || !dev_status || (max_moves > 0 && !moves)) return UP_ERR_ARG;
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
