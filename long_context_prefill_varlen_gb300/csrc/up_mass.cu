// up_kv_mass: the attention weight that every cached row has had, added up step by step: what a cache that takes rows out by
// their weight goes by (up_kv_evict).  The cache is the one that Eqs. 16-17 of "UniPrefill: Universal Long-Context Prefill
// Acceleration via Block-wise Dynamic Sparsification" (arXiv 2605.06221) give slots and lengths to; the records are
// this library's own.
//
// After up_paged_decode has found a step's lse, a row's weight needs no other row:
//   mass_i <- decay mass_i + sum_h exp(q_h . K_i sm_scale - lse_h),
// so the keys are read once more and nothing is joined: 2 dk (dk + 1) bytes a row in bf16 (e4m3) and 8 of records,
// which HBM bounds.  A warp takes units of 16 to 64 rows of one head, straight from memory to registers: lane 4g + t reads
// 16-byte pieces t, t + 4, ... of rows g and g + 8, whose numbers are the products' first operand as they come if the
// queries' columns are taken in the same order (a sum over columns does not care); m16n8k16 with keys in the 16 rows and
// query heads in the 8 columns.
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
    float scale_hi, scale_lo;  // sm_scale * log2 e, in two parts
    float decay;
    FastDiv by_b;
    int32_t* status;
};

template <int DK, bool E4M3>
struct Shape {
    static constexpr int kRowBytes = DK * (E4M3 ? 1 : 2);
    static constexpr int kPieces = kRowBytes / 64;                     // 16-byte pieces of a row that a lane reads
    static constexpr int kTiles = kPieces >= 4 ? 1 : 4 / kPieces;      // tiles of 16 rows in a unit: 8 loads in flight or more
    static constexpr int kRows = 16 * kTiles;
    static constexpr int kCtas = DK == 256 || (DK == 64 && E4M3) ? 4 : DK == 128 && E4M3 ? 5 : 6;      // on an SM: 128, 96 and 80 registers a thread
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
    static constexpr int KS = DK / 16;
    uint32_t b[KS][2];         // head g of the tile, the columns of the lane's pieces
    float hi[2], lo[2];        // factors of heads 2t, 2t + 1 (in two parts), and their lse in log2
    float ref_hi[2], ref_lo[2];
    bool counts[2];

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
            const float l = h < heads ? a.lse[(int64_t)r * a.Hq + head * a.group + h0 + h] : -INFINITY;
            counts[x] = l != -INFINITY;
            // lse * log2 e to about 48 bits: fp32 alone would leave 2^-24 |lse| of a weight's exponent
            ref_hi[x] = l * 1.44269502f;
            ref_lo[x] = fabsf(l) < INFINITY ? fmaf(l, 1.44269502f, -ref_hi[x]) + l * 1.92596303e-8f : 0.f;
            hi[x] = a.scale_hi * back[x];
            lo[x] = a.scale_lo * back[x];
        }
    }
};

// A warp's run of units: of all requests' units in the order request, head, rows, its equal share.
struct Walk {
    int r, head, unit, units;      // units: of the request's head
    int len;
    int64_t left;

    template <int ROWS>
    __device__ __forceinline__ int units_of(const Args& a, int n) const {
        return n < 0 || n > (int64_t)a.max_blocks * static_cast<int64_t>(a.by_b.d) ? 0 : (n + ROWS - 1) / ROWS;
    }
    template <int ROWS>
    __device__ __forceinline__ void seek(const Args& a, int64_t warp, int64_t warps) {
        const int lane = threadIdx.x & 31;
        left = 0;
        int n = 0, mine = 0, upto = 0;
        auto scan = [&](int r0) {
            n = r0 + lane < a.R && UP_IN(r0 + lane, a.R, a.status) ? a.seqused[r0 + lane] : 0;
            mine = units_of<ROWS>(a, n);
            if (mine == 0 && n != 0) set_status(a.status, UP_DEV_BAD_LENGTH);
            upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += y;
            }
        };
        int64_t all = 0;
        for (int r0 = 0; r0 < a.R; r0 += 32) {
            scan(r0);
            all += __shfl_sync(0xffffffffu, upto, 31);
        }
        all *= a.c.Hkv;
        int64_t first;
        if (all == 0) return;
        if (all <= warps) {                            // few units: one each, to warps that lie evenly over the grid
            const int64_t per = warps / all;
            first = warp % per == 0 && warp / per < all ? warp / per : all;
            left = first < all ? 1 : 0;
        } else {
            first = all * warp / warps;
            left = all * (warp + 1) / warps - first;
        }
        if (left == 0) return;
        int64_t before = 0;
        for (int r0 = 0; r0 < a.R; r0 += 32) {
            if (a.R > 32) scan(r0);
            const uint32_t hit = __ballot_sync(0xffffffffu, before + (int64_t)upto * a.c.Hkv > first);
            if (hit) {
                const int l = __ffs(hit) - 1;
                r = r0 + l;
                len = __shfl_sync(0xffffffffu, n, l);
                units = __shfl_sync(0xffffffffu, mine, l);
                const int64_t at = first - before - (int64_t)__shfl_sync(0xffffffffu, upto - mine, l) * a.c.Hkv;
                head = static_cast<int>(at / units);
                unit = static_cast<int>(at - (int64_t)head * units);
                return;
            }
            before += (int64_t)__shfl_sync(0xffffffffu, upto, 31) * a.c.Hkv;
        }
    }
    // on to the next unit; true where it is another head's
    template <int ROWS>
    __device__ __forceinline__ bool next(const Args& a) {
        if (--left == 0 || ++unit < units) return false;
        unit = 0;
        if (++head < a.c.Hkv) return true;
        head = 0;
        do {
            ++r;
            len = UP_IN(r, a.R, a.status) ? a.seqused[r] : 0;
            units = units_of<ROWS>(a, len);
        } while (units == 0);                          // a unit is left, so a request with one follows
        return true;
    }
};

template <int DK, bool E4M3, bool MANY>
__global__ void __launch_bounds__(kThreads, (Shape<DK, E4M3>::kCtas)) mass_kernel(const __grid_constant__ Args a) {
    using S = Shape<DK, E4M3>;
    constexpr int NP = S::kPieces, NT = S::kTiles;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    Walk w{};
    w.seek<S::kRows>(a, (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5), (int64_t)gridDim.x * kWarps);
    Queries<DK, E4M3> q;
    bool fresh = true;
    while (w.left > 0) {
        const int p0 = w.unit * S::kRows;
        if (!MANY && fresh) q.load(a, w.r, w.head, 0);
        // rows 16 i + 8 j + g of the unit: keys, scale bytes
        uint4 x[NT][2][NP];
        float scale[NT][2];
        int64_t at[NT][2];                             // the row's records, -1 for none
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int pos = p0 + 16 * i + 8 * j + g;
                const int col = div_of(pos, a.by_b), tok = pos - col * a.by_b.d;
                const int64_t e = (int64_t)w.r * a.max_blocks + col;
                int page = -1;
                if (pos < w.len) {
                    page = UP_IN(e, (int64_t)a.R * a.max_blocks, a.status) ? a.table[e] : 0;
                    if (page < 0 || page >= a.c.num_blocks) {
                        set_status(a.status, UP_DEV_BAD_PAGE);
                        page = -1;
                    }
                }
                at[i][j] = page < 0 ? -1 : ((int64_t)page * a.c.Hkv + w.head) * a.by_b.d + tok;
                scale[i][j] = 1.f;
                const int64_t row = (int64_t)page * a.c.sb + w.head * a.c.sh + tok * a.c.st + 16 * t;
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    x[i][j][p] = make_uint4(0, 0, 0, 0);
                    if (page >= 0 && UP_IN(row + 64 * p, a.c.row_limit, a.status))
                        x[i][j][p] = *reinterpret_cast<const uint4*>(a.c.k + row + 64 * p);
                }
                if constexpr (E4M3) {
                    const int64_t sc = ((int64_t)page * a.c.Hkv + w.head) * a.c.Bp + tok;
                    if (page >= 0 && UP_IN(sc, a.c.scale_limit, a.status))
                        scale[i][j] = __uint_as_float(max(static_cast<uint32_t>(a.c.ks[sc]) << 23, 0x00400000u));       // 2^(b - 127)
                }
            }
        // lane t of four keeps the records of the rows (i, j) with 2 i + j = t mod 4
        constexpr int OWN = NT == 1 ? 1 : NT / 2;
        float old[OWN];
        const int from = a.counted ? a.counted[w.r] : w.len;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int pos = p0 + 16 * i + 8 * j + g;
                if (((2 * i + j) & 3) == t) {
                    old[(2 * i + j) / 4] = 0.f;
                    if (at[i][j] >= 0 && pos < from && a.decay != 0.f && UP_IN(at[i][j], a.records, a.status))
                        old[(2 * i + j) / 4] = a.mass[at[i][j]];
                }
            }
        float sum[NT][2];
#pragma unroll
        for (int i = 0; i < NT; ++i) sum[i][0] = sum[i][1] = 0.f;
        for (int h0 = 0; h0 < (MANY ? a.group : 1); h0 += 8) {
            if (MANY) q.load(a, w.r, w.head, h0);
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    const uint32_t* u = reinterpret_cast<const uint32_t*>(&x[i][0][p]);
                    const uint32_t* v = reinterpret_cast<const uint32_t*>(&x[i][1][p]);
                    if constexpr (E4M3) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t a0, a1, a2, a3;
                            kv::e4m3x4_to_f16x4(u[k], a0, a2);
                            kv::e4m3x4_to_f16x4(v[k], a1, a3);
                            mma<true>(d, a0, a1, a2, a3, q.b[4 * p + k][0], q.b[4 * p + k][1]);
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            mma<false>(d, u[2 * k], v[2 * k], u[2 * k + 1], v[2 * k + 1], q.b[2 * p + k][0], q.b[2 * p + k][1]);
                    }
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float y[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float z = d[2 * j + k] * scale[i][j];            // exact
                        const float e = fmaf(z, q.hi[k], -q.ref_hi[k]) + fmaf(z, q.lo[k], -q.ref_lo[k]);
                        y[k] = q.counts[k] ? ex2(e) : 0.f;
                    }
                    sum[i][j] += y[0] + y[1];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                sum[i][j] += __shfl_xor_sync(0xffffffffu, sum[i][j], 1);
                sum[i][j] += __shfl_xor_sync(0xffffffffu, sum[i][j], 2);
                const int pos = p0 + 16 * i + 8 * j + g;
                if (((2 * i + j) & 3) == t && at[i][j] >= 0 && UP_IN(at[i][j], a.records, a.status)) {
                    a.out[at[i][j]] = fmaf(a.decay, old[(2 * i + j) / 4], sum[i][j]);
                    if (pos >= from) a.born[at[i][j]] = (a.total ? a.total[w.r] : w.len) - w.len + pos;
                }
            }
        fresh = w.next<S::kRows>(a);
    }
}

template <int DK, bool E4M3, bool MANY>
static cudaError_t launch(const Args& a, cudaStream_t st) {
    const int64_t units = (int64_t)a.R * a.c.Hkv * cdiv((int64_t)a.max_blocks * a.c.B, Shape<DK, E4M3>::kRows);
    const int64_t ctas = std::min<int64_t>(units, (int64_t)Shape<DK, E4M3>::kCtas * num_sms());
    return launch_pdl(mass_kernel<DK, E4M3, MANY>, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), 0, st, a);
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
    const double scale = sm_scale * 1.4426950408889634;
    a.scale_hi = static_cast<float>(scale);
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
