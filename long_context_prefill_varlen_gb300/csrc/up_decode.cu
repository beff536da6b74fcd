// up_paged_decode: attention of one new token per request over its pages of the key-value cache, with the
// lengths that the drop history leaves each layer (up_seqused, section 3.5, Eq. 17 of "UniPrefill:
// Universal Long-Context Prefill Acceleration via Block-wise Dynamic Sparsification", arXiv 2605.06221).
//
// The positions [lo, len) of a request are cut into tiles of kTile rows (whole pages, or parts of one
// page) and the tiles into chunks, by the request's own length alone.  Each (request, KV head, chunk) gives
// for each query head of the group
//   lse2 = log2 sum_i 2^(s_i)   and   o = sum_i 2^(s_i - lse2) v_i,   s_i = q . k_i * sm_scale * log2 e
// and the join adds the chunks in order: out = sum_c 2^(lse2_c - L) o_c, L = log2 sum_c 2^(lse2_c).
#include <stdint.h>

#include <algorithm>

#include "up_kv.cuh"

namespace up {
namespace decode {

using kv::Cache;

constexpr int kTile = 64;            // rows of a tile
constexpr int kMinTiles = 4;         // a chunk holds at least this many tiles, if the request has them
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// How the positions of a request fall into segments (a page, or up to kTile rows of one), tiles of spt
// segments, and chunks of tiles.
struct Cut {
    int B, seg, spp, spt;      // page; rows of a segment; segments of a page; segments of a tile
    int window, s0;            // s0: chunks that spread one request's heads evenly over the grid
    int max_splits;
};

struct Range {
    int len, lo;               // positions [lo, len)
    int seg0, tiles, splits;   // first segment; tiles from there; chunks
};

__host__ __device__ inline int splits_of(int tiles, int s0) {
    const int by_min = (tiles + kMinTiles - 1) / kMinTiles;
    return by_min < s0 ? by_min : s0;
}

__device__ __forceinline__ Range range_of(const Cut& c, int len, int64_t cap) {
    Range r;
    r.len = len < 0 || len > cap ? 0 : len;
    r.lo = c.window > 0 && r.len > c.window ? r.len - c.window : 0;
    const int p0 = r.lo / c.B, p1 = r.len > 0 ? (r.len - 1) / c.B : 0;
    r.seg0 = p0 * c.spp + (r.lo - p0 * c.B) / c.seg;
    const int seg1 = p1 * c.spp + (r.len > 0 ? (r.len - 1 - p1 * c.B) / c.seg : 0);
    r.tiles = r.len > r.lo ? (seg1 - r.seg0) / c.spt + 1 : 0;
    r.splits = splits_of(r.tiles, c.s0);
    return r;
}

// 2^(x - m), and 0 for x = -inf whatever m is (m is the largest of a set that x belongs to; NaN stays)
__device__ __forceinline__ float weight(float x, float m) { return x == -INFINITY ? 0.f : exp2f(x - m); }

struct Args {
    const uint8_t* q;
    int64_t q_stride;          // bytes
    Cache c;
    const int32_t* table;
    const int32_t* seqused;
    int R, max_blocks, Hq, group;
    float scale2;              // sm_scale * log2 e
    Cut cut;
    float* part_lse;           // [R, Hq, max_splits]
    float* part_o;             // [R, Hq, max_splits, dk]
    uint16_t* out;
    float* lse;
    int32_t* status;
};

// ------------------------------------------------------------------------------------------------
// one CTA per (chunk, KV head, request): a warp per row, lanes over dk

template <int DK, bool E4M3>
__global__ void __launch_bounds__(128) chunk_kernel(const __grid_constant__ Args a) {
    pdl_wait();
    pdl_trigger();
    constexpr int E = DK / 32;
    const int r = blockIdx.z, h = blockIdx.y, ch = blockIdx.x, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t cap = (int64_t)a.max_blocks * a.cut.B;
    const int len_in = a.seqused[r];
    if ((len_in < 0 || len_in > cap) && threadIdx.x == 0) set_status(a.status, UP_DEV_BAD_LENGTH);
    const Range g = range_of(a.cut, len_in, cap);
    if (ch >= g.splits) return;
    const int t0 = (int)((int64_t)ch * g.tiles / g.splits), t1 = (int)((int64_t)(ch + 1) * g.tiles / g.splits);
    __shared__ float sm_m[4], sm_l[4], sm_o[4][DK];
    for (int j = 0; j < a.group; ++j) {
        const int hq = h * a.group + j;
        float q[E], o[E];
        for (int e = 0; e < E; ++e) {
            const uint16_t bits = reinterpret_cast<const uint16_t*>(a.q + r * a.q_stride)[hq * DK + lane * E + e];
            q[e] = __uint_as_float((uint32_t)bits << 16);
            o[e] = 0.f;
        }
        float m = -INFINITY, l = 0.f;
        for (int row = t0 * a.cut.spt * a.cut.seg + w; row < t1 * a.cut.spt * a.cut.seg; row += 4) {
            const int s = g.seg0 + row / a.cut.seg, off = row % a.cut.seg;
            const int page_i = s / a.cut.spp, tok = (s % a.cut.spp) * a.cut.seg + off;
            const int64_t pos = (int64_t)page_i * a.cut.B + tok;
            if (tok >= a.cut.B || pos < g.lo || pos >= g.len) continue;
            const int page = a.table[(int64_t)r * a.max_blocks + page_i];
            const bool ok = page >= 0 && page < a.c.num_blocks;
            if (!ok && lane == 0) set_status(a.status, UP_DEV_BAD_PAGE);
            float k[E], v[E];
            for (int e = 0; e < E; ++e) k[e] = v[e] = 0.f;
            if (ok) {
                const int64_t at = (int64_t)page * a.c.sb + h * a.c.sh + (int64_t)tok * a.c.st;
                if constexpr (E4M3) {
                    const int64_t sc = ((int64_t)page * a.c.Hkv + h) * a.c.Bp + tok;
                    const float fk = exp2f((float)a.c.ks[sc] - 127.f), fv = exp2f((float)a.c.vs[sc] - 127.f);
                    for (int e = 0; e < E; ++e) {
                        const uint32_t ck = kv::e4m3x2_to_f16x2(a.c.k[at + lane * E + e]);
                        const uint32_t cv = kv::e4m3x2_to_f16x2(a.c.v[at + lane * E + e]);
                        float x, y;
                        asm("{\n\t.reg .f16 p, q;\n\tmov.b32 {p, q}, %1;\n\tcvt.f32.f16 %0, p;\n\t}" : "=f"(x) : "r"(ck));
                        asm("{\n\t.reg .f16 p, q;\n\tmov.b32 {p, q}, %1;\n\tcvt.f32.f16 %0, p;\n\t}" : "=f"(y) : "r"(cv));
                        k[e] = x * fk;
                        v[e] = y * fv;
                    }
                } else {
                    for (int e = 0; e < E; ++e) {
                        k[e] = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(a.c.k + at)[lane * E + e] << 16);
                        v[e] = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(a.c.v + at)[lane * E + e] << 16);
                    }
                }
            }
            float d = 0.f;
            for (int e = 0; e < E; ++e) d += q[e] * k[e];
            for (int x = 16; x > 0; x >>= 1) d += __shfl_xor_sync(0xffffffffu, d, x);
            d *= a.scale2;
            const float mn = fmaxf(m, d), c0 = weight(m, mn), p = weight(d, mn);
            l = l * c0 + p;
            for (int e = 0; e < E; ++e) o[e] = o[e] * c0 + p * v[e];
            m = mn;
        }
        __syncthreads();
        if (lane == 0) {
            sm_m[w] = m;
            sm_l[w] = l;
        }
        for (int e = 0; e < E; ++e) sm_o[w][lane * E + e] = o[e];
        __syncthreads();
        const float M = fmaxf(fmaxf(sm_m[0], sm_m[1]), fmaxf(sm_m[2], sm_m[3]));
        float L = 0.f;
        for (int i = 0; i < 4; ++i) L += weight(sm_m[i], M) * sm_l[i];
        const int64_t part = ((int64_t)r * a.Hq + hq) * a.cut.max_splits + ch;
        if (threadIdx.x == 0) a.part_lse[part] = M == -INFINITY && L == 0.f ? -INFINITY : M + log2f(L);
        for (int d = threadIdx.x; d < DK; d += 128) {
            float x = 0.f;
            for (int i = 0; i < 4; ++i) x += weight(sm_m[i], M) * sm_o[i][d];
            a.part_o[part * DK + d] = M == -INFINITY && L == 0.f ? 0.f : x / L;
        }
    }
}

// ------------------------------------------------------------------------------------------------
// one CTA per (query head, request): the chunks of a row, in order

template <int DK>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ Args a) {
    pdl_wait();
    pdl_trigger();
    const int hq = blockIdx.x, r = blockIdx.y;
    const int64_t row = (int64_t)r * a.Hq + hq;
    const Range g = range_of(a.cut, a.seqused[r], (int64_t)a.max_blocks * a.cut.B);
    const float* pl = a.part_lse + row * a.cut.max_splits;
    const float* po = a.part_o + row * a.cut.max_splits * DK;
    float m = -INFINITY;
    for (int i = 0; i < g.splits; ++i) m = fmaxf(m, pl[i]);
    float l = 0.f;
    for (int i = 0; i < g.splits; ++i) l += weight(pl[i], m);
    for (int d = threadIdx.x; d < DK; d += 128) {
        float x = 0.f;
        for (int i = 0; i < g.splits; ++i) x += weight(pl[i], m) * po[(int64_t)i * DK + d];
        x = l == 0.f ? 0.f : x / l;
        uint32_t b;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(b) : "f"(0.f), "f"(x));
        a.out[row * DK + d] = static_cast<uint16_t>(b);
    }
    if (a.lse && threadIdx.x == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// ------------------------------------------------------------------------------------------------
// host side

// 0 for arguments that the call refuses
static int make_cut(int R, int Hq, int Hkv, int dk, int B, int max_blocks, int window, Cut* c) {
    if (R <= 0 || R > 65535 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || Hq > 65535 || B <= 0 || B > (1 << 20)) return 0;
    if (max_blocks <= 0 || window < 0) return 0;
    if (dk != 64 && dk != 128 && dk != 256) return 0;
    if ((int64_t)max_blocks * B > 0x7fffffff - 2 * kTile) return 0;
    c->B = B;
    c->seg = B < kTile ? B : kTile;
    c->spp = static_cast<int>(cdiv(B, kTile));
    c->spt = kTile / c->seg;
    c->window = window;
    int s0 = num_sms();
    for (int h = Hkv; s0 % 2 == 0 && h % 2 == 0; h /= 2) s0 /= 2;
    c->s0 = s0;
    int64_t segs = (int64_t)max_blocks * c->spp;
    if (window > 0) segs = std::min<int64_t>(segs, (cdiv(window, B) + 1) * (int64_t)c->spp);
    c->max_splits = splits_of(static_cast<int>(cdiv(segs, c->spt)), s0);
    return 1;
}

}  // namespace decode
}  // namespace up

using namespace up;

extern "C" size_t up_paged_decode_workspace_bytes(int R, int Hq, int Hkv, int dk, int B, int max_blocks, int window) {
    decode::Cut c{};
    if (!decode::make_cut(R, Hq, Hkv, dk, B, max_blocks, window, &c)) return 0;
    const size_t parts = static_cast<size_t>(R) * Hq * c.max_splits;
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
    if (!make_cut(R, Hq, cache->Hkv, cache->dk, cache->B, max_blocks, window, &a.cut)) return UP_ERR_SHAPE;
    if (!aligned16(q) || !aligned16(out) || q_stride % 8 || (R > 1 && q_stride < (int64_t)Hq * cache->dk)) return UP_ERR_SHAPE;
    if (ws_bytes < up_paged_decode_workspace_bytes(R, Hq, cache->Hkv, cache->dk, cache->B, max_blocks, window) ||
        !aligned16(ws))
        return UP_ERR_WORKSPACE;
    const size_t parts = static_cast<size_t>(R) * Hq * a.cut.max_splits;
    a.q = reinterpret_cast<const uint8_t*>(q);
    a.q_stride = q_stride * 2;
    a.table = block_table;
    a.seqused = seqused;
    a.R = R;
    a.max_blocks = max_blocks;
    a.Hq = Hq;
    a.group = Hq / cache->Hkv;
    a.scale2 = sm_scale * kLog2e;
    a.part_lse = static_cast<float*>(ws);
    a.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + align_up(parts * sizeof(float), 256));
    a.out = out;
    a.lse = lse;
    a.status = dev_status;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const dim3 g(a.cut.max_splits, cache->Hkv, R), gj(Hq, R), b(128);
    const bool f8 = cache->format == UP_KV_E4M3;
    cudaError_t e = cudaErrorInvalidValue;
#define UP_DECODE_CASE(DK)                                                                                   \
    case DK:                                                                                                 \
        e = f8 ? launch_pdl(chunk_kernel<DK, true>, g, b, 0, st, a) : launch_pdl(chunk_kernel<DK, false>, g, b, 0, st, a); \
        if (e == cudaSuccess) e = launch_pdl(join_kernel<DK>, gj, b, 0, st, a);                              \
        break
    switch (cache->dk) {
        UP_DECODE_CASE(64);
        UP_DECODE_CASE(128);
        UP_DECODE_CASE(256);
        default: return UP_ERR_SHAPE;
    }
#undef UP_DECODE_CASE
    if (e != cudaSuccess) return UP_ERR_CUDA;
    count_launch(2);
    return check_launch();
}
