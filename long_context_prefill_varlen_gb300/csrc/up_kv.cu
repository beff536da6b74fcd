// up_kv_write and up_kv_read: rows between a packed bf16 stream and the paged cache that up_slot_mapping's
// slots name (section 3.5, Eq. 16 of "UniPrefill: Universal Long-Context Prefill Acceleration via
// Block-wise Dynamic Sparsification", arXiv 2605.06221, gives the slots; the quantised form is this
// library's own).
//
// e4m3 rows: one power of two 2^e per row, the least with max|x| 2^-e <= 448 = 1.75 * 2^8.  For a bf16
// maximum of exponent field E and mantissa field M that is e + 127 = E - 8 + [M > 0x60] (1.75 has mantissa
// 0x60): (pattern + 0x1f) >> 7, less 8, of the row's largest bit pattern.  Scaling by a power of two is exact,
// so a code has one rounding, and reading back is exact: a scale that is not a power of two would round on
// both sides and take four bytes instead of one.
//
// Both kernels only move bytes (write: 2 dk in, dk + 1 or 2 dk out per row; read: the reverse): HBM-bound.  A
// warp takes units of 16 (or 4) tokens of one head: one coalesced load brings their slots, each lane places one
// token, and the tokens' scale bytes, neighbours in a page, leave (or come) in one access.  A row belongs to
// dk / 8 neighbouring lanes, 16 bytes of bf16 each, so that its maximum is a few shuffles; the warps of a CTA
// take the heads of the same tokens, so that they read or write whole tokens of the stream together.
// At 32K tokens of 8 heads of 128 in e4m3 the write takes 32.5 us (6.2 TB/s of what it must move, 0.92 of the
// measured copy rate) and the read 33.9 us (6.0 TB/s, 0.89); with bf16 rows both run at the copy rate (685K tokens written
// in 811 us, 6.9 TB/s).  What the e4m3 forms lack is issue slots: the write's instructions filled 65% of them before
// two rows' maxima shared a shuffle and the scaling moved to pairs of bf16 (35.4 us).
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "up_kv.cuh"

namespace up {
namespace kv {

// 128 threads, 64 registers: 1,024 threads on an SM with up to eight rows (or groups of rows) of 16 bytes in
// flight each.  Units of 16 tokens against 8 and 32 (before the maxima were paired): 35 / 38 / 41 us for a write of 32K
// tokens of 8 heads of 128 in e4m3, 214 / 222 / 218 for a read of 462K of 2 heads of 256.  A call too small to
// give every SM four warps that way takes units of 4: 1.9 against 3.0 us for 64 tokens.
constexpr int kThreads = 128, kCtas = 8;
constexpr int kChunk = 16, kSmallChunk = 4;      // tokens of a warp's unit
constexpr int kSmallWarps = 4;                   // warps of an SM below which units are small
constexpr int kGridPerSm = 32;                   // most CTAs of a side on an SM, where they come in waves
constexpr int kUnroll = 8;

struct Side {              // keys or values of a call
    const uint8_t* src;    // write: the stream; read: the cache
    uint8_t* dst;
    uint8_t* scale;
    int64_t stride;        // bytes from token to token of the stream
};

struct Args {
    Side side[2];
    Cache c;
    FastDiv by_b, by_heads;
    const int64_t* slots;
    int64_t T;
    const int32_t* num_tokens;
    int32_t* status;
};

// tokens of the call, -1 if the device's count is not in [0, T]
__device__ __forceinline__ int64_t token_count(const Args& a) {
    if (!a.num_tokens) return a.T;
    const int c = *a.num_tokens;
    if (c >= 0 && c <= a.T) return c;
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) set_status(a.status, UP_DEV_BAD_TOKEN_COUNT);
    return -1;
}

// page and token of a slot; false (with the status) for one outside the cache
__device__ __forceinline__ bool place(const Args& a, int64_t slot, int64_t* page, int* tok) {
    if (slot >= 0 && slot < (int64_t{1} << 31)) {
        const uint32_t p = div_of(static_cast<uint32_t>(slot), a.by_b);
        *page = p;
        *tok = static_cast<int>(static_cast<uint32_t>(slot) - p * a.by_b.d);
    } else if (slot >= 0) {
        *page = slot / a.c.B;
        *tok = static_cast<int>(slot - *page * a.c.B);
    } else {
        if (slot != -1) set_status(a.status, UP_DEV_BAD_SLOT);
        return false;
    }
    if (*page < a.c.num_blocks) return true;
    set_status(a.status, UP_DEV_BAD_SLOT);
    return false;
}

__device__ __forceinline__ float f_of(uint32_t bits) { return __uint_as_float(bits); }

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

// the larger half of a pair
__device__ __forceinline__ uint32_t top_half(uint32_t m) { return max(m & 0xffffu, m >> 16); }

// the largest of each half over the LPR lanes of a row: two rows' maxima travel together
template <int LPR>
__device__ __forceinline__ uint32_t row_max(uint32_t m) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}

__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// a pair of halves with every half that is infinite or NaN as zero (for the maximum) or as NaN
__device__ __forceinline__ uint32_t finite_or(uint32_t w, uint32_t other) {
    const uint32_t lo = (w & 0x7fffu) >= 0x7f80u ? (other & 0xffffu) : (w & 0xffffu);
    const uint32_t hi = ((w >> 16) & 0x7fffu) >= 0x7f80u ? (other & 0xffff0000u) : (w & 0xffff0000u);
    return lo | hi;
}

// The tokens of a unit: lane i holds where token i's row lies (element bytes and scale byte of head 0), -1 for none.
struct Place {
    int64_t row, scale;
};

__device__ __forceinline__ Place place_of(const Args& a, int64_t t, int64_t n) {
    Place p{-1, -1};
    int64_t page;
    int tok;
    if (t < n && UP_IN(t, a.T, a.status) && place(a, a.slots[t], &page, &tok)) {
        p.row = page * a.c.sb + tok * a.c.st;
        p.scale = page * a.c.Hkv * a.c.Bp + tok;
    }
    return p;
}

template <int DK, bool E4M3, int CHUNK>
__global__ void __launch_bounds__(kThreads, kCtas) write_kernel(const __grid_constant__ Args a) {
    constexpr int LPR = DK / 8, RPI = 32 / LPR, IT = CHUNK / RPI;      // lanes of a row, rows at a time, times
    constexpr int U = IT < kUnroll ? IT : kUnroll;
    pdl_wait();
    pdl_trigger();
    const int64_t n = token_count(a);
    if (n <= 0) return;
    const Side s = a.side[blockIdx.y];
    if (!s.src) return;
    const int lane = threadIdx.x & 31, sub = lane % LPR, grp = lane / LPR;
    const int64_t units = (n + CHUNK - 1) / CHUNK * a.c.Hkv, step = (int64_t)gridDim.x * (kThreads / 32);
    for (int64_t unit = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); unit < units; unit += step) {
        const int64_t chunk = unit < (int64_t{1} << 31) ? div_of(static_cast<uint32_t>(unit), a.by_heads) : unit / a.c.Hkv;
        const int head = static_cast<int>(unit - chunk * a.c.Hkv);
        const int64_t t0 = chunk * CHUNK;
        const Place pl = place_of(a, lane < CHUNK ? t0 + lane : n, n);
        const uint8_t* src = s.src + t0 * s.stride + (head * DK + sub * 8) * 2;
        int scale = 0;
#pragma unroll
        for (int i0 = 0; i0 < IT; i0 += U) {
            uint4 x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int j = (i0 + u) * RPI + grp;
                x[u] = t0 + j < n ? *reinterpret_cast<const uint4*>(src + j * s.stride) : make_uint4(0, 0, 0, 0);
            }
            uint32_t top[(U + 1) / 2];             // largest bit patterns of the rows, two a word
            if constexpr (E4M3) {
                auto maxima = [&](auto finite) {
                    uint32_t all = 0;
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        uint32_t m = 0;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t w = reinterpret_cast<const uint32_t*>(&x[u])[j];
                            m = max_u16x2(m, (decltype(finite)::value ? finite_or(w, 0) : w) & 0x7fff7fffu);
                        }
                        top[u / 2] = u & 1 ? top[u / 2] | (top_half(m) << 16) : top_half(m);
                    }
#pragma unroll
                    for (int u = 0; u < (U + 1) / 2; ++u) {
                        top[u] = row_max<LPR>(top[u]);
                        all = max_u16x2(all, top[u]);
                    }
                    return top_half(all);
                };
                if (__any_sync(0xffffffffu, maxima(std::false_type{}) >= 0x7f80u)) {       // rows with infinities or NaN
                    maxima(std::true_type{});
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t& w = reinterpret_cast<uint32_t*>(&x[u])[j];
                            w = finite_or(w, 0x7fff7fffu);
                        }
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t row = __shfl_sync(0xffffffffu, pl.row, (i0 + u) * RPI + grp);
                const int64_t at = row + head * a.c.sh + sub * (E4M3 ? 8 : 16);
                if constexpr (!E4M3) {
                    if (row >= 0 && UP_IN(at, a.c.row_limit, a.status)) *reinterpret_cast<uint4*>(s.dst + at) = x[u];
                } else {
                    const uint32_t m = u & 1 ? top[u / 2] >> 16 : top[u / 2] & 0xffffu;
                    const int e = static_cast<int>((m + 0x1fu) >> 7) - 8;          // E - 8 + [M > 0x60]
                    const int b = m == 0 ? 127 : max(e, 1);
                    const uint32_t inv = static_cast<uint32_t>(254 - b) * 0x800080u;       // 2^(127 - b), twice
                    uint32_t c[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        // a bf16 number times a power of two is exact down to 2^-126, far below the least code
                        uint32_t w;
                        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(w) : "r"(reinterpret_cast<const uint32_t*>(&x[u])[j]), "r"(inv));
                        c[j] = to_e4m3x2(f_of(w << 16), f_of(w & 0xffff0000u));
                    }
                    if (row >= 0 && UP_IN(at, a.c.row_limit, a.status))
                        *reinterpret_cast<uint2*>(s.dst + at) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
                    // to the lane of the row's token
                    const int v = __shfl_sync(0xffffffffu, b, (lane % RPI) * LPR);
                    if (lane / RPI == i0 + u) scale = v;
                }
            }
        }
        if constexpr (E4M3) {          // neighbouring tokens of a page: one run of bytes
            const int64_t at = pl.scale + head * a.c.Bp;
            if (lane < CHUNK && pl.row >= 0 && UP_IN(at, a.c.scale_limit, a.status)) s.scale[at] = static_cast<uint8_t>(scale);
        }
    }
}

// two f16 numbers that bf16 holds exactly, times a power of two (in both halves of `scale`), in bf16: one rounding
__device__ __forceinline__ uint32_t scaled_bf16x2(uint32_t h2, uint32_t scale) {
    float lo, hi;
    asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}" : "=f"(lo), "=f"(hi) : "r"(h2));
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(r), "r"(scale));
    return r;
}

template <int DK, bool E4M3, int CHUNK>
__global__ void __launch_bounds__(kThreads, kCtas) read_kernel(const __grid_constant__ Args a) {
    constexpr int LPR = DK / 8, RPI = 32 / LPR, IT = CHUNK / RPI;
    constexpr int U = IT < kUnroll ? IT : kUnroll;
    pdl_wait();
    pdl_trigger();
    const int64_t n = token_count(a);
    if (n <= 0) return;
    const Side s = a.side[blockIdx.y];
    if (!s.dst) return;
    const int lane = threadIdx.x & 31, sub = lane % LPR, grp = lane / LPR;
    const int64_t units = (n + CHUNK - 1) / CHUNK * a.c.Hkv, step = (int64_t)gridDim.x * (kThreads / 32);
    for (int64_t unit = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); unit < units; unit += step) {
        const int64_t chunk = unit < (int64_t{1} << 31) ? div_of(static_cast<uint32_t>(unit), a.by_heads) : unit / a.c.Hkv;
        const int head = static_cast<int>(unit - chunk * a.c.Hkv);
        const int64_t t0 = chunk * CHUNK;
        const Place pl = place_of(a, lane < CHUNK ? t0 + lane : n, n);
        uint32_t factor = 0;           // 2^(b - 127) of the lane's token in bf16, twice
        if constexpr (E4M3) {
            const int64_t at = pl.scale + head * a.c.Bp;
            if (lane < CHUNK && pl.row >= 0 && UP_IN(at, a.c.scale_limit, a.status))
                factor = max(static_cast<uint32_t>(s.scale[at]) * 0x800080u, 0x00400040u);
        }
        const int64_t dst = (t0 * a.c.Hkv + head) * DK + sub * 8;
#pragma unroll
        for (int i0 = 0; i0 < IT; i0 += U) {
            uint4 x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t row = __shfl_sync(0xffffffffu, pl.row, (i0 + u) * RPI + grp);
                const int64_t at = row + head * a.c.sh + sub * (E4M3 ? 8 : 16);
                x[u] = make_uint4(0, 0, 0, 0);
                if (row >= 0 && UP_IN(at, a.c.row_limit, a.status)) {
                    if constexpr (E4M3) {
                        const uint2 v = *reinterpret_cast<const uint2*>(s.src + at);
                        x[u].x = v.x;
                        x[u].y = v.y;
                    } else {
                        x[u] = *reinterpret_cast<const uint4*>(s.src + at);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int j = (i0 + u) * RPI + grp;
                const int64_t at = dst + (int64_t)j * a.c.Hkv * DK;
                if constexpr (E4M3) {
                    const uint32_t f = __shfl_sync(0xffffffffu, factor, j);
                    uint32_t h[4];
                    e4m3x4_to_f16x4(x[u].x, h[0], h[1]);
                    e4m3x4_to_f16x4(x[u].y, h[2], h[3]);
                    x[u] = make_uint4(scaled_bf16x2(h[0], f), scaled_bf16x2(h[1], f), scaled_bf16x2(h[2], f), scaled_bf16x2(h[3], f));
                }
                if (t0 + j < n && UP_IN(at, a.T * a.c.Hkv * DK, a.status)) *reinterpret_cast<uint4*>(s.dst + at * 2) = x[u];
            }
        }
    }
}

template <int DK, bool E4M3, int CHUNK>
static cudaError_t launch_one(const Args& a, bool write, cudaStream_t st) {
    const int64_t units = cdiv(a.T, CHUNK) * a.c.Hkv;
    // Reads of e4m3 rows of up to 128, whose units are one batch of loads, go by CTAs that stay: no start and no last wave
    // (32K tokens of 8 heads of 128: 36.3 -> 33.9 us, 131K 129 -> 124).  With two batches a unit (heads of 256: 215 -> 233),
    // and with bf16 rows (32K: 41.5 -> 45.0) or a write's maxima (131K: 117 -> 132), waves keep more loads in flight.
    const int sides = (a.side[0].dst != nullptr) + (a.side[1].dst != nullptr);
    const int per_sm = !write && E4M3 && DK <= 128 ? kCtas / sides : kGridPerSm;
    const dim3 g(static_cast<unsigned>(std::min<int64_t>(cdiv(units, kThreads / 32), per_sm * num_sms())), 2);
    return write ? launch_pdl(write_kernel<DK, E4M3, CHUNK>, g, dim3(kThreads), 0, st, a)
                 : launch_pdl(read_kernel<DK, E4M3, CHUNK>, g, dim3(kThreads), 0, st, a);
}

template <int DK>
static cudaError_t launch_dk(const Args& a, bool write, bool e4m3, cudaStream_t st) {
    const bool small = 2 * cdiv(a.T, kChunk) * a.c.Hkv < kSmallWarps * num_sms();
    if (e4m3) return small ? launch_one<DK, true, kSmallChunk>(a, write, st) : launch_one<DK, true, kChunk>(a, write, st);
    return small ? launch_one<DK, false, kSmallChunk>(a, write, st) : launch_one<DK, false, kChunk>(a, write, st);
}

static up_status launch(const Args& a, bool write, int dk, int format, cudaStream_t st) {
    const bool e4m3 = format == UP_KV_E4M3;
    const cudaError_t e = dk == 64 ? launch_dk<64>(a, write, e4m3, st) : dk == 128 ? launch_dk<128>(a, write, e4m3, st)
                                                                                    : launch_dk<256>(a, write, e4m3, st);
    if (e != cudaSuccess) return failed_launch();
    count_launch();
    return check_launch();
}

}  // namespace kv
}  // namespace up

using namespace up;

extern "C" int up_kv_scale_row(int B) { return kv::scale_row(B); }

extern "C" up_status up_kv_write(const up_kv_cache* cache, const uint16_t* k, int64_t k_stride, const uint16_t* v,
                                 int64_t v_stride, const int64_t* slots, int64_t T, const int32_t* num_tokens,
                                 int32_t* dev_status, void* stream) {
    kv::Args a{};
    if (!dev_status || T < 0) return UP_ERR_ARG;
    const up_status s = kv::check(cache, &a.c);
    if (s != UP_OK) return s;
    if (T == 0 || (!k && !v)) return UP_OK;
    if (!slots) return UP_ERR_ARG;
    const int64_t row = static_cast<int64_t>(cache->Hkv) * cache->dk;
    if ((k && (!aligned16(k) || k_stride % 8)) || (v && (!aligned16(v) || v_stride % 8))) return UP_ERR_SHAPE;
    if (T > 1 && ((k && k_stride < row) || (v && v_stride < row))) return UP_ERR_SHAPE;
    a.side[0] = {reinterpret_cast<const uint8_t*>(k), static_cast<uint8_t*>(cache->k), cache->k_scale, k_stride * 2};
    a.side[1] = {reinterpret_cast<const uint8_t*>(v), static_cast<uint8_t*>(cache->v), cache->v_scale, v_stride * 2};
    a.by_b = kv::fast_div(cache->B);
    a.by_heads = kv::fast_div(cache->Hkv);
    a.slots = slots;
    a.T = T;
    a.num_tokens = num_tokens;
    a.status = dev_status;
    return kv::launch(a, true, cache->dk, cache->format, static_cast<cudaStream_t>(stream));
}

extern "C" up_status up_kv_read(const up_kv_cache* cache, const int64_t* slots, int64_t T, const int32_t* num_tokens,
                                uint16_t* k, uint16_t* v, int32_t* dev_status, void* stream) {
    kv::Args a{};
    if (!dev_status || T < 0) return UP_ERR_ARG;
    const up_status s = kv::check(cache, &a.c);
    if (s != UP_OK) return s;
    if (T == 0 || (!k && !v)) return UP_OK;
    if (!slots) return UP_ERR_ARG;
    if (!aligned16(k) || !aligned16(v)) return UP_ERR_SHAPE;
    a.side[0] = {static_cast<const uint8_t*>(cache->k), reinterpret_cast<uint8_t*>(k), cache->k_scale, 0};
    a.side[1] = {static_cast<const uint8_t*>(cache->v), reinterpret_cast<uint8_t*>(v), cache->v_scale, 0};
    a.by_b = kv::fast_div(cache->B);
    a.by_heads = kv::fast_div(cache->Hkv);
    a.slots = slots;
    a.T = T;
    a.num_tokens = num_tokens;
    a.status = dev_status;
    return kv::launch(a, false, cache->dk, cache->format, static_cast<cudaStream_t>(stream));
}
