// The paged key-value cache as the kernels see it, and the checks that its entry points share.
#pragma once

#include "up_internal.cuh"

namespace up {
namespace kv {

struct Cache {
    const uint8_t* k;
    const uint8_t* v;
    const uint8_t* ks;
    const uint8_t* vs;
    int64_t num_blocks;
    int64_t sb, sh, st;        // strides in bytes
    int64_t row_limit;         // bytes from k (v) to the end of the furthest row
    int64_t scale_limit;       // scale bytes of k (v)
    int Hkv, B, Bp;            // Bp: scale bytes of a page and head
};

// floor(x / d) for 0 <= x < 2^31, 1 <= d < 2^31: the quotient of x by d is the high word of x * m shifted
// by s, m = ceil(2^(32+s) / d), s = ceil(log2 d) - 1 (Granlund & Montgomery, "Division by invariant
// integers using multiplication", 1994, section 4: exact since m * d - 2^(32+s) <= 2^(s+1), x < 2^31).
struct FastDiv {
    uint32_t d, m, s;
};
inline FastDiv fast_div(uint32_t d) {
    FastDiv f{d, 0, 0};
    if (d > 1) {
        uint32_t l = 0;
        while ((1ull << l) < d) ++l;
        f.s = l - 1;
        f.m = static_cast<uint32_t>(((1ull << (32 + f.s)) + d - 1) / d);
    }
    return f;
}
__device__ __forceinline__ uint32_t div_of(uint32_t x, const FastDiv& f) {
    return f.d == 1 ? x : __umulhi(x, f.m) >> f.s;
}

inline int scale_row(int B) { return B > 0 ? static_cast<int>(align_up(static_cast<size_t>(B), 16)) : 0; }
inline int element_bytes(int format) { return format == UP_KV_E4M3 ? 1 : 2; }

// the host-side checks of a cache
inline up_status check(const up_kv_cache* c, Cache* out) {
    if (!c || !c->k || !c->v) return UP_ERR_ARG;
    if (c->format != UP_KV_BF16 && c->format != UP_KV_E4M3) return UP_ERR_ARG;
    if (c->num_blocks <= 0 || c->Hkv <= 0 || c->B <= 0 || c->B > (1 << 20)) return UP_ERR_ARG;
    if (c->num_blocks > (int64_t{1} << 31) - 1) return UP_ERR_ARG;
    if (c->dk != 64 && c->dk != 128 && c->dk != 256) return UP_ERR_SHAPE;
    const int e = element_bytes(c->format);
    if (!aligned16(c->k) || !aligned16(c->v)) return UP_ERR_SHAPE;
    // the stride of an axis of one entry is never used
    const int64_t stride[3] = {c->num_blocks > 1 ? c->stride_block : 16, c->Hkv > 1 ? c->stride_head : 16,
                               c->B > 1 ? c->stride_token : 16};
    for (int64_t s : stride)
        if (s <= 0 || s * e % 16) return UP_ERR_SHAPE;
    if (c->format == UP_KV_E4M3) {
        if (!c->k_scale || !c->v_scale) return UP_ERR_ARG;
        if (!aligned16(c->k_scale) || !aligned16(c->v_scale)) return UP_ERR_SHAPE;
    }
    out->k = static_cast<const uint8_t*>(c->k);
    out->v = static_cast<const uint8_t*>(c->v);
    out->ks = c->k_scale;
    out->vs = c->v_scale;
    out->num_blocks = c->num_blocks;
    out->sb = stride[0] * e;
    out->sh = stride[1] * e;
    out->st = stride[2] * e;
    out->Hkv = c->Hkv;
    out->B = c->B;
    out->Bp = scale_row(c->B);
    out->row_limit = (c->num_blocks - 1) * out->sb + (c->Hkv - 1) * out->sh + (c->B - 1) * out->st + c->dk * e;
    out->scale_limit = c->num_blocks * c->Hkv * out->Bp;
    return UP_OK;
}

// four e4m3 codes (low byte first) to f16, the lower two and the upper two: exact, NaN kept
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(codes));
}

}  // namespace kv
}  // namespace up
