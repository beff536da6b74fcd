// up_rope: rotary positions of the queries and keys of a packed stream (the rotated Q and K that up_score_blocks
// and the cache take; a drop's kept tokens keep their own positions, section 3.5 of "UniPrefill: Universal
// Long-Context Prefill Acceleration via Block-wise Dynamic Sparsification", arXiv 2605.06221), and its gradient.
//
// Pair j of a head turns by x = pos * f_j.  What counts of x is its place within a turn, so the angle is computed as
// turns in 64-bit fixed point: pos * turns_j modulo 2^64, one integer product whose wrap drops the whole turns, for any
// position and sign; the table's last bit leaves |pos| 2^-65 turn.  The upper 32 bits, as a signed number, are the angle in
// [-pi, pi), rounded to the 24 bits of a float for the sine and cosine (pi 2^-24 at most, far below bf16's steps).  With 32-bit
// floats throughout, a position of 100,000 leaves the angles of pairs next to the fastest some 2^-8 off.
//
// The kernel moves bytes (4 dk a row of a head) and HBM bounds it: a thread owns 8 pairs of a token (two 16-byte vectors
// rot/2 numbers apart, in either layout), finds their sines once and turns the pairs of several heads with them, all of
// their loads in flight.  Measured (one GB300, 6.79 TB/s measured copy): 32,513 tokens of 40 heads of 128 97.6 us, 6.8 TB/s; 524,288 of
// 18 heads of 256, a quarter of each turned and the rest copied, 1,393 us, 6.9 TB/s; one token 2.0 us in a replayed graph, the launch (8.9 called from
// Python).  What a partial turn leaves alone is copied in place, too, where nothing would have to move.
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "up_internal.cuh"

namespace up {
namespace rope {

constexpr int kThreads = 128;
constexpr int kUnroll = 4;           // heads in flight
// Heads that a thread turns with the sines it has found: as many of 8, 4, 2 and 1 as leave every SM 64 warps.
constexpr int kHeads = 8;

struct Side {
    const uint16_t* in;
    uint16_t* out;
    int64_t stride, out_stride;      // elements
    int heads;
};

struct Args {
    Side q, k;
    const int64_t* positions;
    int64_t T;
    const int32_t* num_tokens;
    int32_t* status;
    int slice, slices;               // heads of a thread, and threads of a token's heads
    int transpose;
    up_rope_table plan;
};

__device__ __forceinline__ float low_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Eight pairs in two vectors: numbers i of each (halves), or numbers 2i, 2i + 1 of the first and then of the second (pairs).
template <bool PAIRS>
__device__ __forceinline__ void turn(uint4& x, uint4& y, const float (&c)[8], const float (&s)[8]) {
    uint32_t* a = reinterpret_cast<uint32_t*>(&x);
    uint32_t* b = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a0 = low_of(a[i]), a1 = high_of(a[i]), b0 = low_of(b[i]), b1 = high_of(b[i]);
        if constexpr (PAIRS) {
            a[i] = bf16x2(a0 * c[i] - a1 * s[i], a1 * c[i] + a0 * s[i]);
            b[i] = bf16x2(b0 * c[4 + i] - b1 * s[4 + i], b1 * c[4 + i] + b0 * s[4 + i]);
        } else {
            a[i] = bf16x2(a0 * c[2 * i] - b0 * s[2 * i], a1 * c[2 * i + 1] - b1 * s[2 * i + 1]);
            b[i] = bf16x2(b0 * c[2 * i] + a0 * s[2 * i], b1 * c[2 * i + 1] + a1 * s[2 * i + 1]);
        }
    }
}

template <int DK, bool PAIRS>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ Args a) {
    constexpr int LPR = DK / 16, TPW = 32 / LPR;       // threads of a head's row, tokens of a warp
    __shared__ uint64_t turns[UP_ROPE_MAX_PAIRS];
    for (int i = threadIdx.x; i < a.plan.rot / 2; i += kThreads) turns[i] = a.plan.turns[i];
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    int64_t n = a.T;
    if (a.num_tokens) {
        n = *a.num_tokens;
        if (n < 0 || n > a.T) {
            if (blockIdx.x == 0 && threadIdx.x == 0) set_status(a.status, UP_DEV_BAD_TOKEN_COUNT);
            return;
        }
    }
    const int lane = threadIdx.x & 31, job = lane % LPR, jobs = a.plan.rot / 16;
    const int64_t item = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t group = item / a.slices, t = group * TPW + lane / LPR;
    if (t >= n || !UP_IN(t, a.T, a.status)) return;
    // the two vectors of the thread, and how far apart
    const bool turns_here = job < jobs;
    const int at = turns_here ? 8 * job : a.plan.rot + 8 * (job - jobs), apart = turns_here ? a.plan.rot / 2 : (DK - a.plan.rot) / 2;
    float c[8], s[8];
    if (turns_here) {
        const uint64_t pos = static_cast<uint64_t>(a.positions[t]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int pair = PAIRS ? 4 * job + (i & 3) + (i >> 2) * (a.plan.rot / 4) : 8 * job + i;
            const uint64_t x = pos * turns[pair];
            sincospif(static_cast<float>(static_cast<int32_t>(x >> 32)) * 0x1p-31f, &s[i], &c[i]);
            c[i] *= a.plan.gain;
            s[i] *= a.transpose ? -a.plan.gain : a.plan.gain;
        }
    }
    const int first = static_cast<int>(item - group * a.slices) * a.slice, heads = a.q.heads + a.k.heads;
    const int last = min(first + a.slice, heads);
    const uint16_t* const q = a.q.in + t * a.q.stride + at;
    const uint16_t* const k = a.k.in + t * a.k.stride + at;
    uint16_t* const qo = a.q.out + t * a.q.out_stride + at;
    uint16_t* const ko = a.k.out + t * a.k.out_stride + at;
    for (int h0 = first; h0 < last; h0 += kUnroll) {
        uint4 x[kUnroll], y[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int h = h0 + u;
            if (h < last) {
                const uint16_t* p = h < a.q.heads ? q + h * DK : k + (h - a.q.heads) * DK;
                x[u] = *reinterpret_cast<const uint4*>(p);
                y[u] = *reinterpret_cast<const uint4*>(p + apart);
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int h = h0 + u;
            if (h < last) {
                uint16_t* p = h < a.q.heads ? qo + h * DK : ko + (h - a.q.heads) * DK;
                if (turns_here) turn<PAIRS>(x[u], y[u], c, s);
                *reinterpret_cast<uint4*>(p) = x[u];
                *reinterpret_cast<uint4*>(p + apart) = y[u];
            }
        }
    }
}

template <int DK>
static cudaError_t launch(const Args& a, int64_t ctas, cudaStream_t st) {
    const dim3 g(static_cast<unsigned>(ctas));
    return a.plan.layout == UP_ROPE_PAIRS ? launch_pdl(rope_kernel<DK, true>, g, dim3(kThreads), 0, st, a)
                                          : launch_pdl(rope_kernel<DK, false>, g, dim3(kThreads), 0, st, a);
}

// a side's checks; a side without an input has no heads
static up_status check(const uint16_t* in, int64_t stride, uint16_t* out, int64_t out_stride, int heads, int dk, int64_t T, Side* s) {
    *s = Side{in, out, stride, out_stride, in ? heads : 0};
    if (!in && !out) return UP_OK;
    if (!in || !out || heads <= 0) return UP_ERR_ARG;
    if (!aligned16(in) || !aligned16(out) || stride % 8 || out_stride % 8) return UP_ERR_SHAPE;
    const int64_t row = (int64_t)heads * dk;
    if (T > 1 && (stride < row || out_stride < row)) return UP_ERR_SHAPE;
    if (in == out && T > 1 && stride != out_stride) return UP_ERR_SHAPE;
    return UP_OK;
}

}  // namespace rope
}  // namespace up

using namespace up;

extern "C" up_status up_rope_plan(int rot, double theta, int layout, int scaling, double factor, double original_len,
                                  double low, double high, double gain, up_rope_table* plan) {
    if (!plan) return UP_ERR_ARG;
    if (layout != UP_ROPE_HALVES && layout != UP_ROPE_PAIRS) return UP_ERR_ARG;
    if (scaling < UP_ROPE_PLAIN || scaling > UP_ROPE_RAMP) return UP_ERR_ARG;
    if (!(theta > 1 && theta <= 1e300) || !(gain >= 0 && gain < INFINITY)) return UP_ERR_ARG;
    if (scaling != UP_ROPE_PLAIN && !(factor >= 1 && factor < INFINITY)) return UP_ERR_ARG;
    const bool bands = scaling == UP_ROPE_BANDS, ramp = scaling == UP_ROPE_RAMP;
    if ((bands || ramp) && !(original_len > 0 && original_len < INFINITY && low > 0 && low < high && high < INFINITY)) return UP_ERR_ARG;
    if (rot <= 0 || rot % 16 || rot > 2 * UP_ROPE_MAX_PAIRS) return UP_ERR_SHAPE;
    const double two_pi = 6.283185307179586476925286766559;
    *plan = up_rope_table{};
    plan->rot = rot;
    plan->layout = layout;
    plan->gain = static_cast<float>(gain > 0 ? gain : ramp ? 1 + log(factor) / 10 : 1);
    const auto index = [&](double turns) { return rot * log(original_len / (two_pi * turns)) / (2 * log(theta)); };
    const double a = ramp ? std::max(floor(index(high)), 0.0) : 0;
    const double b = ramp ? std::max(std::min(ceil(index(low)), rot - 1.0), a + 0.001) : 1;
    for (int j = 0; j < rot / 2; ++j) {
        const double plain = pow(theta, -2.0 * j / rot), u = plain * original_len / two_pi;
        double f = plain;
        if (scaling == UP_ROPE_LINEAR) f = plain / factor;
        if (bands || ramp) {
            const double x = std::min(1.0, std::max(0.0, bands ? (u - low) / (high - low) : (b - j) / (b - a)));
            f = (1 - x) * plain / factor + x * plain;
        }
        plan->turns[j] = static_cast<uint64_t>(ldexp(f / two_pi, 64) + 0.5);
    }
    return UP_OK;
}

extern "C" up_status up_rope(const up_rope_table* plan, const uint16_t* q, int64_t q_stride, uint16_t* q_out,
                             int64_t q_out_stride, int Hq, const uint16_t* k, int64_t k_stride, uint16_t* k_out,
                             int64_t k_out_stride, int Hkv, int dk, const int64_t* positions, int64_t T,
                             const int32_t* num_tokens, int transpose, int32_t* dev_status, void* stream) {
    if (!plan || !dev_status || T < 0) return UP_ERR_ARG;
    if (plan->layout != UP_ROPE_HALVES && plan->layout != UP_ROPE_PAIRS) return UP_ERR_ARG;
    if (dk != 64 && dk != 128 && dk != 256) return UP_ERR_SHAPE;
    if (plan->rot <= 0 || plan->rot % 16 || plan->rot > dk) return UP_ERR_SHAPE;
    rope::Args a{};
    up_status s = rope::check(q, q_stride, q_out, q_out_stride, Hq, dk, T, &a.q);
    if (s == UP_OK) s = rope::check(k, k_stride, k_out, k_out_stride, Hkv, dk, T, &a.k);
    if (s != UP_OK) return s;
    const int64_t heads = (int64_t)a.q.heads + a.k.heads;
    if (heads * dk > 0x7fffffff) return UP_ERR_SHAPE;
    if (T == 0 || heads == 0) return UP_OK;
    if (!positions) return UP_ERR_ARG;
    a.positions = positions;
    a.T = T;
    a.num_tokens = num_tokens;
    a.status = dev_status;
    a.transpose = transpose;
    a.plan = *plan;
    const int64_t groups = cdiv(T, 32 / (dk / 16));
    a.slice = rope::kHeads;
    while (a.slice > 1 && groups * cdiv(heads, a.slice) < 64 * num_sms()) a.slice /= 2;
    a.slices = static_cast<int>(cdiv(heads, a.slice));
    const int64_t ctas = cdiv(groups * a.slices, rope::kThreads / 32);
    if (ctas > 0x7fffffff) return UP_ERR_SHAPE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dk == 64    ? rope::launch<64>(a, ctas, st)
                          : dk == 128 ? rope::launch<128>(a, ctas, st)
                                      : rope::launch<256>(a, ctas, st);
    if (e != cudaSuccess) return failed_launch();
    count_launch();
    return check_launch();
}
