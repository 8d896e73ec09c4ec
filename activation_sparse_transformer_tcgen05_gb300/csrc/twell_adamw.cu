// twell_adamw.cu — one AdamW step over many tensors, states in 32 or in 8 bits.
//
//   c = norm > max_norm ? max_norm / norm : 1,  g' = c g
//   m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2
//   p = p - lr (m / (1 - b1^t) / (sqrt(v / (1 - b2^t)) + eps) + wd p)
//
// Bound by memory: fp32 parameters with fp32 gradients and states move 28 bytes an
// element, with 8-bit states 16, and the bf16 copy that the layers read two more. The
// clipping factor comes from the norm on the device, so clipped gradients are neither
// written nor read again; the copy is written by the same pass.
//
// 8-bit states. 256 elements of a tensor, one warp's, share a power of two (`scale`),
// the smallest one with their largest magnitude <= 15/16 of it. A code is a small float
// under it: sign, 4 bits of exponent, 3 of fraction for m; 5 and 3 for v, whose range
// has to be the square of m's: an m that is kept beside a v of 0 would be a step of any
// size. Powers of two, so that a new scale moves no value off its code. Codes are
// rounded up or down with the probabilities that keep the mean: v moves by a factor
// 1 - b2 a step, far less than half a code, and would stay where it is if rounded to
// nearest. The 16 random bits of an element come from splitmix64 (Steele, Lea and Flood,
// 2014) at (seed, step, tensor, element), so that a call's results are its inputs' alone.
// A bf16 parameter is rounded the same way. Encoding: the magnitude, scaled to lie just
// above fp32's smallest numbers, has the code as its top bits, gradual underflow included.
//
// Everything that a code depends on is computed with single rounded operations, so that
// it can be reproduced to the bit; the quotient of the step is the fast one (2 units).
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "launch.h"

namespace twell {
namespace {

constexpr int kThreads = 256;
constexpr int kBlocksPerSm = 4, kValueBlocksPerSm = 6;
constexpr int kBlock = TWELL_ADAMW_BLOCK;         // elements that share a scale: one warp's, 8 a lane
constexpr int kUnit = kBlock * (kThreads / 32);   // elements of one unit of work
constexpr int kPer = kBlock / 32;
// Tensors of one launch: two sizes of its parameters (32,764 bytes at most), the larger one without scales and with them.
// (500 tensors of 32-bit states, 4 M elements: 24.1 us, in two launches of 256 27.5.)
constexpr int kSmallTable = 32, kTable = 512, kTable8 = 400;
constexpr int kMost = 32768;
constexpr int kMBits = 4, kVBits = 5;             // exponent bits of the codes

constexpr uint64_t kGamma = 0x9E3779B97F4A7C15ull;

enum { P_F32 = 1, G_F32 = 2, VEC = 4 };  // VEC: everything lies on 16-byte boundaries (copies on 8)

template <int CAP, bool SCALES>
struct Scales {
    float* ms[CAP];
    float* vs[CAP];
    __device__ __forceinline__ float* m_scale(int k) const { return ms[k]; }
    __device__ __forceinline__ float* v_scale(int k) const { return vs[k]; }
};
template <int CAP>
struct Scales<CAP, false> {
    __device__ __forceinline__ float* m_scale(int) const { return nullptr; }
    __device__ __forceinline__ float* v_scale(int) const { return nullptr; }
};

template <int CAP, bool SCALES>
struct Table : Scales<CAP, SCALES> {
    static constexpr int kCap = CAP;
    static constexpr bool kScales = SCALES;
    void* p[CAP];
    const void* g[CAP];
    void* m[CAP];
    void* v[CAP];
    uint16_t* copy[CAP];
    int64_t numel[CAP];
    int32_t first[CAP + 1];  // first unit of each tensor
    int32_t id[CAP];         // its place in the list
    uint8_t flags[CAP];
    int32_t n;

    // Units of block b: a run of them, no run more than one longer than another.
    __device__ __forceinline__ int from(int b) const { return (int)((int64_t)first[n] * b / gridDim.x); }
    __device__ __forceinline__ int find(int u) const
    {
        int lo = 0, hi = n - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (first[mid] <= u)
                lo = mid;
            else
                hi = mid - 1;
        }
        return lo;
    }
};

struct Hyper {
    const float* lr;
    const int32_t* step;
    const float* norm;  // or null
    float max_norm;
    float b1, b2, rest1, rest2;  // rest = 1 - b, rounded once
    float log_b1, log_b2;
    float eps, decay;
    float one;  // 1
    uint64_t seed;
};

__device__ __forceinline__ uint64_t mix(uint64_t z)
{
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
    z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
    return z ^ (z >> 31);
}

// 1 - b^t from log b, without cancellation.
__device__ __forceinline__ float one_minus_power(float log_b, int t) { return -expm1f((float)t * log_b); }

__device__ __forceinline__ float sqrt_approx(float x)
{
    float y;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// (of a normal number below 2^126: eps at least, the root of a float at most)
__device__ __forceinline__ float reciprocal_approx(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Place of a lane's element k in its block: four neighbours, or (V false) neighbours in neighbouring lanes.
template <bool V>
__device__ __forceinline__ int place(int k, int lane)
{
    return V ? (k >> 2) * 128 + lane * 4 + (k & 3) : k * 32 + lane;
}

// A lane's elements as pairs, for the instructions that work on two fp32 values at once: with one at a time the pass
// over 8-bit states is bound by instructions.
constexpr int kPairs = kPer / 2;

template <bool V>
__device__ __forceinline__ void load(const void* p, bool f32, int64_t i0, int left, int lane, float2 (&x)[kPairs])
{
    if constexpr (V) {
#pragma unroll
        for (int k = 0; k < kPer; k += 4) {
            const int64_t i = i0 + place<true>(k, lane);
            if (f32) {
                const float4 q = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
                x[k / 2] = make_float2(q.x, q.y);
                x[k / 2 + 1] = make_float2(q.z, q.w);
            } else {
                const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
                x[k / 2] = make_float2(bf16_lo(q.x), bf16_hi(q.x));
                x[k / 2 + 1] = make_float2(bf16_lo(q.y), bf16_hi(q.y));
            }
        }
    } else {
        float y[kPer];
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int i = place<false>(k, lane);
            y[k] = 0.f;
            if (i < left)
                y[k] = f32 ? static_cast<const float*>(p)[i0 + i] : bf16_to_f32(static_cast<const uint16_t*>(p)[i0 + i]);
        }
#pragma unroll
        for (int k = 0; k < kPairs; ++k) x[k] = make_float2(y[2 * k], y[2 * k + 1]);
    }
}

template <bool V>
__device__ __forceinline__ void store(void* p, bool f32, int64_t i0, int left, int lane, const float2 (&x)[kPairs])
{
    if constexpr (V) {
#pragma unroll
        for (int k = 0; k < kPer; k += 4) {
            const int64_t i = i0 + place<true>(k, lane);
            const float2 a = x[k / 2], b = x[k / 2 + 1];
            if (f32)
                *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(a.x, a.y, b.x, b.y);
            else
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) = make_uint2(cvt_bf16x2(a.x, a.y), cvt_bf16x2(b.x, b.y));
        }
    } else {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int i = place<false>(k, lane);
            if (i >= left) continue;
            const float y = (k & 1) ? x[k / 2].y : x[k / 2].x;
            if (f32)
                static_cast<float*>(p)[i0 + i] = y;
            else
                static_cast<uint16_t*>(p)[i0 + i] = f32_to_bf16_bits(y);
        }
    }
}

// Codes of four elements a word, the first in the lowest byte.
template <bool V>
__device__ __forceinline__ void load_codes(const void* p, int64_t i0, int left, int lane, uint32_t (&w)[kPer / 4])
{
#pragma unroll
    for (int k = 0; k < kPer; k += 4) {
        if constexpr (V) {
            w[k / 4] = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(p) + i0 + place<true>(k, lane));
        } else {
            w[k / 4] = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = place<false>(k + e, lane);
                if (i < left) w[k / 4] |= (uint32_t) static_cast<const uint8_t*>(p)[i0 + i] << (8 * e);
            }
        }
    }
}

template <bool V>
__device__ __forceinline__ void store_codes(void* p, int64_t i0, int left, int lane, const uint32_t (&w)[kPer / 4])
{
#pragma unroll
    for (int k = 0; k < kPer; k += 4) {
        if constexpr (V) {
            *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p) + i0 + place<true>(k, lane)) = w[k / 4];
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = place<false>(k + e, lane);
                if (i < left) static_cast<uint8_t*>(p)[i0 + i] = (uint8_t)(w[k / 4] >> (8 * e));
            }
        }
    }
}

// 16 random bits for each of a lane's elements: for the moments m's in the lower and v's in the upper half of a word,
// two elements' words to one of splitmix64's; for a bf16 parameter four elements' bits. Neighbours of a lane share one.
template <bool V>
__device__ __forceinline__ void moment_bits(uint64_t key, int64_t i0, int lane, uint32_t (&r)[kPer])
{
    if constexpr (V) {
        const uint64_t at = key + (uint64_t)((i0 + lane * 4) / 2 + 1) * kGamma;
#pragma unroll
        for (int k = 0; k < kPer; k += 2) {
            const uint64_t w = mix(at + (uint64_t)((k >> 2) * 64 + ((k >> 1) & 1)) * kGamma);
            r[k] = (uint32_t)w;
            r[k + 1] = (uint32_t)(w >> 32);
        }
    } else {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int64_t e = i0 + place<false>(k, lane);
            r[k] = (uint32_t)(mix(key + (uint64_t)((e >> 1) + 1) * kGamma) >> ((e & 1) * 32));
        }
    }
}
template <bool V>
__device__ __forceinline__ void param_bits(uint64_t key, int64_t i0, int lane, uint32_t (&r)[kPer])
{
    if constexpr (V) {
        const uint64_t at = key + (uint64_t)((i0 + lane * 4) / 4 + 1) * kGamma;
#pragma unroll
        for (int k = 0; k < kPer; k += 4) {
            const uint64_t w = mix(at + (uint64_t)((k >> 2) * 32) * kGamma);
            r[k] = (uint32_t)w & 0xffffu;
            r[k + 1] = (uint32_t)w >> 16;
            r[k + 2] = (uint32_t)(w >> 32) & 0xffffu;
            r[k + 3] = (uint32_t)(w >> 48);
        }
    } else {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int64_t e = i0 + place<false>(k, lane);
            r[k] = (uint32_t)(mix(key + (uint64_t)((e >> 2) + 1) * kGamma) >> ((e & 3) * 16)) & 0xffffu;
        }
    }
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// a + b for pairs, rounded, where a is a rounded product. As a 1 + b with a 1 that the compiler does not know: sums of
// products, the instructions with explicit rounding too, were joined to fused multiply-additions where they work on
// pairs, and a code next to a border then was another one than single operations give (one in 5 million).
__device__ __forceinline__ float2 add_rounded(float2 a, float one, float2 b) { return __ffma2_rn(a, both(one), b); }

// Powers of two that a code and its value lie apart: 2^(127 - 2^E) times the scale. One multiplication as long as their
// product is a normal number, two (rounded the same) for scales above 2^(2^E).
template <int E>
constexpr float kUp = E == kMBits ? 0x1p+111f : 0x1p+95f;

// The values of codes with E exponent bits under `scale`.
template <int E>
__device__ __forceinline__ void decode(const uint32_t (&w)[kPer / 4], float scale, float2 (&x)[kPairs])
{
    const bool large = scale > (E == kMBits ? 0x1p+16f : 0x1p+32f);
    const float2 f = both(large ? kUp<E> : scale * kUp<E>);
#pragma unroll
    for (int k = 0; k < kPer; k += 2) {
        float y[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            // the byte at the top, then 4 bits down: exponent and fraction where fp32 has them, m's sign at its place
            const uint32_t top = w[k / 4] << (24 - 8 * ((k + e) & 3));
            y[e] = __uint_as_float(E == kMBits ? (uint32_t)((int32_t)top >> 4) & 0x87f00000u : (top >> 4) & 0x0ff00000u);
        }
        x[k / 2] = __fmul2_rn(make_float2(y[0], y[1]), f);
        if (large) x[k / 2] = __fmul2_rn(x[k / 2], both(scale));
    }
}

// Codes of a block's values and their scale (the same in all lanes), rounded by 16 random bits each. A block with a
// value that is not finite, or above 15/16 2^127, has NaN as its scale, and all its values are NaN.
template <int E>
__device__ __forceinline__ float encode(const float2 (&x)[kPairs], const uint32_t (&random)[kPer], uint32_t (&w)[kPer / 4])
{
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
        const uint32_t a = __float_as_uint(x[k].x), b = __float_as_uint(x[k].y);
        top = max(top, max(E == kMBits ? a & 0x7fffffffu : a, E == kMBits ? b & 0x7fffffffu : b));
    }
    top = __reduce_max_sync(0xffffffffu, top);
    const uint32_t up = (top >> 23) + 1 + ((top & 0x7fffffu) > 0x700000u ? 1u : 0u);
    const float scale = top == 0 ? 0.f : up > 254u ? __uint_as_float(0x7fc00000u) : __uint_as_float(up << 23);
    // 2^(127 - up) 2^(2^E - 127), the second factor for itself where the product is below fp32's normal numbers
    constexpr uint32_t sum = 127u + (1u << E);
    const bool large = up > sum - 1u;
    const float2 f = both(__uint_as_float(large ? (up >= 254u ? 0x400000u : (254u - up) << 23) : (sum - up) << 23));
    uint32_t least = 0xffffffffu, t[kPer];
#pragma unroll
    for (int k = 0; k < kPer; k += 2) {
        float2 z = __fmul2_rn(x[k / 2], f);
        if (large) z = __fmul2_rn(z, both(1.f / kUp<E>));
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            // Rounded up or down by the bits below the code: at most 15/16 of the scale, so never past the largest
            // code. Four bits up, the code is the top byte, m's sign (which the shift takes away) its first bit.
            const uint32_t bits = __float_as_uint(e ? z.y : z.x), r = random[k + e];
            t[k + e] = (bits + (E == kMBits ? r & 0xffffu : r >> 16) * 16u) << 4;
            if (E == kMBits)
                t[k + e] |= __float_as_uint(e ? x[k / 2].y : x[k / 2].x) & 0x80000000u;
            else
                least = min(least, t[k + e]);
        }
    }
    if (E != kMBits && least < 1u << 24) {  // a code of 0: only 0 has it
#pragma unroll
        for (int k = 0; k < kPer; ++k)
            if (t[k] < 1u << 24 && ((k & 1) ? x[k / 2].y : x[k / 2].x) > 0.f) t[k] = 1u << 24;
    }
#pragma unroll
    for (int k = 0; k < kPer; k += 4)
        w[k / 4] = __byte_perm(__byte_perm(t[k], t[k + 1], 0x0073), __byte_perm(t[k + 2], t[k + 3], 0x0073), 0x5410);
    return scale;
}

struct Scalars {
    float c, rate, decay, root;  // rate = lr / (1 - b1^t), decay so that rate decay = lr wd, root = 1 / sqrt(1 - b2^t)
    uint64_t base;
    int skip;
};

// A block's elements of one tensor. `moments`, `params`: keys of its random bits.
// 8-bit states of fp32 parameters: a warp's next block comes into shared memory by asynchronous copies while the present
// one is worked on (134 M elements: 457 us with loads when their turn came, now 406). bf16 parameters move too few bytes
// for that: their pass is bound by instructions, and the copies cost more of them.
struct Staged {
    uint4 p[kBlock / 4], g[kBlock / 4], m[kBlock / 16], v[kBlock / 16];  // parameters, fp32 or bf16 gradients, codes
};

__device__ __forceinline__ void copy16(void* to, const void* from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}

// Asks for a whole block of a tensor whose addresses allow 16-byte pieces.
__device__ __forceinline__ void stage(Staged& s, const void* p, const void* g, const void* m, const void* v, int flags, int64_t i0,
                                      int lane)
{
    const int gs = flags & G_F32 ? 4 : 2;
    const char* pp = static_cast<const char*>(p) + i0 * 4;
    const char* gg = static_cast<const char*>(g) + i0 * gs;
    copy16(&s.p[lane], pp + lane * 16);
    copy16(&s.p[32 + lane], pp + 512 + lane * 16);
    copy16(&s.g[lane], gg + lane * 16);
    if (gs == 4) copy16(&s.g[32 + lane], gg + 512 + lane * 16);
    const int half = lane & 15;
    if (lane < 16)
        copy16(&s.m[half], static_cast<const char*>(m) + i0 + half * 16);
    else
        copy16(&s.v[half], static_cast<const char*>(v) + i0 + half * 16);
}

// PF, GF: parameter and gradient are fp32 (as template arguments: with both kinds of loads behind a branch each waited for
// the one before).
template <bool V, bool BITS8, bool STAGED, bool PF, bool GF>
__device__ __forceinline__ void step_block(void* p, const void* g, void* m, void* v, float* ms, float* vs, uint16_t* copy,
                                           int64_t i0, int left, int lane, const Hyper& h, const Scalars& s,
                                           uint64_t moments, uint64_t params, const Staged& staged, float2 scales)
{
    float2 x[kPairs], grad[kPairs], mom[kPairs], var[kPairs];
    if constexpr (BITS8) {
        uint32_t cm[kPer / 4], cv[kPer / 4];
        if constexpr (V && STAGED && PF) {
            load<V>(staged.p, PF, 0, left, lane, x);
            load<V>(staged.g, GF, 0, left, lane, grad);
            load_codes<V>(staged.m, 0, left, lane, cm);
            load_codes<V>(staged.v, 0, left, lane, cv);
        } else {
            load<V>(p, PF, i0, left, lane, x);
            load<V>(g, GF, i0, left, lane, grad);
            load_codes<V>(m, i0, left, lane, cm);
            load_codes<V>(v, i0, left, lane, cv);
        }
        decode<kMBits>(cm, scales.x, mom);
        decode<kVBits>(cv, scales.y, var);
    } else {
        load<V>(p, PF, i0, left, lane, x);
        load<V>(g, GF, i0, left, lane, grad);
        load<V>(m, true, i0, left, lane, mom);
        load<V>(v, true, i0, left, lane, var);
    }
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
        // each operation of the moments rounded for itself: the codes are formed of them
        const float2 gs = __fmul2_rn(grad[k], both(s.c));
        mom[k] = add_rounded(__fmul2_rn(both(h.b1), mom[k]), h.one, __fmul2_rn(both(h.rest1), gs));
        var[k] = add_rounded(__fmul2_rn(both(h.b2), var[k]), h.one, __fmul2_rn(both(h.rest2), __fmul2_rn(gs, gs)));
        const float2 under = __ffma2_rn(make_float2(sqrt_approx(var[k].x), sqrt_approx(var[k].y)), both(s.root), both(h.eps));
        const float2 to = __fmul2_rn(mom[k], make_float2(reciprocal_approx(under.x), reciprocal_approx(under.y)));
        x[k] = __ffma2_rn(both(-s.rate), __ffma2_rn(both(s.decay), x[k], to), x[k]);
    }
    if (PF) {
        store<V>(p, true, i0, left, lane, x);
        if (copy) store<V>(copy, false, i0, left, lane, x);
    } else {
        // 16 random bits each: most steps are smaller than half a unit of bf16
        uint32_t r[kPer];
        param_bits<V>(params, i0, lane, r);
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            float& y = (k & 1) ? x[k / 2].y : x[k / 2].x;
            const uint32_t bits = __float_as_uint(y);
            // (not into infinity's or NaN's bits)
            y = __uint_as_float((bits & 0x7f800000u) == 0x7f800000u ? bits : (bits + r[k]) & 0xffff0000u);
        }
        store<V>(p, false, i0, left, lane, x);
    }
    if constexpr (BITS8) {
        uint32_t r[kPer], code[kPer / 4];
        moment_bits<V>(moments, i0, lane, r);
        const float sm = encode<kMBits>(mom, r, code);
        store_codes<V>(m, i0, left, lane, code);
        const float sv = encode<kVBits>(var, r, code);
        store_codes<V>(v, i0, left, lane, code);
        if (lane == 0) {
            ms[i0 / kBlock] = sm;
            vs[i0 / kBlock] = sv;
        }
    } else {
        store<V>(m, true, i0, left, lane, mom);
        store<V>(v, true, i0, left, lane, var);
    }
}

// f(whole pieces, parameter in fp32, gradient in fp32) as types.
template <class F>
__device__ __forceinline__ void by_types(int flags, bool whole, F f)
{
    const std::true_type yes{};
    const std::false_type no{};
    switch (flags & (whole ? VEC | P_F32 | G_F32 : P_F32 | G_F32)) {
        case VEC | P_F32 | G_F32: f(yes, yes, yes); break;
        case VEC | P_F32: f(yes, yes, no); break;
        case VEC | G_F32: f(yes, no, yes); break;
        case VEC: f(yes, no, no); break;
        case P_F32 | G_F32: f(no, yes, yes); break;
        case P_F32: f(no, yes, no); break;
        case G_F32: f(no, no, yes); break;
        default: f(no, no, no); break;
    }
}

// STAGED: 8-bit states, some parameters in fp32. (Without any the ring's shared memory would only take the first-level
// cache away: bf16 parameters 441 instead of 399 us.)
template <int CAP, bool BITS8, bool STAGED>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) k_adamw(const __grid_constant__ Table<CAP, BITS8> t, const Hyper h)
{
    static_assert(sizeof(t) + sizeof(h) <= 32764, "parameters of a launch");
    __shared__ Scalars shared;
    if (threadIdx.x == 0) {
        Scalars s;
        const float norm = h.norm ? *h.norm : 0.f;
        const int step = *h.step;
        s.skip = !(fabsf(norm) < INFINITY) || step < 1;
        // max_norm (1 / norm), as tensor libraries divide a number by a tensor, so that their operations give the same
        // codes to the bit (divided where 1 / norm would pass fp32's range)
        s.c = norm <= h.max_norm ? 1.f : norm > 0x1p-126f ? __fmul_rn(h.max_norm, __frcp_rn(norm)) : __fdiv_rn(h.max_norm, norm);
        const float rest = one_minus_power(h.log_b1, step);
        s.rate = __fdiv_rn(*h.lr, rest);
        s.decay = h.decay * rest;
        s.root = rsqrtf(one_minus_power(h.log_b2, step));
        s.base = mix(h.seed + (uint64_t)(int64_t)step * kGamma);
        shared = s;
    }
    __syncthreads();
    const Scalars s = shared;
    if (s.skip) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int u0 = t.from(blockIdx.x), u1 = t.from(blockIdx.x + 1);
    int k = u0 < u1 ? t.find(u0) - 1 : 0, next = u0;
    uint64_t moments = 0, params = 0;
    __shared__ Staged ring[STAGED ? kThreads / 32 : 1][2];
    bool ready = false;  // this block has been asked for
    int at = 0;          // its place in the ring
    float2 scales = make_float2(0.f, 0.f), next_scales = scales;
    for (int u = u0; u < u1; ++u) {
        if (u >= next) {  // the next tensor (none is empty), or the first
            ++k;
            next = t.first[k + 1];
            const uint64_t key = s.base + (uint64_t)(2 * (int64_t)t.id[k] + 1) * kGamma;
            if (BITS8) moments = mix(key);
            params = mix(key + kGamma);
        }
        const int64_t i0 = (int64_t)(u - t.first[k]) * kUnit + warp * kBlock;
        const int64_t rest = t.numel[k] - i0;
        if (rest <= 0) continue;
        const int left = (int)min((int64_t)kBlock, rest);
        if constexpr (BITS8) {
            scales = ready ? next_scales : make_float2(t.ms[k][i0 / kBlock], t.vs[k][i0 / kBlock]);
            if (STAGED && left == kBlock && (t.flags[k] & VEC) && (t.flags[k] & P_F32)) {
                if (!ready) stage(ring[warp][at], t.p[k], t.g[k], t.m[k], t.v[k], t.flags[k], i0, lane);
                asm volatile("cp.async.commit_group;" ::: "memory");
                ready = u + 1 < min(u1, next) && rest >= kUnit + kBlock;
                if (ready) {
                    stage(ring[warp][at ^ 1], t.p[k], t.g[k], t.m[k], t.v[k], t.flags[k], i0 + kUnit, lane);
                    const int64_t b = i0 / kBlock + kUnit / kBlock;
                    next_scales = make_float2(t.ms[k][b], t.vs[k][b]);
                }
                asm volatile("cp.async.commit_group;\n cp.async.wait_group 1;" ::: "memory");
                __syncwarp();
            } else {
                ready = false;
            }
        }
        by_types(t.flags[k], left == kBlock, [&](auto v, auto pf, auto gf) {
            step_block<decltype(v)::value, BITS8, STAGED, decltype(pf)::value, decltype(gf)::value>(
                t.p[k], t.g[k], t.m[k], t.v[k], t.m_scale(k), t.v_scale(k), t.copy[k], i0, left, lane, h, s, moments, params,
                ring[STAGED ? warp : 0][at], scales);
        });
        at ^= 1;
        if (STAGED) __syncwarp();  // the ring's other half may be filled again
    }
}

// The values that 8-bit states stand for: m to p's tensor of the table, v to g's.
template <int CAP>
__global__ void __launch_bounds__(kThreads, kValueBlocksPerSm) k_adamw_values(const __grid_constant__ Table<CAP, true> t)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int u0 = t.from(blockIdx.x), u1 = t.from(blockIdx.x + 1);
    int k = u0 < u1 ? t.find(u0) : 0;
    for (int u = u0; u < u1; ++u) {
        while (u >= t.first[k + 1]) ++k;
        const int64_t i0 = (int64_t)(u - t.first[k]) * kUnit + warp * kBlock;
        const int64_t rest = t.numel[k] - i0;
        if (rest <= 0) continue;
        const int left = (int)min((int64_t)kBlock, rest);
        const int flags = t.flags[k];
        auto block = [&](auto tag) {
            constexpr bool V = decltype(tag)::value;
            uint32_t cm[kPer / 4], cv[kPer / 4];
            float2 x[kPairs];
            load_codes<V>(t.m[k], i0, left, lane, cm);
            load_codes<V>(t.v[k], i0, left, lane, cv);
            const float sm = t.ms[k][i0 / kBlock], sv = t.vs[k][i0 / kBlock];
            decode<kMBits>(cm, sm, x);
            store<V>(t.p[k], flags & P_F32, i0, left, lane, x);
            decode<kVBits>(cv, sv, x);
            store<V>(const_cast<void*>(t.g[k]), flags & G_F32, i0, left, lane, x);
        };
        if (left == kBlock && (flags & VEC))
            block(std::true_type{});
        else
            block(std::false_type{});
    }
}

bool aligned(const void* p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool type_ok(int t) { return t == TWELL_BF16 || t == TWELL_F32; }

int sms_current()
{
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) !=
                                                  cudaSuccess)
        return 0;
    return n;
}

twell_status check_list(const twell_adamw_list* l)
{
    if (!l || l->n < 0 || (l->state_bits != 8 && l->state_bits != 32)) return TWELL_ERR_INVALID_ARG;
    if (l->n == 0) return TWELL_OK;
    const bool eight = l->state_bits == 8;
    if (!l->param || !l->grad || !l->m || !l->v || !l->numel || !l->param_type || !l->grad_type ||
        (eight && (!l->m_scale || !l->v_scale)))
        return TWELL_ERR_INVALID_ARG;
    if (l->n > kMost) return TWELL_ERR_UNSUPPORTED;
    for (int i = 0; i < l->n; ++i) {
        const int64_t n = l->numel[i];
        if (n < 0 || !type_ok(l->param_type[i]) || !type_ok(l->grad_type[i])) return TWELL_ERR_INVALID_ARG;
        if (n == 0) continue;
        const void* copy = l->copy ? l->copy[i] : nullptr;
        if (!l->param[i] || !l->grad[i] || !l->m[i] || !l->v[i] || (copy && l->param_type[i] != TWELL_F32)) return TWELL_ERR_INVALID_ARG;
        const size_t ps = l->param_type[i] == TWELL_F32 ? 4 : 2, gs = l->grad_type[i] == TWELL_F32 ? 4 : 2, ss = eight ? 1 : 4;
        if (!aligned(l->param[i], ps) || !aligned(l->grad[i], gs) || !aligned(l->m[i], ss) || !aligned(l->v[i], ss) ||
            !aligned(copy, 2))
            return TWELL_ERR_INVALID_ARG;
        if (eight && (!l->m_scale[i] || !l->v_scale[i] || !aligned(l->m_scale[i], 4) || !aligned(l->v_scale[i], 4)))
            return TWELL_ERR_INVALID_ARG;
        if (l->m[i] == l->v[i] || l->param[i] == l->grad[i] || l->param[i] == l->m[i] || l->param[i] == l->v[i] ||
            copy == l->param[i] || (copy && (copy == l->grad[i] || copy == l->m[i] || copy == l->v[i])))
            return TWELL_ERR_INVALID_ARG;
        if (n > (int64_t)kUnit * (INT32_MAX / 2)) return TWELL_ERR_UNSUPPORTED;
    }
    return TWELL_OK;
}

// f(table, blocks) for the list's tensors, CAP of them a launch. p and g of entry i: of(i, &p, &g, &flags).
template <int CAP, bool SCALES, class Of, class F>
twell_status by_tables(const twell_adamw_list* l, int most, Of of, F f)
{
    int next = 0;
    while (next < l->n) {
        Table<CAP, SCALES> t;
        t.n = 0;
        int64_t units = 0;
        while (next < l->n && t.n < CAP) {
            const int64_t n = l->numel[next], more = (n + kUnit - 1) / kUnit;
            if (units + more > INT32_MAX / 2 && t.n > 0) break;
            if (n > 0) {
                const int i = t.n++;
                of(next, &t.p[i], &t.g[i], &t.copy[i], &t.flags[i]);
                t.m[i] = l->m[next];
                t.v[i] = l->v[next];
                if constexpr (SCALES) {
                    t.ms[i] = l->m_scale[next];
                    t.vs[i] = l->v_scale[next];
                }
                t.numel[i] = n;
                t.first[i] = (int32_t)units;
                t.id[i] = next;
                if (aligned(t.p[i], 16) && aligned(t.g[i], 16) && aligned(t.m[i], 16) && aligned(t.v[i], 16) && aligned(t.copy[i], 8))
                    t.flags[i] |= VEC;
                units += more;
            }
            ++next;
        }
        if (t.n == 0) break;
        t.first[t.n] = (int32_t)units;
        count_launches(1);
        f(t, (int)(units < most ? units : most));
        if (cudaGetLastError() != cudaSuccess) return TWELL_ERR_CUDA;
    }
    return TWELL_OK;
}

}  // namespace
}  // namespace twell

using namespace twell;

extern "C" twell_status twell_adamw(const twell_adamw_list* list, const float* lr, const int32_t* step, double beta1,
                                    double beta2, double eps, double weight_decay, const float* norm, float max_norm,
                                    uint64_t seed, void* stream)
{
    const twell_status ok = check_list(list);
    if (ok != TWELL_OK) return ok;
    if (!lr || !step || !aligned(lr, 4) || !aligned(step, 4) || !aligned(norm, 4) || !(beta1 >= 0.0 && beta1 < 1.0) ||
        !(beta2 >= 0.0 && beta2 < 1.0) || !(eps > 0.0 && eps < INFINITY) || !(weight_decay >= 0.0 && weight_decay < INFINITY) ||
        !((float)eps >= 0x1p-126f) || (norm && !(max_norm >= 0.f)))
        return TWELL_ERR_INVALID_ARG;
    if (list->n == 0) return TWELL_OK;
    const int sms = sms_current();
    if (sms <= 0) return TWELL_ERR_CUDA;
    Hyper h{};
    h.lr = lr;
    h.step = step;
    h.norm = norm;
    h.max_norm = norm ? max_norm : INFINITY;
    h.b1 = (float)beta1;
    h.b2 = (float)beta2;
    h.rest1 = (float)(1.0 - beta1);
    h.rest2 = (float)(1.0 - beta2);
    h.log_b1 = (float)log(beta1);  // -infinity for 0: 1 - 0^t = 1
    h.log_b2 = (float)log(beta2);
    h.eps = (float)eps;
    h.decay = (float)weight_decay;
    h.one = 1.f;
    h.seed = seed;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool eight = list->state_bits == 8;
    auto of = [&](int i, void** p, const void** g, uint16_t** copy, uint8_t* flags) {
        *p = list->param[i];
        *g = list->grad[i];
        *copy = list->copy ? static_cast<uint16_t*>(list->copy[i]) : nullptr;
        *flags = (uint8_t)((list->param_type[i] == TWELL_F32 ? P_F32 : 0) | (list->grad_type[i] == TWELL_F32 ? G_F32 : 0));
    };
    bool any_f32 = false;
    for (int i = 0; i < list->n; ++i) any_f32 = any_f32 || (list->numel[i] > 0 && list->param_type[i] == TWELL_F32);
    auto launch = [&](const auto& table, int blocks) {
        using T = std::decay_t<decltype(table)>;
        if constexpr (!T::kScales)
            k_adamw<T::kCap, false, false><<<blocks, kThreads, 0, s>>>(table, h);
        else if (any_f32)
            k_adamw<T::kCap, true, true><<<blocks, kThreads, 0, s>>>(table, h);
        else
            k_adamw<T::kCap, true, false><<<blocks, kThreads, 0, s>>>(table, h);
    };
    const int most = sms * kBlocksPerSm;
    if (list->n <= kSmallTable)
        return eight ? by_tables<kSmallTable, true>(list, most, of, launch) : by_tables<kSmallTable, false>(list, most, of, launch);
    return eight ? by_tables<kTable8, true>(list, most, of, launch) : by_tables<kTable, false>(list, most, of, launch);
}

extern "C" twell_status twell_adamw_values(const twell_adamw_list* list, const twell_tensor_list* m_out,
                                           const twell_tensor_list* v_out, void* stream)
{
    const twell_status ok = check_list(list);
    if (ok != TWELL_OK) return ok;
    if (!m_out || !v_out || list->state_bits != 8 || m_out->n != list->n || v_out->n != list->n) return TWELL_ERR_INVALID_ARG;
    if (list->n == 0) return TWELL_OK;
    for (const twell_tensor_list* o : {m_out, v_out}) {
        if (!o->out || !o->numel || !o->type) return TWELL_ERR_INVALID_ARG;
        for (int i = 0; i < list->n; ++i) {
            if (o->numel[i] != list->numel[i] || !type_ok(o->type[i])) return TWELL_ERR_INVALID_ARG;
            if (list->numel[i] > 0 && (!o->out[i] || !aligned(o->out[i], o->type[i] == TWELL_F32 ? 4 : 2))) return TWELL_ERR_INVALID_ARG;
        }
    }
    const int sms = sms_current();
    if (sms <= 0) return TWELL_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto of = [&](int i, void** p, const void** g, uint16_t** copy, uint8_t* flags) {
        *p = m_out->out[i];
        *g = v_out->out[i];
        *copy = nullptr;
        *flags = (uint8_t)((m_out->type[i] == TWELL_F32 ? P_F32 : 0) | (v_out->type[i] == TWELL_F32 ? G_F32 : 0));
    };
    auto launch = [&](const auto& table, int blocks) {
        k_adamw_values<std::decay_t<decltype(table)>::kCap><<<blocks, kThreads, 0, s>>>(table);
    };
    const int most = sms * kValueBlocksPerSm;
    return list->n <= kSmallTable ? by_tables<kSmallTable, true>(list, most, of, launch) : by_tables<kTable8, true>(list, most, of, launch);
}
