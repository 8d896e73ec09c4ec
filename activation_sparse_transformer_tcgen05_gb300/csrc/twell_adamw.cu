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
constexpr int kBlocksPerSm = 4;
constexpr int kBlock = TWELL_ADAMW_BLOCK;         // elements that share a scale: one warp's, 8 a lane
constexpr int kUnit = kBlock * (kThreads / 32);   // elements of one unit of work
constexpr int kPer = kBlock / 32;
constexpr int kTable = 256, kSmallTable = 32;     // tensors of one launch: two sizes of its parameters
constexpr int kMost = 32768;
constexpr int kMBits = 4, kVBits = 5;             // exponent bits of the codes

constexpr uint64_t kGamma = 0x9E3779B97F4A7C15ull;

enum { P_F32 = 1, G_F32 = 2, VEC = 4 };

template <int CAP>
struct Table {
    void* p[CAP];
    const void* g[CAP];
    void* m[CAP];
    void* v[CAP];
    float* ms[CAP];
    float* vs[CAP];
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

// Place of a lane's element k in its block: four neighbours, or (VEC false) neighbours in neighbouring lanes.
template <bool V>
__device__ __forceinline__ int place(int k, int lane)
{
    return V ? (k >> 2) * 128 + lane * 4 + (k & 3) : k * 32 + lane;
}

template <bool V>
__device__ __forceinline__ void load(const void* p, bool f32, int64_t i0, int left, int lane, float (&x)[kPer])
{
    if constexpr (V) {
#pragma unroll
        for (int k = 0; k < kPer; k += 4) {
            const int64_t i = i0 + place<true>(k, lane);
            if (f32) {
                const float4 q = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
                x[k] = q.x, x[k + 1] = q.y, x[k + 2] = q.z, x[k + 3] = q.w;
            } else {
                const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
                x[k] = bf16_lo(q.x), x[k + 1] = bf16_hi(q.x), x[k + 2] = bf16_lo(q.y), x[k + 3] = bf16_hi(q.y);
            }
        }
    } else {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int i = place<false>(k, lane);
            x[k] = 0.f;
            if (i < left)
                x[k] = f32 ? static_cast<const float*>(p)[i0 + i] : bf16_to_f32(static_cast<const uint16_t*>(p)[i0 + i]);
        }
    }
}

template <bool V>
__device__ __forceinline__ void store(void* p, bool f32, int64_t i0, int left, int lane, const float (&x)[kPer])
{
    if constexpr (V) {
#pragma unroll
        for (int k = 0; k < kPer; k += 4) {
            const int64_t i = i0 + place<true>(k, lane);
            if (f32)
                *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(x[k], x[k + 1], x[k + 2], x[k + 3]);
            else
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) =
                    make_uint2(cvt_bf16x2(x[k], x[k + 1]), cvt_bf16x2(x[k + 2], x[k + 3]));
        }
    } else {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int i = place<false>(k, lane);
            if (i >= left) continue;
            if (f32)
                static_cast<float*>(p)[i0 + i] = x[k];
            else
                static_cast<uint16_t*>(p)[i0 + i] = f32_to_bf16_bits(x[k]);
        }
    }
}

template <bool V>
__device__ __forceinline__ void load_codes(const void* p, int64_t i0, int left, int lane, uint32_t (&x)[kPer])
{
    if constexpr (V) {
#pragma unroll
        for (int k = 0; k < kPer; k += 4) {
            const uint32_t q = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(p) + i0 + place<true>(k, lane));
#pragma unroll
            for (int e = 0; e < 4; ++e) x[k + e] = (q >> (8 * e)) & 255u;
        }
    } else {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int i = place<false>(k, lane);
            x[k] = i < left ? static_cast<const uint8_t*>(p)[i0 + i] : 0u;
        }
    }
}

template <bool V>
__device__ __forceinline__ void store_codes(void* p, int64_t i0, int left, int lane, const uint32_t (&x)[kPer])
{
    if constexpr (V) {
#pragma unroll
        for (int k = 0; k < kPer; k += 4)
            *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p) + i0 + place<true>(k, lane)) =
                x[k] | x[k + 1] << 8 | x[k + 2] << 16 | x[k + 3] << 24;
    } else {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int i = place<false>(k, lane);
            if (i < left) static_cast<uint8_t*>(p)[i0 + i] = (uint8_t)x[k];
        }
    }
}

// The values of codes with E exponent bits under `scale`.
template <int E>
__device__ __forceinline__ void decode(const uint32_t (&code)[kPer], float scale, float (&x)[kPer])
{
    const float up = __uint_as_float((uint32_t)(254 - (1 << E)) << 23);  // 2^(127 - 2^E)
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const uint32_t size = E == kMBits ? code[k] & 127u : code[k];
        const float y = __fmul_rn(__fmul_rn(__uint_as_float(size << 20), up), scale);
        x[k] = E == kMBits && (code[k] & 128u) ? -y : y;
    }
}

// Codes of a block's values and their scale (the same in all lanes), rounded by 16 random bits each. A block with a
// value that is not finite has NaN as its scale, and all its values are NaN.
template <int E>
__device__ __forceinline__ float encode(const float (&x)[kPer], const uint32_t (&random)[kPer], uint32_t (&code)[kPer])
{
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) top = max(top, __float_as_uint(x[k]) & 0x7fffffffu);
    top = __reduce_max_sync(0xffffffffu, top);
    uint32_t up = (top >> 23) + 1 + ((top & 0x7fffffu) > 0x700000u ? 1u : 0u);
    up = min(up, 254u);
    const float scale = top == 0 ? 0.f : top >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : __uint_as_float(up << 23);
    // 1 / scale: 2^(127 - up), below fp32's normal numbers for up = 254
    const float inv = top == 0 ? 0.f : up == 254u ? __uint_as_float(0x400000u) : __uint_as_float((254u - up) << 23);
    const float down = E == kMBits ? 0x1p-111f : 0x1p-95f;  // 2^(2^E - 127)
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const float z = __fmul_rn(__fmul_rn(fabsf(x[k]), inv), down);
        uint32_t q = (__float_as_uint(z) + (random[k] << 4)) >> 20;
        q = min(q, (8u << E) - 1u);
        if (E == kMBits)
            q |= (__float_as_uint(x[k]) >> 24) & 128u;
        else if (q == 0 && x[k] > 0.f)
            q = 1;
        code[k] = q;
    }
    return scale;
}

struct Scalars {
    float c, lr, by_m, by_v;
    uint64_t base;
    int skip;
};

// A block's elements of one tensor.
template <bool V, bool BITS8>
__device__ __forceinline__ void step_block(void* p, const void* g, void* m, void* v, float* ms, float* vs, uint16_t* copy,
                                           int flags, int64_t i0, int left, int lane, const Hyper& h, const Scalars& s,
                                           uint64_t key)
{
    float x[kPer], grad[kPer], mom[kPer], var[kPer];
    load<V>(p, flags & P_F32, i0, left, lane, x);
    load<V>(g, flags & G_F32, i0, left, lane, grad);
    if constexpr (BITS8) {
        uint32_t cm[kPer], cv[kPer];
        load_codes<V>(m, i0, left, lane, cm);
        load_codes<V>(v, i0, left, lane, cv);
        const float sm = ms[i0 / kBlock], sv = vs[i0 / kBlock];
        decode<kMBits>(cm, sm, mom);
        decode<kVBits>(cv, sv, var);
    } else {
        load<V>(m, true, i0, left, lane, mom);
        load<V>(v, true, i0, left, lane, var);
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const float gs = __fmul_rn(grad[k], s.c);
        mom[k] = __fadd_rn(__fmul_rn(h.b1, mom[k]), __fmul_rn(h.rest1, gs));
        var[k] = __fadd_rn(__fmul_rn(h.b2, var[k]), __fmul_rn(h.rest2, __fmul_rn(gs, gs)));
        const float to = __fdividef(mom[k] * s.by_m, sqrt_approx(var[k] * s.by_v) + h.eps);
        x[k] -= s.lr * fmaf(h.decay, x[k], to);
    }
    if (flags & P_F32) {
        store<V>(p, true, i0, left, lane, x);
        if (copy) store<V>(copy, false, i0, left, lane, x);
    } else {
        // 16 random bits each: most steps are smaller than half a unit of bf16
        const uint64_t pkey = mix(key + kGamma);
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int64_t e = i0 + place<V>(k, lane);
            const uint32_t r = (uint32_t)(mix(pkey + (uint64_t)((e >> 2) + 1) * kGamma) >> ((e & 3) * 16)) & 0xffffu;
            const uint32_t bits = __float_as_uint(x[k]);
            // (not into infinity's or NaN's bits)
            x[k] = __uint_as_float((bits & 0x7f800000u) == 0x7f800000u ? bits : (bits + r) & 0xffff0000u);
        }
        store<V>(p, false, i0, left, lane, x);
    }
    if constexpr (BITS8) {
        const uint64_t mkey = mix(key);
        uint32_t rm[kPer], rv[kPer], code[kPer];
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int64_t e = i0 + place<V>(k, lane);
            const uint32_t w = (uint32_t)(mix(mkey + (uint64_t)((e >> 1) + 1) * kGamma) >> ((e & 1) * 32));
            rm[k] = w & 0xffffu;
            rv[k] = w >> 16;
        }
        const float sm = encode<kMBits>(mom, rm, code);
        store_codes<V>(m, i0, left, lane, code);
        const float sv = encode<kVBits>(var, rv, code);
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

template <int CAP, bool BITS8>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) k_adamw(const __grid_constant__ Table<CAP> t, const Hyper h)
{
    __shared__ Scalars shared;
    if (threadIdx.x == 0) {
        Scalars s;
        const float norm = h.norm ? *h.norm : 0.f;
        s.c = norm > h.max_norm ? __fdiv_rn(h.max_norm, norm) : 1.f;
        s.lr = *h.lr;
        const int step = *h.step;
        s.skip = !(fabsf(norm) < INFINITY) || step < 1;
        s.by_m = __fdiv_rn(1.f, one_minus_power(h.log_b1, step));
        s.by_v = __fdiv_rn(1.f, one_minus_power(h.log_b2, step));
        s.base = mix(h.seed + (uint64_t)(int64_t)step * kGamma);
        shared = s;
    }
    __syncthreads();
    const Scalars s = shared;
    if (s.skip) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int u0 = t.from(blockIdx.x), u1 = t.from(blockIdx.x + 1);
    int k = u0 < u1 ? t.find(u0) : 0;
    for (int u = u0; u < u1; ++u) {
        while (u >= t.first[k + 1]) ++k;
        const int64_t i0 = (int64_t)(u - t.first[k]) * kUnit + warp * kBlock;
        const int64_t rest = t.numel[k] - i0;
        if (rest <= 0) continue;
        const int left = (int)min((int64_t)kBlock, rest);
        const uint64_t key = s.base + (uint64_t)(2 * (int64_t)t.id[k] + 1) * kGamma;
        if (left == kBlock && (t.flags[k] & VEC))
            step_block<true, BITS8>(t.p[k], t.g[k], t.m[k], t.v[k], t.ms[k], t.vs[k], t.copy[k], t.flags[k], i0, left, lane, h, s,
                                    key);
        else
            step_block<false, BITS8>(t.p[k], t.g[k], t.m[k], t.v[k], t.ms[k], t.vs[k], t.copy[k], t.flags[k], i0, left, lane, h,
                                     s, key);
    }
}

// The values that 8-bit states stand for: m to p's tensor of the table, v to g's.
template <int CAP>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) k_adamw_values(const __grid_constant__ Table<CAP> t)
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
        auto both = [&](auto tag) {
            constexpr bool V = decltype(tag)::value;
            uint32_t cm[kPer], cv[kPer];
            float x[kPer];
            load_codes<V>(t.m[k], i0, left, lane, cm);
            load_codes<V>(t.v[k], i0, left, lane, cv);
            const float sm = t.ms[k][i0 / kBlock], sv = t.vs[k][i0 / kBlock];
            decode<kMBits>(cm, sm, x);
            store<V>(t.p[k], flags & P_F32, i0, left, lane, x);
            decode<kVBits>(cv, sv, x);
            store<V>(const_cast<void*>(t.g[k]), flags & G_F32, i0, left, lane, x);
        };
        if (left == kBlock && (flags & VEC))
            both(std::true_type{});
        else
            both(std::false_type{});
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
template <int CAP, class Of, class F>
twell_status by_tables(const twell_adamw_list* l, int sms, Of of, F f)
{
    int next = 0;
    while (next < l->n) {
        Table<CAP> t;
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
                t.ms[i] = l->state_bits == 8 ? l->m_scale[next] : nullptr;
                t.vs[i] = l->state_bits == 8 ? l->v_scale[next] : nullptr;
                t.numel[i] = n;
                t.first[i] = (int32_t)units;
                t.id[i] = next;
                // 16-byte pieces of fp32, 8 of bf16, 4 of codes
                const size_t ss = l->state_bits == 8 ? 4 : 16;
                if (aligned(t.p[i], t.flags[i] & P_F32 ? 16 : 8) && aligned(t.g[i], t.flags[i] & G_F32 ? 16 : 8) &&
                    aligned(t.m[i], ss) && aligned(t.v[i], ss) && aligned(t.copy[i], 8))
                    t.flags[i] |= VEC;
                units += more;
            }
            ++next;
        }
        if (t.n == 0) break;
        t.first[t.n] = (int32_t)units;
        const int most = sms * kBlocksPerSm;
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
        !((float)eps > 0.f) || (norm && !(max_norm >= 0.f)))
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
    h.seed = seed;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool eight = list->state_bits == 8;
    auto of = [&](int i, void** p, const void** g, uint16_t** copy, uint8_t* flags) {
        *p = list->param[i];
        *g = list->grad[i];
        *copy = list->copy ? static_cast<uint16_t*>(list->copy[i]) : nullptr;
        *flags = (uint8_t)((list->param_type[i] == TWELL_F32 ? P_F32 : 0) | (list->grad_type[i] == TWELL_F32 ? G_F32 : 0));
    };
    if (list->n <= kSmallTable)
        return by_tables<kSmallTable>(list, sms, of, [&](const Table<kSmallTable>& t, int blocks) {
            if (eight)
                k_adamw<kSmallTable, true><<<blocks, kThreads, 0, s>>>(t, h);
            else
                k_adamw<kSmallTable, false><<<blocks, kThreads, 0, s>>>(t, h);
        });
    return by_tables<kTable>(list, sms, of, [&](const Table<kTable>& t, int blocks) {
        if (eight)
            k_adamw<kTable, true><<<blocks, kThreads, 0, s>>>(t, h);
        else
            k_adamw<kTable, false><<<blocks, kThreads, 0, s>>>(t, h);
    });
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
    if (list->n <= kSmallTable)
        return by_tables<kSmallTable>(list, sms, of, [&](const Table<kSmallTable>& t, int blocks) {
            k_adamw_values<kSmallTable><<<blocks, kThreads, 0, s>>>(t);
        });
    return by_tables<kTable>(list, sms, of, [&](const Table<kTable>& t, int blocks) {
        k_adamw_values<kTable><<<blocks, kThreads, 0, s>>>(t);
    });
}
