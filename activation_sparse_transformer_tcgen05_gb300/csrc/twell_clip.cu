// twell_clip.cu — L2 norm over many tensors, and the tensors scaled so that it
// is at most a bound.
//
//   norm = sqrt(sum over all elements of g^2),  c = 1 where norm <= max_norm, else max_norm / norm
//   out = c g, rounded once to the tensor's type
//
// Bound by memory: every element is read for the norm, and read and written
// again scaled (12 bytes in fp32). The tensors' addresses travel in the
// launch's parameters (up to 512 of them a launch), so nothing is copied to the
// device first.
//
//   k_sumsq       every block sums the squares of a run of consecutive units
//   k_clip_scale  every block adds the blocks' sums in the same fixed order and
//                 scales the same run, last unit first: what the first kernel
//                 read last is still in L2
#include "common.cuh"
#include "launch.h"

namespace twell {
namespace {

constexpr int kThreads = 256;
constexpr int kBlocksPerSm = 4;
constexpr int kUnit = 8192;                     // elements of one unit of work: 32 a thread
constexpr int kPer = kUnit / kThreads;
constexpr int kMaxBlocks = 152 * kBlocksPerSm;  // of one launch, each with one partial sum
constexpr int kTable = 512, kSmallTable = 32;   // tensors of one launch: two sizes of its parameters
constexpr int kMaxLaunches = 64;                // 32768 tensors

template <int CAP>
struct Table {
    const void* in[CAP];
    void* out[CAP];
    int64_t numel[CAP];
    int32_t first[CAP + 1];  // first unit of each tensor
    uint8_t f32[CAP];
    uint8_t vec[CAP];        // 16-byte accesses: both addresses allow them
    int32_t n;

    // Units of block b: a run of them, no run more than one longer than another.
    __device__ __forceinline__ int from(int b) const { return (int)((int64_t)first[n] * b / gridDim.x); }
};

// One thread's elements of a unit as floats: 16-byte loads where the tensor
// allows them, else element by element, neighbours in neighbouring threads.
// at(k) is the place of element k in the unit.
template <bool F32, bool VEC>
struct Slice {
    static constexpr int W = VEC ? (F32 ? 4 : 8) : 1;
    static __device__ __forceinline__ int at(int k) { return (k / W * kThreads + (int)threadIdx.x) * W + k % W; }

    // `left` elements of the unit exist; a whole unit takes the branch without tests
    // for each piece (2.1 GB of gradients, both passes: 1.26 ms, with them 1.29).
    static __device__ __forceinline__ void load(const void* p, int64_t i0, int left, float (&v)[kPer])
    {
        if (left == kUnit)
            load_pieces<true>(p, i0, left, v);
        else
            load_pieces<false>(p, i0, left, v);
    }
    static __device__ __forceinline__ void store(void* p, int64_t i0, int left, const float (&v)[kPer])
    {
        if (left == kUnit)
            store_pieces<true>(p, i0, left, v);
        else
            store_pieces<false>(p, i0, left, v);
    }

    template <bool FULL>
    static __device__ __forceinline__ void load_pieces(const void* p, int64_t i0, int left, float (&v)[kPer])
    {
#pragma unroll
        for (int k = 0; k < kPer; k += W) {
            const int i = at(k);
            if (VEC && (FULL || i + W <= left)) {
                if constexpr (F32) {
                    const float4 q = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i0 + i);
                    v[k] = q.x, v[k + 1 < kPer ? k + 1 : k] = q.y, v[k + 2 < kPer ? k + 2 : k] = q.z,
                    v[k + 3 < kPer ? k + 3 : k] = q.w;
                } else if constexpr (VEC) {
                    const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i0 + i);
                    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                    for (int e = 0; e < W; ++e) v[k + e] = (e & 1) ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < W; ++e) {
                    float x = 0.f;
                    if (FULL || i + e < left)
                        x = F32 ? static_cast<const float*>(p)[i0 + i + e]
                                : bf16_to_f32(static_cast<const uint16_t*>(p)[i0 + i + e]);
                    v[k + e] = x;
                }
            }
        }
    }

    template <bool FULL>
    static __device__ __forceinline__ void store_pieces(void* p, int64_t i0, int left, const float (&v)[kPer])
    {
#pragma unroll
        for (int k = 0; k < kPer; k += W) {
            const int i = at(k);
            if (VEC && (FULL || i + W <= left)) {
                if constexpr (F32) {
                    *reinterpret_cast<float4*>(static_cast<float*>(p) + i0 + i) =
                        make_float4(v[k], v[k + 1 < kPer ? k + 1 : k], v[k + 2 < kPer ? k + 2 : k],
                                    v[k + 3 < kPer ? k + 3 : k]);
                } else if constexpr (VEC) {
                    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i0 + i) =
                        make_uint4(cvt_bf16x2(v[k], v[k + 1]), cvt_bf16x2(v[k + 2], v[k + 3]),
                                   cvt_bf16x2(v[k + 4], v[k + 5]), cvt_bf16x2(v[k + 6], v[k + 7]));
                }
            } else {
#pragma unroll
                for (int e = 0; e < W; ++e) {
                    if (!FULL && i + e >= left) continue;
                    if (F32)
                        static_cast<float*>(p)[i0 + i + e] = v[k + e];
                    else
                        static_cast<uint16_t*>(p)[i0 + i + e] = f32_to_bf16_bits(v[k + e]);
                }
            }
        }
    }
};

// f(tag) with the Slice for a tensor's type and alignment.
template <class F>
__device__ __forceinline__ void by_slice(bool f32, bool vec, F f)
{
    if (f32)
        vec ? f(Slice<true, true>{}) : f(Slice<true, false>{});
    else
        vec ? f(Slice<false, true>{}) : f(Slice<false, false>{});
}

// The tensor that unit u belongs to.
template <int CAP>
__device__ __forceinline__ int find_tensor(const Table<CAP>& t, int u)
{
    int lo = 0, hi = t.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.first[mid] <= u)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ double warp_sum_f64(double v)
{
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// Sum of the squares of a warp's 1024 elements. In fp32, unless the largest is so
// large that its square overflows or so small that squares are lost below fp32's
// range: then in 64 bits from the same registers (unrolled as well: a loop that
// indexes them moves all elements to local memory, and both passes over 2.1 GB took
// 1.26 instead of 1.00 ms). 64-bit additions are rare on purpose: this GPU does two
// a clock and SM, and sums of blocks in which every thread took part in them cost 8
// of the 15 us of a call on 500 one-element tensors.
__device__ __forceinline__ double sum_squares(const float (&v)[kPer])
{
    float s[4] = {0.f, 0.f, 0.f, 0.f}, m = 0.f;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        s[k & 3] = fmaf(v[k], v[k], s[k & 3]);
        m = fmaxf(m, fabsf(v[k]));
    }
    if (__any_sync(0xffffffffu, m > 0x1p+58f || (m < 0x1p-40f && m > 0.f))) {
        double d = 0.0;
#pragma unroll
        for (int k = 0; k < kPer; ++k) d = fma((double)v[k], (double)v[k], d);
        return warp_sum_f64(d);
    }
    return (double)warp_sum((s[0] + s[1]) + (s[2] + s[3]));
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    k_sumsq(const __grid_constant__ Table<CAP> t, double* __restrict__ partial)
{
    double s = 0.0;
    const int u0 = t.from(blockIdx.x), u1 = t.from(blockIdx.x + 1);
    int k = u0 < u1 ? find_tensor(t, u0) : 0;
    for (int u = u0; u < u1; ++u) {
        while (u >= t.first[k + 1]) ++k;
        const int64_t i0 = (int64_t)(u - t.first[k]) * kUnit;
        const int left = (int)min((int64_t)kUnit, t.numel[k] - i0);
        by_slice(t.f32[k], t.vec[k], [&](auto slice) {
            float v[kPer];
            slice.load(t.in[k], i0, left, v);
            s += sum_squares(v);
        });
    }
    __shared__ double part[kThreads / 32];
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x < 32) {  // one warp: the others' additions would wait for the same unit
        s = part[0];
#pragma unroll
        for (int i = 1; i < kThreads / 32; ++i) s += part[i];
        if (threadIdx.x == 0) partial[blockIdx.x] = s;
    }
}

// n_partial sums were written; this launch scales the tensors of its table.
template <int CAP>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    k_clip_scale(const __grid_constant__ Table<CAP> t, const double* __restrict__ partial, int n_partial,
                 float max_norm, float* __restrict__ norm_out)
{
    __shared__ float norm_s, factor_s, shift_s;
    if (threadIdx.x < 32) {
        double s = 0.0;
        for (int i = threadIdx.x; i < n_partial; i += 32 * 8) {
            double v[8];  // asked for together
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = i + 32 * k < n_partial ? partial[i + 32 * k] : 0.0;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (i + 32 * k < n_partial) s += v[k];
        }
        s = warp_sum_f64(s);
        if (threadIdx.x == 0) {
            const double norm64 = sqrt(s);
            const float norm = (float)norm64;
            // by comparison, as the quotient of two zeros or two infinities has no value: an infinite bound
            // leaves everything, a NaN norm gives a NaN factor, an infinite one 0 (NaN where g is infinite);
            // finite elements whose norm passes fp32's range still have a factor. Factors that fp32 would hold
            // with few bits, or not at all, leave a power of two of theirs aside. (Only those are divided in 64
            // bits, which would cost every call a microsecond.)
            float c = norm <= max_norm || max_norm == INFINITY ? 1.f : max_norm / norm, shift = 1.f;
            if (c < 0x1p-100f && isfinite(norm64)) {
                shift = 0x1p-60f;
                c = (float)((double)max_norm / norm64 * 0x1p+60);
            }
            norm_s = norm;
            factor_s = c;
            shift_s = shift;
        }
    }
    __syncthreads();
    const float c = factor_s, shift = shift_s;
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm_out = norm_s;
    const int u0 = t.from(blockIdx.x), u1 = t.from(blockIdx.x + 1);
    int k = u0 < u1 ? find_tensor(t, u1 - 1) : 0;
    for (int u = u1 - 1; u >= u0; --u) {
        while (u < t.first[k]) --k;
        if (c == 1.f && t.in[k] == t.out[k]) continue;
        const int64_t i0 = (int64_t)(u - t.first[k]) * kUnit;
        const int left = (int)min((int64_t)kUnit, t.numel[k] - i0);
        by_slice(t.f32[k], t.vec[k], [&](auto slice) {
            float v[kPer];
            slice.load(t.in[k], i0, left, v);
            if (c != 1.f) {
#pragma unroll
                for (int e = 0; e < kPer; ++e) v[e] = v[e] * shift * c;
            }
            slice.store(t.out[k], i0, left, v);
        });
    }
}

// Both passes over the tensors, CAP of them a launch.
template <int CAP>
twell_status run_clip(const twell_tensor_list* list, float max_norm, float* norm, double* partial, cudaStream_t s)
{
    int n_partial = 0;
    Table<CAP> t;
    for (int pass = 0; pass < 2; ++pass) {
        int next = 0;
        do {
            if (pass == 0 || list->n > CAP) {  // a list of one table: pass 1 takes pass 0's
                t.n = 0;
                int64_t units = 0;
                while (next < list->n && t.n < CAP) {
                    const int64_t n = list->numel[next];
                    const int64_t more = (n + kUnit - 1) / kUnit;
                    if (units + more > INT32_MAX / 2 && t.n > 0) break;
                    if (n > 0) {
                        t.in[t.n] = list->in[next];
                        t.out[t.n] = list->out[next];
                        t.numel[t.n] = n;
                        t.first[t.n] = (int32_t)units;
                        t.f32[t.n] = list->type[next] == TWELL_F32;
                        t.vec[t.n] = ((reinterpret_cast<uintptr_t>(list->in[next]) |
                                       reinterpret_cast<uintptr_t>(list->out[next])) & 15u) == 0;
                        units += more;
                        ++t.n;
                    }
                    ++next;
                }
                t.first[t.n] = (int32_t)units;
                if (list->n <= CAP && next < list->n) return TWELL_ERR_UNSUPPORTED;  // more units than a table counts
            }
            const int units = t.first[t.n];
            const int blocks = units < 1 ? 1 : units < kMaxBlocks ? units : kMaxBlocks;
            if (pass == 0 && n_partial + blocks > kMaxBlocks * kMaxLaunches) return TWELL_ERR_UNSUPPORTED;
            count_launches(1);
            if (pass == 0) {
                k_sumsq<CAP><<<blocks, kThreads, 0, s>>>(t, partial + n_partial);
                n_partial += blocks;
            } else {
                k_clip_scale<CAP><<<blocks, kThreads, 0, s>>>(t, partial, n_partial, max_norm, norm);
            }
            if (cudaGetLastError() != cudaSuccess) return TWELL_ERR_CUDA;
        } while (next < list->n && list->n > CAP);
    }
    return TWELL_OK;
}

}  // namespace
}  // namespace twell

using namespace twell;

extern "C" size_t twell_grad_clip_workspace_bytes(void) { return (size_t)kMaxBlocks * kMaxLaunches * sizeof(double); }

extern "C" twell_status twell_grad_clip(const twell_tensor_list* list, float max_norm, float* norm, void* ws,
                                        size_t ws_bytes, void* stream)
{
    if (!list || !norm || list->n < 0 || !(max_norm >= 0.f)) return TWELL_ERR_INVALID_ARG;
    if (list->n > 0 && (!list->in || !list->out || !list->numel || !list->type)) return TWELL_ERR_INVALID_ARG;
    if (list->n > kTable * kMaxLaunches) return TWELL_ERR_UNSUPPORTED;
    for (int i = 0; i < list->n; ++i) {
        const int64_t n = list->numel[i];
        const int type = list->type[i];
        if (n < 0 || (type != TWELL_BF16 && type != TWELL_F32)) return TWELL_ERR_INVALID_ARG;
        const uintptr_t mask = type == TWELL_F32 ? 3 : 1;
        if (n > 0 && (!list->in[i] || !list->out[i] || (reinterpret_cast<uintptr_t>(list->in[i]) & mask) ||
                      (reinterpret_cast<uintptr_t>(list->out[i]) & mask)))
            return TWELL_ERR_INVALID_ARG;
        if (n > (int64_t)kUnit * (INT32_MAX / 2)) return TWELL_ERR_UNSUPPORTED;
    }
    if (!ws || ws_bytes < twell_grad_clip_workspace_bytes()) return TWELL_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(ws) & 255u) return TWELL_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    double* partial = static_cast<double*>(ws);
    return list->n <= kSmallTable ? run_clip<kSmallTable>(list, max_norm, norm, partial, s)
                                  : run_clip<kTable>(list, max_norm, norm, partial, s);
}
