// twell_clip.cu — L2 norm over many tensors, and the tensors scaled so that it
// is at most a bound.
//
//   norm = sqrt(sum over all elements of g^2),  c = min(1, max_norm / norm)
//   out = c g, rounded once to the tensor's type
//
// Bound by memory: every element is read for the norm, and read and written
// again scaled (12 bytes in fp32). The tensors' addresses travel in the
// launch's parameters (up to kTable of them a launch), so nothing is copied to
// the device first.
//
//   k_sumsq       every block sums the squares of its share of the elements
//   k_clip_scale  every block adds the blocks' sums in the same fixed order and
//                 scales its share
#include "common.cuh"
#include "launch.h"

namespace twell {
namespace {

constexpr int kThreads = 256;
constexpr int kTable = 512;         // tensors of one launch
constexpr int kChunk = 8192;        // elements of one unit of work
constexpr int kMaxBlocks = 608;     // four blocks on each of 152 SMs; partial sums of one launch
constexpr int kMaxLaunches = 64;    // 32768 tensors

struct Table {
    const void* in[kTable];
    void* out[kTable];
    int64_t numel[kTable];
    int32_t first[kTable + 1];  // first unit of each tensor
    uint8_t f32[kTable];
    int n;
};

// The tensor that unit u belongs to.
__device__ __forceinline__ int find_tensor(const Table& t, int u)
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

__device__ __forceinline__ float load1(const void* p, bool f32, int64_t i)
{
    return f32 ? static_cast<const float*>(p)[i] : bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
}

__device__ double block_sum(double v)
{
    __shared__ double part[kThreads / 32];
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) s += part[i];
    return s;
}

__global__ void __launch_bounds__(kThreads) k_sumsq(const __grid_constant__ Table t, double* __restrict__ partial)
{
    double s = 0.0;
    for (int u = blockIdx.x; u < t.first[t.n]; u += gridDim.x) {
        const int k = find_tensor(t, u);
        const int64_t i0 = (int64_t)(u - t.first[k]) * kChunk;
        const int64_t i1 = i0 + kChunk < t.numel[k] ? i0 + kChunk : t.numel[k];
        for (int64_t i = i0 + threadIdx.x; i < i1; i += kThreads) {
            const double g = (double)load1(t.in[k], t.f32[k], i);
            s += g * g;
        }
    }
    s = block_sum(s);
    if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// n_partial sums were written; this launch scales the tensors of its table.
__global__ void __launch_bounds__(kThreads)
    k_clip_scale(const __grid_constant__ Table t, const double* __restrict__ partial, int n_partial, float max_norm,
                 float* __restrict__ norm_out)
{
    double s = 0.0;
    for (int i = threadIdx.x; i < n_partial; i += kThreads) s += partial[i];
    const float norm = (float)sqrt(block_sum(s));
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm_out = norm;
    // a norm that is NaN keeps a NaN factor; an infinite one gives 0 (NaN where g is infinite)
    const float r = max_norm / norm;
    const float c = r >= 1.f ? 1.f : r;
    for (int u = blockIdx.x; u < t.first[t.n]; u += gridDim.x) {
        const int k = find_tensor(t, u);
        if (c == 1.f && t.in[k] == t.out[k]) continue;
        const int64_t i0 = (int64_t)(u - t.first[k]) * kChunk;
        const int64_t i1 = i0 + kChunk < t.numel[k] ? i0 + kChunk : t.numel[k];
        for (int64_t i = i0 + threadIdx.x; i < i1; i += kThreads) {
            const float g = load1(t.in[k], t.f32[k], i) * c;
            if (t.f32[k])
                static_cast<float*>(t.out[k])[i] = g;
            else
                static_cast<uint16_t*>(t.out[k])[i] = f32_to_bf16_bits(g);
        }
    }
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
        if (n > (int64_t)kChunk * (INT32_MAX / 2)) return TWELL_ERR_UNSUPPORTED;
    }
    if (!ws || ws_bytes < twell_grad_clip_workspace_bytes()) return TWELL_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(ws) & 255u) return TWELL_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    double* partial = static_cast<double*>(ws);
    int n_partial = 0;
    for (int pass = 0; pass < 2; ++pass) {
        int next = 0;
        do {
            Table t;
            t.n = 0;
            int64_t units = 0;
            while (next < list->n && t.n < kTable) {
                const int64_t n = list->numel[next];
                const int64_t more = (n + kChunk - 1) / kChunk;
                if (units + more > INT32_MAX / 2 && t.n > 0) break;
                if (n > 0) {
                    t.in[t.n] = list->in[next];
                    t.out[t.n] = list->out[next];
                    t.numel[t.n] = n;
                    t.first[t.n] = (int32_t)units;
                    t.f32[t.n] = list->type[next] == TWELL_F32;
                    units += more;
                    ++t.n;
                }
                ++next;
            }
            t.first[t.n] = (int32_t)units;
            const int blocks = units < 1 ? 1 : units < kMaxBlocks ? (int)units : kMaxBlocks;
            if (pass == 0 && n_partial + blocks > kMaxBlocks * kMaxLaunches) return TWELL_ERR_UNSUPPORTED;
            count_launches(1);
            if (pass == 0) {
                k_sumsq<<<blocks, kThreads, 0, s>>>(t, partial + n_partial);
                n_partial += blocks;
            } else {
                k_clip_scale<<<blocks, kThreads, 0, s>>>(t, partial, n_partial, max_norm, norm);
            }
            if (cudaGetLastError() != cudaSuccess) return TWELL_ERR_CUDA;
        } while (next < list->n);
    }
    return TWELL_OK;
}
