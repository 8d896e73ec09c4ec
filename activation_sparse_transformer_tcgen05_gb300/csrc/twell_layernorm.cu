// twell_layernorm.cu — layer norm's forward and backward pass around the
// feed-forward layer, with the residual sum and the weight's gradient.
//
//   forward   s = x + res, hat = (s - mean) rstd, y = hat w + b
//   backward  v = w dy, dx = rstd (v - mean(v) - hat mean(v hat)) + dres,
//             dw = sum_r dy hat, db = sum_r dy
#include "common.cuh"
#include "launch.h"

namespace twell {
namespace {

struct f32_t {
    using type = float;
    static __device__ __forceinline__ float load(const float* p) { return *p; }
    static __device__ __forceinline__ void store(float* p, float v) { *p = v; }
};
struct bf16_t {
    using type = uint16_t;
    static __device__ __forceinline__ float load(const uint16_t* p) { return bf16_to_f32(*p); }
    static __device__ __forceinline__ void store(uint16_t* p, float v) { *p = f32_to_bf16_bits(v); }
};

struct FwdArgs {
    const void *x, *res, *w, *b;
    void *sum, *y;
    int64_t ldx, ldres, ldsum, ldy, N;
    int d;
    float eps;
    float *mean, *rstd;
};

struct BwdArgs {
    const void *dy, *x, *w, *dres;
    void* dx;
    int64_t lddy, ldx, lddres, lddx, N;
    int d;
    const float *mean, *rstd;
    float* part;  // [parts, 2, d] partial sums of dw and db; null: not wanted
    int parts;
};

constexpr int kRowThreads = 256;
constexpr int kMaxParts = 304;

// Sums of a and b over the block; every thread gets them.
__device__ __forceinline__ float2 block_sum2(float a, float b, float2* buf)
{
    a = warp_sum(a);
    b = warp_sum(b);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    float2 s = buf[0];
    for (int i = 1; i < (int)(blockDim.x >> 5); ++i) {
        s.x += buf[i].x;
        s.y += buf[i].y;
    }
    return s;
}

// One block per row, the row read three times (from L2 after the first).
template <class TX, class TY, class TW>
__global__ void __launch_bounds__(kRowThreads) k_ln_fwd_long(const FwdArgs a)
{
    __shared__ float2 buf[kRowThreads / 32];
    const typename TW::type* w = static_cast<const typename TW::type*>(a.w);
    const typename TW::type* b = static_cast<const typename TW::type*>(a.b);
    for (int64_t r = blockIdx.x; r < a.N; r += gridDim.x) {
        const typename TX::type* x = static_cast<const typename TX::type*>(a.x) + r * a.ldx;
        const typename TX::type* res = a.res ? static_cast<const typename TX::type*>(a.res) + r * a.ldres : nullptr;
        typename TX::type* sum = res ? static_cast<typename TX::type*>(a.sum) + r * a.ldsum : nullptr;
        typename TY::type* y = static_cast<typename TY::type*>(a.y) + r * a.ldy;
        float s = 0.f;
        for (int i = threadIdx.x; i < a.d; i += kRowThreads) {
            float v = TX::load(x + i);
            if (res) {
                TX::store(sum + i, v + TX::load(res + i));
                v = TX::load(sum + i);
            }
            s += v;
        }
        const typename TX::type* from = res ? sum : x;
        const float mean = block_sum2(s, 0.f, buf).x / (float)a.d;
        float q = 0.f;
        for (int i = threadIdx.x; i < a.d; i += kRowThreads) {
            const float c = TX::load(from + i) - mean;
            q += c * c;
        }
        const float rstd = 1.f / sqrtf(block_sum2(q, 0.f, buf).x / (float)a.d + a.eps);
        for (int i = threadIdx.x; i < a.d; i += kRowThreads) {
            const float hat = (TX::load(from + i) - mean) * rstd;
            TY::store(y + i, fmaf(hat, w ? TW::load(w + i) : 1.f, b ? TW::load(b + i) : 0.f));
        }
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
    }
}

// dx, one block per row, the row read twice.
template <class TX, class TY, class TW>
__global__ void __launch_bounds__(kRowThreads) k_ln_bwd_long(const BwdArgs a)
{
    __shared__ float2 buf[kRowThreads / 32];
    const typename TW::type* w = static_cast<const typename TW::type*>(a.w);
    for (int64_t r = blockIdx.x; r < a.N; r += gridDim.x) {
        const typename TX::type* x = static_cast<const typename TX::type*>(a.x) + r * a.ldx;
        const typename TX::type* dres = a.dres ? static_cast<const typename TX::type*>(a.dres) + r * a.lddres : nullptr;
        const typename TY::type* dy = static_cast<const typename TY::type*>(a.dy) + r * a.lddy;
        typename TX::type* dx = static_cast<typename TX::type*>(a.dx) + r * a.lddx;
        const float mean = a.mean[r], rstd = a.rstd[r];
        float s1 = 0.f, s2 = 0.f;
        for (int i = threadIdx.x; i < a.d; i += kRowThreads) {
            const float hat = (TX::load(x + i) - mean) * rstd;
            const float v = TY::load(dy + i) * (w ? TW::load(w + i) : 1.f);
            s1 += v;
            s2 += v * hat;
        }
        const float2 s = block_sum2(s1, s2, buf);
        const float c1 = s.x / (float)a.d, c2 = s.y / (float)a.d;
        for (int i = threadIdx.x; i < a.d; i += kRowThreads) {
            const float hat = (TX::load(x + i) - mean) * rstd;
            const float v = TY::load(dy + i) * (w ? TW::load(w + i) : 1.f);
            float g = rstd * (v - c1 - hat * c2);
            if (dres) g += TX::load(dres + i);
            TX::store(dx + i, g);
        }
    }
}

// Column sums of dy hat and dy over the rows of one part: block (32 columns,
// part), eight rows at a time.
template <class TX, class TY>
__global__ void __launch_bounds__(256) k_ln_cols_long(const BwdArgs a)
{
    const int col = blockIdx.x * 32 + threadIdx.x, ty = threadIdx.y;
    float dw = 0.f, db = 0.f;
    if (col < a.d) {
        for (int64_t r = (int64_t)blockIdx.y * 8 + ty; r < a.N; r += (int64_t)gridDim.y * 8) {
            const float x = TX::load(static_cast<const typename TX::type*>(a.x) + r * a.ldx + col);
            const float g = TY::load(static_cast<const typename TY::type*>(a.dy) + r * a.lddy + col);
            dw += g * ((x - a.mean[r]) * a.rstd[r]);
            db += g;
        }
    }
    __shared__ float2 buf[8][32];
    buf[ty][threadIdx.x] = make_float2(dw, db);
    __syncthreads();
    if (ty == 0 && col < a.d) {
        float2 s = buf[0][threadIdx.x];
        for (int i = 1; i < 8; ++i) {
            s.x += buf[i][threadIdx.x].x;
            s.y += buf[i][threadIdx.x].y;
        }
        a.part[((size_t)blockIdx.y * 2) * a.d + col] = s.x;
        a.part[((size_t)blockIdx.y * 2 + 1) * a.d + col] = s.y;
    }
}

// dw and db: the parts of 32 columns added by eight warps (every eighth part
// each, ascending), then the eight sums in order.
__global__ void __launch_bounds__(256)
    k_ln_reduce(const float* __restrict__ part, int parts, int d, float* __restrict__ dw, float* __restrict__ db)
{
    const int i = blockIdx.x * 32 + threadIdx.x, ty = threadIdx.y;  // column of [dw | db]
    float s = 0.f;
    if (i < 2 * d)
        for (int p = ty; p < parts; p += 8) s += part[(size_t)p * 2 * d + i];
    __shared__ float buf[8][32];
    buf[ty][threadIdx.x] = s;
    __syncthreads();
    if (ty == 0 && i < 2 * d) {
        for (int j = 1; j < 8; ++j) s += buf[j][threadIdx.x];
        if (i < d)
            dw[i] = s;
        else
            db[i - d] = s;
    }
}

int parts_for(int64_t N) { return N < kMaxParts * 8 ? (int)((N + 7) / 8) : kMaxParts; }

bool type_ok(int t) { return t == TWELL_BF16 || t == TWELL_F32; }

bool elem_aligned(const void* p, int type)
{
    return (reinterpret_cast<uintptr_t>(p) & (type == TWELL_F32 ? 3u : 1u)) == 0;
}

template <class TX, class TY, class TW>
cudaError_t fwd(const FwdArgs& a, cudaStream_t s)
{
    const unsigned grid = (unsigned)(a.N < 65536 ? a.N : 65536);
    count_launches(1);
    k_ln_fwd_long<TX, TY, TW><<<grid, kRowThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <class TX, class TY, class TW>
cudaError_t bwd(const BwdArgs& a, float* dw, float* db, cudaStream_t s)
{
    const unsigned grid = (unsigned)(a.N < 65536 ? a.N : 65536);
    count_launches(1);
    k_ln_bwd_long<TX, TY, TW><<<grid, kRowThreads, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !dw) return e;
    count_launches(2);
    k_ln_cols_long<TX, TY><<<dim3((unsigned)((a.d + 31) / 32), (unsigned)a.parts), dim3(32, 8), 0, s>>>(a);
    k_ln_reduce<<<(unsigned)((2 * (int64_t)a.d + 31) / 32), dim3(32, 8), 0, s>>>(a.part, a.parts, a.d, dw, db);
    return cudaGetLastError();
}

// f with the tags of the three types.
template <class F>
cudaError_t by_types(int x, int y, int w, F f)
{
    auto with_w = [&](auto tx, auto ty) {
        return w == TWELL_F32 ? f(tx, ty, f32_t{}) : f(tx, ty, bf16_t{});
    };
    auto with_y = [&](auto tx) { return y == TWELL_F32 ? with_w(tx, f32_t{}) : with_w(tx, bf16_t{}); };
    return x == TWELL_F32 ? with_y(f32_t{}) : with_y(bf16_t{});
}

}  // namespace
}  // namespace twell

using namespace twell;

extern "C" twell_status twell_layernorm_fwd(const void* x, int64_t ldx, const void* res, int64_t ldres, const void* w,
                                            const void* b, int64_t N, int d, float eps, int x_type, int y_type,
                                            int w_type, void* sum, int64_t ldsum, void* y, int64_t ldy, float* mean,
                                            float* rstd, void* stream)
{
    if (N < 0 || d < 1 || !type_ok(x_type) || !type_ok(y_type) || !type_ok(w_type) || !(eps >= 0.f))
        return TWELL_ERR_INVALID_ARG;
    if (N == 0) return TWELL_OK;
    if (!x || !y || (res != nullptr) != (sum != nullptr) || ldx < d || ldy < d || (res && (ldres < d || ldsum < d)))
        return TWELL_ERR_INVALID_ARG;
    if (y == x || y == res || (sum && (sum == x || sum == res || sum == y))) return TWELL_ERR_INVALID_ARG;
    if (!elem_aligned(x, x_type) || !elem_aligned(res, x_type) || !elem_aligned(sum, x_type) ||
        !elem_aligned(y, y_type) || !elem_aligned(w, w_type) || !elem_aligned(b, w_type) ||
        !elem_aligned(mean, TWELL_F32) || !elem_aligned(rstd, TWELL_F32))
        return TWELL_ERR_INVALID_ARG;
    const FwdArgs a{x, res, w, b, sum, y, ldx, ldres, ldsum, ldy, N, d, eps, mean, rstd};
    const cudaError_t e = by_types(x_type, y_type, w_type, [&](auto tx, auto ty, auto tw) {
        return fwd<decltype(tx), decltype(ty), decltype(tw)>(a, static_cast<cudaStream_t>(stream));
    });
    return e == cudaSuccess ? TWELL_OK : TWELL_ERR_CUDA;
}

extern "C" size_t twell_layernorm_bwd_workspace_bytes(int64_t N, int d)
{
    if (N < 0 || d < 1) return 0;
    const size_t n = (size_t)parts_for(N) * 2 * d * sizeof(float);
    return n > 256 ? n : 256;
}

extern "C" twell_status twell_layernorm_bwd(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* w,
                                            const float* mean, const float* rstd, const void* dres, int64_t lddres,
                                            int64_t N, int d, int x_type, int y_type, int w_type, void* dx,
                                            int64_t lddx, float* dw, float* db, void* ws, size_t ws_bytes,
                                            void* stream)
{
    if (N < 0 || d < 1 || !type_ok(x_type) || !type_ok(y_type) || !type_ok(w_type) || (dw != nullptr) != (db != nullptr))
        return TWELL_ERR_INVALID_ARG;
    if (!elem_aligned(dw, TWELL_F32) || !elem_aligned(db, TWELL_F32)) return TWELL_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (N == 0) {
        if (dw && (cudaMemsetAsync(dw, 0, (size_t)d * 4, s) != cudaSuccess ||
                   cudaMemsetAsync(db, 0, (size_t)d * 4, s) != cudaSuccess))
            return TWELL_ERR_CUDA;
        return TWELL_OK;
    }
    if (!dy || !x || !mean || !rstd || !dx || lddy < d || ldx < d || lddx < d || (dres && lddres < d))
        return TWELL_ERR_INVALID_ARG;
    if (dx == x || dx == dy || dx == dres) return TWELL_ERR_INVALID_ARG;
    if (!elem_aligned(x, x_type) || !elem_aligned(dres, x_type) || !elem_aligned(dx, x_type) ||
        !elem_aligned(dy, y_type) || !elem_aligned(w, w_type) || !elem_aligned(mean, TWELL_F32) ||
        !elem_aligned(rstd, TWELL_F32))
        return TWELL_ERR_INVALID_ARG;
    if (!ws || ws_bytes < twell_layernorm_bwd_workspace_bytes(N, d)) return TWELL_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(ws) & 255u) return TWELL_ERR_INVALID_ARG;
    const BwdArgs a{dy, x, w, dres, dx, lddy, ldx, lddres, lddx, N, d, mean, rstd,
                    dw ? static_cast<float*>(ws) : nullptr, parts_for(N)};
    const cudaError_t e = by_types(x_type, y_type, w_type, [&](auto tx, auto ty, auto tw) {
        return bwd<decltype(tx), decltype(ty), decltype(tw)>(a, dw, db, s);
    });
    return e == cudaSuccess ? TWELL_OK : TWELL_ERR_CUDA;
}
