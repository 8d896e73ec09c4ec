// twell_linear.cu — linear layer with bias, activation and residual, and its backward.
//
//   pre = x W^T + bias, y = act(pre) + res
//   dpre = dy act'(pre);  dx = dpre W,  dW = dpre^T x,  dbias = column sums of dpre
//
// The products are twell_mm.cu's; W is read as it lies, [N, K] or [K, N], in all three.
// k_linear_dpre forms dpre once for both gradients, rounded to bf16 as the tensor cores'
// operand (dbias is summed from the fp32 values); without an activation dy itself is the
// operand, unless its rows do not start on 16-byte boundaries, and this pass only sums.
#include "activation.cuh"
#include "common.cuh"
#include "launch.h"
#include "mm.h"

namespace twell {
namespace {

int sms_current()
{
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) !=
                                                  cudaSuccess)
        return 0;
    return n;
}

bool aligned(const void* p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

constexpr int kMostDim = 1 << 30;
constexpr int kDpreThreads = 128;

size_t round256(size_t v) { return (v + 255) & ~size_t(255); }
int64_t padded(int n) { return ((int64_t)n + 63) / 64 * 64; }

// kSumRows rows a block: dpre = dy act'(pre) (pre null: dy) to out, if there is one, and the rows' sums in fp32 to part,
// if there is one. V = 8: rows of dy, pre and out in 16-byte pieces. Narrow matrices: `split` threads share a column's
// rows (each every split-th) and their sums are added in order (3789 x 16: 32 rows in a row took 25 us).
template <int V, bool SPLIT>
__global__ void __launch_bounds__(kDpreThreads)
    k_linear_dpre(const uint16_t* __restrict__ dy, int64_t lddy, const uint16_t* __restrict__ pre, int64_t ldpre, int M, int N,
                  int act, uint16_t* __restrict__ out, int64_t ldout, float* __restrict__ part, int split_arg, int col0,
                  const int32_t* __restrict__ status)
{
    if (has_error(status)) return;
    __shared__ float shared[V][SPLIT ? kDpreThreads : 1];
    const int split = SPLIT ? split_arg : 1;
    const int r0 = (int)blockIdx.x * kSumRows, rows = min(kSumRows, M - r0);
    const int wide = kDpreThreads / split, first = (int)threadIdx.x / wide;  // threads across, this one's first row
    const int c = col0 + ((int)blockIdx.y * wide + (int)threadIdx.x % wide) * V;
    if (!SPLIT && c >= N) return;
    float sum[V];
#pragma unroll
    for (int e = 0; e < V; ++e) sum[e] = 0.f;
    if (c < N) by_activation(pre ? act : TWELL_ACT_NONE, [&](auto tag) {
        constexpr int ACT = decltype(tag)::value;
#pragma unroll 2  // (more at once: fewer threads on an SM; sums of 8192 x 16384: 1 105 us, 2 103, 4 140, 8 152)
        for (int r = SPLIT ? first : 0; r < rows; r += split) {
            const size_t row = (size_t)r0 + r;
            float d[V];
            if constexpr (V == 8) {
                const uint4 q = *reinterpret_cast<const uint4*>(dy + row * lddy + c);
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
                uint32_t z[4] = {0, 0, 0, 0};
                if (ACT != TWELL_ACT_NONE) {
                    const uint4 p = *reinterpret_cast<const uint4*>(pre + row * ldpre + c);
                    z[0] = p.x, z[1] = p.y, z[2] = p.z, z[3] = p.w;
                }
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    float2 g = make_float2(bf16_lo(w[e >> 1]), bf16_hi(w[e >> 1]));
                    if (ACT != TWELL_ACT_NONE) {
                        float2 da;
                        activate<ACT>(make_float2(bf16_lo(z[e >> 1]), bf16_hi(z[e >> 1])), &da);
                        g = __fmul2_rn(g, da);
                    }
                    d[e] = g.x;
                    d[e + 1] = g.y;
                }
                if (out)
                    *reinterpret_cast<uint4*>(out + row * ldout + c) =
                        make_uint4(cvt_bf16x2(d[0], d[1]), cvt_bf16x2(d[2], d[3]), cvt_bf16x2(d[4], d[5]),
                                   cvt_bf16x2(d[6], d[7]));
            } else {
                d[0] = bf16_to_f32(dy[row * lddy + c]);
                if (ACT != TWELL_ACT_NONE) {
                    float2 da;
                    activate<ACT>(pair(bf16_to_f32(pre[row * ldpre + c])), &da);
                    d[0] *= da.x;
                }
                if (out) out[row * ldout + c] = f32_to_bf16_bits(d[0]);
            }
#pragma unroll
            for (int e = 0; e < V; ++e) sum[e] += d[e];
        }
    });
    if (SPLIT && part) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < V; ++e) shared[e][threadIdx.x] = sum[e];
        __syncthreads();
        if (first == 0) {
            for (int k = 1; k < split; ++k)
#pragma unroll
                for (int e = 0; e < V; ++e) sum[e] += shared[e][threadIdx.x + k * wide];
        }
    }
    if (part && first == 0 && c < N) {
#pragma unroll
        for (int e = 0; e < V; ++e) part[(size_t)blockIdx.x * N + c + e] = sum[e];
    }
}

bool act_ok(int act) { return act >= TWELL_ACT_NONE && act <= TWELL_ACT_GELU_TANH; }

bool dims_ok(int M, int N, int K, int w_kn)
{
    return M >= 0 && N > 0 && K > 0 && K % 8 == 0 && (w_kn == 0 || (w_kn == 1 && N % 8 == 0));
}
bool dims_fit(int M, int N, int K) { return M <= kMostDim && N <= kMostDim && K <= kMostDim; }

// Rows of bf16 that the tensor cores' loads can start on.
bool operand_ok(const void* p, int64_t ld, int width) { return p && aligned(p, 16) && ld >= width && ld % 8 == 0 && ld <= kMostDim; }

}  // namespace
}  // namespace twell

using namespace twell;

extern "C" twell_status twell_linear_fwd(const uint16_t* x, int64_t ldx, const uint16_t* W, int w_kn, const float* bias,
                                         int act, const void* res, int64_t ldres, int M, int N, int K, uint16_t* pre,
                                         int64_t ldpre, void* y, int64_t ldy, int y_type, int32_t* status, void* stream)
{
    if (!dims_ok(M, N, K, w_kn) || !act_ok(act) || (y_type != TWELL_BF16 && y_type != TWELL_F32)) return TWELL_ERR_INVALID_ARG;
    if (!dims_fit(M, N, K)) return TWELL_ERR_UNSUPPORTED;
    if (M == 0) return TWELL_OK;
    const size_t es = y_type == TWELL_F32 ? 4 : 2;
    if (!operand_ok(x, ldx, K) || !operand_ok(W, w_kn ? N : K, 1) || !y || !status || !aligned(y, es) || ldy < N ||
        !aligned(bias, 4) || !aligned(status, 4))
        return TWELL_ERR_INVALID_ARG;
    if ((res && (ldres < N || !aligned(res, es))) || (pre && (ldpre < N || !aligned(pre, 2)))) return TWELL_ERR_INVALID_ARG;
    if (shared({y, pre}, {x, W, bias}) || (pre && res == pre)) return TWELL_ERR_INVALID_ARG;
    // (in place: rows of y that lie elsewhere than those of res would replace some that are not read yet)
    if (y == res && ldy != ldres && M > 1) return TWELL_ERR_INVALID_ARG;
    const int sms = sms_current();
    if (sms <= 0) return TWELL_ERR_CUDA;
    MmLinear m{};
    m.M = M;
    m.N = N;
    m.K = K;
    m.segments = m.problems = 1;
    m.a[0] = {x, ldx, false};
    m.b[0] = {W, w_kn ? N : K, w_kn != 0};
    m.bias = bias;
    m.act = act;
    m.res = res;
    m.ldres = ldres;
    m.pre = pre;
    m.ldpre = ldpre;
    m.out[0] = y;
    m.ldo = ldy;
    m.out_f32 = y_type == TWELL_F32;
    m.status = status;
    return launch_mm_linear(m, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? TWELL_OK : TWELL_ERR_CUDA;
}

extern "C" size_t twell_linear_bwd_workspace_bytes(int M, int N, int K)
{
    if (!dims_ok(M, N, K, 0) || !dims_fit(M, N, K)) return 0;
    return round256((size_t)M * padded(N) * 2) + round256(((size_t)M + kSumRows - 1) / kSumRows * N * 4) + 256;
}

extern "C" twell_status twell_linear_bwd(const uint16_t* dy, int64_t lddy, const uint16_t* x, int64_t ldx, const uint16_t* W,
                                         int w_kn, int act, const uint16_t* pre, int64_t ldpre, int M, int N, int K,
                                         uint16_t* dx, int64_t lddx, void* dW, int dw_type, int accumulate, float* dbias,
                                         void* ws, size_t ws_bytes, int32_t* status, void* stream)
{
    if (!dims_ok(M, N, K, w_kn) || !act_ok(act) || (dw_type != TWELL_BF16 && dw_type != TWELL_F32) ||
        (accumulate && dw_type != TWELL_F32) || (!dx && !dW && !dbias))
        return TWELL_ERR_INVALID_ARG;
    if (!dims_fit(M, N, K)) return TWELL_ERR_UNSUPPORTED;
    if (!status || !aligned(status, 4) || !aligned(dW, 16) || !aligned(dbias, 4)) return TWELL_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (M == 0) {
        cudaError_t e = cudaSuccess;
        if (dW && !accumulate) e = cudaMemsetAsync(dW, 0, (size_t)N * K * (dw_type == TWELL_F32 ? 4 : 2), s);
        if (dbias && e == cudaSuccess) e = cudaMemsetAsync(dbias, 0, (size_t)N * 4, s);
        return e == cudaSuccess ? TWELL_OK : TWELL_ERR_CUDA;
    }
    if (!dy || lddy < N || !aligned(dy, 2) || (dW && !operand_ok(x, ldx, K)) || (dx && !operand_ok(W, w_kn ? N : K, 1)) ||
        (dx && (lddx < K || !aligned(dx, 2))))
        return TWELL_ERR_INVALID_ARG;
    if (act != TWELL_ACT_NONE && (!pre || ldpre < N || !aligned(pre, 2))) return TWELL_ERR_INVALID_ARG;
    if (shared({dx, dW, dbias, ws}, {dy, x, W, pre})) return TWELL_ERR_INVALID_ARG;
    if (!ws || ws_bytes < twell_linear_bwd_workspace_bytes(M, N, K)) return TWELL_ERR_WORKSPACE;
    if (!aligned(ws, 256)) return TWELL_ERR_INVALID_ARG;
    const int sms = sms_current();
    if (sms <= 0) return TWELL_ERR_CUDA;

    if (act == TWELL_ACT_NONE) pre = nullptr;
    uint16_t* own = static_cast<uint16_t*>(ws);
    float* part = reinterpret_cast<float*>(static_cast<char*>(ws) + round256((size_t)M * padded(N) * 2));
    MmOperand dpre{dy, lddy, false};
    const bool form = (dx || dW) && (pre || !operand_ok(dy, lddy, N));
    if (form) dpre = {own, padded(N), false};
    const int blocks = (M + kSumRows - 1) / kSumRows;
    cudaError_t e = cudaSuccess;
    if (form || dbias) {
        const bool vec = N % 8 == 0 && operand_ok(dy, lddy, N) && (!pre || operand_ok(pre, ldpre, N));
        const int v = vec ? 8 : 1;
        int split = 1;
        while (split < kSumRows && (int64_t)N * 2 * split <= (int64_t)kDpreThreads * v) split *= 2;
        const int wide = kDpreThreads / split;
        auto kern = vec ? (split > 1 ? k_linear_dpre<8, true> : k_linear_dpre<8, false>)
                        : (split > 1 ? k_linear_dpre<1, true> : k_linear_dpre<1, false>);
        // (a launch has at most 65535 blocks across)
        for (int64_t c = 0; c < N && e == cudaSuccess; c += 65535ll * wide * v) {
            const int64_t across = (N - c + wide * v - 1) / (wide * v);
            count_launches(1);
            kern<<<dim3((unsigned)blocks, (unsigned)(across < 65535 ? across : 65535)), kDpreThreads, 0, s>>>(
                dy, lddy, pre, ldpre, M, N, act, form ? own : nullptr, padded(N), dbias ? part : nullptr, split, (int)c, status);
            e = cudaGetLastError();
        }
        if (e == cudaSuccess && dbias) e = launch_block_sums(part, blocks, N, dbias, status, s);
    }
    MmLinear in{}, w{};
    in.M = M;
    in.N = K;
    in.K = N;
    in.segments = in.problems = 1;
    in.a[0] = dpre;
    in.b[0] = {W, w_kn ? N : K, w_kn == 0};  // [K, N]: K-major for this product
    in.out[0] = dx;
    in.ldo = lddx;
    in.status = status;
    const MmOperand rows{dpre.p, dpre.ld, true}, cols{x, ldx, true};
    w.M = w_kn ? K : N;
    w.N = w_kn ? N : K;
    w.K = M;
    w.segments = w.problems = 1;
    w.a[0] = w_kn ? cols : rows;
    w.b[0] = w_kn ? rows : cols;
    w.out[0] = dW;
    w.ldo = w.N;
    w.out_f32 = dw_type == TWELL_F32;
    w.accumulate = accumulate != 0;
    w.status = status;
    if (e == cudaSuccess) e = launch_mm_two(in, w, dx != nullptr, dW != nullptr, sms, s);
    return e == cudaSuccess ? TWELL_OK : TWELL_ERR_CUDA;
}
