// twell_gated.cu — the gated feed-forward layer computed densely, forward and backward.
//
//   g = x W_gate^T + b, u = x W_up^T, h = act(g) u, y = h W_down + res
//   dh = dy W_down^T + l1 sign(h), dg = dh u act'(g), du = dh act(g)
//   dx = dg W_gate + du W_up, dW_gate = dg^T x, dW_up = du^T x, dW_down = h^T dy, db = column sums of dg
//
// With act = ReLU this is the layer that twell_ffn_fwd serves sparsely (h packed by the gate's
// active units): here its weights are trained, and rows too dense to pack are served.
// Forward: two launches, h formed in the first one's epilogue from both projections. Backward:
// dg and du from dh's product, then dx as one product over both of them and the three weight
// gradients, in one launch or two; h, g and u are what the forward kept, in bf16.
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

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool dims_ok(int M, int d, int F) { return M >= 0 && d > 0 && F > 0 && d % 8 == 0 && F % 8 == 0; }
constexpr int kMostDim = 1 << 30;
bool dims_fit(int M, int d, int F) { return M <= kMostDim && d <= kMostDim && F <= kMostDim; }
bool act_ok(int act) { return act >= TWELL_ACT_NONE && act <= TWELL_ACT_GELU_TANH; }
size_t round256(size_t v) { return (v + 255) & ~size_t(255); }

}  // namespace
}  // namespace twell

using namespace twell;

extern "C" twell_status twell_dense_gated_ffn_fwd(const uint16_t* x, const uint16_t* W_gate, const uint16_t* W_up,
                                                  const float* b, const uint16_t* W_down, int act, const uint16_t* res, int M,
                                                  int d, int F, uint16_t* g, uint16_t* u, uint16_t* h, uint16_t* y,
                                                  int32_t* status, void* stream)
{
    if (!dims_ok(M, d, F) || !act_ok(act)) return TWELL_ERR_INVALID_ARG;
    if (!dims_fit(M, d, F)) return TWELL_ERR_UNSUPPORTED;
    if (M == 0) return TWELL_OK;
    if (!x || !W_gate || !W_up || !W_down || !h || !y || !status || (g == nullptr) != (u == nullptr)) return TWELL_ERR_INVALID_ARG;
    for (const void* p : {(const void*)x, (const void*)W_gate, (const void*)W_up, (const void*)W_down, (const void*)res,
                          (const void*)g, (const void*)u, (const void*)h, (const void*)y})
        if (!aligned16(p)) return TWELL_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(b) | reinterpret_cast<uintptr_t>(status)) & 3u) return TWELL_ERR_INVALID_ARG;
    // (g, u and h are written before res is read)
    if (shared({g, u, h, y}, {x, W_gate, W_up, b, W_down}) || shared({g, u, h}, {res})) return TWELL_ERR_INVALID_ARG;
    const int sms = sms_current();
    if (sms <= 0) return TWELL_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    MmGated up{};
    up.M = M;
    up.F = F;
    up.K = d;
    up.x = x;
    up.Wg = W_gate;
    up.Wu = W_up;
    up.bias = b;
    up.act = act;
    up.g = g;
    up.u = u;
    up.h = h;
    up.status = status;
    cudaError_t e = launch_mm_gated(up, sms, s);
    MmLinear down{};
    down.M = M;
    down.N = d;
    down.K = F;
    down.segments = down.problems = 1;
    down.a[0] = {h, F, false};
    down.b[0] = {W_down, d, true};
    down.res = res;
    down.ldres = d;
    down.out[0] = y;
    down.ldo = d;
    down.after_gated = true;
    down.status = status;
    if (e == cudaSuccess) e = launch_mm_linear(down, sms, s);
    return e == cudaSuccess ? TWELL_OK : TWELL_ERR_CUDA;
}

extern "C" size_t twell_dense_gated_bwd_workspace_bytes(int M, int d, int F)
{
    if (!dims_ok(M, d, F) || !dims_fit(M, d, F)) return 0;
    return 2 * round256((size_t)M * F * 2) + round256(((size_t)M + kSumRows - 1) / kSumRows * F * 4) + 256;
}

extern "C" twell_status twell_dense_gated_ffn_bwd(const uint16_t* x, const uint16_t* W_gate, const uint16_t* W_up,
                                                  const uint16_t* W_down, int act, const uint16_t* g, const uint16_t* u,
                                                  const uint16_t* h, const uint16_t* dy, float l1_coef, int M, int d, int F,
                                                  uint16_t* dx, void* dW_gate, void* dW_up, void* dW_down, int dw_type,
                                                  int accumulate, float* db, void* ws, size_t ws_bytes, int32_t* status,
                                                  void* stream)
{
    if (!dims_ok(M, d, F) || !act_ok(act) || (dw_type != TWELL_BF16 && dw_type != TWELL_F32) ||
        (accumulate && dw_type != TWELL_F32) || !status)
        return TWELL_ERR_INVALID_ARG;
    if (!dims_fit(M, d, F)) return TWELL_ERR_UNSUPPORTED;
    const int grads = (dW_gate != nullptr) + (dW_up != nullptr) + (dW_down != nullptr);
    if ((grads != 0 && grads != 3) || (!dx && !grads && !db)) return TWELL_ERR_INVALID_ARG;
    for (const void* p : {(const void*)x, (const void*)W_gate, (const void*)W_up, (const void*)W_down, (const void*)g,
                          (const void*)u, (const void*)h, (const void*)dy, (const void*)dx, (const void*)dW_gate,
                          (const void*)dW_up, (const void*)dW_down})
        if (!aligned16(p)) return TWELL_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(db) | reinterpret_cast<uintptr_t>(status)) & 3u) return TWELL_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    void* const dW[3] = {dW_gate, dW_up, dW_down};
    if (M == 0) {
        for (int i = 0; i < 3 && e == cudaSuccess; ++i)
            if (dW[i] && !accumulate) e = cudaMemsetAsync(dW[i], 0, (size_t)F * d * (dw_type == TWELL_F32 ? 4 : 2), s);
        if (db && e == cudaSuccess) e = cudaMemsetAsync(db, 0, (size_t)F * 4, s);
        return e == cudaSuccess ? TWELL_OK : TWELL_ERR_CUDA;
    }
    if (!W_down || !g || !u || !dy || (dx && (!W_gate || !W_up)) || (grads && (!x || !h))) return TWELL_ERR_INVALID_ARG;
    if (shared({dx, dW_gate, dW_up, dW_down, db, ws}, {x, W_gate, W_up, W_down, g, u, h, dy})) return TWELL_ERR_INVALID_ARG;
    if (!ws || ws_bytes < twell_dense_gated_bwd_workspace_bytes(M, d, F)) return TWELL_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return TWELL_ERR_INVALID_ARG;
    const int sms = sms_current();
    if (sms <= 0) return TWELL_ERR_CUDA;

    const size_t each = round256((size_t)M * F * 2);
    uint16_t* dg = static_cast<uint16_t*>(ws);
    uint16_t* du = reinterpret_cast<uint16_t*>(static_cast<char*>(ws) + each);
    float* part = reinterpret_cast<float*>(static_cast<char*>(ws) + 2 * each);
    MmGatedBwd hid{};
    hid.M = M;
    hid.F = F;
    hid.K = d;
    hid.dy = dy;
    hid.Wd = W_down;
    hid.g = g;
    hid.u = u;
    hid.act = act;
    hid.l1 = l1_coef;
    hid.dg = dg;
    hid.du = du;
    hid.part = db ? part : nullptr;
    hid.status = status;
    e = launch_mm_gated_bwd(hid, sms, s);
    if (e == cudaSuccess && db) e = launch_block_sums(part, (M + kSumRows - 1) / kSumRows, F, db, status, s);
    MmLinear in{}, w{};
    in.M = M;
    in.N = d;
    in.K = F;
    in.segments = 2;
    in.problems = 1;
    in.a[0] = {dg, F, false};
    in.a[1] = {du, F, false};
    in.b[0] = {W_gate, d, true};
    in.b[1] = {W_up, d, true};
    in.out[0] = dx;
    in.ldo = d;
    in.status = status;
    w.M = F;
    w.N = d;
    w.K = M;
    w.segments = 1;
    w.problems = 3;
    w.a[0] = {dg, F, true};
    w.a[1] = {du, F, true};
    w.a[2] = {h, F, true};
    w.b[0] = w.b[1] = {x, d, true};
    w.b[2] = {dy, d, true};
    for (int i = 0; i < 3; ++i) w.out[i] = dW[i];
    w.ldo = d;
    w.out_f32 = dw_type == TWELL_F32;
    w.accumulate = accumulate != 0;
    w.status = status;
    if (e == cudaSuccess) e = launch_mm_two(in, w, dx != nullptr, grads != 0, sms, s);
    return e == cudaSuccess ? TWELL_OK : TWELL_ERR_CUDA;
}
