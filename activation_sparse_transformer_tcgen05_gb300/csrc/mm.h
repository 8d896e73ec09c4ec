// mm.h — launchers of the dense products behind the linear and gated layers (twell_mm.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

namespace twell {

// Whether an output is an input or another output (null ones are neither).
inline bool shared(std::initializer_list<const void*> out, std::initializer_list<const void*> in)
{
    for (const void* const* o = out.begin(); o != out.end(); ++o) {
        if (!*o) continue;
        for (const void* i : in)
            if (i == *o) return true;
        for (const void* const* p = o + 1; p != out.end(); ++p)
            if (*p == *o) return true;
    }
    return false;
}

// A bf16 operand: `rows` x K, either K-major ([rows, K], ld >= K) or with mn set as its
// transpose ([K, rows], ld >= rows). ld a multiple of 8, p 16-byte aligned.
struct MmOperand {
    const uint16_t* p;
    int64_t ld;
    bool mn;
};

constexpr int kMmParts = 3;  // most products that one launch adds up or computes side by side

// out = act(sum over segments of A_s B_s^T + bias) + res, [M, N]; or with `problems` products side by
// side, out[p] = A_p B_p^T. All have the same M, N, K and operand layouts.
struct MmLinear {
    int M, N, K;
    int segments, problems;  // one of the two is 1
    MmOperand a[kMmParts], b[kMmParts];
    const float* bias;       // [N] or null
    int act;
    const void* res;         // [M, ldres] of out's type, or null; may be out itself
    int64_t ldres;
    uint16_t* pre;           // [M, ldpre] bf16: what the activation is taken of, or null
    int64_t ldpre;
    void* out[kMmParts];
    int64_t ldo;
    bool out_f32;
    bool accumulate;         // out += (fp32 only; no res)
    bool after_gated;        // the stream's launch before is launch_mm_gated's: it does not write W, so that W may be
                             //   loaded while it still runs
    int32_t* status;
};
cudaError_t launch_mm_linear(const MmLinear& m, int sms, cudaStream_t s);

// Two of them that do not need one another, in one launch or in two, whichever should be faster: A K-major in the first,
// A and B as transposes in the second. Or one of them alone (with_one, with_two): its sums are taken in the order that they
// have beside the other, so that its bits do not depend on it; of the other only sizes and strides are looked at.
cudaError_t launch_mm_two(const MmLinear& one, const MmLinear& two, bool with_one, bool with_two, int sms, cudaStream_t s);

// g = x Wg^T + bias, u = x Wu^T, h = act(g) u, all [M, F] bf16; g and u may be null (not kept).
struct MmGated {
    int M, F, K;
    const uint16_t *x, *Wg, *Wu;
    const float* bias;
    int act;
    uint16_t *g, *u, *h;
    int32_t* status;
};
cudaError_t launch_mm_gated(const MmGated& m, int sms, cudaStream_t s);

// dh = dy Wd^T + l1 sign(act(g) u), dg = dh u act'(g), du = dh act(g) [M, F] bf16; part [ceil(M / 32), F]:
// sums of dg in fp32 over 32 rows each, or null.
struct MmGatedBwd {
    int M, F, K;
    const uint16_t *dy, *Wd, *g, *u;
    int act;
    float l1;
    uint16_t *dg, *du;
    float* part;
    int32_t* status;
};
cudaError_t launch_mm_gated_bwd(const MmGatedBwd& m, int sms, cudaStream_t s);

// db[c] = sum over b of part[b, c], b ascending within 16 interleaved runs joined in order.
cudaError_t launch_block_sums(const float* part, int blocks, int n, float* db, const int32_t* status, cudaStream_t s);
constexpr int kSumRows = 32;  // rows of one partial column sum

}  // namespace twell
