// twell_xent.cu — softmax cross entropy of a linear head over a large
// vocabulary, with its gradient, without the logits.
//
//   z = x W^T          x [N, d] hidden rows, W [V, d] the head, one row per word
//   lse_r = log sum_j exp z_rj,   nll_r = lse_r - z_r,target(r)
//   dz_rj = exp(z_rj - lse_r) - [j = target(r)]
//   dx = g dz W,  dW = g dz^T x     g = grad_scale, or grad_scale / scored rows
//
// Three products of 2 N V d operations bound it. The softmax needs a whole row
// before its first gradient, so a gradient without stored logits either
// computes the logits twice (a fourth product) or keeps something smaller. What
// is kept here, for one chunk of rows at a time, are 16-bit codes of the
// logits' distances to their (row, 128 words) maximum, written by the first
// product's epilogue (twell_gemm.cu). One pass rewrites the codes in place as
// bf16 dz, the operand of the two other products; g enters with their fp32
// results, so that a target's -1 stays exact whatever g is. Six bytes a logit cost
// 0.9 ps at the memory's rate, a fourth product d * 1.03 fs: the codes cost
// less from d = 860 on, and they round dz once, as any bf16 operand is.
//
// Rows that are not scored (target == ignore_index) take no part: the scored
// rows are copied together first, so that a prompt or padding costs nothing in
// the products and whatever stands there (NaN too) reaches no gradient.
//
//   k_xent_prep    orders the rows (scored first), counts them, checks the targets
//   k_xent_gather  the scored rows of x together; zeros for the others (few rows:
//                  both in k_xent_prep_gather)
//   GEMM_XENT      codes, per-(row, 128 words) maxima and sums, target logits
//   k_xent_lse     one warp per row: lse, nll; the sum or mean of the losses
//   k_xent_dz      codes -> bf16 dz, in place
//   GEMM_SPLITK    dx; with few output tiles the vocabulary (its depth) is split
//                  over the GPU and k_xent_dx adds the parts in order
//   GEMM_SCALED    dx as a whole, and dW (operands read MN-major, nothing is transposed)
// Every sum is taken in a fixed order.
#include "common.cuh"
#include "launch.h"

namespace twell {
namespace {

constexpr int kPrepThreads = 1024;
constexpr int kPairsNominal = 76;  // CTA pairs the split of dx is planned for (152 SMs)
constexpr int kMaxSplits = 32;

struct XentWs {
    int32_t* count;     // scored rows
    float* gscale;      // gradient factor of a scored row
    int32_t* rows_dev;  // [chunks] scored rows of each chunk
    int32_t* k_dev;     // [chunks] the same as a depth of dW (at least 1 in chunk 0, so that dW is written)
    int2* split;        // [chunks] parts of dx and the k-blocks of one
    int32_t* perm;      // [N] scored rows ascending, then the others
    int32_t* target;    // [N] targets of the scored rows, in perm's order
    uint16_t* xs;       // [N, row_stride(d)] scored rows of x, zeros in the 64 rows after them
    int32_t* done;      // blocks of k_xent_lse that have finished
    float2* stat;       // [chunk, tiles] (maximum in log2 units, sum relative to it)
    float* ztarget;     // [chunk]
    float* lse2;        // [chunk] log2 of the sum of exponentials
    float* nll;         // [chunk]
    uint16_t* codes;    // [chunk, ldcode] codes, then bf16 dz
    float* parts;       // [parts, scored rows, d] partial dx
    float* dw_acc;      // [V, d] when a bf16 dW is summed over several chunks
};

size_t round256(size_t v) { return (v + 255) & ~size_t(255); }

// Row stride of the codes and of the scored rows of x: whole 128-byte lines. (Rows
// that start inside a line cost the tiles' loads a second line each: with rows of
// W and x of 1000 elements, 777 x 50001 losses took 85 us, of 1024 62 us.)
size_t row_stride(int n) { return ((size_t)n + 63) & ~size_t(63); }

// Parts of the depth V of dx = dz W, and the k-blocks of a part: each (256 x 256
// tile, part) is one unit of work of a CTA pair; the time is the waves of units
// times a unit's k-blocks (0.28 us each) plus its epilogue (about 8 k-blocks'
// worth), and what the parts' fp32 sums cost to write and read again. At most
// three waves of units, which bounds the parts' room.
constexpr int kMaxUnits = 3 * kPairsNominal;

// Estimated time of `s` parts (1 <= s <= kMaxSplits) in us; infinite where a part would be empty
// or the units too many.
__host__ __device__ inline float split_time(int s, int rows, int d, int V)
{
    const unsigned tiles = (unsigned)((rows + 255) / 256) * (unsigned)((d + 255) / 256);
    const unsigned num_kb = (unsigned)(V + 63) / 64;
    if ((unsigned)s > num_kb || (s > 1 && tiles > (unsigned)(kMaxUnits / s))) return INFINITY;
    const unsigned per = (num_kb + s - 1) / s;
    if ((num_kb + per - 1) / per != (unsigned)s) return INFINITY;
    const unsigned waves = (tiles * s + kPairsNominal - 1) / kPairsNominal;
    const float t = (float)waves * (float)(per + 8) * 0.28f;
    return s == 1 ? t : t + (float)s * (float)rows * (float)d * 1.6e-6f + 3.f;  // 8 bytes at ~5 TB/s, a launch
}

bool in_parts(int rows, int d, int V)
{
    for (int s = 2; s <= kMaxSplits; ++s)
        if (split_time(s, rows, d, V) < split_time(1, rows, d, V)) return true;
    return false;
}

// The best split for a number of rows known on the device; one warp, a lane for each number of parts.
__device__ __forceinline__ void plan_splits(int rows, int d, int V, int lane, int2* out)
{
    static_assert(kMaxSplits == 32, "one lane each");
    const float mine = split_time(lane + 1, rows, d, V);
    float best = mine;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) best = fminf(best, __shfl_xor_sync(0xffffffffu, best, off));
    const int s = __ffs(__ballot_sync(0xffffffffu, mine == best));
    const int num_kb = (V + 63) / 64;
    if (lane == 0) *out = make_int2(s, (num_kb + s - 1) / s);
}

// Elements of the parts for any number of scored rows up to `rows`.
size_t parts_elements(int rows, int d)
{
    const size_t most = (size_t)kMaxUnits * 256 * 256, all = (size_t)kMaxSplits * rows * d;
    return most < all ? most : all;
}

size_t carve(void* ws, int N, int chunk, int d, int V, bool grad, bool acc, XentWs* out)
{
    char* base = static_cast<char*>(ws);
    size_t used = 0;
    auto take = [&](size_t bytes) {
        char* p = base ? base + used : nullptr;
        used += round256(bytes);
        return p;
    };
    const size_t tiles = (size_t)(V + kXentTile - 1) / kXentTile;
    const size_t chunks = chunk > 0 ? ((size_t)N + chunk - 1) / chunk : 0;
    XentWs w{};
    w.count = reinterpret_cast<int32_t*>(take(4));
    w.gscale = reinterpret_cast<float*>(take(4));
    w.rows_dev = reinterpret_cast<int32_t*>(take(chunks * 4));
    w.k_dev = reinterpret_cast<int32_t*>(take(chunks * 4));
    w.split = reinterpret_cast<int2*>(take(chunks * 8));
    w.perm = reinterpret_cast<int32_t*>(take((size_t)N * 4));
    w.target = reinterpret_cast<int32_t*>(take((size_t)N * 4));
    w.xs = reinterpret_cast<uint16_t*>(take((size_t)N * row_stride(d) * 2));
    w.done = reinterpret_cast<int32_t*>(take(4));
    w.stat = reinterpret_cast<float2*>(take((size_t)chunk * tiles * 8));
    w.ztarget = reinterpret_cast<float*>(take((size_t)chunk * 4));
    w.lse2 = reinterpret_cast<float*>(take((size_t)chunk * 4));
    w.nll = reinterpret_cast<float*>(take((size_t)chunk * 4));
    if (grad) {
        w.codes = reinterpret_cast<uint16_t*>(take((size_t)chunk * row_stride(V) * 2));
        w.parts = reinterpret_cast<float*>(take(parts_elements(chunk, d) * 4));
        if (acc) w.dw_acc = reinterpret_cast<float*>(take((size_t)V * d * 4));
    }
    if (out) *out = w;
    return used;
}

// Inclusive sum over the lanes of a warp.
__device__ __forceinline__ int warp_scan(int v, int lane)
{
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += u;
    }
    return v;
}

// Order of the rows: scored ones ascending, then the others. Each thread of a block
// takes a run of consecutive rows: their counts are scanned, then each thread
// places its rows. place(position, row, target of a scored row).
struct Order {
    int total;  // scored rows
    bool bad;   // this thread saw a target outside the vocabulary
};
template <class F>
__device__ __forceinline__ Order order_rows(const int64_t* __restrict__ target, int N, int V, int64_t ignore_index, F place)
{
    const int run = (N + kPrepThreads - 1) / kPrepThreads;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long first = (long long)threadIdx.x * run;
    const int i0 = (int)(first < N ? first : N), i1 = (int)(first + run < N ? first + run : N);
    int n = 0;
    bool bad = false;
    for (int i = i0; i < i1; ++i) {
        const int64_t t = target[i];
        if (t == ignore_index) continue;
        ++n;
        bad |= t < 0 || t >= V;
    }
    const int incl = warp_scan(n, lane);
    __shared__ int part[kPrepThreads / 32], before[kPrepThreads / 32], total_s;
    if (lane == 31) part[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        const int p = part[lane];
        const int pi = warp_scan(p, lane);
        before[lane] = pi - p;
        if (lane == 31) total_s = pi;
    }
    __syncthreads();
    const int total = total_s;
    int at = before[warp] + incl - n;   // scored rows before this run
    int other = total + (i0 - at);      // place of the run's first unscored row
    for (int i = i0; i < i1; ++i) {
        const int64_t t = target[i];
        if (t == ignore_index)
            place(other++, i, 0, false);
        else
            place(at++, i, (int)t, true);
    }
    return Order{total, bad};
}

// What the later kernels read of the order: counts, gradient factor, splits of dx.
__device__ __forceinline__ void publish_order(const Order& o, int N, int d, int V, int chunk, int mean, float grad_scale,
                                              const XentWs& w)
{
    for (long long c = threadIdx.x; c * chunk < N; c += kPrepThreads) {
        const long long left = (long long)o.total - c * chunk;
        const int rows = (int)(left < 0 ? 0 : left < chunk ? left : chunk);
        w.rows_dev[c] = rows;
        w.k_dev[c] = rows == 0 && c == 0 ? 1 : rows;
    }
    if (w.parts) {  // gradients
        for (long long c = threadIdx.x >> 5; c * chunk < N; c += kPrepThreads / 32) {
            const long long left = (long long)o.total - c * chunk;
            plan_splits((int)(left < 0 ? 0 : left < chunk ? left : chunk), d, V, threadIdx.x & 31, w.split + c);
        }
    }
    if (threadIdx.x == 0) {
        *w.done = 0;
        *w.count = o.total;
        *w.gscale = mean ? grad_scale / (float)(o.total > 0 ? o.total : 1) : grad_scale;
    }
}

// Row i of the order, one warp: a scored row of x to its place, zeros in the 64
// rows after them (the depth of dW is read in steps of 64), and zero results for a
// row that is not scored.
__device__ __forceinline__ void gather_row(const uint16_t* __restrict__ x, int d, const XentWs& w, int ldx, long long i,
                                           int row, int count, int lane, float* __restrict__ nll,
                                           float* __restrict__ lse, uint16_t* __restrict__ dx)
{
    const int d8 = d / 8;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint4* to = reinterpret_cast<uint4*>(w.xs + (size_t)i * ldx);
    if (i < count) {
        const uint4* from = reinterpret_cast<const uint4*>(x + (size_t)row * d);
        for (int c = lane; c < d8; c += 32) to[c] = from[c];
        return;
    }
    if (i < (long long)count + 64)
        for (int c = lane; c < d8; c += 32) to[c] = zero;
    if (dx)
        for (int c = lane; c < d8; c += 32) reinterpret_cast<uint4*>(dx + (size_t)row * d)[c] = zero;
    if (lane == 0) {
        nll[row] = 0.f;
        lse[row] = 0.f;
    }
}

// The order by one block (16384 targets take 13 us) ...
__global__ void __launch_bounds__(kPrepThreads)
    k_xent_prep(const int64_t* __restrict__ target, int N, int d, int V, int64_t ignore_index, int chunk, int mean,
                float grad_scale, XentWs w, int32_t* status)
{
    const Order o = order_rows(target, N, V, ignore_index, [&](int pos, int row, int t, bool scored) {
        w.perm[pos] = row;
        if (scored) w.target[pos] = t;
    });
    if (o.bad) set_error(status, TWELL_ERR_INVALID_ARG);
    publish_order(o, N, d, V, chunk, mean, grad_scale, w);
}

// ... and then the rows of x; one warp per row.
__global__ void __launch_bounds__(256)
    k_xent_gather(const uint16_t* __restrict__ x, int N, int d, XentWs w, int ldx, float* __restrict__ nll,
                  float* __restrict__ lse, uint16_t* __restrict__ dx, const int32_t* status)
{
    if (has_error(status)) return;
    const int count = *w.count;
    for (long long i = blockIdx.x * 8 + (threadIdx.x >> 5); i < N; i += gridDim.x * 8)
        gather_row(x, d, w, ldx, i, w.perm[i], count, threadIdx.x & 31, nll, lse, dx);
}

// Both in one launch for few rows: every block orders all rows for itself and
// gathers its 32; block 0 publishes the order. Saves a launch (61 x 512 x 50001: 29.2
// against 30.7 us a call); with more rows every block would read more targets.
constexpr int kFewRows = 2048;

__global__ void __launch_bounds__(kPrepThreads)
    k_xent_prep_gather(const int64_t* __restrict__ target, const uint16_t* __restrict__ x, int N, int d, int V,
                       int64_t ignore_index, int chunk, int mean, float grad_scale, XentWs w, int ldx,
                       float* __restrict__ nll, float* __restrict__ lse, uint16_t* __restrict__ dx, int32_t* status)
{
    __shared__ int perm[kFewRows];
    const bool failed = has_error(status);  // asked for here, together with the targets; nothing is written then
    const bool first = blockIdx.x == 0;
    const Order o = order_rows(target, N, V, ignore_index, [&](int pos, int row, int t, bool scored) {
        perm[pos] = row;
        if (first) {
            w.perm[pos] = row;
            if (scored) w.target[pos] = t;
        }
    });
    if (o.bad) set_error(status, TWELL_ERR_INVALID_ARG);
    if (first) publish_order(o, N, d, V, chunk, mean, grad_scale, w);
    __syncthreads();
    const int i = blockIdx.x * (kPrepThreads / 32) + (threadIdx.x >> 5);
    if (i < N && !failed) gather_row(x, d, w, ldx, i, perm[i], o.total, threadIdx.x & 31, nll, lse, dx);
}

// a + b rounded, and what the rounding lost (operations that the compiler does not
// join with others).
__device__ __forceinline__ float two_sum(float a, float b, float* lost)
{
    const float s = __fadd_rn(a, b), bb = __fsub_rn(s, a);
    *lost = __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb));
    return s;
}

// One warp per scored row: the tiles' (maximum, sum) pairs joined, in the order
// of the lanes' strides and then a butterfly. In the call's last chunk the block
// that finishes last adds up the N losses, in a fixed order and with what each
// addition lost.
__device__ __forceinline__ void row_lse(const XentWs& w, int tiles, int row, int lane, const int32_t* targets,
                                        const int32_t* perm, float* nll, float* lse)
{
    // asked for first: each load a row waits for is a third of a microsecond of the call
    const float2* st = w.stat + (size_t)row * tiles;
    const float zt = w.ztarget[row];
    const float mt = st[targets[row] / kXentTile].x;
    const int to = perm[row];
    float m = -INFINITY;
    for (int t = lane; t < tiles; t += 32) m = fmaxf(m, st[t].x);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    // every logit -inf: the sum stays 0 and lse is -inf; a maximum of +inf or a
    // NaN logit leaves a NaN sum, and with it a NaN loss and gradient row
    float s = 0.f;
    for (int t = lane; t < tiles; t += 32) {
        const float2 v = st[t];
        if (v.x != -INFINITY || v.y != 0.f) s += v.y * exp2_approx(v.x - m);
    }
    s = warp_sum(s);
    if (lane != 0) return;
    const float lg = s == 0.f ? -INFINITY : logf(s);
    // The exponentials were taken of z c - m, with c log2(e) rounded to fp32 and m the maximum
    // of z c: m / c brings the maximum back as it was.
    constexpr double to_nats = 1.0 / (double)kXentLog2e;
    constexpr float hi = (float)to_nats, lo = (float)(to_nats - (double)hi);
    lse[to] = isfinite(lg) ? fmaf(m, hi, fmaf(m, lo, lg)) : lg;
    // The target's exponent t is the one its tile's sum has, so that it cancels against the log-sum: the loss of a
    // likely target keeps its digits beside logits of any size. A sum of approximate exponentials may
    // still be a little less than its largest one. (A tile without a finite logit has no maximum: t is then -inf.)
    const float t = mt == -INFINITY ? zt : fmaf(zt, kXentLog2e, -mt);
    const float below = (m - (mt == -INFINITY ? 0.f : mt)) - t;
    const float value = fmaf(below, hi, lg);
    const float loss = value < 0.f ? 0.f : value;
    nll[to] = loss;
    w.nll[row] = loss;
    w.lse2[row] = s == 0.f ? -INFINITY : m + log2f(s);
}

__global__ void __launch_bounds__(256)
    k_xent_lse(XentWs w, int tiles, const int32_t* __restrict__ rows_dev, const int32_t* __restrict__ targets,
               const int32_t* __restrict__ perm, float* nll, float* lse, int last_chunk, int N, int mean, float* loss,
               const int32_t* status)
{
    const int rows = *rows_dev, scored = *w.count;
    if (has_error(status)) return;
    const int row = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row < rows) row_lse(w, tiles, row, threadIdx.x & 31, targets, perm, nll, lse);
    if (!last_chunk) return;
    __shared__ bool last;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(w.done, 1) == (int)gridDim.x - 1;
    __syncthreads();
    if (!last) return;
    float s = 0.f, c = 0.f, lost;
    for (int i = threadIdx.x; i < N; i += 256) {
        s = two_sum(s, __ldcg(nll + i), &lost);
        c += lost;
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        c += __shfl_xor_sync(0xffffffffu, c, off);
        s = two_sum(s, __shfl_xor_sync(0xffffffffu, s, off), &lost);
        c += lost;
    }
    __shared__ float2 part[8];
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = make_float2(s, c);
    __syncthreads();
    if (threadIdx.x == 0) {
        // (a 64-bit division alone would take a microsecond here)
        for (int i = 1; i < 8; ++i) {
            s = two_sum(s, part[i].x, &lost);
            c += part[i].y + lost;
        }
        const float total = isfinite(s) ? s + c : s;
        *loss = scored == 0 ? 0.f : mean ? total / (float)scored : total;
    }
}

// Codes to bf16 dz in place, one warp per (row, 256 words), eight words a lane:
// dz = 2^(m2 - q / 2048 - lse2). The target's entry is p - 1 = expm1(-nll), which
// stays exact where p is close to 1. A row without a finite lse is NaN throughout.
// Bound by memory (4 bytes a logit). A code becomes a float as the low mantissa
// bits of 2^23 + code: an integer conversion shares the special-function unit with
// the exponential. Few registers and many warps do better than several pieces a
// thread (777 x 50001: 26 against 37 us with two; 8192 x 65536: 335 against 465).
__global__ void __launch_bounds__(256, 8)
    k_xent_dz(XentWs w, unsigned ldcode, int tiles, const int32_t* __restrict__ targets,
              const int32_t* __restrict__ rows_dev, int max_rows, const int32_t* status)
{
    if (has_error(status)) return;
    const int lane = threadIdx.x & 31;
    const int rows = *rows_dev;
    const int padded = min(max_rows, max((rows + 63) / 64 * 64, 64));  // zeros up to the depth dW reads
    const unsigned spans = (ldcode + 255) / 256;
    const unsigned step = gridDim.x * 8;
    // (row, span) of this warp, advanced by `step` spans at a time
    unsigned i = blockIdx.x * 8 + (threadIdx.x >> 5);
    unsigned row = i / spans, span = i % spans;
    const unsigned rows_step = step / spans, span_step = step % spans;
    for (; row < (unsigned)padded;) {
        const unsigned col = span * 256 + lane * 8;
        if (col < ldcode) {
            uint4* p = reinterpret_cast<uint4*>(w.codes + (size_t)row * ldcode + col);
            if (row >= (unsigned)rows) {
                *p = make_uint4(0, 0, 0, 0);
            } else {
                const uint4 q = *p;
                const float l2 = w.lse2[row];
                // (the padding past the last word has no tile of its own)
                const float m2 = w.stat[(size_t)row * tiles + min((int)(col / kXentTile), tiles - 1)].x;
                const int target = targets[row] - (int)col;
                const float shift = m2 - l2;
                const float one = isfinite(l2) ? 1.f : NAN;
                const uint32_t qw[4] = {q.x, q.y, q.z, q.w};
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float v =
                        __uint_as_float(__byte_perm(qw[e >> 1], 0x4b00u, (e & 1) ? 0x5432 : 0x5410)) - 8388608.f;
                    f[e] = v == (float)kXentZero ? 0.f : exp2_approx(fmaf(v, -1.f / kXentSteps, shift));
                    f[e] *= one;
                }
                if (target >= 0 && target < 8) {
                    const float ft = one * expm1f(-w.nll[row]);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (e == target) f[e] = ft;
                }
                *p = make_uint4(cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]), cvt_bf16x2(f[4], f[5]),
                                cvt_bf16x2(f[6], f[7]));
            }
        }
        row += rows_step;
        span += span_step;
        if (span >= spans) {
            span -= spans;
            ++row;
        }
    }
}

// dx = bf16 of g times the parts added in order, each scored row at its place.
__global__ void __launch_bounds__(256)
    k_xent_dx(const float* __restrict__ parts, const int2* __restrict__ split, const int32_t* __restrict__ rows_dev, int d,
              const float* __restrict__ scale, const int32_t* __restrict__ perm, uint16_t* __restrict__ dx,
              const int32_t* status)
{
    if (has_error(status)) return;
    const float g = *scale;
    const int d4 = d / 4, splits = split->x;
    const size_t n4 = (size_t)*rows_dev * d4, stride = n4 * 4;
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n4; i += (size_t)gridDim.x * 256) {
        float4 a = reinterpret_cast<const float4*>(parts)[i];
        for (int p = 1; p < splits; ++p) {
            const float4 b = reinterpret_cast<const float4*>(parts + p * stride)[i];
            a.x += b.x;
            a.y += b.y;
            a.z += b.z;
            a.w += b.w;
        }
        const size_t row = i / d4, c = i % d4;
        reinterpret_cast<uint2*>(dx + (size_t)perm[row] * d)[c] =
            make_uint2(cvt_bf16x2(g * a.x, g * a.y), cvt_bf16x2(g * a.z, g * a.w));
    }
}

// dW in bf16 from the sum over chunks; n4 groups of four elements.
__global__ void __launch_bounds__(256)
    k_xent_round(const float* __restrict__ acc, size_t n4, uint16_t* __restrict__ out, const int32_t* status)
{
    if (has_error(status)) return;
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n4; i += (size_t)gridDim.x * 256) {
        const float4 a = reinterpret_cast<const float4*>(acc)[i];
        reinterpret_cast<uint2*>(out)[i] = make_uint2(cvt_bf16x2(a.x, a.y), cvt_bf16x2(a.z, a.w));
    }
}

int sms_current()
{
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    return n;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool dims_ok(int N, int d, int V) { return N >= 0 && d > 0 && V > 0 && d % 8 == 0; }

// Sizes rounded up to tiles and strides still count in int.
constexpr int kMaxSize = 1 << 30;
bool dims_fit(int N, int d, int V) { return N <= kMaxSize && d <= kMaxSize && V <= kMaxSize; }

unsigned blocks_for(size_t work, size_t per_block, int sms)
{
    const size_t b = (work + per_block - 1) / per_block, most = (size_t)sms * 16;
    return (unsigned)(b < 1 ? 1 : b < most ? b : most);
}

struct Grads {
    float scale;
    uint16_t* dx;
    void* dW;  // null: losses only
    int dw_type, accumulate;
};

// One chunk's gradients, after its losses: dz, dx, and its share of dW.
cudaError_t chunk_grads(const XentWs& w, const uint16_t* W, int r0, int c, int rows, int d, int V, const Grads& g,
                        int sms, int32_t* status, cudaStream_t s)
{
    const int tiles = (V + kXentTile - 1) / kXentTile;
    const size_t ldcode = row_stride(V);
    count_launches(1);
    k_xent_dz<<<blocks_for((size_t)rows * ((ldcode + 255) / 256), 8, sms), 256, 0, s>>>(
        w, (unsigned)ldcode, tiles, w.target + r0, w.rows_dev + c, rows, status);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;

    GemmArgs g2{};
    g2.rowsA = rows;
    g2.rowsA_dev = w.rows_dev + c;
    g2.rowsB = d;
    g2.K = V;
    g2.lda = (int)ldcode;
    g2.b_mn = 1;
    g2.ldo = d;
    g2.status = status;
    // whole or in parts by the rows there may be; how many parts by those that are scored
    if (!in_parts(rows, d, V)) {
        g2.out = g.dx;
        g2.row_map = w.perm + r0;
        g2.scale = w.gscale;
        e = launch_gemm(GEMM_SCALED, w.codes, W, g2, sms, s);
    } else {
        g2.split = w.split + c;
        g2.out_f32 = w.parts;
        e = launch_gemm(GEMM_SPLITK, w.codes, W, g2, sms, s);
        if (e != cudaSuccess) return e;
        count_launches(1);
        k_xent_dx<<<blocks_for((size_t)rows * d / 4, 256, sms), 256, 0, s>>>(
            w.parts, w.split + c, w.rows_dev + c, d, w.gscale, w.perm + r0, g.dx, status);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) return e;

    GemmArgs g3{};
    g3.rowsA = V;
    g3.rowsB = d;
    g3.K = rows;
    g3.K_dev = w.k_dev + c;
    g3.lda = (int)ldcode;
    g3.a_mn = 1;
    g3.b_mn = 1;
    g3.ldo = d;
    g3.scale = w.gscale;
    g3.status = status;
    if (w.dw_acc || g.dw_type == TWELL_F32) {
        g3.out_f32 = w.dw_acc ? w.dw_acc : static_cast<float*>(g.dW);
        g3.accumulate = r0 > 0 || (!w.dw_acc && g.accumulate);
    } else {
        g3.out = static_cast<uint16_t*>(g.dW);
    }
    g3.ldb = (int)row_stride(d);
    return launch_gemm(GEMM_SCALED, w.codes, w.xs + (size_t)r0 * row_stride(d), g3, sms, s);
}

// Both entry points: losses, and with g.dW the gradients.
cudaError_t run_xent(const uint16_t* x, const uint16_t* W, const int64_t* target, int N, int d, int V,
                     int64_t ignore_index, int mean, int chunk, float* nll, float* lse, float* loss, const Grads& g,
                     void* ws, int32_t* status, cudaStream_t s)
{
    const int sms = sms_current();
    if (sms <= 0) return cudaErrorInvalidDevice;
    const bool grad = g.dW != nullptr;
    XentWs w{};
    carve(ws, N, chunk, d, V, grad, grad && g.dw_type == TWELL_BF16 && chunk < N, &w);
    const int tiles = (V + kXentTile - 1) / kXentTile;
    const int per_chunk = chunk > 0 ? chunk : 1, ldx = (int)row_stride(d);
    cudaError_t e = cudaSuccess;
    if (N == 0) {
        e = cudaMemsetAsync(loss, 0, sizeof(float), s);
        if (e == cudaSuccess && grad && !g.accumulate)
            e = cudaMemsetAsync(g.dW, 0, (size_t)V * d * (g.dw_type == TWELL_F32 ? 4 : 2), s);
        return e;
    }
    if (N <= kFewRows) {
        count_launches(1);
        k_xent_prep_gather<<<(unsigned)((N + 31) / 32), kPrepThreads, 0, s>>>(
            target, x, N, d, V, ignore_index, per_chunk, mean, g.scale, w, ldx, nll, lse, g.dx, status);
    } else {
        count_launches(2);
        k_xent_prep<<<1, kPrepThreads, 0, s>>>(target, N, d, V, ignore_index, per_chunk, mean, g.scale, w, status);
        k_xent_gather<<<blocks_for((size_t)N, 8, sms), 256, 0, s>>>(x, N, d, w, ldx, nll, lse, g.dx, status);
    }
    e = cudaGetLastError();
    for (int r0 = 0, c = 0; r0 < N && e == cudaSuccess; r0 += chunk, ++c) {
        const int rows = N - r0 < chunk ? N - r0 : chunk;
        GemmArgs g1{};
        g1.rowsA = rows;
        g1.rowsA_dev = w.rows_dev + c;
        g1.rowsB = V;
        g1.K = d;
        g1.NB = tiles;
        g1.codes = w.codes;
        g1.ldcode = row_stride(V);
        g1.xstat = w.stat;
        g1.target = w.target + r0;
        g1.ztarget = w.ztarget;
        g1.status = status;
        g1.lda = ldx;
        e = launch_gemm(GEMM_XENT, w.xs + (size_t)r0 * row_stride(d), W, g1, sms, s);
        if (e != cudaSuccess) return e;
        count_launches(1);
        k_xent_lse<<<(unsigned)((rows + 7) / 8), 256, 0, s>>>(w, tiles, w.rows_dev + c, w.target + r0, w.perm + r0, nll, lse,
                                                              N - r0 <= chunk ? 1 : 0, N, mean, loss, status);
        e = cudaGetLastError();
        if (e == cudaSuccess && grad) e = chunk_grads(w, W, r0, c, rows, d, V, g, sms, status, s);
        if (rows < chunk) break;  // the last chunk; r0 + chunk may pass the range of int
    }
    if (e == cudaSuccess && w.dw_acc) {
        const size_t n4 = (size_t)V * d / 4;
        count_launches(1);
        k_xent_round<<<blocks_for(n4, 256, sms), 256, 0, s>>>(w.dw_acc, n4, static_cast<uint16_t*>(g.dW), status);
        e = cudaGetLastError();
    }
    return e;
}

int chunk_of(int N, int chunk_rows) { return chunk_rows == 0 || chunk_rows > N ? N : chunk_rows; }

bool type_ok(int t) { return t == TWELL_BF16 || t == TWELL_F32; }

}  // namespace
}  // namespace twell

using namespace twell;

extern "C" size_t twell_xent_fwd_workspace_bytes(int N, int d, int V)
{
    if (!dims_ok(N, d, V) || !dims_fit(N, d, V)) return 0;
    return carve(nullptr, N, N, d, V, false, false, nullptr);
}

extern "C" size_t twell_xent_bwd_workspace_bytes(int N, int d, int V, int chunk_rows, int dw_type)
{
    if (!dims_ok(N, d, V) || !dims_fit(N, d, V) || chunk_rows < 0 || !type_ok(dw_type)) return 0;
    const int chunk = chunk_of(N, chunk_rows);
    return carve(nullptr, N, chunk, d, V, true, dw_type == TWELL_BF16 && chunk < N, nullptr);
}

extern "C" twell_status twell_xent_fwd(const uint16_t* x, const uint16_t* W, const int64_t* target, int N, int d,
                                       int V, int64_t ignore_index, int mean, float* nll, float* lse, float* loss,
                                       void* ws, size_t ws_bytes, int32_t* status, void* stream)
{
    if (!dims_ok(N, d, V) || !W || !loss || !status || (N > 0 && (!x || !target || !nll || !lse)))
        return TWELL_ERR_INVALID_ARG;
    if (!dims_fit(N, d, V)) return TWELL_ERR_UNSUPPORTED;
    if (!aligned(x, 16) || !aligned(W, 16) || !aligned(target, 8)) return TWELL_ERR_INVALID_ARG;
    if (!ws || ws_bytes < twell_xent_fwd_workspace_bytes(N, d, V)) return TWELL_ERR_WORKSPACE;
    if (!aligned(ws, 256)) return TWELL_ERR_INVALID_ARG;
    const cudaError_t e = run_xent(x, W, target, N, d, V, ignore_index, mean, N, nll, lse, loss, Grads{}, ws, status,
                                   static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? TWELL_OK : TWELL_ERR_CUDA;
}

extern "C" twell_status twell_xent_fwd_bwd(const uint16_t* x, const uint16_t* W, const int64_t* target, int N, int d,
                                           int V, int64_t ignore_index, int mean, float grad_scale, int chunk_rows,
                                           float* nll, float* lse, float* loss, uint16_t* dx, void* dW, int dw_type,
                                           int accumulate, void* ws, size_t ws_bytes, int32_t* status, void* stream)
{
    if (!dims_ok(N, d, V) || chunk_rows < 0 || !type_ok(dw_type) || (accumulate && dw_type != TWELL_F32))
        return TWELL_ERR_INVALID_ARG;
    if (!W || !loss || !status || !dW || (N > 0 && (!x || !target || !nll || !lse || !dx)))
        return TWELL_ERR_INVALID_ARG;
    if (!dims_fit(N, d, V)) return TWELL_ERR_UNSUPPORTED;
    if (!aligned(x, 16) || !aligned(W, 16) || !aligned(target, 8) || !aligned(dx, 16) || !aligned(dW, 16))
        return TWELL_ERR_INVALID_ARG;
    if (!ws || ws_bytes < twell_xent_bwd_workspace_bytes(N, d, V, chunk_rows, dw_type)) return TWELL_ERR_WORKSPACE;
    if (!aligned(ws, 256)) return TWELL_ERR_INVALID_ARG;
    const Grads g{grad_scale, dx, dW, dw_type, accumulate};
    const cudaError_t e = run_xent(x, W, target, N, d, V, ignore_index, mean, chunk_of(N, chunk_rows), nll, lse, loss,
                                   g, ws, status, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? TWELL_OK : TWELL_ERR_CUDA;
}
