// twell_layernorm.cu — layer norm's forward and backward pass around the
// feed-forward layer, with the residual sum and the weight's gradient.
//
//   forward   s = x + res, hat = (s - mean) rstd, y = hat w + b
//   backward  v = w dy, dx = rstd (v - mean(v) - hat mean(v hat)) + dres,
//             dw = sum_r dy hat, db = sum_r dy
//
// Bound by memory: every element read once and written once (forward: x, res in,
// sum, y out; backward: x, dy, dres in, dx out). 16384 x 4096 bf16 with residual, 537
// MB either way, 79 us at the measured copy rate: forward 82 us, backward 84.5 us (5 us
// of it the column sums).
//
//   k_ln_fwd       rows up to 8192 elements, held by their threads
//   k_ln_bwd       the same: dx, and partial dw, db of each block
//   k_ln_reduce    the blocks' partial sums added in order (few rows: blocks of
//                  k_ln_bwd sum whole columns instead)
//   k_ln_fwd_long, k_ln_bwd_long, k_ln_cols_long   longer rows, read several times
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
    bool w_f32;
};

struct BwdArgs {
    const void *dy, *x, *w, *dres;
    void* dx;
    int64_t lddy, ldx, lddres, lddx, N;
    int d;
    const float *mean, *rstd;
    float* part;  // [parts, 2, d] partial sums of dw and db; null: not wanted, or dw and db direct
    int parts;    // blocks that work on rows
    float *dw, *db;  // few rows: blocks after those sum whole columns
    bool w_f32;
};

constexpr int kRowThreads = 256;
constexpr int kMaxLongParts = 304;  // two blocks on each of 152 SMs
// Up to so many rows the column sums are taken by blocks of their own in the same
// launch. Backward with those / with partial sums and a second launch, us, bf16:
// 256 x 1024 3.2 / 6.3, 768 x 1024 5.4 / 7.6, 768 x 4096 10.7 / 11.9, 1024 x 1024 7.6 / 7.3,
// 1024 x 4096 13.1 / 14.3, 1536 x 4096 20.6 / 17.7.
constexpr int64_t kFewRows = 896;

// Element i of a weight vector of either type; `none` where there is no vector.
__device__ __forceinline__ float weight(const void* p, int i, bool f32, float none)
{
    if (!p) return none;
    return f32 ? static_cast<const float*>(p)[i] : bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
}

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
template <class TX, class TY>
__global__ void __launch_bounds__(kRowThreads) k_ln_fwd_long(const FwdArgs a)
{
    __shared__ float2 buf[kRowThreads / 32];
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
            TY::store(y + i, fmaf(hat, weight(a.w, i, a.w_f32, 1.f), weight(a.b, i, a.w_f32, 0.f)));
        }
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
    }
}

// dx, one block per row, the row read twice.
template <class TX, class TY>
__global__ void __launch_bounds__(kRowThreads) k_ln_bwd_long(const BwdArgs a)
{
    __shared__ float2 buf[kRowThreads / 32];
    for (int64_t r = blockIdx.x; r < a.N; r += gridDim.x) {
        const typename TX::type* x = static_cast<const typename TX::type*>(a.x) + r * a.ldx;
        const typename TX::type* dres = a.dres ? static_cast<const typename TX::type*>(a.dres) + r * a.lddres : nullptr;
        const typename TY::type* dy = static_cast<const typename TY::type*>(a.dy) + r * a.lddy;
        typename TX::type* dx = static_cast<typename TX::type*>(a.dx) + r * a.lddx;
        const float mean = a.mean[r], rstd = a.rstd[r];
        float s1 = 0.f, s2 = 0.f;
        for (int i = threadIdx.x; i < a.d; i += kRowThreads) {
            const float hat = (TX::load(x + i) - mean) * rstd;
            const float v = TY::load(dy + i) * weight(a.w, i, a.w_f32, 1.f);
            s1 += v;
            s2 += v * hat;
        }
        const float2 s = block_sum2(s1, s2, buf);
        const float c1 = s.x / (float)a.d, c2 = s.y / (float)a.d;
        for (int i = threadIdx.x; i < a.d; i += kRowThreads) {
            const float hat = (TX::load(x + i) - mean) * rstd;
            const float v = TY::load(dy + i) * weight(a.w, i, a.w_f32, 1.f);
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

// dw and db: the parts of 32 columns added by 32 warps (every 32nd part each,
// ascending), then the 32 sums in order.
__global__ void __launch_bounds__(1024)
    k_ln_reduce(const float* __restrict__ part, int parts, int d, float* __restrict__ dw, float* __restrict__ db)
{
    const int i = blockIdx.x * 32 + threadIdx.x, ty = threadIdx.y;  // column of [dw | db]
    float s = 0.f;
    if (i < 2 * d)
        for (int p = ty; p < parts; p += 32) s += part[(size_t)p * 2 * d + i];
    __shared__ float buf[32][32];
    buf[ty][threadIdx.x] = s;
    __syncthreads();
    if (ty == 0 && i < 2 * d) {
        for (int j = 1; j < 32; ++j) s += buf[j][threadIdx.x];
        if (i < d)
            dw[i] = s;
        else
            db[i - d] = s;
    }
}

// ---------------------------------------------- rows held by their threads --
//
// A row is held by G threads (a warp to 512 threads, 8 or 16 elements each), so
// that it is read from memory once. Blocks stay and walk over the rows: w, b and
// the column sums live in registers. Each thread copies its pieces of the next
// rows (16 bytes where the rows' addresses allow it, else two elements, else one)
// asynchronously into shared memory, where only it reads them: bytes in flight
// without registers and without barriers. Odd rows of bf16, whose single elements
// such copies do not move, are read when their turn comes. The mean is
// summed first and the variance from the centred values, which holds for rows
// whose mean is far larger than their deviation.

constexpr int kMaxGroup = 512;  // threads of a row at most: rows up to 512 * 16 = 8192 elements

// VEC consecutive elements of type T as they are in memory.
template <class T, int VEC>
struct Piece;
template <int VEC>
struct Piece<bf16_t, VEC> {
    static_assert(VEC == 8, "");
    uint4 v;
    __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ float get(int i) const
    {
        const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
        return (i & 1) ? bf16_hi(w) : bf16_lo(w);
    }
    __device__ __forceinline__ void set(const float* f)
    {
        v = make_uint4(cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]), cvt_bf16x2(f[4], f[5]), cvt_bf16x2(f[6], f[7]));
    }
    __device__ __forceinline__ void store(uint16_t* p) const { *reinterpret_cast<uint4*>(p) = v; }
};
template <>
struct Piece<bf16_t, 1> {
    // a whole register: two halves packed into one would wait for both loads at once
    uint32_t v;
    __device__ __forceinline__ void load(const uint16_t* p) { v = *p; }
    __device__ __forceinline__ void zero() { v = 0; }
    __device__ __forceinline__ float get(int) const { return bf16_lo(v); }
    __device__ __forceinline__ void set(const float* f) { v = f32_to_bf16_bits(f[0]); }
    __device__ __forceinline__ void store(uint16_t* p) const { *p = (uint16_t)v; }
};
template <>
struct Piece<bf16_t, 4> {
    uint2 v;
    __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const uint2*>(p); }
    __device__ __forceinline__ void zero() { v = make_uint2(0, 0); }
    __device__ __forceinline__ float get(int i) const
    {
        const uint32_t w = i < 2 ? v.x : v.y;
        return (i & 1) ? bf16_hi(w) : bf16_lo(w);
    }
    __device__ __forceinline__ void set(const float* f)
    {
        v = make_uint2(cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]));
    }
    __device__ __forceinline__ void store(uint16_t* p) const { *reinterpret_cast<uint2*>(p) = v; }
};
template <>
struct Piece<bf16_t, 2> {
    uint32_t v;
    __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const uint32_t*>(p); }
    __device__ __forceinline__ void zero() { v = 0; }
    __device__ __forceinline__ float get(int i) const { return i ? bf16_hi(v) : bf16_lo(v); }
    __device__ __forceinline__ void set(const float* f) { v = cvt_bf16x2(f[0], f[1]); }
    __device__ __forceinline__ void store(uint16_t* p) const { *reinterpret_cast<uint32_t*>(p) = v; }
};
template <>
struct Piece<f32_t, 2> {
    float2 v;
    __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float2*>(p); }
    __device__ __forceinline__ void zero() { v = make_float2(0.f, 0.f); }
    __device__ __forceinline__ float get(int i) const { return i ? v.y : v.x; }
    __device__ __forceinline__ void set(const float* f) { v = make_float2(f[0], f[1]); }
    __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<float2*>(p) = v; }
};
template <>
struct Piece<f32_t, 4> {
    float4 v;
    __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ void zero() { v = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ float get(int i) const { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
    __device__ __forceinline__ void set(const float* f) { v = make_float4(f[0], f[1], f[2], f[3]); }
    __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<float4*>(p) = v; }
};
template <int VEC>
struct Piece<f32_t, VEC> {  // (weights only)
    static_assert(VEC == 8, "");
    float4 a, b;
    __device__ __forceinline__ void load(const float* p)
    {
        a = reinterpret_cast<const float4*>(p)[0];
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ float get(int i) const
    {
        return i == 0 ? a.x : i == 1 ? a.y : i == 2 ? a.z : i == 3 ? a.w : i == 4 ? b.x : i == 5 ? b.y : i == 6 ? b.z : b.w;
    }
};
template <>
struct Piece<f32_t, 1> {
    float v;
    __device__ __forceinline__ void load(const float* p) { v = *p; }
    __device__ __forceinline__ void zero() { v = 0.f; }
    __device__ __forceinline__ float get(int) const { return v; }
    __device__ __forceinline__ void set(const float* f) { v = f[0]; }
    __device__ __forceinline__ void store(float* p) const { *p = v; }
};

// Sums over the G threads of a row, the same bits in all of them: a butterfly in
// each warp, then one over the warps' sums. `buf` alternates between two halves
// from one sum to the next, so one barrier each is enough.
struct RowSum {
    float2* buf;  // [2][16]
    int mine, from, warps, bar;
    __device__ RowSum(float2* b, int G) : buf(b)
    {
        const int group = threadIdx.x / G;
        warps = G >> 5;
        mine = threadIdx.x >> 5;
        from = group * warps + (threadIdx.x & (warps - 1));
        bar = 1 + group;
    }
    __device__ __forceinline__ float2 sum2(float x, float y)
    {
        x = warp_sum(x);
        y = warp_sum(y);
        if (warps == 1) return make_float2(x, y);
        if ((threadIdx.x & 31) == 0) buf[mine] = make_float2(x, y);
        named_bar_sync(bar, warps * 32);
        float2 s = buf[from];
        turn();
        for (int off = warps >> 1; off >= 1; off >>= 1) {
            s.x += __shfl_xor_sync(0xffffffffu, s.x, off);
            s.y += __shfl_xor_sync(0xffffffffu, s.y, off);
        }
        return s;
    }
    __device__ __forceinline__ float sum(float x)
    {
        x = warp_sum(x);
        if (warps == 1) return x;
        if ((threadIdx.x & 31) == 0) buf[mine].x = x;
        named_bar_sync(bar, warps * 32);
        float s = buf[from].x;
        turn();
        for (int off = warps >> 1; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        return s;
    }
    __device__ __forceinline__ void turn()
    {
        mine ^= 16;
        from ^= 16;
    }
};

template <class T>
__device__ __forceinline__ const typename T::type* row_of(const void* p, int64_t r, int64_t ld)
{
    return static_cast<const typename T::type*>(p) + r * ld;
}
template <class T>
__device__ __forceinline__ typename T::type* row_of(void* p, int64_t r, int64_t ld)
{
    return static_cast<typename T::type*>(p) + r * ld;
}

// VEC weights as floats; `f32`: their type.
template <int VEC>
__device__ __forceinline__ void load_weights(const void* p, int i, bool f32, float* out)
{
    if (f32) {
        Piece<f32_t, VEC> w;
        w.load(static_cast<const float*>(p) + i);
#pragma unroll
        for (int e = 0; e < VEC; ++e) out[e] = w.get(e);
    } else {
        Piece<bf16_t, VEC> w;
        w.load(static_cast<const uint16_t*>(p) + i);
#pragma unroll
        for (int e = 0; e < VEC; ++e) out[e] = w.get(e);
    }
}

template <int BYTES>
__device__ __forceinline__ void copy_async(void* smem, const void* global)
{
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(smem)), "l"(global) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(smem)), "l"(global), "n"(BYTES)
                     : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

// Elements of an aligned piece: 16 bytes of the wider type, so that neighbouring
// threads' pieces touch (two halves of 32 bytes a thread took each sector twice:
// 4096 x 2048 fp32 with residual 29.6 us instead of 20.7).
template <class TX, class TY>
constexpr int vec_of()
{
    return sizeof(typename TX::type) + sizeof(typename TY::type) == 4 ? 8 : 4;
}

// Whether rows come through the ring: its copies move at least 4 bytes.
template <class TX, class TY, int VEC>
constexpr bool ringed()
{
    return VEC > 1 || sizeof(typename TX::type) + sizeof(typename TY::type) == 8;
}

template <class T, int VEC>
constexpr int piece_bytes()
{
    return (int)sizeof(typename T::type) * VEC;
}

// Rows on their way: STAGES rows of every stream (x; res or dy; dres), BYTES of a
// row to a thread. A piece is named by its offset in those bytes; the pieces of all
// threads at one offset lie side by side. `stage`: the bytes before the oldest row.
template <int STAGES, int BYTES>
struct Ring {
    char* base;
    int threads, stage = 0;
    __device__ Ring(void* smem) : base(static_cast<char*>(smem)), threads(blockDim.x) {}
    static size_t bytes(int threads) { return (size_t)STAGES * BYTES * threads; }

    __device__ __forceinline__ void turn()
    {
        stage += BYTES * threads;
        if (stage == STAGES * BYTES * threads) stage = 0;
    }
    template <class T, int VEC>
    __device__ __forceinline__ char* at(int off)
    {
        return base + (off * threads + (int)threadIdx.x * piece_bytes<T, VEC>()) + stage;
    }
    template <class T, int VEC>
    __device__ __forceinline__ void get(int off, Piece<T, VEC>& p)
    {
        p.load(reinterpret_cast<const typename T::type*>(at<T, VEC>(off)));
    }
    template <class T, int VEC>
    __device__ __forceinline__ void ask(int off, const typename T::type* from)
    {
        copy_async<piece_bytes<T, VEC>()>(at<T, VEC>(off), from);
    }
};

// Rows of a stream on their way: the next one while a row is worked on is enough,
// and more of them slow the memory down (16384 x 4096 bf16 with residual, forward: two
// rows 82 us, three 86, four 90, six 96).
constexpr int kStages = 2;

// Blocks of 512 threads that share an SM: two (64 registers a thread) with 8
// elements a thread, one with 16.
constexpr int blocks_per_sm(int per) { return per == 8 ? 2 : 1; }

template <class TX, int PER, bool RES>
constexpr int fwd_bytes()
{
    return PER * (int)sizeof(typename TX::type) * (RES ? 2 : 1);
}

template <class TX, class TY, int VEC, int PER, bool RES>
__global__ void __launch_bounds__(kMaxGroup, blocks_per_sm(PER)) k_ln_fwd(const FwdArgs a, int G)
{
    constexpr int NV = PER / VEC, BYTES = fwd_bytes<TX, PER, RES>(), STAGES = kStages;
    constexpr int SX = piece_bytes<TX, VEC>();
    constexpr bool RING = ringed<TX, TY, VEC>();
    extern __shared__ uint4 dyn[];
    __shared__ float2 buf[32];
    RowSum rs(buf, G);
    Ring<STAGES, BYTES> ring(dyn);
    const int t = threadIdx.x % G;
    const float inv_d = 1.f / (float)a.d;
    float w[PER], b[PER];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int i = (v * G + t) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            w[v * VEC + e] = 1.f;
            b[v * VEC + e] = 0.f;
        }
        if (i < a.d && a.w) load_weights<VEC>(a.w, i, a.w_f32, w + v * VEC);
        if (i < a.d && a.b) load_weights<VEC>(a.b, i, a.w_f32, b + v * VEC);
    }
    const int64_t step = (int64_t)gridDim.x * (blockDim.x / G);
    int64_t r = (int64_t)blockIdx.x * (blockDim.x / G) + threadIdx.x / G;
    // this thread's first element in the row asked for next
    int64_t asked = r;
    const typename TX::type* ax = row_of<TX>(a.x, r, a.ldx) + t * VEC;
    const typename TX::type* aq = RES ? row_of<TX>(a.res, r, a.ldres) + t * VEC : nullptr;
    auto request = [&] {
        if constexpr (RING) {
            if (asked < a.N) {
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    if ((v * G + t) * VEC < a.d) {
                        ring.template ask<TX, VEC>(v * SX, ax + v * G * VEC);
                        if (RES) ring.template ask<TX, VEC>((NV + v) * SX, aq + v * G * VEC);
                    }
                }
            }
            copies_commit();
            asked += step;
            ax += step * a.ldx;
            if (RES) aq += step * a.ldres;
        }
    };
#pragma unroll
    for (int i = 0; i < STAGES; ++i) {
        request();
        ring.turn();
    }
    for (; r < a.N; r += step) {
        float f[PER];
        float s = 0.f;
        if (RING) copies_wait<STAGES - 1>();
        // all of the row is asked for before any of it is used, at an address that is
        // always there (a load under a branch waits for the one before it)
        Piece<TX, VEC> xs[NV], qs[RES ? NV : 1];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int i = (v * G + t) * VEC;
            const bool in = i < a.d;
            if constexpr (RING) {
                ring.get(v * SX, xs[v]);
                if (RES) ring.get((NV + v) * SX, qs[v]);
            } else {
                xs[v].load(row_of<TX>(a.x, r, a.ldx) + (in ? i : 0));
                if (RES) qs[v].load(row_of<TX>(a.res, r, a.ldres) + (in ? i : 0));
            }
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int i = (v * G + t) * VEC;
            Piece<TX, VEC> x = xs[v];
            if (i >= a.d) x.zero();
#pragma unroll
            for (int e = 0; e < VEC; ++e) f[v * VEC + e] = x.get(e);
            if (RES) {
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (i < a.d) f[v * VEC + e] += qs[v].get(e);
                x.set(f + v * VEC);
                if (i < a.d) x.store(row_of<TX>(a.sum, r, a.ldsum) + i);
#pragma unroll
                for (int e = 0; e < VEC; ++e) f[v * VEC + e] = x.get(e);
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) s += f[v * VEC + e];
        }
        request();
        ring.turn();
        const float mean = rs.sum(s) * inv_d;
        float c2 = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const bool in = (v * G + t) * VEC < a.d;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                f[v * VEC + e] -= mean;
                if (in) c2 = fmaf(f[v * VEC + e], f[v * VEC + e], c2);
            }
        }
        const float rstd = rsqrtf(rs.sum(c2) * inv_d + a.eps);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int i = (v * G + t) * VEC;
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                f[v * VEC + e] = fmaf(f[v * VEC + e] * rstd, w[v * VEC + e], b[v * VEC + e]);
            Piece<TY, VEC> o;
            o.set(f + v * VEC);
            if (i < a.d) o.store(row_of<TY>(a.y, r, a.ldy) + i);
        }
        if (t == 0) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
    }
    if (RING) copies_wait<0>();
}

template <class TX, class TY, int PER, bool RES>
constexpr int bwd_bytes()
{
    return PER * ((int)sizeof(typename TX::type) * (RES ? 2 : 1) + (int)sizeof(typename TY::type));
}

// VEC column sums (d is a multiple of VEC; element by element these stores took 6 us
// of a backward over 300 x 4096).
template <int VEC>
__device__ __forceinline__ void store_sums(float* p, const float* s)
{
    if constexpr (VEC == 1) {
        *p = s[0];
    } else if constexpr (VEC == 2) {
        *reinterpret_cast<float2*>(p) = make_float2(s[0], s[1]);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; e += 4)
            *reinterpret_cast<float4*>(p + e) = make_float4(s[e], s[e + 1], s[e + 2], s[e + 3]);
    }
}

// dw and db of 16 columns over all rows, one block: sixteenths (or 32nds) of the
// rows summed side by side, then joined in order.
constexpr int kColBlock = 16;
template <class TX, class TY>
__device__ __forceinline__ void column_sums(const BwdArgs& a, int block)
{
    __shared__ float2 sums[kMaxGroup / kColBlock][kColBlock];
    const int c = threadIdx.x % kColBlock, lane = threadIdx.x / kColBlock, lanes = blockDim.x / kColBlock;
    const int col = block * kColBlock + c;
    float dw = 0.f, db = 0.f;
    if (col < a.d) {
#pragma unroll 8
        for (int64_t r = lane; r < a.N; r += lanes) {
            const float x = TX::load(row_of<TX>(a.x, r, a.ldx) + col);
            const float g = TY::load(row_of<TY>(a.dy, r, a.lddy) + col);
            dw = fmaf(g, (x - a.mean[r]) * a.rstd[r], dw);
            db += g;
        }
    }
    sums[lane][c] = make_float2(dw, db);
    __syncthreads();
    if (lane == 0 && col < a.d) {
        for (int i = 1; i < lanes; ++i) {
            dw += sums[i][c].x;
            db += sums[i][c].y;
        }
        a.dw[col] = dw;
        a.db[col] = db;
    }
}

// The normalised values and w dy are formed twice from what was read (before
// and after the row's sums): two products cost less than the registers.
template <class TX, class TY, int VEC, int PER, bool RES>
__global__ void __launch_bounds__(kMaxGroup, blocks_per_sm(PER)) k_ln_bwd(const BwdArgs a, int G)
{
    constexpr int NV = PER / VEC, BYTES = bwd_bytes<TX, TY, PER, RES>(), STAGES = kStages;
    constexpr int SX = piece_bytes<TX, VEC>(), SY = piece_bytes<TY, VEC>();
    constexpr bool RING = ringed<TX, TY, VEC>();
    constexpr int G0 = NV * SX, Q0 = G0 + NV * SY;  // offsets of dy and dres
    if ((int)blockIdx.x >= a.parts) {
        column_sums<TX, TY>(a, blockIdx.x - a.parts);
        return;
    }
    extern __shared__ uint4 dyn[];
    __shared__ float2 buf[32];
    RowSum rs(buf, G);
    Ring<STAGES, BYTES> ring(dyn);
    const int t = threadIdx.x % G, groups = blockDim.x / G;
    const float inv_d = 1.f / (float)a.d;
    float w[PER], dw[PER], db[PER];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int i = (v * G + t) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            w[v * VEC + e] = 1.f;
            dw[v * VEC + e] = db[v * VEC + e] = 0.f;
        }
        if (i < a.d && a.w) load_weights<VEC>(a.w, i, a.w_f32, w + v * VEC);
    }
    const int64_t step = (int64_t)a.parts * groups;
    int64_t r = (int64_t)blockIdx.x * groups + threadIdx.x / G;
    int64_t asked = r;
    const typename TX::type* ax = row_of<TX>(a.x, r, a.ldx) + t * VEC;
    const typename TY::type* ag = row_of<TY>(a.dy, r, a.lddy) + t * VEC;
    const typename TX::type* aq = RES ? row_of<TX>(a.dres, r, a.lddres) + t * VEC : nullptr;
    auto request = [&] {
        if constexpr (RING) {
            if (asked < a.N) {
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    if ((v * G + t) * VEC < a.d) {
                        ring.template ask<TX, VEC>(v * SX, ax + v * G * VEC);
                        ring.template ask<TY, VEC>(G0 + v * SY, ag + v * G * VEC);
                        if (RES) ring.template ask<TX, VEC>(Q0 + v * SX, aq + v * G * VEC);
                    }
                }
            }
            copies_commit();
            asked += step;
            ax += step * a.ldx;
            ag += step * a.lddy;
            if (RES) aq += step * a.lddres;
        }
    };
#pragma unroll
    for (int i = 0; i < STAGES; ++i) {
        request();
        ring.turn();
    }
    float next_mean = r < a.N ? a.mean[r] : 0.f, next_rstd = r < a.N ? a.rstd[r] : 0.f;
    for (; r < a.N; r += step) {
        const float mean = next_mean, rstd = next_rstd;
        if (r + step < a.N) {
            next_mean = a.mean[r + step];
            next_rstd = a.rstd[r + step];
        }
        Piece<TX, VEC> x[NV], add[RES && !RING ? NV : 1];
        Piece<TY, VEC> g[NV];
        if (RING) copies_wait<STAGES - 1>();
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int i = (v * G + t) * VEC;
            if constexpr (RING) {
                ring.get(v * SX, x[v]);
                ring.get(G0 + v * SY, g[v]);
            } else {
                const int at = i < a.d ? i : 0;
                x[v].load(row_of<TX>(a.x, r, a.ldx) + at);
                g[v].load(row_of<TY>(a.dy, r, a.lddy) + at);
                if constexpr (RES) add[v].load(row_of<TX>(a.dres, r, a.lddres) + at);
            }
        }
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if ((v * G + t) * VEC >= a.d) g[v].zero();  // beyond the row
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int k = v * VEC + e;
                const float dy = g[v].get(e);
                const float hat = (v * G + t) * VEC < a.d ? (x[v].get(e) - mean) * rstd : 0.f;
                dw[k] = fmaf(dy, hat, dw[k]);
                db[k] += dy;
                const float dv = dy * w[k];
                s1 += dv;
                s2 = fmaf(dv, hat, s2);
            }
        }
        const float2 c = rs.sum2(s1, s2);
        const float c1 = c.x * inv_d, c2 = c.y * inv_d;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int i = (v * G + t) * VEC;
            if (i >= a.d) continue;
            Piece<TX, VEC> q;
            if constexpr (RES) {
                if constexpr (RING)
                    ring.get(Q0 + v * SX, q);
                else
                    q = add[v];
            }
            float f[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float hat = (x[v].get(e) - mean) * rstd;
                f[e] = rstd * (g[v].get(e) * w[v * VEC + e] - c1 - hat * c2);
                if constexpr (RES) f[e] += q.get(e);
            }
            q.set(f);
            q.store(row_of<TX>(a.dx, r, a.lddx) + i);
        }
        request();
        ring.turn();
    }
    if (RING) copies_wait<0>();
    if (!a.part) return;
    float* part = a.part + (size_t)blockIdx.x * 2 * a.d;
    if (groups == 1) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int i = (v * G + t) * VEC;
            if (i < a.d) {
                store_sums<VEC>(part + i, dw + v * VEC);
                store_sums<VEC>(part + a.d + i, db + v * VEC);
            }
        }
        return;
    }
    // several rows at a time in the block: the groups' sums side by side (over the
    // ring), then added in order
    float* sums = reinterpret_cast<float*>(dyn);
    float* mine = sums + (int)threadIdx.x / G * 2 * a.d;
    __syncthreads();
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int i = (v * G + t) * VEC;
        if (i < a.d) {
            store_sums<VEC>(mine + i, dw + v * VEC);
            store_sums<VEC>(mine + a.d + i, db + v * VEC);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.d; i += blockDim.x) {
        float s = sums[i];
        for (int k = 1; k < groups; ++k) s += sums[k * 2 * a.d + i];
        part[i] = s;
    }
}

// Elements of a row per thread. What a warp does once a row (sums over lanes and
// warps, addresses) weighs more than the bytes with 8 elements a lane (16384 x 4096
// bf16 with residual: forward 117 us with 8, issue slots 74 % busy); rows that a
// warp holds with 8 take 8.
int per_thread(int d) { return d <= 256 ? 8 : 16; }

// Threads of a row: the fewest that hold it; 0 where kMaxGroup do not.
int group_of(int d)
{
    for (int G = 32; G <= kMaxGroup; G *= 2)
        if (G * per_thread(d) >= d) return G;
    return 0;
}

// Longest rows: twice as many column sums, and the threads past the last, still count in int.
constexpr int kMaxWidth = 1 << 29;

int rows_per_block(int G) { return G < 256 ? 256 / G : 1; }

// Blocks on 152 SMs at once: 128 registers a thread with 16 elements, 64 with 8.
int resident_blocks(int G, int d) { return 152 * (G > 256 ? 1 : per_thread(d) == 16 ? 2 : 4); }

// Blocks of the backward, each with its own partial sums (long rows: parts of
// eight rows at a time).
int parts_for(int64_t N, int d)
{
    const int G = group_of(d);
    const int64_t rows = G ? rows_per_block(G) : 8;
    const int64_t n = (N + rows - 1) / rows, most = G ? resident_blocks(G, d) : kMaxLongParts;
    return (int)(n < most ? n : most);
}

bool type_ok(int t) { return t == TWELL_BF16 || t == TWELL_F32; }

bool elem_aligned(const void* p, int type)
{
    return (reinterpret_cast<uintptr_t>(p) & (type == TWELL_F32 ? 3u : 1u)) == 0;
}

// Elements of a piece every row of p allows (by its address and stride), at most `most`: most, 2 or 1.
int pieces(const void* p, int64_t ld, int64_t N, int type, int most)
{
    const int64_t size = type == TWELL_F32 ? 4 : 2;
    for (int v = most; v > 1; v = v > 2 ? 2 : 1)
        if (reinterpret_cast<uintptr_t>(p) % (v * size) == 0 && (N <= 1 || ld % v == 0)) return v;
    return 1;
}

// The same for a vector of weights, whose pieces are read in loads of 16 bytes at most
// (16384 x 4096 bf16 with residual, fp32 weights on any 16-byte boundary: forward 85, backward
// 90 us a call; in single elements 251 and 412).
int weight_pieces(const void* p, int type, int most)
{
    const int size = type == TWELL_F32 ? 4 : 2;
    for (int v = most; v > 1; v = v > 2 ? 2 : 1)
        if (reinterpret_cast<uintptr_t>(p) % (v * size < 16 ? v * size : 16) == 0) return v;
    return 1;
}

// Launches a kernel that may want more than 48 KB of shared memory (its static part included).
template <class Args>
cudaError_t launch_rows(void (*kern)(Args, int), const Args& a, int G, unsigned blocks, unsigned threads, size_t smem,
                        cudaStream_t s)
{
    if (smem > 47 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    kern<<<blocks, threads, smem, s>>>(a, G);
    return cudaGetLastError();
}

template <class TX, class TY, int PER, bool RES>
cudaError_t launch_fwd(const FwdArgs& a, int G, int vec, unsigned blocks, unsigned threads, cudaStream_t s)
{
    constexpr int B = fwd_bytes<TX, PER, RES>();
    const size_t ring = Ring<kStages, B>::bytes(threads);
    if (vec == 1)
        return launch_rows(k_ln_fwd<TX, TY, 1, PER, RES>, a, G, blocks, threads, ringed<TX, TY, 1>() ? ring : 0, s);
    if (vec == 2) return launch_rows(k_ln_fwd<TX, TY, 2, PER, RES>, a, G, blocks, threads, ring, s);
    return launch_rows(k_ln_fwd<TX, TY, vec_of<TX, TY>(), PER, RES>, a, G, blocks, threads, ring, s);
}

template <class TX, class TY>
cudaError_t fwd(const FwdArgs& a, int vec, cudaStream_t s)
{
    const int G = group_of(a.d);
    count_launches(1);
    if (G) {
        const int64_t n = (a.N + rows_per_block(G) - 1) / rows_per_block(G);
        const int64_t most = resident_blocks(G, a.d);
        const unsigned blocks = (unsigned)(n < most ? n : most), threads = G < 256 ? 256 : G;
        if (per_thread(a.d) == 8)
            return a.res ? launch_fwd<TX, TY, 8, true>(a, G, vec, blocks, threads, s)
                         : launch_fwd<TX, TY, 8, false>(a, G, vec, blocks, threads, s);
        return a.res ? launch_fwd<TX, TY, 16, true>(a, G, vec, blocks, threads, s)
                     : launch_fwd<TX, TY, 16, false>(a, G, vec, blocks, threads, s);
    }
    k_ln_fwd_long<TX, TY><<<(unsigned)(a.N < 65536 ? a.N : 65536), kRowThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <class TX, class TY, int PER, bool RES>
cudaError_t launch_bwd(const BwdArgs& a, int G, int vec, unsigned threads, cudaStream_t s)
{
    constexpr int B = bwd_bytes<TX, TY, PER, RES>();
    const unsigned blocks = a.parts + (a.dw ? (a.d + kColBlock - 1) / kColBlock : 0);
    // the groups' column sums, when a block holds several rows at a time (over the ring where there is one)
    const size_t sums = a.part && G < 256 ? (size_t)rows_per_block(G) * 2 * a.d * sizeof(float) : 0;
    const size_t ring = Ring<kStages, B>::bytes(threads), both = ring > sums ? ring : sums;
    if (vec == 1)
        return launch_rows(k_ln_bwd<TX, TY, 1, PER, RES>, a, G, blocks, threads, ringed<TX, TY, 1>() ? both : sums, s);
    if (vec == 2) return launch_rows(k_ln_bwd<TX, TY, 2, PER, RES>, a, G, blocks, threads, both, s);
    return launch_rows(k_ln_bwd<TX, TY, vec_of<TX, TY>(), PER, RES>, a, G, blocks, threads, both, s);
}

template <class TX, class TY>
cudaError_t bwd(const BwdArgs& a, int vec, float* dw, float* db, cudaStream_t s)
{
    const int G = group_of(a.d);
    cudaError_t e;
    count_launches(1);
    if (G) {
        const unsigned threads = G < 256 ? 256 : G;
        if (per_thread(a.d) == 8)
            e = a.dres ? launch_bwd<TX, TY, 8, true>(a, G, vec, threads, s)
                       : launch_bwd<TX, TY, 8, false>(a, G, vec, threads, s);
        else
            e = a.dres ? launch_bwd<TX, TY, 16, true>(a, G, vec, threads, s)
                       : launch_bwd<TX, TY, 16, false>(a, G, vec, threads, s);
    } else {
        k_ln_bwd_long<TX, TY><<<(unsigned)(a.N < 65536 ? a.N : 65536), kRowThreads, 0, s>>>(a);
        if (a.part) {
            count_launches(1);
            k_ln_cols_long<TX, TY><<<dim3((unsigned)((a.d + 31) / 32), (unsigned)a.parts), dim3(32, 8), 0, s>>>(a);
        }
        e = cudaGetLastError();
    }
    if (e != cudaSuccess || !a.part) return e;
    count_launches(1);
    k_ln_reduce<<<(unsigned)((2 * (int64_t)a.d + 31) / 32), dim3(32, 32), 0, s>>>(a.part, a.parts, a.d, dw, db);
    return cudaGetLastError();
}

// f with the tags of the two types.
template <class F>
cudaError_t by_types(int x, int y, F f)
{
    if (x == TWELL_F32) return y == TWELL_F32 ? f(f32_t{}, f32_t{}) : f(f32_t{}, bf16_t{});
    return y == TWELL_F32 ? f(bf16_t{}, f32_t{}) : f(bf16_t{}, bf16_t{});
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
    if (d > kMaxWidth) return TWELL_ERR_UNSUPPORTED;
    if (N == 0) return TWELL_OK;
    if (!x || !y || (res != nullptr) != (sum != nullptr) || ldx < d || ldy < d || (res && (ldres < d || ldsum < d)))
        return TWELL_ERR_INVALID_ARG;
    if (y == x || y == res || (sum && (sum == x || sum == res || sum == y))) return TWELL_ERR_INVALID_ARG;
    if (!elem_aligned(x, x_type) || !elem_aligned(res, x_type) || !elem_aligned(sum, x_type) ||
        !elem_aligned(y, y_type) || !elem_aligned(w, w_type) || !elem_aligned(b, w_type) ||
        !elem_aligned(mean, TWELL_F32) || !elem_aligned(rstd, TWELL_F32))
        return TWELL_ERR_INVALID_ARG;
    int vec = x_type == TWELL_BF16 && y_type == TWELL_BF16 ? 8 : 4;
    while (vec > 1 && d % vec) vec = vec > 2 ? 2 : 1;
    vec = pieces(x, ldx, N, x_type, vec);
    vec = pieces(res, ldres, N, x_type, vec);
    vec = pieces(sum, ldsum, N, x_type, vec);
    vec = pieces(y, ldy, N, y_type, vec);
    vec = weight_pieces(w, w_type, vec);
    vec = weight_pieces(b, w_type, vec);
    const FwdArgs a{x, res, w, b, sum, y, ldx, ldres, ldsum, ldy, N, d, eps, mean, rstd,
                    w_type == TWELL_F32};
    const cudaError_t e = by_types(x_type, y_type, [&](auto tx, auto ty) {
        return fwd<decltype(tx), decltype(ty)>(a, vec, static_cast<cudaStream_t>(stream));
    });
    return e == cudaSuccess ? TWELL_OK : TWELL_ERR_CUDA;
}

extern "C" size_t twell_layernorm_bwd_workspace_bytes(int64_t N, int d)
{
    if (N < 0 || d < 1 || d > kMaxWidth) return 0;
    const size_t n = (size_t)parts_for(N, d) * 2 * d * sizeof(float);
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
    if (d > kMaxWidth) return TWELL_ERR_UNSUPPORTED;
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
    int vec = x_type == TWELL_BF16 && y_type == TWELL_BF16 ? 8 : 4;
    while (vec > 1 && d % vec) vec = vec > 2 ? 2 : 1;
    vec = pieces(dy, lddy, N, y_type, vec);
    vec = pieces(x, ldx, N, x_type, vec);
    vec = pieces(dres, lddres, N, x_type, vec);
    vec = pieces(dx, lddx, N, x_type, vec);
    vec = weight_pieces(w, w_type, vec);
    // few rows: the column sums by blocks of their own, which read the rows again (from L2)
    const bool direct = dw && N <= kFewRows && group_of(d) != 0;
    const BwdArgs a{dy, x, w, dres, dx, lddy, ldx, lddres, lddx, N, d, mean, rstd,
                    dw && !direct ? static_cast<float*>(ws) : nullptr, parts_for(N, d),
                    direct ? dw : nullptr, direct ? db : nullptr, w_type == TWELL_F32};
    const cudaError_t e = by_types(x_type, y_type, [&](auto tx, auto ty) {
        return bwd<decltype(tx), decltype(ty)>(a, vec, dw, db, s);
    });
    return e == cudaSuccess ? TWELL_OK : TWELL_ERR_CUDA;
}
