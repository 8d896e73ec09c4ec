// twell_mm.cu — dense products with the linear and gated layers' epilogues.
//
// D = A B^T on CTA pairs (tcgen05.mma.cta_group::2, 256 x 256 tiles), bf16 operands
// by TMA, fp32 accumulators in tensor memory, two of them so that a tile's epilogue
// runs under the next tile's products. Bound by the tensor cores for hundreds of
// rows and more.
//
//   LINEAR     act(D + bias) + res in bf16 or fp32, the pre-activation kept on demand.
//              Several products can be added up (segments: the gated layer's
//              dx = dg Wg + du Wu, one accumulator for both), or several of the same sizes
//              computed side by side (problems: dWg, dWu, dWd), so that only one launch
//              ends with partly filled waves of tiles.
//   GATED      one CTA of the pair brings 128 rows of W_gate, the other 128 of W_up:
//              a tile's accumulator holds g in its first and u in its last 128 columns,
//              so the same thread has both, and neither has to be written for h.
//   GATED_BWD  D = dh; with g and u, dg and du are formed while the next tile is
//              computed; dh itself is never written.
//
// Few rows (decode batches): the weights' rows are the tensor cores' 128-row operand and
// the tokens its columns, so that a tile reads 128 rows of W once, whatever the batch
// (k_mm_few). Bound by memory: the depth is split over a cluster of CTAs until the whole GPU
// streams, and the parts are added up through the cluster's shared memory, in order.
//
// Roles as in twell_gemm.cu: warp 0 loads, warp 1 (even CTA) issues the products, 8 or 16
// warps form the results of 32 rows x 128 or 64 columns each and store them through 4 KB of
// their own shared memory, whole pieces of rows at a time.
#include "activation.cuh"
#include "common.cuh"
#include "gemm_common.cuh"
#include "launch.h"
#include "mm.h"

#include <atomic>

namespace twell {
namespace {

enum Epilogue { LINEAR, GATED, GATED_BWD };

constexpr int kBox = 4096;  // 32 rows x 128 bytes of one epilogue warp

// GATED_BWD's results take the longest to form (two matrices in, two out, column sums): 16 warps of 64 columns, and a
// ring one stage shorter for their boxes. With eight of 128 the epilogue took longer than a tile's products (8192 x 4096 x
// 14336 807 us; with 16, and g and u asked for early, 690 in pieces of 1024 of depth, 709 of 768, 748 of 512).
template <int EPI>
struct Smem {
    static constexpr int STAGES = EPI == GATED_BWD ? 5 : 6;
    static constexpr int WARPS = EPI == GATED_BWD ? 16 : 8;    // of the epilogue
    static constexpr int COLS = EPI == LINEAR ? 128 : 64;      // output columns of one of them
    static constexpr int THREADS = 64 + 32 * WARPS;
    static constexpr int A_BYTES = HALF * BK * 2;
    static constexpr int STAGE_BYTES = 2 * A_BYTES;
    static constexpr int BOX_OFF = STAGES * STAGE_BYTES;
    static constexpr int BAR_OFF = BOX_OFF + WARPS * kBox;
    static constexpr int NBARS = 2 * STAGES + 5;
    static constexpr int MISC_OFF = BAR_OFF + NBARS * 8;
    static constexpr int TOTAL = MISC_OFF + 16 + 1024;  // + alignment slack
    static_assert(TOTAL <= 227 * 1024, "shared memory of one CTA");
};

// The tensor cores' fp32 sums drop what does not fit, towards zero, at each step of 16 of depth: over 512 by 2 to 3
// units of 2^-23 of the result, over 1024 by 7, over 4096 by 31 to 70, over 16384 four times that. Results that leave in
// fp32, and the dh that db is summed from, are therefore summed 512 at a time and the pieces added up with rounding: 4.8e-7
// off 64 bits in norm at any depth, where fp32 matrix products by torch are 2.5e-7 (depth 1000), 6.1e-7 (4096) and 9.6e-7
// (8192) off. Both sides of the length: 768, 7.2e-7; 256, 2.5e-7. Linear backward 8192 x 4096 -> 16384 with fp32 dW 1266 us
// at 768, 1289 at 512, 1341 at 256; gated backward 8192 x 4096 x 14336 with bf16 dW 3144, 3189 and 3273. Few rows (k_mm_few),
// whose time goes into W, 256 at a time, which costs 0 to 1 us (61 x 50001 x 2048 39.5 us at 768, 39.8 at 256; 128 rows
// 53.5 and 54.3).
// Results that leave in bf16, 16384 at a time: the loss is then 280 units of 2^-23 at most, a hundredth of their own
// rounding, whatever the depth (of a weight gradient the number of rows).
constexpr int kPieceBlocks = 8, kFewPieceBlocks = 4, kPieceBlocksBf16 = 256;

struct Maps {
    CUtensorMap a[kMmParts], b[kMmParts];
};

struct Args {
    int rowsA, rowsB, num_kb;  // output rows and columns, 64-deep k-blocks of one segment
    int segments, problems;
    int piece;                 // k-blocks that the tensor cores sum by themselves
    const float* bias;
    int act;
    const void* res;
    int64_t ldres;
    uint16_t* pre;
    int64_t ldpre;
    void* out[kMmParts];
    int64_t ldo;
    int out_f32;
    int accumulate;
    int vec;                   // bits: out, res, pre have 16-byte pieces (base, row stride and width allow them)
    // gated
    uint16_t *g, *u, *h;
    const uint16_t *g_in, *u_in;
    float l1;
    float* part;
    int early;                 // few rows: W does not come from the launch before, and may be loaded before that has ended
    int32_t* status;
};
enum { VEC_OUT = 1, VEC_RES = 2, VEC_PRE = 4 };

__device__ __forceinline__ void fail(int32_t* status, volatile int* abort_flag)
{
    set_error(status, TWELL_ERR_TIMEOUT);
    *abort_flag = 1;
}

// 32 rows of 128 bytes between a warp's accumulator rows (lane = row) and global memory, where eight lanes share
// a row. 16-byte pieces are permuted within a row so that both sides touch different banks.
struct Box {
    uint8_t* box;
    int lane;
    __device__ __forceinline__ uint4* at(int row, int c) const
    {
        // (eight rows' same piece, two rows' same four and one row's eight each touch all banks)
        return reinterpret_cast<uint4*>(box + row * 128 + ((c ^ ((row & 1) << 2 | (row >> 1 & 3))) << 4));
    }
    __device__ __forceinline__ void put(int c, const uint4& v) { *at(lane, c) = v; }
    __device__ __forceinline__ uint4 get(int c) const { return *at(lane, c); }

    // The box's first `rows` rows and `cols` columns (elements of ES bytes) to rows of `stride` bytes at `to`.
    template <int ES>
    __device__ __forceinline__ void store(void* to, size_t stride, int rows, int cols, bool vec)
    {
        constexpr int E = 16 / ES;
        __syncwarp();
        const int c = lane & 7, r0 = lane >> 3;
        char* p = static_cast<char*>(to) + r0 * stride + c * 16;
        if (vec) {
            if (c * E < cols) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (i * 4 + r0 < rows) *reinterpret_cast<uint4*>(p) = *at(i * 4 + r0, c);
                    p += 4 * stride;
                }
            }
        } else {
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {
                const uint4 q = *at(i * 4 + r0, c);
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
                if (i * 4 + r0 < rows) {
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        if (c * E + e < cols) {
                            if constexpr (ES == 4)
                                reinterpret_cast<uint32_t*>(p)[e] = w[e];
                            else
                                reinterpret_cast<uint16_t*>(p)[e] = (uint16_t)(w[e >> 1] >> ((e & 1) * 16));
                        }
                }
                p += 4 * stride;
            }
        }
        __syncwarp();
    }

    // The same way back; what lies outside is 0.
    template <int ES>
    __device__ __forceinline__ void load(const void* from, size_t stride, int rows, int cols, bool vec)
    {
        constexpr int E = 16 / ES;
        const int c = lane & 7, r0 = lane >> 3;
        const char* p = static_cast<const char*>(from) + r0 * stride + c * 16;
        if (vec) {
            uint4 q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                q[i] = make_uint4(0, 0, 0, 0);
                if (i * 4 + r0 < rows && c * E < cols) q[i] = *reinterpret_cast<const uint4*>(p);
                p += 4 * stride;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) *at(i * 4 + r0, c) = q[i];
        } else {
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {
                uint32_t w[4] = {0, 0, 0, 0};
                if (i * 4 + r0 < rows) {
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        if (c * E + e < cols) {
                            if constexpr (ES == 4)
                                w[e] = reinterpret_cast<const uint32_t*>(p)[e];
                            else
                                w[e >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[e] << ((e & 1) * 16);
                        }
                }
                *at(i * 4 + r0, c) = make_uint4(w[0], w[1], w[2], w[3]);
                p += 4 * stride;
            }
        }
        __syncwarp();
    }

    // N values of the lane's row as bf16 in the pieces from c0 on.
    template <int N>
    __device__ __forceinline__ void put_bf16(const float (&v)[N], int c0 = 0)
    {
#pragma unroll
        for (int c = 0; c < N / 8; ++c) put(c0 + c, pack8(v + c * 8));
    }
    static __device__ __forceinline__ uint4 pack8(const float* v)
    {
        return make_uint4(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]), cvt_bf16x2(v[4], v[5]), cvt_bf16x2(v[6], v[7]));
    }

    // Two bf16 matrices of one layout side by side: 32 columns of the first in pieces 0 to 3, of the second in 4 to
    // 7. `at` is the element of row 0 and column 0, rows have `ld` elements and lie on 16-byte boundaries.
    __device__ __forceinline__ void store_two(uint16_t* m0, uint16_t* m1, size_t at, int64_t ld, int rows, int cols)
    {
        __syncwarp();
        const int c = lane & 3, r0 = lane >> 2;
        if (c * 8 < cols) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (i * 8 + r0 < rows) {
                    const size_t o = at + (size_t)(i * 8 + r0) * ld + c * 8;
                    *reinterpret_cast<uint4*>(m0 + o) = *this->at(i * 8 + r0, c);
                    *reinterpret_cast<uint4*>(m1 + o) = *this->at(i * 8 + r0, 4 + c);
                }
            }
        }
        __syncwarp();
    }
};

template <int N>
__device__ __forceinline__ void read_columns(uint32_t taddr, float (&v)[N])
{
#pragma unroll
    for (int ch = 0; ch < N / 32; ++ch) {
        uint32_t r[32];
        tmem_ld32_wait(taddr + ch * 32, r);
#pragma unroll
        for (int c = 0; c < 32; ++c) v[ch * 32 + c] = __uint_as_float(r[c]);
    }
}

template <int ACT, int N>
__device__ __forceinline__ void activate_all(float (&v)[N])
{
#pragma unroll
    for (int c = 0; c < N; c += 2) {
        const float2 y = activate<ACT>(make_float2(v[c], v[c + 1]));
        v[c] = y.x;
        v[c + 1] = y.y;
    }
}

// bias[col .. col + N - 1] (0 past `cols` of them, or without a bias) added to v, by way of the lanes' registers.
template <int N>
__device__ __forceinline__ void add_bias(const float* bias, int col, int cols, int lane, float (&v)[N])
{
    if (!bias) return;
#pragma unroll
    for (int ch = 0; ch < N / 32; ++ch) {
        const float b = ch * 32 + lane < cols ? bias[col + ch * 32 + lane] : 0.f;
#pragma unroll
        for (int c = 0; c < 32; ++c) v[ch * 32 + c] += __shfl_sync(0xffffffffu, b, c);
    }
}

// 32 rows x `width` columns from col0 on: bias, activation, residual. read(offset, v): 64 sums of the lane's row from
// col0 + offset on (those past the width may be anything).
template <class Read>
__device__ __forceinline__ void epi_linear(Read read, int width, int row0, int col0, int problem, const Args& a, Box& box)
{
    const int rows = a.rowsA - row0;
#pragma unroll 1
    for (int ch = 0; ch * 64 < width; ++ch) {
        const int col = col0 + ch * 64, cols = min(a.rowsB - col, width - ch * 64);
        if (cols <= 0) break;
        float v[64];
        read(ch * 64, v);
        add_bias(a.bias, col, cols, box.lane, v);
        if (a.pre) {
            box.put_bf16(v);
            box.store<2>(a.pre + (size_t)row0 * a.ldpre + col, (size_t)a.ldpre * 2, rows, cols, a.vec & VEC_PRE);
        }
        if (a.act != TWELL_ACT_NONE)
            by_activation(a.act, [&](auto tag) {
                activate_all<decltype(tag)::value>(v);
            });
        if (a.out_f32) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (half * 32 >= cols) break;
                if (a.res || a.accumulate) {
                    // (an element of out is read and written by the same lane)
                    const float* from = static_cast<const float*>(a.accumulate ? a.out[problem] : a.res);
                    const int64_t ld = a.accumulate ? a.ldo : a.ldres;
                    box.load<4>(from + (size_t)row0 * ld + col + half * 32, (size_t)ld * 4, rows, cols - half * 32,
                                a.vec & (a.accumulate ? VEC_OUT : VEC_RES));
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const uint4 q = box.get(c);
                        float* w = v + half * 32 + c * 4;
                        w[0] += __uint_as_float(q.x);
                        w[1] += __uint_as_float(q.y);
                        w[2] += __uint_as_float(q.z);
                        w[3] += __uint_as_float(q.w);
                    }
                }
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const float* w = v + half * 32 + c * 4;
                    box.put(c, make_uint4(__float_as_uint(w[0]), __float_as_uint(w[1]), __float_as_uint(w[2]),
                                          __float_as_uint(w[3])));
                }
                box.store<4>(static_cast<float*>(a.out[problem]) + (size_t)row0 * a.ldo + col + half * 32, (size_t)a.ldo * 4, rows,
                             cols - half * 32, a.vec & VEC_OUT);
            }
        } else {
            if (a.res) {
                box.load<2>(static_cast<const uint16_t*>(a.res) + (size_t)row0 * a.ldres + col, (size_t)a.ldres * 2, rows, cols,
                            a.vec & VEC_RES);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const uint4 q = box.get(c);
                    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v[c * 8 + 2 * e] += bf16_lo(w[e]);
                        v[c * 8 + 2 * e + 1] += bf16_hi(w[e]);
                    }
                }
            }
            box.put_bf16(v);
            box.store<2>(static_cast<uint16_t*>(a.out[problem]) + (size_t)row0 * a.ldo + col, (size_t)a.ldo * 2, rows, cols,
                         a.vec & VEC_OUT);
        }
    }
}

// 32 rows x 64 hidden units from col on; g at taddr, u 128 columns further.
__device__ __forceinline__ void epi_gated(uint32_t taddr, int row0, int col, const Args& a, Box& box)
{
    const int rows = a.rowsA - row0, cols = a.rowsB - col;
    uint4 h[8];
#pragma unroll
    for (int ch = 0; ch < 2; ++ch) {
        float g[32], u[32];
        read_columns(taddr + ch * 32, g);
        add_bias(a.bias, col + ch * 32, cols - ch * 32, box.lane, g);
        read_columns(taddr + HALF + ch * 32, u);
        if (a.g) {
            box.put_bf16(g);
            box.put_bf16(u, 4);
            box.store_two(a.g, a.u, (size_t)row0 * a.ldo + col + ch * 32, a.ldo, rows, cols - ch * 32);
        }
        by_activation(a.act, [&](auto tag) {
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
                const float2 h = __fmul2_rn(activate<decltype(tag)::value>(make_float2(g[c], g[c + 1])), make_float2(u[c], u[c + 1]));
                g[c] = h.x;
                g[c + 1] = h.y;
            }
        });
#pragma unroll
        for (int c = 0; c < 4; ++c) h[ch * 4 + c] = Box::pack8(g + c * 8);
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) box.put(c, h[c]);
    box.store<2>(a.h + (size_t)row0 * a.ldo + col, (size_t)a.ldo * 2, rows, cols, true);
}

// GATED_BWD: g and u come into a warp's shared memory by asynchronous copies, 16 columns of both at a time, while the 16
// columns before are worked on (those of the next tile too): two halves of a box, each 32 rows of 64 bytes (g's two
// pieces, then u's), which dg and du take the place of on their way out. (Loaded when their turn came, they were two
// fifths of the epilogue: 8192 x 512 x 14336 337 us, 201 without.)
struct HalfBox {
    uint8_t* box;
    int lane;
    __device__ __forceinline__ uint4* at(int half, int row, int c) const
    {
        // (eight rows' same piece and two rows' all four touch all banks)
        return reinterpret_cast<uint4*>(box + half * 2048 + row * 64 + ((c ^ (row >> 1 & 3)) << 4));
    }
    // Lane's place in a matrix for rows i * 8 + lane / 4: pieces 0 and 1 are the first matrix's, 2 and 3 the second's.
    __device__ __forceinline__ int piece() const { return lane & 3; }

    // Asks for rows row0 .. row0 + 31 and columns col .. col + 15; what lies outside becomes 0.
    __device__ __forceinline__ void fetch(int half, int row0, int col, const Args& a) const
    {
        const int c = piece(), r0 = lane >> 2;
        const uint16_t* m = c < 2 ? a.g_in : a.u_in;
        const int mc = col + (c & 1) * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = row0 + i * 8 + r0;
            const bool ok = row < a.rowsA && mc < a.rowsB;
            const uint16_t* from = ok ? m + (size_t)row * a.ldo + mc : m;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(at(half, i * 8 + r0, c))), "l"(from),
                         "r"(ok ? 16 : 0)
                         : "memory");
        }
    }
    __device__ __forceinline__ void store(int half, int row0, int col, const Args& a) const
    {
        const int c = piece(), r0 = lane >> 2;
        uint16_t* m = c < 2 ? a.g : a.u;
        const int mc = col + (c & 1) * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = row0 + i * 8 + r0;
            if (row < a.rowsA && mc < a.rowsB) *reinterpret_cast<uint4*>(m + (size_t)row * a.ldo + mc) = *at(half, i * 8 + r0, c);
        }
    }
};
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the last group have landed.
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

// l1 with the sign of act u, 0 where either is 0.
__device__ __forceinline__ float l1_term(float l1, float act, float u)
{
    const uint32_t sign = (__float_as_uint(act) ^ __float_as_uint(u)) & 0x80000000u;
    return act != 0.f && u != 0.f ? __uint_as_float(__float_as_uint(l1) ^ sign) : 0.f;
}

// 32 rows x 64 hidden units from col0 on of dh, the first 16 columns of g and u already asked for. next_row0, next_col0:
// where the next tile's begin (next_row0 < 0: there is none). Rows and columns outside have g = u = 0 and dh = 0, so
// dg = du = 0.
__device__ __forceinline__ void epi_gated_bwd(uint32_t taddr, int row0, int col0, int next_row0, int next_col0, const Args& a,
                                              const HalfBox& box)
{
#pragma unroll 1
    for (int ch = 0; ch < 4; ++ch) {
        const int col = col0 + ch * 16, half = ch & 1, lane = box.lane;
        if (ch < 3)
            box.fetch(half ^ 1, row0, col + 16, a);
        else if (next_row0 >= 0)
            box.fetch(half ^ 1, next_row0, next_col0, a);
        copies_commit();
        uint32_t dh[16];
        tmem_ld16_wait(taddr + ch * 16, dh);
        copies_wait();
        __syncwarp();
        float dg[16];
        by_activation(a.act, [&](auto tag) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const uint4 qg = *box.at(half, lane, c), qu = *box.at(half, lane, 2 + c);
                const uint32_t wg[4] = {qg.x, qg.y, qg.z, qg.w}, wu[4] = {qu.x, qu.y, qu.z, qu.w};
                float du[8];
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float2 g = make_float2(bf16_lo(wg[e >> 1]), bf16_hi(wg[e >> 1]));
                    const float2 u = make_float2(bf16_lo(wu[e >> 1]), bf16_hi(wu[e >> 1]));
                    float2 da, d = make_float2(__uint_as_float(dh[c * 8 + e]), __uint_as_float(dh[c * 8 + e + 1]));
                    const float2 act = activate<decltype(tag)::value>(g, &da);
                    if (a.l1 != 0.f) {
                        d.x += l1_term(a.l1, act.x, u.x);
                        d.y += l1_term(a.l1, act.y, u.y);
                    }
                    const float2 by_g = __fmul2_rn(__fmul2_rn(d, u), da), by_u = __fmul2_rn(d, act);
                    dg[c * 8 + e] = by_g.x;
                    dg[c * 8 + e + 1] = by_g.y;
                    du[e] = by_u.x;
                    du[e + 1] = by_u.y;
                }
                // rounded to bf16 once, as operands of the products that follow; the bias's gradient is summed before
                *box.at(half, lane, c) = Box::pack8(dg + c * 8);
                *box.at(half, lane, 2 + c) = Box::pack8(du);
            }
        });
        __syncwarp();
        box.store(half, row0, col, a);
        if (a.part && row0 < a.rowsA) {
            transpose_reduce16(dg, lane);  // lane u: column u over the 32 rows
            if (lane < 16 && col + lane < a.rowsB) a.part[(size_t)(row0 / kSumRows) * a.rowsB + col + lane] = dg[0];
        }
        __syncwarp();
    }
}

// N accumulator columns of a thread's row added to sum; or sum put in their place.
template <int N>
__device__ __forceinline__ void add_columns(uint32_t taddr, float (&sum)[N])
{
#pragma unroll
    for (int ch = 0; ch < N / 16; ++ch) {
        uint32_t v[16];
        tmem_ld16_wait(taddr + ch * 16, v);
#pragma unroll
        for (int c = 0; c < 16; ++c) sum[ch * 16 + c] += __uint_as_float(v[c]);
    }
}
template <int N>
__device__ __forceinline__ void set_columns(uint32_t taddr, const float (&sum)[N])
{
#pragma unroll
    for (int ch = 0; ch < N / 32; ++ch) {
        uint32_t v[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) v[c] = __float_as_uint(sum[ch * 32 + c]);
        tmem_st32(taddr + ch * 32, v);
    }
    tmem_st_wait();
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// LINEAR with few tiles: the pairs of a cluster have a part of the depth of one tile each. Every pair finishes its share
// of the tile's columns: its own sums stay in tensor memory, the others' go to shared memory, in the place of the
// operands' ring, and are read from there by the pair that needs them; parts are added in order. (4096 x 4096, 512 rows:
// 25 us in one part, 20 in two; 1024 x 4096, 256 rows: 24 us in one, 18 in two, 16 in four.)
// Four columns of a row lie together, then the rows, then the next four columns: a warp's 16-byte accesses touch 512
// bytes in a row. (Rows apart, each lane's piece crossed the cluster by itself: 5 us more for each part.)
__device__ __forceinline__ float* part_row(uint8_t* smem, int share, int owner, int row)
{
    return reinterpret_cast<float*>(smem) + (size_t)owner * HALF * share + row * 4;
}

// 32 sums of a row from the tile's column c0 on, for the pair that finishes them.
__device__ __forceinline__ void put_part(uint8_t* smem, int share, int my_part, int row, int c0, const float* v)
{
    const int owner = c0 / share;
    if (owner == my_part) return;
    float4* to = reinterpret_cast<float4*>(part_row(smem, share, owner, row) + (c0 - owner * share) * HALF);
#pragma unroll
    for (int c = 0; c < 8; ++c) to[c * HALF] = make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
}

// The products of one launch. Two of them (JOBS = 2, LINEAR): a backward pass' dx and its weight gradients, which need the
// same operands and nothing of one another. Each by itself seldom fills its last wave of tiles; together the short tiles
// (the weight gradients', as deep as there are rows) fill up what the long ones leave: first the long ones, then the
// short ones, `delay` rounds of them by the pairs without a long tile in the last round of those alone. (`delay` is what
// a long tile takes in short ones. In two launches, and in one: linear backward 1000 x 1024 -> 1024 24 us, 14; 4096 x 4096 ->
// 4096 174, 157; gated backward 2048 x 1000 x 2696 107, 93.)
template <int JOBS>
struct Jobs {
    Maps maps[JOBS];
    Args args[JOBS];
    int delay;
    float us[JOBS];  // about, of a tile (the host's)
};

__device__ __forceinline__ int tiles_of(const Args& a, int tile_n)
{
    return ((a.rowsA + PAIR_M - 1) / PAIR_M) * ((a.rowsB + tile_n - 1) / tile_n) * a.problems;
}

// A pair's tiles in their order; all roles of both CTAs walk along the same ones. What does not change lies in shared
// memory (the epilogue has no registers left).
struct Route {
    int pair, pairs, count[2];
    int start, free, head;  // of job 1: first tile, pairs without a tile in the last round of job 0, tiles for those alone
};

template <int JOBS, int TILE_N>
__device__ __forceinline__ void set_route(Route& r, const Jobs<JOBS>& jobs, int pair, int pairs)
{
    r.pair = pair;
    r.pairs = pairs;
    r.count[0] = tiles_of(jobs.args[0], TILE_N);
    if constexpr (JOBS > 1) {
        r.count[1] = tiles_of(jobs.args[1], TILE_N);
        const int busy = r.count[0] % pairs;
        r.free = pairs - busy;
        r.head = jobs.delay * r.free;
        r.start = pair >= busy ? pair - busy : r.head + pair;
    }
}

template <int JOBS>
struct Walk {
    const Route& r;
    int job, tile;
    __device__ __forceinline__ Walk(const Route& route) : r(route), job(0), tile(route.pair) { enter(); }
    __device__ __forceinline__ bool more() const { return tile < r.count[JOBS > 1 ? job : 0]; }
    __device__ __forceinline__ void next()
    {
        if (JOBS > 1 && job == 1 && tile < r.head) {
            tile += r.free;
            if (tile >= r.head) tile = r.head + r.pair;
        } else {
            tile += r.pairs;
            enter();
        }
    }
    __device__ __forceinline__ void enter()
    {
        if (JOBS > 1 && job == 0 && tile >= r.count[0]) {
            job = 1;
            tile = r.start;
        }
    }
};

// (of two jobs the first has K-major rows and B_MN, the second both as their transposes)
template <int EPI, bool A_MN, bool B_MN, int JOBS>
__global__ void __launch_bounds__(Smem<EPI>::THREADS, 1) k_mm_pair(const __grid_constant__ Jobs<JOBS> jobs, int parts_arg, int per)
{
    static_assert(JOBS == 1 || (EPI == LINEAR && !A_MN), "two jobs");
    const int parts = EPI == LINEAR && JOBS == 1 ? parts_arg : 1;
    using L = Smem<EPI>;
    constexpr int kStages = L::STAGES;
    constexpr int TILE_N = EPI == GATED ? HALF : PAIR_N;  // output columns of a tile
    const Args& first = jobs.args[0];
    int32_t* const status = first.status;
    extern __shared__ uint8_t smem_raw[];
    // Same offset in both CTAs: the pair's products address the peer's operands with the leader's descriptors.
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::BAR_OFF);
    uint64_t* empty = full + kStages;
    uint64_t* tfull = empty + kStages;
    uint64_t* tempty = tfull + 2;
    uint64_t* mma_done = tempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::MISC_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* skip = reinterpret_cast<volatile int*>(tmem_slot + 2);
    __shared__ Route route;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t crank = cluster_rank(), rank = crank & 1u, lead = crank & ~1u;  // rank in the pair, its even CTA
    const int my_part = (int)(crank >> 1);
    const uint16_t both_ctas = (uint16_t)(3u << lead);
    const bool leader = rank == 0;
    if (threadIdx.x == 0) {
        // (in parts: one tile for each cluster)
        set_route<JOBS, TILE_N>(route, jobs, (int)blockIdx.x / (2 * parts), (int)gridDim.x / (2 * parts));
        *skip = (crank == 0 && has_error(status)) ? 1 : 0;
        *abort_flag = 0;
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], 2 * L::WARPS);
        }
        mbar_init(mma_done, 1);
        fence_mbar_init();
    }
    cluster_sync();  // barriers of both CTAs initialised before either uses the other's
    const int sk = ld_cluster_s32(cluster_addr(const_cast<int*>(skip), 0));
    cluster_sync();  // the leader's flag has been read before anyone may leave
    if (sk) return;  // an earlier kernel of this call failed; uniform over the cluster
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, 2 * PAIR_N);
        tmem_relinquish_pair();
    }
    if (warp == 0 && lane == 0) {
#pragma unroll
        for (int j = 0; j < JOBS; ++j)
            for (int i = 0; i < jobs.args[j].segments * jobs.args[j].problems; ++i) {
                tma_prefetch_map(&jobs.maps[j].a[i]);
                tma_prefetch_map(&jobs.maps[j].b[i]);
            }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    // this pair's k-blocks of a job's tiles
    auto from = [&](const Args& a) { return parts > 1 ? min(my_part * per, a.num_kb * a.segments) : 0; };
    auto to = [&](const Args& a) { return parts > 1 ? min(from(a) + per, a.num_kb * a.segments) : a.num_kb * a.segments; };
    // a tile's product and coordinates
    auto locate = [&](const Args& a, int tile, int* problem, int* mb, int* nb) {
        const int num_m = (a.rowsA + PAIR_M - 1) / PAIR_M, num_n = (a.rowsB + TILE_N - 1) / TILE_N;
        *problem = tile / (num_m * num_n);
        pair_tile_coords(tile - *problem * (num_m * num_n), num_m, num_n, mb, nb);
    };
    Box box{smem + L::BOX_OFF + (warp >= 2 ? warp - 2 : 0) * kBox, lane};
    int last_acc = 0;

    if (warp == 0) {
        // ------------------------------------------------ TMA producer ----
        if (lane == 0) {
            const uint32_t full_leader = cluster_addr(full, lead);
            int stage = 0;
            uint32_t phase = 0;
            long long issued = 0;
            bool ok = true;
            for (Walk<JOBS> at(route); ok && at.more(); at.next()) {
                const int job = JOBS > 1 ? at.job : 0;
                const Args& a = jobs.args[job];
                const Maps& maps = jobs.maps[job];
                const bool a_mn = JOBS > 1 ? job == 1 : A_MN, b_mn = JOBS > 1 ? job == 1 || B_MN : B_MN;
                int mb, nb, problem;
                locate(a, at.tile, &problem, &mb, &nb);
                const int k0 = from(a), k1 = to(a);
                const int ma = mb * PAIR_M + (int)rank * HALF;
                // GATED: 128 rows of W_gate in the even CTA, the same rows of W_up in the odd one
                const int nbr = EPI == GATED ? nb * HALF : nb * PAIR_N + (int)rank * HALF;
                for (int k = k0; ok && k < k1;) {
                    const int seg = k / a.num_kb, end = min(k1, (seg + 1) * a.num_kb) - seg * a.num_kb;
                    const CUtensorMap* ta = &maps.a[problem + seg];
                    const CUtensorMap* tb = &maps.b[EPI == GATED ? (int)rank : problem + seg];
                    for (int kb = k - seg * a.num_kb; kb < end; ++kb, ++k) {
                        if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag)) {
                            ok = false;
                            break;
                        }
                        uint8_t* sa = smem + stage * L::STAGE_BYTES;
                        if (leader) mbar_arrive_expect_tx(&full[stage], 2 * L::STAGE_BYTES);
                        const uint32_t fb = full_leader + 8u * (uint32_t)stage;
                        if (a_mn) {
                            tma_load_2d_pair(sa, ta, ma, kb * BK, fb);
                            tma_load_2d_pair(sa + kMnBox * BK * 2, ta, ma + kMnBox, kb * BK, fb);
                        } else {
                            tma_load_2d_pair(sa, ta, kb * BK, ma, fb);
                        }
                        if (b_mn) {
                            tma_load_2d_pair(sa + L::A_BYTES, tb, nbr, kb * BK, fb);
                            tma_load_2d_pair(sa + L::A_BYTES + kMnBox * BK * 2, tb, nbr + kMnBox, kb * BK, fb);
                        } else {
                            tma_load_2d_pair(sa + L::A_BYTES, tb, kb * BK, nbr, fb);
                        }
                        ++issued;
                        if (++stage == kStages) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                }
            }
            if (!ok) fail(status, abort_flag);
            // The last load issued into each stage must land before the CTA exits: the leader sees it on its full
            // barrier, the peer on its empty barrier (the leader's products consumed it).
            for (int s = 0; s < kStages; ++s) {
                const long long n_s = issued / kStages + (s < issued % kStages ? 1 : 0);
                if (n_s > 0) mbar_wait(leader ? &full[s] : &empty[s], (uint32_t)((n_s - 1) & 1), nullptr);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------- MMA issuer (even CTA) -----
        if (leader && lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            int acc = 0;
            uint32_t acc_phase = 0;
            bool ok = true;
            for (Walk<JOBS> at(route); ok && at.more(); at.next()) {
                const int job = JOBS > 1 ? at.job : 0;
                const Args& a = jobs.args[job];
                const bool a_mn = JOBS > 1 ? job == 1 : A_MN, b_mn = JOBS > 1 ? job == 1 || B_MN : B_MN;
                const uint32_t idesc = idesc_bf16_f32(PAIR_M, PAIR_N) | (a_mn ? kIdescAMn : 0u) | (b_mn ? kIdescBMn : 0u);
                // descriptor units (16 B) per 16-deep K step
                const uint64_t a_kstep = a_mn ? (16u * 128u) >> 4 : 2u, b_kstep = b_mn ? (16u * 128u) >> 4 : 2u;
                const int depth = to(a) - from(a);
                for (int kb0 = 0, kb1; ok && kb0 < depth; kb0 = kb1) {
                    kb1 = min(kb0 + a.piece, depth);
                    if (!mbar_wait(&tempty[acc], acc_phase ^ 1u, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d_tmem = tmem_base + (uint32_t)(acc * PAIR_N);
                    for (int kb = kb0; kb < kb1; ++kb) {
                        if (!mbar_wait(&full[stage], phase, abort_flag)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t sa = smem_u32(smem + stage * L::STAGE_BYTES);
                        const uint64_t adesc = operand_desc(a_mn, sa);
                        const uint64_t bdesc = operand_desc(b_mn, sa + L::A_BYTES);
#pragma unroll
                        for (int k = 0; k < BK / 16; ++k)
                            umma_bf16_pair(d_tmem, adesc + a_kstep * k, bdesc + b_kstep * k, idesc, ((kb - kb0) | k) != 0);
                        umma_commit_pair(&empty[stage], both_ctas);
                        if (++stage == kStages) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                    if (!ok) break;
                    umma_commit_pair(&tfull[acc], both_ctas);
                    acc ^= 1;
                    if (acc == 0) acc_phase ^= 1u;
                }
            }
            if (!ok) fail(status, abort_flag);
            umma_commit_pair(mma_done, (uint16_t)(1u << lead));  // every product issued above has finished once this arrives
            mbar_wait(mma_done, 0, nullptr);
        }
    } else {
        // --------------------------------------------------- epilogue -----
        const int q = warp & 3;              // TMEM lane quarter this warp may read
        const int slice = (warp - 2) >> 2;   // its columns of the accumulator
        const uint32_t tempty_leader = cluster_addr(tempty, lead);
        const uint32_t lanes_at = tmem_base + ((uint32_t)(32 * q) << 16);
        Walk<JOBS> at(route);
        if (EPI == GATED_BWD && at.more()) {
            int mb, nb, problem;
            locate(first, at.tile, &problem, &mb, &nb);
            HalfBox{box.box, lane}.fetch(0, mb * PAIR_M + (int)rank * HALF + 32 * q, nb * TILE_N + L::COLS * slice, first);
            copies_commit();
        }
        int acc = 0;
        uint32_t acc_phase = 0;
        bool ok = true;
        auto finish = [&](const Args& a) {
            const int depth = to(a) - from(a);
            const bool pieces = depth > a.piece;
            int mb, nb, problem;
            locate(a, at.tile, &problem, &mb, &nb);
            const int row0 = mb * PAIR_M + (int)rank * HALF + 32 * q;
            const int col0 = nb * TILE_N + L::COLS * slice;
            const bool live = row0 < a.rowsA && col0 < a.rowsB;  // not all past the last row or column
            ok = __all_sync(0xffffffffu, mbar_wait(&tfull[acc], acc_phase, abort_flag));
            if (!ok) return;
            tc_fence_after();
            if (pieces) {
                constexpr int W = EPI == GATED ? 2 : 1;  // (g and u)
                float sum[W][L::COLS];
#pragma unroll
                for (int w = 0; w < W; ++w)
#pragma unroll
                    for (int k = 0; k < L::COLS; ++k) sum[w][k] = 0.f;
                int done = 0;
                while (true) {
                    const uint32_t sums = lanes_at + (uint32_t)(acc * PAIR_N + L::COLS * slice);
                    done += a.piece;
                    if (live) {
#pragma unroll
                        for (int w = 0; w < W; ++w) add_columns(sums + (uint32_t)(w * HALF), sum[w]);
                    }
                    if (done >= depth) {
                        if (live) {
#pragma unroll
                            for (int w = 0; w < W; ++w) set_columns(sums + (uint32_t)(w * HALF), sum[w]);
                        }
                        break;
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster_relaxed(tempty_leader + 8u * (uint32_t)acc);
                    acc ^= 1;
                    if (acc == 0) acc_phase ^= 1u;
                    ok = __all_sync(0xffffffffu, mbar_wait(&tfull[acc], acc_phase, abort_flag));
                    if (!ok) break;
                    tc_fence_after();
                }
                if (!ok) return;
            }
            if (EPI == LINEAR && parts > 1) {
                // (the pair's products are done: its ring is free)
                const uint32_t sums = lanes_at + (uint32_t)(acc * PAIR_N);
                last_acc = acc;
                const int share = PAIR_N / parts;
#pragma unroll 1
                for (int c0 = L::COLS * slice; c0 < L::COLS * (slice + 1); c0 += 32) {
                    if (c0 / share == my_part) continue;
                    float v[32];
                    read_columns(sums + (uint32_t)c0, v);
                    put_part(smem, share, my_part, 32 * q + lane, c0, v);
                }
            } else if (live || EPI == GATED_BWD) {  // (there also to ask for what comes next)
                const uint32_t sums = lanes_at + (uint32_t)(acc * PAIR_N + L::COLS * slice);
                if constexpr (EPI == LINEAR)
                    epi_linear([&](int c, float (&v)[64]) { read_columns(sums + (uint32_t)c, v); }, L::COLS, row0, col0, problem, a,
                               box);
                else if constexpr (EPI == GATED)
                    epi_gated(sums, row0, col0, a, box);
                else {
                    int next_row0 = -1, next_col0 = 0;
                    Walk<JOBS> then = at;
                    then.next();
                    if (then.more()) {
                        locate(a, then.tile, &problem, &mb, &nb);
                        next_row0 = mb * PAIR_M + (int)rank * HALF + 32 * q;
                        next_col0 = nb * TILE_N + L::COLS * slice;
                    }
                    epi_gated_bwd(sums, row0, col0, next_row0, next_col0, a, HalfBox{box.box, lane});
                }
            }
            tc_fence_before();
            __syncwarp();
            // relaxed: it says that tensor memory has been read; a release would wait for the results' stores
            if (lane == 0) mbar_arrive_cluster_relaxed(tempty_leader + 8u * (uint32_t)acc);
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
        };
        for (; ok && at.more(); at.next()) {
            if (JOBS == 1 || at.job == 0)  // (each with its own, so that they need no registers)
                finish(jobs.args[0]);
            else
                finish(jobs.args[JOBS - 1]);
        }
        if (!ok) fail(status, abort_flag);
        if (EPI == GATED_BWD) asm volatile("cp.async.wait_all;" ::: "memory");  // (copies may be left after a wait that ran out)
    }

    if constexpr (EPI == LINEAR && JOBS == 1) {
        if (parts > 1) {
            const Args& a = first;
            __syncwarp();
            tc_fence_before();
            cluster_sync();
            tc_fence_after();
            if (warp >= 2 && !has_error(a.status)) {  // (a wait that ran out has left a part undefined)
                const int q = warp & 3, half = (warp - 2) >> 2;
                int mb, nb, problem;
                locate(a, route.pair, &problem, &mb, &nb);
                const int share = PAIR_N / parts, width = share / 2;  // 64 or 32 columns of a warp
                const int first = my_part * share + half * width;
                const int row0 = mb * PAIR_M + (int)rank * HALF + 32 * q, col0 = nb * PAIR_N + first;
                const uint32_t own = tmem_base + ((uint32_t)(32 * q) << 16) + (uint32_t)(last_acc * PAIR_N + first);
                if (row0 < a.rowsA && col0 < a.rowsB)
                    epi_linear(
                        [&](int c0, float (&v)[64]) {
                            const float* mine = part_row(smem, share, my_part, 32 * q + lane) + (half * width + c0) * HALF;
#pragma unroll
                            for (int c = 0; c < 64; ++c) v[c] = 0.f;
#pragma unroll 1
                            for (int p = 0; p < parts; ++p) {
                                const uint32_t at = cluster_addr(mine, (uint32_t)(2 * p) + rank);
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    if (h * 32 >= width) break;
                                    float w[32];
                                    if (p == my_part) {
                                        read_columns(own + (uint32_t)(c0 + h * 32), w);
                                    } else {
#pragma unroll
                                        for (int c = 0; c < 8; ++c) {
                                            const float4 f = ld_cluster_f4(at + (uint32_t)((h * 32 + c * 4) * HALF * 4));
                                            w[4 * c] = f.x, w[4 * c + 1] = f.y, w[4 * c + 2] = f.z, w[4 * c + 3] = f.w;
                                        }
                                    }
#pragma unroll
                                    for (int c = 0; c < 32; ++c) v[h * 32 + c] += w[c];
                                }
                            }
                        },
                        width, row0, col0, problem, a, box);
            }
        }
    }

    // Neither CTA deallocates or exits while the pair's products, loads or arrivals may still touch the other's
    // tensor or shared memory, or the cluster's CTAs read its part.
    __syncwarp();
    tc_fence_before();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 2 * PAIR_N);
    }
}

// ---------------------------------------------------------------- few rows --
//
// One CTA: 128 rows of W (GATED: 64 of W_gate and the same 64 of W_up) x up to BN tokens x one part of the depth; a
// cluster of `parts` CTAs has the whole depth. Two or three CTAs share an SM: set-up and ends overlap
// with the others' loads.
//   warp 0  loads, warp 1  tensor memory and products, warps 2-5  parts to shared memory; then all threads add the
//   parts of their columns up and form the results.
// An earlier error is only looked at before the results are stored: no CTA may leave its cluster early.

// Lets the stream's next launch start if it waits for this one's end by itself (launch_wait).
__device__ __forceinline__ void launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void launch_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

constexpr int kFewThreads = 192;
constexpr int kFewRows = 128;  // rows of W in a tile

// Shared memory of a CTA: a ring of `stages`, then the barriers.
template <int BN>
struct FewSmem {
    static constexpr int W_BYTES = kFewRows * BK * 2;
    static constexpr int STAGE_BYTES = W_BYTES + BN * BK * 2;
    static constexpr int MOST = 5;  // stages
    static constexpr int total(int stages) { return stages * STAGE_BYTES + (2 * MOST + 5) * 8 + 16 + 1024; }  // + alignment slack
    // Two or three CTAs on an SM (each with 1 KB of the system's)
    static constexpr int TWO = BN <= 32 ? 5 : BN == 64 ? 4 : 3;
    static constexpr int THREE = BN == 16 ? 4 : BN <= 64 ? 3 : 2;
    // Accumulators. Up to 64 tokens: a second one for results in pieces, which the epilogue's threads add up in
    // registers while the next piece is formed; with 128 (too many for registers) the first one keeps the sum, and each
    // later piece is formed in the second and added to it before the next may begin (128 x 50001 x 2048, fp32: 54 us;
    // 70 in two blocks of 64 tokens, which read W twice).
    static constexpr bool DRAINED = BN <= 64;
    static_assert(TWO <= MOST && 2 * (total(TWO) + 1024) <= 228 * 1024 && 3 * (total(THREE) + 1024) <= 228 * 1024, "the SM's");
    static_assert(kFewRows * BN * 4 <= THREE * STAGE_BYTES, "the parts take the ring's place");
};

// Four results of one row: neighbours, in one piece (VEC), or `apart` columns from one another, of which those with
// col + e apart < n exist.
template <bool VEC>
__device__ __forceinline__ void few_store(void* out, bool f32, size_t at, int apart, int left, const float (&v)[4])
{
    if constexpr (VEC) {
        if (f32)
            *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = make_float4(v[0], v[1], v[2], v[3]);
        else
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = make_uint2(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]));
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (e * apart >= left) break;
            if (f32)
                static_cast<float*>(out)[at + e * apart] = v[e];
            else
                static_cast<uint16_t*>(out)[at + e * apart] = f32_to_bf16_bits(v[e]);
        }
    }
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// A CTA's share of its tile's results (`share` columns from `base` on, `tokens` rows), four a thread: neighbours where
// everything lies on 16-byte boundaries, else a quarter of the share apart, so that lanes store neighbours. A thread keeps
// its columns (their number divides the threads). (Four rows at once were slower: 128 x 4096 x 4096 21 us instead of 17.)
template <int EPI, bool VEC>
__device__ __forceinline__ void few_finish(const float* part, int parts, int base, int share, int tokens, int row0, int col0,
                                           const Args& a)
{
    const int per_row = share / 4, apart = VEC ? 1 : per_row, step = kFewThreads / per_row;
    const int c = base + (int)threadIdx.x % per_row * (VEC ? 4 : 1), col = col0 + c, left = a.rowsB - col;
    if (left <= 0) return;
    float bias[4] = {0.f, 0.f, 0.f, 0.f};
    if (a.bias) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (VEC || e * apart < left) bias[e] = a.bias[col + e * apart];
    }
#pragma unroll 1
    for (int t = (int)threadIdx.x / per_row; t < tokens; t += step) {
        const size_t row = (size_t)row0 + t;
        float v[4], u[4] = {0.f, 0.f, 0.f, 0.f}, res[4] = {0.f, 0.f, 0.f, 0.f};
        if (EPI == LINEAR && a.res) {
            const size_t at = row * a.ldres + col;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (VEC || e * apart < left)
                    res[e] = a.out_f32 ? static_cast<const float*>(a.res)[at + e * apart]
                                       : bf16_to_f32(static_cast<const uint16_t*>(a.res)[at + e * apart]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = bias[e];
        const float* from = part + t * kFewRows + c;
        for (int r = 0; r < parts; ++r) {
            const uint32_t addr = parts > 1 ? cluster_addr(from, (uint32_t)r) : smem_u32(from);
            if constexpr (VEC) {
                const float4 f = ld_cluster_f4(addr);
                v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w;
                if constexpr (EPI == GATED) {
                    const float4 w = ld_cluster_f4(addr + (kFewRows / 2) * 4);
                    u[0] += w.x, u[1] += w.y, u[2] += w.z, u[3] += w.w;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] += ld_cluster_f32(addr + (uint32_t)(e * apart * 4));
            }
        }
        if constexpr (EPI == GATED) {
            const size_t at = row * a.ldo + col;
            if (a.g) {
                few_store<true>(a.g, false, at, 1, left, v);
                few_store<true>(a.u, false, at, 1, left, u);
            }
            by_activation(a.act, [&](auto tag) { activate_all<decltype(tag)::value>(v); });
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] *= u[e];
            few_store<true>(a.h, false, at, 1, left, v);
        } else {
            if (a.pre) few_store<VEC>(a.pre, false, row * a.ldpre + col, apart, left, v);
            if (a.act != TWELL_ACT_NONE) by_activation(a.act, [&](auto tag) { activate_all<decltype(tag)::value>(v); });
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += res[e];
            few_store<VEC>(a.out[0], a.out_f32, row * a.ldo + col, apart, left, v);
        }
    }
}

// The whole depth in one CTA (LINEAR): 16 tokens' results of a column, stored by the thread that has them in its
// tensor memory lane. A warp's lanes are neighbouring columns of one row. The residual's values are asked for before
// the sums are ready, or while the 16 tokens before are worked on.
__device__ __forceinline__ void few_residual(float (&r)[16], int tokens, size_t row, int col, const Args& a)
{
#pragma unroll
    for (int c = 0; c < 16; ++c) {
        r[c] = 0.f;
        if (c < tokens)
            r[c] = a.out_f32 ? static_cast<const float*>(a.res)[(row + c) * a.ldres + col]
                             : bf16_to_f32(static_cast<const uint16_t*>(a.res)[(row + c) * a.ldres + col]);
    }
}
__device__ __forceinline__ void few_direct(float (&v)[16], const float (&res)[16], int tokens, size_t row, int col, float bias,
                                           const Args& a)
{
#pragma unroll
    for (int c = 0; c < 16; ++c) v[c] += bias;
    if (a.pre) {
#pragma unroll
        for (int c = 0; c < 16; ++c)
            if (c < tokens) a.pre[(row + c) * a.ldpre + col] = f32_to_bf16_bits(v[c]);
    }
    if (a.act != TWELL_ACT_NONE)
        by_activation(a.act, [&](auto tag) { activate_all<decltype(tag)::value>(v); });
    if (a.res) {
#pragma unroll
        for (int c = 0; c < 16; ++c) v[c] += res[c];
    }
#pragma unroll
    for (int c = 0; c < 16; ++c) {
        if (c >= tokens) break;
        if (a.out_f32)
            static_cast<float*>(a.out[0])[(row + c) * a.ldo + col] = v[c];
        else
            static_cast<uint16_t*>(a.out[0])[(row + c) * a.ldo + col] = f32_to_bf16_bits(v[c]);
    }
}

template <int EPI, int BN, bool W_MN>
__global__ void __launch_bounds__(kFewThreads, 3)
    k_mm_few(const __grid_constant__ Maps maps, const Args a, int parts, int per, int stages, uint32_t tmem_cols)
{
    using L = FewSmem<BN>;
    constexpr uint32_t IDESC = idesc_bf16_f32(kFewRows, BN) | (W_MN ? kIdescAMn : 0u);
    constexpr uint64_t W_KSTEP = W_MN ? (16u * 128u) >> 4 : 2u;
    constexpr int COLS = EPI == GATED ? kFewRows / 2 : kFewRows;  // output columns of a tile
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + stages * L::STAGE_BYTES);
    uint64_t* empty = full + L::MOST;
    uint64_t* done = empty + L::MOST;
    uint64_t* tfull = done + 1;
    uint64_t* tempty = tfull + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 2);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = parts > 1 ? (int)cluster_rank() : 0;
    const int col0 = (int)(blockIdx.x / (unsigned)parts) * COLS, row0 = (int)blockIdx.y * BN;
    const int depth = a.num_kb * a.segments;
    const int kb0 = min(rank * per, depth), kb1 = min(kb0 + per, depth);
    const uint64_t once = l2_policy_evict_first();  // W goes by once
    auto load_w = [&](int kb, int at) {
        const int seg = kb / a.num_kb, x = (kb - seg * a.num_kb) * BK;
        uint8_t* sw = smem + at * L::STAGE_BYTES;
        mbar_arrive_expect_tx(&full[at], L::STAGE_BYTES);
        if constexpr (EPI == GATED) {
            tma_load_2d_hint(sw, &maps.b[0], x, col0, &full[at], once);
            tma_load_2d_hint(sw + L::W_BYTES / 2, &maps.b[1], x, col0, &full[at], once);
        } else if constexpr (W_MN) {
            tma_load_2d_hint(sw, &maps.b[seg], col0, x, &full[at], once);
            tma_load_2d_hint(sw + L::W_BYTES / 2, &maps.b[seg], col0 + kMnBox, x, &full[at], once);
        } else {
            tma_load_2d_hint(sw, &maps.b[seg], x, col0, &full[at], once);
        }
    };
    auto load_x = [&](int kb, int at) {
        const int seg = kb / a.num_kb;
        tma_load_2d(smem + at * L::STAGE_BYTES + L::W_BYTES, &maps.a[seg], (kb - seg * a.num_kb) * BK, row0, &full[at]);
    };
    const int pieces = (kb1 - kb0 + a.piece - 1) / a.piece;
    const bool drain = L::DRAINED && pieces > 1;
    const bool merge = !L::DRAINED && pieces > 2;
    const int ahead = min(kb1 - kb0, stages);  // the ring's first round, which needs no wait
    if (threadIdx.x == 0) {
        *abort_flag = 0;
        for (int s = 0; s < stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(done, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], 4);
        }
        fence_mbar_init();
        // under way before the others are set up; the tokens' rows when the launch before has ended
        for (int i = 0; i < ahead; ++i) load_w(kb0 + i, i);
        if (!a.early)
            for (int i = 0; i < ahead; ++i) load_x(kb0 + i, i);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, tmem_cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    if (EPI == GATED) launch_next();  // (this launch has its tensor memory: the next one's cannot come first)

    if (warp == 0) {
        if (lane == 0) {
            bool ok = true;
            if (a.early) {
                launch_wait();
                for (int i = 0; i < ahead; ++i) load_x(kb0 + i, i);
            }
            int stage = 0;
            uint32_t phase = 0;
            for (int kb = kb0 + ahead; kb < kb1; ++kb) {  // (ahead = stages, or nothing is left)
                if (!mbar_wait(&empty[stage], phase, abort_flag)) {
                    ok = false;
                    break;
                }
                load_w(kb, stage);
                load_x(kb, stage);
                if (++stage == stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!ok) fail(a.status, abort_flag);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            bool ok = true;
            int stage = 0;
            uint32_t phase = 0;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!mbar_wait(&full[stage], phase, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int i = kb - kb0, piece = i / a.piece, in_piece = i - piece * a.piece;
                const int acc = drain ? piece & 1 : min(piece, 1);
                if (drain && in_piece == 0 && piece >= 2) {  // its last sums have been read
                    if (!mbar_wait(&tempty[acc], (uint32_t)((piece >> 1) & 1) ^ 1u, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                }
                if (merge && in_piece == 0 && piece >= 2) {  // the piece before has been added to the sum
                    if (!mbar_wait(&tempty[1], (uint32_t)piece & 1u, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                }
                const uint32_t d_tmem = tmem_base + (uint32_t)(acc * BN);
                const uint32_t sw = smem_u32(smem + stage * L::STAGE_BYTES);
                const uint64_t wdesc = operand_desc(W_MN, sw);
                const uint64_t xdesc = sw128_kmajor_desc(sw + L::W_BYTES);
#pragma unroll
                for (int k = 0; k < BK / 16; ++k)
                    umma_bf16(d_tmem, wdesc + W_KSTEP * k, xdesc + 2u * k, IDESC, (in_piece | k) != 0);
                umma_commit(&empty[stage]);
                if (drain && (in_piece == a.piece - 1 || kb == kb1 - 1)) umma_commit(&tfull[acc]);
                if (merge && in_piece == a.piece - 1 && piece > 0 && piece < pieces - 1) umma_commit(&tfull[1]);
                if (++stage == stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!ok) fail(a.status, abort_flag);
            umma_commit(done);
        }
    }
    const uint32_t lanes_at = tmem_base + ((uint32_t)(32 * (warp & 3)) << 16);
    float sum[L::DRAINED ? BN : 1];
    if constexpr (L::DRAINED) {
        if (warp >= 2 && drain) {
#pragma unroll
            for (int c = 0; c < BN; ++c) sum[c] = 0.f;
            for (int p = 0; p < pieces; ++p) {
                if (!__all_sync(0xffffffffu, mbar_wait(&tfull[p & 1], (uint32_t)(p >> 1) & 1u, abort_flag))) break;
                tc_fence_after();
#pragma unroll
                for (int c0 = 0; c0 < BN; c0 += 16) {
                    uint32_t v[16];
                    tmem_ld16_wait(lanes_at + (uint32_t)((p & 1) * BN + c0), v);
#pragma unroll
                    for (int c = 0; c < 16; ++c) sum[c0 + c] += __uint_as_float(v[c]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&tempty[p & 1]);
            }
        }
    } else if (warp >= 2 && merge) {
        for (int p = 1; p < pieces - 1; ++p) {  // (the last one is added below)
            if (!__all_sync(0xffffffffu, mbar_wait(&tfull[1], (uint32_t)(p - 1) & 1u, abort_flag))) break;
            tc_fence_after();
#pragma unroll 1
            for (int c0 = 0; c0 < BN; c0 += 32) {
                uint32_t v[32], w[32];
                tmem_ld32_wait(lanes_at + (uint32_t)c0, v);
                tmem_ld32_wait(lanes_at + (uint32_t)(BN + c0), w);
#pragma unroll
                for (int c = 0; c < 32; ++c) v[c] = __float_as_uint(__uint_as_float(v[c]) + __uint_as_float(w[c]));
                tmem_st32(lanes_at + (uint32_t)c0, v);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[1]);
        }
    }
    __syncwarp();
    if (a.early) launch_wait();  // nothing of the launch before is read, and nothing written, ahead of this
    // Every load has landed when the products that read it are done, so the ring is free from here on. (Loads in
    // flight after a wait that ran out still land in it: the results are not used then, but the CTA must not end.)
    bool ok = mbar_wait(done, 0, nullptr);
    if (!ok) fail(a.status, abort_flag);
    if (__syncthreads_or(*abort_flag)) {
        if (threadIdx.x == 0)
            for (int s = 0; s < stages; ++s) {
                mbar_wait(&full[s], 0, nullptr);
                mbar_wait(&full[s], 1, nullptr);
            }
        __syncthreads();
    }
    tc_fence_after();
    float* part = reinterpret_cast<float*>(smem);  // [token][kFewRows]
    const bool direct = EPI == LINEAR && parts == 1;
    const int tokens = min(BN, a.rowsA - row0);
    if (warp >= 2) {
        const int row = 32 * (warp & 3) + lane, col = col0 + row;
        const bool failed = direct && has_error(a.status);
        const float bias = direct && a.bias && col < a.rowsB ? a.bias[col] : 0.f;
        const bool with_res = direct && a.res && col < a.rowsB;
        float res[16];
        if (with_res) few_residual(res, tokens, (size_t)row0, col, a);
        auto put16 = [&](int c0, float (&v)[16]) {
            if (direct) {
                float now[16];
#pragma unroll
                for (int c = 0; c < 16; ++c) now[c] = res[c];
                if (with_res && c0 + 16 < tokens) few_residual(res, tokens - c0 - 16, (size_t)row0 + c0 + 16, col, a);
                if (col < a.rowsB && !failed) few_direct(v, now, tokens - c0, (size_t)row0 + c0, col, bias, a);
            } else {
#pragma unroll
                for (int c = 0; c < 16; ++c) part[(c0 + c) * kFewRows + row] = v[c];
            }
        };
        if (drain) {
            if constexpr (L::DRAINED) {
#pragma unroll
                for (int c0 = 0; c0 < BN; c0 += 16) {
                    if (c0 >= tokens) break;
                    float v[16];
#pragma unroll
                    for (int c = 0; c < 16; ++c) v[c] = sum[c0 + c];
                    put16(c0, v);
                }
            }
        } else {
#pragma unroll 1
            for (int c0 = 0; c0 < tokens; c0 += 16) {
                float v[16];
#pragma unroll
                for (int c = 0; c < 16; ++c) v[c] = 0.f;
                for (int p = 0; p < min(pieces, 2); ++p) {
                    uint32_t w[16];
                    tmem_ld16_wait(lanes_at + (uint32_t)(p * BN + c0), w);
#pragma unroll
                    for (int c = 0; c < 16; ++c) v[c] += __uint_as_float(w[c]);
                }
                put16(c0, v);
            }
        }
        tc_fence_before();
    }
    __syncwarp();
    if (parts > 1)
        cluster_sync();
    else
        __syncthreads();

    // this CTA's share of the tile's columns; parts in the cluster's order
    const int share = COLS / parts;
    const int base = rank * share;
    if (!direct && !has_error(a.status)) {
        if (EPI == GATED || (a.vec & VEC_OUT && (!a.pre || a.vec & VEC_PRE)))
            few_finish<EPI, true>(part, parts, base, share, tokens, row0, col0, a);
        else
            few_finish<EPI, false>(part, parts, base, share, tokens, row0, col0, a);
    }
    __syncwarp();
    // no CTA ends while another may still read its part
    if (parts > 1)
        cluster_sync();
    else
        __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, tmem_cols);
    }
}

// ------------------------------------------------------------- one to four tokens --
//
// Products of W's rows (K-major) with up to four tokens' rows, on the fp32 units: bound by memory like the kernel above, but
// nothing has to be set up, and nothing joined. A warp (SPLIT of them where there are few rows) has a row of W, GATED the
// same row of both; x comes from the first-level cache, past which W goes.
constexpr int kMvThreads = 256, kMvWarps = kMvThreads / 32;

__device__ __forceinline__ uint4 ld_once(const uint16_t* p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

struct MvArgs {
    const uint16_t *x, *w0, *w1;  // w1: GATED's W_up
    int64_t ldx, ldw;
    int K, tokens;
};

template <int TOK>
__device__ __forceinline__ void mv_piece(const uint4& w, const MvArgs& m, int piece, float (&sum)[TOK])
{
    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int t = 0; t < TOK; ++t) {
        if (TOK == 4 && t == 3 && m.tokens < 4) break;
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(m.x + t * m.ldx) + piece);
        const uint32_t xx[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            sum[t] = fmaf(bf16_lo(ww[e]), bf16_lo(xx[e]), sum[t]);
            sum[t] = fmaf(bf16_hi(ww[e]), bf16_hi(xx[e]), sum[t]);
        }
    }
}

// The tokens' results of output column n, one in each of the first TOK lanes.
template <int EPI>
__device__ __forceinline__ void mv_finish(float v, float u, int n, int t, const Args& a)
{
    const size_t row = (size_t)t;
    if (a.bias) v += a.bias[n];
    float y[2] = {v, 0.f};
    if constexpr (EPI == GATED) {
        if (a.g) {
            a.g[row * a.ldo + n] = f32_to_bf16_bits(v);
            a.u[row * a.ldo + n] = f32_to_bf16_bits(u);
        }
        by_activation(a.act, [&](auto tag) { activate_all<decltype(tag)::value>(y); });
        a.h[row * a.ldo + n] = f32_to_bf16_bits(y[0] * u);
    } else {
        if (a.pre) a.pre[row * a.ldpre + n] = f32_to_bf16_bits(v);
        if (a.act != TWELL_ACT_NONE) by_activation(a.act, [&](auto tag) { activate_all<decltype(tag)::value>(y); });
        if (a.res)
            y[0] += a.out_f32 ? static_cast<const float*>(a.res)[row * a.ldres + n]
                              : bf16_to_f32(static_cast<const uint16_t*>(a.res)[row * a.ldres + n]);
        if (a.out_f32)
            static_cast<float*>(a.out[0])[row * a.ldo + n] = y[0];
        else
            static_cast<uint16_t*>(a.out[0])[row * a.ldo + n] = f32_to_bf16_bits(y[0]);
    }
}

template <int EPI, int TOK, int SPLIT>
__global__ void __launch_bounds__(kMvThreads) k_mv(const MvArgs m, const Args a)
{
    constexpr int W = EPI == GATED ? 2 : 1;
    constexpr int AT_ONCE = 8 / W;  // pieces of a row under way in a lane
    __shared__ float shared[W * TOK][kMvWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n = (int)blockIdx.x * (kMvWarps / SPLIT) + warp / SPLIT;
    if (EPI == GATED) launch_next();
    float sum[W][TOK];
#pragma unroll
    for (int i = 0; i < W; ++i)
#pragma unroll
        for (int t = 0; t < TOK; ++t) sum[i][t] = 0.f;
    if (n < a.rowsB) {
        const int pieces = m.K / 8;
        const uint16_t* w0 = m.w0 + (size_t)n * m.ldw;
        const uint16_t* w1 = EPI == GATED ? m.w1 + (size_t)n * m.ldw : nullptr;
        for (int p = warp % SPLIT * 32 + lane; p < pieces; p += AT_ONCE * 32 * SPLIT) {
            uint4 q[W][AT_ONCE];
#pragma unroll
            for (int j = 0; j < AT_ONCE; ++j) {
                const int at = p + j * 32 * SPLIT;
                if (at < pieces) {
                    q[0][j] = ld_once(w0 + (size_t)at * 8);
                    if constexpr (EPI == GATED) q[1][j] = ld_once(w1 + (size_t)at * 8);
                }
            }
#pragma unroll
            for (int j = 0; j < AT_ONCE; ++j) {
                const int at = p + j * 32 * SPLIT;
                if (at < pieces) {
#pragma unroll
                    for (int i = 0; i < W; ++i) mv_piece<TOK>(q[i][j], m, at, sum[i]);
                }
            }
        }
    }
    float v = 0.f, u = 0.f;  // lane t: token t's
#pragma unroll
    for (int i = 0; i < W; ++i)
#pragma unroll
        for (int t = 0; t < TOK; ++t) {
            float s = sum[i][t];
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
            if (SPLIT > 1) {
                if (lane == 0) shared[i * TOK + t][warp] = s;
            } else if (lane == t) {
                (i ? u : v) = s;
            }
        }
    if constexpr (SPLIT > 1) {
        __syncthreads();
        if (warp % SPLIT != 0) return;
        if (lane < TOK) {
#pragma unroll
            for (int k = 0; k < SPLIT; ++k) {
                v += shared[lane][warp + k];
                if (EPI == GATED) u += shared[(W - 1) * TOK + lane][warp + k];
            }
        }
    }
    if (lane < TOK && lane < a.rowsA && n < a.rowsB && !has_error(a.status)) mv_finish<EPI>(v, u, n, lane, a);
}

__global__ void __launch_bounds__(512) k_block_sums(const float* __restrict__ part, int blocks, int n,
                                                    float* __restrict__ db, const int32_t* __restrict__ status)
{
    __shared__ float sum[16][33];
    if (has_error(status)) return;
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), run = threadIdx.x >> 5;
    float s = 0.f;
    if (c < n) {
#pragma unroll 4
        for (int b = run; b < blocks; b += 16) s += part[(size_t)b * n + c];
    }
    sum[run][threadIdx.x & 31] = s;
    __syncthreads();
    if (run == 0 && c < n) {
#pragma unroll
        for (int i = 1; i < 16; ++i) s += sum[i][threadIdx.x];
        db[c] = s;
    }
}

// ---------------------------------------------------------------- launches --

bool map_of(CUtensorMap* m, const MmOperand& o, int rows, int K, int box_rows)
{
    return o.mn ? make_map_mn(m, o.p, rows, K, (int)o.ld) : make_map(m, o.p, rows, K, box_rows, (int)o.ld);
}

// What a tile of 256 x 256 takes a pair among others, in us: 0.3 a k-block, and 1 between tiles. (Depths of 64 to 14336;
// rows that do not lie on 128-byte boundaries: 0.41 a k-block.)
float tile_us(const Args& a, bool rows128)
{
    return 1.f + (rows128 ? 0.3f : 0.41f) * (float)a.num_kb * (float)a.segments;
}

// How two jobs' tiles share the pairs.
struct Split {
    int delay;   // rounds of the second's tiles for the pairs without a last tile of the first
    float most;  // of the pair with the most
    Split(const Args& one, const Args& two, float us1, float us2, int pairs)
    {
        auto tiles = [](const Args& a) {
            return ((int64_t)a.rowsA + PAIR_M - 1) / PAIR_M * (((int64_t)a.rowsB + PAIR_N - 1) / PAIR_N) * a.problems;
        };
        const int64_t t1 = tiles(one), t2 = tiles(two), busy = t1 % pairs, free = pairs - busy;
        const int64_t enough = (t2 + free - 1) / free;
        const float about = us1 / us2 + 0.5f;
        const int64_t rounds = about < 1.f ? 1 : about > (float)enough ? enough : (int64_t)about;
        delay = (int)rounds;
        const int64_t later = t2 > rounds * free ? (t2 - rounds * free + pairs - 1) / pairs : 0;
        const float with = (float)(t1 / pairs + (busy > 0)) * us1 + (float)later * us2;
        const float without = (float)(t1 / pairs) * us1 + (float)(rounds + later) * us2;
        most = with > without ? with : without;
    }
};

// Clusters of 2, 4 and 8 CTAs of a kernel of pairs that can be resident at once on the current device (0: none, or not
// needed), as the driver says.
struct AtOnce {
    int n[3];
};
template <int EPI, bool A_MN, bool B_MN, int JOBS>
cudaError_t clusters_at_once(AtOnce* out)
{
    // (one word for a device, so that threads whose first calls meet see all three numbers or none)
    static std::atomic<uint64_t> known[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    uint64_t all = known[dev].load(std::memory_order_relaxed);
    if (all == 0) {
        auto kern = k_mm_pair<EPI, A_MN, B_MN, JOBS>;
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<EPI>::TOTAL);
        if (e != cudaSuccess) return e;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.blockDim = dim3(Smem<EPI>::THREADS, 1, 1);
        cfg.dynamicSmemBytes = Smem<EPI>::TOTAL;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        for (int i = 0; i < 3; ++i) {
            if (i > 0 && (EPI != LINEAR || JOBS > 1)) continue;
            int n = 0;
            attr[0].val.clusterDim.x = 2u << i;
            cfg.gridDim = dim3(2u << i, 1, 1);
            e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
            if (e != cudaSuccess && i == 0) return e;
            if (e != cudaSuccess) (void)cudaGetLastError();
            if (n <= 0 && i == 0) return cudaErrorNotSupported;
            if (e == cudaSuccess) all |= (uint64_t)(n & 0xffff) << (16 * i);
        }
        known[dev].store(all, std::memory_order_relaxed);
    }
    for (int i = 0; i < 3; ++i) out->n[i] = (int)(all >> (16 * i) & 0xffff);
    return cudaSuccess;
}

// Parts of a tile's depth: where there are few tiles, as many as run at once, if none is shorter than 12 k-blocks (joining
// takes about 2.5 us for each part more, as long as 9 k-blocks); so no part is empty.
int parts_of(int64_t tiles, int depth, const AtOnce& at_once)
{
    int parts = 1;
    for (int i = 1; i <= 2; ++i)
        if (tiles <= at_once.n[i] && depth >= (12 << i)) parts = 1 << i;
    return parts;
}

// whole: a tile's depth in one part, however few tiles there are.
template <int EPI, bool A_MN, bool B_MN, int JOBS>
cudaError_t run_jobs(Jobs<JOBS>& jobs, bool whole, cudaStream_t s)
{
    auto kern = k_mm_pair<EPI, A_MN, B_MN, JOBS>;
    AtOnce at_once;
    cudaError_t e = clusters_at_once<EPI, A_MN, B_MN, JOBS>(&at_once);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<EPI>::TOTAL);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(Smem<EPI>::THREADS, 1, 1);
    cfg.dynamicSmemBytes = Smem<EPI>::TOTAL;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    constexpr int TILE_N = EPI == GATED ? HALF : PAIR_N;
    int64_t tiles = 0;
    for (const Args& a : jobs.args)
        tiles += ((int64_t)a.rowsA + PAIR_M - 1) / PAIR_M * (((int64_t)a.rowsB + TILE_N - 1) / TILE_N) * a.problems;
    if (tiles > INT32_MAX / 2) return cudaErrorInvalidValue;
    const int depth = jobs.args[0].num_kb * jobs.args[0].segments;
    const int parts = EPI == LINEAR && JOBS == 1 && !whole ? parts_of(tiles, depth, at_once) : 1;
    const int per = (depth + parts - 1) / parts;
    const int clusters = (int)(parts > 1 || tiles < at_once.n[0] ? tiles : at_once.n[0]);
    if constexpr (JOBS > 1) jobs.delay = Split(jobs.args[0], jobs.args[1], jobs.us[0], jobs.us[1], clusters).delay;
    attr[0].val.clusterDim.x = 2u * (unsigned)parts;
    cfg.gridDim = dim3(2u * (unsigned)parts * (unsigned)clusters, 1, 1);
    count_launches(1);
    return cudaLaunchKernelEx(&cfg, kern, jobs, parts, per);
}

template <int EPI, bool A_MN, bool B_MN>
cudaError_t run_pair(const Maps& maps, const Args& a, cudaStream_t s, bool whole = false)
{
    Jobs<1> jobs{{maps}, {a}, 0, {0.f}};
    return run_jobs<EPI, A_MN, B_MN, 1>(jobs, whole, s);
}

cudaError_t run_linear(const MmLinear& m, const Maps& maps, const Args& a, cudaStream_t s, bool whole)
{
    const bool amn = m.a[0].mn, bmn = m.b[0].mn;
    if (amn && bmn) return run_pair<LINEAR, true, true>(maps, a, s, whole);
    if (amn) return cudaErrorInvalidValue;
    if (bmn) return run_pair<LINEAR, false, true>(maps, a, s, whole);
    return run_pair<LINEAR, false, false>(maps, a, s, whole);
}

// Few rows: up to this many always, up to kFewTry where an estimate says so.
constexpr int kFewMost = 128, kFewTry = 1024;

// How k_mm_few would work on `rows` rows and `tiles` tiles of output columns.
struct FewPlan {
    int tokens, blocks, parts, per;  // of a tile, blocks of them, parts of the depth, k-blocks of one
    float us;                        // about
};

FewPlan few_plan(int rows, int64_t tiles, int depth, int sms)
{
    FewPlan p{};
    p.tokens = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
    p.blocks = (rows + p.tokens - 1) / p.tokens;
    // parts of the depth: as few as keep about one CTA on each SM, and none shorter than four k-blocks
    p.parts = 1;
    while (p.parts < 8 && tiles * p.blocks * p.parts < sms && depth / (2 * p.parts) >= 4) p.parts *= 2;
    p.per = (depth + p.parts - 1) / p.parts;
    const float ctas = (float)(tiles * p.blocks * p.parts), slots = 2.f * (float)sms;
    const float at_once = ctas < slots ? ctas : slots;
    // a k-block takes 0.2 us by itself, 0.55 where two CTAs share each SM (256 to 512 rows x 128 to 4096 x 512 to 14336)
    const float each = 0.0018f * at_once;
    p.us = 9.5f + ceilf(ctas / slots) * (float)p.per * (each > 0.2f ? each : 0.2f);
    return p;
}

// The same of the CTA pairs' kernel, whose parts are 2.5 us each (parts_of).
float pair_us(int64_t rows, int64_t cols, int problems, int depth, bool rows128, const AtOnce& at_once)
{
    const int64_t tiles = (rows + PAIR_M - 1) / PAIR_M * ((cols + PAIR_N - 1) / PAIR_N) * problems, pairs = at_once.n[0];
    const int parts = parts_of(tiles, depth, at_once);
    const float waves = parts > 1 ? 1.f : (float)((tiles + pairs - 1) / pairs);
    Args a{};
    a.num_kb = (depth + parts - 1) / parts;
    a.segments = 1;
    return 6.6f + (parts == 4 ? 5.f : parts == 2 ? 2.5f : 0.f) + waves * tile_us(a, rows128);
}

// Whether k_mv takes `tokens` rows and `weights` weights: one token always (4096 x 4096 8.7 us, k_mm_few 11.4; 256 x 8192 3.2,
// 12.1; 50001 x 2048 32.8, 34.5). x's rows are read from the cache as often as W's, so more of them count: two tokens as long
// as that is hidden (4096 x 4096 10.3, 11.5; 16384 x 4096 26.6, 26.5; 50001 x 2048 36.1, 34.8), three or four where W is small
// (256 x 8192 4.0, 12.1; 1024 x 1024 4.2, 6.7; 4096 x 4096 17.9, 11.5).
bool mv_takes(int tokens, int64_t weights)
{
    return tokens == 1 || (tokens == 2 && weights <= 1 << 26) || (tokens <= 4 && weights <= 1 << 22);
}

template <int EPI, int TOK>
cudaError_t run_mv_tokens(const MvArgs& m, const Args& a, int sms, cudaStream_t s)
{
    // as many warps on a row as give every SM about 24
    int split = 1;
    while (split < 8 && (int64_t)a.rowsB * split < (int64_t)sms * 24 && m.K >= 512 * split) split *= 2;
    const int rows = kMvWarps / split;
    const unsigned blocks = (unsigned)(((int64_t)a.rowsB + rows - 1) / rows);
    count_launches(1);
    switch (split) {
        case 1: k_mv<EPI, TOK, 1><<<blocks, kMvThreads, 0, s>>>(m, a); break;
        case 2: k_mv<EPI, TOK, 2><<<blocks, kMvThreads, 0, s>>>(m, a); break;
        case 4: k_mv<EPI, TOK, 4><<<blocks, kMvThreads, 0, s>>>(m, a); break;
        default: k_mv<EPI, TOK, 8><<<blocks, kMvThreads, 0, s>>>(m, a); break;
    }
    return cudaGetLastError();
}

template <int EPI>
cudaError_t run_mv(const MvArgs& m, const Args& a, int sms, cudaStream_t s)
{
    switch (a.rowsA) {
        case 1: return run_mv_tokens<EPI, 1>(m, a, sms, s);
        case 2: return run_mv_tokens<EPI, 2>(m, a, sms, s);
        default: return run_mv_tokens<EPI, 4>(m, a, sms, s);
    }
}

// Length of the pieces of `depth` k-blocks: as few as the results' type allows, as even as they can be.
int piece_of(int depth, bool f32)
{
    const int most = f32 ? kPieceBlocks : kPieceBlocksBf16;
    const int pieces = (depth + most - 1) / most;
    return (depth + pieces - 1) / pieces;
}

template <int EPI, int BN, bool W_MN>
cudaError_t run_few(const Maps& maps, Args a, const FewPlan& plan, int sms, cudaStream_t s)
{
    using L = FewSmem<BN>;
    auto kern = k_mm_few<EPI, BN, W_MN>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::total(L::MOST));
    if (e != cudaSuccess) return e;
    constexpr int COLS = EPI == GATED ? kFewRows / 2 : kFewRows;
    const int64_t tiles = ((int64_t)a.rowsB + COLS - 1) / COLS;
    const int blocks = plan.blocks, parts = plan.parts, per = plan.per;
    if (tiles * parts > INT32_MAX) return cudaErrorInvalidValue;
    a.piece = a.out_f32 ? kFewPieceBlocks : piece_of(per, false);
    const int held = per > a.piece ? 2 : 1;  // accumulators
    uint32_t cols = 32;
    while (cols < (uint32_t)(held * BN)) cols *= 2;
    // More CTAs than two on each SM: a third one there, with shorter rings, if tensor memory has room. (64 rows x 50000 x
    // 2048: 46 us with two, 38.5 with three; the gated layer's 224 tiles of 4096 x 14336 58 us with long rings, 61.)
    const bool three = tiles * parts * blocks > 2 * sms && 3 * cols <= 512;
    const int stages = three ? L::THREE : L::TWO;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)parts;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * parts), (unsigned)blocks, 1);
    cfg.blockDim = dim3(kFewThreads, 1, 1);
    cfg.dynamicSmemBytes = (size_t)L::total(stages);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = a.early ? 2 : 1;
    count_launches(1);
    return cudaLaunchKernelEx(&cfg, kern, maps, a, parts, per, stages, cols);
}

template <int EPI, bool W_MN>
cudaError_t run_few_rows(const Maps& maps, const Args& a, const FewPlan& plan, int sms, cudaStream_t s)
{
    switch (plan.tokens) {
        case 16: return run_few<EPI, 16, W_MN>(maps, a, plan, sms, s);
        case 32: return run_few<EPI, 32, W_MN>(maps, a, plan, sms, s);
        case 64: return run_few<EPI, 64, W_MN>(maps, a, plan, sms, s);
        default: return run_few<EPI, 128, W_MN>(maps, a, plan, sms, s);
    }
}

bool pieces_of_16(const void* p, int64_t ld, int n, int es)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld * es % 16 == 0 && (int64_t)n * es % 16 == 0;
}

}  // namespace

namespace {

// What a launch of m needs, with boxes of `box` rows of A (few rows: the tokens of a tile).
bool fill(const MmLinear& m, int box, Maps* maps, Args* args)
{
    const int n = m.segments * m.problems;
    for (int i = 0; i < n; ++i)
        if (!map_of(&maps->a[i], m.a[i], m.M, m.K, box) || !map_of(&maps->b[i], m.b[i], m.N, m.K, HALF)) return false;
    for (int i = n; i < kMmParts; ++i) maps->a[i] = maps->a[0], maps->b[i] = maps->b[0];
    Args& a = *args;
    a = Args{};
    a.rowsA = m.M;
    a.rowsB = m.N;
    a.num_kb = (m.K + BK - 1) / BK;
    a.segments = m.segments;
    a.problems = m.problems;
    a.piece = piece_of(a.num_kb * m.segments, m.out_f32);
    a.bias = m.bias;
    a.act = m.act;
    a.res = m.res;
    a.ldres = m.ldres;
    a.pre = m.pre;
    a.ldpre = m.ldpre;
    for (int i = 0; i < m.problems; ++i) a.out[i] = m.out[i];
    a.ldo = m.ldo;
    a.out_f32 = m.out_f32;
    a.accumulate = m.accumulate;
    const int es = m.out_f32 ? 4 : 2;
    bool out_vec = true;
    for (int i = 0; i < m.problems; ++i) out_vec = out_vec && pieces_of_16(m.out[i], m.ldo, m.N, es);
    a.vec = (out_vec ? VEC_OUT : 0) | (m.res && pieces_of_16(m.res, m.ldres, m.N, es) ? VEC_RES : 0) |
            (m.pre && pieces_of_16(m.pre, m.ldpre, m.N, 2) ? VEC_PRE : 0);
    a.status = m.status;
    return true;
}

// Whether all operands' rows lie on 128-byte boundaries.
bool rows128(const MmLinear& m)
{
    for (int i = 0; i < m.segments * m.problems; ++i)
        if (m.a[i].ld % 64 != 0 || m.b[i].ld % 64 != 0) return false;
    return true;
}

// The kernel for m, and about its time.
struct Choice {
    FewPlan plan;
    bool few;
    float us;
    Choice(const MmLinear& m, int sms, const AtOnce& at_once)
    {
        const int depth = (m.K + BK - 1) / BK * m.segments;
        plan = few_plan(m.M, ((int64_t)m.N + kFewRows - 1) / kFewRows, depth, sms);
        us = pair_us(m.M, m.N, m.problems, depth, rows128(m), at_once);
        few = m.problems == 1 && !m.accumulate && !m.a[0].mn && (m.M <= kFewMost || (m.M <= kFewTry && plan.us < us));
        if (few) us = plan.us;
    }
};

}  // namespace

cudaError_t launch_mm_linear(const MmLinear& m, int sms, cudaStream_t s)
{
    AtOnce at_once;
    const cudaError_t e = clusters_at_once<LINEAR, false, false, 1>(&at_once);
    if (e != cudaSuccess) return e;
    const Choice choice(m, sms, at_once);
    const bool few = choice.few;
    Maps maps;
    Args a;
    if (!fill(m, few ? choice.plan.tokens : HALF, &maps, &a)) return cudaErrorInvalidValue;
    a.early = few && m.M <= kFewMost && m.after_gated;  // (then that launch lets this one start)
    const bool bmn = m.b[0].mn;
    if (few && !bmn && m.segments == 1 && mv_takes(m.M, (int64_t)m.N * m.K))
        return run_mv<LINEAR>(MvArgs{m.a[0].p, m.b[0].p, nullptr, m.a[0].ld, m.b[0].ld, m.K, m.M}, a, sms, s);
    if (few)
        return bmn ? run_few_rows<LINEAR, true>(maps, a, choice.plan, sms, s)
                   : run_few_rows<LINEAR, false>(maps, a, choice.plan, sms, s);
    return run_linear(m, maps, a, s, false);
}

cudaError_t launch_mm_two(const MmLinear& one, const MmLinear& two, bool with_one, bool with_two, int sms, cudaStream_t s)
{
    if (one.a[0].mn || !two.a[0].mn || !two.b[0].mn || one.status != two.status) return cudaErrorInvalidValue;
    AtOnce at_once;
    cudaError_t e = clusters_at_once<LINEAR, false, false, 1>(&at_once);
    if (e != cudaSuccess) return e;
    Args args[2];
    for (int i = 0; i < 2; ++i) {
        const MmLinear& m = i ? two : one;
        args[i].rowsA = m.M, args[i].rowsB = m.N, args[i].problems = m.problems, args[i].segments = m.segments;
        args[i].num_kb = (m.K + BK - 1) / BK;
    }
    const float us[2] = {tile_us(args[0], rows128(one)), tile_us(args[1], rows128(two))};
    const Split split(args[0], args[1], us[0], us[1], at_once.n[0]);
    // (tiles that run far apart in depth read more from memory, so that a gain of 2 to 4 % by this estimate was a loss of 1
    // to 3, 8192 x 4096 x 14336 and -> 16384; one of 8 % was a gain of 1.5, 2048 x 4096 x 14336)
    const bool together = 6.6f + split.most < 0.95f * (Choice(one, sms, at_once).us + Choice(two, sms, at_once).us);
    if (together && with_one && with_two) {
        Jobs<2> jobs;
        if (!fill(one, HALF, &jobs.maps[0], &jobs.args[0]) || !fill(two, HALF, &jobs.maps[1], &jobs.args[1])) return cudaErrorInvalidValue;
        for (int i = 0; i < 2; ++i) jobs.us[i] = us[i];
        return one.b[0].mn ? run_jobs<LINEAR, false, true, 2>(jobs, true, s) : run_jobs<LINEAR, false, false, 2>(jobs, true, s);
    }
    for (int i = 0; i < 2 && e == cudaSuccess; ++i) {
        if (!(i ? with_two : with_one)) continue;
        const MmLinear& m = i ? two : one;
        if (!together) {
            e = launch_mm_linear(m, sms, s);
            continue;
        }
        Maps maps;
        Args a;
        e = fill(m, HALF, &maps, &a) ? run_linear(m, maps, a, s, true) : cudaErrorInvalidValue;
    }
    return e;
}

cudaError_t launch_mm_gated(const MmGated& m, int sms, cudaStream_t s)
{
    Maps maps;
    const bool few = m.M <= kFewMost;
    const FewPlan plan = few_plan(m.M, ((int64_t)m.F + kFewRows / 2 - 1) / (kFewRows / 2), (m.K + BK - 1) / BK, sms);
    const int w_rows = few ? kFewRows / 2 : HALF;
    if (!make_map(&maps.a[0], m.x, m.M, m.K, few ? plan.tokens : HALF) || !make_map(&maps.b[0], m.Wg, m.F, m.K, w_rows) ||
        !make_map(&maps.b[1], m.Wu, m.F, m.K, w_rows))
        return cudaErrorInvalidValue;
    maps.a[1] = maps.a[2] = maps.a[0];
    maps.b[2] = maps.b[0];
    Args a{};
    a.rowsA = m.M;
    a.rowsB = m.F;
    a.num_kb = (m.K + BK - 1) / BK;
    a.segments = a.problems = 1;
    a.piece = piece_of(a.num_kb, false);
    a.bias = m.bias;
    a.act = m.act;
    a.g = m.g;
    a.u = m.u;
    a.h = m.h;
    a.ldo = m.F;
    a.status = m.status;
    if (mv_takes(m.M, 2ll * m.F * m.K)) return run_mv<GATED>(MvArgs{m.x, m.Wg, m.Wu, m.K, m.K, m.K, m.M}, a, sms, s);
    if (few) return run_few_rows<GATED, false>(maps, a, plan, sms, s);
    return run_pair<GATED, false, false>(maps, a, s);
}

cudaError_t launch_mm_gated_bwd(const MmGatedBwd& m, int sms, cudaStream_t s)
{
    (void)sms;
    Maps maps;
    if (!make_map(&maps.a[0], m.dy, m.M, m.K, HALF) || !make_map(&maps.b[0], m.Wd, m.F, m.K, HALF))
        return cudaErrorInvalidValue;
    maps.a[1] = maps.a[2] = maps.a[0];
    maps.b[1] = maps.b[2] = maps.b[0];
    Args a{};
    a.rowsA = m.M;
    a.rowsB = m.F;
    a.num_kb = (m.K + BK - 1) / BK;
    a.segments = a.problems = 1;
    a.piece = piece_of(a.num_kb, true);  // without db too: dx and the weight gradients have the same bits
    a.act = m.act;
    a.l1 = m.l1;
    a.g_in = m.g;
    a.u_in = m.u;
    a.g = m.dg;
    a.u = m.du;
    a.part = m.part;
    a.ldo = m.F;
    a.status = m.status;
    return run_pair<GATED_BWD, false, false>(maps, a, s);
}

cudaError_t launch_block_sums(const float* part, int blocks, int n, float* db, const int32_t* status, cudaStream_t s)
{
    count_launches(1);
    k_block_sums<<<(unsigned)((n + 31) / 32), 512, 0, s>>>(part, blocks, n, db, status);
    return cudaGetLastError();
}

}  // namespace twell
