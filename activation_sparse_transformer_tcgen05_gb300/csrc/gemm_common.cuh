// gemm_common.cuh — what the tcgen05 GEMM kernels share: tile sizes and order of
// the CTA-pair kernels, operand descriptors, and the tensor maps (host).
#pragma once

#include "common.cuh"

namespace twell {

constexpr int BK = 64;        // one 128-byte swizzle row of bf16
constexpr int PAIR_M = 256;   // tile rows over the pair
constexpr int PAIR_N = 256;   // tile columns (B rows over the pair)
constexpr int HALF = 128;     // rows of A and of B held by one CTA

// Tile order of the CTA-pair kernel: groups of kRasterN consecutive column
// tiles; inside a group the column tile varies fastest. The ~76 pairs at work
// at any time then cover about 5 row tiles x 16 column tiles, whose A rows and
// B rows (~42 MB at K = 4096) stay in L2, so A is read from DRAM once per
// group instead of once per column tile. At 16384 x 16384 x 4096: 16 column
// tiles per group 1.6-2 % faster than 8, 32 slower (its group's rows no
// longer stay in L2), 4 slower still.
constexpr int kRasterN = 16;

__device__ __forceinline__ void pair_tile_coords(int tile, int num_m, int num_n, int* mb, int* nb)
{
    const int group = tile / (kRasterN * num_m);
    const int first_n = group * kRasterN;
    const int gn = min(kRasterN, num_n - first_n);
    const int local = tile - group * kRasterN * num_m;
    *mb = local / gn;
    *nb = first_n + local % gn;
}

// Operands stored MN-major (A_MN, B_MN: the matrix is given as its transpose,
// [K, rows] row-major) arrive as two 64-row x 64-element TMA boxes per CTA
// half and k-block, 8 KB apart: the 128-byte-swizzled MN-major layout whose
// 64-element blocks along MN are 8 KB apart and whose 8-row groups along K
// are 1024 bytes apart. A 16-deep K step then advances 2048 bytes instead of
// the K-major operand's 32.
constexpr int kMnBox = 64;

__device__ __forceinline__ uint64_t operand_desc(bool mn, uint32_t addr)
{
    return mn ? sw128_mnmajor_desc(addr, kMnBox * BK * 2) : sw128_kmajor_desc(addr);
}

// ------------------------------------------------------- tensor maps (host) --

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn()
{
    static EncodeTiledFn fn = nullptr;
    if (!fn) {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    }
    return fn;
}

// [rows, K] bf16 row-major, box = 64 (K) x box_rows, 128-byte swizzle, zero fill.
inline bool make_map(CUtensorMap* m, const void* ptr, int rows, int K, int box_rows, int ld = 0)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)(ld ? ld : K) * 2};
    cuuint32_t box[2] = {(cuuint32_t)BK, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [K, mn] bf16 row-major (an MN-major operand), box = 64 (MN) x 64 (K), 128-byte swizzle, zero fill.
inline bool make_map_mn(CUtensorMap* m, const void* ptr, int mn, int K, int ld = 0)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)mn, (cuuint64_t)K};
    cuuint64_t strides[1] = {(cuuint64_t)(ld ? ld : mn) * 2};
    cuuint32_t box[2] = {(cuuint32_t)kMnBox, (cuuint32_t)BK};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace twell
