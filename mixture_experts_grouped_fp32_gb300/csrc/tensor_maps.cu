// tensor_maps.cu — tensor maps of the training products (grouped_mm.cu); the layer's own are in grouped_gemm.cu.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "common.cuh"

namespace moe {
namespace {

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q);
        return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p)
                                                                    : nullptr;
    }();
    return fn;
}

bool encode_bf16(CUtensorMap* m, const void* base, uint32_t rank, const cuuint64_t* dims, const cuuint64_t* strides,
                 const cuuint32_t* box) {
    const auto enc = encoder();
    const cuuint32_t steps[4] = {1, 1, 1, 1};
    return enc && enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, steps,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// [d2, rows, cols] (cols contiguous), box = [1, box_rows, 64 cols].
bool make_tensor_map_bf16_3d(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint64_t d2,
                             uint32_t box_rows) {
    const cuuint64_t dims[3] = {cols, rows, d2}, strides[2] = {cols * 2, cols * rows * 2};
    const cuuint32_t box[3] = {64, box_rows, 1};
    return encode_bf16(m, base, 3, dims, strides, box);
}

// [d3, rows, cols] viewed as [d3, cols / 64, rows, 64] (cols a multiple of 64): box = [1, blocks, box_rows, 64], i.e.
// `blocks` neighbouring 64-column boxes in one copy, one after another in shared memory.
bool make_tensor_map_bf16_blocks(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint64_t d3,
                                 uint32_t box_rows, uint32_t blocks) {
    if (cols % 64) return false;
    const cuuint64_t dims[4] = {64, rows, cols / 64, d3}, strides[3] = {cols * 2, 128, cols * rows * 2};
    const cuuint32_t box[4] = {64, box_rows, blocks, 1};
    return encode_bf16(m, base, 4, dims, strides, box);
}

}  // namespace moe
