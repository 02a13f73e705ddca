// Test kernels over the bulk 4-bit eviction's tensor-core product: the
// product and its error bound for given rows, and single MMA sums.  The
// library's own source is compiled in, so that what is measured is what it runs.
#include "../../bit_kv_cache_evict_gb300/csrc/evict_bulk.cu"

namespace oscar {
namespace {

// Block = one matrix U; its warps take tiles of 16 of its rows in turn.
__global__ void __launch_bounds__(kBulkThreads, 1) product_kernel(const float* U, const __nv_bfloat16* x, int tiles,
                                                                  float* y, float* bound) {
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gID = lane >> 2, tq = lane & 3;
    int q;
    float rnorm;
    bulk_matrix(U + (size_t)blockIdx.x * kD * kD, smem, q, rnorm);
    uint8_t* xs = smem + BulkSmem::kX + warp * kTile * kXPitch;
    __syncthreads();
    for (int tile = warp; tile < tiles; tile += kBulkWarps) {
        const size_t row0 = ((size_t)blockIdx.x * tiles + tile) * kTile;
        for (int c = lane; c < kTile * 16; c += 32)
            *reinterpret_cast<uint4*>(xs + (c >> 4) * kXPitch + 16 * (c & 15)) =
                *reinterpret_cast<const uint4*>(x + (row0 + (c >> 4)) * kD + 8 * (c & 15));
        __syncwarp();
        float acc[16][4], delta[2];
        bulk_product(smem, xs, pow2f_bits(-q), rnorm, acc, delta);
#pragma unroll
        for (int n = 0; n < 16; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) y[(row0 + gID + 8 * (e >> 1)) * kD + 8 * n + 2 * tq + (e & 1)] = acc[n][e];
        if (tq < 2) bound[row0 + gID + 8 * tq] = delta[tq];
        __syncwarp();
    }
}

// d[i] = c[i] + sum_k a[i][k] b[i][k] by one MMA (row 0, column 0).
__global__ void sum_kernel(const __half* a, const __half* b, const float* c, float* d) {
    const int lane = threadIdx.x, gID = lane >> 2, tq = lane & 3;
    const size_t at = (size_t)blockIdx.x * 16 + 2 * tq;
    const uint32_t a0 = gID ? 0u : *reinterpret_cast<const uint32_t*>(a + at), a2 = gID ? 0u : *reinterpret_cast<const uint32_t*>(a + at + 8);
    const uint32_t b0 = gID ? 0u : *reinterpret_cast<const uint32_t*>(b + at), b1 = gID ? 0u : *reinterpret_cast<const uint32_t*>(b + at + 8);
    float acc[4] = {lane ? 0.f : c[blockIdx.x], 0.f, 0.f, 0.f};
    mma_f16_16816(acc, a0, 0u, a2, 0u, b0, b1);
    if (lane == 0) d[blockIdx.x] = acc[0];
}

}  // namespace
}  // namespace oscar

using namespace oscar;

// Device pointers: U fp32 [mats][128][128], x bf16 [mats][16 tiles][128], y fp32 like x, bound fp32 [mats][16 tiles].
extern "C" int run_product(int mats, int tiles, const float* U, const void* x, float* y, float* bound) {
    cudaError_t e = cudaFuncSetAttribute(product_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, BulkSmem::kBytes);
    if (e != cudaSuccess) return (int)e;
    product_kernel<<<mats, kBulkThreads, BulkSmem::kBytes>>>(U, static_cast<const __nv_bfloat16*>(x), tiles, y, bound);
    e = cudaGetLastError();
    return (int)(e != cudaSuccess ? e : cudaDeviceSynchronize());
}

// Device pointers: a, b fp16 [n][16], c, d fp32 [n].
extern "C" int run_sums(int n, const void* a, const void* b, const float* c, float* d) {
    sum_kernel<<<n, 32>>>(static_cast<const __half*>(a), static_cast<const __half*>(b), c, d);
    const cudaError_t e = cudaGetLastError();
    return (int)(e != cudaSuccess ? e : cudaDeviceSynchronize());
}
