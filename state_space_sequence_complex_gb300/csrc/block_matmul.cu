// 8-bit product (include/ssdc_block.h): C[m, n] = sum over groups of 128 columns of
// a_scale[g][m] b_scale[..] sum_k A[m, k] B[n, k].
//
// One CTA computes a 64 x 64 tile with fp32 multiply-adds.
#include <cuda_runtime.h>

#include "block_common.cuh"
#include "block_kernels.h"

namespace ssdc {
namespace block {

namespace {

constexpr int kTile = 64, kStep = 32, kThreads = 256;

__device__ __forceinline__ float from_e4m3(uint8_t v) {
    __nv_fp8_e4m3 f;
    f.__x = v;
    return (float)f;
}

__global__ void __launch_bounds__(kThreads) matmul(Matmul p) {
    __shared__ float a[kStep][kTile + 1], b[kStep][kTile + 1];
    const int64_t m0 = (int64_t)blockIdx.y * kTile, n0 = (int64_t)blockIdx.x * kTile;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    const int64_t KB = (p.K + 127) / 128;
    float acc[4][4] = {};
    for (int64_t g = 0; g < KB; ++g) {
        float part[4][4] = {};
        for (int64_t k0 = g * 128; k0 < (g + 1) * 128 && k0 < p.K; k0 += kStep) {
            __syncthreads();
            for (int e = threadIdx.x; e < kTile * kStep; e += kThreads) {
                const int r = e / kStep, k = e % kStep;
                a[k][r] = m0 + r < p.M && k0 + k < p.K ? from_e4m3(p.a[(m0 + r) * p.a_ld + k0 + k]) : 0.0f;
                b[k][r] = n0 + r < p.N && k0 + k < p.K ? from_e4m3(p.b[(n0 + r) * p.b_ld + k0 + k]) : 0.0f;
            }
            __syncthreads();
            for (int k = 0; k < kStep; ++k)
                for (int i = 0; i < 4; ++i)
                    for (int j = 0; j < 4; ++j) part[i][j] = fmaf(a[k][ty + 16 * i], b[k][tx + 16 * j], part[i][j]);
        }
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < 4; ++j) {
                const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
                if (m < p.M && n < p.N) {
                    const float sb = p.b_blocks ? p.b_scale[(n / 128) * KB + g] : p.b_scale[g * p.N + n];
                    acc[i][j] = fmaf(part[i][j], p.a_scale[g * p.M + m] * sb, acc[i][j]);
                }
            }
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (m < p.M && n < p.N) {
                if (p.out_bf16) static_cast<__nv_bfloat16*>(p.c)[m * p.c_ld + n] = __float2bfloat16_rn(acc[i][j]);
                else static_cast<float*>(p.c)[m * p.c_ld + n] = acc[i][j];
            }
        }
}

}  // namespace

size_t matmul_workspace(int64_t, int64_t, int64_t) { return 256; }

int matmul_launch(const Matmul& p, cudaStream_t stream) {
    const dim3 grid((unsigned)((p.N + kTile - 1) / kTile), (unsigned)((p.M + kTile - 1) / kTile));
    if (grid.y > 65535) return SSDC_ERR_UNSUPPORTED;
    matmul<<<grid, kThreads, 0, stream>>>(p);
    return 1;
}

}  // namespace block
}  // namespace ssdc
