// Residual norm, its gradients, and the 8-bit quantiser (include/ssdc_block.h).
#include <cuda_runtime.h>

#include "block_common.cuh"
#include "block_kernels.h"

namespace ssdc {
namespace block {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ float block_sum(float v) {
    __shared__ float part[kWarps];
    v = warp_sum(v);
    __syncthreads();
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    float s = 0.0f;
    for (int k = 0; k < kWarps; ++k) s += part[k];
    return s;
}

// One CTA a row; a warp owns whole groups of 128 features.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_fwd(Norm p) {
    const int64_t m = blockIdx.x;
    const T* x = static_cast<const T*>(p.x) + m * p.x_ld;
    const T* res = p.res ? static_cast<const T*>(p.res) + m * p.res_ld : nullptr;
    T* r = p.r ? static_cast<T*>(p.r) + m * p.r_ld : nullptr;
    float sq = 0.0f;
    for (int d = threadIdx.x; d < p.D; d += kThreads) {
        const float v = to_f32(x[d]) + (res ? to_f32(res[d]) : 0.0f);
        sq = fmaf(v, v, sq);
    }
    const float rstd = rsqrtf(block_sum(sq) / (float)p.D + p.eps);
    if (p.rstd && threadIdx.x == 0) p.rstd[m] = rstd;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    for (int d0 = warp * 128; d0 < p.D; d0 += kWarps * 128) {
        float y[4], amax = 0.0f;
        for (int j = 0; j < 4; ++j) {
            const int d = d0 + lane + 32 * j;
            y[j] = 0.0f;
            if (d < p.D) {
                const float v = to_f32(x[d]) + (res ? to_f32(res[d]) : 0.0f);
                if (r) r[d] = from_f32<T>(v);
                y[j] = v * rstd * (p.w ? p.w[d] : 1.0f);
                if (p.out_type == SSD_TYPE_F32) static_cast<float*>(p.y)[m * p.y_ld + d] = y[j];
                if (p.out_type == SSD_TYPE_BF16)
                    static_cast<__nv_bfloat16*>(p.y)[m * p.y_ld + d] = __float2bfloat16_rn(y[j]);
            }
            amax = fmaxf(amax, fabsf(y[j]));
        }
        if (p.out_type == SSD_TYPE_E4M3) {
            const float s = group_scale(warp_max(amax));
            if (lane == 0) p.scale[(int64_t)(d0 / 128) * p.M + m] = s;
            for (int j = 0; j < 4; ++j) {
                const int d = d0 + lane + 32 * j;
                if (d < p.D) static_cast<uint8_t*>(p.y)[m * p.y_ld + d] = e4m3(y[j] / s);
            }
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) norm_bwd(NormBwd p) {
    const int64_t m = blockIdx.x;
    const T* dy = static_cast<const T*>(p.dy) + m * p.dy_ld;
    const T* dr = p.dr ? static_cast<const T*>(p.dr) + m * p.dr_ld : nullptr;
    const T* r = static_cast<const T*>(p.r) + m * p.r_ld;
    T* dx = static_cast<T*>(p.dx) + m * p.dx_ld;
    const float rstd = p.rstd[m];
    float s = 0.0f;
    for (int d = threadIdx.x; d < p.D; d += kThreads)
        s += to_f32(dy[d]) * (p.w ? p.w[d] : 1.0f) * (to_f32(r[d]) * rstd);
    const float mean = block_sum(s) / (float)p.D;
    for (int d = threadIdx.x; d < p.D; d += kThreads) {
        const float xh = to_f32(r[d]) * rstd, gy = to_f32(dy[d]) * (p.w ? p.w[d] : 1.0f);
        dx[d] = from_f32<T>((dr ? to_f32(dr[d]) : 0.0f) + rstd * (gy - xh * mean));
    }
}

// dw: one CTA for 32 features and one part of the rows, before dx may overwrite dy.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_bwd_dw(NormBwd p, int parts) {
    const int d = blockIdx.x * 32 + threadIdx.x % 32;
    const int64_t per = (p.M + parts - 1) / parts, m0 = blockIdx.y * per;
    const int64_t m1 = m0 + per < p.M ? m0 + per : p.M;
    __shared__ float part[kWarps][32];
    float s = 0.0f;
    if (d < p.D)
        for (int64_t m = m0 + threadIdx.x / 32; m < m1; m += kWarps)
            s += to_f32(static_cast<const T*>(p.dy)[m * p.dy_ld + d]) *
                 (to_f32(static_cast<const T*>(p.r)[m * p.r_ld + d]) * p.rstd[m]);
    part[threadIdx.x / 32][threadIdx.x % 32] = s;
    __syncthreads();
    if (threadIdx.x < 32 && d < p.D) {
        s = 0.0f;
        for (int k = 0; k < kWarps; ++k) s += part[k][threadIdx.x];
        p.partial[(int64_t)blockIdx.y * p.D + d] = s;
    }
}

__global__ void __launch_bounds__(kThreads) norm_bwd_sum(NormBwd p, int parts) {
    const int d = blockIdx.x * kThreads + threadIdx.x;
    if (d >= p.D) return;
    float s = 0.0f;
    for (int k = 0; k < parts; ++k) s += p.partial[(int64_t)k * p.D + d];
    p.dw[d] = s;
}

// One CTA a tile of 128 x 128; threads re-read the tile.
template <typename T>
__global__ void __launch_bounds__(128) quantize(Quant p) {
    __shared__ float amax[128];
    const int64_t m0 = (int64_t)blockIdx.y * 128, k0 = (int64_t)blockIdx.x * 128;
    const int t = threadIdx.x;
    const int64_t MB = (p.M + 127) / 128, KB = (p.K + 127) / 128;
    auto at = [&](int64_t m, int64_t k) {
        return m < p.M && k < p.K ? to_f32(static_cast<const T*>(p.x)[m * p.x_ld + k]) : 0.0f;
    };
    float by_row = 0.0f, by_col = 0.0f;
    for (int j = 0; j < 128; ++j) {
        by_row = fmaxf(by_row, fabsf(at(m0 + t, k0 + j)));
        by_col = fmaxf(by_col, fabsf(at(m0 + j, k0 + t)));
    }
    if (p.blocks) {
        amax[t] = by_row;
        __syncthreads();
        for (int j = 0; j < 128; ++j) by_row = fmaxf(by_row, amax[j]);
        by_col = by_row;
    }
    const float sr = group_scale(by_row), sc = group_scale(by_col);
    if (p.q) {
        if (p.blocks && t == 0) p.scale[blockIdx.y * KB + blockIdx.x] = sr;
        if (!p.blocks && m0 + t < p.M) p.scale[blockIdx.x * p.M + m0 + t] = sr;
        for (int j = 0; j < 128; ++j)
            if (m0 + t < p.M && k0 + j < p.K) p.q[(m0 + t) * p.q_ld + k0 + j] = e4m3(at(m0 + t, k0 + j) / sr);
    }
    if (p.qt) {
        if (p.blocks && t == 0) p.scale_t[blockIdx.x * MB + blockIdx.y] = sc;
        if (!p.blocks && k0 + t < p.K) p.scale_t[blockIdx.y * p.K + k0 + t] = sc;
        for (int j = 0; j < 128; ++j)
            if (m0 + j < p.M && k0 + t < p.K) p.qt[(k0 + t) * p.qt_ld + m0 + j] = e4m3(at(m0 + j, k0 + t) / sc);
    }
}

}  // namespace

int norm_fwd_launch(const Norm& p, cudaStream_t stream) {
    if (p.bf16) norm_fwd<__nv_bfloat16><<<(unsigned)p.M, kThreads, 0, stream>>>(p);
    else norm_fwd<float><<<(unsigned)p.M, kThreads, 0, stream>>>(p);
    return 1;
}

int norm_bwd_parts(int64_t M, int64_t) { return (int)(M < 1024 ? 1 : M / 1024 < 64 ? M / 1024 : 64); }

int norm_bwd_launch(const NormBwd& p, cudaStream_t stream) {
    int launches = 1;
    if (p.dw) {
        const int parts = norm_bwd_parts(p.M, p.D);
        const dim3 grid((p.D + 31) / 32, parts);
        if (p.bf16) norm_bwd_dw<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(p, parts);
        else norm_bwd_dw<float><<<grid, kThreads, 0, stream>>>(p, parts);
        norm_bwd_sum<<<(p.D + kThreads - 1) / kThreads, kThreads, 0, stream>>>(p, parts);
        launches += 2;
    }
    if (p.bf16) norm_bwd<__nv_bfloat16><<<(unsigned)p.M, kThreads, 0, stream>>>(p);
    else norm_bwd<float><<<(unsigned)p.M, kThreads, 0, stream>>>(p);
    return launches;
}

int quantize_launch(const Quant& p, cudaStream_t stream) {
    const dim3 grid((unsigned)((p.K + 127) / 128), (unsigned)((p.M + 127) / 128));
    if (grid.y > 65535) return SSDC_ERR_UNSUPPORTED;
    if (p.bf16) quantize<__nv_bfloat16><<<grid, 128, 0, stream>>>(p);
    else quantize<float><<<grid, 128, 0, stream>>>(p);
    return 1;
}

}  // namespace block
}  // namespace ssdc
