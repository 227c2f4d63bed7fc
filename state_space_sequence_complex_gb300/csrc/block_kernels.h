// Declarations shared by the host entry points (block_host.cu) and the kernels of the
// operators around the scan: gated scan, residual norm, 8-bit quantiser and product.
#pragma once

#include <atomic>
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/ssdc_block.h"

namespace ssdc {
namespace block {

// A kernel's dynamic shared memory, allowed once on each device.
template <typename K>
inline cudaError_t allow_smem(K kernel, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

// A kernel on `groups` clusters of R CTAs of so many threads, as a programmatic dependent.
// `together`: all of them at the same time or not at all (they wait for one another).
template <typename... KArgs, typename... Args>
inline int launch_clusters(void (*kernel)(KArgs...), int64_t groups, int R, bool together, int threads, size_t smem,
                           cudaStream_t stream, const Args&... args) {
    if (groups * R > INT32_MAX) return SSDC_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(groups * R));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = R;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    if (together) {
        attr[1].id = cudaLaunchAttributeCooperative;
        attr[1].val.cooperative = 1;
    } else {
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? 1 : SSDC_ERR_CUDA;
}

// The current device's SMs, asked once (0: an error).
int device_sms();

// One gated-scan call. Strides in elements; reset, h0, h_last, states may be null.
struct Gated {
    const void *x, *f, *i;  // i null: coupled gates
    int64_t x_b, x_t, f_b, f_t, i_b, i_t;
    const uint8_t* reset;
    int64_t T;
    int B, D;
    bool bf16;
    // forward
    const float* h0;
    void* h;
    int64_t h_b, h_t;
    float *h_last, *states;
    // a sequence in segments of `segment` tokens, walked by CTAs of their own (segments > 1): what takes
    // the state that enters a segment from the one before, (B, segments, D) pairs
    float2* joints;
    int segments, segment;
    // backward
    const float* in_states;
    const void* dh;
    int64_t dh_b, dh_t;
    const float* dh_last;
    void *dx, *df, *di;
    int64_t dx_b, dx_t, df_b, df_t, di_b, di_t;
    float* dh0;
    int* status;  // or null
};
int gated_fwd_launch(const Gated& p, cudaStream_t stream);
int gated_segments(int64_t B, int64_t T, int64_t D, bool bf16);  // that a call with a workspace takes
int gated_bwd_launch(const Gated& p, cudaStream_t stream);
int gated_step_launch(const Gated& p, cudaStream_t stream);

// One residual-norm call; out_type as in the header.
struct Norm {
    const void *x, *res;
    int64_t x_ld, res_ld;
    const float* w;
    float eps;
    int64_t M;
    int D;
    bool bf16;
    void* r;
    int64_t r_ld;
    int out_type;
    void* y;
    int64_t y_ld;
    float *scale, *rstd;
};
int norm_fwd_launch(const Norm& p, cudaStream_t stream);

struct NormBwd {
    const void *dy, *dr, *r;
    int64_t dy_ld, dr_ld, r_ld;
    const float *w, *rstd;
    int64_t M;
    int D;
    bool bf16;
    void* dx;
    int64_t dx_ld;
    float *dw, *partial;
};
int norm_bwd_parts(int64_t M, int64_t D);  // rows of D floats that `partial` holds
int norm_bwd_launch(const NormBwd& p, cudaStream_t stream);

struct Quant {
    const void* x;
    int64_t x_ld;
    int64_t M, K;
    bool bf16, blocks;
    uint8_t *q, *qt;
    int64_t q_ld, qt_ld;
    float *scale, *scale_t;
};
int quantize_launch(const Quant& p, cudaStream_t stream);

struct Matmul {
    const uint8_t *a, *b;
    int64_t a_ld, b_ld;
    const float *a_scale, *b_scale;
    bool b_blocks;
    int64_t M, N, K;
    bool out_bf16;
    void* c;
    int64_t c_ld;
    int* status;
    float* partial;
};
size_t matmul_workspace(int64_t M, int64_t N, int64_t K);
int matmul_launch(const Matmul& p, cudaStream_t stream);
// The same for few rows of A (block_matmul_few.cu), and whether it is taken.
bool matmul_is_few(int64_t M, int64_t N, int64_t K);
int matmul_few_launch(const Matmul& p, cudaStream_t stream);

}  // namespace block
}  // namespace ssdc
