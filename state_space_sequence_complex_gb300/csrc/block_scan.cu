// Gated scan (include/ssdc_block.h): h_t = c_t h_{t-1} + v_t per channel.
//
// One thread walks one channel of one batch row.
#include <cuda_runtime.h>

#include "block_common.cuh"
#include "block_kernels.h"

namespace ssdc {
namespace block {

namespace {

constexpr int kThreads = 128;
constexpr int kChunk = SSD_GATED_STATE_TOKENS;

template <typename T, bool kGate>
__global__ void __launch_bounds__(kThreads) gated_fwd(Gated p) {
    const int64_t k = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (k >= (int64_t)p.B * p.D) return;
    const int b = (int)(k / p.D), d = (int)(k % p.D);
    const T* x = static_cast<const T*>(p.x) + b * p.x_b + d;
    const T* f = static_cast<const T*>(p.f) + b * p.f_b + d;
    const T* g = kGate ? static_cast<const T*>(p.i) + b * p.i_b + d : nullptr;
    T* h = static_cast<T*>(p.h) + b * p.h_b + d;
    float s = p.h0 ? p.h0[k] : 0.0f;
    const int64_t chunks = (p.T + kChunk - 1) / kChunk;
    for (int64_t t = 0; t < p.T; ++t) {
        if (p.states && t % kChunk == 0) p.states[((int64_t)b * chunks + t / kChunk) * p.D + d] = s;
        float a, r;
        sigmoid_pair(to_f32(f[t * p.f_t]), a, r);
        float u = r;
        if (kGate) sigmoid_pair(to_f32(g[t * p.i_t]), u, r);
        const float v = u * to_f32(x[t * p.x_t]);
        const bool stop = p.reset && p.reset[(int64_t)b * p.T + t];
        s = stop ? v : fmaf(a, s, v);
        h[t * p.h_t] = from_f32<T>(s);
    }
    p.h_last[k] = s;
}

template <typename T, bool kGate>
__global__ void __launch_bounds__(kThreads) gated_bwd(Gated p) {
    const int64_t k = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (k >= (int64_t)p.B * p.D) return;
    const int b = (int)(k / p.D), d = (int)(k % p.D);
    const T* x = static_cast<const T*>(p.x) + b * p.x_b + d;
    const T* f = static_cast<const T*>(p.f) + b * p.f_b + d;
    const T* g = kGate ? static_cast<const T*>(p.i) + b * p.i_b + d : nullptr;
    const T* dh = static_cast<const T*>(p.dh) + b * p.dh_b + d;
    T* dx = static_cast<T*>(p.dx) + b * p.dx_b + d;
    T* df = static_cast<T*>(p.df) + b * p.df_b + d;
    T* di = kGate ? static_cast<T*>(p.di) + b * p.di_b + d : nullptr;
    const uint8_t* reset = p.reset ? p.reset + (int64_t)b * p.T : nullptr;
    const int64_t chunks = (p.T + kChunk - 1) / kChunk;
    float carry = p.dh_last ? p.dh_last[k] : 0.0f;  // c_{t+1} g_{t+1}
    for (int64_t c = chunks - 1; c >= 0; --c) {
        const int64_t t0 = c * kChunk;
        const int n = (int)(p.T - t0 < kChunk ? p.T - t0 : kChunk);
        float before[kChunk];
        float s = p.in_states[((int64_t)b * chunks + c) * p.D + d];
        for (int j = 0; j < n; ++j) {
            const int64_t t = t0 + j;
            float a, r;
            sigmoid_pair(to_f32(f[t * p.f_t]), a, r);
            float u = r;
            if (kGate) sigmoid_pair(to_f32(g[t * p.i_t]), u, r);
            const bool stop = reset && reset[t];
            before[j] = stop ? 0.0f : s;
            const float v = u * to_f32(x[t * p.x_t]);
            s = stop ? v : fmaf(a, s, v);
        }
        for (int j = n - 1; j >= 0; --j) {
            const int64_t t = t0 + j;
            float a, na, u, nu;
            sigmoid_pair(to_f32(f[t * p.f_t]), a, na);
            const float xv = to_f32(x[t * p.x_t]);
            const float gr = to_f32(dh[t * p.dh_t]) + carry;
            if (kGate) {
                sigmoid_pair(to_f32(g[t * p.i_t]), u, nu);
                di[t * p.di_t] = from_f32<T>(xv * u * nu * gr);
                df[t * p.df_t] = from_f32<T>(a * na * gr * before[j]);
            } else {
                u = na;
                df[t * p.df_t] = from_f32<T>(a * na * gr * (before[j] - xv));
            }
            dx[t * p.dx_t] = from_f32<T>(u * gr);
            carry = reset && reset[t] ? 0.0f : a * gr;
        }
    }
    if (p.dh0) p.dh0[k] = carry;
}

template <typename T, bool kGate>
__global__ void __launch_bounds__(kThreads) gated_step(Gated p) {
    const int64_t k = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (k >= (int64_t)p.B * p.D) return;
    const int b = (int)(k / p.D), d = (int)(k % p.D);
    float a, r;
    sigmoid_pair(to_f32(static_cast<const T*>(p.f)[b * p.f_b + d]), a, r);
    float u = r;
    if (kGate) sigmoid_pair(to_f32(static_cast<const T*>(p.i)[b * p.i_b + d]), u, r);
    const float s = fmaf(a, p.h0[k], u * to_f32(static_cast<const T*>(p.x)[b * p.x_b + d]));
    static_cast<T*>(p.h)[b * p.h_b + d] = from_f32<T>(s);
    p.h_last[k] = s;
}

unsigned grid_for(const Gated& p) { return (unsigned)(((int64_t)p.B * p.D + kThreads - 1) / kThreads); }

}  // namespace

#define SSD_GATED_LAUNCH(kernel)                                                       \
    do {                                                                               \
        const unsigned grid = grid_for(p);                                             \
        if (p.bf16 && p.i) kernel<__nv_bfloat16, true><<<grid, kThreads, 0, stream>>>(p); \
        else if (p.bf16) kernel<__nv_bfloat16, false><<<grid, kThreads, 0, stream>>>(p);  \
        else if (p.i) kernel<float, true><<<grid, kThreads, 0, stream>>>(p);           \
        else kernel<float, false><<<grid, kThreads, 0, stream>>>(p);                   \
    } while (0)

int gated_fwd_launch(const Gated& p, cudaStream_t stream) {
    SSD_GATED_LAUNCH(gated_fwd);
    return 1;
}
int gated_bwd_launch(const Gated& p, cudaStream_t stream) {
    SSD_GATED_LAUNCH(gated_bwd);
    return 1;
}
int gated_step_launch(const Gated& p, cudaStream_t stream) {
    SSD_GATED_LAUNCH(gated_step);
    return 1;
}

}  // namespace block
}  // namespace ssdc
