// Host side of the C ABI declared in include/ssdc_block.h: argument checks, then one
// launch sequence per call on the caller's stream. Nothing is allocated.
#include <atomic>
#include <cstdint>
#include <cstring>
#include <initializer_list>

#include <cuda_runtime.h>

#include "block_args.h"

namespace {

using namespace ssdc::block;

constexpr int kMaxDevices = 64;
std::atomic<int> g_device_ok[kMaxDevices];  // an sm_103 device's SMs

Array seq(const void* p, int64_t sb, int64_t st, const ssd_gated_dims& d) {
    return Array{p, d.B, d.T, d.D, taken(sb, d.B), taken(st, d.T), type_bytes(d.type)};
}
int check_gated(const ssd_gated_dims& d) {
    if (d.B <= 0 || d.T <= 0 || d.D <= 0) return SSDC_ERR_INVALID;
    if (d.type != SSD_TYPE_F32 && d.type != SSD_TYPE_BF16) return SSDC_ERR_INVALID;
    if (d.B > INT32_MAX || d.D > INT32_MAX || d.B > INT32_MAX / d.D || d.T > INT32_MAX) return SSDC_ERR_UNSUPPORTED;
    if ((double)d.B * (double)d.T * (double)d.D > (double)kBig) return SSDC_ERR_UNSUPPORTED;
    return SSDC_OK;
}

int64_t state_rows(const ssd_gated_dims& d) {
    return (d.T + SSD_GATED_STATE_TOKENS - 1) / SSD_GATED_STATE_TOKENS;
}

// The kernels step from token to token in 32 bits.
int check_token_strides(const ssd_gated_dims& d, std::initializer_list<int64_t> strides) {
    for (int64_t s : strides)
        if (taken(s, d.T) >= (int64_t(1) << 31) / (int64_t)type_bytes(d.type)) return SSDC_ERR_UNSUPPORTED;
    return SSDC_OK;
}

Gated gated_problem(const ssd_seq_in& x, const ssd_seq_in& f, const ssd_seq_in& i, const ssd_gated_dims& d) {
    Gated p = {};
    p.x = x.p; p.x_b = taken(x.stride_b, d.B); p.x_t = taken(x.stride_t, d.T);
    p.f = f.p; p.f_b = taken(f.stride_b, d.B); p.f_t = taken(f.stride_t, d.T);
    p.i = i.p; p.i_b = taken(i.stride_b, d.B); p.i_t = taken(i.stride_t, d.T);
    p.T = d.T; p.B = (int)d.B; p.D = (int)d.D;
    p.bf16 = d.type == SSD_TYPE_BF16;
    return p;
}

int check_rows(int64_t M, int64_t D, int type) {
    if (M <= 0 || D <= 0) return SSDC_ERR_INVALID;
    if (type != SSD_TYPE_F32 && type != SSD_TYPE_BF16) return SSDC_ERR_INVALID;
    if (D > 32768 || M > INT32_MAX) return SSDC_ERR_UNSUPPORTED;
    return SSDC_OK;
}

}  // namespace

int ssdc::block::check_device() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return SSDC_ERR_CUDA;
    if (g_device_ok[dev].load(std::memory_order_acquire)) return SSDC_OK;
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
        return SSDC_ERR_CUDA;
    if (major != 10 || minor != 3) return SSDC_ERR_DEVICE;
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 2) return SSDC_ERR_CUDA;
    g_device_ok[dev].store(sms, std::memory_order_release);
    return SSDC_OK;
}

int ssdc::block::device_sms() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
    return g_device_ok[dev].load(std::memory_order_acquire);
}

extern "C" {

size_t ssd_gated_scan_states_bytes(ssd_gated_dims dims) {
    if (check_gated(dims) != SSDC_OK) return 0;
    return (size_t)(dims.B * state_rows(dims) * dims.D) * sizeof(float);
}

size_t ssd_gated_scan_workspace_bytes(ssd_gated_dims d) {
    if (check_gated(d) != SSDC_OK) return 0;
    const int segments = gated_segments(d.B, d.T, d.D, d.type == SSD_TYPE_BF16);
    return segments > 1 ? (size_t)(d.B * segments * d.D) * sizeof(float2) : 0;
}

int ssd_gated_scan_fwd(ssd_seq_in x, ssd_seq_in f, ssd_seq_in i, const float* h0, const uint8_t* reset,
                       ssd_gated_dims d, ssd_seq_out h, float* h_last, float* states, int32_t* status,
                       cudaStream_t stream) {
    return ssd_gated_scan_fwd_ws(x, f, i, h0, reset, d, h, h_last, states, status, nullptr, 0, stream);
}

int ssd_gated_scan_fwd_ws(ssd_seq_in x, ssd_seq_in f, ssd_seq_in i, const float* h0, const uint8_t* reset,
                          ssd_gated_dims d, ssd_seq_out h, float* h_last, float* states, int32_t* status,
                          void* workspace, size_t ws_bytes, cudaStream_t stream) {
    int rc = check_gated(d);
    if (rc != SSDC_OK) return rc;
    const size_t need = workspace ? ssd_gated_scan_workspace_bytes(d) : 0;
    if (workspace != nullptr && (ws_bytes < need || !aligned_to(workspace, 16))) return SSDC_ERR_WORKSPACE;
    Args a;
    a.input(seq(x.p, x.stride_b, x.stride_t, d));
    a.input(seq(f.p, f.stride_b, f.stride_t, d));
    a.input(seq(i.p, i.stride_b, i.stride_t, d), false);
    a.input(dense(h0, d.B * d.D), false);
    a.input(dense(reset, d.B * d.T, 1), false);
    a.output(seq(h.p, h.stride_b, h.stride_t, d));
    a.output(dense(h_last, d.B * d.D), true, h0);
    a.output(dense(states, d.B * state_rows(d) * d.D), false);
    a.output(dense(status, 1), false);
    if (need > 0) a.output(dense(workspace, (int64_t)(need / 4)));
    if (a.rc != SSDC_OK) return a.rc;
    rc = check_token_strides(d, {x.stride_t, f.stride_t, i.stride_t, h.stride_t});
    if (rc == SSDC_OK) rc = check_device();
    if (rc != SSDC_OK) return rc;
    Gated p = gated_problem(x, f, i, d);
    p.h0 = h0; p.reset = reset;
    p.h = h.p; p.h_b = taken(h.stride_b, d.B); p.h_t = taken(h.stride_t, d.T);
    p.h_last = h_last; p.states = states; p.status = status;
    p.joints = need > 0 ? static_cast<float2*>(workspace) : nullptr;
    (void)cudaGetLastError();
    return done(gated_fwd_launch(p, stream));
}

int ssd_gated_scan_step(ssd_seq_in x, ssd_seq_in f, ssd_seq_in i, const float* state_in, int64_t B, int64_t D,
                        int32_t type, ssd_seq_out h, float* state_out, cudaStream_t stream) {
    const ssd_gated_dims d = {B, 1, D, type};
    int rc = check_gated(d);
    if (rc != SSDC_OK) return rc;
    Args a;
    a.input(seq(x.p, x.stride_b, 0, d));
    a.input(seq(f.p, f.stride_b, 0, d));
    a.input(seq(i.p, i.stride_b, 0, d), false);
    a.input(dense(state_in, B * D));
    a.output(seq(h.p, h.stride_b, 0, d));
    a.output(dense(state_out, B * D), true, state_in);
    if (a.rc != SSDC_OK) return a.rc;
    rc = check_device();
    if (rc != SSDC_OK) return rc;
    Gated p = gated_problem(x, f, i, d);
    p.h0 = state_in; p.h = h.p; p.h_b = taken(h.stride_b, B); p.h_last = state_out;
    (void)cudaGetLastError();
    return done(gated_step_launch(p, stream));
}

int ssd_gated_scan_bwd(ssd_seq_in x, ssd_seq_in f, ssd_seq_in i, const float* states, const uint8_t* reset,
                       ssd_seq_in dh, const float* dh_last, ssd_gated_dims d, ssd_seq_out dx, ssd_seq_out df,
                       ssd_seq_out di, float* dh0, int32_t* status, cudaStream_t stream) {
    int rc = check_gated(d);
    if (rc != SSDC_OK) return rc;
    if ((i.p == nullptr) != (di.p == nullptr)) return SSDC_ERR_INVALID;
    Args a;
    a.input(seq(x.p, x.stride_b, x.stride_t, d));
    a.input(seq(f.p, f.stride_b, f.stride_t, d));
    a.input(seq(i.p, i.stride_b, i.stride_t, d), false);
    a.input(dense(states, d.B * state_rows(d) * d.D));
    a.input(dense(reset, d.B * d.T, 1), false);
    a.input(seq(dh.p, dh.stride_b, dh.stride_t, d));
    a.input(dense(dh_last, d.B * d.D), false);
    a.output(seq(dx.p, dx.stride_b, dx.stride_t, d));
    a.output(seq(df.p, df.stride_b, df.stride_t, d));
    a.output(seq(di.p, di.stride_b, di.stride_t, d), false);
    a.output(dense(dh0, d.B * d.D), false, dh_last);
    a.output(dense(status, 1), false);
    if (a.rc != SSDC_OK) return a.rc;
    rc = check_token_strides(d, {x.stride_t, f.stride_t, i.stride_t, dh.stride_t, dx.stride_t, df.stride_t, di.stride_t});
    if (rc == SSDC_OK) rc = check_device();
    if (rc != SSDC_OK) return rc;
    Gated p = gated_problem(x, f, i, d);
    p.in_states = states; p.reset = reset;
    p.dh = dh.p; p.dh_b = taken(dh.stride_b, d.B); p.dh_t = taken(dh.stride_t, d.T); p.dh_last = dh_last;
    p.dx = dx.p; p.dx_b = taken(dx.stride_b, d.B); p.dx_t = taken(dx.stride_t, d.T);
    p.df = df.p; p.df_b = taken(df.stride_b, d.B); p.df_t = taken(df.stride_t, d.T);
    p.di = di.p; p.di_b = taken(di.stride_b, d.B); p.di_t = taken(di.stride_t, d.T);
    p.dh0 = dh0; p.status = status;
    (void)cudaGetLastError();
    return done(gated_bwd_launch(p, stream));
}

int ssd_residual_norm_fwd(ssd_rows_in x, ssd_rows_in residual, const float* w, float eps, int64_t M, int64_t D,
                          int32_t type, ssd_rows_out r, int32_t out_type, ssd_rows_out y, float* scale, float* rstd,
                          cudaStream_t stream) {
    int rc = check_rows(M, D, type);
    if (rc != SSDC_OK) return rc;
    if (out_type != SSD_TYPE_F32 && out_type != SSD_TYPE_BF16 && out_type != SSD_TYPE_E4M3) return SSDC_ERR_INVALID;
    if (!(eps >= 0.0f)) return SSDC_ERR_INVALID;
    const bool fp8 = out_type == SSD_TYPE_E4M3;
    if (fp8 != (scale != nullptr)) return SSDC_ERR_INVALID;
    if (fp8 && (rc = check_fp8_rows(y.p, y.ld, M, D)) != SSDC_OK) return rc;
    Args a;
    a.input(rows(x.p, x.ld, M, D, type_bytes(type)));
    a.input(rows(residual.p, residual.ld, M, D, type_bytes(type)), false);
    a.input(dense(w, D), false);
    a.output(rows(r.p, r.ld, M, D, type_bytes(type)), false, x.p, residual.p);
    a.output(rows(y.p, y.ld, M, D, type_bytes(out_type)));
    a.output(dense(scale, M * groups(D)), fp8);
    a.output(dense(rstd, M), false);
    if (a.rc != SSDC_OK) return a.rc;
    rc = check_device();
    if (rc != SSDC_OK) return rc;
    Norm p = {};
    const size_t e = type_bytes(type), eo = type_bytes(out_type);
    p.x = x.p; p.x_ld = row_stride(x.ld, M, D, e); p.res = residual.p; p.res_ld = row_stride(residual.ld, M, D, e);
    p.w = w; p.eps = eps; p.M = M; p.D = (int)D; p.bf16 = type == SSD_TYPE_BF16;
    p.r = r.p; p.r_ld = row_stride(r.ld, M, D, e); p.out_type = out_type; p.y = y.p; p.y_ld = row_stride(y.ld, M, D, eo);
    p.scale = scale; p.rstd = rstd;
    (void)cudaGetLastError();
    return done(norm_fwd_launch(p, stream));
}

size_t ssd_residual_norm_bwd_workspace_bytes(int64_t M, int64_t D) {
    if (check_rows(M, D, SSD_TYPE_F32) != SSDC_OK) return 0;
    return (size_t)norm_bwd_parts(M, D) * (size_t)D * sizeof(float);
}

int ssd_residual_norm_bwd(ssd_rows_in dy, ssd_rows_in dr, ssd_rows_in r, const float* w, const float* rstd, int64_t M,
                          int64_t D, int32_t type, ssd_rows_out dx, float* dw, void* workspace, size_t ws_bytes,
                          cudaStream_t stream) {
    int rc = check_rows(M, D, type);
    if (rc != SSDC_OK) return rc;
    const size_t e = type_bytes(type), need = ssd_residual_norm_bwd_workspace_bytes(M, D);
    if (dw != nullptr && (workspace == nullptr || !aligned_to(workspace, 256) || ws_bytes < need))
        return SSDC_ERR_WORKSPACE;
    Args a;
    a.input(rows(dy.p, dy.ld, M, D, e));
    a.input(rows(dr.p, dr.ld, M, D, e), false);
    a.input(rows(r.p, r.ld, M, D, e));
    a.input(dense(w, D), false);
    a.input(dense(rstd, M));
    a.output(rows(dx.p, dx.ld, M, D, e), true, dy.p, dr.p);
    a.output(dense(dw, D), false);
    if (dw != nullptr) a.output(dense(workspace, (int64_t)(need / 4)));
    if (a.rc != SSDC_OK) return a.rc;
    rc = check_device();
    if (rc != SSDC_OK) return rc;
    NormBwd p = {};
    p.dy = dy.p; p.dy_ld = row_stride(dy.ld, M, D, e); p.dr = dr.p; p.dr_ld = row_stride(dr.ld, M, D, e);
    p.r = r.p; p.r_ld = row_stride(r.ld, M, D, e);
    p.w = w; p.rstd = rstd; p.M = M; p.D = (int)D; p.bf16 = type == SSD_TYPE_BF16;
    p.dx = dx.p; p.dx_ld = row_stride(dx.ld, M, D, e); p.dw = dw; p.partial = static_cast<float*>(workspace);
    (void)cudaGetLastError();
    return done(norm_bwd_launch(p, stream));
}

int ssd_fp8_quantize(ssd_rows_in x, int64_t M, int64_t K, int32_t type, int32_t scales, ssd_rows_out q, float* scale,
                     ssd_rows_out qt, float* scale_t, cudaStream_t stream) {
    if (M <= 0 || K <= 0) return SSDC_ERR_INVALID;
    if (type != SSD_TYPE_F32 && type != SSD_TYPE_BF16) return SSDC_ERR_INVALID;
    if (scales != SSD_SCALE_ROWS && scales != SSD_SCALE_BLOCKS) return SSDC_ERR_INVALID;
    if (M > INT32_MAX - 128 || K > INT32_MAX - 128) return SSDC_ERR_UNSUPPORTED;
    if (q.p == nullptr && qt.p == nullptr) return SSDC_ERR_INVALID;
    if ((q.p == nullptr) != (scale == nullptr) || (qt.p == nullptr) != (scale_t == nullptr)) return SSDC_ERR_INVALID;
    int rc;
    if ((rc = check_fp8_rows(q.p, q.ld, M, K)) != SSDC_OK || (rc = check_fp8_rows(qt.p, qt.ld, K, M)) != SSDC_OK) return rc;
    const bool blocks = scales == SSD_SCALE_BLOCKS;
    Args a;
    a.input(rows(x.p, x.ld, M, K, type_bytes(type)));
    a.output(rows(q.p, q.ld, M, K, 1), false);
    a.output(dense(scale, blocks ? groups(M) * groups(K) : M * groups(K)), false);
    a.output(rows(qt.p, qt.ld, K, M, 1), false);
    a.output(dense(scale_t, blocks ? groups(M) * groups(K) : K * groups(M)), false);
    if (a.rc != SSDC_OK) return a.rc;
    rc = check_device();
    if (rc != SSDC_OK) return rc;
    Quant p = {};
    p.x = x.p; p.x_ld = row_stride(x.ld, M, K, type_bytes(type)); p.M = M; p.K = K; p.bf16 = type == SSD_TYPE_BF16; p.blocks = blocks;
    p.q = static_cast<uint8_t*>(q.p); p.q_ld = q.ld; p.scale = scale;
    p.qt = static_cast<uint8_t*>(qt.p); p.qt_ld = qt.ld; p.scale_t = scale_t;
    (void)cudaGetLastError();
    return done(quantize_launch(p, stream));
}

size_t ssd_fp8_matmul_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (M <= 0 || N <= 0 || K <= 0 || M > INT32_MAX - 256 || N > INT32_MAX - 256 || K > INT32_MAX - 256) return 0;
    return matmul_workspace(M, N, K);
}

int ssd_fp8_matmul(ssd_rows_in a8, const float* a_scale, ssd_rows_in b8, const float* b_scale, int32_t b_scales,
                   int64_t M, int64_t N, int64_t K, int32_t out_type, ssd_rows_out c, void* workspace,
                   size_t ws_bytes, cudaStream_t stream) {
    if (M <= 0 || N <= 0 || K <= 0) return SSDC_ERR_INVALID;
    if (out_type != SSD_TYPE_F32 && out_type != SSD_TYPE_BF16) return SSDC_ERR_INVALID;
    if (b_scales != SSD_SCALE_ROWS && b_scales != SSD_SCALE_BLOCKS) return SSDC_ERR_INVALID;
    if (M > INT32_MAX - 256 || N > INT32_MAX - 256 || K > INT32_MAX - 256) return SSDC_ERR_UNSUPPORTED;
    int rc;
    if ((rc = check_fp8_rows(a8.p, a8.ld, M, K)) != SSDC_OK || (rc = check_fp8_rows(b8.p, b8.ld, N, K)) != SSDC_OK) return rc;
    const size_t need = matmul_workspace(M, N, K);
    if (workspace == nullptr || !aligned_to(workspace, 256) || ws_bytes < need) return SSDC_ERR_WORKSPACE;
    const bool blocks = b_scales == SSD_SCALE_BLOCKS;
    Args a;
    a.input(rows(a8.p, a8.ld, M, K, 1));
    a.input(dense(a_scale, M * groups(K)));
    a.input(rows(b8.p, b8.ld, N, K, 1));
    a.input(dense(b_scale, blocks ? groups(N) * groups(K) : N * groups(K)));
    a.output(rows(c.p, c.ld, M, N, type_bytes(out_type)));
    a.output(dense(workspace, (int64_t)(need / 4)));
    if (a.rc != SSDC_OK) return a.rc;
    rc = check_device();
    if (rc != SSDC_OK) return rc;
    Matmul p = {};
    p.a = static_cast<const uint8_t*>(a8.p); p.a_ld = row_stride(a8.ld, M, K, 1); p.a_scale = a_scale;
    p.b = static_cast<const uint8_t*>(b8.p); p.b_ld = row_stride(b8.ld, N, K, 1); p.b_scale = b_scale; p.b_blocks = blocks;
    p.M = M; p.N = N; p.K = K; p.out_bf16 = out_type == SSD_TYPE_BF16;
    p.c = c.p; p.c_ld = row_stride(c.ld, M, N, type_bytes(out_type));
    p.status = static_cast<int*>(workspace);
    p.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + 256);
    (void)cudaGetLastError();
    return done(matmul_launch(p, stream));
}

int ssd_block_call(int32_t call, const int64_t* words, cudaStream_t stream) {
    if (words == nullptr) return SSDC_ERR_INVALID;
    const int64_t* w = words;
    auto ptr = [&] { return reinterpret_cast<void*>(*w++); };
    auto f32 = [&] { return static_cast<float*>(ptr()); };
    auto i64 = [&] { return *w++; };
    auto i32 = [&] { return (int32_t)*w++; };
    auto seq_in = [&] { ssd_seq_in a; a.p = ptr(); a.stride_b = i64(); a.stride_t = i64(); return a; };
    auto seq_out = [&] { ssd_seq_out a; a.p = ptr(); a.stride_b = i64(); a.stride_t = i64(); return a; };
    auto rows_in = [&] { ssd_rows_in a; a.p = ptr(); a.ld = i64(); return a; };
    auto rows_out = [&] { ssd_rows_out a; a.p = ptr(); a.ld = i64(); return a; };
    auto dims = [&] { ssd_gated_dims d; d.B = i64(); d.T = i64(); d.D = i64(); d.type = i32(); return d; };
    switch (call) {
        case SSD_CALL_GATED_SCAN_FWD: {
            const ssd_seq_in x = seq_in(), f = seq_in(), i = seq_in();
            const float* h0 = f32();
            const uint8_t* reset = static_cast<const uint8_t*>(ptr());
            const ssd_gated_dims d = dims();
            const ssd_seq_out h = seq_out();
            float *h_last = f32(), *states = f32();
            return ssd_gated_scan_fwd(x, f, i, h0, reset, d, h, h_last, states, static_cast<int32_t*>(ptr()), stream);
        }
        case SSD_CALL_GATED_SCAN_FWD_WS: {
            const ssd_seq_in x = seq_in(), f = seq_in(), i = seq_in();
            const float* h0 = f32();
            const uint8_t* reset = static_cast<const uint8_t*>(ptr());
            const ssd_gated_dims d = dims();
            const ssd_seq_out h = seq_out();
            float *h_last = f32(), *states = f32();
            int32_t* status = static_cast<int32_t*>(ptr());
            void* ws = ptr();
            return ssd_gated_scan_fwd_ws(x, f, i, h0, reset, d, h, h_last, states, status, ws, (size_t)i64(), stream);
        }
        case SSD_CALL_GATED_SCAN_STEP: {
            const ssd_seq_in x = seq_in(), f = seq_in(), i = seq_in();
            const float* state = f32();
            const int64_t B = i64(), D = i64();
            const int32_t type = i32();
            const ssd_seq_out h = seq_out();
            return ssd_gated_scan_step(x, f, i, state, B, D, type, h, f32(), stream);
        }
        case SSD_CALL_GATED_SCAN_BWD: {
            const ssd_seq_in x = seq_in(), f = seq_in(), i = seq_in();
            const float* states = f32();
            const uint8_t* reset = static_cast<const uint8_t*>(ptr());
            const ssd_seq_in dh = seq_in();
            const float* dh_last = f32();
            const ssd_gated_dims d = dims();
            const ssd_seq_out dx = seq_out(), df = seq_out(), di = seq_out();
            float* dh0 = f32();
            return ssd_gated_scan_bwd(x, f, i, states, reset, dh, dh_last, d, dx, df, di, dh0, static_cast<int32_t*>(ptr()),
                                      stream);
        }
        case SSD_CALL_RESIDUAL_NORM_FWD: {
            const ssd_rows_in x = rows_in(), res = rows_in();
            const float* weights = f32();
            const uint32_t bits = (uint32_t)i64();
            float eps;
            std::memcpy(&eps, &bits, sizeof eps);
            const int64_t M = i64(), D = i64();
            const int32_t type = i32();
            const ssd_rows_out r = rows_out();
            const int32_t out_type = i32();
            const ssd_rows_out y = rows_out();
            float* scale = f32();
            return ssd_residual_norm_fwd(x, res, weights, eps, M, D, type, r, out_type, y, scale, f32(), stream);
        }
        case SSD_CALL_RESIDUAL_NORM_BWD: {
            const ssd_rows_in dy = rows_in(), dr = rows_in(), r = rows_in();
            const float *weights = f32(), *rstd = f32();
            const int64_t M = i64(), D = i64();
            const int32_t type = i32();
            const ssd_rows_out dx = rows_out();
            float* dw = f32();
            void* ws = ptr();
            return ssd_residual_norm_bwd(dy, dr, r, weights, rstd, M, D, type, dx, dw, ws, (size_t)i64(), stream);
        }
        case SSD_CALL_FP8_QUANTIZE: {
            const ssd_rows_in x = rows_in();
            const int64_t M = i64(), K = i64();
            const int32_t type = i32(), scales = i32();
            const ssd_rows_out q = rows_out();
            float* scale = f32();
            const ssd_rows_out qt = rows_out();
            return ssd_fp8_quantize(x, M, K, type, scales, q, scale, qt, f32(), stream);
        }
        case SSD_CALL_FP8_MATMUL: {
            const ssd_rows_in a = rows_in();
            const float* a_scale = f32();
            const ssd_rows_in b = rows_in();
            const float* b_scale = f32();
            const int32_t b_scales = i32();
            const int64_t M = i64(), N = i64(), K = i64();
            const int32_t out_type = i32();
            const ssd_rows_out c = rows_out();
            void* ws = ptr();
            return ssd_fp8_matmul(a, a_scale, b, b_scale, b_scales, M, N, K, out_type, c, ws, (size_t)i64(), stream);
        }
        default: return delta_call(call, words, stream);
    }
}

}  // extern "C"
