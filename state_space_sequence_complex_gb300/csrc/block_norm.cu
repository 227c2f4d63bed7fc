// Residual norm and its gradients (include/ssdc_block.h).
//
//   r = x + residual,  rstd = 1 / sqrt(mean(r^2) + eps),  y = r rstd w
//
// Bound by HBM. A row is read once and stays in registers between the sum of squares and
// the output: a lane holds 8 to 32 features (kVals), and up to 32 warps share a row. A
// lane's features are vectors of 16 bytes (bfloat16: 8, so that a group of 128 features is
// half a warp; fp32: 4, a whole one), or, for rows that do not start at multiples of 16
// bytes, single features 32 apart.
//
// Measured: M 32768 D 1024 bfloat16 to 8 bits with a residual 41 us (5.7 TB/s), gradients 53 us
// (5.0 TB/s, the sum of dw's shares in it); M 3001 D 1537 fp32 16 us (4.6 TB/s, half of it in L2).
#include <type_traits>

#include <cuda_runtime.h>

#include "block_common.cuh"
#include "block_kernels.h"
#include "ptx.cuh"
#include "ssdc_kernels.h"

namespace ssdc {
namespace block {

namespace {

// Which features a lane holds: value i of lane l is feature base + at(i, l). A run is kRun
// adjacent features, one load.
template <typename T, bool kAligned, int kVals>
struct Layout {
    static constexpr int kWarpSpan = 32 * kVals;  // features of a warp
    static constexpr int kRun = kAligned ? 16 / (int)sizeof(T) : 1;
    static constexpr int kRuns = kVals / kRun;
    static constexpr int kGroupRuns = kAligned ? 1 : 4;              // runs of a lane in a group of 128
    static constexpr int kGroupLanes = 128 / (kRun * kGroupRuns);    // lanes that share a group
    static __device__ __forceinline__ int run_at(int run, int lane) { return (run * 32 + lane) * kRun; }
};

// kRun values at a feature inside the row, as floats.
template <typename T, bool kAligned>
__device__ __forceinline__ void load_run(const T* p, float* v) {
    if constexpr (!kAligned) {
        v[0] = to_f32(*p);
    } else if constexpr (sizeof(T) == 2) {
        const uint4 w = *reinterpret_cast<const uint4*>(p);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = ptx::bf16_lo(u[i]);
            v[2 * i + 1] = ptx::bf16_hi(u[i]);
        }
    } else {
        const float4 w = *reinterpret_cast<const float4*>(p);
        v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
    }
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&t);
}
// kN values to an array of T (kN is a run of the input's type; the output's may be another).
template <typename T, int kN>
__device__ __forceinline__ void store_run(T* p, const float* v) {
    if constexpr (kN == 1) {
        *p = from_f32<T>(v[0]);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < kN; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    } else if constexpr (kN == 8) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                                  pack_bf16(v[6], v[7]));
    } else {
        *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    }
}
template <int kN>
__device__ __forceinline__ void load_w(const float* w, float* v) {
    if constexpr (kN == 1) {
        v[0] = __ldg(w);
    } else {
#pragma unroll
        for (int i = 0; i < kN; i += 4) {
            const float4 t = __ldg(reinterpret_cast<const float4*>(w + i));
            v[i] = t.x; v[i + 1] = t.y; v[i + 2] = t.z; v[i + 3] = t.w;
        }
    }
}

// 1 / sqrt(m) to within a unit of its last place: the hardware's approximation and one step of
// Newton's method, the residual 1 - m y^2 formed with the product's rounding error.
__device__ __forceinline__ float rsqrt_refined(float m) {
    const float y = rsqrtf(m), h = m * y, l = fmaf(m, y, -h);
    const float e = fmaf(-h, y, 1.0f) - l * y;
    const float r = fmaf(0.5f * y, e, y);
    return isfinite(r) ? r : y;  // (m infinite or zero)
}

// The sum over the warps of a row (`row` of the CTA's kRows, kRowWarps each); every warp of the
// CTA takes part. `slot` alternates between calls.
template <int kRowWarps>
__device__ __forceinline__ float row_sum(float v, float (*part)[32], int slot, int warp) {
    v = warp_sum(v);
    if constexpr (kRowWarps == 1) return v;
    if (threadIdx.x % 32 == 0) part[slot][warp] = v;
    __syncthreads();
    float s = 0.0f;
    const int first = warp / kRowWarps * kRowWarps;
#pragma unroll
    for (int k = 0; k < kRowWarps; ++k) s += part[slot][first + k];
    return s;
}

// CTAs of the gradients' kernel an SM takes (its registers), by a lane's features.
constexpr int bwd_ctas(int vals) { return vals == 32 ? 2 : vals == 16 ? 3 : 4; }

template <int kRowWarps>
constexpr int cta_warps() { return kRowWarps > 8 ? kRowWarps : 8; }

template <typename T, typename TO, bool kFp8, int kVals, int kRowWarps, bool kAligned>
__global__ void __launch_bounds__(32 * cta_warps<kRowWarps>(), kRowWarps > 8 ? 1 : 4) norm_fwd(const Norm p) {
    using L = Layout<T, kAligned, kVals>;
    constexpr int kWarps = cta_warps<kRowWarps>(), kRun = L::kRun, kWarpSpan = L::kWarpSpan;
    __shared__ float part[1][32];
    launch_dependents();
    grid_dependency_wait();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t m = (int64_t)blockIdx.x * (kWarps / kRowWarps) + warp / kRowWarps;
    const int base = warp % kRowWarps * kWarpSpan;
    const bool in = m < p.M;
    const T* x = static_cast<const T*>(p.x) + m * p.x_ld + base;
    const T* res = static_cast<const T*>(p.res) + m * p.res_ld + base;
    float v[kVals];
#pragma unroll
    for (int i = 0; i < L::kRuns; ++i) {
        const int at = L::run_at(i, lane);
#pragma unroll
        for (int e = 0; e < kRun; ++e) v[i * kRun + e] = 0.0f;
        if (in && base + at < p.D) load_run<T, kAligned>(x + at, v + i * kRun);
    }
    if (p.res) {
#pragma unroll
        for (int i = 0; i < L::kRuns; ++i) {
            const int at = L::run_at(i, lane);
            if (in && base + at < p.D) {
                float u[kRun];
                load_run<T, kAligned>(res + at, u);
#pragma unroll
                for (int e = 0; e < kRun; ++e) v[i * kRun + e] += u[e];
            }
        }
    }
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < kVals; ++i) sq = fmaf(v[i], v[i], sq);
    sq = row_sum<kRowWarps>(sq, part, 0, warp);
    if (!in) return;
    const float rstd = rsqrt_refined(sq / (float)p.D + p.eps);
    if (p.rstd && lane == 0 && base == 0) p.rstd[m] = rstd;
    if (p.r) {
        T* r = static_cast<T*>(p.r) + m * p.r_ld + base;
#pragma unroll
        for (int i = 0; i < L::kRuns; ++i) {
            const int at = L::run_at(i, lane);
            if (base + at < p.D) store_run<T, kRun>(r + at, v + i * kRun);
        }
    }
#pragma unroll
    for (int i0 = 0; i0 < L::kRuns; i0 += L::kGroupRuns) {
        float lo[kRun * L::kGroupRuns];  // what rounding the two products left out of y
        float amax = 0.0f;
#pragma unroll
        for (int i = i0; i < i0 + L::kGroupRuns; ++i) {
            const int at = L::run_at(i, lane);
            float w[kRun];
#pragma unroll
            for (int e = 0; e < kRun; ++e) w[e] = 1.0f;
            if (p.w && base + at < p.D) load_w<kRun>(p.w + base + at, w);
#pragma unroll
            for (int e = 0; e < kRun; ++e) {
                float& t = v[i * kRun + e];
                const float n = t * rstd, y = n * w[e];
                if (kFp8) {
                    lo[(i - i0) * kRun + e] = fmaf(fmaf(t, rstd, -n), w[e], fmaf(n, w[e], -y));
                    amax = fmaxf(amax, fabsf(y));
                }
                t = y;
            }
            if (!kFp8 && base + at < p.D)
                store_run<TO, kRun>(static_cast<TO*>(p.y) + m * p.y_ld + base + at, v + i * kRun);
        }
        if (kFp8) {
            amax = warp_max<L::kGroupLanes>(amax);
            const Scale s(amax);
            const int first = base + L::run_at(i0, lane);  // in the same group for all its lanes and runs
            if (lane % L::kGroupLanes == 0 && first < p.D) p.scale[(int64_t)(first / SSD_FP8_GROUP) * p.M + m] = s.s;
#pragma unroll
            for (int i = i0; i < i0 + L::kGroupRuns; ++i) {
                const int at = L::run_at(i, lane);
                float q[kRun];
#pragma unroll
                for (int e = 0; e < kRun; ++e) q[e] = s.quotient(v[i * kRun + e], lo[(i - i0) * kRun + e]);
                if (base + at < p.D) store_e4m3<kRun>(static_cast<uint8_t*>(p.y) + m * p.y_ld + base + at, q);
            }
        }
    }
}

// Gradients. A warp walks rows kRows apart and adds up its share of dw in registers; the CTA's
// warps that hold the same features join theirs at the end, one row of `partial` a CTA. The next
// row is on its way meanwhile: into shared memory where it fits, each lane copying what it will
// itself read, else into L2.
template <typename T, int kVals, int kRowWarps, bool kAligned>
constexpr int bwd_smem() {  // two rows of three arrays a warp
    constexpr int bytes = cta_warps<kRowWarps>() * 2 * 3 * 32 * kVals * (int)sizeof(T);
    return kAligned && bytes <= 200 * 1024 ? bytes : 0;
}
template <typename T, int kVals, int kRowWarps, bool kAligned>
__global__ void __launch_bounds__(32 * cta_warps<kRowWarps>(), kRowWarps > 8 ? 1 : bwd_ctas(kVals)) norm_bwd(const NormBwd p) {
    using L = Layout<T, kAligned, kVals>;
    constexpr int kWarps = cta_warps<kRowWarps>(), kRun = L::kRun, kRows = kWarps / kRowWarps, kWarpSpan = L::kWarpSpan;
    __shared__ float part[2][32];
    __shared__ float join[kRows > 1 ? kWarps - kRowWarps : 1][kRows > 1 ? kWarpSpan / 4 : 1];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int base = warp % kRowWarps * kWarpSpan;
    launch_dependents();
    grid_dependency_wait();
    float dw[kVals];
#pragma unroll
    for (int i = 0; i < kVals; ++i) dw[i] = 0.0f;
    constexpr bool kStaged = bwd_smem<T, kVals, kRowWarps, kAligned>() > 0;
    extern __shared__ __align__(16) char staged[];
    T* rows = reinterpret_cast<T*>(staged) + warp * 6 * kWarpSpan;
    auto copy = [&](int64_t m, int stage) {  // this lane's runs of a row of dy, r and dr
        if (m < p.M)
#pragma unroll
            for (int i = 0; i < L::kRuns; ++i) {
                const int at = L::run_at(i, lane);
                if (base + at < p.D) {
                    T* to = rows + 3 * stage * kWarpSpan + at;
                    ptx::cp_async_16(to, static_cast<const T*>(p.dy) + m * p.dy_ld + base + at);
                    ptx::cp_async_16(to + kWarpSpan, static_cast<const T*>(p.r) + m * p.r_ld + base + at);
                    if (p.dr) ptx::cp_async_16(to + 2 * kWarpSpan, static_cast<const T*>(p.dr) + m * p.dr_ld + base + at);
                }
            }
        ptx::cp_async_commit();
    };
    int slot = 0;
    float rstd_next = (int64_t)blockIdx.x * kRows + warp / kRowWarps < p.M ? __ldg(p.rstd + (int64_t)blockIdx.x * kRows + warp / kRowWarps) : 0.0f;
    if constexpr (kStaged) copy((int64_t)blockIdx.x * kRows + warp / kRowWarps, 0);
    for (int64_t m0 = (int64_t)blockIdx.x * kRows; m0 < p.M; m0 += (int64_t)gridDim.x * kRows, slot ^= 1) {
        const int64_t m = m0 + warp / kRowWarps;
        const bool in = m < p.M;
        const T* dy = static_cast<const T*>(p.dy) + m * p.dy_ld + base;
        const T* r = static_cast<const T*>(p.r) + m * p.r_ld + base;
        const T* dr = static_cast<const T*>(p.dr) + m * p.dr_ld + base;
        const int64_t next = (int64_t)gridDim.x * kRows;
        const float rstd = rstd_next;
        rstd_next = m + next < p.M ? __ldg(p.rstd + m + next) : 0.0f;
        if constexpr (kStaged) {
            copy(m + next, slot ^ 1);
            ptx::cp_async_wait<1>();
            dy = rows + 3 * slot * kWarpSpan;
            r = dy + kWarpSpan;
            dr = r + kWarpSpan;
        } else {  // a lane a line of each array
            const int ahead = lane * (128 / (int)sizeof(T));
            if (m + next < p.M && ahead < kWarpSpan && base + ahead < p.D) {
                ptx::prefetch_l2(dy + next * p.dy_ld + ahead);
                ptx::prefetch_l2(r + next * p.r_ld + ahead);
                if (p.dr) ptx::prefetch_l2(dr + next * p.dr_ld + ahead);
            }
        }
        float g[kVals], xh[kVals], s = 0.0f;
#pragma unroll
        for (int i = 0; i < L::kRuns; ++i) {
            const int at = L::run_at(i, lane);
#pragma unroll
            for (int e = 0; e < kRun; ++e) g[i * kRun + e] = xh[i * kRun + e] = 0.0f;
            if (in && base + at < p.D) {
                load_run<T, kAligned>(dy + at, g + i * kRun);
                load_run<T, kAligned>(r + at, xh + i * kRun);
            }
        }
#pragma unroll
        for (int i = 0; i < L::kRuns; ++i) {
            const int at = L::run_at(i, lane);
            float w[kRun];
#pragma unroll
            for (int e = 0; e < kRun; ++e) w[e] = 1.0f;
            if (p.w && base + at < p.D) load_w<kRun>(p.w + base + at, w);
#pragma unroll
            for (int e = 0; e < kRun; ++e) {
                const int j = i * kRun + e;
                xh[j] *= rstd;
                dw[j] = fmaf(g[j], xh[j], dw[j]);
                g[j] *= w[e];
                s = fmaf(g[j], xh[j], s);
            }
        }
        const float mean = row_sum<kRowWarps>(s, part, slot, warp) / (float)p.D;
        if (!in) continue;
        T* dx = static_cast<T*>(p.dx) + m * p.dx_ld + base;
#pragma unroll
        for (int i = 0; i < L::kRuns; ++i) {
            const int at = L::run_at(i, lane);
            if (base + at < p.D) {
                float o[kRun];
#pragma unroll
                for (int e = 0; e < kRun; ++e) o[e] = 0.0f;
                if (p.dr) load_run<T, kAligned>(dr + at, o);
#pragma unroll
                for (int e = 0; e < kRun; ++e) {
                    const int j = i * kRun + e;
                    o[e] = fmaf(rstd, fmaf(-xh[j], mean, g[j]), o[e]);
                }
                store_run<T, kRun>(dx + at, o);
            }
        }
    }
    if (!p.dw) return;
    float* to = p.partial + (int64_t)blockIdx.x * p.D + base;
    if constexpr (kRows > 1) {
        // a quarter of the lanes' values at a time, so that the rows' shares fit into shared memory
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            __syncthreads();
            if (warp >= kRowWarps)
#pragma unroll
                for (int i = 0; i < kVals / 4; ++i) join[warp - kRowWarps][i * 32 + lane] = dw[q * (kVals / 4) + i];
            __syncthreads();
            if (warp < kRowWarps)
#pragma unroll
                for (int i = 0; i < kVals / 4; ++i)
                    for (int k = 1; k < kRows; ++k) dw[q * (kVals / 4) + i] += join[k * kRowWarps + warp - kRowWarps][i * 32 + lane];
        }
        if (warp >= kRowWarps) return;
    }
#pragma unroll
    for (int i = 0; i < L::kRuns; ++i) {
        const int at = L::run_at(i, lane);
        if (base + at < p.D)
#pragma unroll
            for (int e = 0; e < kRun; ++e) to[at + e] = dw[i * kRun + e];
    }
}

// dw from the CTAs' shares, in a fixed order: a CTA sums 32 features, each of its warps its part of
// the shares, with all loads under way at once (304 shares: 10 a warp).
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(32 * kSumWarps) norm_bwd_sum(const float* partial, float* dw, int D, int parts) {
    __shared__ float join[kSumWarps][32];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, d = blockIdx.x * 32 + lane;
    grid_dependency_wait();
    float s = 0.0f;
    const int per = (parts + kSumWarps - 1) / kSumWarps;
    if (d < D) {
#pragma unroll 10
        for (int k = warp * per; k < min((warp + 1) * per, parts); ++k) s += partial[(int64_t)k * D + d];
    }
    join[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && d < D) {
        s = 0.0f;
#pragma unroll
        for (int k = 0; k < kSumWarps; ++k) s += join[k][lane];
        dw[d] = s;
    }
}

bool rows16(const void* q, int64_t ld, size_t elem) {
    return q == nullptr || (reinterpret_cast<uintptr_t>(q) % 16 == 0 && ld * (int64_t)elem % 16 == 0);
}

// Features a lane holds, and warps of a row (a power of two). Rows in 16-byte loads: 32 bfloat16
// (M 32768 D 1024, 8-bit output: 44 us; 16: 52 us) or 16 fp32 (M 3001 D 1536: 12.6 us; 32: 14.8 us),
// which is four or eight loads under way. Rows in single loads: 8, for more warps to a row
// (M 3001 D 1537 fp32: 17 us; 32: 35 us). The widest rows need 32 either way.
int lane_vals(int64_t D, bool bf16, bool aligned) {
    const int v = !aligned ? 8 : bf16 ? 32 : 16;
    return D <= 32 * 32 * v ? v : 32;
}
int row_warps(int64_t D, int vals) {
    int w = 1;
    while (w * 32 * vals < D) w *= 2;
    return w;
}

// Calls f.template operator()<kVals, kRowWarps, kAligned>() for a row of D features.
template <typename T, typename F>
void by_row(int64_t D, bool aligned, const F& f) {
    const int vals = lane_vals(D, sizeof(T) == 2, aligned), w = row_warps(D, vals);
    auto warps = [&](auto v, auto al) {
        constexpr int kVals = decltype(v)::value;
        constexpr bool kAligned = decltype(al)::value;
        constexpr bool kWide = kVals == 32 && !(kAligned && sizeof(T) == 2);  // taken for the widest rows only
        if constexpr (!kWide) {
            switch (w) {
                case 1: return f.template run<kVals, 1, kAligned>();
                case 2: return f.template run<kVals, 2, kAligned>();
                case 4: return f.template run<kVals, 4, kAligned>();
                case 8: return f.template run<kVals, 8, kAligned>();
                default: break;
            }
        }
        if constexpr (!kWide || !kAligned) {
            if (w <= 16) return f.template run<kVals, 16, kAligned>();
        }
        f.template run<kVals, 32, kAligned>();
    };
    using std::integral_constant;
    constexpr int kOwn = sizeof(T) == 2 ? 32 : 16;
    if (aligned && vals == kOwn) warps(integral_constant<int, kOwn>{}, std::true_type{});
    else if (aligned) warps(integral_constant<int, 32>{}, std::true_type{});
    else if (vals == 8) warps(integral_constant<int, 8>{}, std::false_type{});
    else warps(integral_constant<int, 32>{}, std::false_type{});
}

template <typename T, typename TO, bool kFp8>
struct Fwd {
    const Norm& p;
    cudaStream_t stream;
    template <int kVals, int W, bool kAligned>
    void run() const {
        constexpr int rows = cta_warps<W>() / W;
        launch_dependent(norm_fwd<T, TO, kFp8, kVals, W, kAligned>, dim3((unsigned)((p.M + rows - 1) / rows)),
                         dim3(32 * cta_warps<W>()), 0, stream, p);
    }
};
template <typename T>
void fwd(const Norm& p, bool aligned, cudaStream_t stream) {
    if (p.out_type == SSD_TYPE_E4M3) by_row<T>(p.D, aligned, Fwd<T, T, true>{p, stream});
    else if (p.out_type == SSD_TYPE_BF16) by_row<T>(p.D, aligned, Fwd<T, __nv_bfloat16, false>{p, stream});
    else by_row<T>(p.D, aligned, Fwd<T, float, false>{p, stream});
}
template <typename T>
struct Bwd {
    const NormBwd& p;
    int ctas;
    cudaStream_t stream;
    template <int kVals, int W, bool kAligned>
    void run() const {
        constexpr int smem = bwd_smem<T, kVals, W, kAligned>();
        auto* k = norm_bwd<T, kVals, W, kAligned>;
        static std::atomic<uint64_t> allowed;
        if (smem > 0 && allow_smem(k, smem, allowed) != cudaSuccess) return;  // (left for the caller to see)
        launch_dependent(k, dim3(ctas), dim3(32 * cta_warps<W>()), smem, stream, p);
    }
};

// The CTAs that walk the rows: as many as the SMs hold, fewer for few rows and (their shares of dw
// being written and read again) for wide ones.
int bwd_parts(int64_t M, int64_t D, bool bf16, bool aligned) {
    const int vals = lane_vals(D, bf16, aligned), w = row_warps(D, vals), rows = w > 8 ? 1 : 8 / w;
    const int64_t ctas = (M + rows - 1) / rows, most = D <= 2048 ? 152 * bwd_ctas(vals) : 152;
    return (int)(ctas < most ? ctas : most);
}

}  // namespace

int norm_fwd_launch(const Norm& p, cudaStream_t stream) {
    const size_t e = p.bf16 ? 2 : 4, eo = p.out_type == SSD_TYPE_F32 ? 4 : p.out_type == SSD_TYPE_BF16 ? 2 : 1;
    const bool aligned = p.D % (16 / (int)e) == 0 && rows16(p.x, p.x_ld, e) && rows16(p.res, p.res_ld, e) &&
                         rows16(p.r, p.r_ld, e) && rows16(p.y, p.y_ld, eo) && rows16(p.w, 0, 4);
    if (p.bf16) fwd<__nv_bfloat16>(p, aligned, stream);
    else fwd<float>(p, aligned, stream);
    return 1;
}

int norm_bwd_parts(int64_t M, int64_t D) {  // for any type and alignment
    int most = 0;
    for (int k = 0; k < 4; ++k) {
        const int n = bwd_parts(M, D, (k & 1) != 0, (k & 2) != 0);
        most = n > most ? n : most;
    }
    return most;
}

int norm_bwd_launch(const NormBwd& p, cudaStream_t stream) {
    const size_t e = p.bf16 ? 2 : 4;
    const bool aligned = p.D % (16 / (int)e) == 0 && rows16(p.dy, p.dy_ld, e) && rows16(p.dr, p.dr_ld, e) &&
                         rows16(p.r, p.r_ld, e) && rows16(p.dx, p.dx_ld, e) && rows16(p.w, 0, 4);
    const int parts = bwd_parts(p.M, p.D, p.bf16, aligned);
    if (p.bf16) by_row<__nv_bfloat16>(p.D, aligned, Bwd<__nv_bfloat16>{p, parts, stream});
    else by_row<float>(p.D, aligned, Bwd<float>{p, parts, stream});
    if (!p.dw) return 1;
    if (launch_dependent(norm_bwd_sum, dim3((p.D + 31) / 32), dim3(32 * kSumWarps), 0, stream, (const float*)p.partial, p.dw, p.D, parts) !=
        cudaSuccess)
        return SSDC_ERR_CUDA;
    return 2;
}

}  // namespace block
}  // namespace ssdc
