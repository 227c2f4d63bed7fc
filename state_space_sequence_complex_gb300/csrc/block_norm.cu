// Residual norm and its gradients (include/ssdc_block.h).
//
//   r = x + residual,  rstd = 1 / sqrt(mean(r^2) + eps),  y = r rstd w
//
// Bound by HBM. A row is read once and stays in registers between the sum of squares and
// the output: a lane holds 8 to 32 features (kVals), and up to 32 warps share a row. A
// lane's features are vectors of 16 bytes (bfloat16: 8, so that a group of 128 features is
// half a warp; fp32: 4, a whole one). Rows that do not start at multiples of 16 bytes, but at the
// same place in 16 bytes in every array, are held the same way from the multiple before their
// start on, shifted by up to 7 features: rows 8 apart are then shifted alike, so a CTA takes such
// rows. Other rows are held as single features 32 apart.
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
enum { kSingle, kAligned, kShifted };
template <typename T, int kAlign, int kVals>
struct Layout {
    static constexpr int kWarpSpan = 32 * kVals;  // features of a warp
    static constexpr int kRun = kAlign != kSingle ? 16 / (int)sizeof(T) : 1;
    static constexpr int kRuns = kVals / kRun;
    static __device__ __forceinline__ int run_at(int run, int lane) { return (run * 32 + lane) * kRun; }
};

// kRun values at a feature inside the row, as floats.
template <typename T, int kAlign>
__device__ __forceinline__ void load_run(const T* p, float* v) {
    if constexpr (kAlign == kSingle) {
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

// A shifted row's run from feature f on may begin before the row or end behind it: what of it lies
// inside is then loaded and stored singly, the rest is zeros and stays as it is.
template <int kRun>
__device__ __forceinline__ bool whole(int f, int D) { return f >= 0 && f + kRun <= D; }
template <typename T, int kAlign, int kRun>
__device__ __forceinline__ void load_part(const T* p, int f, int D, float* v) {
    if (kAlign != kShifted || whole<kRun>(f, D)) {
        load_run<T, kAlign>(p, v);
    } else {
#pragma unroll
        for (int e = 0; e < kRun; ++e) v[e] = f + e >= 0 && f + e < D ? to_f32(p[e]) : 0.0f;
    }
}
template <typename T, int kAlign, int kRun>
__device__ __forceinline__ void store_part(T* p, int f, int D, const float* v) {
    if (kAlign != kShifted || whole<kRun>(f, D)) {
        store_run<T, kRun>(p, v);
    } else {
#pragma unroll
        for (int e = 0; e < kRun; ++e)
            if (f + e >= 0 && f + e < D) p[e] = from_f32<T>(v[e]);
    }
}

// The weights as a shifted row's features lie, in shared memory.
__device__ __forceinline__ void shift_weights(float* to, const float* w, int shift, int D, int n) {
    for (int k = threadIdx.x; k < n; k += blockDim.x)
        to[k] = k < shift || k - shift >= D ? 0.0f : w ? __ldg(w + k - shift) : 1.0f;
    __syncthreads();
}

// kBy of the steps that take a warp's values from a shifted layout to the one from the row's start
// on: every value moves that many places towards the first. `next`: the first values of the
// row's next warp.
template <int kBy, int kRun, int kRuns>
__device__ __forceinline__ void move_down(float* v, float* next, int lane) {
#pragma unroll
    for (int i = 0; i < kRuns; ++i) {
        float in[kBy];
#pragma unroll
        for (int e = 0; e < kBy; ++e) {
            const float after = i + 1 < kRuns ? v[(i + 1) % kRuns * kRun + e] : next[e];
            in[e] = __shfl_sync(0xffffffffu, lane == 0 ? after : v[i * kRun + e], (lane + 1) % 32);
        }
#pragma unroll
        for (int e = 0; e < kRun - kBy; ++e) v[i * kRun + e] = v[i * kRun + e + kBy];
#pragma unroll
        for (int e = 0; e < kBy; ++e) v[i * kRun + kRun - kBy + e] = in[e];
    }
#pragma unroll
    for (int e = 0; e < kRun - kBy; ++e) next[e] = next[e + kBy];
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

// CTAs of the gradients' kernel an SM takes: two with rows copied ahead (96 KB of shared memory each), else
// as many as a lane's features leave registers for. (fp32, 16 features, two and three CTAs an SM of which two
// fit at a time: M 32768 D 1024 93 / 103 us, M 16384 D 1024 54 / 60 us, M 8192 D 4096 93 / 105 us.)
constexpr int bwd_ctas(int vals, int align) { return vals == 32 || align == kAligned ? 2 : vals == 16 ? 3 : 4; }

template <int kRowWarps>
constexpr int cta_warps() { return kRowWarps > 8 ? kRowWarps : 8; }

template <typename T, typename TO, bool kFp8, int kVals, int kRowWarps, int kAlign>
__global__ void __launch_bounds__(32 * cta_warps<kRowWarps>(), kRowWarps > 8 ? 1 : 4) norm_fwd(const Norm p) {
    using L = Layout<T, kAlign, kVals>;
    constexpr int kWarps = cta_warps<kRowWarps>(), kRun = L::kRun, kWarpSpan = L::kWarpSpan;
    constexpr int kRows = kWarps / kRowWarps;
    constexpr int kGroupRuns = kAlign != kSingle ? 1 : 4;              // runs of a lane in a group of 128
    constexpr int kGroupLanes = SSD_FP8_GROUP / (kRun * kGroupRuns);   // lanes that share a group
    __shared__ float part[1][32];
    constexpr bool kWeights = kAlign == kShifted && !kFp8, kMoved = kAlign == kShifted && kFp8;
    __shared__ __align__(16) float weights[kWeights ? kRowWarps * kWarpSpan : 4];
    __shared__ float firsts[kMoved ? kWarps + 1 : 1][8];
    launch_dependents();
    grid_dependency_wait();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t m = kAlign == kShifted ? ((int64_t)(blockIdx.x / 8) * kRows + warp / kRowWarps) * 8 + blockIdx.x % 8
                                         : (int64_t)blockIdx.x * kRows + warp / kRowWarps;
    const bool in = m < p.M;
    // (the same for all rows of the CTA)
    const int shift = kAlign == kShifted ? (int)(reinterpret_cast<uintptr_t>(static_cast<const T*>(p.x) + m * p.x_ld) / sizeof(T) % kRun) : 0;
    int base = warp % kRowWarps * kWarpSpan - shift;
    const T* x = static_cast<const T*>(p.x) + m * p.x_ld + base;
    const T* res = static_cast<const T*>(p.res) + m * p.res_ld + base;
    float v[kVals];
#pragma unroll
    for (int i = 0; i < L::kRuns; ++i) {
        const int at = L::run_at(i, lane);
#pragma unroll
        for (int e = 0; e < kRun; ++e) v[i * kRun + e] = 0.0f;
        if (in && base + at < p.D) load_part<T, kAlign, kRun>(x + at, base + at, p.D, v + i * kRun);
    }
    if (p.res) {
#pragma unroll
        for (int i = 0; i < L::kRuns; ++i) {
            const int at = L::run_at(i, lane);
            if (in && base + at < p.D) {
                float u[kRun];
                load_part<T, kAlign, kRun>(res + at, base + at, p.D, u);
#pragma unroll
                for (int e = 0; e < kRun; ++e) v[i * kRun + e] += u[e];
            }
        }
    }
    if constexpr (kWeights) shift_weights(weights, p.w, shift, p.D, kRowWarps * kWarpSpan);
    if constexpr (kMoved && kRowWarps > 1) {  // (there before the row's sum is)
        if (lane == 0)
#pragma unroll
            for (int e = 0; e < kRun; ++e) firsts[warp][e] = v[e];
    }
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < kVals; ++i) sq = fmaf(v[i], v[i], sq);
    sq = row_sum<kRowWarps>(sq, part, 0, warp);
    if (!in) return;
    const float rstd = rsqrt_refined(sq / (float)p.D + p.eps);
    if (p.rstd && lane == 0 && warp % kRowWarps == 0) p.rstd[m] = rstd;
    if (p.r) {
        T* r = static_cast<T*>(p.r) + m * p.r_ld + base;
#pragma unroll
        for (int i = 0; i < L::kRuns; ++i) {
            const int at = L::run_at(i, lane);
            if (base + at < p.D) store_part<T, kAlign, kRun>(r + at, base + at, p.D, v + i * kRun);
        }
    }
    if constexpr (kMoved) {
        // groups of 128 and 8-bit values count from the row's start
        float next[kRun];
#pragma unroll
        for (int e = 0; e < kRun; ++e) next[e] = kRowWarps > 1 && warp % kRowWarps + 1 < kRowWarps ? firsts[warp + 1][e] : 0.0f;
        if constexpr (kRun == 8)
            if (shift & 4) move_down<4, kRun, L::kRuns>(v, next, lane);
        if (shift & 2) move_down<2, kRun, L::kRuns>(v, next, lane);
        if (shift & 1) move_down<1, kRun, L::kRuns>(v, next, lane);
        base += shift;
    }
#pragma unroll
    for (int i0 = 0; i0 < L::kRuns; i0 += kGroupRuns) {
        float lo[kRun * kGroupRuns];  // what rounding the two products left out of y
        float amax = 0.0f;
#pragma unroll
        for (int i = i0; i < i0 + kGroupRuns; ++i) {
            const int at = L::run_at(i, lane);
            __align__(16) float w[kRun];
#pragma unroll
            for (int e = 0; e < kRun; ++e) w[e] = 1.0f;
            if constexpr (kWeights) {
#pragma unroll
                for (int e = 0; e < kRun; e += 4) *reinterpret_cast<float4*>(w + e) = *reinterpret_cast<const float4*>(weights + base + shift + at + e);
            } else if (p.w && base + at < p.D) {
                if (!kMoved || base + at + kRun <= p.D) load_w<kRun>(p.w + base + at, w);
                else
#pragma unroll
                    for (int e = 0; e < kRun; ++e) w[e] = base + at + e < p.D ? __ldg(p.w + base + at + e) : 0.0f;
            }
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
                store_part<TO, kAlign, kRun>(static_cast<TO*>(p.y) + m * p.y_ld + base + at, base + at, p.D, v + i * kRun);
        }
        if (kFp8) {
            amax = warp_max<kGroupLanes>(amax);
            const Scale s(amax);
            const int first = base + L::run_at(i0, lane);  // in the same group for all its lanes and runs
            if (lane % kGroupLanes == 0 && first < p.D) p.scale[(int64_t)(first / SSD_FP8_GROUP) * p.M + m] = s.s;
#pragma unroll
            for (int i = i0; i < i0 + kGroupRuns; ++i) {
                const int at = L::run_at(i, lane);
                float q[kRun];
#pragma unroll
                for (int e = 0; e < kRun; ++e) q[e] = s.quotient(v[i * kRun + e], lo[(i - i0) * kRun + e]);
                uint8_t* to = static_cast<uint8_t*>(p.y) + m * p.y_ld + base + at;
                if (kMoved ? base + at + kRun <= p.D : base + at < p.D) {
                    store_e4m3<kRun>(to, q);
                } else if (kMoved) {
#pragma unroll
                    for (int e = 0; e < kRun; ++e)
                        if (base + at + e < p.D) to[e] = e4m3(q[e]);
                }
            }
        }
    }
}

// Gradients. A warp walks rows kRows apart and adds up its share of dw in registers; the CTA's
// warps that hold the same features join theirs at the end, one row of `partial` a CTA. The next
// row is on its way meanwhile: into shared memory where it fits, each lane copying what it will
// itself read, else into L2.
template <typename T, int kVals, int kRowWarps, int kAlign>
constexpr int bwd_staging() {  // bytes: two rows of three arrays a warp
    constexpr int bytes = cta_warps<kRowWarps>() * 2 * 3 * 32 * kVals * (int)sizeof(T);
    return kAlign == kAligned && bytes <= 200 * 1024 || kAlign == kShifted && kRowWarps <= 2 ? bytes : 0;
}
template <typename T, int kVals, int kRowWarps, int kAlign>
constexpr int bwd_smem() {  // and, for shifted rows, the weights
    return bwd_staging<T, kVals, kRowWarps, kAlign>() + (kAlign == kShifted ? kRowWarps * 32 * kVals * 4 : 0);
}
template <typename T, int kVals, int kRowWarps, int kAlign>
__global__ void __launch_bounds__(32 * cta_warps<kRowWarps>(), kRowWarps > 8 ? 1 : bwd_ctas(kVals, kAlign)) norm_bwd(const NormBwd p) {
    using L = Layout<T, kAlign, kVals>;
    constexpr int kWarps = cta_warps<kRowWarps>(), kRun = L::kRun, kRows = kWarps / kRowWarps, kWarpSpan = L::kWarpSpan;
    __shared__ float part[2][32];
    __shared__ float join[kRows > 1 ? kWarps - kRowWarps : 1][kRows > 1 ? kWarpSpan / 4 : 1];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    // Rows: kRows at a time. Shifted ones are 8 apart, and gridDim.x is a multiple of 8.
    constexpr int kApart = kAlign == kShifted ? 8 : 1;
    const int64_t row0 = kAlign == kShifted ? (int64_t)(blockIdx.x / 8) * kRows * 8 + blockIdx.x % 8 : (int64_t)blockIdx.x * kRows;
    const int in_cta = warp / kRowWarps * kApart;
    const int shift = kAlign == kShifted ? (int)(reinterpret_cast<uintptr_t>(static_cast<const T*>(p.dy) + row0 * p.dy_ld) / sizeof(T) % kRun) : 0;
    const int base = warp % kRowWarps * kWarpSpan - shift;
    launch_dependents();
    grid_dependency_wait();
    float dw[kVals];
#pragma unroll
    for (int i = 0; i < kVals; ++i) dw[i] = 0.0f;
    constexpr int kStaging = bwd_staging<T, kVals, kRowWarps, kAlign>();
    constexpr bool kStaged = kStaging > 0;
    extern __shared__ __align__(16) char staged[];
    T* rows = reinterpret_cast<T*>(staged) + warp * 6 * kWarpSpan;
    float* weights = reinterpret_cast<float*>(staged + kStaging);
    auto fetch = [&](T* to, const T* from, int f) {
        if (kAlign != kShifted || whole<kRun>(f, p.D)) {
            ptx::cp_async_16(to, from);
        } else {
#pragma unroll
            for (int e = 0; e < kRun; ++e) to[e] = f + e >= 0 && f + e < p.D ? from[e] : from_f32<T>(0.0f);
        }
    };
    auto copy = [&](int64_t m, int stage) {  // this lane's runs of a row of dy, r and dr
        if (m < p.M)
#pragma unroll
            for (int i = 0; i < L::kRuns; ++i) {
                const int at = L::run_at(i, lane);
                if (base + at < p.D) {
                    T* to = rows + 3 * stage * kWarpSpan + at;
                    fetch(to, static_cast<const T*>(p.dy) + m * p.dy_ld + base + at, base + at);
                    fetch(to + kWarpSpan, static_cast<const T*>(p.r) + m * p.r_ld + base + at, base + at);
                    if (p.dr) fetch(to + 2 * kWarpSpan, static_cast<const T*>(p.dr) + m * p.dr_ld + base + at, base + at);
                }
            }
        ptx::cp_async_commit();
    };
    int slot = 0;
    float rstd_next = row0 + in_cta < p.M ? __ldg(p.rstd + row0 + in_cta) : 0.0f;
    if constexpr (kStaged) copy(row0 + in_cta, 0);
    if constexpr (kAlign == kShifted) shift_weights(weights, p.w, shift, p.D, kRowWarps * kWarpSpan);
    for (int64_t m0 = row0; m0 < p.M; m0 += (int64_t)gridDim.x * kRows, slot ^= 1) {
        const int64_t m = m0 + in_cta;
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
            const int ahead = lane * (128 / (int)sizeof(T)) + shift;
            if (m + next < p.M && ahead < kWarpSpan && base + ahead < p.D) {
                ptx::prefetch_l2(dy + next * p.dy_ld + ahead);
                ptx::prefetch_l2(r + next * p.r_ld + ahead);
                if (p.dr) ptx::prefetch_l2(dr + next * p.dr_ld + ahead);
            }
        }
        auto load = [&](const T* from, int f, float* to) {
            if constexpr (kStaged) load_run<T, kAlign>(from, to);
            else load_part<T, kAlign, kRun>(from, f, p.D, to);
        };
        float g[kVals], xh[kVals], s = 0.0f;
#pragma unroll
        for (int i = 0; i < L::kRuns; ++i) {
            const int at = L::run_at(i, lane);
#pragma unroll
            for (int e = 0; e < kRun; ++e) g[i * kRun + e] = xh[i * kRun + e] = 0.0f;
            if (in && base + at < p.D) {
                load(dy + at, base + at, g + i * kRun);
                load(r + at, base + at, xh + i * kRun);
            }
        }
#pragma unroll
        for (int i = 0; i < L::kRuns; ++i) {
            const int at = L::run_at(i, lane);
            __align__(16) float w[kRun];
#pragma unroll
            for (int e = 0; e < kRun; ++e) w[e] = 1.0f;
            if constexpr (kAlign == kShifted) {
#pragma unroll
                for (int e = 0; e < kRun; e += 4) *reinterpret_cast<float4*>(w + e) = *reinterpret_cast<const float4*>(weights + base + shift + at + e);
            } else if (p.w && base + at < p.D) {
                load_w<kRun>(p.w + base + at, w);
            }
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
                if (p.dr) load(dr + at, base + at, o);
#pragma unroll
                for (int e = 0; e < kRun; ++e) {
                    const int j = i * kRun + e;
                    o[e] = fmaf(rstd, fmaf(-xh[j], mean, g[j]), o[e]);
                }
                store_part<T, kAlign, kRun>(dx + at, base + at, p.D, o);
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
            for (int e = 0; e < kRun; ++e)
                if (kAlign != kShifted || (base + at + e >= 0 && base + at + e < p.D)) to[at + e] = dw[i * kRun + e];
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

// How the rows of a call's arrays lie: all from multiples of 16 bytes on; all from the same place in
// 16 bytes on, row by row; or otherwise.
struct Rows {
    size_t elem;
    bool start = true, alike = true;
    uintptr_t at = 0;
    int64_t ld = 0;
    bool any = false;
    void add(const void* q, int64_t q_ld) {
        if (q == nullptr) return;
        const uintptr_t a = reinterpret_cast<uintptr_t>(q) % 16;
        const int64_t l = q_ld % (int64_t)(16 / elem);
        start = start && a == 0 && l == 0;
        if (any) alike = alike && a == at && l == ld;
        any = true;
        at = a;
        ld = l;
    }
};
bool words16(const void* q) { return reinterpret_cast<uintptr_t>(q) % 16 == 0; }

// Features a lane holds, and warps of a row (a power of two). Rows in 16-byte loads: 32 bfloat16
// (M 32768 D 1024, 8-bit output: 44 us; 16: 52 us) or 16 fp32 (M 3001 D 1536: 12.6 us; 32: 14.8 us),
// which is four or eight loads under way. Rows in single loads: 8, for more warps to a row
// (M 3001 D 1537 fp32: 17 us; 32: 35 us). The widest rows need 32 either way.
int lane_vals(int64_t D, bool bf16, int align) {
    const int v = align == kSingle ? 8 : bf16 ? 32 : 16;
    return D <= 32 * 32 * v ? v : 32;
}
int row_warps(int64_t D, int vals) {
    int w = 1;
    while (w * 32 * vals < D) w *= 2;
    return w;
}
int64_t spread(int64_t D, bool bf16, int align) { return align == kShifted ? D + (bf16 ? 7 : 3) : D; }
// Rows that are held shifted: of up to 8 warps (their weights are in shared memory), that take no
// more lanes so than in single loads. Backward, bfloat16 (single / shifted): M 18000 D 901 63 / 49 us,
// M 10000 D 1601 86 / 41 us, M 4000 D 4001 132 / 58 us; but M 40000 D 417, in twice the lanes,
// 75 / 83 us. fp32: M 4000 D 3001 102 / 50 us, M 18000 D 901 66 / 73 us. Forward, bfloat16: to 8 bits
// M 10000 D 1601 56 / 49 us, M 4000 D 4001 51 / 42 us, but M 16384 D 1022 41 / 70 us, in twice the
// lanes; to bfloat16 M 4000 D 4001 36 / 39 us, and M 2000 D 5501, 32 warps in single loads, 52 /
// 35 us. fp32 forward M 4000 D 3001 41 / 45 us: in single loads.
bool may_shift(int64_t D, bool bf16) {
    const int vals = bf16 ? 32 : 16, w = row_warps(spread(D, bf16, kShifted), vals);
    return w <= 8 && w * vals == 8 * row_warps(D, 8);
}
bool shift_fwd(const Norm& p) { return p.bf16 && may_shift(p.D, true) && (p.out_type == SSD_TYPE_E4M3 || p.D > 4096); }
bool shift_bwd(int64_t D, bool bf16) { return may_shift(D, bf16) && (bf16 || D > 1024); }

// Calls f.template run<kVals, kRowWarps, kAlign>() for a row of D features. kLeast: the fewest warps
// of a shifted row (0: rows are not held so).
template <typename T, int kLeast, typename F>
void by_row(int64_t D, int align, const F& f) {
    const int vals = lane_vals(D, sizeof(T) == 2, align), w = row_warps(spread(D, sizeof(T) == 2, align), vals);
    auto warps = [&](auto v, auto al) {
        constexpr int kVals = decltype(v)::value, kAlign = decltype(al)::value;
        constexpr bool kWide = kVals == 32 && !(kAlign != kSingle && sizeof(T) == 2);  // taken for the widest rows only
        if constexpr (!kWide) {
            constexpr int kFrom = kAlign == kShifted ? kLeast : 1;
            if constexpr (kFrom <= 1) {
                if (w == 1) return f.template run<kVals, 1, kAlign>();
            }
            if constexpr (kFrom <= 2) {
                if (w == 2) return f.template run<kVals, 2, kAlign>();
            }
            if constexpr (kFrom <= 4) {
                if (w == 4) return f.template run<kVals, 4, kAlign>();
            }
            if (w == 8) return f.template run<kVals, 8, kAlign>();
        }
        if constexpr (kAlign != kShifted) {
            if constexpr (!kWide || kAlign == kSingle) {
                if (w <= 16) return f.template run<kVals, 16, kAlign>();
            }
            f.template run<kVals, 32, kAlign>();
        }
    };
    using std::integral_constant;
    constexpr int kOwn = sizeof(T) == 2 ? 32 : 16;
    if constexpr (kLeast > 0) {
        if (align == kShifted) return warps(integral_constant<int, kOwn>{}, integral_constant<int, kShifted>{});
    }
    if (align == kAligned && vals == kOwn) warps(integral_constant<int, kOwn>{}, integral_constant<int, kAligned>{});
    else if (align == kAligned) warps(integral_constant<int, 32>{}, integral_constant<int, kAligned>{});
    else if (vals == 8) warps(integral_constant<int, 8>{}, integral_constant<int, kSingle>{});
    else warps(integral_constant<int, 32>{}, integral_constant<int, kSingle>{});
}

template <typename T, typename TO, bool kFp8>
struct Fwd {
    const Norm& p;
    cudaStream_t stream;
    template <int kVals, int W, int kAlign>
    void run() const {
        constexpr int rows = cta_warps<W>() / W * (kAlign == kShifted ? 8 : 1), ctas = kAlign == kShifted ? 8 : 1;
        launch_dependent(norm_fwd<T, TO, kFp8, kVals, W, kAlign>, dim3((unsigned)((p.M + rows - 1) / rows * ctas)),
                         dim3(32 * cta_warps<W>()), 0, stream, p);
    }
};
template <typename T>
void fwd(const Norm& p, int align, cudaStream_t stream) {
    constexpr bool kHalf = sizeof(T) == 2;
    if (p.out_type == SSD_TYPE_E4M3) by_row<T, kHalf ? 1 : 0>(p.D, align, Fwd<T, T, true>{p, stream});
    else if (p.out_type == SSD_TYPE_BF16) by_row<T, kHalf ? 8 : 0>(p.D, align, Fwd<T, __nv_bfloat16, false>{p, stream});
    else by_row<T, 0>(p.D, align, Fwd<T, float, false>{p, stream});
}
template <typename T>
struct Bwd {
    const NormBwd& p;
    int ctas;
    cudaStream_t stream;
    template <int kVals, int W, int kAlign>
    void run() const {
        constexpr int smem = bwd_smem<T, kVals, W, kAlign>();
        auto* k = norm_bwd<T, kVals, W, kAlign>;
        static std::atomic<uint64_t> allowed;
        if (smem > 0 && allow_smem(k, smem, allowed) != cudaSuccess) return;  // (left for the caller to see)
        launch_dependent(k, dim3(ctas), dim3(32 * cta_warps<W>()), smem, stream, p);
    }
};

// The CTAs that walk the rows: as many as the SMs hold, fewer for few rows (M 4000 D 4000 bfloat16:
// 37 us with two an SM, 47 us with one). Those of shifted rows are a multiple of 8.
int bwd_parts(int64_t M, int64_t D, bool bf16, int align) {
    const int vals = lane_vals(D, bf16, align), w = row_warps(spread(D, bf16, align), vals), rows = w > 8 ? 1 : 8 / w;
    int64_t ctas = (M + rows - 1) / rows;
    if (align == kShifted) ctas = (M + 8 * rows - 1) / (8 * rows) * 8;
    const int64_t most = w > 8 ? 152 : 152 * bwd_ctas(vals, align);
    return (int)(ctas < most ? ctas : most);
}

}  // namespace

int norm_fwd_launch(const Norm& p, cudaStream_t stream) {
    const bool same = p.out_type == SSD_TYPE_BF16, fp8 = p.out_type == SSD_TYPE_E4M3;
    const size_t e = p.bf16 ? 2 : 4, eo = fp8 ? 1 : p.out_type == SSD_TYPE_F32 ? 4 : 2;
    Rows in{e}, out{eo};
    in.add(p.x, p.x_ld);
    in.add(p.res, p.res_ld);
    in.add(p.r, p.r_ld);
    out.add(p.y, p.y_ld);
    int align = kSingle;
    if (p.D % (16 / (int)e) == 0 && in.start && out.start && words16(p.w)) {
        align = kAligned;
    } else if (shift_fwd(p) && in.alike) {
        if (same) in.add(p.y, p.y_ld);
        if (same ? in.alike : fp8 && out.start && words16(p.w)) align = kShifted;
    }
    if (p.bf16) fwd<__nv_bfloat16>(p, align, stream);
    else fwd<float>(p, align, stream);
    return 1;
}

int norm_bwd_parts(int64_t M, int64_t D) {  // for any type and alignment
    int most = 0;
    for (int align : {kSingle, kAligned, kShifted})
        for (bool bf16 : {false, true}) {
            const int n = align == kShifted && !shift_bwd(D, bf16) ? 0 : bwd_parts(M, D, bf16, align);
            most = n > most ? n : most;
        }
    return most;
}

int norm_bwd_launch(const NormBwd& p, cudaStream_t stream) {
    Rows rows{(size_t)(p.bf16 ? 2 : 4)};
    rows.add(p.dy, p.dy_ld);
    rows.add(p.dr, p.dr_ld);
    rows.add(p.r, p.r_ld);
    rows.add(p.dx, p.dx_ld);
    int align = kSingle;
    if (p.D % (p.bf16 ? 8 : 4) == 0 && rows.start && words16(p.w)) align = kAligned;
    else if (shift_bwd(p.D, p.bf16) && rows.alike) align = kShifted;
    const int parts = bwd_parts(p.M, p.D, p.bf16, align);
    if (p.bf16) by_row<__nv_bfloat16, 1>(p.D, align, Bwd<__nv_bfloat16>{p, parts, stream});
    else by_row<float, 4>(p.D, align, Bwd<float>{p, parts, stream});
    if (!p.dw) return 1;
    if (launch_dependent(norm_bwd_sum, dim3((p.D + 31) / 32), dim3(32 * kSumWarps), 0, stream, (const float*)p.partial, p.dw, p.D, parts) !=
        cudaSuccess)
        return SSDC_ERR_CUDA;
    return 2;
}

}  // namespace block
}  // namespace ssdc
