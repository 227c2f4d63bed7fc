// 8-bit operands of a matrix (include/ssdc_block.h): e4m3 values with a scale for each row and
// 128 columns, or for each block of 128 x 128, as the matrix stands and transposed.
//
// A CTA reads a tile of 128 x 128 once, holds it in registers, and writes both operands' tiles.
// A thread owns kCols adjacent columns (one 16-byte load) of kRows adjacent rows, so that a group
// of 128 along a row is half a warp (bfloat16) or one (fp32), and the transposed tile's bytes go
// to shared memory kRows at a time: a column there is 128 bytes, its pieces exchanged by an
// exclusive or with the column's thread, which spreads both the writes by column and the reads by
// row over the banks.
//
// Measured, 32768 x 1024 bfloat16: row scales one way 20 us (5.0 TB/s), both ways 32 us (4.3 TB/s),
// a block's scale both ways 32 us; fp32 both ways 37 us (5.5 TB/s). Between memory and issue slots:
// 17 instructions a value both ways, nearly half of all slots, in two CTAs an SM. Quotients two at
// a time and one scale a lane took it from 35 us to 32; the next tile's loads ahead of this
// one's work, or three or four CTAs with fewer registers, gained nothing.
#include <cuda_runtime.h>

#include "block_common.cuh"
#include "block_kernels.h"
#include "ptx.cuh"
#include "ssdc_kernels.h"

namespace ssdc {
namespace block {

namespace {

constexpr int kThreads = 256, kTile = SSD_FP8_GROUP;

template <typename T, bool kBlocks, bool kAligned>
__global__ void __launch_bounds__(kThreads, 2) quantize(const Quant p) {
    constexpr int kCols = 16 / sizeof(T), kLanes = kTile / kCols, kRows = kTile * kLanes / kThreads;
    __shared__ __align__(16) uint8_t tile[kTile][kTile];
    __shared__ float col_max[kThreads / kLanes][kTile];
    __shared__ Scale col_scale[kTile];
    launch_dependents();
    grid_dependency_wait();
    const int t = threadIdx.x, lane = t % kLanes, strip = t / kLanes;  // columns kCols lane .., rows kRows strip ..
    const int64_t tiles_k = (p.K + kTile - 1) / kTile, tiles_m = (p.M + kTile - 1) / kTile;
    const int64_t tk = blockIdx.x % tiles_k, tm = blockIdx.x / tiles_k;
    const int64_t m0 = tm * kTile + strip * kRows, k0 = tk * kTile + lane * kCols;
    const int cols = (int)max((int64_t)0, min((int64_t)kCols, p.K - k0)), rows = (int)max((int64_t)0, min((int64_t)kRows, p.M - m0));
    float v[kRows][kCols];
    const T* x = static_cast<const T*>(p.x) + m0 * p.x_ld + k0;
    if (kAligned && rows == kRows && cols == kCols) {
        uint4 w[kRows];  // all on their way before the first is used
#pragma unroll
        for (int r = 0; r < kRows; ++r) w[r] = __ldg(reinterpret_cast<const uint4*>(x + r * p.x_ld));
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const uint32_t u[4] = {w[r].x, w[r].y, w[r].z, w[r].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (sizeof(T) == 2) {
                    v[r][2 * i] = ptx::bf16_lo(u[i]);
                    v[r][2 * i + 1] = ptx::bf16_hi(u[i]);
                } else {
                    v[r][i] = __uint_as_float(u[i]);
                }
            }
        }
    } else {
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int c = 0; c < kCols; ++c) v[r][c] = r < rows && c < cols ? to_f32(x[r * p.x_ld + c]) : 0.0f;
    }
    float row_amax[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        row_amax[r] = 0.0f;
#pragma unroll
        for (int c = 0; c < kCols; ++c) row_amax[r] = fmaxf(row_amax[r], fabsf(v[r][c]));
    }
    if (kBlocks) {
        float a = 0.0f;
#pragma unroll
        for (int r = 0; r < kRows; ++r) a = fmaxf(a, row_amax[r]);
        a = warp_max(a);
        if (t % 32 == 0) col_max[0][t / 32] = a;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) a = fmaxf(a, col_max[0][w]);
#pragma unroll
        for (int r = 0; r < kRows; ++r) row_amax[r] = a;
    }
    Scale mine;
    if (kBlocks) {
        mine = Scale(row_amax[0]);
        if (p.q && t == 0) p.scale[tm * tiles_k + tk] = mine.s;
    } else if (p.q) {
        // Each step leaves a lane half the rows, of twice the columns, so that each two lanes end
        // with one row's maximum (row lane / 2) and make its scale.
        int o = kLanes / 2;
#pragma unroll
        for (int n = kRows / 2; n > 0; n /= 2, o /= 2) {
            const bool upper = lane & o;
#pragma unroll
            for (int k = 0; k < n; ++k) {
                const float other = __shfl_xor_sync(0xffffffffu, upper ? row_amax[k] : row_amax[k + n], o);
                row_amax[k] = fmaxf(upper ? row_amax[k + n] : row_amax[k], other);
            }
        }
        mine = Scale(fmaxf(row_amax[0], __shfl_xor_sync(0xffffffffu, row_amax[0], 1)));
        if (lane % 2 == 0 && lane / 2 < rows) p.scale[tk * p.M + m0 + lane / 2] = mine.s;
    }
    if (p.q) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            Scale s = mine;
            if (!kBlocks) {
                s.s = __shfl_sync(0xffffffffu, mine.s, 2 * r, kLanes);
                s.inv = __shfl_sync(0xffffffffu, mine.inv, 2 * r, kLanes);
            }
            if (r < rows && cols > 0) {
                float q[kCols];
#pragma unroll
                for (int c = 0; c < kCols; c += 2) {
                    const float2 u = s.quotient(make_float2(v[r][c], v[r][c + 1]));
                    q[c] = u.x;
                    q[c + 1] = u.y;
                }
                uint8_t* to = p.q + (m0 + r) * p.q_ld + k0;
                if (cols == kCols) {
                    store_e4m3<kCols>(to, q);
                } else {
#pragma unroll
                    for (int c = 0; c < kCols; ++c)
                        if (c < cols) to[c] = e4m3(q[c]);
                }
            }
        }
    }
    if (!p.qt) return;
    Scale cs[kCols];
    if (kBlocks) {
#pragma unroll
        for (int c = 0; c < kCols; ++c) cs[c] = mine;
        if (t == 0) p.scale_t[tk * tiles_m + tm] = cs[0].s;
    } else {
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
            float a = 0.0f;
#pragma unroll
            for (int r = 0; r < kRows; ++r) a = fmaxf(a, fabsf(v[r][c]));
            col_max[strip][lane * kCols + c] = a;
        }
        __syncthreads();
        if (t < kTile) {  // one thread a column
            float a = 0.0f;
#pragma unroll
            for (int k = 0; k < kThreads / kLanes; ++k) a = fmaxf(a, col_max[k][t]);
            const Scale s(a);
            col_scale[t] = s;
            if (tk * kTile + t < p.K) p.scale_t[tm * p.K + tk * kTile + t] = s.s;
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < kCols; ++c) cs[c] = col_scale[lane * kCols + c];
    }
    // a column's kRows bytes as one piece; pieces of a column exchanged by the column's thread
    constexpr int kPieces = kTile / kRows;
#pragma unroll
    for (int c = 0; c < kCols; ++c) {
        float q[kRows];
#pragma unroll
        for (int r = 0; r < kRows; r += 2) {
            const float2 u = cs[c].quotient(make_float2(v[r][c], v[r + 1][c]));
            q[r] = u.x;
            q[r + 1] = u.y;
        }
        store_e4m3<kRows>(&tile[lane * kCols + c][(strip ^ (lane % kPieces)) * kRows], q);
    }
    __syncthreads();
    const int64_t mt = tm * kTile;
#pragma unroll
    for (int i = 0; i < kTile * kTile / 16 / kThreads; ++i) {
        const int at = i * kThreads + t, k = at / 8, j = at % 8;  // 16 bytes j of column k
        const int x = k / kCols % kPieces;
        uint4 w;
        if constexpr (kRows == 16) {
            w = *reinterpret_cast<const uint4*>(&tile[k][(j ^ x) * 16]);
        } else {
            w = *reinterpret_cast<const uint4*>(&tile[k][((2 * j ^ x) & ~1) * 8]);
            if (x & 1) w = make_uint4(w.z, w.w, w.x, w.y);
        }
        const int64_t row = tk * kTile + k, m = mt + 16 * j;
        if (row < p.K && m < p.M) {
            uint8_t* to = p.qt + row * p.qt_ld + m;
            if (m + 16 <= p.M) {
                *reinterpret_cast<uint4*>(to) = w;
            } else {
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (m + e < p.M) to[e] = (uint8_t)(u[e / 4] >> (8 * (e % 4)));
            }
        }
    }
}

template <typename T, bool kBlocks>
void launch(const Quant& p, bool aligned, unsigned grid, cudaStream_t stream) {
    launch_dependent(aligned ? quantize<T, kBlocks, true> : quantize<T, kBlocks, false>, dim3(grid), dim3(kThreads), 0, stream, p);
}

}  // namespace

int quantize_launch(const Quant& p, cudaStream_t stream) {
    const int64_t tiles = ((p.K + kTile - 1) / kTile) * ((p.M + kTile - 1) / kTile);
    if (tiles > INT32_MAX) return SSDC_ERR_UNSUPPORTED;
    const size_t e = p.bf16 ? 2 : 4;
    const bool aligned = reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && p.x_ld * (int64_t)e % 16 == 0;
    const unsigned grid = (unsigned)tiles;
    if (p.bf16) p.blocks ? launch<__nv_bfloat16, true>(p, aligned, grid, stream) : launch<__nv_bfloat16, false>(p, aligned, grid, stream);
    else p.blocks ? launch<float, true>(p, aligned, grid, stream) : launch<float, false>(p, aligned, grid, stream);
    return 1;
}

}  // namespace block
}  // namespace ssdc
