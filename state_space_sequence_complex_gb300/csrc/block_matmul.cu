// 8-bit product (include/ssdc_block.h): C[m, n] = sum over groups g of 128 columns of
// a_scale[g][m] b_scale[g, n] sum_{k in g} A[m, k] B[n, k].
//
// The inner sums are e4m3 matrix products on the tensor cores. Their scales differ from
// group to group, so the sum over groups cannot stay in the tensor memory: each group's
// product is read back, scaled and added in fp32 registers while the next group's is being
// computed (two tensor-memory buffers).
//
// A pair of CTAs works on a tile of 256 rows x BN columns (cta_group::2): each CTA
// stages half of A's rows and half of B's, which halves the operand bytes an SM takes in
// for its part of the product. Roles: warp 0 loads (TMA, a ring of stages of one group),
// warps 1 and 2 of the even CTA issue the MMAs of every other group, warp 3 fetches the
// scales, warps 4 .. 19 scale, add and store; each of those owns 32 rows x BN / 4 columns in registers, and takes registers that the first
// four warps give up. (The issue of an MMA returns shortly before it is done, so a single
// issuer's waits between two groups left the tensor cores idle for as long as they worked.)
#include <cuda.h>
#include <cuda_runtime.h>

#include "block_common.cuh"
#include "block_kernels.h"
#include "ptx.cuh"
#include "ssdc_kernels.h"
#include "tc_common.cuh"

namespace ssdc {
namespace block {

namespace {

constexpr uint64_t kWaitNs = 2000000000ull;  // wait limit
constexpr int kAddWarps = 16, kThreads = 128 + 32 * kAddWarps;
// Registers a thread: 96 x 640 = 61440 at launch, 56 x 128 + 104 x 512 = 60416 after the split
constexpr int kCtlRegs = 56, kAddRegs = 104;
constexpr int kGroup = SSD_FP8_GROUP;

struct Product {
    const float *a_scale, *b_scale;
    int64_t M, N, c_ld;
    int KB, m_tiles, n_tiles;
    void* c;
    bool aligned;  // every row of c starts at a multiple of 32 bytes
    int* status;
};

// Tiles are walked in bands of 8 row tiles, so that the pairs at work at one time share
// both operands' tiles in L2.
constexpr int kBand = 8;
__device__ __forceinline__ void tile_at(const Product& p, int idx, int& mt, int& nt) {
    const int band = idx / (kBand * p.n_tiles), first = band * kBand;
    const int rows = min(kBand, p.m_tiles - first), in = idx - band * kBand * p.n_tiles;
    nt = in / rows;
    mt = first + in % rows;
}

template <int BN>
struct Shape {
    static constexpr uint32_t kA = 128 * kGroup, kB = BN / 2 * kGroup, kStage = kA + kB;
    static constexpr int kCols = BN / 4;  // columns of one warp
    // Scales, a ring of groups: 128 rows' for each of B's two blocks (already multiplied), or 128
    // rows' and then the columns'
    static constexpr int kRing = 8, kSlot = 128 + 256;
    static constexpr uint32_t kScales = kRing * kSlot * 4;
    // per adding warp: 32 rows of 32 values of C, a bank apart, for rows that start unaligned
    static constexpr uint32_t kOut = 32 * 33 * 4;
    static constexpr int kStages = BN == 256 ? 4 : 5;
    static constexpr uint32_t kBytes = 1024 + kStages * kStage + kScales + kAddWarps * kOut;
};

// 32 consecutive values of each of a warp's 32 rows to C, one row a lane. Rows aligned to
// 32 bytes take whole sectors straight from registers; others go through shared memory, a
// row at a time. Columns from n on; rows and columns outside C are left out.
template <typename T>
__device__ __forceinline__ void store_rows(const Product& p, char* stage, const float2* v, int64_t m0, int64_t n, int lane) {
    T* c = static_cast<T*>(p.c) + n;
    const int cols = (int)min((int64_t)32, p.N - n), rows = (int)min((int64_t)32, p.M - m0);
    if (p.aligned && cols == 32) {
        if (lane < rows) {
            T* to = c + (m0 + lane) * p.c_ld;
            if constexpr (sizeof(T) == 2) {
#pragma unroll
                for (int e = 0; e < 32; e += 16) {
                    uint32_t w[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const __nv_bfloat162 t = __float22bfloat162_rn(v[e / 2 + k]);
                        w[k] = *reinterpret_cast<const uint32_t*>(&t);
                    }
                    ptx::st_global_v8(to + e, w);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    uint32_t w[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) w[k] = __float_as_uint(k & 1 ? v[(e + k) / 2].y : v[(e + k) / 2].x);
                    ptx::st_global_v8(to + e, w);
                }
            }
        }
    } else {
        float* st = reinterpret_cast<float*>(stage);
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            st[lane * 33 + 2 * e] = v[e].x;
            st[lane * 33 + 2 * e + 1] = v[e].y;
        }
        __syncwarp();
        if (lane < cols)
            for (int r = 0; r < rows; ++r) c[(m0 + r) * p.c_ld + lane] = from_f32<T>(st[r * 33 + lane]);
    }
}

template <int BN, bool kBlocks, typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
product_pair(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, const Product p) {
    using S = Shape<BN>;
    extern __shared__ char smem_raw[];
    char* smem = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t full[S::kStages], empty[S::kStages], tfull[2], tempty[2];
    __shared__ uint32_t tmem_slot;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = ptx::cluster_ctarank();
    const int pair = blockIdx.x / 2, pairs = gridDim.x / 2, tiles = p.m_tiles * p.n_tiles;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            ptx::mbar_init(&full[s], 1);
            ptx::mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(&tfull[b], 2);  // the product, and its scales
            ptx::mbar_init(&tempty[b], 2 * kAddWarps);
        }
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&map_a);
        ptx::prefetch_tmap(&map_b);
    }
    if (warp == 1) {
        ptx::tmem_alloc_pair(&tmem_slot, 512);
        ptx::tmem_relinquish_pair();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();  // the peer's barriers are initialised
    ptx::tc_fence_after();
    const uint32_t tmem = tmem_slot;
    float* scales = reinterpret_cast<float*>(smem + S::kStages * S::kStage);
    bool ok = true;

    if (warp < 4) {
        ptx::regs_dec<kCtlRegs>();
        if (warp == 0 && lane == 0) {
            uint32_t it = 0;
            for (int idx = pair; idx < tiles && ok; idx += pairs) {
                int mt, nt;
                tile_at(p, idx, mt, nt);
                for (int g = 0; g < p.KB; ++g, ++it) {
                    const uint32_t s = it % S::kStages;
                    ok = ptx::mbar_wait(&empty[s], ((it / S::kStages) & 1) ^ 1, kWaitNs);
                    if (!ok) break;
                    // both CTAs' bytes count on the even CTA's barrier
                    if (rank == 0) ptx::mbar_arrive_expect_tx(&full[s], 2 * S::kStage);
                    const uint32_t bar = ptx::mapa(ptx::smem_addr(&full[s]), 0);
                    char* st = smem + s * S::kStage;
                    ptx::tma_load_2d_pair(st, &map_a, bar, g * kGroup, mt * 256 + (int)rank * 128);
                    ptx::tma_load_2d_pair(st + S::kA, &map_b, bar, g * kGroup, nt * BN + (int)rank * (BN / 2));
                }
            }
            // every stage has been read, and no arrival at this CTA's barriers is on its way
            for (uint32_t k = it < S::kStages ? 0 : it - S::kStages; k < it && ok; ++k)
                ok = ptx::mbar_wait(&empty[k % S::kStages], (k / S::kStages) & 1, kWaitNs);
        }
        if ((warp == 1 || warp == 2) && lane == 0 && rank == 0) {
            // one issuer for each tensor-memory buffer
            constexpr uint32_t idesc = ptx::idesc_e4m3(256, BN);
            const uint32_t b = warp - 1, d = tmem + b * BN;
            const uint64_t base = ptx::smem_desc_sw128(ptx::smem_addr(smem), 16, 1024);
            const uint32_t total = (uint32_t)((tiles - pair + pairs - 1) / pairs) * p.KB;
            uint32_t s = b, s_phase = 0, b_phase = 1;
            for (uint32_t it = b; it < total; it += 2) {
                ok = ptx::mbar_wait(&tempty[b], b_phase, kWaitNs) && ptx::mbar_wait(&full[s], s_phase, kWaitNs);
                if (!ok) break;
                ptx::tc_fence_after();
                const uint64_t da = base + s * (S::kStage / 16), db = da + S::kA / 16;
#pragma unroll
                for (int k = 0; k < 4; ++k) ptx::mma_f8_ss_pair(d, da + 2 * k, db + 2 * k, idesc, k > 0);
                ptx::mma_commit_pair(&tfull[b]);
                ptx::mma_commit_pair(&empty[s]);
                b_phase ^= 1;
                s += 2;
                if (s >= S::kStages) {
                    s -= S::kStages;
                    s_phase ^= 1;
                }
            }
        }
        if (warp == 3) {
            // The scales of every group, for the adding warps of this CTA: loaded two groups ahead
            // (under load they take longer than a group's product), put into the ring once the
            // product two groups back is complete. That one was begun when every adding warp had
            // read the one before it, so none still uses the ring's slots from five groups back.
            constexpr int kB = kBlocks ? BN / 128 : BN / 32;  // scales of B a lane holds
            const float *sa_at = nullptr, *sb_at = nullptr;
            int rows_in = 0, cols_in = 0, idx = pair, g = 0;  // the group to load next
            float sa[2][4], sb[2][kB];
            auto load = [&](float (&a)[4], float (&b)[kB]) {
                if (idx >= tiles) return;
                if (g == 0) {
                    int mt, nt;
                    tile_at(p, idx, mt, nt);
                    const int64_t m = min((int64_t)mt * 256 + rank * 128, p.M - 1), n = (int64_t)nt * BN;
                    sa_at = p.a_scale + m;
                    rows_in = (int)min((int64_t)128, p.M - m) - 1;
                    sb_at = kBlocks ? p.b_scale + n / kGroup * p.KB : p.b_scale + n;
                    cols_in = (int)min((int64_t)BN, p.N - n) - 1;
                }
                // rows and columns outside C take the last one's
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] = __ldg(sa_at + min(lane + 32 * i, rows_in));
#pragma unroll
                for (int i = 0; i < kB; ++i)
                    b[i] = __ldg(sb_at + (kBlocks ? min(i, cols_in / kGroup) * p.KB : min(lane + 32 * i, cols_in)));
                sa_at += p.M;
                sb_at += kBlocks ? 1 : p.N;
                if (++g == p.KB) {
                    g = 0;
                    idx += pairs;
                }
            };
            load(sa[0], sb[0]);
            load(sa[1], sb[1]);
            const uint32_t total = (uint32_t)((tiles - pair + pairs - 1) / pairs) * p.KB;
            uint32_t phase = 1;
            for (uint32_t it = 0; it < total && ok; it += 2) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    if (it + k >= total) break;
                    ok = __all_sync(0xffffffffu, ptx::mbar_wait(&tfull[k], phase, kWaitNs));
                    if (!ok) break;
                    float* slot = scales + (it + k) % S::kRing * S::kSlot;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (kBlocks) {
#pragma unroll
                            for (int j = 0; j < kB; ++j) slot[128 * j + 32 * i + lane] = sa[k][i] * sb[k][j];
                        } else {
                            slot[32 * i + lane] = sa[k][i];
                        }
                    }
                    if (!kBlocks) {
#pragma unroll
                        for (int j = 0; j < kB; ++j) slot[128 + 32 * j + lane] = sb[k][j];
                    }
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&tfull[k]);
                    load(sa[k], sb[k]);
                }
                phase ^= 1;
            }
        }
    } else {
        ptx::regs_inc<kAddRegs>();
        constexpr int kCols = S::kCols;
        const int quad = warp % 4, part = (warp - 4) / 4;
        const uint32_t taddr = tmem + ((uint32_t)(32 * quad) << 16) + part * kCols;
        char* stage = smem + S::kStages * S::kStage + S::kScales + (warp - 4) * S::kOut;
        // this lane's row's scale in a slot, and the warp's columns'
        const int row_at = 32 * quad + lane + (kBlocks ? part * kCols / kGroup * 128 : 0), col_at = 128 + part * kCols;
        const uint32_t tempty_at = ptx::mapa(ptx::smem_addr(&tempty[0]), 0);
        uint32_t it = 0;
        for (int idx = pair; idx < tiles && ok; idx += pairs) {
            int mt, nt;
            tile_at(p, idx, mt, nt);
            const int64_t m0 = (int64_t)mt * 256 + rank * 128 + 32 * quad;
            const int64_t n0 = (int64_t)nt * BN + part * kCols;
            float2 acc[kCols / 2];
#pragma unroll
            for (int j = 0; j < kCols / 2; ++j) acc[j] = make_float2(0.0f, 0.0f);
            for (int g = 0; g < p.KB; ++g, ++it) {
                const uint32_t b = it & 1;
                ok = __all_sync(0xffffffffu, ptx::mbar_wait(&tfull[b], (it >> 1) & 1, kWaitNs));
                if (!ok) break;
                const float* slot = scales + it % S::kRing * S::kSlot;
                const float s = slot[row_at];
                const float2 ss = make_float2(s, s);
                ptx::tc_fence_after();
#pragma unroll
                for (int j = 0; j < kCols / 32; ++j) {
                    float v[32];
                    ptx::tmem_ld32(taddr + b * BN + 32 * j, v);
                    ptx::tmem_wait_ld();
                    if (j == kCols / 32 - 1) {  // read: the next product but one may take its place
                        ptx::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive_remote_relaxed(tempty_at + 8 * b);
                    }
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        float2* to = acc + 16 * j + e / 2;
                        float2 lo = make_float2(v[e], v[e + 1]), hi = make_float2(v[e + 2], v[e + 3]);
                        if (!kBlocks) {
                            const float4 w = *reinterpret_cast<const float4*>(slot + col_at + 32 * j + e);
                            lo = ptx::mul2(lo, make_float2(w.x, w.y));
                            hi = ptx::mul2(hi, make_float2(w.z, w.w));
                        }
                        to[0] = ptx::fma2(lo, ss, to[0]);
                        to[1] = ptx::fma2(hi, ss, to[1]);
                    }
                }
            }
            if (!ok) break;
#pragma unroll
            for (int j = 0; j < kCols / 32; ++j)
                if (n0 + 32 * j < p.N) store_rows<T>(p, stage, acc + 16 * j, m0, n0 + 32 * j, lane);
        }
    }
    if (!ok) {
        // a wait gave up: report it, and leave copies and products in flight the time to end
        tc::fail(p.status);
        const uint64_t t0 = ptx::globaltimer_ns();
        while (ptx::globaltimer_ns() - t0 < 2000000) {
        }
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();  // no arrival at the peer's barriers and no MMA on its tensor memory is left
    if (warp == 1) ptx::tmem_dealloc_pair(tmem, 512);
}

int device_sms() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    return sms;
}

template <int BN, bool kBlocks, typename T>
int launch_pair(const Matmul& p, Product q, int sms, cudaStream_t stream) {
    CUtensorMap ma, mb;
    if (!tc::encode_tiled_u8(&ma, p.a, p.K, p.M, p.a_ld, 128) || !tc::encode_tiled_u8(&mb, p.b, p.K, p.N, p.b_ld, BN / 2))
        return SSDC_ERR_CUDA;
    q.n_tiles = (int)((p.N + BN - 1) / BN);
    const int64_t tiles = (int64_t)q.m_tiles * q.n_tiles;
    if (tiles > INT32_MAX / 2) return SSDC_ERR_UNSUPPORTED;
    const int pairs = (int)(tiles < sms / 2 ? tiles : sms / 2);
    auto* k = product_pair<BN, kBlocks, T>;
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Shape<BN>::kBytes) != cudaSuccess)
        return SSDC_ERR_CUDA;
    k<<<2 * pairs, kThreads, Shape<BN>::kBytes, stream>>>(ma, mb, q);
    return 1;
}

template <int BN>
int launch_pair_types(const Matmul& p, const Product& q, int sms, cudaStream_t stream) {
    if (p.b_blocks)
        return p.out_bf16 ? launch_pair<BN, true, __nv_bfloat16>(p, q, sms, stream)
                          : launch_pair<BN, true, float>(p, q, sms, stream);
    return p.out_bf16 ? launch_pair<BN, false, __nv_bfloat16>(p, q, sms, stream)
                      : launch_pair<BN, false, float>(p, q, sms, stream);
}

}  // namespace

size_t matmul_workspace(int64_t, int64_t, int64_t) { return 256; }

int matmul_launch(const Matmul& p, cudaStream_t stream) {
    const int sms = device_sms();
    if (sms < 2) return SSDC_ERR_CUDA;
    Product q = {};
    q.a_scale = p.a_scale; q.b_scale = p.b_scale;
    q.M = p.M; q.N = p.N; q.c_ld = p.c_ld;
    q.KB = (int)((p.K + kGroup - 1) / kGroup);
    q.m_tiles = (int)((p.M + 255) / 256);
    q.c = p.c;
    const size_t e = p.out_bf16 ? 2 : 4;
    q.aligned = (reinterpret_cast<uintptr_t>(p.c) | (uintptr_t)(p.c_ld * e)) % 32 == 0;
    q.status = p.status;
    // The tile width whose rounds over the SM pairs cover fewer columns in all
    auto rounds = [&](int bn) {
        const int64_t tiles = (int64_t)q.m_tiles * ((p.N + bn - 1) / bn);
        return (tiles + sms / 2 - 1) / (sms / 2) * bn;
    };
    return rounds(128) < rounds(256) ? launch_pair_types<128>(p, q, sms, stream)
                                     : launch_pair_types<256>(p, q, sms, stream);
}

}  // namespace block
}  // namespace ssdc
