// 8-bit product (include/ssdc_block.h) for few rows of A (tokens): bound by reading B (weights).
//
// The operands change places: a tile of 128 of B's rows is the matrix unit's 128 rows, and
// the tokens, padded to kRows (16 or 32), its columns, so that no work goes into rows that
// are not there. The columns of K are dealt over the CTAs of a cluster where B has fewer tiles
// than the GPU SMs; their sums meet in distributed shared memory, each CTA adding up a share of
// the tokens in the order of K. Scaling between groups of 128 as in block_matmul.cu: a B-row a
// lane, a token a register.
//
// Warp 0 loads (TMA), warp 1 issues the MMAs, warps 2 .. 5 scale, add and store.
//
// Measured: M 8 N 50257 K 1024 (51 MB, from L2) 11.4 us, 4.5 TB/s; M 8 N 5136 K 1024 5.5 us in a graph, a
// call after another 5.9 us: latency (copies, products, the cluster's meeting), not bytes (0.8 us).
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
constexpr int kGroup = SSD_FP8_GROUP, kThreads = 192, kStages = 4, kBufs = 4;

struct Few {
    const float *a_scale, *b_scale;
    int64_t N, c_ld;
    int M, KB, per_cta;  // groups a CTA takes
    uint32_t cluster;
    void* c;
    int* status;
};

template <int kRows>
struct Shape {
    static constexpr uint32_t kB = 128 * kGroup, kA = kRows * kGroup, kStage = kB + kA;
    static constexpr uint32_t kMeet = 128 * kRows * 4;       // sums from the cluster's CTAs
    static constexpr uint32_t kScales = 4 * 2 * kRows * 4;   // tokens' scales, two groups for each warp
    // (with 4 kRows tensor-memory columns a CTA, no more CTAs share an SM's shared memory than its
    // tensor memory: a CTA never waits for columns that a waiting cluster holds)
    static constexpr uint32_t kBytes = 1024 + kStages * kStage + kMeet + kScales;
};

template <int kRows, bool kBlocks, typename T>
__global__ void __launch_bounds__(kThreads)
product_few(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, const Few p) {
    using S = Shape<kRows>;
    extern __shared__ char smem_raw[];
    char* smem = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* meet = reinterpret_cast<float*>(smem + kStages * S::kStage);
    float* scales = meet + 128 * kRows;
    __shared__ uint64_t full[kStages], empty[kStages], tfull[kBufs], tempty[kBufs];
    __shared__ uint32_t tmem_slot;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t R = p.cluster, rank = blockIdx.x % R;
    const int64_t n0 = (int64_t)(blockIdx.x / R) * 128;
    const int g0 = (int)rank * p.per_cta, groups = max(0, min(p.per_cta, p.KB - g0));

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(&full[s], 1);
            ptx::mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < kBufs; ++b) {
            ptx::mbar_init(&tfull[b], 1);
            ptx::mbar_init(&tempty[b], 4);
        }
        ptx::fence_mbar_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc(&tmem_slot, kBufs * kRows);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    launch_dependents();
    grid_dependency_wait();
    if (R > 1) ptx::cluster_arrive_relaxed();  // (a CTA's shared memory may be written to once it runs)
    const uint32_t tmem = tmem_slot;
    bool ok = true;

    if (warp == 0) {
        if (lane == 0) {
            for (int i = 0; i < groups; ++i) {
                const int s = i % kStages;
                ok = ptx::mbar_wait(&empty[s], ((i / kStages) & 1) ^ 1, kWaitNs);
                if (!ok) break;
                ptx::mbar_arrive_expect_tx(&full[s], S::kStage);
                ptx::tma_load_2d(smem + s * S::kStage, &map_b, &full[s], (g0 + i) * kGroup, (int)n0);
                ptx::tma_load_2d(smem + s * S::kStage + S::kB, &map_a, &full[s], (g0 + i) * kGroup, 0);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t idesc = ptx::idesc_e4m3(128, kRows);
            for (int i = 0; i < groups; ++i) {
                const int s = i % kStages, b = i % kBufs;
                ok = ptx::mbar_wait(&full[s], (i / kStages) & 1, kWaitNs) &&
                     ptx::mbar_wait(&tempty[b], ((i / kBufs) & 1) ^ 1, kWaitNs);
                if (!ok) break;
                ptx::tc_fence_after();
                const uint32_t w = ptx::smem_addr(smem + s * S::kStage), x = w + S::kB;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    ptx::mma_f8_ss(tmem + b * kRows, ptx::smem_desc_sw128(w + 32 * k, 16, 1024),
                                   ptx::smem_desc_sw128(x + 32 * k, 16, 1024), idesc, k > 0);
                ptx::mma_commit(&empty[s]);
                ptx::mma_commit(&tfull[b]);
            }
        }
    } else {
        constexpr int kPiece = kRows < 32 ? kRows : 32, kOf = (kRows + 31) / 32;  // scales a lane fetches
        const int quad = warp % 4, row = 32 * quad + lane;
        const int64_t n = n0 + row;
        const uint32_t taddr = tmem + ((uint32_t)(32 * quad) << 16);
        float* mine = scales + quad * 2 * kRows;
        // the scale of this lane's row of B, and of the tokens (those past M take the last one's), a
        // group ahead
        const float* sb_at = kBlocks ? p.b_scale + n0 / kGroup * p.KB + g0 : p.b_scale + (int64_t)g0 * p.N + min(n, p.N - 1);
        const float* sa_at = p.a_scale + (int64_t)g0 * p.M;
        float sb = 0.0f, sa[kOf];
        auto fetch = [&]() {
            sb = __ldg(sb_at);
#pragma unroll
            for (int j = 0; j < kOf; ++j) sa[j] = __ldg(sa_at + min(32 * j + lane, p.M - 1));
            sb_at += kBlocks ? 1 : p.N;
            sa_at += p.M;
        };
        float acc[kRows];
#pragma unroll
        for (int c = 0; c < kRows; ++c) acc[c] = 0.0f;
        if (groups > 0) fetch();
        for (int i = 0; i < groups; ++i) {
            const int b = i % kBufs;
            float* slot = mine + (i & 1) * kRows;
#pragma unroll
            for (int j = 0; j < kOf; ++j)
                if (32 * j + lane < kRows) slot[32 * j + lane] = sa[j];
            const float s = sb;
            __syncwarp();
            if (i + 1 < groups) fetch();
            ok = __all_sync(0xffffffffu, ptx::mbar_wait(&tfull[b], (i / kBufs) & 1, kWaitNs));
            if (!ok) break;
            ptx::tc_fence_after();
#pragma unroll
            for (int j = 0; j < kRows / kPiece; ++j) {
                float v[kPiece];
                if constexpr (kPiece == 32) ptx::tmem_ld32(taddr + b * kRows + 32 * j, v);
                else ptx::tmem_ld16(taddr + b * kRows, v);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < kPiece; e += 4) {
                    const float4 w = *reinterpret_cast<const float4*>(slot + kPiece * j + e);
                    float* to = acc + kPiece * j + e;
                    to[0] = fmaf(v[e], s * w.x, to[0]);
                    to[1] = fmaf(v[e + 1], s * w.y, to[1]);
                    to[2] = fmaf(v[e + 2], s * w.z, to[2]);
                    to[3] = fmaf(v[e + 3], s * w.w, to[3]);
                }
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&tempty[b]);
        }
        T* c = static_cast<T*>(p.c) + n;
        if (R == 1) {
#pragma unroll
            for (int m = 0; m < kRows; ++m)
                if (ok && m < p.M && n < p.N) c[m * p.c_ld] = from_f32<T>(acc[m]);
        } else {
            // token m's sums go to the CTA m / (kRows / R), place (rank, row, m % (kRows / R))
            ptx::cluster_wait();
            const int share = kRows / R;
            const uint32_t at = ptx::smem_addr(meet) + (uint32_t)((rank * 128 + row) * share) * 4;
#pragma unroll
            for (int m = 0; m < kRows; m += 2) {
                const uint32_t to = ptx::mapa(at + (uint32_t)(m % share) * 4, m / share);
                asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(acc[m]), "f"(acc[m + 1]) : "memory");
            }
        }
    }
    if (!ok) {
        // a wait gave up: report it, and leave copies and products in flight the time to end
        tc::fail(p.status);
        const uint64_t t0 = ptx::globaltimer_ns();
        while (ptx::globaltimer_ns() - t0 < 2000000) {
        }
    }
    if (R > 1) {
        if (warp < 2) ptx::cluster_wait();
        __syncwarp();
        ptx::cluster_sync();
        if (warp >= 2) {
            const int row = 32 * (warp % 4) + lane, share = kRows / R;
            const int64_t n = n0 + row;
            for (int k = 0; k < share; ++k) {
                const int m = (int)rank * share + k;
                if (m >= p.M) break;
                float v = 0.0f;
                for (uint32_t r = 0; r < R; ++r) v += meet[(r * 128 + row) * share + k];
                if (n < p.N) static_cast<T*>(p.c)[m * p.c_ld + n] = from_f32<T>(v);
            }
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) ptx::tmem_dealloc(tmem, kBufs * kRows);
}

template <int kRows, bool kBlocks, typename T>
int launch(const Matmul& p, const Few& q, cudaStream_t stream) {
    using S = Shape<kRows>;
    CUtensorMap ma, mb;
    if (!tc::encode_tiled_2d(&ma, p.a, 1, p.K, p.M, p.a_ld, kRows) || !tc::encode_tiled_2d(&mb, p.b, 1, p.K, p.N, p.b_ld, 128))
        return SSDC_ERR_CUDA;
    auto* k = product_few<kRows, kBlocks, T>;
    static std::atomic<uint64_t> allowed;
    if (allow_smem(k, (int)S::kBytes, allowed) != cudaSuccess) return SSDC_ERR_CUDA;
    return launch_clusters(k, (p.N + 127) / 128, (int)q.cluster, false, kThreads, S::kBytes, stream, ma, mb, q);
}

template <int kRows>
int launch_types(const Matmul& p, const Few& q, cudaStream_t stream) {
    if (p.b_blocks) return p.out_bf16 ? launch<kRows, true, __nv_bfloat16>(p, q, stream) : launch<kRows, true, float>(p, q, stream);
    return p.out_bf16 ? launch<kRows, false, __nv_bfloat16>(p, q, stream) : launch<kRows, false, float>(p, q, stream);
}

}  // namespace

// CTAs of a cluster: until every SM has one, with 8 groups each at least (M 8 N 1024 K 8192: 29 us
// with one CTA a tile, 7.3 us with 8; M 8 N 5136 K 1024, 8 groups in all: 5.9 us undivided, 6.6 us
// over four).
uint32_t few_cluster(int64_t N, int KB) {
    const int64_t tiles = (N + 127) / 128;
    uint32_t r = 1;
    while (r < 8 && tiles * r < 152 && KB >= 16 * (int)r) r *= 2;
    return r;
}

// Up to 16 rows always (M 16, bfloat16, in a graph, here / by block_matmul.cu: N 64 K 64 2.7 / 3.7 us, N 64
// K 8192 6.6 / 22, N 1024 K 1024 5.7 / 5.9, N 5136 K 1024 5.8 / 6.6, N 20000 K 2048 9.6 / 20, N 50257 K 128
// 6.0 / 8.7, N 50257 K 4096 42 / 52); up to 32 where K is dealt over a cluster (M 32 N 1024 K 8192 13 / 23 us;
// where it is not, M 32 N 5136 K 1024 7.5 / 7.2 us).
bool matmul_is_few(int64_t M, int64_t N, int64_t K) {
    return M <= 16 || (M <= 32 && few_cluster(N, (int)((K + kGroup - 1) / kGroup)) > 1);
}

int matmul_few_launch(const Matmul& p, cudaStream_t stream) {
    Few q = {};
    q.a_scale = p.a_scale; q.b_scale = p.b_scale;
    q.N = p.N; q.c_ld = p.c_ld; q.M = (int)p.M;
    q.KB = (int)((p.K + kGroup - 1) / kGroup);
    q.c = p.c; q.status = p.status;
    q.cluster = few_cluster(p.N, q.KB);
    q.per_cta = (q.KB + (int)q.cluster - 1) / (int)q.cluster;
    return p.M <= 16 ? launch_types<16>(p, q, stream) : launch_types<32>(p, q, stream);
}

}  // namespace block
}  // namespace ssdc
