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
// scales, the others scale, add and store; each of those owns 32 rows x BN / 2 columns in
// registers, and takes registers that the first four warps give up. (The issue of an MMA returns shortly before it is done, so a single
// issuer's waits between two groups left the tensor cores idle for as long as they worked.)
//
// Measured: M 9728 N 8192 K 8192 455 us (2.87 PFLOP/s); M 32768 N 5136 K 1024 174 us
// (1.98 PFLOP/s), 1021 x 50257 x 1024 60 us (1.75 PFLOP/s), 4096 x 5136 x 1024 28 us. A group's
// product waits for its operands from L2 (32 KB a CTA, 0.38 us at the 13 TB/s that the SMs take
// in together) and its sums for the adding warps (0.41 us); with eight groups a tile,
// storing a tile costs about a fifth on top: its rows go through the shared memory that the
// operands stream through (stored or not: 174 and 145 us).
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
constexpr int kGroup = SSD_FP8_GROUP;

struct Product {
    const float *a_scale, *b_scale;
    int64_t M, N, c_ld;
    int KB, m_tiles, n_tiles;
    void* c;
    bool tma_out;  // c's rows start at multiples of 16 bytes: stored by TMA
    int* status;
    int whole;       // tiles that pairs take whole, in turn; the others' groups are dealt out evenly
    int* flags;      // a pair's warps' marks that their sums of a tile's end are in `sums`
    float4* sums;
    int64_t copied;  // (tma_out) the columns that are copied out, whole 16-byte units
};

constexpr int kFlags = 16;  // of a pair: 8 adding warps of two CTAs

// What a pair works on, one piece after another: groups g0 .. g1 of a tile. First the tiles that
// it takes whole. Then its even share of the other tiles' groups, which may begin inside a
// tile and end inside one. A tile's first part is always some pair's last piece and its later
// parts are other pairs' first pieces: the one with the first part waits for the others'
// sums, adds them in the order of K and stores the tile.
struct Walk {
    const Product& p;
    int pair, pairs, tile;
    int64_t at, end;
    __device__ __forceinline__ Walk(const Product& q, int pr, int prs) : p(q), pair(pr), pairs(prs), tile(pr), at(first(pr)), end(first(pr + 1)) {}
    __device__ __forceinline__ int64_t first(int pr) const {
        return (int64_t)(p.m_tiles * p.n_tiles - p.whole) * p.KB * pr / pairs;
    }
    __device__ __forceinline__ uint32_t groups() const {
        return (uint32_t)((tile < p.whole ? (p.whole - tile + pairs - 1) / pairs : 0) * p.KB + (int)(end - at));
    }
    __device__ __forceinline__ bool next(int& idx, int& g0, int& g1) {
        if (tile < p.whole) {
            idx = tile;
            g0 = 0;
            g1 = p.KB;
            tile += pairs;
            return true;
        }
        if (at >= end) return false;
        const int t = (int)(at / p.KB);
        idx = p.whole + t;
        g0 = (int)(at - (int64_t)t * p.KB);
        g1 = (int)min((int64_t)p.KB, g0 + (end - at));
        at += g1 - g0;
        return true;
    }
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
    static constexpr int kBufs = 512 / BN;  // tensor-memory buffers
    // adding warps: four quarters of the rows x two halves of the columns
    static constexpr int kCols = BN / 2, kAddWarps = 8, kThreads = 128 + 32 * kAddWarps;
    // Registers a thread: 384 x 168 at launch = 128 x 56 + 256 x 224 after the split
    static constexpr int kCtlRegs = 56, kAddRegs = 224;
    // Scales, a ring of groups: 128 rows' for each of B's two blocks (already multiplied), or 128
    // rows' and then the columns'
    static constexpr int kRing = 4 * kBufs, kSlot = 128 + 256;
    static constexpr uint32_t kScales = kRing * kSlot * 4;
    // per adding warp: twice 32 rows of 128 bytes of C (of 132 where they are stored one by one)
    static constexpr uint32_t kOut = 8 * 1024;
    static constexpr int kStages = BN == 256 ? 4 : 5;
    static constexpr uint32_t kBytes = 1024 + kStages * kStage + kAddWarps * kOut + kScales;
};

__device__ __forceinline__ uint32_t bf16_pair(float2 v) {
    const __nv_bfloat162 t = __float22bfloat162_rn(v);
    return *reinterpret_cast<const uint32_t*>(&t);
}

// kRest: C's columns are copied out and end inside a 16-byte unit. (An instance of its own: with the test
// for it in the other, 32768 x 5120 x 1024 bfloat16 took 168 us for 163.)

// Which of a warp's 32 x 16 sums a lane holds. Along: its row's, acc[8 j + e] columns 16 j + 2 e and
// the next. Across (as the tensor memory gives 8 x 8 blocks to a warp): acc[8 j + 4 i + 2 c + h] is
// row 16 i + 8 h + lane / 4, columns 16 j + 8 c + 2 (lane % 4) and the next. Where every column has
// its own scale it is then read for 4 rows' sums rather than one's: M 9728 N 2048 K 4096 117 us
// along, 93 us across (65 us with a scale for each 128 columns, along).

// 128 bytes (64 bfloat16 or 32 fp32 values) of each of a warp's 32 rows to C from row m0 and
// column n on, through the warp's staging rows: piece j of the warp's part of a tile takes half
// j & 1 of them. A tile's first piece waits until all copies before it have read their rows (the
// tile before may have ended with either half), a later one until all but the last have.
template <typename T, bool kAcross, bool kRest>
__device__ __forceinline__ void store_piece(const Product& p, const CUtensorMap* map_c, char* stage, int j,
                                            const float2* v, int64_t m0, int64_t n, int lane) {
    constexpr bool kHalf = sizeof(T) == 2;
    constexpr int kPiece = 128 / sizeof(T);
    auto word = [&](int e) {  // the e-th of the row's 32 words
        if constexpr (kHalf) return bf16_pair(v[e]);
        else return __float_as_uint(e & 1 ? v[e / 2].y : v[e / 2].x);
    };
    // across: the two values of block c8 (of 8 columns), row 8 k + lane / 4
    auto pair_of = [&](int c8, int k) { return v[8 * (c8 / 2) + 4 * (k / 2) + 2 * (c8 % 2) + k % 2]; };
    if (p.tma_out) {
        // asynchronous: the warp goes on to the next tile while the rows are copied out; rows outside C
        // are left out by the copy, and columns from C's last whole 16-byte unit on
        if (lane == 0) {
            if (j == 0) ptx::bulk_wait_read<0>();
            else ptx::bulk_wait_read<1>();
        }
        __syncwarp();
        char* to = stage + 4096 * (j & 1);  // (with the 128-byte swizzle of the tensor map)
        if constexpr (!kAcross) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
                *reinterpret_cast<uint4*>(to + lane * 128 + (((e / 4) ^ (lane & 7)) << 4)) =
                    make_uint4(word(e), word(e + 1), word(e + 2), word(e + 3));
        } else if constexpr (kHalf) {
#pragma unroll
            for (int c = 0; c < 8; ++c)
                ptx::stmatrix4(to + lane * 128 + ((c ^ (lane & 7)) << 4), bf16_pair(pair_of(c, 0)), bf16_pair(pair_of(c, 1)),
                               bf16_pair(pair_of(c, 2)), bf16_pair(pair_of(c, 3)));
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    *reinterpret_cast<float2*>(to + (8 * k + lane / 4) * 128 + (((2 * c + lane % 4 / 2) ^ (lane / 4)) << 4) +
                                               lane % 2 * 8) = pair_of(c, k);
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && (!kRest || n < p.copied)) {
            ptx::tma_store_2d(map_c, to, (int)n, (int)m0);
            ptx::bulk_commit();
        }
        return;
    }
    // Rows that start anywhere: word by word, a row a store. A row of bfloat16 that starts between
    // two words is shifted by one value, its first and last values stored alone.
    uint32_t* st = reinterpret_cast<uint32_t*>(stage);
    __syncwarp();
    if constexpr (!kAcross) {
#pragma unroll
        for (int e = 0; e < 32; ++e) st[lane * 33 + e] = word(e);
    } else {
#pragma unroll
        for (int c = 0; c < kPiece / 8; ++c)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 u = pair_of(c, k);
                uint32_t* to = st + (8 * k + lane / 4) * 33;
                if constexpr (kHalf) {
                    to[4 * c + lane % 4] = bf16_pair(u);
                } else {
                    to[8 * c + 2 * (lane % 4)] = __float_as_uint(u.x);
                    to[8 * c + 2 * (lane % 4) + 1] = __float_as_uint(u.y);
                }
            }
    }
    __syncwarp();
    const int cols = (int)min((int64_t)kPiece, p.N - n), rows = (int)min((int64_t)32, p.M - m0);
    if (kHalf && cols == kPiece) {
        // many rows under way at a time; a row is shifted by none or one of its values
        constexpr int kAtOnce = 8;
        char* c = reinterpret_cast<char*>(static_cast<T*>(p.c) + m0 * p.c_ld + n) + 4 * lane;
        const int64_t pitch = p.c_ld * (int64_t)sizeof(T);
#pragma unroll
        for (int r0 = 0; r0 < 32; r0 += kAtOnce) {
            uint32_t w[kAtOnce], next[kAtOnce];
#pragma unroll
            for (int r = 0; r < kAtOnce; ++r) {
                w[r] = st[(r0 + r) * 33 + lane];
                next[r] = st[(r0 + r) * 33 + lane + 1];  // (the 33rd word of a row is not used)
            }
#pragma unroll
            for (int r = 0; r < kAtOnce; ++r) {
                char* row = c + (r0 + r) * pitch;
                if (r0 + r < rows) {
                    const uint32_t odd = (uint32_t)(reinterpret_cast<uintptr_t>(row) >> 1) & 1;
                    if (!odd || lane < 31) *reinterpret_cast<uint32_t*>(row + 2 * odd) = __funnelshift_r(w[r], next[r], 16 * odd);
                    else *reinterpret_cast<uint16_t*>(row + 2) = (uint16_t)(w[r] >> 16);
                    if (odd && lane == 0) *reinterpret_cast<uint16_t*>(row) = (uint16_t)w[r];
                }
            }
        }
        return;
    }
    for (int r = 0; r < rows; ++r) {
        T* c = static_cast<T*>(p.c) + (m0 + r) * p.c_ld + n;
        const uint32_t w = st[r * 33 + lane];
        if constexpr (kHalf) {
            if ((reinterpret_cast<uintptr_t>(c) & 2) == 0) {
                if (2 * lane + 1 < cols) reinterpret_cast<uint32_t*>(c)[lane] = w;
                else if (2 * lane < cols) reinterpret_cast<uint16_t*>(c)[2 * lane] = (uint16_t)w;
            } else {
                const uint32_t next = st[r * 33 + min(lane + 1, 31)];
                if (lane == 0) reinterpret_cast<uint16_t*>(c)[0] = (uint16_t)w;
                if (2 * lane + 2 < cols)
                    *reinterpret_cast<uint32_t*>(c + 2 * lane + 1) = __byte_perm(w, next, 0x5432);
                else if (2 * lane + 1 < cols) reinterpret_cast<uint16_t*>(c)[2 * lane + 1] = (uint16_t)(w >> 16);
            }
        } else {
            if (lane < cols) reinterpret_cast<uint32_t*>(c)[lane] = w;
        }
    }
}

// A copy writes whole 16-byte units: where C's columns end inside one it would overwrite what is behind
// them. The columns that are no whole unit (from p.copied on) are stored one by one, a row a lane, from
// the staging rows of a warp's part of a tile, columns n0 on, after its pieces.
template <typename T>
__device__ __forceinline__ void store_rest(const Product& p, const char* stage, int64_t m0, int64_t n0, int lane) {
    constexpr int kPiece = 128 / sizeof(T);
    if (m0 + lane >= p.M) return;
    const int first = (int)(p.copied - n0), piece = first / kPiece;
    const char* row = stage + 4096 * (piece & 1) + lane * 128;
    T* c = static_cast<T*>(p.c) + (m0 + lane) * p.c_ld + p.copied;
    for (int k = 0; k < (int)(p.N - p.copied); ++k) {
        const int at = (first - piece * kPiece + k) * (int)sizeof(T);
        c[k] = *reinterpret_cast<const T*>(row + (((at / 16) ^ (lane & 7)) << 4) + at % 16);
    }
}

template <int BN, bool kBlocks, typename T, bool kRest>
__global__ void __launch_bounds__(Shape<BN>::kThreads, 1)
product_pair(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
             const __grid_constant__ CUtensorMap map_c, const Product p) {
    using S = Shape<BN>;
    constexpr int kBufs = S::kBufs;
    extern __shared__ char smem_raw[];
    char* smem = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t full[S::kStages], empty[S::kStages], tfull[kBufs], tempty[kBufs];
    __shared__ uint32_t tmem_slot;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = ptx::cluster_ctarank();
    Walk walk(p, blockIdx.x / 2, gridDim.x / 2);
    const uint32_t total = walk.groups();

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            ptx::mbar_init(&full[s], 1);
            ptx::mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < kBufs; ++b) {
            ptx::mbar_init(&tfull[b], 2);  // the product, and its scales
            ptx::mbar_init(&tempty[b], 2 * S::kAddWarps);
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
    launch_dependents();
    grid_dependency_wait();
    const uint32_t tmem = tmem_slot;
    char* out = smem + S::kStages * S::kStage;
    float* scales = reinterpret_cast<float*>(out + S::kAddWarps * S::kOut);
    bool ok = true;

    if (warp < 4) {
        ptx::regs_dec<S::kCtlRegs>();
        if (warp == 0 && lane == 0) {
            uint32_t it = 0;
            int idx, g0, g1;
            while (ok && walk.next(idx, g0, g1)) {
                int mt, nt;
                tile_at(p, idx, mt, nt);
                for (int g = g0; g < g1; ++g, ++it) {
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
            // two issuers, each of every other group
            constexpr uint32_t idesc = ptx::idesc_e4m3(256, BN);
            const uint64_t base = ptx::smem_desc_sw128(ptx::smem_addr(smem), 16, 1024);
            uint32_t s = warp - 1, s_phase = 0;
            for (uint32_t it = warp - 1; it < total; it += 2) {
                const uint32_t b = it % kBufs, b_phase = it / kBufs & 1 ^ 1, d = tmem + b * BN;
                // (the operands come early: waited for first, the buffer's release is acted on at once)
                ok = ptx::mbar_wait(&full[s], s_phase, kWaitNs) && ptx::mbar_wait(&tempty[b], b_phase, kWaitNs);
                if (!ok) break;
                ptx::tc_fence_after();
                const uint64_t da = base + s * (S::kStage / 16), db = da + S::kA / 16;
#pragma unroll
                for (int k = 0; k < 4; ++k) ptx::mma_f8_ss_pair(d, da + 2 * k, db + 2 * k, idesc, k > 0);
                ptx::mma_commit_pair(&tfull[b]);
                ptx::mma_commit_pair(&empty[s]);
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
            // product kBufs groups back is complete. That one was begun when every adding warp had
            // read the one in its buffer before, 2 kBufs groups back, and so had done with all
            // earlier ones: of a ring of more than 2 kBufs slots the oldest is free.
            constexpr int kB = kBlocks ? BN / 128 : BN / 32;  // scales of B a lane holds
            const float *sa_at = nullptr, *sb_at = nullptr;
            int rows_in = 0, cols_in = 0, g = 0, g_end = 0;  // the group to load next, of a piece that ends before g_end
            float sa[2][4], sb[2][kB];
            auto load = [&](float (&a)[4], float (&c)[kB]) {
                if (g == g_end) {
                    int idx, mt, nt;
                    if (!walk.next(idx, g, g_end)) return;
                    tile_at(p, idx, mt, nt);
                    const int64_t m = min((int64_t)mt * 256 + rank * 128, p.M - 1), n = (int64_t)nt * BN;
                    sa_at = p.a_scale + g * p.M + m;
                    rows_in = (int)min((int64_t)128, p.M - m) - 1;
                    sb_at = kBlocks ? p.b_scale + n / kGroup * p.KB + g : p.b_scale + g * p.N + n;
                    cols_in = (int)min((int64_t)BN, p.N - n) - 1;
                }
                // rows and columns outside C take the last one's
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] = __ldg(sa_at + min(lane + 32 * i, rows_in));
#pragma unroll
                for (int i = 0; i < kB; ++i)
                    c[i] = __ldg(sb_at + (kBlocks ? min(i, cols_in / kGroup) * p.KB : min(lane + 32 * i, cols_in)));
                sa_at += p.M;
                sb_at += kBlocks ? 1 : p.N;
                ++g;
            };
            load(sa[0], sb[0]);
            load(sa[1], sb[1]);
            for (uint32_t it = 0; it < total && ok; it += 2) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    if (it + k >= total) break;
                    const uint32_t b = (it + k) % kBufs, phase = (it + k) / kBufs & 1 ^ 1;
                    ok = __all_sync(0xffffffffu, ptx::mbar_wait(&tfull[b], phase, kWaitNs));
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
                    if (lane == 0) ptx::mbar_arrive(&tfull[b]);
                    load(sa[k], sb[k]);
                }
            }
        }
    } else {
        ptx::regs_inc<S::kAddRegs>();
        constexpr int kCols = S::kCols;
        const int quad = warp % 4, part = (warp - 4) / 4;
        const uint32_t taddr = tmem + ((uint32_t)(32 * quad) << 16) + part * kCols;
        char* stage = out + (warp - 4) * S::kOut;
        // this lane's rows' scales in a slot, and its columns'
        constexpr int kRows = kBlocks ? 1 : 4;
        const int row_at = 32 * quad + (kBlocks ? lane + part * kCols / kGroup * 128 : lane / 4);
        const int col_at = 128 + part * kCols + 2 * (lane % 4);
        const uint32_t tempty_at = ptx::mapa(ptx::smem_addr(&tempty[0]), 0);
        // Pieces of kP columns are read while the one before is added, and the first of a group
        // while the last of the group before is: accesses to shared memory and its barriers take
        // 200 cycles while operands stream through it, and must not stand between two pieces. With
        // a scale for every column the pieces are smaller, for the registers.
        constexpr int kP = kBlocks ? 32 : 16, kPieces = kCols / kP;
        float v[2][kP], s[kRows] = {};
        float2 w[2][kBlocks ? 1 : 2];
        auto read = [&](int j, uint32_t b, const float* slot) {  // piece j
            if constexpr (kBlocks) {
                ptx::tmem_ld32(taddr + b * BN + kP * j, v[j & 1]);
            } else {
                ptx::tmem_ld_16x16(taddr + b * BN + kP * j, v[j & 1]);
                ptx::tmem_ld_16x16(taddr + (16u << 16) + b * BN + kP * j, v[j & 1] + 8);
#pragma unroll
                for (int c = 0; c < 2; ++c) w[j & 1][c] = *reinterpret_cast<const float2*>(slot + col_at + kP * j + 8 * c);
            }
        };
        uint32_t it = 0;  // the group that begin() reads next
        bool ready = false;
        auto begin = [&]() {
            const uint32_t b = it % kBufs, phase = it / kBufs & 1;
            ok = __all_sync(0xffffffffu, ready || ptx::mbar_wait(&tfull[b], phase, kWaitNs));
            if (!ok) return;
            ptx::tc_fence_after();
            const float* slot = scales + it % S::kRing * S::kSlot;
            read(0, b, slot);
#pragma unroll
            for (int k = 0; k < kRows; ++k) s[k] = slot[row_at + 8 * k];
            ++it;
        };
        begin();
        const int flag_at = (int)rank * 8 + warp - 4;  // this warp among its pair's, and its sums
        const int64_t sums_at = (int64_t)flag_at * (kCols / 4) * 32 + lane, sums_pair = (int64_t)kFlags * (kCols / 4) * 32;
        int idx, g0, g1;
        while (ok && walk.next(idx, g0, g1)) {
            int mt, nt;
            tile_at(p, idx, mt, nt);
            const int64_t m0 = (int64_t)mt * 256 + rank * 128 + 32 * quad;
            const int64_t n0 = (int64_t)nt * BN + part * kCols;
            float2 acc[kCols / 2];
#pragma unroll
            for (int j = 0; j < kCols / 2; ++j) acc[j] = make_float2(0.0f, 0.0f);
            for (int g = g0; g < g1 && ok; ++g) {
                const uint32_t b = (it - 1) % kBufs;
                const float* slot = scales + (it - 1) % S::kRing * S::kSlot;
                float2 ss[kRows];
#pragma unroll
                for (int k = 0; k < kRows; ++k) ss[k] = make_float2(s[k], s[k]);
#pragma unroll
                for (int j = 0; j < kPieces; ++j) {
                    ptx::tmem_wait_ld();
                    if (j == kPieces - 2) ready = ptx::mbar_test_wait(&tfull[it % kBufs], it / kBufs & 1);
                    if (j + 1 < kPieces) {
                        read(j + 1, b, slot);
                    } else {  // read: the next product but kBufs - 1 may take its place
                        ptx::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive_remote_relaxed(tempty_at + 8 * b);
                        if (it < total) begin();
                    }
                    const float* u = v[j & 1];
#pragma unroll
                    for (int e = 0; e < kP / 2; ++e) {
                        float2& to = acc[kP / 2 * j + e];
                        const float2 t = make_float2(u[2 * e], u[2 * e + 1]);
                        if constexpr (kBlocks) to = ptx::fma2(t, ss[0], to);
                        else to = ptx::fma2(ptx::mul2(t, w[j & 1][e / 2 % 2]), ss[e / 4 * 2 + e % 2], to);
                    }
                }
            }
            if (!ok) break;
            if (g0 > 0) {  // a later part of a tile: the sums for the pair that has the first
                float4* to = p.sums + walk.pair * sums_pair + sums_at;
#pragma unroll
                for (int j = 0; j < kCols / 4; ++j)
                    __stcg(to + j * 32, make_float4(acc[2 * j].x, acc[2 * j].y, acc[2 * j + 1].x, acc[2 * j + 1].y));
                __threadfence();
                __syncwarp();
                if (lane == 0) ptx::st_release(p.flags + walk.pair * kFlags + flag_at, 1);
                continue;
            }
            for (int q = walk.pair + 1; g1 < p.KB; ++q) {  // the first part: the others' sums
                int* flag = p.flags + q * kFlags + flag_at;
                ok = __all_sync(0xffffffffu, lane != 0 || ptx::wait_flag(flag, 1, kWaitNs));
                if (!ok) break;
                __syncwarp();  // (lane 0's acquire is ordered before the other lanes' reads)
                const float4* from = p.sums + q * sums_pair + sums_at;
#pragma unroll
                for (int j = 0; j < kCols / 4; ++j) {
                    const float4 w = __ldcg(from + j * 32);
                    acc[2 * j].x += w.x;
                    acc[2 * j].y += w.y;
                    acc[2 * j + 1].x += w.z;
                    acc[2 * j + 1].y += w.w;
                }
                __syncwarp();
                if (lane == 0) *flag = 0;  // for the next call
                g1 += (int)min((int64_t)(p.KB - g1), walk.first(q + 1) - walk.first(q));
            }
            if (!ok) break;
            constexpr int kPiece = 128 / sizeof(T);
#pragma unroll
            for (int j = 0; j < kCols / kPiece; ++j)
                if (m0 < p.M && n0 + kPiece * j < p.N)
                    store_piece<T, !kBlocks, kRest>(p, &map_c, stage, j, acc + kPiece / 2 * j, m0, n0 + kPiece * j, lane);
            if constexpr (kRest) {
                if (n0 <= p.copied && p.copied < n0 + kCols) store_rest<T>(p, stage, m0, n0, lane);
            }
        }
        if (lane == 0) ptx::bulk_wait_all();
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

// How a product is dealt out over the pairs of SMs.
constexpr int kPairs = 76;
struct Plan {
    int width, pairs, whole;
    int64_t tiles;
    bool split;  // tiles are shared between pairs
};

// By estimated time, in a wide tile's group (0.38 us at M 9728 N 8192 K 8192; a narrow tile's takes
// 0.6 of that): rounds of whole tiles, wide or narrow; or, wide, all full rounds but one of whole
// tiles and the rest's groups dealt evenly, with 14 for the exchange of sums and 8 for each more
// that a tile takes. Whole tiles and dealt evenly: M 5136 N 1024 K 4096 (84 wide tiles) 36 and
// 31 us, with row scales 47 and 39 us; M = N = 1024, K 32768 84 and 48 us.
Plan plan_for(int64_t M, int64_t N, int64_t K, int64_t most, bool may_split = true) {
    const int64_t KB = (K + kGroup - 1) / kGroup, mt = (M + 255) / 256;
    const int64_t wide = mt * ((N + 255) / 256), narrow = mt * ((N + 127) / 128);
    auto rounds = [&](int64_t tiles) { return (tiles + most - 1) / most; };
    const double by_wide = (double)(rounds(wide) * KB), by_narrow = 0.6 * (double)(rounds(narrow) * KB);
    Plan plan = by_narrow < by_wide ? Plan{128, (int)(narrow < most ? narrow : most), 0, narrow, false}
                                    : Plan{256, (int)(wide < most ? wide : most), 0, wide, false};
    plan.whole = (int)(plan.tiles < INT32_MAX ? plan.tiles : INT32_MAX);
    if (!may_split || wide % most == 0 || wide * KB > INT32_MAX) return plan;
    const int64_t before = wide < most ? 0 : wide / most - 1, rest = wide - before * most;
    int64_t pairs = most;
    if (wide < most) {
        pairs = wide * KB / 8;  // 8 groups each at least
        pairs = pairs < wide ? wide : pairs > most ? most : pairs;
    }
    const double share = (double)(rest * KB) / (double)pairs;
    const double by_share = (double)(before * KB) + share + 14.0 + 8.0 * (share < (double)KB ? (double)KB / share - 1.0 : 0.0);
    if (by_share < (by_narrow < by_wide ? by_narrow : by_wide)) return Plan{256, (int)pairs, (int)(before * most), wide, true};
    return plan;
}

template <int BN, bool kBlocks, typename T>
int launch_pair(const Matmul& p, Product q, const Plan& plan, cudaStream_t stream) {
    using S = Shape<BN>;
    CUtensorMap ma, mb, mc;
    if (!tc::encode_tiled_2d(&ma, p.a, 1, p.K, p.M, p.a_ld, 128) || !tc::encode_tiled_2d(&mb, p.b, 1, p.K, p.N, p.b_ld, BN / 2))
        return SSDC_ERR_CUDA;
    if (q.tma_out) {
        if (!tc::encode_tiled_2d(&mc, p.c, sizeof(T), q.copied, p.M, p.c_ld * (int64_t)sizeof(T), 32)) return SSDC_ERR_CUDA;
    } else {
        mc = ma;  // not used
    }
    q.n_tiles = (int)((p.N + BN - 1) / BN);
    q.whole = plan.whole;
    const int pairs = plan.pairs;
    auto launch = [&](auto* k, std::atomic<uint64_t>& allowed) {
        if (allow_smem(k, (int)S::kBytes, allowed) != cudaSuccess) return (int)SSDC_ERR_CUDA;
        return launch_clusters(k, pairs, 2, plan.split, S::kThreads, S::kBytes, stream, ma, mb, mc, q);
    };
    static std::atomic<uint64_t> allowed, allowed_rest;
    if (q.tma_out && q.copied < p.N) return launch(product_pair<BN, kBlocks, T, true>, allowed_rest);
    return launch(product_pair<BN, kBlocks, T, false>, allowed);
}

template <int BN>
int launch_pair_types(const Matmul& p, const Product& q, const Plan& plan, cudaStream_t stream) {
    if (p.b_blocks)
        return p.out_bf16 ? launch_pair<BN, true, __nv_bfloat16>(p, q, plan, stream)
                          : launch_pair<BN, true, float>(p, q, plan, stream);
    return p.out_bf16 ? launch_pair<BN, false, __nv_bfloat16>(p, q, plan, stream)
                      : launch_pair<BN, false, float>(p, q, plan, stream);
}

}  // namespace

// The workspace: the status word, the flags, the sums.
constexpr size_t kHead = 16384, kSumsOfPair = (size_t)kFlags * 32 * 32 * sizeof(float4);

size_t matmul_workspace(int64_t M, int64_t N, int64_t K) {
    if (matmul_is_few(M, N, K)) return 256;
    const Plan plan = plan_for(M, N, K, kPairs);
    return plan.split ? kHead + plan.pairs * kSumsOfPair : 256;
}

int matmul_launch(const Matmul& p, cudaStream_t stream) {
    const int sms = device_sms();
    if (sms < 2) return SSDC_ERR_CUDA;
    if (matmul_is_few(p.M, p.N, p.K)) return matmul_few_launch(p, stream);
    Product q = {};
    q.a_scale = p.a_scale; q.b_scale = p.b_scale;
    q.M = p.M; q.N = p.N; q.c_ld = p.c_ld;
    q.KB = (int)((p.K + kGroup - 1) / kGroup);
    q.m_tiles = (int)((p.M + 255) / 256);
    q.c = p.c;
    const size_t e = p.out_bf16 ? 2 : 4;
    q.copied = p.N / (int64_t)(16 / e) * (int64_t)(16 / e);
    q.tma_out = (reinterpret_cast<uintptr_t>(p.c) | (uintptr_t)(p.c_ld * e)) % 16 == 0 && q.copied > 0;
    q.status = p.status;
    char* ws = reinterpret_cast<char*>(p.status);
    q.flags = reinterpret_cast<int*>(ws + 256);
    q.sums = reinterpret_cast<float4*>(ws + kHead);
    Plan plan = plan_for(p.M, p.N, p.K, kPairs);
    if (sms / 2 < kPairs) plan = plan_for(p.M, p.N, p.K, sms / 2, false);
    if (plan.tiles * q.KB > INT32_MAX) return SSDC_ERR_UNSUPPORTED;
    return plan.width == 128 ? launch_pair_types<128>(p, q, plan, stream) : launch_pair_types<256>(p, q, plan, stream);
}

}  // namespace block
}  // namespace ssdc
