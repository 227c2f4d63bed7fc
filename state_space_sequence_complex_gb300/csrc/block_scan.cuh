// What the gated scan's kernels share (block_scan.cu, block_scan_tma.cu): how runs of tokens
// are joined, within a tile and across the tiles of a cluster.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "block_common.cuh"
#include "block_kernels.h"
#include "ptx.cuh"

namespace ssdc {
namespace block {
namespace gated {

constexpr int kMaxCluster = 8;

// A reset stops everything that comes before it, an infinity or a NaN too, so it is not the
// factor 0 but a mark of its own in A: the value -0, which no product of gates takes.
constexpr float kStop = -0.0f;
__device__ __forceinline__ bool stops(float A) { return __float_as_uint(A) == 0x80000000u; }
// The state behind a run, from the one before it.
template <bool kReset>
__device__ __forceinline__ float through(float A, float H, float h) {
    return kReset && stops(A) ? H : fmaf(A, h, H);
}
// The factor of two runs, the first one first.
template <bool kReset>
__device__ __forceinline__ float both(float A1, float A2) {
    return kReset && (stops(A1) || stops(A2)) ? kStop : A1 * A2;
}

// A run of tokens for a lane's channels, as it goes through shared memory.
template <int kVec>
struct alignas(8 * kVec) Run {
    float A[kVec], H[kVec];
};
template <int kVec>
struct alignas(4 * kVec) Lane {
    float v[kVec];
};

// The totals of the cluster's tiles, by tile, for this CTA's channels: A and H of each of a
// lane's channels. Two of them, with a barrier each, by the parity of the round: a CTA that
// sends its total of round i + 2 has taken every CTA's of round i + 1, which each sent when
// it had used round i's.
template <int kVec>
struct Totals {
    Run<kVec> v[2][kMaxCluster][32];
    uint64_t full[2];
};
constexpr uint64_t kWaitNs = 2000000000ull;  // wait limit

// Before the first totals are sent, every CTA of the cluster has to run and to have its barriers: it
// arrives on the cluster's barrier (totals_init) and waits for it (totals_wait). Where the last state
// takes the place of the first (h_last is h0, dh0 dh_last), every CTA must have read that first: it
// arrives behind this load (totals_arrive), and behind the first rows', which would else wait for it. So
// late an arrival costs 0.7 us (B 2 T 2048 D 1024 bfloat16, forward: 10.0 us for 9.3).
__device__ __forceinline__ void totals_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void totals_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
template <int kVec>
__device__ __forceinline__ void totals_init(Totals<kVec>& t, bool in_place) {
    if (threadIdx.x == 0) {
        ptx::mbar_init(&t.full[0], 1);
        ptx::mbar_init(&t.full[1], 1);
        ptx::fence_mbar_init();
    }
    if (!in_place) totals_arrive();
}

// This CTA's total to every CTA of the cluster, its own too; by one warp.
template <int kVec>
__device__ __forceinline__ void send_total(Totals<kVec>& t, int64_t round, uint32_t rank, uint32_t R, int lane,
                                           const float (&A)[kVec], const float (&H)[kVec]) {
    const int parity = (int)(round & 1);
    if (lane == 0) ptx::mbar_arrive_expect_tx(&t.full[parity], R * 32 * 8 * kVec);
    const uint32_t at = ptx::smem_addr(&t.v[parity][rank][lane]), full = ptx::smem_addr(&t.full[parity]);
    for (uint32_t r = 0; r < R; ++r) {
        const uint32_t to = ptx::mapa(at, r), bar = ptx::mapa(full, r);
        if constexpr (kVec == 2) ptx::st_async_v4(to, make_float4(A[0], A[1], H[0], H[1]), bar);
        else ptx::st_async_v2(to, make_float2(A[0], H[0]), bar);
    }
}

// A wait that gives up makes the results NaN from there on, and later waits give up at once.
template <int kVec, bool kReset>
__device__ __forceinline__ void receive_totals(Totals<kVec>& t, int64_t round, uint32_t rank, uint32_t R, int lane,
                                               float (&carry)[kVec], float (&in)[kVec], bool& ok) {
    const int parity = (int)(round & 1);
    ok = ptx::mbar_wait(&t.full[parity], (uint32_t)(round >> 1) & 1, ok ? kWaitNs : 0) && ok;
    if (!ok) {
#pragma unroll
        for (int c = 0; c < kVec; ++c) carry[c] = __int_as_float(0x7fffffff);
    }
#pragma unroll
    for (int c = 0; c < kVec; ++c) in[c] = carry[c];
    for (uint32_t r = 0; r < R; ++r) {
        const Run<kVec> o = t.v[parity][r][lane];
#pragma unroll
        for (int c = 0; c < kVec; ++c) {
            carry[c] = through<kReset>(o.A[c], o.H[c], carry[c]);
            if (r < rank) in[c] = carry[c];
        }
    }
}

// No CTA leaves while another may still send to it (where a wait gave up).
__device__ __forceinline__ void leave(uint32_t R, bool ok, int* status) {
    if (!ok && status) atomicCAS(status, SSDC_OK, SSDC_ERR_TIMEOUT);
    if (R > 1) {
        ptx::cluster_arrive_relaxed();
        ptx::cluster_wait();
    }
}

// The marks of a warp's tokens that start a document, one bit each: the lane's token is marked.
// (The vote waits for the load. Voted on when loaded, a round ahead, B 16 T 2048 D 1024 bfloat16
// took 54 us forward and 119 backward; a round later, where it is used, 50 and 108.)
__device__ __forceinline__ uint32_t mark(const uint8_t* reset, int64_t t0, int n, int lane) {
    return lane < n ? __ldg(reset + t0 + lane) : 0;
}
__device__ __forceinline__ uint32_t marked(uint32_t mark) { return __ballot_sync(0xffffffffu, mark != 0); }

// Tiles that a cluster takes at a time: so many that the clusters reach `ctas` CTAs, which each
// kernel's launch gives, with as few exchanges as that allows.
inline int cluster_size(int64_t tiles, int64_t groups, int ctas) {
    int R = 1;
    while (R < kMaxCluster && R < tiles && groups * R < ctas) R *= 2;
    return R;
}

// The forward and backward passes by TMA copies (block_scan_tma.cu): the launches, or 0 where
// the arrays or sizes do not allow it.
int tma_fwd_launch(const Gated& p, cudaStream_t stream);
int tma_bwd_launch(const Gated& p, cudaStream_t stream);

}  // namespace gated
}  // namespace block
}  // namespace ssdc
