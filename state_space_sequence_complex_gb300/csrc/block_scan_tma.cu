// Gated scan by TMA copies: the forward and backward passes of block_scan.cu, joined the same
// way, for arrays that tensor maps can describe (rows and strides of whole 16-byte units).
//
// The scan costs about as many instructions as HBM allows it: 2.9 elements a cycle and SM at
// 8 bytes an element leave 44 of them each. A thread that loads its rows itself spends a
// third of those on addresses. Here a warp's rows come and go as one copy for each array:
// an element is then read from shared memory at a constant offset, its result is written
// over it and copied out from there, and the next rows are on their way meanwhile.
//
// Every warp copies its own tokens and waits for them alone; the CTA meets once a tile.
//
// Measured, bfloat16 with an input gate, B 16 T 2048 D 1024: forward 49 us (5.5 TB/s; 50 with
// resets), backward 95 us (5.0 TB/s; 108 with resets); B 4 T 65536: 409 us (5.2 TB/s) and 830 us.
// Four in ten issue slots are taken, in the 16 (8 backward) warps that the registers allow: what
// is left is waits for shared memory and for the special-function unit between dependent steps.
#include <type_traits>

#include <cuda.h>
#include <cuda_runtime.h>

#include "block_common.cuh"
#include "block_kernels.h"
#include "block_scan.cuh"
#include "ptx.cuh"
#include "ssdc_kernels.h"
#include "tc_common.cuh"

namespace ssdc {
namespace block {
namespace gated {

namespace {

constexpr int kStages = 2;

struct FwdMaps {
    CUtensorMap x, f, i, h;
};
struct BwdMaps {
    CUtensorMap x, f, i, dh, dx, df, di;
};

// A lane's word of a row in shared memory: two bfloat16 channels or one fp32.
template <typename T>
struct Word;
template <>
struct Word<__nv_bfloat16> {
    static constexpr int kVec = 2;
    static __device__ __forceinline__ void get(const char* at, float (&v)[2]) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(at);
        v[0] = ptx::bf16_lo(w);
        v[1] = ptx::bf16_hi(w);
    }
    static __device__ __forceinline__ void put(char* at, const float (&v)[2]) {
        *reinterpret_cast<__nv_bfloat162*>(at) = __floats2bfloat162_rn(v[0], v[1]);
    }
};
template <>
struct Word<float> {
    static constexpr int kVec = 1;
    static __device__ __forceinline__ void get(const char* at, float (&v)[1]) { v[0] = *reinterpret_cast<const float*>(at); }
    static __device__ __forceinline__ void put(char* at, const float (&v)[1]) { *reinterpret_cast<float*>(at) = v[0]; }
};

// Copies in flight get the time to end before a CTA leaves after a wait that gave up.
__device__ __forceinline__ void pause_if(bool failed) {
    if (!failed) return;
    const uint64_t t0 = ptx::globaltimer_ns();
    while (ptx::globaltimer_ns() - t0 < 2000000) {
    }
}

// Shared memory of a CTA: for every stage and warp the rows of each array, 128 bytes a row.
template <int kTok, int kArrays>
constexpr uint32_t warp_bytes() { return kTok * 128 * kArrays; }
template <int kWarps, int kTok, int kArrays>
constexpr uint32_t smem_bytes() { return kStages * kWarps * warp_bytes<kTok, kArrays>() + 128; }

// Warps of a CTA, and tokens that a thread holds in registers. Forward (B 16 T 2048 / B 2 T 2048 /
// B 1 T 65536, D 1024, bfloat16): eight warps 49 / 11 / 205 us, four (twice the exchanges, half
// the waits for each other) 59 / 13 / 277 us.
constexpr int kFwdWarps = 8, kFwdTok = 16;
// Backward a token takes twice the registers. Two bfloat16 channels a lane: four warps of 16
// tokens (B 16 T 2048 D 1024: 94 us; eight of 8: 106 us); one fp32 channel: eight of 8
// (167 us; four of 16: 187 us).
template <typename T>
constexpr int bwd_warps() { return sizeof(T) == 2 ? 4 : 8; }
template <typename T>
constexpr int bwd_tok() { return 64 / bwd_warps<T>(); }

// Few sequences and channels leave most SMs idle, however many CTAs a cluster has. Long sequences are
// then cut into segments, and two kernels take the place of one: the first reads the segments (but
// each sequence's last) for their maps (kTotals; nothing else is written), the second walks them
// all, each from the state that the joints before it make. The inputs are read twice, by many
// more SMs.
template <typename T, bool kGate, bool kReset, bool kTotals>
__global__ void __launch_bounds__(32 * kFwdWarps, 16 / kFwdWarps) gated_fwd_tma(const __grid_constant__ FwdMaps maps, const Gated p) {
    constexpr int kVec = Word<T>::kVec, kWarps = kFwdWarps, kTok = kFwdTok, kTile = kWarps * kTok, kArrays = kGate ? 3 : 2;
    constexpr uint32_t kWarp = warp_bytes<kTok, kArrays>(), kArray = kTok * 128;
    extern __shared__ char smem_raw[];
    char* smem = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    __shared__ Totals<kVec> totals;
    __shared__ Run<kVec> part[2][kWarps][32];
    __shared__ bool stopped[2][kWarps];  // whether a warp's tokens hold a reset
    __shared__ uint64_t full[kStages][kWarps];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = ptx::cluster_ctarank(), R = ptx::cluster_nctarank();
    if (lane == 0) {
        for (int s = 0; s < kStages; ++s) ptx::mbar_init(&full[s][warp], 1);
        ptx::fence_mbar_init();
    }
    const bool in_place = R > 1 && p.h0 == p.h_last;
    if (R > 1) totals_init(totals, in_place);
    const int groups = (p.D + 32 * kVec - 1) / (32 * kVec);
    const int mine_of = p.segments - (kTotals ? 1 : 0);  // segments of a sequence in this launch
    const int group = blockIdx.x / R / mine_of, segment = blockIdx.x / R % mine_of;
    const int t_begin = segment * p.segment;
    const int b = group / groups, d0 = group % groups * 32 * kVec, d = d0 + lane * kVec;
    const bool in_d = d < p.D;
    const int T_ = p.segments > 1 ? (int)min(p.T, (int64_t)t_begin + p.segment) : (int)p.T, tiles = (T_ - t_begin + kTile - 1) / kTile;
    const int64_t state_at = (int64_t)b * p.D + d, state_rows = (p.T + SSD_GATED_STATE_TOKENS - 1) / SSD_GATED_STATE_TOKENS;
    const uint8_t* reset = kReset ? p.reset + (int64_t)b * p.T : nullptr;

    launch_dependents();
    grid_dependency_wait();
    float carry[kVec];
#pragma unroll
    for (int c = 0; c < kVec; ++c) carry[c] = p.h0 && in_d ? p.h0[state_at + c] : 0.0f;
    float through_all[kVec];  // kTotals: the factor of all tiles so far
#pragma unroll
    for (int c = 0; c < kVec; ++c) through_all[c] = 1.0f;
    if (p.segments > 1) {
        float2* joint = p.joints + (int64_t)b * p.segments * p.D + d;
#pragma unroll
        for (int c = 0; c < kVec; ++c) {
            if (kTotals) {
                // (h_last may be h0: the second kernel takes h0 from here)
                if (segment == 0 && warp == 0 && in_d) joint[c] = make_float2(kStop, carry[c]);
                carry[c] = 0.0f;
            } else {
                carry[c] = 0.0f;
                if (in_d) {
#pragma unroll 8
                    for (int s = 0; s <= segment; ++s) {
                        const float2 j = joint[(int64_t)s * p.D + c];
                        carry[c] = through<true>(j.x, j.y, carry[c]);
                    }
                }
            }
        }
    }

    // the copies of this warp's rows of the CTA's tile of a round (none where they are all past the end: the barrier's phase passes all the same)
    auto fetch = [&](int round) {
        const int t0 = t_begin + (round * (int)R + (int)rank) * kTile + warp * kTok;
        uint64_t* bar = &full[round % kStages][warp];
        if (t0 >= T_) return ptx::mbar_arrive(bar);
        char* at = smem + (round % kStages * kWarps + warp) * kWarp;
        ptx::mbar_arrive_expect_tx(bar, kWarp);
        ptx::tma_load_3d(at, &maps.x, bar, d0, t0, b);
        ptx::tma_load_3d(at + kArray, &maps.f, bar, d0, t0, b);
        if (kGate) ptx::tma_load_3d(at + 2 * kArray, &maps.i, bar, d0, t0, b);
    };
    __syncwarp();
    if (lane == 0) fetch(0);
    bool ok = true;
    const int rounds = (tiles + (int)R - 1) / (int)R;
    const int t_first = t_begin + (int)rank * kTile + warp * kTok;
    uint32_t mark_next = kReset ? mark(reset, t_first, min(kTok, T_ - t_first), lane) : 0;
    if (in_place) totals_arrive();
    for (int round = 0; round < rounds; ++round) {
        const int parity = round & 1, t0 = t_begin + (round * (int)R + (int)rank) * kTile + warp * kTok, n = min(kTok, T_ - t0);
        if (lane == 0 && round + 1 < rounds) {
            ptx::bulk_wait_read<0>();  // the rows of the round before last have been copied out
            fetch(round + 1);
        }
        __syncwarp();
        ok = ptx::mbar_wait(&full[round % kStages][warp], round / kStages & 1, ok ? kWaitNs : 0) && ok;
        char* at = smem + (round % kStages * kWarps + warp) * kWarp + lane * 4;
        float C[kTok][kVec], v[kTok][kVec], A[kVec], H[kVec];
#pragma unroll
        for (int c = 0; c < kVec; ++c) {
            A[c] = 1.0f;
            H[c] = 0.0f;
        }
#pragma unroll
        for (int k = 0; k < kTok; ++k) {
            float x[kVec], f[kVec], g[kVec];
            Word<T>::get(at + k * 128, x);
            Word<T>::get(at + kArray + k * 128, f);
            if (kGate) Word<T>::get(at + 2 * kArray + k * 128, g);
#pragma unroll
            for (int c = 0; c < kVec; ++c) {
                float u;
                if (kGate) {
                    C[k][c] = sigmoid(f[c]);
                    u = sigmoid(g[c]);
                } else {
                    sigmoid_pair(f[c], C[k][c], u);
                }
                v[k][c] = u * x[c];
            }
        }
        // (the vote waits for the load, a round ahead)
        const uint32_t stop = kReset ? marked(mark_next) : 0;
        if (kReset && round + 1 < rounds) {
            const int t1 = t0 + (int)R * kTile;
            mark_next = mark(reset, t1, min(kTok, T_ - t1), lane);
        }
        // a warp whose tokens are all there and start no document takes the short way
        const bool plain = n == kTok && (!kReset || stop == 0);
        if (plain) {
#pragma unroll
            for (int k = 0; k < kTok; ++k)
#pragma unroll
                for (int c = 0; c < kVec; ++c) {
                    H[c] = fmaf(C[k][c], H[c], v[k][c]);
                    A[c] *= C[k][c];
                }
        } else {
#pragma unroll
            for (int k = 0; k < kTok; ++k)
#pragma unroll
                for (int c = 0; c < kVec; ++c) {
                    // tokens past the end leave the state as it is
                    if (k >= n) {
                        C[k][c] = 1.0f;
                        v[k][c] = 0.0f;
                    } else if (kReset && (stop >> k & 1)) {
                        C[k][c] = kStop;
                    }
                    H[c] = through<kReset>(C[k][c], v[k][c], H[c]);
                    A[c] = both<kReset>(A[c], C[k][c]);
                }
        }
        Run<kVec> mine;
#pragma unroll
        for (int c = 0; c < kVec; ++c) {
            mine.A[c] = A[c];
            mine.H[c] = H[c];
        }
        part[parity][warp][lane] = mine;
        if (kReset && lane == 0) stopped[parity][warp] = stop != 0;
        __syncthreads();
        // the tile's warps before this one (pre); and all of them, in every warp or, where the
        // total goes to the cluster's CTAs, in the last one
        float preA[kVec], preH[kVec], allA[kVec], allH[kVec];
#pragma unroll
        for (int c = 0; c < kVec; ++c) {
            allA[c] = preA[c] = 1.0f;
            allH[c] = preH[c] = 0.0f;
        }
        const bool whole = !kReset || !__any_sync(0xffffffffu, stopped[parity][lane % kWarps]);
        auto join = [&](auto with_resets) {
            constexpr bool kStops = decltype(with_resets)::value;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                if (w > warp && R > 1) break;
                const Run<kVec> o = part[parity][w][lane];
#pragma unroll
                for (int c = 0; c < kVec; ++c) {
                    if (w == warp) {
                        preA[c] = allA[c];
                        preH[c] = allH[c];
                    }
                    allH[c] = through<kStops>(o.A[c], o.H[c], allH[c]);
                    allA[c] = both<kStops>(allA[c], o.A[c]);
                }
            }
        };
        if (whole) join(std::false_type());
        else join(std::true_type());
        float in[kVec];
        if (R > 1) {
            if (round == 0) totals_wait();
            if (warp == kWarps - 1) send_total<kVec>(totals, round, rank, R, lane, allA, allH);
            receive_totals<kVec, kReset>(totals, round, rank, R, lane, carry, in, ok);
        } else {
#pragma unroll
            for (int c = 0; c < kVec; ++c) {
                in[c] = carry[c];
                carry[c] = through<kReset>(allA[c], allH[c], carry[c]);
                if (kTotals) through_all[c] = both<kReset>(through_all[c], allA[c]);
            }
        }
        if constexpr (!kTotals) {
#pragma unroll
            for (int c = 0; c < kVec; ++c) in[c] = through<kReset>(preA[c], preH[c], in[c]);
            if (p.states && t0 % SSD_GATED_STATE_TOKENS == 0 && n > 0 && in_d) {
                float* s = p.states + ((int64_t)b * state_rows + t0 / SSD_GATED_STATE_TOKENS) * p.D + d;
#pragma unroll
                for (int c = 0; c < kVec; ++c) s[c] = in[c];
            }
            // h over x (rows past the end are not copied out)
            if (plain) {
#pragma unroll
                for (int k = 0; k < kTok; ++k) {
#pragma unroll
                    for (int c = 0; c < kVec; ++c) in[c] = fmaf(C[k][c], in[c], v[k][c]);
                    Word<T>::put(at + k * 128, in);
                }
            } else {
#pragma unroll
                for (int k = 0; k < kTok; ++k) {
#pragma unroll
                    for (int c = 0; c < kVec; ++c) in[c] = through<kReset>(C[k][c], v[k][c], in[c]);
                    Word<T>::put(at + k * 128, in);
                }
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && n > 0) {
                ptx::tma_store_3d(&maps.h, at, d0, t0, b);
                ptx::bulk_commit();
            }
        }
    }
    if (rank == 0 && warp == 0 && in_d) {
#pragma unroll
        for (int c = 0; c < kVec; ++c) {
            if (kTotals) p.joints[((int64_t)b * p.segments + segment + 1) * p.D + d + c] = make_float2(through_all[c], ok ? carry[c] : __int_as_float(0x7fffffff));
            else if (segment == p.segments - 1) p.h_last[state_at + c] = carry[c];
        }
    }
    if (lane == 0) ptx::bulk_wait_all();
    pause_if(!ok);
    leave(R, ok, p.status);
}

template <typename T, bool kGate, bool kReset>
__global__ void __launch_bounds__(32 * bwd_warps<T>(), 2) gated_bwd_tma(const __grid_constant__ BwdMaps maps, const Gated p) {
    constexpr int kVec = Word<T>::kVec, kWarps = bwd_warps<T>(), kTok = bwd_tok<T>(), kTile = kWarps * kTok, kArrays = kGate ? 4 : 3;
    static_assert(kTile == SSD_GATED_STATE_TOKENS, "a state is kept for every tile");
    constexpr uint32_t kWarp = warp_bytes<kTok, kArrays>(), kArray = kTok * 128;
    extern __shared__ char smem_raw[];
    char* smem = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    __shared__ Totals<kVec> totals;
    __shared__ Run<kVec> part[2][kWarps][32];     // A and G
    __shared__ Lane<kVec> part_h[2][kWarps][32];  // H
    __shared__ bool stopped[2][kWarps];           // whether a warp's tokens hold a reset
    __shared__ uint64_t full[kStages][kWarps];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = ptx::cluster_ctarank(), R = ptx::cluster_nctarank();
    if (lane == 0) {
        for (int s = 0; s < kStages; ++s) ptx::mbar_init(&full[s][warp], 1);
        ptx::fence_mbar_init();
    }
    const bool in_place = R > 1 && p.dh0 && p.dh0 == p.dh_last;
    if (R > 1) totals_init(totals, in_place);
    const int groups = (p.D + 32 * kVec - 1) / (32 * kVec), group = blockIdx.x / R;
    const int b = group / groups, d0 = group % groups * 32 * kVec, d = d0 + lane * kVec;
    const bool in_d = d < p.D;
    const int T_ = (int)p.T, tiles = (T_ + kTile - 1) / kTile;
    const int64_t state_at = (int64_t)b * p.D + d;
    const uint8_t* reset = kReset ? p.reset + (int64_t)b * p.T : nullptr;

    launch_dependents();
    grid_dependency_wait();
    float carry[kVec];
#pragma unroll
    for (int c = 0; c < kVec; ++c) carry[c] = p.dh_last && in_d ? p.dh_last[state_at + c] : 0.0f;

    // the first token of this warp in a round, counted from the last tile; negative: none
    auto first = [&](int round) { return (tiles - 1 - (round * (int)R + (int)rank)) * kTile + warp * kTok; };
    auto has = [&](int t0) { return t0 >= warp * kTok && t0 < T_; };
    float s_next[kVec];
    uint32_t mark_next = 0;
    auto fetch = [&](int round) {
        const int t0 = first(round);
        uint64_t* bar = &full[round % kStages][warp];
        if (!has(t0)) return ptx::mbar_arrive(bar);
        char* at = smem + (round % kStages * kWarps + warp) * kWarp;
        ptx::mbar_arrive_expect_tx(bar, kWarp);
        ptx::tma_load_3d(at + kArray, &maps.f, bar, d0, t0, b);
        if (kGate) ptx::tma_load_3d(at + 3 * kArray, &maps.i, bar, d0, t0, b);
        ptx::tma_load_3d(at, &maps.x, bar, d0, t0, b);
        ptx::tma_load_3d(at + 2 * kArray, &maps.dh, bar, d0, t0, b);
    };
    auto load_ahead = [&](int round) {  // the tile's state
        const int t0 = first(round), tile = tiles - 1 - (round * (int)R + (int)rank);
#pragma unroll
        for (int c = 0; c < kVec; ++c)
            s_next[c] = tile >= 0 && in_d ? __ldg(p.in_states + ((int64_t)b * tiles + tile) * p.D + d + c) : 0.0f;
    };
    __syncwarp();
    if (lane == 0) fetch(0);
    load_ahead(0);
    if (kReset) mark_next = mark(reset, first(0), has(first(0)) ? min(kTok, T_ - first(0)) : 0, lane);
    if (in_place) totals_arrive();
    bool ok = true;
    const int rounds = (tiles + (int)R - 1) / (int)R;
    for (int round = 0; round < rounds; ++round) {
        const int parity = round & 1, t0 = first(round), n = has(t0) ? min(kTok, T_ - t0) : 0;

        float s[kVec];
#pragma unroll
        for (int c = 0; c < kVec; ++c) s[c] = s_next[c];
        if (lane == 0 && round + 1 < rounds) {
            ptx::bulk_wait_read<0>();
            fetch(round + 1);
        }
        __syncwarp();
        ok = ptx::mbar_wait(&full[round % kStages][warp], round / kStages & 1, ok ? kWaitNs : 0) && ok;
        // x, f, dh and i in, dx, df and di out
        char *at = smem + (round % kStages * kWarps + warp) * kWarp + lane * 4, *at_f = at + kArray, *at_h = at + 2 * kArray,
             *at_i = at + 3 * kArray;
        if (round + 1 < rounds) load_ahead(round + 1);
        // a token's factor C, its input's factor u and both factors' derivatives (ca; cu with x
        // in it), and the run's A, H (states) and G (gradients)
        float C[kTok][kVec], ca[kTok][kVec], u[kTok][kVec], cu[kTok][kVec], v[kTok][kVec], A[kVec], H[kVec], G[kVec];
#pragma unroll
        for (int c = 0; c < kVec; ++c) {
            A[c] = 1.0f;
            H[c] = G[c] = 0.0f;
        }
#pragma unroll
        for (int k = 0; k < kTok; ++k) {
            float x[kVec], f[kVec], g[kVec];
            Word<T>::get(at + k * 128, x);
            Word<T>::get(at_f + k * 128, f);
            if (kGate) Word<T>::get(at_i + k * 128, g);
#pragma unroll
            for (int c = 0; c < kVec; ++c) {
                float na, nu;
                sigmoid_pair(f[c], C[k][c], na);
                ca[k][c] = C[k][c] * na;
                u[k][c] = na;
                if (kGate) sigmoid_pair(g[c], u[k][c], nu);
                v[k][c] = u[k][c] * x[c];
                if (kGate) cu[k][c] = v[k][c] * nu;
                else cu[k][c] = x[c];
            }
        }
        // (the vote waits for the load, a round ahead)
        const uint32_t stop = kReset ? marked(mark_next) : 0;
        if (kReset && round + 1 < rounds) {
            const int t1 = first(round + 1);
            mark_next = mark(reset, t1, has(t1) ? min(kTok, T_ - t1) : 0, lane);
        }
        const bool plain = n == kTok && (!kReset || stop == 0);
        if (plain) {
#pragma unroll
            for (int k = 0; k < kTok; ++k)
#pragma unroll
                for (int c = 0; c < kVec; ++c) {
                    H[c] = fmaf(C[k][c], H[c], v[k][c]);
                    A[c] *= C[k][c];
                }
#pragma unroll
            for (int k = kTok - 1; k >= 0; --k) {
                float dh[kVec];
                Word<T>::get(at_h + k * 128, dh);
#pragma unroll
                for (int c = 0; c < kVec; ++c) G[c] = C[k][c] * (dh[c] + G[c]);
            }
        } else {
#pragma unroll
            for (int k = 0; k < kTok; ++k)
#pragma unroll
                for (int c = 0; c < kVec; ++c) {
                    // tokens past the end change nothing
                    if (k >= n) {
                        C[k][c] = 1.0f;
                        v[k][c] = 0.0f;
                    } else if (kReset && (stop >> k & 1)) {
                        C[k][c] = kStop;
                    }
                    H[c] = through<kReset>(C[k][c], v[k][c], H[c]);
                    A[c] = both<kReset>(A[c], C[k][c]);
                }
#pragma unroll
            for (int k = kTok - 1; k >= 0; --k) {
                float dh[kVec];
                Word<T>::get(at_h + k * 128, dh);
#pragma unroll
                for (int c = 0; c < kVec; ++c) G[c] = through<kReset>(C[k][c], 0.0f, k < n ? dh[c] + G[c] : G[c]);
            }
        }
        Run<kVec> mine;
        Lane<kVec> mine_h;
#pragma unroll
        for (int c = 0; c < kVec; ++c) {
            mine.A[c] = A[c];
            mine.H[c] = G[c];
            mine_h.v[c] = H[c];
        }
        part[parity][warp][lane] = mine;
        if (kReset && lane == 0) stopped[parity][warp] = stop != 0;
        part_h[parity][warp][lane] = mine_h;
        __syncthreads();
        // the gradient's run through the tile's warps after this one (suf); and through all, in
        // every warp or, where the total goes to the cluster's CTAs, in the first one
        float sufA[kVec], sufG[kVec], allA[kVec], allG[kVec];
#pragma unroll
        for (int c = 0; c < kVec; ++c) {
            allA[c] = sufA[c] = 1.0f;
            allG[c] = sufG[c] = 0.0f;
        }
        const bool whole = !kReset || !__any_sync(0xffffffffu, stopped[parity][lane % kWarps]);
        auto join = [&](auto with_resets) {
            constexpr bool kStops = decltype(with_resets)::value;
#pragma unroll
            for (int w = kWarps - 1; w >= 0; --w) {
                if (w < warp && R > 1) break;
                const Run<kVec> o = part[parity][w][lane];
#pragma unroll
                for (int c = 0; c < kVec; ++c) {
                    if (w == warp) {
                        sufA[c] = allA[c];
                        sufG[c] = allG[c];
                    }
                    allG[c] = through<kStops>(o.A[c], o.H[c], allG[c]);
                    allA[c] = both<kStops>(allA[c], o.A[c]);
                }
            }
            // the state behind the tile's warps before this one
#pragma unroll
            for (int w = 0; w < kWarps - 1; ++w) {
                const Run<kVec> o = part[parity][w][lane];
                const Lane<kVec> oh = part_h[parity][w][lane];
#pragma unroll
                for (int c = 0; c < kVec; ++c)
                    if (w < warp) s[c] = through<kStops>(o.A[c], oh.v[c], s[c]);
            }
        };
        if (whole) join(std::false_type());
        else join(std::true_type());
        if (R > 1) {
            if (round == 0) totals_wait();
            if (warp == 0) send_total<kVec>(totals, round, rank, R, lane, allA, allG);
        }
        // token by token: what enters a token (nothing at a reset) makes its gate's gradient
        if (plain) {
#pragma unroll
            for (int k = 0; k < kTok; ++k)
#pragma unroll
                for (int c = 0; c < kVec; ++c) {
                    ca[k][c] *= kGate ? s[c] : s[c] - cu[k][c];
                    s[c] = fmaf(C[k][c], s[c], v[k][c]);
                }
        } else {
#pragma unroll
            for (int k = 0; k < kTok; ++k)
#pragma unroll
                for (int c = 0; c < kVec; ++c) {
                    const float before = kReset && stops(C[k][c]) ? 0.0f : s[c];
                    ca[k][c] *= kGate ? before : before - cu[k][c];
                    s[c] = through<kReset>(C[k][c], v[k][c], s[c]);
                }
        }
        float in[kVec];
        if (R > 1) {
            receive_totals<kVec, kReset>(totals, round, rank, R, lane, carry, in, ok);
        } else {
#pragma unroll
            for (int c = 0; c < kVec; ++c) {
                in[c] = carry[c];
                carry[c] = through<kReset>(allA[c], allG[c], carry[c]);
            }
        }
#pragma unroll
        for (int c = 0; c < kVec; ++c) in[c] = through<kReset>(sufA[c], sufG[c], in[c]);
#pragma unroll
        for (int k = kTok - 1; k >= 0; --k) {
            float dh[kVec], ox[kVec], of[kVec], oi[kVec];
            Word<T>::get(at_h + k * 128, dh);
#pragma unroll
            for (int c = 0; c < kVec; ++c) {
                // (rows past the end were filled with zeros)
                const float gr = dh[c] + in[c];
                ox[c] = u[k][c] * gr;
                of[c] = ca[k][c] * gr;
                oi[c] = cu[k][c] * gr;
                in[c] = C[k][c] * gr;
                if (kReset && !plain && stops(C[k][c])) in[c] = 0.0f;
            }
            Word<T>::put(at + k * 128, ox);
            Word<T>::put(at_f + k * 128, of);
            if (kGate) Word<T>::put(at_i + k * 128, oi);
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && n > 0) {
            ptx::tma_store_3d(&maps.dx, at, d0, t0, b);
            ptx::tma_store_3d(&maps.df, at_f, d0, t0, b);
            if (kGate) ptx::tma_store_3d(&maps.di, at_i, d0, t0, b);
            ptx::bulk_commit();
        }
    }
    if (p.dh0 && rank == 0 && warp == 0 && in_d) {
#pragma unroll
        for (int c = 0; c < kVec; ++c) p.dh0[state_at + c] = carry[c];
    }
    if (lane == 0) ptx::bulk_wait_all();
    pause_if(!ok);
    leave(R, ok, p.status);
}

// Whether a map can describe an array, and the map. Rows are whole 16-byte units, not only their pitch: a
// copy out of shared memory ends at such a unit, so that it would overwrite up to seven values behind a
// row that ends inside one (seen with D 33 in rows of 40: the last seven were zeros), and a lane's
// two bfloat16 channels are then always both there.
bool make_map(CUtensorMap* m, const void* q, int64_t sb, int64_t st, const Gated& p, int rows) {
    const int64_t e = p.bf16 ? 2 : 4;
    if (p.B == 1) sb = st * p.T;  // not used
    if (reinterpret_cast<uintptr_t>(q) % 16 || p.D * e % 16 || st * e % 16 || sb * e % 16 || st < p.D || sb < st) return false;
    return tc::encode_rows_3d(m, q, (int)e, p.D, p.T, p.B, st * e, sb * e, rows);
}

template <auto kKernel, typename M>
int launch(const M& maps, const Gated& p, int warps, int tile, uint32_t smem, cudaStream_t stream) {
    static std::atomic<uint64_t> allowed;
    if (allow_smem(kKernel, (int)smem, allowed) != cudaSuccess) return SSDC_ERR_CUDA;
    const int per = p.bf16 ? 64 : 32;
    const int64_t groups = (int64_t)p.B * ((p.D + per - 1) / per);
    // (B 8 T 2048 D 1024, forward / backward: clusters up to 76 CTAs 46 / 91 us, 152: 28 / 53 us, 304: 33 / 60 us)
    return launch_clusters(kKernel, groups, cluster_size((p.T + tile - 1) / tile, groups, 152), false, 32 * warps, smem, stream, maps, p);
}

// Tokens of a segment: whole tiles.
int segment_tokens(int64_t T, int64_t segments, int64_t tile) {
    const int64_t tiles = (T + tile - 1) / tile;
    return (int)((tiles + segments - 1) / segments * tile);
}

template <auto kKernel>
int launch_segments(const FwdMaps& maps, const Gated& p, int segments, uint32_t smem, cudaStream_t stream) {
    static std::atomic<uint64_t> allowed;
    if (allow_smem(kKernel, (int)smem, allowed) != cudaSuccess) return SSDC_ERR_CUDA;
    const int per = p.bf16 ? 64 : 32;
    return launch_clusters(kKernel, (int64_t)p.B * ((p.D + per - 1) / per) * segments, 1, false, 32 * kFwdWarps, smem, stream, maps, p);
}

// Fewer tokens than this are one tile of the other kernels, which start sooner: B 8 T 64 D 1024,
// calls one after another, forward 6.9 us there and 7.5 here, backward 8.0 and 8.4.
constexpr int64_t kMinTokens = 65;

template <typename T, bool kGate, bool kReset>
int fwd(const FwdMaps& m, const Gated& p, cudaStream_t stream) {
    constexpr uint32_t smem = smem_bytes<kFwdWarps, kFwdTok, kGate ? 3 : 2>();
    if (p.segments == 1) return launch<gated_fwd_tma<T, kGate, kReset, false>>(m, p, kFwdWarps, kFwdWarps * kFwdTok, smem, stream);
    const int first = launch_segments<gated_fwd_tma<T, kGate, kReset, true>>(m, p, p.segments - 1, smem, stream);
    if (first < 0) return first;
    const int second = launch_segments<gated_fwd_tma<T, kGate, kReset, false>>(m, p, p.segments, smem, stream);
    return second < 0 ? second : first + second;
}
template <typename T, bool kGate>
int fwd(const FwdMaps& m, const Gated& p, cudaStream_t stream) {
    return p.reset ? fwd<T, kGate, true>(m, p, stream) : fwd<T, kGate, false>(m, p, stream);
}
template <typename T, bool kGate>
int bwd(const BwdMaps& m, const Gated& p, cudaStream_t stream) {
    constexpr uint32_t smem = smem_bytes<bwd_warps<T>(), bwd_tok<T>(), kGate ? 4 : 3>();
    return p.reset ? launch<gated_bwd_tma<T, kGate, true>>(m, p, bwd_warps<T>(), 64, smem, stream)
                   : launch<gated_bwd_tma<T, kGate, false>>(m, p, bwd_warps<T>(), 64, smem, stream);
}

}  // namespace

int tma_fwd_launch(const Gated& call, cudaStream_t stream) {
    Gated p = call;
    if (p.T < kMinTokens || p.T > INT32_MAX - 4096) return 0;
    p.segments = 1;
    p.segment = 0;
    const int64_t segments = p.joints ? gated_segments(p.B, p.T, p.D, p.bf16) : 1;
    if (segments > 1) {
        constexpr int kTile = kFwdWarps * kFwdTok;  // (a state is kept at multiples of its half)
        p.segment = segment_tokens(p.T, segments, kTile);
        p.segments = (int)((p.T + p.segment - 1) / p.segment);
    }
    FwdMaps m;
    if (!make_map(&m.x, p.x, p.x_b, p.x_t, p, kFwdTok) || !make_map(&m.f, p.f, p.f_b, p.f_t, p, kFwdTok) ||
        !make_map(&m.h, p.h, p.h_b, p.h_t, p, kFwdTok))
        return 0;
    m.i = m.x;
    if (p.i && !make_map(&m.i, p.i, p.i_b, p.i_t, p, kFwdTok)) return 0;
    if (p.bf16) return p.i ? fwd<__nv_bfloat16, true>(m, p, stream) : fwd<__nv_bfloat16, false>(m, p, stream);
    return p.i ? fwd<float, true>(m, p, stream) : fwd<float, false>(m, p, stream);
}

int tma_bwd_launch(const Gated& p, cudaStream_t stream) {
    if (p.T < kMinTokens || p.T > INT32_MAX - 4096) return 0;
    const int rows = p.bf16 ? bwd_tok<__nv_bfloat16>() : bwd_tok<float>();
    BwdMaps m;
    if (!make_map(&m.x, p.x, p.x_b, p.x_t, p, rows) || !make_map(&m.f, p.f, p.f_b, p.f_t, p, rows) ||
        !make_map(&m.dh, p.dh, p.dh_b, p.dh_t, p, rows) || !make_map(&m.dx, p.dx, p.dx_b, p.dx_t, p, rows) ||
        !make_map(&m.df, p.df, p.df_b, p.df_t, p, rows))
        return 0;
    m.i = m.x;
    m.di = m.dx;
    if (p.i && (!make_map(&m.i, p.i, p.i_b, p.i_t, p, rows) || !make_map(&m.di, p.di, p.di_b, p.di_t, p, rows)))
        return 0;
    if (p.bf16) return p.i ? bwd<__nv_bfloat16, true>(m, p, stream) : bwd<__nv_bfloat16, false>(m, p, stream);
    return p.i ? bwd<float, true>(m, p, stream) : bwd<float, false>(m, p, stream);
}

}  // namespace gated

// Segments that fill two places on each SM, for sequences of which even clusters of eight CTAs would
// leave SMs idle, and long enough to pay for reading the inputs twice. In segments / in
// clusters, B 1, bfloat16 with an input gate: T 65536 D 64 35 / 158 us, T 65536 D 1024 160 / 208 us,
// T 16384 D 512 28 / 51 us, T 8192 D 512 18 / 26 us, fp32 T 30000 D 512 77 / 74 us; T 5000 D 1152 21 / 18 us,
// T 4096 D 64 11.6 / 11.4 us.
int gated_segments(int64_t B, int64_t T, int64_t D, bool bf16) {
    constexpr int64_t kTile = gated::kFwdWarps * gated::kFwdTok, kSlots = 2 * 152;
    const int64_t groups = B * ((D + (bf16 ? 63 : 31)) / (bf16 ? 64 : 32));
    if (groups * gated::kMaxCluster >= 152 || T < 8192) return 1;
    int64_t segments = kSlots / groups;
    const int64_t most = T / kTile < 128 ? T / kTile : 128;
    segments = segments < most ? segments : most;
    const int64_t tokens = gated::segment_tokens(T, segments, kTile);
    return (int)((T + tokens - 1) / tokens);
}

}  // namespace block
}  // namespace ssdc
