// Gated scan (include/ssdc_block.h): h_t = c_t h_{t-1} + v_t for every channel, with
// a_t = sigmoid(f_t), c_t = a_t (0 at a reset), v_t = sigmoid(i_t) x_t or (1 - a_t) x_t.
//
// A run of tokens maps the state that enters it to the one that leaves it by h -> A h + H
// with A the product of its c and H its own end state; (A2, H2) after (A1, H1) is
// (A1 A2, A2 H1 + H2). So the tokens are split in three levels: 8 tokens a thread, in
// registers; 8 warps a CTA, a tile of 64 tokens, joined through shared memory; and R tiles
// a cluster, joined through distributed shared memory. A cluster walks its channels'
// sequence R tiles at a time, the running state in registers, and every input is read
// once. All joins run in the order of the tokens, so results do not depend on timing. The
// tiles' totals travel by st.async, counted on an mbarrier of the CTA that takes them: a
// cluster barrier's release would wait for the last tile's rows to reach memory.
//
// A lane owns two adjacent channels (one where the arrays do not allow it), a warp 64: a row
// of a warp is one 128-byte line of bfloat16. Bound by HBM: 8 bytes an element (bfloat16
// with an input gate) forward, 14 backward; the next tile's rows are loaded while this
// one is joined and written. These kernels take arrays of any alignment, and sequences of one
// tile; longer ones whose rows tensor maps can describe are block_scan_tma.cu's, which need fewer
// instructions: B 16 T 2048, bfloat16, D 1023 here 96 us forward and 175 us backward, D 1024
// there 49 us (5.5 TB/s) and 95 us (5.0 TB/s).
#include <cuda_runtime.h>

#include "block_common.cuh"
#include "block_kernels.h"
#include "block_scan.cuh"
#include "ptx.cuh"
#include "ssdc_kernels.h"

namespace ssdc {
namespace block {

namespace {

using namespace gated;

constexpr int kWarps = 8, kThreads = 32 * kWarps, kTok = 8, kTile = kWarps * kTok;
static_assert(kTile == SSD_GATED_STATE_TOKENS, "a state is kept for every tile");

// kVec adjacent channels of one token, as they are in memory.
template <typename T, int kVec>
struct Raw;
template <>
struct Raw<__nv_bfloat16, 2> {
    uint32_t w;
    __device__ __forceinline__ void zero() { w = 0; }
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = __ldg(reinterpret_cast<const uint32_t*>(p)); }
    __device__ __forceinline__ float get(int k) const { return k ? ptx::bf16_hi(w) : ptx::bf16_lo(w); }
};
template <>
struct Raw<__nv_bfloat16, 1> {
    uint16_t w;
    __device__ __forceinline__ void zero() { w = 0; }
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = __ldg(reinterpret_cast<const uint16_t*>(p)); }
    __device__ __forceinline__ float get(int) const { return ptx::bf16_lo(w); }
};
template <>
struct Raw<float, 2> {
    float2 w;
    __device__ __forceinline__ void zero() { w = make_float2(0.0f, 0.0f); }
    __device__ __forceinline__ void load(const float* p) { w = __ldg(reinterpret_cast<const float2*>(p)); }
    __device__ __forceinline__ float get(int k) const { return k ? w.y : w.x; }
};
template <>
struct Raw<float, 1> {
    float w;
    __device__ __forceinline__ void zero() { w = 0.0f; }
    __device__ __forceinline__ void load(const float* p) { w = __ldg(p); }
    __device__ __forceinline__ float get(int) const { return w; }
};

template <int kVec>
__device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[kVec]) {
    if constexpr (kVec == 2) *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v[0], v[1]);
    else *p = __float2bfloat16_rn(v[0]);
}
template <int kVec>
__device__ __forceinline__ void store(float* p, const float (&v)[kVec]) {
    if constexpr (kVec == 2) *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
    else *p = v[0];
}

// Row k of a few, from the first: the token stride in bytes has 32 bits, so that this is one instruction.
template <typename T>
__device__ __forceinline__ T* row(T* first, int k, int32_t stride) {
    return reinterpret_cast<T*>(reinterpret_cast<uintptr_t>(first) + (int64_t)k * stride);
}

template <typename T, int kVec, bool kGate, bool kReset>
__global__ void __launch_bounds__(kThreads, kVec == 2 ? 2 : 3) gated_fwd(const Gated p) {
    __shared__ Totals<kVec> totals;
    __shared__ Run<kVec> part[2][kWarps][32];
    // (the warp's index from a shuffle: what depends on it alone is then computed once a warp)
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    const uint32_t rank = ptx::cluster_ctarank(), R = ptx::cluster_nctarank();
    const bool in_place = R > 1 && p.h0 == p.h_last;
    totals_init(totals, in_place);
    const int64_t groups = (p.D + 32 * kVec - 1) / (32 * kVec), group = blockIdx.x / R;
    const int b = (int)(group / groups), d = (int)(group % groups) * 32 * kVec + lane * kVec;
    const bool in_d = d < p.D;
    const int64_t tiles = (p.T + kTile - 1) / kTile;
    // rows of the batch row b; dl: this lane's channels, or the last ones where there are none
    constexpr int32_t e = sizeof(T);
    const int32_t st_x = (int32_t)p.x_t * e, st_f = (int32_t)p.f_t * e, st_i = (int32_t)p.i_t * e, st_h = (int32_t)p.h_t * e;
    const T* x = static_cast<const T*>(p.x) + b * p.x_b;
    const T* f = static_cast<const T*>(p.f) + b * p.f_b;
    const T* g = kGate ? static_cast<const T*>(p.i) + b * p.i_b : nullptr;
    T* h = static_cast<T*>(p.h) + b * p.h_b;
    const uint32_t dl = in_d ? d : p.D - kVec;
    const uint8_t* reset = kReset ? p.reset + (int64_t)b * p.T : nullptr;

    launch_dependents();
    grid_dependency_wait();
    float carry[kVec];
#pragma unroll
    for (int c = 0; c < kVec; ++c) carry[c] = p.h0 && in_d ? p.h0[(int64_t)b * p.D + d + c] : 0.0f;

    Raw<T, kVec> rx[kTok], rf[kTok], rg[kTok];
    int n = 0;          // tokens of this warp, the same for all lanes
    uint32_t first = 0;  // whether a document starts at the lane's token
    auto load = [&](int64_t tile) {
        const int64_t t0 = tile * kTile + warp * kTok;
        n = (int)max((int64_t)0, min((int64_t)kTok, p.T - t0));
        if (kReset) first = mark(reset, t0, n, lane);
        const T *px = x + t0 * p.x_t + dl, *pf = f + t0 * p.f_t + dl, *pg = kGate ? g + t0 * p.i_t + dl : nullptr;
        if (n == kTok) {
#pragma unroll
            for (int k = 0; k < kTok; ++k) {
                rf[k].load(row(pf, k, st_f));
                if (kGate) rg[k].load(row(pg, k, st_i));
                rx[k].load(row(px, k, st_x));
            }
        } else {
#pragma unroll
            for (int k = 0; k < kTok; ++k) {
                rx[k].zero();
                rf[k].zero();
                if (kGate) rg[k].zero();
                if (k < n) {
                    rf[k].load(row(pf, k, st_f));
                    if (kGate) rg[k].load(row(pg, k, st_i));
                    rx[k].load(row(px, k, st_x));
                }
            }
        }
    };
    load(rank);
    if (in_place) totals_arrive();
    bool ok = true;
    int64_t round = 0;
    for (int64_t tile = rank; tile - rank < tiles; tile += R, ++round) {
        const int parity = (int)(round & 1);
        const int rows = n;
        const uint32_t stop = kReset ? marked(first) : 0;
        // a warp whose tokens are all there and start no document takes the short way
        const bool plain = rows == kTok && (!kReset || stop == 0);
        float C[kTok][kVec], v[kTok][kVec], A[kVec], H[kVec];
#pragma unroll
        for (int c = 0; c < kVec; ++c) {
            A[c] = 1.0f;
            H[c] = 0.0f;
        }
#pragma unroll
        for (int k = 0; k < kTok; ++k)
#pragma unroll
            for (int c = 0; c < kVec; ++c) {
                float u;
                if (kGate) {
                    C[k][c] = sigmoid(rf[k].get(c));
                    u = sigmoid(rg[k].get(c));
                } else {
                    sigmoid_pair(rf[k].get(c), C[k][c], u);
                }
                v[k][c] = u * rx[k].get(c);
            }
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
                    if (k >= rows) {
                        C[k][c] = 1.0f;
                        v[k][c] = 0.0f;
                    } else if (kReset && (stop >> k & 1)) {
                        C[k][c] = kStop;
                    }
                    H[c] = through<kReset>(C[k][c], v[k][c], H[c]);
                    A[c] = both<kReset>(A[c], C[k][c]);
                }
        }
        if (tile - rank + R < tiles) load(tile + R);
        Run<kVec> mine;
#pragma unroll
        for (int c = 0; c < kVec; ++c) {
            mine.A[c] = A[c];
            mine.H[c] = H[c];
        }
        part[parity][warp][lane] = mine;
        __syncthreads();
        // the tile's warps before this one; the last warp adds its own and has the tile's total
        float preA[kVec], preH[kVec];
#pragma unroll
        for (int c = 0; c < kVec; ++c) {
            preA[c] = 1.0f;
            preH[c] = 0.0f;
        }
#pragma unroll 1
        for (int w = 0; w < warp; ++w) {
            const Run<kVec> o = part[parity][w][lane];
#pragma unroll
            for (int c = 0; c < kVec; ++c) {
                preH[c] = through<kReset>(o.A[c], o.H[c], preH[c]);
                preA[c] = both<kReset>(preA[c], o.A[c]);
            }
        }
        if (round == 0) totals_wait();
        if (warp == kWarps - 1) {
#pragma unroll
            for (int c = 0; c < kVec; ++c) {
                H[c] = through<kReset>(A[c], H[c], preH[c]);
                A[c] = both<kReset>(preA[c], A[c]);
            }
            send_total<kVec>(totals, round, rank, R, lane, A, H);
        }
        float in[kVec];
        receive_totals<kVec, kReset>(totals, round, rank, R, lane, carry, in, ok);
        if (p.states && warp == 0 && in_d && tile < tiles) {
            float* s = p.states + ((int64_t)b * tiles + tile) * p.D + d;
#pragma unroll
            for (int c = 0; c < kVec; ++c) s[c] = in[c];
        }
#pragma unroll
        for (int c = 0; c < kVec; ++c) in[c] = through<kReset>(preA[c], preH[c], in[c]);
        T* ph = h + (tile * kTile + warp * kTok) * p.h_t + dl;
        if (plain) {
#pragma unroll
            for (int k = 0; k < kTok; ++k) {
#pragma unroll
                for (int c = 0; c < kVec; ++c) in[c] = fmaf(C[k][c], in[c], v[k][c]);
                if (in_d) store<kVec>(row(ph, k, st_h), in);
            }
        } else {
#pragma unroll
            for (int k = 0; k < kTok; ++k) {
#pragma unroll
                for (int c = 0; c < kVec; ++c) in[c] = through<kReset>(C[k][c], v[k][c], in[c]);
                if (k < rows && in_d) store<kVec>(row(ph, k, st_h), in);
            }
        }
    }
    if (rank == 0 && warp == 0 && in_d) {
#pragma unroll
        for (int c = 0; c < kVec; ++c) p.h_last[(int64_t)b * p.D + d + c] = carry[c];
    }
    leave(R, ok, p.status);
}

// Backward, from the last tile to the first: with k_t = c_{t+1} g_{t+1} the gradient that enters
// token t from its right, g_t = dh_t + k_t and k_{t-1} = c_t g_t, so a run of tokens maps
// k -> A k + G with the same A as forward. Each tile's states are recomputed from the one
// that the forward pass kept for it. The next tile's rows are fetched into L2 meanwhile.
template <typename T, int kVec, bool kGate, bool kReset>
__global__ void __launch_bounds__(kThreads, 2) gated_bwd(const Gated p) {
    __shared__ Totals<kVec> totals;
    __shared__ Run<kVec> part[2][kWarps][32];        // A and G
    __shared__ Lane<kVec> part_h[2][kWarps][32];     // H
    // (the warp's index from a shuffle: what depends on it alone is then computed once a warp)
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    const uint32_t rank = ptx::cluster_ctarank(), R = ptx::cluster_nctarank();
    const bool in_place = R > 1 && p.dh0 && p.dh0 == p.dh_last;
    totals_init(totals, in_place);
    const int64_t groups = (p.D + 32 * kVec - 1) / (32 * kVec), group = blockIdx.x / R;
    const int b = (int)(group / groups), d0 = (int)(group % groups) * 32 * kVec, d = d0 + lane * kVec;
    const bool in_d = d < p.D;
    const int64_t tiles = (p.T + kTile - 1) / kTile;
    const T* x = static_cast<const T*>(p.x) + b * p.x_b;
    const T* f = static_cast<const T*>(p.f) + b * p.f_b;
    const T* g = kGate ? static_cast<const T*>(p.i) + b * p.i_b : nullptr;
    constexpr int32_t e = sizeof(T);
    const int32_t st_x = (int32_t)p.x_t * e, st_f = (int32_t)p.f_t * e, st_i = (int32_t)p.i_t * e, st_dh = (int32_t)p.dh_t * e;
    const int32_t st_dx = (int32_t)p.dx_t * e, st_df = (int32_t)p.df_t * e, st_di = (int32_t)p.di_t * e;
    const T* dh = static_cast<const T*>(p.dh) + b * p.dh_b;
    T* dx = static_cast<T*>(p.dx) + b * p.dx_b;
    T* df = static_cast<T*>(p.df) + b * p.df_b;
    T* di = kGate ? static_cast<T*>(p.di) + b * p.di_b : nullptr;
    const uint32_t dl = in_d ? d : p.D - kVec;
    const uint8_t* reset = kReset ? p.reset + (int64_t)b * p.T : nullptr;
    // the row that this lane fetches for its warp: one of 8 tokens of one of the 4 arrays
    const int fetch = lane / kTok;
    const T* fetch_at = (fetch == 0 ? x : fetch == 1 ? f : fetch == 2 ? dh : kGate ? g : x) + d0;
    const int64_t fetch_t = fetch == 0 ? p.x_t : fetch == 1 ? p.f_t : fetch == 2 ? p.dh_t : kGate ? p.i_t : p.x_t;

    launch_dependents();
    grid_dependency_wait();
    float carry[kVec];
#pragma unroll
    for (int c = 0; c < kVec; ++c) carry[c] = p.dh_last && in_d ? p.dh_last[(int64_t)b * p.D + d + c] : 0.0f;

    bool ok = true;
    int64_t round = 0;
    for (int64_t back = rank; back - rank < tiles; back += R, ++round) {
        const int parity = (int)(round & 1);
        const int64_t tile = tiles - 1 - back, t0 = tile * kTile + warp * kTok;
        const int n = tile < 0 ? 0 : (int)max((int64_t)0, min((int64_t)kTok, p.T - t0));
        const uint32_t first = kReset ? mark(reset, t0, n, lane) : 0;
        Raw<T, kVec> rx[kTok], rf[kTok], rg[kTok], rh[kTok];
        float s[kVec];
#pragma unroll
        for (int c = 0; c < kVec; ++c)
            s[c] = tile >= 0 && in_d ? __ldg(p.in_states + ((int64_t)b * tiles + tile) * p.D + d + c) : 0.0f;
        {
            const T *px = x + t0 * p.x_t + dl, *pf = f + t0 * p.f_t + dl, *ph = dh + t0 * p.dh_t + dl;
            const T* pg = kGate ? g + t0 * p.i_t + dl : nullptr;
            if (n == kTok) {
#pragma unroll
                for (int k = 0; k < kTok; ++k) {
                    rf[k].load(row(pf, k, st_f));
                    if (kGate) rg[k].load(row(pg, k, st_i));
                    rx[k].load(row(px, k, st_x));
                    rh[k].load(row(ph, k, st_dh));
                }
            } else {
#pragma unroll
                for (int k = 0; k < kTok; ++k) {
                    rx[k].zero();
                    rf[k].zero();
                    rh[k].zero();
                    if (kGate) rg[k].zero();
                    if (k < n) {
                        rf[k].load(row(pf, k, st_f));
                        if (kGate) rg[k].load(row(pg, k, st_i));
                        rx[k].load(row(px, k, st_x));
                        rh[k].load(row(ph, k, st_dh));
                    }
                }
            }
            // (a tile before this one is full)
            const int64_t next = tile - R;
            if (next >= 0) {
                const T* q = fetch_at + (next * kTile + warp * kTok + lane % kTok) * fetch_t;
                ptx::prefetch_l2(q);
                if (sizeof(T) * kVec * 32 > 128 && d0 + 32 < p.D) ptx::prefetch_l2(q + 32);
            }
        }
        if (in_place && round == 0) totals_arrive();
        const uint32_t stop = kReset ? marked(first) : 0;
        const bool plain = n == kTok && (!kReset || stop == 0);
        // a token's factor C, its input's factor u and both factors' derivatives (ca; cu with x
        // in it), and the run's A, H (states) and G (gradients)
        float C[kTok][kVec], ca[kTok][kVec], u[kTok][kVec], cu[kTok][kVec], A[kVec], H[kVec], G[kVec];
#pragma unroll
        for (int c = 0; c < kVec; ++c) {
            A[c] = 1.0f;
            H[c] = G[c] = 0.0f;
        }
#pragma unroll
        for (int k = 0; k < kTok; ++k)
#pragma unroll
            for (int c = 0; c < kVec; ++c) {
                float na, nu;
                sigmoid_pair(rf[k].get(c), C[k][c], na);
                ca[k][c] = C[k][c] * na;
                u[k][c] = na;
                if (kGate) {
                    sigmoid_pair(rg[k].get(c), u[k][c], nu);
                    cu[k][c] = rx[k].get(c) * (u[k][c] * nu);
                }
            }
        if (plain) {
#pragma unroll
            for (int k = 0; k < kTok; ++k)
#pragma unroll
                for (int c = 0; c < kVec; ++c) {
                    H[c] = fmaf(C[k][c], H[c], u[k][c] * rx[k].get(c));
                    A[c] *= C[k][c];
                }
#pragma unroll
            for (int k = kTok - 1; k >= 0; --k)
#pragma unroll
                for (int c = 0; c < kVec; ++c) G[c] = C[k][c] * (rh[k].get(c) + G[c]);
        } else {
#pragma unroll
            for (int k = 0; k < kTok; ++k)
#pragma unroll
                for (int c = 0; c < kVec; ++c) {
                    // tokens past the end change nothing (their rows are zero)
                    if (k >= n) C[k][c] = 1.0f;
                    else if (kReset && (stop >> k & 1)) C[k][c] = kStop;
                    H[c] = through<kReset>(C[k][c], u[k][c] * rx[k].get(c), H[c]);
                    A[c] = both<kReset>(A[c], C[k][c]);
                }
#pragma unroll
            for (int k = kTok - 1; k >= 0; --k)
#pragma unroll
                for (int c = 0; c < kVec; ++c) G[c] = through<kReset>(C[k][c], 0.0f, rh[k].get(c) + G[c]);
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
        part_h[parity][warp][lane] = mine_h;
        __syncthreads();
        // the gradient's run through the tile's warps after this one; the first warp adds its own
        // and has the tile's total
        float sufA[kVec], sufG[kVec];
#pragma unroll
        for (int c = 0; c < kVec; ++c) {
            sufA[c] = 1.0f;
            sufG[c] = 0.0f;
        }
#pragma unroll 1
        for (int w = kWarps - 1; w > warp; --w) {
            const Run<kVec> o = part[parity][w][lane];
#pragma unroll
            for (int c = 0; c < kVec; ++c) {
                sufG[c] = through<kReset>(o.A[c], o.H[c], sufG[c]);
                sufA[c] = both<kReset>(sufA[c], o.A[c]);
            }
        }
        if (round == 0) totals_wait();
        if (warp == 0) {
#pragma unroll
            for (int c = 0; c < kVec; ++c) {
                G[c] = through<kReset>(A[c], G[c], sufG[c]);
                A[c] = both<kReset>(sufA[c], A[c]);
            }
            send_total<kVec>(totals, round, rank, R, lane, A, G);
        }
        // the state behind the tile's warps before this one, then token by token: what enters a
        // token (nothing at a reset) makes its gate's gradient
#pragma unroll 1
        for (int w = 0; w < warp; ++w) {
            const Run<kVec> o = part[parity][w][lane];
            const Lane<kVec> oh = part_h[parity][w][lane];
#pragma unroll
            for (int c = 0; c < kVec; ++c) s[c] = through<kReset>(o.A[c], oh.v[c], s[c]);
        }
#pragma unroll
        for (int k = 0; k < kTok; ++k)
#pragma unroll
            for (int c = 0; c < kVec; ++c) {
                const float xv = rx[k].get(c), before = kReset && stops(C[k][c]) ? 0.0f : s[c];
                ca[k][c] *= kGate ? before : before - xv;
                s[c] = through<kReset>(C[k][c], u[k][c] * xv, s[c]);
            }
        float in[kVec];
        receive_totals<kVec, kReset>(totals, round, rank, R, lane, carry, in, ok);
#pragma unroll
        for (int c = 0; c < kVec; ++c) in[c] = through<kReset>(sufA[c], sufG[c], in[c]);
        T *px = dx + t0 * p.dx_t + dl, *pf = df + t0 * p.df_t + dl, *pi = kGate ? di + t0 * p.di_t + dl : nullptr;
#pragma unroll
        for (int k = kTok - 1; k >= 0; --k) {
            float ox[kVec], of[kVec], oi[kVec];
#pragma unroll
            for (int c = 0; c < kVec; ++c) {
                const float gr = rh[k].get(c) + in[c];
                ox[c] = u[k][c] * gr;
                of[c] = ca[k][c] * gr;
                if (kGate) oi[c] = cu[k][c] * gr;
                in[c] = kReset && stops(C[k][c]) ? 0.0f : C[k][c] * gr;
            }
            if (in_d && k < n) {
                store<kVec>(row(px, k, st_dx), ox);
                store<kVec>(row(pf, k, st_df), of);
                if (kGate) store<kVec>(row(pi, k, st_di), oi);
            }
        }
    }
    if (p.dh0 && rank == 0 && warp == 0 && in_d) {
#pragma unroll
        for (int c = 0; c < kVec; ++c) p.dh0[(int64_t)b * p.D + d + c] = carry[c];
    }
    leave(R, ok, p.status);
}

// One token: a thread a channel pair (or channel). Bound by the launch.
template <typename T, int kVec, bool kGate>
__global__ void __launch_bounds__(128) gated_step(const Gated p) {
    launch_dependents();
    grid_dependency_wait();
    const int64_t per = (p.D + kVec - 1) / kVec, i = (int64_t)blockIdx.x * 128 + threadIdx.x;
    if (i >= p.B * per) return;
    const int64_t b = i / per, d = (i - b * per) * kVec;
    Raw<T, kVec> rx, rf, rg;
    rx.load(static_cast<const T*>(p.x) + b * p.x_b + d);
    rf.load(static_cast<const T*>(p.f) + b * p.f_b + d);
    if (kGate) rg.load(static_cast<const T*>(p.i) + b * p.i_b + d);
    float s[kVec];
#pragma unroll
    for (int c = 0; c < kVec; ++c) {
        float a, r, u;
        sigmoid_pair(rf.get(c), a, r);
        u = r;
        if (kGate) sigmoid_pair(rg.get(c), u, r);
        s[c] = fmaf(a, p.h0[b * p.D + d + c], u * rx.get(c));
        p.h_last[b * p.D + d + c] = s[c];
    }
    store<kVec>(static_cast<T*>(p.h) + b * p.h_b + d, s);
}

// Whether every row of an array allows loads of two channels.
bool pairs_ok(const void* q, int64_t sb, int64_t st, size_t elem) {
    return q == nullptr || (reinterpret_cast<uintptr_t>(q) % (2 * elem) == 0 && sb % 2 == 0 && st % 2 == 0);
}

template <typename K>
int launch_cluster(K kernel, const Gated& p, int vec, int ctas, cudaStream_t stream) {
    const int64_t groups = (int64_t)p.B * ((p.D + 32 * vec - 1) / (32 * vec));
    return launch_clusters(kernel, groups, cluster_size((p.T + kTile - 1) / kTile, groups, ctas), false, kThreads, 0, stream, p);
}

// CTAs that the clusters are made to reach, bfloat16, D 1023 (forward / backward): B 2 T 2048
// 456: 17.7 / 27.9 us, 152: 19.1 / 25.3 us; B 4 T 4096 456: 54.6 / 92.7 us, 152: 66.9 / 90.7 us.
constexpr int kFwdCtas = 3 * 152, kBwdCtas = 152;

template <typename T, int kVec, bool kGate>
int launch(const Gated& p, int what, cudaStream_t stream) {
    if (what == 0 && p.reset) return launch_cluster(gated_fwd<T, kVec, kGate, true>, p, kVec, kFwdCtas, stream);
    if (what == 0) return launch_cluster(gated_fwd<T, kVec, kGate, false>, p, kVec, kFwdCtas, stream);
    if (what == 1 && p.reset) return launch_cluster(gated_bwd<T, kVec, kGate, true>, p, kVec, kBwdCtas, stream);
    if (what == 1) return launch_cluster(gated_bwd<T, kVec, kGate, false>, p, kVec, kBwdCtas, stream);
    const int64_t n = (int64_t)p.B * ((p.D + kVec - 1) / kVec);
    return launch_dependent(gated_step<T, kVec, kGate>, dim3((unsigned)((n + 127) / 128)), dim3(128), 0, stream, p) == cudaSuccess
               ? 1
               : SSDC_ERR_CUDA;
}

template <typename T>
int launch_types(const Gated& p, int what, cudaStream_t stream) {
    const size_t e = sizeof(T);
    const bool two = p.D % 2 == 0 && pairs_ok(p.x, p.x_b, p.x_t, e) && pairs_ok(p.f, p.f_b, p.f_t, e) &&
                     pairs_ok(p.i, p.i_b, p.i_t, e) && pairs_ok(p.h, p.h_b, p.h_t, e) &&
                     pairs_ok(p.dh, p.dh_b, p.dh_t, e) && pairs_ok(p.dx, p.dx_b, p.dx_t, e) &&
                     pairs_ok(p.df, p.df_b, p.df_t, e) && pairs_ok(p.di, p.di_b, p.di_t, e);
    if (p.i) return two ? launch<T, 2, true>(p, what, stream) : launch<T, 1, true>(p, what, stream);
    return two ? launch<T, 2, false>(p, what, stream) : launch<T, 1, false>(p, what, stream);
}

int launch_scan(const Gated& p, int what, cudaStream_t stream) {
    return p.bf16 ? launch_types<__nv_bfloat16>(p, what, stream) : launch_types<float>(p, what, stream);
}

}  // namespace

int gated_fwd_launch(const Gated& p, cudaStream_t stream) {
    const int n = gated::tma_fwd_launch(p, stream);
    return n != 0 ? n : launch_scan(p, 0, stream);
}
int gated_bwd_launch(const Gated& p, cudaStream_t stream) {
    const int n = gated::tma_bwd_launch(p, stream);
    return n != 0 ? n : launch_scan(p, 1, stream);
}
int gated_step_launch(const Gated& p, cudaStream_t stream) { return launch_scan(p, 2, stream); }

}  // namespace block
}  // namespace ssdc
