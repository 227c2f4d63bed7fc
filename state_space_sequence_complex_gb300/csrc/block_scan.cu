// Gated scan (include/ssdc_block.h): h_t = c_t h_{t-1} + v_t for every channel, with
// a_t = sigmoid(f_t), c_t = a_t (0 at a reset), v_t = sigmoid(i_t) x_t or (1 - a_t) x_t.
//
// A run of tokens maps the state that enters it to the one that leaves it by h -> A h + H
// with A the product of its c and H its own end state; (A2, H2) after (A1, H1) is
// (A1 A2, A2 H1 + H2). So the tokens are split in three levels: 8 tokens a thread, in
// registers; 8 warps a CTA, a tile of 64 tokens, joined through shared memory; and R tiles
// a cluster, joined through distributed shared memory. A cluster walks its channels'
// sequence R tiles at a time, the running state in registers, and every input is read
// once. All joins run in the order of the tokens, so results do not depend on timing.
//
// A lane owns two adjacent channels (one where the arrays do not allow it), a warp 64: a row
// of a warp is one 128-byte line of bfloat16. Bound by HBM: 8 bytes an element (bfloat16
// with an input gate) forward, 14 backward; the next tile's rows are loaded while this
// one is joined and written.
#include <cuda_runtime.h>

#include "block_common.cuh"
#include "block_kernels.h"
#include "ptx.cuh"
#include "ssdc_kernels.h"

namespace ssdc {
namespace block {

namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps, kTok = 8, kTile = kWarps * kTok;
static_assert(kTile == SSD_GATED_STATE_TOKENS, "a state is kept for every tile");
constexpr int kMaxCluster = kWarps;  // one warp sends to each CTA of the cluster

// A reset stops everything that comes before it, an infinity or a NaN too, so it is not the
// factor 0 but a mark of its own in A: the value -0, which no product of gates takes.
constexpr float kStop = -0.0f;
__device__ __forceinline__ bool stops(float A) { return __float_as_uint(A) == 0x80000000u; }
// The state behind a run, from the one before it.
__device__ __forceinline__ float through(float A, float H, float h) { return stops(A) ? H : fmaf(A, h, H); }
// The factor of two runs, the first one first.
__device__ __forceinline__ float both(float A1, float A2) { return stops(A1) || stops(A2) ? kStop : A1 * A2; }

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

// The totals of the cluster's tiles, by tile, for this CTA's channels: A and H of each of a
// lane's channels. Two of them: a CTA may be a round ahead of another.
template <int kVec>
struct Totals {
    float v[2][kMaxCluster][32][2 * kVec];
};

// This CTA's total to every CTA of the cluster (one warp each), then the first half of the
// cluster's barrier.
template <int kVec>
__device__ __forceinline__ void send_total(Totals<kVec>& t, int parity, uint32_t rank, uint32_t R, int warp, int lane,
                                           const float (&A)[kVec], const float (&H)[kVec]) {
    if (warp < (int)R) {
        const uint32_t to = ptx::mapa(ptx::smem_addr(t.v[parity][rank][lane]), warp);
        if constexpr (kVec == 2)
            asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to), "f"(A[0]), "f"(A[1]), "f"(H[0]),
                         "f"(H[1])
                         : "memory");
        else
            asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(A[0]), "f"(H[0]) : "memory");
    }
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}

// The second half, then: `carry` through the tiles before this one (in), and through all (carry).
template <int kVec>
__device__ __forceinline__ void receive_totals(const Totals<kVec>& t, int parity, uint32_t rank, uint32_t R, int lane,
                                               float (&carry)[kVec], float (&in)[kVec]) {
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
#pragma unroll
    for (int c = 0; c < kVec; ++c) in[c] = carry[c];
    for (uint32_t r = 0; r < R; ++r) {
        const float* v = t.v[parity][r][lane];
#pragma unroll
        for (int c = 0; c < kVec; ++c) {
            carry[c] = through(v[c], v[kVec + c], carry[c]);
            if (r < rank) in[c] = carry[c];
        }
    }
}

template <typename T, int kVec, bool kGate>
__global__ void __launch_bounds__(kThreads, 2) gated_fwd(const Gated p) {
    __shared__ Totals<kVec> totals;
    __shared__ float part[2][kWarps][32][2 * kVec];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = ptx::cluster_ctarank(), R = ptx::cluster_nctarank();
    const int64_t groups = (p.D + 32 * kVec - 1) / (32 * kVec), group = blockIdx.x / R;
    const int b = (int)(group / groups), d = (int)(group % groups) * 32 * kVec + lane * kVec;
    const bool in_d = d < p.D;
    const int64_t tiles = (p.T + kTile - 1) / kTile;
    const T* x = static_cast<const T*>(p.x) + b * p.x_b + d;
    const T* f = static_cast<const T*>(p.f) + b * p.f_b + d;
    const T* g = kGate ? static_cast<const T*>(p.i) + b * p.i_b + d : nullptr;
    T* h = static_cast<T*>(p.h) + b * p.h_b + d;
    const uint8_t* reset = p.reset ? p.reset + (int64_t)b * p.T : nullptr;

    // (a CTA's shared memory may be written to once the CTA runs)
    if (R > 1) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
    float carry[kVec];
#pragma unroll
    for (int c = 0; c < kVec; ++c) carry[c] = p.h0 && in_d ? p.h0[(int64_t)b * p.D + d + c] : 0.0f;

    Raw<T, kVec> rx[kTok], rf[kTok], rg[kTok];
    uint32_t stop = 0;
    auto load = [&](int64_t tile) {
        const int64_t t0 = tile * kTile + warp * kTok;
        stop = 0;
#pragma unroll
        for (int k = 0; k < kTok; ++k) {
            const int64_t t = t0 + k;
            rx[k].zero();
            rf[k].zero();
            if (kGate) rg[k].zero();
            if (t < p.T) {
                if (in_d) {
                    rx[k].load(x + t * p.x_t);
                    rf[k].load(f + t * p.f_t);
                    if (kGate) rg[k].load(g + t * p.i_t);
                }
                if (reset && __ldg(reset + t)) stop |= 1u << k;
            }
        }
    };
    load(rank);
    int parity = 0;
    for (int64_t tile0 = 0; tile0 < tiles; tile0 += R, parity ^= 1) {
        const int64_t tile = tile0 + rank, t0 = tile * kTile + warp * kTok;
        const int n = (int)max((int64_t)0, min((int64_t)kTok, p.T - t0));  // tokens of this warp
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
                float a, r, u;
                sigmoid_pair(rf[k].get(c), a, r);
                u = r;
                if (kGate) sigmoid_pair(rg[k].get(c), u, r);
                // tokens past the end leave the state as it is
                C[k][c] = k >= n ? 1.0f : (stop >> k & 1) ? kStop : a;
                v[k][c] = k >= n ? 0.0f : u * rx[k].get(c);
                H[c] = through(C[k][c], v[k][c], H[c]);
                A[c] = both(A[c], C[k][c]);
            }
        if (tile0 + R < tiles) load(tile + R);
        float* mine = part[parity][warp][lane];
#pragma unroll
        for (int c = 0; c < kVec; ++c) {
            mine[c] = A[c];
            mine[kVec + c] = H[c];
        }
        __syncthreads();
        // the tile's warps before this one, and all of them
        float preA[kVec], preH[kVec];
#pragma unroll
        for (int c = 0; c < kVec; ++c) {
            A[c] = preA[c] = 1.0f;
            H[c] = preH[c] = 0.0f;
        }
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float* o = part[parity][w][lane];
#pragma unroll
            for (int c = 0; c < kVec; ++c) {
                if (w == warp) {
                    preA[c] = A[c];
                    preH[c] = H[c];
                }
                H[c] = through(o[c], o[kVec + c], H[c]);
                A[c] = both(A[c], o[c]);
            }
        }
        float in[kVec];
        if (R > 1) {
            if (tile0 == 0) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
            send_total<kVec>(totals, parity, rank, R, warp, lane, A, H);
            receive_totals<kVec>(totals, parity, rank, R, lane, carry, in);
        } else {
#pragma unroll
            for (int c = 0; c < kVec; ++c) {
                in[c] = carry[c];
                carry[c] = through(A[c], H[c], carry[c]);
            }
        }
        if (p.states && warp == 0 && in_d && tile < tiles) {
            float* s = p.states + ((int64_t)b * tiles + tile) * p.D + d;
#pragma unroll
            for (int c = 0; c < kVec; ++c) s[c] = in[c];
        }
#pragma unroll
        for (int c = 0; c < kVec; ++c) in[c] = through(preA[c], preH[c], in[c]);
#pragma unroll
        for (int k = 0; k < kTok; ++k) {
#pragma unroll
            for (int c = 0; c < kVec; ++c) in[c] = through(C[k][c], v[k][c], in[c]);
            if (k < n && in_d) store<kVec>(h + (t0 + k) * p.h_t, in);
        }
    }
    if (rank == 0 && warp == 0 && in_d) {
#pragma unroll
        for (int c = 0; c < kVec; ++c) p.h_last[(int64_t)b * p.D + d + c] = carry[c];
    }
}

// Backward, from the last tile to the first: with k_t = c_{t+1} g_{t+1} the gradient that enters
// token t from its right, g_t = dh_t + k_t and k_{t-1} = c_t g_t, so a run of tokens maps
// k -> A k + G with the same A as forward. Each tile's states are recomputed from the one
// that the forward pass kept for it.
template <typename T, int kVec, bool kGate>
__global__ void __launch_bounds__(kThreads, 2) gated_bwd(const Gated p) {
    __shared__ Totals<kVec> totals;
    __shared__ float part[2][kWarps][32][3 * kVec];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = ptx::cluster_ctarank(), R = ptx::cluster_nctarank();
    const int64_t groups = (p.D + 32 * kVec - 1) / (32 * kVec), group = blockIdx.x / R;
    const int b = (int)(group / groups), d = (int)(group % groups) * 32 * kVec + lane * kVec;
    const bool in_d = d < p.D;
    const int64_t tiles = (p.T + kTile - 1) / kTile;
    const T* x = static_cast<const T*>(p.x) + b * p.x_b + d;
    const T* f = static_cast<const T*>(p.f) + b * p.f_b + d;
    const T* g = kGate ? static_cast<const T*>(p.i) + b * p.i_b + d : nullptr;
    const T* dh = static_cast<const T*>(p.dh) + b * p.dh_b + d;
    T* dx = static_cast<T*>(p.dx) + b * p.dx_b + d;
    T* df = static_cast<T*>(p.df) + b * p.df_b + d;
    T* di = kGate ? static_cast<T*>(p.di) + b * p.di_b + d : nullptr;
    const uint8_t* reset = p.reset ? p.reset + (int64_t)b * p.T : nullptr;

    // (a CTA's shared memory may be written to once the CTA runs)
    if (R > 1) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
    float carry[kVec];
#pragma unroll
    for (int c = 0; c < kVec; ++c) carry[c] = p.dh_last && in_d ? p.dh_last[(int64_t)b * p.D + d + c] : 0.0f;

    int parity = 0;
    for (int64_t back0 = 0; back0 < tiles; back0 += R, parity ^= 1) {
        const int64_t tile = tiles - 1 - (back0 + rank), t0 = tile * kTile + warp * kTok;
        const int n = tile < 0 ? 0 : (int)max((int64_t)0, min((int64_t)kTok, p.T - t0));
        Raw<T, kVec> rx[kTok], rf[kTok], rg[kTok], rh[kTok];
        uint32_t stop = 0;
        float s[kVec];
#pragma unroll
        for (int c = 0; c < kVec; ++c)
            s[c] = tile >= 0 && in_d ? __ldg(p.in_states + ((int64_t)b * tiles + tile) * p.D + d + c) : 0.0f;
#pragma unroll
        for (int k = 0; k < kTok; ++k) {
            const int64_t t = t0 + k;
            rx[k].zero();
            rf[k].zero();
            rh[k].zero();
            if (kGate) rg[k].zero();
            if (k < n) {
                if (in_d) {
                    rf[k].load(f + t * p.f_t);
                    if (kGate) rg[k].load(g + t * p.i_t);
                    rx[k].load(x + t * p.x_t);
                    rh[k].load(dh + t * p.dh_t);
                }
                if (reset && __ldg(reset + t)) stop |= 1u << k;
            }
        }
        // C, the factors' derivatives, and the run's A, H (states) and G (gradients)
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
                float a, na, nu;
                sigmoid_pair(rf[k].get(c), a, na);
                ca[k][c] = a * na;
                u[k][c] = na;
                if (kGate) {
                    sigmoid_pair(rg[k].get(c), u[k][c], nu);
                    cu[k][c] = u[k][c] * nu;
                }
                C[k][c] = k >= n ? 1.0f : (stop >> k & 1) ? kStop : a;
                H[c] = through(C[k][c], k >= n ? 0.0f : u[k][c] * rx[k].get(c), H[c]);
                A[c] = both(A[c], C[k][c]);
            }
#pragma unroll
        for (int k = kTok - 1; k >= 0; --k)
#pragma unroll
            for (int c = 0; c < kVec; ++c) G[c] = through(C[k][c], 0.0f, rh[k].get(c) + G[c]);
        float* mine = part[parity][warp][lane];
#pragma unroll
        for (int c = 0; c < kVec; ++c) {
            mine[c] = A[c];
            mine[kVec + c] = H[c];
            mine[2 * kVec + c] = G[c];
        }
        __syncthreads();
        // the state behind the tile's warps before this one; the gradient's run through those after
        // it (suf), and through all
        float sufA[kVec], sufG[kVec];
#pragma unroll
        for (int c = 0; c < kVec; ++c) {
            A[c] = sufA[c] = 1.0f;
            G[c] = sufG[c] = 0.0f;
        }
#pragma unroll
        for (int w = kWarps - 1; w >= 0; --w) {
            const float* o = part[parity][w][lane];
#pragma unroll
            for (int c = 0; c < kVec; ++c) {
                if (w == warp) {
                    sufA[c] = A[c];
                    sufG[c] = G[c];
                }
                G[c] = through(o[c], o[2 * kVec + c], G[c]);
                A[c] = both(A[c], o[c]);
            }
        }
        if (R > 1) {
            if (back0 == 0) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
            send_total<kVec>(totals, parity, rank, R, warp, lane, A, G);
        }
#pragma unroll
        for (int w = 0; w < kWarps - 1; ++w)
            if (w < warp) {
                const float* o = part[parity][w][lane];
#pragma unroll
                for (int c = 0; c < kVec; ++c) s[c] = through(o[c], o[kVec + c], s[c]);
            }
        float before[kTok][kVec];  // the state that enters each token (0 at a reset)
#pragma unroll
        for (int k = 0; k < kTok; ++k)
#pragma unroll
            for (int c = 0; c < kVec; ++c) {
                before[k][c] = stops(C[k][c]) ? 0.0f : s[c];
                s[c] = through(C[k][c], u[k][c] * rx[k].get(c), s[c]);
            }
        float in[kVec];
        if (R > 1) {
            receive_totals<kVec>(totals, parity, rank, R, lane, carry, in);
        } else {
#pragma unroll
            for (int c = 0; c < kVec; ++c) {
                in[c] = carry[c];
                carry[c] = through(A[c], G[c], carry[c]);
            }
        }
#pragma unroll
        for (int c = 0; c < kVec; ++c) in[c] = through(sufA[c], sufG[c], in[c]);
#pragma unroll
        for (int k = kTok - 1; k >= 0; --k) {
            float ox[kVec], of[kVec], oi[kVec];
#pragma unroll
            for (int c = 0; c < kVec; ++c) {
                const float gr = rh[k].get(c) + in[c], xv = rx[k].get(c);
                ox[c] = u[k][c] * gr;
                of[c] = ca[k][c] * gr * (kGate ? before[k][c] : before[k][c] - xv);
                if (kGate) oi[c] = xv * cu[k][c] * gr;
                if (k < n) in[c] = stops(C[k][c]) ? 0.0f : C[k][c] * gr;
            }
            if (k < n && in_d) {
                store<kVec>(dx + (t0 + k) * p.dx_t, ox);
                store<kVec>(df + (t0 + k) * p.df_t, of);
                if (kGate) store<kVec>(di + (t0 + k) * p.di_t, oi);
            }
        }
    }
    if (p.dh0 && rank == 0 && warp == 0 && in_d) {
#pragma unroll
        for (int c = 0; c < kVec; ++c) p.dh0[(int64_t)b * p.D + d + c] = carry[c];
    }
}

// One token: a thread a channel pair (or channel). Bound by the launch.
template <typename T, int kVec, bool kGate>
__global__ void __launch_bounds__(128) gated_step(const Gated p) {
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

// Tiles a cluster takes at a time: enough CTAs to fill the GPU's SMs several times over with
// as few exchanges as that allows.
int cluster_size(const Gated& p, int64_t groups) {
    const int64_t tiles = (p.T + kTile - 1) / kTile;
    int R = 1;
    while (R < kMaxCluster && R < tiles && groups * R < 152 * 3) R *= 2;
    return R;
}

template <typename K>
int launch_cluster(K kernel, const Gated& p, int vec, cudaStream_t stream) {
    const int64_t groups = (int64_t)p.B * ((p.D + 32 * vec - 1) / (32 * vec));
    const int R = cluster_size(p, groups);
    if (groups * R > INT32_MAX) return SSDC_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(groups * R));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = R;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? 1 : SSDC_ERR_CUDA;
}

template <typename T, int kVec, bool kGate>
int launch(const Gated& p, int what, cudaStream_t stream) {
    if (what == 0) return launch_cluster(gated_fwd<T, kVec, kGate>, p, kVec, stream);
    if (what == 1) return launch_cluster(gated_bwd<T, kVec, kGate>, p, kVec, stream);
    const int64_t n = (int64_t)p.B * ((p.D + kVec - 1) / kVec);
    gated_step<T, kVec, kGate><<<(unsigned)((n + 127) / 128), 128, 0, stream>>>(p);
    return 1;
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

int gated_fwd_launch(const Gated& p, cudaStream_t stream) { return launch_scan(p, 0, stream); }
int gated_bwd_launch(const Gated& p, cudaStream_t stream) { return launch_scan(p, 1, stream); }
int gated_step_launch(const Gated& p, cudaStream_t stream) { return launch_scan(p, 2, stream); }

}  // namespace block
}  // namespace ssdc
