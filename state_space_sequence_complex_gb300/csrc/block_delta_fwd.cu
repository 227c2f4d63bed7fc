// The delta rule over sequences of bfloat16, forward, in chunks on the tensor cores (the formulas are in
// block_delta.cuh).
//
// A CTA walks one state, or some columns of it, chunk by chunk. Four warps prepare the next chunk (products of
// keys and queries, decays, the inverses of the 16 x 16 blocks), and up to eight warps with 16 columns of the state
// each carry the chain of the current one:
//   S k^T, S q^T  ->  X  ->  U in four blocks  ->  O, S
// S stays in registers in fp32, transposed (columns of the state are rows of the tiles). Products that end up in S
// have operands in two bf16 parts (16 bits or more); those that only end up in O, which is rounded to 8 bits
// itself, have one.
//
// A chunk of 64 tokens, 64 rows and 64 columns takes 240 matrix instructions of each of four column warps, 1,920
// clocks of an SM's 1,024 multiply-adds, and 0.5 KB of memory a token.
#include "block_delta_prepare.cuh"

namespace ssdc {
namespace block {
namespace delta {
namespace {

template <int KP, int NW, int kGroups, bool kUnitRows>
__device__ __forceinline__ void walk(const Delta& p, char* smem, int b, int h, int w, int col0, int column_threads) {
    using L = Layout<KP, NW, false, kGroups>;
    constexpr int KT = KP / 8;  // 8-row tiles of the state
    const uint32_t base = ptx::smem_addr(smem);
    const int lane = threadIdx.x % 32, all = kPrep + column_threads;
    const int columns = min(16, p.V - col0);
    const int chunks = (int)((p.T + C - 1) / C);
    const int64_t seq = (int64_t)b * p.H + h;
    const uint32_t strips = base + L::kStripOff + w * 2 * L::kStrip;
    const Lanes<L::kKeyPitch> key_lanes(base);
    const Lanes<L::kPitch> lanes(base);
    const int fetch_u = lane % 2, fetch_r = lane / 2;
    const bool has_unit = 8 * fetch_u < columns;
    const __nv_bfloat16* v_row = bf16(p.v.p) + b * p.v.b + h * p.v.h + fetch_r * p.v.t + col0 + (has_unit ? 8 * fetch_u : 0);
    auto fetch_v = [&](int c) {  // chunks in order
        const int left = (int)min((int64_t)C, p.T - (int64_t)c * C) - fetch_r;
        const __nv_bfloat16* v = v_row;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            fetch<kUnitRows>(strip_at(strips + (c & 1) * L::kStrip, fetch_r + 16 * i, fetch_u), v, has_unit && 16 * i < left);
            v += 16 * p.v.t;
        }
        ptx::cp_async_commit();
        v_row += C * p.v.t;
    };
    fetch_v(0);
    // state[row 8 i + 2 (lane % 4) + e % 2][column lane / 4 + 8 (e / 2)]
    float S[KT][4];
    const int64_t state = seq * p.K * p.V + col0;
#pragma unroll
    for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = 8 * i + 2 * (lane % 4) + e % 2, cl = lane / 4 + 8 * (e / 2);
            S[i][e] = p.h0 != nullptr && r < p.K && cl < columns ? p.h0[state + (int64_t)r * p.V + cl] : 0.0f;
        }
    const int64_t o_stride = (int64_t)p.H * p.V, o_step = C * o_stride, o_first = (b * p.T * p.H + h) * p.V + col0;
    __nv_bfloat16* o_rows = static_cast<__nv_bfloat16*>(p.o) + o_first;
    __nv_bfloat16* u_rows = static_cast<__nv_bfloat16*>(p.updates) + o_first;
    int stage = 0;
    for (int c = 0; c < chunks; ++c, stage = L::next_stage(stage, 1)) {
        const int turn = c & 1, set = c & (L::kSets - 1), half = c % kGroups;
        // The strip of this chunk has its v, and when that has been read its u and o. The other one has the last
        // chunk's o, which goes to memory beside the first products; then the state, where it is kept; then the next v.
        const uint32_t mine = strips + turn * L::kStrip, other = strips + (turn ^ 1) * L::kStrip;
        bar_sync(kBarKeys + (c & 3), all);
        const uint32_t keys = stage * L::kStage, queries = keys + L::kKeyTile;
        StripRows rows;
        rows.take(other);
        float X[8][4], O[8][4];
        Split a;
        uint32_t kb[2][4], qb[2][4];  // the next products' operands are read before this one's are used
        ldsm(kb[0], keys + key_lanes.down[0]);
        ldsm(qb[0], queries + key_lanes.down[0]);
#pragma unroll
        for (int it = 0; it < KP / 4; ++it) {
            const int s = it / 4, n = it % 4, now = it % 2;
            if (n == 0) {
                a.set(S[2 * s], S[2 * s + 1]);
                if (p.states != nullptr) stsm_t(strip_rows(other, 16 * s % C), a.hi[0], a.hi[1], a.hi[2], a.hi[3]);
            }
            if (it + 1 < KP / 4) {
                const int s1 = (it + 1) / 4, n1 = (it + 1) % 4;
                ldsm(kb[1 - now], keys + 16 * n1 * L::kKeyPitch + key_lanes.down[s1]);
                ldsm(qb[1 - now], queries + 16 * n1 * L::kKeyPitch + key_lanes.down[s1]);
            }
            const uint32_t *k = kb[now], *q = qb[now];
            mma_at(s, X[2 * n], a.hi, k[0], k[1]);
            mma_at(s, X[2 * n + 1], a.hi, k[2], k[3]);
            mma_at(s, O[2 * n], a.hi, q[0], q[1]);
            mma_at(s, O[2 * n + 1], a.hi, q[2], q[3]);
            mma(X[2 * n], a.lo, k[0], k[1]);
            mma(X[2 * n + 1], a.lo, k[2], k[3]);
            if (it == 3 && c > 0) rows.give(o_rows - o_step, o_stride, C, columns);
            if (p.states != nullptr && it % 16 == 15) {
                const int first = it / 16 * C;
                rows.take(other);
                rows.give(static_cast<__nv_bfloat16*>(p.states) + (seq * chunks + c) * p.K * p.V + (int64_t)first * p.V + col0, p.V,
                          p.K - first, columns);
            }
        }
        if (c + 1 < chunks) fetch_v(c + 1);
        else ptx::cp_async_commit();
        ptx::cp_async_wait<1>();
        __syncwarp();
        bar_sync(kBarFull + half, all);
        const Factors* factors = reinterpret_cast<const Factors*>(smem + L::kFactorsOff) + set * C;
        const uint32_t hi = L::kLOff + half * L::kBlocks, lo = hi + L::kSquare, ps = lo + L::kSquare;
        const float gam = reinterpret_cast<const float*>(smem + L::kGamOff)[set];
        // A chunk that cuts the state off (a reset in it, as a rule): what a token does not take from it is zero,
        // whatever the state holds; an infinity or a NaN of one document stays out of the next.
        if (gam == 0.0f) {
#pragma unroll
            for (int n = 0; n < 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (factors[8 * n + 2 * (lane % 4) + e % 2].k == 0.0f) X[n][e] = O[n][e] = 0.0f;
        }
#pragma unroll
        for (int n = 0; n < 8; n += 2) {
            uint32_t r[4];
            ldsm_t(r, strip_rows(mine, 8 * n));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int j = 8 * (n + e) + 2 * (lane % 4);
                const float2 f0 = *reinterpret_cast<const float2*>(&factors[j]), f1 = *reinterpret_cast<const float2*>(&factors[j + 1]);
                float *x = X[n + e], *o = O[n + e];
                x[0] = fmaf(-f0.x, x[0], ptx::bf16_lo(r[2 * e]));
                x[1] = fmaf(-f1.x, x[1], ptx::bf16_hi(r[2 * e]));
                x[2] = fmaf(-f0.x, x[2], ptx::bf16_lo(r[2 * e + 1]));
                x[3] = fmaf(-f1.x, x[3], ptx::bf16_hi(r[2 * e + 1]));
                o[0] *= f0.y; o[1] *= f1.y; o[2] *= f0.y; o[3] *= f1.y;
            }
        }
#pragma unroll
        for (int i = 0; i < KT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) S[i][e] *= gam;
        if (gam == 0.0f) {
#pragma unroll
            for (int i = 0; i < KT; ++i) S[i][0] = S[i][1] = S[i][2] = S[i][3] = 0.0f;
        }
        const int64_t left = p.T - (int64_t)c * C;
        const int n_tokens = left < C ? (int)left : C;
        // Block by block: what a block adds to O and S keeps the instructions coming while the next one, which
        // waits for each of its products, is solved.
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            Split a;
            uint32_t bh[4], bl[4];
            float *x0 = X[2 * r], *x1 = X[2 * r + 1];
            a.set(x0, x1);
            ldsm_t(bh, hi + 16 * r * L::kPitch + lanes.across[r]);
            ldsm_t(bl, lo + 16 * r * L::kPitch + lanes.across[r]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float* x = X[2 * r + e];
                mma0(x, a.lo, bh[2 * e], bh[2 * e + 1]);
                mma(x, a.hi, bl[2 * e], bl[2 * e + 1]);
                mma(x, a.hi, bh[2 * e], bh[2 * e + 1]);
            }
            a.set(x0, x1);  // U of this block
#pragma unroll
            for (int n = r + 1; n < 4; ++n) {
                ldsm(bh, hi + 16 * n * L::kPitch + lanes.down[r]);
                ldsm(bl, lo + 16 * n * L::kPitch + lanes.down[r]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    mma(X[2 * n + e], a.hi, bh[2 * e], bh[2 * e + 1]);
                    mma(X[2 * n + e], a.lo, bh[2 * e], bh[2 * e + 1]);
                    mma(X[2 * n + e], a.hi, bl[2 * e], bl[2 * e + 1]);
                }
            }
            if (p.updates != nullptr)
                stsm_t(strip_rows(mine, 16 * r), a.hi[0], a.hi[1], a.hi[2], a.hi[3]);
#pragma unroll
            for (int n = r; n < 4; ++n) {
                ldsm(bh, ps + 16 * n * L::kPitch + lanes.down[r]);
                mma(O[2 * n], a.hi, bh[0], bh[1]);
                mma(O[2 * n + 1], a.hi, bh[2], bh[3]);
                mma(O[2 * n], a.lo, bh[0], bh[1]);
                mma(O[2 * n + 1], a.lo, bh[2], bh[3]);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int j = 16 * r + 8 * e + 2 * (lane % 4);
                const float f0 = factors[j].s, f1 = factors[j + 1].s;
                float* x = X[2 * r + e];
                x[0] *= f0; x[1] *= f1; x[2] *= f0; x[3] *= f1;
                if (gam == 0.0f) {  // what a reset keeps from the next chunk is left out, too
                    if (f0 == 0.0f) x[0] = x[2] = 0.0f;
                    if (f1 == 0.0f) x[1] = x[3] = 0.0f;
                }
            }
            a.set(x0, x1);
#pragma unroll
            for (int i = 0; i < KT; i += 2) {
                uint32_t kb[4];
                ldsm_t(kb, keys + 16 * r * L::kKeyPitch + key_lanes.across[i / 2]);
                mma(S[i], a.hi, kb[0], kb[1]);
                mma(S[i + 1], a.hi, kb[2], kb[3]);
                mma(S[i], a.lo, kb[0], kb[1]);
                mma(S[i + 1], a.lo, kb[2], kb[3]);
            }
        }
        if (c + kGroups < chunks) bar_arrive(kBarFree + half, all);
        if (c + 2 * kGroups < chunks) bar_arrive(kBarStage + (c & 3), all);
        if (p.updates != nullptr) {
            rows.take(mine);
            rows.give(u_rows, o_stride, n_tokens, columns);
            u_rows += o_step;
        }
#pragma unroll
        for (int n = 0; n < 8; n += 2)
            stsm_t(strip_rows(mine, 8 * n), pack(O[n][0], O[n][1]), pack(O[n][2], O[n][3]), pack(O[n + 1][0], O[n + 1][1]),
                   pack(O[n + 1][2], O[n + 1][3]));
        o_rows += o_step;
    }
    StripRows rows;
    rows.take(strips + ((chunks - 1) & 1) * L::kStrip);
    rows.give(o_rows - o_step, o_stride, (int)(p.T - (int64_t)(chunks - 1) * C), columns);
#pragma unroll
    for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = 8 * i + 2 * (lane % 4) + e % 2, cl = lane / 4 + 8 * (e / 2);
            if (r < p.K && cl < columns) p.h_last[state + (int64_t)r * p.V + cl] = S[i][e];
        }
}

template <int KP, int NW, int kGroups, bool kUnitRows>
__global__ void __launch_bounds__(kGroups * kPrep + 32 * NW, KP == 64 && NW == 4 && kGroups == 1 ? 2 : 1) delta_fwd(const __grid_constant__ Delta p) {
    extern __shared__ __align__(128) char smem[];
    const int parts = (p.V + 16 * NW - 1) / (16 * NW), item = blockIdx.x / parts, col0 = blockIdx.x % parts * 16 * NW;
    const int b = item / p.H, h = item % p.H;
    const int warps = min(NW, (p.V - col0 + 15) / 16);  // that have columns
    if (threadIdx.x < kGroups * kPrep) {
        Registers<KP, NW, false, kGroups>::prepare();
        prepare_chunks<KP, NW, false, kGroups, kUnitRows>(p, smem, b, h, 32 * warps);
    } else {
        Registers<KP, NW, false, kGroups>::walk();
        const int w = threadIdx.x / 32 - kGroups * kPrep / 32;
        if (w < warps) walk<KP, NW, kGroups, kUnitRows>(p, smem, b, h, w, col0 + 16 * w, 32 * warps);
    }
}

template <int KP, int NW, int kGroups>
int launch(const Delta& p, cudaStream_t stream) {
    using L = Layout<KP, NW, false, kGroups>;
    const bool units = whole_units(p.k) && whole_units(p.q) && whole_units(p.v);
    const auto kernel = units ? delta_fwd<KP, NW, kGroups, true> : delta_fwd<KP, NW, kGroups, false>;
    static std::atomic<uint64_t> done[2];
    if (allow_smem(kernel, L::kBytes, done[units]) != cudaSuccess) return SSDC_ERR_CUDA;
    const int parts = (p.V + 16 * NW - 1) / (16 * NW);
    kernel<<<p.B * p.H * parts, kGroups * kPrep + 32 * NW, L::kBytes, stream>>>(p);
    return 1;
}

}  // namespace
}  // namespace delta

int delta_fwd_launch(const Delta& p, cudaStream_t stream) {
    using namespace delta;
    if (few_states(p)) return p.K <= 64 ? launch<64, 4, 2>(p, stream) : launch<128, 4, 2>(p, stream);
    if (p.K <= 64) return p.V <= 64 ? launch<64, 4, 1>(p, stream) : launch<64, 8, 1>(p, stream);
    return p.V <= 64 ? launch<128, 4, 1>(p, stream) : launch<128, 8, 1>(p, stream);
}

}  // namespace block
}  // namespace ssdc
