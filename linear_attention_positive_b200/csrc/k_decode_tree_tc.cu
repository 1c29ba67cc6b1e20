// favor_decode_tree on tensor cores: bf16 trees of enough nodes to fill tiles, one CTA per head.
//
// With P = w_r.x the projections and X_r a scale per feature (below), in log2 units:
//   b_ir = 2^(P_ir + X_r - f_i),   f_i = max_r (P_ir + X_r), rounded up      query rows
//   a_jr = 2^(P_jr - X_r - g_j),   g_j = max_r (P_jr - X_r), rounded up      key rows
//   A_ij = sum_r b_ir a_jr,   Y_ic = sum_r b_ir s_r S'_r[c],   y_i = sum_r b_ir s_r z'_r,   s_r = 2^(D_r - X_r)
//   G_j = g_j - |k_j|^2/2,    w_ij = 2^G_j A_ij for j in J(i), else 0
//   out_i = [Y_i + sum_j w_ij v_j] / [y_i + sum_j w_ij].
// X_r = D_r + log2 z'_r, the feature's own sum over the state, makes s_r S'_r a weighted mean of the
// values (of one size for all features) and y_i at least about 1. Where a feature is empty or some key
// lies far above the state (kTreeTcRaise), X_r is raised to the largest logit of the tree's keys. X, f
// and g are whole numbers, so that the exponents of a row's large terms are small and rounded once.
//
// Precision: a, b and s S' enter the MMAs as hi + lo, two fp16 values (22 bits), products hi hi,
// hi lo, lo hi; a and b are scaled by 2^15, so that a term 2^-18 below its maximum keeps all 22 bits
// and fp16's smallest step is an error of at most 2^-40 of the maximum. Each column of s S' is scaled by
// its first 64 features' largest magnitude to about 2^6 (1000 times that still fits). Weights of values are
// three bf16 parts against the bf16 values. The steps' error in a row is at most
//   2^-40 sum_{j in J(i)} 2^G_j (sum_r a_jr + sum_r b_ir) + 2^-31 sum_r b_ir
// (the second part: s S', at most 2^-25 2^-6 of its column's largest magnitude); a row where that bound exceeds
// 2^-20 of the denominator (its own terms lie far below the scales of other rows'), and every row of a
// head with a non-finite value or s S' beyond fp16's range, is
// computed by tree_row_exact_bf16. (The bound is nearly attained: where 2^-14 was allowed, rows behind two
// tokens of context came out with errors of 3e-4. At N(0, 1) inputs no row is beyond it behind a long
// context, at most 0.02 % are behind 16 tokens and 0.05 to 0.6 % behind one.)
//
// T <= 64: keys and queries are the two halves of one 128-row tile, and at d = 64 two CTAs share an
// SM (TMEM 256 columns, 112 KB), so that one head's copies and MMAs run under another's exponentials.
// T <= 128: a tile each, one CTA an SM.
//
// Features are taken 128 at a time (the logits of both halves are formed once for the maxima, then
// the second half's again: TMEM holds one half next to the accumulators); a and S' are rows of one
// operand, so that A and Y are one MMA of N = T + d columns (two of half the size took 1.6 times as
// long). At d = 128, T > 64, a and S' take 64 features at a time, for shared memory.
//
// Bound: the state's bytes, (m d + 2 m) 4 a head, and next to it the exponentials and splits of
// 2 T m features on CUDA cores, and 3 (T + d) m 128 products on the tensor cores: about equal at
// T = d = 64. What is measured is the latency of the chain copy, logits, maxima, exponentials, MMA,
// exponentials, MMA, weights, MMA, rows out.

#include "common.cuh"

namespace favor {

// Keys at most this far (log2) above the state's features leave X_r as it is.
constexpr float kTreeTcRaise = 10.f;
// A column of s S' is scaled so that its first 64 features' largest magnitude is about 2^this.
constexpr float kTreeTcState = 6.f;

template <int D_, bool STACK_>
struct TreeTc {
    static constexpr int D = D_, NB = D / 64;
    // Column groups of a TMEM lane, a warpgroup each. Two CTAs an SM leave 64 registers to 512 threads, and
    // their spills go to L2 (shared memory takes all of L1): 96 us for 1024 heads, 77 with 256 threads.
    static constexpr int NCG = (STACK_ && D == 64) ? 2 : 4, THREADS = 128 * NCG;
    static constexpr int MR = STACK_ ? 64 : 128;             // key rows
    static constexpr uint32_t BLK = 128 * 128;               // 64 columns of a 128-row tile
    static constexpr uint32_t KQ = (STACK_ ? 1 : 2) * NB * BLK;
    static constexpr uint32_t WB = 2 * NB * BLK;             // both halves of W
    static constexpr uint32_t XB = (MR + D) * 128;           // a and S', 64 features, one part
    static constexpr int NSB = (!STACK_ && D == 128) ? 1 : 2;  // such blocks a step
    static constexpr bool OVER = STACK_ && D == 64;          // the second low block takes W's first half
    static constexpr uint32_t OFF_W = KQ, OFF_XH = OFF_W + WB, OFF_XL = OFF_XH + NSB * XB,
                              OFF_F = OFF_XL + (OVER ? 1 : NSB) * XB;
    static constexpr uint32_t OFF_BAR = OFF_F + 4 * (3 * 256 + 8 * 128 + 8 * 128 + 128 + D + 16 + 6 * 128), BYTES = OFF_BAR + 128 + 1024;
    // TMEM columns: logits of a half (keys and queries), accumulators of A and Y, of the values' sum
    static constexpr uint32_t T_K = 0, T_Q = STACK_ ? 0 : 128, T_H = STACK_ ? 128 : 256, T_A = T_H, T_Y = T_A + MR,
                              T_O = (STACK_ && D == 128) ? 320 : T_A;
    static constexpr uint32_t OFF_Y = OFF_W + (OVER ? NB * BLK : 0);  // the first half's Y, fp32 [MR][D], in W's place
    static constexpr uint32_t COLS = (STACK_ && D == 64) ? 256 : 512;
    static_assert(MR * D * 4 <= WB && (!OVER || (XB <= NB * BLK && MR * D * 4 <= NB * BLK)),
                  "output rows, the low block and the first half's Y fit in W's place");
};

// fp32 order as signed integers (for the integer warp maximum) and back.
__device__ __forceinline__ int order_bits(float x) {
    const int i = __float_as_int(x);
    return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float from_order_bits(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }

// The 11 leading bits of x, rounded to nearest.
__device__ __forceinline__ float hi_round(float x) { return __uint_as_float((__float_as_uint(x) + 0x1000u) & 0xFFFFE000u); }

template <int D, bool STACK>
__global__ void __launch_bounds__(TreeTc<D, STACK>::THREADS, (STACK && D == 64) ? 2 : 1)
k_decode_tree_tc(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                 const __grid_constant__ CUtensorMap mapV, const __grid_constant__ CUtensorMap mapW,
                 const __grid_constant__ CUtensorMap mapS, TreeParams p) {
    using C = TreeTc<D, STACK>;
    constexpr int NB = C::NB, MR = C::MR, NSB = C::NSB, NCG = C::NCG;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t *sKQ = smem, *sW = smem + C::OFF_W, *sXH = smem + C::OFF_XH, *sXL = smem + C::OFF_XL;
    uint8_t *sXL1 = C::OVER ? sW : sXL + C::XB;
    uint8_t *sV = sKQ;                                    // the values take the keys' place
    float *sX = (float *)(smem + C::OFF_F), *sZ = sX + 256, *sFac = sZ + 256;  // X_r, s_r z'_r, s_r
    float *sMx = sFac + 256;                              // [keys, queries][column group][128] maxima
    float *sDen = sMx, *sErr = sMx + 4 * 128;             // then [column group][128] parts of denominators and their errors
    float *sSum = sMx + 8 * 128;                          // [keys, queries][4][128] sums of a and b
    float *sGe = sSum + 8 * 128;                          // 2^(G_j - 30)
    float *sUp = sGe + 128;                               // [D] what the columns of s S' are multiplied by
    int *sFlag = (int *)(sUp + D);
    int *sPar = sFlag + 16, *sPtr = sPar + 128;
    uint32_t *sAnc = (uint32_t *)(sPtr + 128);            // [128][MR / 32] rows of J
    uint64_t *bars = (uint64_t *)(smem + C::OFF_BAR);
    uint64_t *kq_full = bars, *w_full = bars + 1, *v_full = bars + 2, *mma_done = bars + 3, *s_full = bars + 4;
    uint32_t *tmem_slot = (uint32_t *)(bars + 6);
    volatile int *abort_flag = (volatile int *)(tmem_slot + 1);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int bh = blockIdx.x, b = bh / p.H, m = p.m, T = p.T;
    const int n = tree_count(p.n_nodes, b, T);
    if (n == 0) return;
    const int nh = m > 128 ? 2 : 1, nch = (m + 63) / 64;

    // chunk c of S' (64 features): its two raw blocks of 32 lie where its high and low block will
    auto load_chunk = [&](int c) {  // one thread
        const int s = c % NSB;
        mbar_arrive_expect_tx(&s_full[s], D * 256);
        tma_load_3d(sXH + s * C::XB + MR * 128, &mapS, &s_full[s], 64 * c, 0, bh);
        tma_load_3d((s == 0 ? sXL : sXL1) + MR * 128, &mapS, &s_full[s], 64 * c + 32, 0, bh);
    };
    int ns = min(C::OVER ? 1 : NSB, nch);  // chunks asked for
    auto load_state = [&]() {
        if (warp == 0 && elect_one()) load_chunk(ns);
        __syncwarp();
        ++ns;
    };
    if (tid == 0) {  // barriers and the first copies, while another warp asks for TMEM
        for (int i = 0; i < 6; ++i) mbar_init(&bars[i], 1);
        *abort_flag = 0;
        sFlag[0] = 0;
        fence_barrier_init();
        mbar_arrive_expect_tx(kq_full, C::KQ);
        for (int nb = 0; nb < NB; ++nb) {
            tma_load_3d(sKQ + nb * C::BLK, &mapK, kq_full, 64 * nb, 0, bh);
            tma_load_3d(sKQ + (STACK ? nb * C::BLK + 64 * 128 : (NB + nb) * C::BLK), &mapQ, kq_full, 64 * nb, 0, bh);
        }
        mbar_arrive_expect_tx(w_full, nh * NB * C::BLK);
        for (int h = 0; h < nh; ++h)
            for (int nb = 0; nb < NB; ++nb) tma_load_2d(sW + (h * NB + nb) * C::BLK, &mapW, w_full, 64 * nb, 128 * h);
        for (int c = 0; c < ns; ++c) load_chunk(c);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, C::COLS);
        tmem_relinquish();
    }
    // the state's scales, asked for here, used under the logits
    float z = 0.f, Dr = 0.f;
    if (tid < m) {
        const float *zp = p.state + (size_t)bh * ((size_t)D * m + 2 * m) + (size_t)D * m;
        z = zp[tid];
        Dr = zp[m + tid];
    }
    int ptr = -1;
    const int node = tid - C::THREADS / 2;  // the threads that form J's rows
    if (node >= 0 && node < n) ptr = tree_parent(p.parents + (size_t)b * T, node);

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    // (descriptors are formed where they are used, by one warp)
    auto logits = [&](int h, uint32_t col) {  // warp 0
        constexpr uint32_t idesc_p = make_idesc(128, 128, kFmtBF16, 0, 0);
        const uint64_t dKQ = make_sdesc(smem_u32(sKQ), 16, 1024), dW = make_sdesc(smem_u32(sW), 16, 1024);
        for (int nb = 0; nb < NB; ++nb) {
            const uint64_t w = dW + (h * NB + nb) * (C::BLK / 16);
            mma_ss_x4_w(tmem + col + C::T_K, dKQ + nb * (C::BLK / 16), w, idesc_p, nb > 0, 2, 2);
            if (!STACK) mma_ss_x4_w(tmem + col + C::T_Q, dKQ + (NB + nb) * (C::BLK / 16), w, idesc_p, nb > 0, 2, 2);
        }
    };
    int nm = 0, nc = 0;  // commits waited for, commits made
    bool ok = true;
    // a bounded wait of the whole CTA, with one result
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        const bool w = ok && mbar_wait(bar, parity, abort_flag);
        ok = __syncthreads_and(w);
        return ok;
    };

    // TMEM lanes are rows: STACK keeps keys in lanes 0-63 and queries in 64-127; cg: column group
    const int row = STACK ? (warp & 1) * 32 + lane : (warp & 3) * 32 + lane, cg = warp >> 2;
    const bool is_key = !STACK || (warp & 3) < 2, is_query = !STACK || (warp & 3) >= 2;
    const uint32_t tL = tmem + (((uint32_t)(warp & 3) * 32u) << 16);
    float *sY = (float *)(smem + C::OFF_Y);
    auto row_chunk = [&](int c) { return row * D + (((c >> 2) ^ (row & 7)) << 2); };  // 16-byte chunks XOR-swizzled by row
    float eN = 0.f;     // -|k|^2/2 of this thread's key, log2 units
    bool v_asked = false;
    auto load_values = [&]() {
        if (warp == 0 && elect_one()) {
            mbar_arrive_expect_tx(v_full, NB * MR * 128);
            for (int nb = 0; nb < NB; ++nb) tma_load_3d(sV + nb * MR * 128, &mapV, v_full, 64 * nb, 0, bh);
        }
        __syncwarp();
        v_asked = true;
    };

    do {
        if (!wait(kq_full, 0) || !wait(w_full, 0)) break;
        if (warp == 0) {
            for (int h = 0; h < nh; ++h) logits(h, h * C::T_H);
            mma_commit_w(mma_done);
        }
        ++nc;
        if (is_key) eN = -0.5f * kLog2e * key_sq_norm<NB, 128>(sKQ, row);
        // rows of J: ancestors by pointer doubling
        if (node >= 0 && node < MR) {
            constexpr int NW = MR / 32;
            uint32_t anc[NW];
#pragma unroll
            for (int w = 0; w < NW; ++w) anc[w] = node < n && (node >> 5) == w ? 1u << (node & 31) : 0u;
            sPar[node] = ptr;
            sPtr[node] = ptr;
#pragma unroll
            for (int w = 0; w < NW; ++w) sAnc[node * NW + w] = anc[w];
            for (int k = 1; k < n; k <<= 1) {
                named_bar_sync(1, MR);
                int next = -1;
                if (ptr >= 0) {
                    next = sPtr[ptr];
#pragma unroll
                    for (int w = 0; w < NW; ++w) anc[w] |= sAnc[ptr * NW + w];
                }
                named_bar_sync(1, MR);
                sPtr[node] = ptr = next;
#pragma unroll
                for (int w = 0; w < NW; ++w) sAnc[node * NW + w] = anc[w];
            }
        }
        const bool some = z > 0.f;
        if (tid < m) {
            const double D2 = (double)Dr * 1.4426950408889634074;
            const float X = rintf((float)D2 + log2f(z)), s = some ? exp2f((float)(D2 - (double)X)) : 0.f;
            sX[tid] = some ? X : -INFINITY;
            sZ[tid] = some ? s * z : 0.f;
            sFac[tid] = s;
        }
        const bool any_empty = __syncthreads_or(tid < m && !some), has_state = __syncthreads_or(tid < m && some);
        // the columns' sizes in s S', from its first 64 features: a lane a column and 16 features. (A column that
        // is 0 there gets a scale that takes what later features may hold out of range, unless it is 0 in effect.)
        if (!wait(&s_full[0], 0)) break;
        {
            for (int rg = warp; rg < D / 8; rg += C::THREADS / 32) {
                const int q = lane >> 3;
                float mx = 0.f;
                const uint8_t *src = (q < 2 ? sXH : sXL) + MR * 128 + rg * 1024;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 x = *(const float4 *)(src + sw128_offset(lane & 7, 4 * (q & 1) + i));
                    const int r = 16 * q + 4 * i;
                    if (r < m) {
                        const float4 f = *(const float4 *)(sFac + r);
                        const float y[4] = {fabsf(x.x * f.x), fabsf(x.y * f.y), fabsf(x.z * f.z), fabsf(x.w * f.w)};
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (y[k] < INFINITY) mx = fmaxf(mx, y[k]);
                    }
                }
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                const int e = mx > 0.f ? min(max((int)(__float_as_uint(mx) >> 23) - 127, -100), 110) : -100;
                if (lane < 8) sUp[8 * rg + lane] = __uint_as_float((uint32_t)(127 + (int)kTreeTcState - e) << 23);
            }
        }
        if (!wait(mma_done, nm++ & 1)) break;
        tc_fence_after();
        if (C::OVER && nch > 1) load_state();
        if (nh == 1) load_values();

        // row maxima of P + sgn X over this thread's columns of a half
        auto row_max = [&](uint32_t col, int h, float sgn) {
            float mx = -INFINITY;
            const int f0 = 128 * h + 128 / NCG * cg;
#pragma unroll 1
            for (int q = 0; q < 128 / NCG; q += 16) {
                if (f0 + q >= m) break;
                float v[16];
                tmem_ld16(tL + col + 128 / NCG * cg + q, v);
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const float4 x = *(const float4 *)(sX + f0 + q + e);
                    float t[4];
                    ffma2(v[e], v[e + 1], sgn * kLog2e, sgn * kLog2e, x.x, x.y, t[0], t[1]);
                    ffma2(v[e + 2], v[e + 3], sgn * kLog2e, sgn * kLog2e, x.z, x.w, t[2], t[3]);
#pragma unroll
                    for (int k = 0; k < 4; k += 2) mx = fmax3(mx, sgn * t[k], sgn * t[k + 1]);
                }
            }
            return mx;
        };
        float g2 = 0.f, f2 = 0.f;
        auto maxima = [&]() {
            if (is_key) {
                float x = row_max(C::T_K, 0, -1.f);
                if (nh == 2) x = fmaxf(x, row_max(C::T_H + C::T_K, 1, -1.f));
                sMx[cg * 128 + row] = x;
            }
            if (is_query) {
                float x = row_max(C::T_Q, 0, 1.f);
                if (nh == 2) x = fmaxf(x, row_max(C::T_H + C::T_Q, 1, 1.f));
                sMx[(NCG + cg) * 128 + row] = x;
            }
            __syncthreads();
            auto over_groups = [&](const float *at) {
                float x = at[row];
#pragma unroll
                for (int i = 1; i < NCG; ++i) x = fmaxf(x, at[i * 128 + row]);
                return ceilf(x);
            };
            if (is_key) g2 = over_groups(sMx);
            if (is_query) f2 = over_groups(sMx + NCG * 128);
        };
        bool raise = any_empty;
        if (!raise) {
            maxima();
            const float G = g2 + eN;
            raise = __syncthreads_or(is_key && row < n && G > kTreeTcRaise && G < INFINITY);
        }
        if (raise) {
            float *sE = (float *)sXH;  // [4][256], the lane quarters' maxima
            if (is_key) {
                for (int h = 0; h < nh; ++h) {
                    const int f0 = 128 * h + 128 / NCG * cg;
#pragma unroll 1
                    for (int q = 0; q < 128 / NCG; q += 16) {
                        if (f0 + q >= m) break;
                        float v[16], mine = -INFINITY;
                        tmem_ld16(tL + h * C::T_H + C::T_K + 128 / NCG * cg + q, v);
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float u = fmaf(v[e], kLog2e, eN);
                            if (!(row < n && fabsf(u) < INFINITY)) u = -INFINITY;
                            u = from_order_bits(__reduce_max_sync(0xffffffffu, order_bits(u)));
                            if (e == lane) mine = u;
                        }
                        if (lane < 16) sE[(warp & 3) * 256 + f0 + q + lane] = mine;
                    }
                }
            }
            __syncthreads();
            if (tid < m) {
                float E = sE[tid];
#pragma unroll
                for (int w = 1; w < MR / 32; ++w) E = fmaxf(E, sE[w * 256 + tid]);
                const float old = sX[tid];
                float x = fmaxf(old, rintf(E));
                if (!(fabsf(x) < INFINITY)) x = 0.f;
                const float s = exp2f(old - x);
                sX[tid] = x;
                sZ[tid] *= s;
                sFac[tid] *= s;
            }
            __syncthreads();
            maxima();
        }
        if (is_key && cg == 0) sGe[row] = row < n ? exp2f(g2 + eN) * 0x1p-30f : 0.f;

        float den_s[2] = {0.f, 0.f}, sum_a[2] = {0.f, 0.f}, sum_q[2] = {0.f, 0.f};  // 2^15 y_i, sum_r a_jr and b_ir, of this thread's features
        float(&sum_b)[2] = STACK ? sum_a : sum_q;  // (a thread of a stacked tile has a key or a query)
        // 16 features from TMEM: 2^(15 + P + sgn X - max) as hi + lo
        auto split = [&](uint32_t col, int f, float sgn, float c, uint32_t(&hi)[8], uint32_t(&lo)[8], float(&sum)[2], bool state) {
            float v[16];
            tmem_ld16(tL + col, v);
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                const float4 x4 = *(const float4 *)(sX + f + e);
                const float x[4] = {x4.x, x4.y, x4.z, x4.w};
                float4 s4 = make_float4(0.f, 0.f, 0.f, 0.f);
                if (state) s4 = *(const float4 *)(sZ + f + e);
                const float s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
                for (int k = 0; k < 4; k += 2) {
                    float y0, y1, l0, l1;
                    ffma2(x[k], x[k + 1], sgn, sgn, c, c, y0, y1);  // whole numbers: exact
                    ffma2(v[e + k], v[e + k + 1], kLog2e, kLog2e, y0, y1, y0, y1);
                    y0 = ex2_approx(y0);
                    y1 = ex2_approx(y1);
                    ffma2(y0, y1, 0x1p15f, 0x1p15f, 0.f, 0.f, y0, y1);
                    // (the keys' hi is rounded, the queries' truncated: lo lo, which is left out, then has no sign)
                    const float h0 = state ? tf32_trunc(y0) : hi_round(y0), h1 = state ? tf32_trunc(y1) : hi_round(y1);
                    ffma2(y0, y1, 1.f, 1.f, sum[0], sum[1], sum[0], sum[1]);
                    if (state) ffma2(y0, y1, s[k], s[k + 1], den_s[0], den_s[1], den_s[0], den_s[1]);
                    ffma2(h0, h1, -1.f, -1.f, y0, y1, l0, l1);
                    hi[(e + k) >> 1] = pack_f16x2(h0, h1);
                    lo[(e + k) >> 1] = pack_f16x2(l0, l1);
                }
            }
        };
        for (int c0 = 0; c0 < nch; c0 += NSB) {  // steps of 64 NSB features
            const int c1 = min(nch, c0 + NSB), h = c0 >> 1;
            // exponentials: a to shared memory, b in place of its logits
#pragma unroll 2
            for (int u = 0; u < 4 * NSB / NCG; ++u) {
                const int col = (NSB == 2 ? 0 : 64 * (c0 & 1)) + 64 * NSB / NCG * cg + 16 * u;  // in this half
                const int f = 128 * h + col, blk = NSB == 2 ? col >> 6 : 0;
                if (f >= m) break;
                uint32_t hi[8], lo[8];
                if (is_key) {
                    split(C::T_K + col, f, -1.f, -g2, hi, lo, sum_a, false);
                    uint8_t *xh = sXH + blk * C::XB, *xl = blk == 0 ? sXL : sXL1;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t at = sw128_offset(row, ((col & 63) >> 3) + i);
                        *(uint4 *)(xh + at) = make_uint4(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
                        *(uint4 *)(xl + at) = make_uint4(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
                    }
                }
                if (is_query) {
                    split(C::T_Q + col, f, 1.f, -f2, hi, lo, sum_b, true);
                    tmem_st8u(tL + C::T_Q + col, hi);
                    tmem_st8u(tL + C::T_Q + col + 8, lo);
                }
            }
            tmem_wait_st();
            // s S' of the step in place: the rows of a chunk's raw blocks (32 features each) become its
            // high and low block of 64 features
            for (int c = c0; c < c1; ++c)
                if (!wait(&s_full[c % NSB], (c / NSB) & 1)) break;
            if (!ok) break;
            bool bad = false;
            for (int t = warp; t < (c1 - c0) * (D / 8); t += C::THREADS / 32) {
                const int c = c0 + t / (D / 8), rg = t % (D / 8), s = c % NSB, q = lane >> 3, r = 64 * c + 16 * q;
                uint8_t *xh = sXH + s * C::XB + MR * 128 + rg * 1024, *xl = (s == 0 ? sXL : sXL1) + MR * 128 + rg * 1024;
                const float up = sUp[8 * rg + (lane & 7)];
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 x = *(const float4 *)((q < 2 ? xh : xl) + sw128_offset(lane & 7, 4 * (q & 1) + i));
                    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (r < m) f = *(const float4 *)(sFac + r + 4 * i);
                    const float y[4] = {x.x * up * f.x, x.y * up * f.y, x.z * up * f.z, x.w * up * f.w};
                    float yh[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        yh[k] = hi_round(y[k]);
                        bad = bad || !(fabsf(yh[k]) < 65504.f);
                    }
                    hi[2 * i] = pack_f16x2(yh[0], yh[1]);
                    hi[2 * i + 1] = pack_f16x2(yh[2], yh[3]);
                    lo[2 * i] = pack_f16x2(y[0] - yh[0], y[1] - yh[1]);
                    lo[2 * i + 1] = pack_f16x2(y[2] - yh[2], y[3] - yh[3]);
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t at = sw128_offset(lane & 7, 2 * q + i);
                    *(uint4 *)(xh + at) = make_uint4(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
                    *(uint4 *)(xl + at) = make_uint4(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
                }
            }
            if (bad) sFlag[0] = 1;
            fence_async_smem();
            tc_fence_before();
            __syncthreads();
            tc_fence_after();
            const bool next_half = (c1 & 1) == 0 && c1 < nch;
            if (warp == 0) {
                // K-steps of 16 features: hi lo and lo hi of all, then hi hi. (Each addition truncates the
                // accumulator; the first two thirds of a first half's then truncate a small one.)
                constexpr uint32_t idesc_x = make_idesc(128, MR + D, kFmtF16, 0, 0);
                constexpr uint32_t idesc_a = make_idesc(128, MR, kFmtF16, 0, 0), idesc_y = make_idesc(128, D, kFmtF16, 0, 0);
                const uint64_t dXH = make_sdesc(smem_u32(sXH), 16, 1024), dXL = make_sdesc(smem_u32(sXL), 16, 1024);
                const uint64_t dXL1 = make_sdesc(smem_u32(sXL1), 16, 1024);
#pragma unroll 1
                for (int i = 0; i < 3; ++i)
#pragma unroll 1
                    for (int c = c0; c < c1; ++c) {  // 64 features: four steps, or two at the end of m
                        const int s = c % NSB;
                        const uint64_t x = i != 0 ? dXH + s * (C::XB / 16) : s == 0 ? dXL : dXL1;
                        const uint32_t b = tmem + C::T_Q + 64 * (c & 1) + (i == 1 ? 8 : 0);
                        if (c == 2 && i == 0) {  // the second half's Y starts anew
                            mma_f16_ts_w(tmem + C::T_A, b, x, idesc_a, 1u);
                            mma_f16_ts_w(tmem + C::T_Y, b, x + MR * 128 / 16, idesc_y, 0u);
                            for (int k = 1; k < (m - 128 < 64 ? 2 : 4); ++k)
                                mma_f16_ts_w(tmem + C::T_A, b + 16 * k, x + 2 * k, idesc_x, 1u);
                        } else if (64 * c + 64 <= m) {
                            mma_ts_x4_w(tmem + C::T_A, b, x, idesc_x, c + i > 0, 2, 16);
                        } else {
                            mma_f16_ts_w(tmem + C::T_A, b, x, idesc_x, c + i > 0);
                            mma_f16_ts_w(tmem + C::T_A, b + 16, x + 2, idesc_x, 1u);
                        }
                    }
                mma_commit_w(mma_done);
            }
            ++nc;
            if (!wait(mma_done, nm++ & 1)) break;
            tc_fence_after();
            if (next_half) {  // over this half's b: the MMAs that read it are done
                if (warp == 0) {
                    logits(h + 1, 0);
                    mma_commit_w(mma_done);
                }
                ++nc;
            }
            while (ns < min(nch, c1 + NSB)) load_state();
            if (next_half) {
                if (!wait(mma_done, nm++ & 1)) break;
                tc_fence_after();
                load_values();
                // Y of the first half moves out (T_Y starts anew): each addition truncates the accumulator by up to
                // 2^-23 of it, while y_i is summed with rounding. Equal values then come out 6e-7 low at m = 256, and
                // 2e-6 low where one accumulator holds both halves (0.6 us of 43 for 256 heads of 60 nodes at d = 128).
                if (is_query) {
#pragma unroll 1
                    for (int c = cg * (D / NCG); c < (cg + 1) * (D / NCG); c += 16) {
                        float y[16];
                        tmem_ld16(tL + C::T_Y + c, y);
#pragma unroll
                        for (int e = 0; e < 16; e += 4) *(float4 *)(sY + row_chunk(c + e)) = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
                    }
                }
            }
        }
        if (!ok) break;
        if (is_key) sSum[cg * 128 + row] = sum_a[0] + sum_a[1];
        if (is_query) sSum[(NCG + cg) * 128 + row] = sum_b[0] + sum_b[1];

        // values: rows past the tree are not the tree's; non-finite ones must not meet a zero weight
        if (!wait(v_full, 0)) break;
        {
            bool bad = false;
            for (int i = tid; i < NB * MR * 8; i += C::THREADS) {
                uint4 *at = (uint4 *)(sV + (size_t)i * 16);
                if (((i >> 3) & (MR - 1)) >= n) {
                    *at = make_uint4(0u, 0u, 0u, 0u);
                } else {
                    const uint4 x = *at;
                    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) bad = bad || __vcmpgeu2(u[k] & 0x7FFF7FFFu, 0x7F807F80u) != 0u;
                }
            }
            if (bad) sFlag[0] = 1;
        }
        // weights of the visible nodes
        if (is_query) {
            constexpr int KT = MR / NCG;  // keys a thread takes
            static_assert(KT <= 32, "one word of J");
            auto over_groups = [&](const float *at, int i) {
                float x = at[i];
#pragma unroll
                for (int k = 1; k < NCG; ++k) x += at[k * 128 + i];
                return x;
            };
            const float sb = over_groups(sSum + NCG * 128, row);
            float den = has_state ? (den_s[0] + den_s[1]) * 0x1p-15f : 0.f;
            float err = has_state && cg == 0 ? sb * 0x1p-21f : 0.f;  // (S''s own: 2^-31 of sb, in err's units)
            const int j0 = KT * cg;
            const uint32_t seen = sAnc[row * (MR / 32) + (j0 >> 5)] >> (j0 & 31);
#pragma unroll
            for (int q = 0; q < KT; q += 16) {
                float v[16];
                uint32_t part[3][8];
                tmem_ld16(tL + C::T_A + j0 + q, v);
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    uint32_t w0[2], w1[2], w2[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int j = j0 + q + e + k;
                        float w = 0.f;
                        if ((seen >> (q + e + k)) & 1u) {
                            w = v[e + k] * sGe[j];
                            err = fmaf(sGe[j], sb + over_groups(sSum, j), err);
                        }
                        den += w;
                        // w in three bf16 parts of 8 bits, by truncation
                        w0[k] = __float_as_uint(w);
                        const float r1 = w - __uint_as_float(w0[k] & 0xFFFF0000u);
                        w1[k] = __float_as_uint(r1);
                        w2[k] = __float_as_uint(r1 - __uint_as_float(w1[k] & 0xFFFF0000u));
                    }
                    part[0][e >> 1] = __byte_perm(w0[0], w0[1], 0x7632);
                    part[1][e >> 1] = __byte_perm(w1[0], w1[1], 0x7632);
                    part[2][e >> 1] = __byte_perm(w2[0], w2[1], 0x7632);
                }
#pragma unroll
                for (int t = 0; t < 3; ++t) tmem_st8u(tL + t * (MR / 2) + ((j0 + q) >> 1), part[t]);
            }
            tmem_wait_st();
            sDen[cg * 128 + row] = den;
            sErr[cg * 128 + row] = err;
        }
        fence_async_smem();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (warp == 0) {
            const uint32_t idesc = make_idesc(128, D, kFmtBF16, 0, 1);
            const uint64_t dV = make_sdesc(smem_u32(sV), MR * 128, 1024);
            for (int t = 2; t >= 0; --t)  // the small parts first, as above
                for (int k = 0; k < (n + 15) / 16; ++k)
                    mma_f16_ts_w(tmem + C::T_O, tmem + t * (MR / 2) + 8 * k, dV + k * (16 * 128 / 16), idesc, t < 2 || k > 0);
            mma_commit_w(mma_done);
        }
        ++nc;
        // rows that stand: a finite denominator, 2^20 times its error bound (2^-25 of sErr's sum)
        bool good = false;
        float inv = 0.f;
        if (is_query) {
            float den = sDen[row], err = sErr[row];
#pragma unroll
            for (int k = 1; k < NCG; ++k) {
                den += sDen[k * 128 + row];
                err += sErr[k * 128 + row];
            }
            good = den >= 1e-30f && den < INFINITY && den >= err * 0x1p-5f;
            inv = 1.f / den;
        }
        if (!wait(mma_done, nm++ & 1)) break;
        tc_fence_after();
        // rows out, through shared memory (16-byte chunks XOR-swizzled by row)
        float *sOut = (float *)sW;
        if (is_query) {
            if (cg == 0) sPtr[row] = good && sFlag[0] == 0;
            constexpr int CT = D / NCG;  // columns a thread takes
#pragma unroll
            for (int q = 0; q < CT; q += 16) {
                const int c0 = cg * CT + q;
                float y[16], o[16];
                tmem_ld16_nowait(tL + C::T_Y + c0, y);
                tmem_ld16_nowait(tL + C::T_O + c0, o);
                tmem_wait_ld16(y);
                tmem_wait_ld16(o);
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    float x[4];
                    if (nh == 2) {
                        const float4 y1 = *(const float4 *)(sY + row_chunk(c0 + e));
                        y[e] += y1.x, y[e + 1] += y1.y, y[e + 2] += y1.z, y[e + 3] += y1.w;
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {  // (2^-15 / up: powers of two)
                        const float down = __uint_as_float((239u << 23) - __float_as_uint(sUp[c0 + e + k]));
                        x[k] = (has_state ? fmaf(down, y[e + k], o[e + k]) : o[e + k]) * inv;
                    }
                    *(float4 *)(sOut + row_chunk(c0 + e)) = make_float4(x[0], x[1], x[2], x[3]);
                }
            }
        }
        __syncthreads();
        float *out = p.out + (size_t)bh * T * D;
        for (int i = tid; i < n * (D / 4); i += C::THREADS) {
            const int r = i / (D / 4), c = i % (D / 4);
            if (sPtr[r]) *(float4 *)(out + (size_t)i * 4) = *(const float4 *)(sOut + r * D + ((c ^ (r & 7)) << 2));
        }
        // the others: a warp a row in turn, or where there are few rows two or four warps
        constexpr int NW = C::THREADS / 32;
        uint32_t left[MR / 32];
        int rows = 0;
#pragma unroll
        for (int w = 0; w < MR / 32; ++w) {
            left[w] = __ballot_sync(0xffffffffu, 32 * w + lane < n && !sPtr[32 * w + lane]);
            rows += __popc(left[w]);
        }
        if (rows != 0) {
            const int parts = 4 * rows <= NW ? 4 : 2 * rows <= NW ? 2 : 1, share = NW / parts;
            float *part_out = (float *)sXH;  // [row][part][D + 2]
            int k = 0;
            for (int w = 0; w < MR / 32; ++w)
                for (uint32_t x = left[w]; x != 0; x &= x - 1, ++k)
                    if (k % share == warp / parts)
                        tree_row_exact_bf16<D>(p, bh, 32 * w + __ffs(x) - 1, sPar, warp % parts, parts,
                                               part_out + (k * parts + warp % parts) * (D + 2));
            if (parts > 1) {
                __syncthreads();
                k = 0;
                for (int w = 0; w < MR / 32; ++w)
                    for (uint32_t x = left[w]; x != 0; x &= x - 1, ++k)
                        if (k == warp) tree_row_join<D>(p, bh, 32 * w + __ffs(x) - 1, parts, part_out + k * parts * (D + 2));
            }
        }
    } while (false);

    if (!ok && warp == 0) {  // a wait ran out: nothing of this CTA stays in flight
        volatile int no_abort = 0;
        mma_commit_w(mma_done);
        if (nc > 0) mbar_wait_all(mma_done, (nc - 1) & 1, &no_abort);
        mbar_wait_all(mma_done, nc & 1, &no_abort);
        mbar_wait_all(kq_full, 0, &no_abort);
        mbar_wait_all(w_full, 0, &no_abort);
        for (int c = max(ns - NSB, 0); c < ns; ++c) mbar_wait_all(&s_full[c % NSB], (c / NSB) & 1, &no_abort);
        if (v_asked) mbar_wait_all(v_full, 0, &no_abort);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::COLS);
    }
}

template <int D, bool STACK>
static cudaError_t launch_tree_tc_t(const CUtensorMap &mQ, const CUtensorMap &mK, const CUtensorMap &mV,
                                    const CUtensorMap &mW, const CUtensorMap &mS, const TreeParams &p, cudaStream_t st) {
    using C = TreeTc<D, STACK>;
    const cudaError_t e =
        cudaFuncSetAttribute(k_decode_tree_tc<D, STACK>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::BYTES);
    if (e != cudaSuccess) return e;
    k_decode_tree_tc<D, STACK><<<p.B * p.H, C::THREADS, C::BYTES, st>>>(mQ, mK, mV, mW, mS, p);
    return cudaGetLastError();
}

cudaError_t launch_decode_tree_tc(const CUtensorMap &mQ, const CUtensorMap &mK, const CUtensorMap &mV,
                                  const CUtensorMap &mW, const CUtensorMap &mS, const TreeParams &p, int d, cudaStream_t st) {
    if (p.T <= 64) return d == 64 ? launch_tree_tc_t<64, true>(mQ, mK, mV, mW, mS, p, st) : launch_tree_tc_t<128, true>(mQ, mK, mV, mW, mS, p, st);
    return d == 64 ? launch_tree_tc_t<64, false>(mQ, mK, mV, mW, mS, p, st) : launch_tree_tc_t<128, false>(mQ, mK, mV, mW, mS, p, st);
}

}  // namespace favor
