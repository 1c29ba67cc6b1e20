// Tokens added to the carried state of favor_decode_step: a prompt's, or the nodes of an accepted
// path, S_r += sum_j e^(u_r(k_j)) v_j, z_r += sum_j e^(u_r(k_j)), u_r(x) = w_r.x - |x|^2/2, each
// feature held relative to e^(D_r) with D_r the largest u_r so far (as favor_decode_step keeps it).

#include "common.cuh"

namespace favor {

struct ExtendParams {
    int B, H, L, m;
    int bf16;               // k, v, W bf16 (else fp32)
    const void *k, *v;      // [B, H, L, d]
    const void *W;          // [m, d]
    const int *index;       // [B, n_tok] token positions, or NULL (0, 1, ...)
    const int *counts;      // [B] or NULL (n_tok each)
    int n_tok;              // tokens a sequence may add: the index's width, or L
    float *state;           // [B * H][d m + 2 m]
    float *part;            // n_split > 1: [B * H][n_split][d m + 2 m]
    int n_split, tok_per_split;
};

// Tokens sequence b adds, clamped to what its row holds (a count outside it is recorded).
__device__ __forceinline__ int extend_count(const ExtendParams &p, int b) {
    if (p.counts == nullptr) return p.n_tok;
    const int n = p.counts[b];
    if (n < 0 || n > p.n_tok) record_status(FAVOR_ERR_INVALID_ARG);
    return min(max(n, 0), p.n_tok);
}

// Position of token t of sequence b, or -1 for an index outside the buffer (recorded, not added).
__device__ __forceinline__ int extend_token(const ExtendParams &p, int b, int t) {
    if (p.index == nullptr) return t;
    const int j = p.index[(size_t)b * p.n_tok + t];
    if (j < 0 || j >= p.L) {
        record_status(FAVOR_ERR_INVALID_ARG);
        return -1;
    }
    return j;
}

// ------------------------------------------------------------------------------- rows on warp MMAs
//
// fp32 tokens, and bf16 ones by index or too few for tiles. One CTA per (run of tokens, head, 64 value
// columns), a warp per 32 features, W in shared memory, 16 tokens at a time, double-buffered. All in
// registers: P's accumulator fragments (features x tokens) become phi and are the next MMA's A operand as
// they stand, with tokens 2t, 2t + 1 in the places of K = t, t + 4 on both sides. Products are tf32 with
// both operands hi + lo (three MMAs, 2^-22; bf16 operands are exact in one part); the S accumulators are
// added to fp32 registers every 64 tokens, since the tensor core truncates as it accumulates.
// Bound: the rate of these MMAs and the splits around them: 1.8 ms for 65536 fp32 tokens in 16 heads at
// d = 64, m = 256 (sums on CUDA cores, a feature a thread: 5.7 ms).

constexpr int kExtBlk = 16;
constexpr int kExtRowCols = 64;

template <int D, bool BF16>
struct ExtRows {
    static constexpr int ES = BF16 ? 2 : 4;
    // row strides in bytes: 64 mod 128 for 16-byte fragments, 16 mod 64 apart by two rows for values
    static constexpr int LDW = D * ES + 64, LDV = kExtRowCols * ES + 16;
    static constexpr size_t KV = (size_t)kExtBlk * (LDW + LDV);
    static size_t bytes(int m) { return (size_t)m * LDW + 2 * KV + 2 * kExtBlk * 4; }
};

__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

template <int D, bool BF16>
__global__ void __launch_bounds__(256, 1) k_decode_extend_rows(ExtendParams p) {
    using C = ExtRows<D, BF16>;
    constexpr int ES = C::ES, NT = kExtRowCols / 8;
    extern __shared__ __align__(16) uint8_t sm8[];
    const int split = blockIdx.x, bh = blockIdx.y, b = bh / p.H, v0 = blockIdx.z * kExtRowCols, m = p.m;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3, f0 = 32 * warp;
    const int n = extend_count(p, b);
    if (n == 0) return;  // the state stays as it is
    const int t0 = split * p.tok_per_split, t1 = min(n, t0 + p.tok_per_split);
    if (t0 >= t1) return;  // an empty run
    const bool whole = p.n_split == 1 && D == 64;  // (two CTAs of a head must not meet in its state)
    const size_t len = (size_t)D * m + 2 * m;
    uint8_t *sW = sm8, *sTok = sW + (size_t)m * C::LDW;
    int *sUse = (int *)(sTok + 2 * C::KV);  // [2][16]: a token that is added
    const size_t row0 = (size_t)bh * p.L;

    for (int i = tid; i < m * (D * ES / 16); i += blockDim.x) {
        const int r = i / (D * ES / 16), c = i % (D * ES / 16);
        cp_async16(sW + (size_t)r * C::LDW + 16 * c, (const char *)p.W + (size_t)r * D * ES + 16 * c);
    }
    auto fetch = [&](int blk) {  // tokens of block blk into its buffer
        uint8_t *kb = sTok + (blk & 1) * C::KV, *vb = kb + kExtBlk * C::LDW;
        constexpr int KC = D * ES / 16, VC = kExtRowCols * ES / 16;
        for (int i = tid; i < kExtBlk * (KC + VC); i += blockDim.x) {
            const int j = i / (KC + VC), c = i % (KC + VC), tok = t0 + blk * kExtBlk + j;
            const int at = tok < t1 ? extend_token(p, b, tok) : -1;
            uint8_t *dst = c < KC ? kb + j * C::LDW + 16 * c : vb + j * C::LDV + 16 * (c - KC);
            if (at >= 0)
                cp_async16(dst, c < KC ? (const char *)p.k + (row0 + at) * D * ES + 16 * c
                                       : (const char *)p.v + ((row0 + at) * D + v0) * ES + 16 * (c - KC));
            else
                *(uint4 *)dst = make_uint4(0u, 0u, 0u, 0u);
            if (c == 0) sUse[(blk & 1) * kExtBlk + j] = at >= 0;
        }
        cp_async_commit();
    };
    const int nblk = (t1 - t0 - 1) / kExtBlk + 1;
    fetch(0);

    float S[2][NT][4], acc[2][NT][4], z[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
    float Dr[2][2] = {{-INFINITY, -INFINITY}, {-INFINITY, -INFINITY}};
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int c = 0; c < NT; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) S[a][c][e] = acc[a][c][e] = 0.f;

    for (int blk = 0; blk < nblk; ++blk) {
        cp_async_wait_all();
        __syncthreads();
        if (blk + 1 < nblk) fetch(blk + 1);
        const uint8_t *kb = sTok + (blk & 1) * C::KV, *vb = kb + kExtBlk * C::LDW;
        // P: [32 features][16 tokens]
        float P[2][2][4], Q[2][2][4], sq[2] = {0.f, 0.f};
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) P[a][c][e] = Q[a][c][e] = 0.f;
        const uint8_t *wr = sW + (size_t)(f0 + g) * C::LDW + 16 * t, *kr = kb + g * C::LDW + 16 * t;
#pragma unroll 2
        for (int j = 0; j < D * ES / 64; ++j) {
            uint4 w[2][2], x[2];
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int h = 0; h < 2; ++h) w[a][h] = *(const uint4 *)(wr + (size_t)(16 * a + 8 * h) * C::LDW + 64 * j);
#pragma unroll
            for (int c = 0; c < 2; ++c) x[c] = *(const uint4 *)(kr + (size_t)8 * c * C::LDW + 64 * j);
            if constexpr (BF16) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const uint32_t u[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float lo = __uint_as_float(u[e] << 16), hi = __uint_as_float(u[e] & 0xFFFF0000u);
                        sq[c] = fmaf(lo, lo, sq[c]);
                        sq[c] = fmaf(hi, hi, sq[c]);
                    }
#pragma unroll
                    for (int a = 0; a < 2; ++a) {
                        mma_bf16_16x8x16(P[a][c], w[a][0].x, w[a][1].x, w[a][0].y, w[a][1].y, x[c].x, x[c].y);
                        mma_bf16_16x8x16(P[a][c], w[a][0].z, w[a][1].z, w[a][0].w, w[a][1].w, x[c].z, x[c].w);
                    }
                }
            } else {
                uint32_t xh[2][4], xl[2][4];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const uint32_t u[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float f = __uint_as_float(u[e]);
                        sq[c] = fmaf(f, f, sq[c]);
                        tf32_split(f, xh[c][e], xl[c][e]);
                    }
                }
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    const uint32_t u0[4] = {w[a][0].x, w[a][0].y, w[a][0].z, w[a][0].w};
                    const uint32_t u1[4] = {w[a][1].x, w[a][1].y, w[a][1].z, w[a][1].w};
                    uint32_t h0[4], l0[4], h1[4], l1[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        tf32_split(__uint_as_float(u0[e]), h0[e], l0[e]);
                        tf32_split(__uint_as_float(u1[e]), h1[e], l1[e]);
                    }
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            mma_tf32_16x8x8(Q[a][c], l0[e], l1[e], l0[e + 1], l1[e + 1], xh[c][e], xh[c][e + 1]);
                            mma_tf32_16x8x8(Q[a][c], h0[e], h1[e], h0[e + 1], h1[e + 1], xl[c][e], xl[c][e + 1]);
                            mma_tf32_16x8x8(P[a][c], h0[e], h1[e], h0[e + 1], h1[e + 1], xh[c][e], xh[c][e + 1]);
                        }
                }
            }
        }
        // u = P - |k|^2/2 of tokens 8c + 2t, 8c + 2t + 1 (-inf for one that is not added)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            sq[c] += __shfl_xor_sync(0xffffffffu, sq[c], 1);
            sq[c] += __shfl_xor_sync(0xffffffffu, sq[c], 2);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float h = 0.5f * __shfl_sync(0xffffffffu, sq[c], 4 * (2 * t + e));
                const bool use = sUse[(blk & 1) * kExtBlk + 8 * c + 2 * t + e] != 0;
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    P[a][c][e] = use ? P[a][c][e] + Q[a][c][e] - h : -INFINITY;
                    P[a][c][2 + e] = use ? P[a][c][2 + e] + Q[a][c][2 + e] - h : -INFINITY;
                }
            }
        }
        // D_r, then phi (in P's place)
        bool raise = false;
        float Dn[2][2];
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float x = fmaxf(fmaxf(P[a][0][2 * h], P[a][0][2 * h + 1]), fmaxf(P[a][1][2 * h], P[a][1][2 * h + 1]));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                Dn[a][h] = fmaxf(Dr[a][h], x);
                raise = raise || Dn[a][h] > Dr[a][h];
            }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float keep = Dr[a][h] == -INFINITY ? 0.f : expf(Dr[a][h] - Dn[a][h]);
                    Dr[a][h] = Dn[a][h];
                    z[a][h] *= keep;
#pragma unroll
                    for (int c = 0; c < NT; ++c)
#pragma unroll
                        for (int e = 2 * h; e < 2 * h + 2; ++e) {
                            S[a][c][e] *= keep;
                            acc[a][c][e] *= keep;
                        }
                }
        }
        uint32_t ph[2][2][4], pl[2][2][4];
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float u = P[a][c][e];
                    const float x = u == -INFINITY ? 0.f : ex2_approx((u - Dr[a][e >> 1]) * kLog2e);
                    z[a][e >> 1] += x;
                    tf32_split(x, ph[a][c][e], pl[a][c][e]);
                }
        // acc += phi v
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int q = 0; q < NT; ++q) {
                const uint8_t *at = vb + (size_t)(8 * c + 2 * t) * C::LDV + (8 * q + g) * ES;
                uint32_t vh[2], vl[2] = {0u, 0u};
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if constexpr (BF16)
                        vh[e] = (uint32_t)*(const uint16_t *)(at + e * C::LDV) << 16;
                    else
                        tf32_split(*(const float *)(at + e * C::LDV), vh[e], vl[e]);
                }
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    mma_tf32_16x8x8(acc[a][q], pl[a][c][0], pl[a][c][2], pl[a][c][1], pl[a][c][3], vh[0], vh[1]);
                    if constexpr (!BF16)
                        mma_tf32_16x8x8(acc[a][q], ph[a][c][0], ph[a][c][2], ph[a][c][1], ph[a][c][3], vl[0], vl[1]);
                    mma_tf32_16x8x8(acc[a][q], ph[a][c][0], ph[a][c][2], ph[a][c][1], ph[a][c][3], vh[0], vh[1]);
                }
            }
        if ((blk & 3) == 3 || blk + 1 == nblk) {
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int c = 0; c < NT; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        S[a][c][e] += acc[a][c][e];
                        acc[a][c][e] = 0.f;
                    }
        }
    }
    // the run's sums, joined with the carried state by the first run
    const float *old = p.state + (size_t)bh * len;
    float *dst = whole ? p.state + (size_t)bh * len : p.part + ((size_t)bh * p.n_split + split) * len;
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = f0 + 16 * a + 8 * h + g;
            float zr = z[a][h], fx = 1.f, fy = 0.f, Dn = Dr[a][h];
            zr += __shfl_xor_sync(0xffffffffu, zr, 1);
            zr += __shfl_xor_sync(0xffffffffu, zr, 2);
            if (split == 0) {
                const float z_old = old[(size_t)D * m + r], D_old = old[(size_t)D * m + m + r];
                if (z_old != 0.f) {
                    Dn = fmaxf(D_old, Dn);
                    fy = expf(D_old - Dn);
                    fx = zr != 0.f ? expf(Dr[a][h] - Dn) : 0.f;
                    zr = fmaf(z_old, fy, zr * fx);
                }
            }
            float y[2 * NT];
#pragma unroll
            for (int c = 0; c < NT; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    y[2 * c + e] = fy != 0.f ? __ldcg(old + (size_t)(v0 + 8 * c + 2 * t + e) * m + r) : 0.f;
            __syncwarp();  // the row's four lanes have read z' and D of the carried state
            if (zr != 0.f || !whole) {
#pragma unroll
                for (int c = 0; c < NT; ++c)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        dst[(size_t)(v0 + 8 * c + 2 * t + e) * m + r] = fmaf(y[2 * c + e], fy, S[a][c][2 * h + e] * fx);
                if (v0 == 0 && t == 0) {
                    dst[(size_t)D * m + r] = zr;
                    dst[(size_t)D * m + m + r] = Dn;
                }
            }
        }
}

// ------------------------------------------------------------------------------- accepted paths
//
// Up to kExtPath tokens a head: one CTA per head, two features a thread. All tokens' feature values are
// formed first (registers), then the state streams through, kExtCols value columns in flight at a time,
// each read, rescaled, added to and written once; the traffic, (m d + 2 m) * 8 bytes a head, is the bound.
// What has to stay out of its way is shared memory and L1 (one feature a thread, each reading its own
// row of W and every value: 50 us for 1024 heads at d = 64, m = 256, with L1 77 % busy): two features
// share each value read, and bf16 projections are warp MMAs, whose W fragments are 64-byte runs.

constexpr int kExtPath = 16;
constexpr int kExtCols = 8;

template <int D, bool BF16>
__global__ void __launch_bounds__(128, 5) k_decode_extend_path(ExtendParams p) {
    constexpr int LD = kExtPath + 1;
    __shared__ __align__(16) float sV[kExtPath * D], sU[4 * 64 * LD];
    __shared__ float sN[kExtPath];  // |k|^2 / 2, -1 for a token that is not added
    const int bh = blockIdx.x, b = bh / p.H, m = p.m, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n = extend_count(p, b);
    if (n == 0) return;  // the state stays as it is
    const int nw = blockDim.x >> 5, f0 = 64 * warp;
    const bool two = f0 + 32 < m;  // m is a multiple of 32: the last warp may have one feature a lane
    float *S = p.state + (size_t)bh * ((size_t)D * m + 2 * m) + f0 + lane;
    float *z = S + (size_t)D * m, *Dl = z + m;
    const int second = two ? 32 : 0;  // (a lane without a second feature computes its first twice, stores it once)
    float zr[2], Dr[2], s[2][kExtCols];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        zr[h] = z[h * second];
        Dr[h] = Dl[h * second];
    }
    auto columns = [&](int c0) {
#pragma unroll
        for (int c = 0; c < kExtCols; ++c) {
            s[0][c] = S[(size_t)(c0 + c) * m];
            s[1][c] = S[(size_t)(c0 + c) * m + second];
        }
    };
    columns(0);
    const size_t row0 = (size_t)bh * p.L;
    for (int t = warp; t < n; t += nw) {  // a warp a value row
        const int j = extend_token(p, b, t);
        for (int c = lane; c < D; c += 32) sV[t * D + c] = j < 0 ? 0.f : ld_elem(p.v, BF16, (row0 + j) * D + c);
    }
    for (int i = n * D + tid; i < kExtPath * D; i += blockDim.x) sV[i] = 0.f;
    float u[2][kExtPath], *su = sU + warp * 64 * LD;
    for (int t0 = 0; t0 < n; t0 += 8) {
        const int t = t0 + (lane >> 2), j = t < n ? extend_token(p, b, t) : -1;
        const void *x = j < 0 ? nullptr : (const char *)p.k + (row0 + j) * D * (BF16 ? 2 : 4);
        const float sq = warp_logits<D, LD, 4, BF16>(p.W, m, f0, x, su, t0, lane);
        if (warp == 0 && (lane & 3) == 0) sN[t] = j < 0 ? -1.f : 0.5f * sq;
    }
    if (n <= 8 && warp == 0 && lane < 8) sN[8 + lane] = -1.f;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kExtPath; ++i) {
        u[0][i] = i < 8 || n > 8 ? su[lane * LD + i] : 0.f;
        u[1][i] = i < 8 || n > 8 ? su[(lane + second) * LD + i] : 0.f;
    }
    float keep[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const bool old = zr[h] != 0.f;
        float Dn = old ? Dr[h] : -INFINITY;
#pragma unroll
        for (int i = 0; i < kExtPath; ++i) {
            u[h][i] = sN[i] < 0.f ? -INFINITY : u[h][i] - sN[i];
            Dn = fmaxf(Dn, u[h][i]);
        }
        keep[h] = old ? expf(Dr[h] - Dn) : 0.f;
        zr[h] *= keep[h];
#pragma unroll
        for (int i = 0; i < kExtPath; ++i) {
            u[h][i] = u[h][i] == -INFINITY ? 0.f : expf(u[h][i] - Dn);
            zr[h] += u[h][i];
        }
        if (zr[h] != 0.f && (h == 0 || two)) {  // else no token entered this feature
            z[h * second] = zr[h];
            Dl[h * second] = Dn;
        }
    }
#pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += kExtCols) {
        float x[2][kExtCols];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int c = 0; c < kExtCols; ++c) x[h][c] = keep[h] != 0.f ? s[h][c] * keep[h] : 0.f;
        if (c0 + kExtCols < D) columns(c0 + kExtCols);
#pragma unroll
        for (int i0 = 0; i0 < kExtPath; i0 += 4) {
            if (i0 < n) {
#pragma unroll
                for (int i = i0; i < i0 + 4; ++i)
#pragma unroll
                    for (int c = 0; c < kExtCols; c += 4) {
                        const float4 v = *(const float4 *)(sV + i * D + c0 + c);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            ffma2(u[h][i], u[h][i], v.x, v.y, x[h][c], x[h][c + 1], x[h][c], x[h][c + 1]);
                            ffma2(u[h][i], u[h][i], v.z, v.w, x[h][c + 2], x[h][c + 3], x[h][c + 2], x[h][c + 3]);
                        }
                    }
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (zr[h] != 0.f && (h == 0 || two)) {
#pragma unroll
                for (int c = 0; c < kExtCols; ++c) S[(size_t)(c0 + c) * m + h * second] = x[h][c];
            }
    }
}

template <int D>
static cudaError_t launch_extend_path(const ExtendParams &p, cudaStream_t st) {
    const int threads = 32 * ((p.m + 63) / 64);
    if (p.bf16)
        k_decode_extend_path<D, true><<<p.B * p.H, threads, 0, st>>>(p);
    else
        k_decode_extend_path<D, false><<<p.B * p.H, threads, 0, st>>>(p);
    return cudaGetLastError();
}

// Adds the partial states of a head's runs (the first holds the carried state) into the state: one
// thread per feature, kCombCols value columns per CTA; the CTA of the first columns writes z' and D. One
// pass with a running maximum, kCombRuns runs' loads in flight at a time (left to the compiler they were
// taken one after another: 2 us a run).
constexpr int kCombCols = 4, kCombRuns = 8;

__global__ void __launch_bounds__(256) k_extend_combine(ExtendParams p, int d) {
    const int bh = blockIdx.y, r = threadIdx.x, m = p.m, c0 = blockIdx.x * kCombCols;
    const size_t len = (size_t)d * m + 2 * m;
    const int n = extend_count(p, bh / p.H);
    if (n == 0) return;
    const int runs = (n - 1) / p.tok_per_split + 1;  // the others are empty, and not written
    const float *part = p.part + (size_t)bh * p.n_split * len + r;
    float *S = p.state + (size_t)bh * len + r;
    const size_t oz = (size_t)d * m, oD = oz + m;
    float D = -INFINITY, acc[kCombCols], z = 0.f;
#pragma unroll
    for (int c = 0; c < kCombCols; ++c) acc[c] = 0.f;
    for (int s0 = 0; s0 < runs; s0 += kCombRuns) {
        float zs[kCombRuns], Ds[kCombRuns], x[kCombRuns][kCombCols];
#pragma unroll
        for (int i = 0; i < kCombRuns; ++i) {
            const float *at = part + min(s0 + i, runs - 1) * len;
            zs[i] = __ldcg(at + oz);
            Ds[i] = __ldcg(at + oD);
#pragma unroll
            for (int c = 0; c < kCombCols; ++c) x[i][c] = __ldcg(at + (size_t)(c0 + c) * m);
        }
        float Dn = D;
#pragma unroll
        for (int i = 0; i < kCombRuns; ++i) {
            if (s0 + i >= runs) zs[i] = 0.f;
            Dn = zs[i] != 0.f ? fmaxf(Dn, Ds[i]) : Dn;
        }
        const float keep = z != 0.f ? expf(D - Dn) : 0.f;
        D = Dn;
        z *= keep;
#pragma unroll
        for (int c = 0; c < kCombCols; ++c) acc[c] *= keep;
#pragma unroll
        for (int i = 0; i < kCombRuns; ++i) {
            const float w = zs[i] != 0.f ? expf(Ds[i] - Dn) : 0.f;
            z = fmaf(w, zs[i], z);
#pragma unroll
            for (int c = 0; c < kCombCols; ++c) acc[c] = s0 + i < runs ? fmaf(w, x[i][c], acc[c]) : acc[c];
        }
    }
    if (z == 0.f) return;
#pragma unroll
    for (int c = 0; c < kCombCols; ++c) S[(size_t)(c0 + c) * m] = acc[c];
    if (c0 == 0) {
        S[oz] = z;
        S[oD] = D;
    }
}

template <int D, bool BF16>
static cudaError_t launch_extend_rows(const ExtendParams &p, cudaStream_t st) {
    const size_t sm = ExtRows<D, BF16>::bytes(p.m);
    const cudaError_t e = cudaFuncSetAttribute(k_decode_extend_rows<D, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm);
    if (e != cudaSuccess) return e;
    k_decode_extend_rows<D, BF16><<<dim3(p.n_split, p.B * p.H, D / kExtRowCols), p.m, sm, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_decode_extend(const ExtendParams &p, int d, cudaStream_t st) {
    const int BH = p.B * p.H;
    if (p.n_tok <= kExtPath) return d == 64 ? launch_extend_path<64>(p, st) : launch_extend_path<128>(p, st);
    const cudaError_t e = d == 64 ? (p.bf16 ? launch_extend_rows<64, true>(p, st) : launch_extend_rows<64, false>(p, st))
                                  : (p.bf16 ? launch_extend_rows<128, true>(p, st) : launch_extend_rows<128, false>(p, st));
    if (e != cudaSuccess) return e;
    if (p.n_split > 1 || d != 64) k_extend_combine<<<dim3(d / kCombCols, BH), p.m, 0, st>>>(p, d);
    return cudaGetLastError();
}

}  // namespace favor
