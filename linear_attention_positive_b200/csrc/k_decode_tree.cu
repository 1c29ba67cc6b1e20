// Attention of a tree of drafted tokens over the carried state of favor_decode_step: node i sees
// every committed token (through S', z', D) and J(i), its ancestors and itself,
//   out_i = [sum_r e^(w_r.q_i) (S_r + sum_{j in J(i)} e^(u_r(k_j)) v_j)]
//           / [sum_r e^(w_r.q_i) (z_r + sum_{j in J(i)} e^(u_r(k_j)))],   u_r(x) = w_r.x - |x|^2/2.
//
// Scaled form, so that nothing overflows and a node that a row does not see cannot push the row's
// own terms out of range by its norm: with E_r = max_j w_r.k_j over the tree's (finite) logits,
//   a_rj = e^(w_r.k_j - E_r) <= 1,           e_j = -|k_j|^2/2         (one scale per token),
//   s_r  = e^(D_r - E_r - e_S) <= 1,         e_S = max_r (D_r - E_r)  (one scale for the state),
//   b_ri = e^(w_r.q_i + E_r - f_i) <= 1,     f_i its row maximum (cancels),
//   A_ij = sum_r b_ri a_rj,  M_i = the largest of e_S and e_j over J(i),
//   out_i = [e^(e_S - M_i) sum_r b_ri s_r S'_r + sum_{j in J(i)} e^(e_j - M_i) A_ij v_j] / [same of z', 1].
// What can still be lost is a row whose visible terms are all e^-87 or more below the features'
// maxima E_r, which nodes it does not see may have set. Its denominator then comes out below
// kTreeDenMin and the row is recomputed in log space from its own visible terms alone
// (tree_row_exact); the same path takes nothing from nodes outside J(i), so NaN or infinities there
// never reach a row.

#include "common.cuh"

namespace favor {

// Terms lost to underflow are at most m T 2^-126 < 4e-34 in the scaled denominator: 4e-14 of one
// that is at least this.
constexpr float kTreeDenMin = 1e-20f;

struct TreeParams {
    int B, H, T, m;
    int bf16;                  // q, k, v, W bf16 (else fp32)
    const void *q, *k, *v;     // [B, H, T, d]
    const void *W;             // [m, d]
    const float *state;        // [B * H][d m + 2 m]
    const int *parents;        // [B, T]
    const int *n_nodes;        // [B] or NULL
    float *out;                // [B, H, T, d]
};

__device__ __forceinline__ float ld_elem(const void *p, int bf16, size_t i) {
    return bf16 ? __uint_as_float((uint32_t)((const uint16_t *)p)[i] << 16) : ((const float *)p)[i];
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Number of nodes of sequence b, clamped to the buffer (a count outside it is recorded).
__device__ __forceinline__ int tree_count(const int *n_nodes, int b, int T) {
    if (n_nodes == nullptr) return T;
    const int n = n_nodes[b];
    if (n < 0 || n > T) record_status(FAVOR_ERR_INVALID_ARG);
    return min(max(n, 0), T);
}

// A node's parent, -1 for a root. A parent outside -1 .. i-1 is recorded and read as -1, so that a
// walk up the tree always ends.
__device__ __forceinline__ int tree_parent(const int *parents, int i) {
    const int p = parents[i];
    if (p < -1 || p >= i) {
        record_status(FAVOR_ERR_INVALID_ARG);
        return -1;
    }
    return p;
}

// w_r . x from global memory (one thread; 16-byte loads).
template <int D>
__device__ float dot_global(const void *W, const void *x, int bf16, int r, size_t x0) {
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    if (bf16) {
        const uint4 *w = (const uint4 *)((const uint16_t *)W + (size_t)r * D), *y = (const uint4 *)((const uint16_t *)x + x0);
#pragma unroll 4
        for (int i = 0; i < D / 8; ++i) {
            const uint4 a = __ldg(w + i), c = __ldg(y + i);
            const uint32_t u[4] = {a.x, a.y, a.z, a.w}, v[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[j] = fmaf(__uint_as_float(u[j] << 16), __uint_as_float(v[j] << 16), acc[j]);
                acc[j] = fmaf(__uint_as_float(u[j] & 0xFFFF0000u), __uint_as_float(v[j] & 0xFFFF0000u), acc[j]);
            }
        }
    } else {
        const float4 *w = (const float4 *)((const float *)W + (size_t)r * D), *y = (const float4 *)((const float *)x + x0);
#pragma unroll 4
        for (int i = 0; i < D / 4; ++i) {
            const float4 a = __ldg(w + i), c = __ldg(y + i);
            acc[0] = fmaf(a.x, c.x, acc[0]);
            acc[1] = fmaf(a.y, c.y, acc[1]);
            acc[2] = fmaf(a.z, c.z, acc[2]);
            acc[3] = fmaf(a.w, c.w, acc[3]);
        }
    }
    return (acc[0] + acc[1]) + (acc[2] + acc[3]);
}

// One output row in log space over its own visible terms (one warp; lanes over features, then over
// value columns): F = the row's largest exponent, weight_j = sum_r e^(w_r.q + u_r(k_j) - F). `par`
// holds the checked parents. Rare, so its projections are simply recomputed.
template <int D>
__device__ __noinline__ void tree_row_exact(const TreeParams &p, int bh, int i, const int *par) {
    const int lane = threadIdx.x & 31, nk = p.m >> 5;
    const size_t row0 = (size_t)bh * p.T * D;
    const float *S = p.state + (size_t)bh * ((size_t)D * p.m + 2 * p.m);
    const float *z = S + (size_t)D * p.m, *Dl = z + p.m;
    float uq[8], F = -INFINITY;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        uq[k] = k < nk ? dot_global<D>(p.W, p.q, p.bf16, lane + 32 * k, row0 + (size_t)i * D) : -INFINITY;
        if (k < nk && z[lane + 32 * k] != 0.f) F = fmaxf(F, uq[k] + Dl[lane + 32 * k]);
    }
    auto half_norm = [&](int j) {
        float s = 0.f;
        for (int c = lane; c < D; c += 32) {
            const float x = ld_elem(p.k, p.bf16, row0 + (size_t)j * D + c);
            s = fmaf(x, x, s);
        }
        return 0.5f * warp_sum(s);
    };
    for (int j = i; j >= 0; j = par[j]) {
        const float h = half_norm(j);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < nk)
                F = fmaxf(F, uq[k] + dot_global<D>(p.W, p.k, p.bf16, lane + 32 * k, row0 + (size_t)j * D) - h);
    }
    F = warp_max(F);
    float num[D / 32], den = 0.f;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) num[c] = 0.f;
    float wz = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int r = lane + 32 * k;
        uq[k] = k < nk ? uq[k] - F : -INFINITY;
        if (k < nk && z[r] != 0.f) wz = fmaf(expf(uq[k] + Dl[r]), z[r], wz);
    }
    den = warp_sum(wz);
    for (int c = 0; c < D; ++c) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int r = lane + 32 * k;
            if (k < nk && z[r] != 0.f) s = fmaf(expf(uq[k] + Dl[r]), S[(size_t)c * p.m + r], s);
        }
        s = warp_sum(s);
        if ((c & 31) == lane) num[c >> 5] = s;
    }
    for (int j = i; j >= 0; j = par[j]) {
        const float h = half_norm(j);
        float w = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < nk) w += expf(uq[k] + dot_global<D>(p.W, p.k, p.bf16, lane + 32 * k, row0 + (size_t)j * D) - h);
        w = warp_sum(w);
        den += w;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            const float x = ld_elem(p.v, p.bf16, row0 + (size_t)j * D + lane + 32 * c);
            num[c] = w == 0.f ? num[c] : fmaf(w, x, num[c]);
        }
    }
#pragma unroll
    for (int c = 0; c < D / 32; ++c) p.out[row0 + (size_t)i * D + lane + 32 * c] = num[c] / den;
}

// ------------------------------------------------------------------------------- CUDA-core kernel
//
// One CTA per (head, tile of TQ rows), 256 threads, fp32 throughout. Feature phases: thread = feature
// (W row streamed once per 16 tokens). Product phase: every column x over the features (the d state
// columns, z', and a_j of the tile's and earlier nodes) is met by all TQ rows at once: a warp's lanes
// hold b for their features and all rows in registers, read the column coalesced, and reduce the TQ
// sums by a halving exchange.

constexpr int kTreeThreads = 256;
constexpr int kTreeTok = 16;  // tokens projected together

template <int D>
struct TreeSmem {
    // floats: x tile, a [nk][m], b [TQ][m], y [TQ][D + 1 + T], s, s z, e [T], reductions
    __host__ __device__ static size_t floats(int TQ, int T, int m) {
        return (size_t)kTreeTok * D + (size_t)T * m + (size_t)TQ * m + (size_t)TQ * (D + 1 + T) + 2 * m + T + 8 * 16 + 16 +
               TQ * 2;
    }
    __host__ __device__ static size_t bytes(int TQ, int T, int m) { return floats(TQ, T, m) * 4 + (size_t)T * 4; }
};

// acc[t] = w_r . x_t for NT tokens held in shared memory as fp32 rows.
template <int D, int NT>
__device__ __forceinline__ void feature_dots(const void *W, int bf16, int r, const float *sX, float (&acc)[NT]) {
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = 0.f;
#pragma unroll 2
    for (int c = 0; c < D; c += 8) {
        float w[8];
        if (bf16) {
            const uint4 u = __ldg((const uint4 *)((const uint16_t *)W + (size_t)r * D + c));
            const uint32_t uu[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[2 * i] = __uint_as_float(uu[i] << 16);
                w[2 * i + 1] = __uint_as_float(uu[i] & 0xFFFF0000u);
            }
        } else {
            const float4 a = __ldg((const float4 *)((const float *)W + (size_t)r * D + c));
            const float4 b = __ldg((const float4 *)((const float *)W + (size_t)r * D + c + 4));
            w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const float4 x0 = *(const float4 *)(sX + t * D + c), x1 = *(const float4 *)(sX + t * D + c + 4);
            acc[t] = fmaf(w[0], x0.x, acc[t]);
            acc[t] = fmaf(w[1], x0.y, acc[t]);
            acc[t] = fmaf(w[2], x0.z, acc[t]);
            acc[t] = fmaf(w[3], x0.w, acc[t]);
            acc[t] = fmaf(w[4], x1.x, acc[t]);
            acc[t] = fmaf(w[5], x1.y, acc[t]);
            acc[t] = fmaf(w[6], x1.z, acc[t]);
            acc[t] = fmaf(w[7], x1.w, acc[t]);
        }
    }
}

// sU[f][t0 + g] = w_(f0 + f) . x_g for 16 MT of a warp's features and 8 tokens (x: this lane's token row
// g, NULL for none; g = lane / 4); returns |x_g|^2. As warp MMAs: bf16 products are exact, fp32 rows are
// hi + lo in tf32 (three products, 2^-22). K runs in the order in which 16-byte loads hand it out, the
// same for both operands, so that W's fragments are 64-byte runs.
template <int D, int LD, int MT, bool BF16>
__device__ __forceinline__ float warp_logits(const void *Wv, int m, int f0, const void *xv, float *sU, int t0, int lane) {
    const int g = lane >> 2, t = lane & 3;
    float sq = 0.f;
    if constexpr (BF16) {
        const uint16_t *W = (const uint16_t *)Wv, *x = (const uint16_t *)xv;
        uint4 xb[D / 32];
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
            xb[j] = x != nullptr ? __ldg((const uint4 *)(x + 32 * j + 8 * t)) : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t u[4] = {xb[j].x, xb[j].y, xb[j].z, xb[j].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float lo = __uint_as_float(u[i] << 16), hi = __uint_as_float(u[i] & 0xFFFF0000u);
                sq = fmaf(lo, lo, sq);
                sq = fmaf(hi, hi, sq);
            }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            if (f0 + 16 * mt < m) {
                const uint16_t *w = W + (size_t)(f0 + 16 * mt + g) * D + 8 * t;
                float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int j = 0; j < D / 32; ++j) {
                    const uint4 a = __ldg((const uint4 *)(w + 32 * j)), b = __ldg((const uint4 *)(w + 8 * D + 32 * j));
                    mma_bf16_16x8x16(d, a.x, b.x, a.y, b.y, xb[j].x, xb[j].y);
                    mma_bf16_16x8x16(d, a.z, b.z, a.w, b.w, xb[j].z, xb[j].w);
                }
                float *o = sU + (16 * mt + g) * LD + t0 + 2 * t;
                o[0] = d[0];
                o[1] = d[1];
                o[8 * LD] = d[2];
                o[8 * LD + 1] = d[3];
            }
        }
    } else {
        const float *W = (const float *)Wv, *x = (const float *)xv;
        float d[MT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) d[mt][0] = d[mt][1] = d[mt][2] = d[mt][3] = 0.f;
#pragma unroll 2
        for (int j = 0; j < D / 16; ++j) {
            const float4 b = x != nullptr ? __ldg((const float4 *)(x + 16 * j + 4 * t)) : make_float4(0.f, 0.f, 0.f, 0.f);
            sq += (b.x * b.x + b.y * b.y) + (b.z * b.z + b.w * b.w);
            uint32_t bh[4], bl[4];
            tf32_split(b.x, bh[0], bl[0]);
            tf32_split(b.y, bh[1], bl[1]);
            tf32_split(b.z, bh[2], bl[2]);
            tf32_split(b.w, bh[3], bl[3]);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                if (f0 + 16 * mt < m) {
                    const float *w = W + (size_t)(f0 + 16 * mt + g) * D + 16 * j + 4 * t;
                    const float4 a0 = __ldg((const float4 *)w), a1 = __ldg((const float4 *)(w + 8 * D));
                    const float a[2][4] = {{a0.x, a0.y, a0.z, a0.w}, {a1.x, a1.y, a1.z, a1.w}};
                    uint32_t ah[2][4], al[2][4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        tf32_split(a[0][i], ah[0][i], al[0][i]);
                        tf32_split(a[1][i], ah[1][i], al[1][i]);
                    }
#pragma unroll
                    for (int i = 0; i < 4; i += 2) {
                        mma_tf32_16x8x8(d[mt], al[0][i], al[1][i], al[0][i + 1], al[1][i + 1], bh[i], bh[i + 1]);
                        mma_tf32_16x8x8(d[mt], ah[0][i], ah[1][i], ah[0][i + 1], ah[1][i + 1], bl[i], bl[i + 1]);
                        mma_tf32_16x8x8(d[mt], ah[0][i], ah[1][i], ah[0][i + 1], ah[1][i + 1], bh[i], bh[i + 1]);
                    }
                }
            }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
            if (f0 + 16 * mt < m) {
                float *o = sU + (16 * mt + g) * LD + t0 + 2 * t;
                o[0] = d[mt][0];
                o[1] = d[mt][1];
                o[8 * LD] = d[mt][2];
                o[8 * LD + 1] = d[mt][3];
            }
    }
    sq += __shfl_xor_sync(0xffffffffu, sq, 1);
    sq += __shfl_xor_sync(0xffffffffu, sq, 2);
    return sq;
}

// Sums of TQ per-lane values over the warp: on return lane l holds in v[0] the sum of value
// l * TQ / 32 (TQ <= 32, a power of two).
template <int TQ>
__device__ __forceinline__ void halving_sum(float (&v)[TQ], int lane) {
    int o = 16;
#pragma unroll
    for (int n = TQ; n > 1; n >>= 1, o >>= 1) {
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const float send = up ? v[i] : v[n / 2 + i];
            const float keep = up ? v[n / 2 + i] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
    for (; o > 0; o >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
}

template <int D, int TQ>
__global__ void __launch_bounds__(kTreeThreads) k_decode_tree_rows(TreeParams p) {
    extern __shared__ __align__(16) float sm[];
    const int bh = blockIdx.x, b = bh / p.H, m = p.m, T = p.T;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nw = kTreeThreads / 32;
    const int n = tree_count(p.n_nodes, b, T);
    const int i0 = blockIdx.y * TQ;
    if (i0 >= n) return;
    const int rows = min(TQ, n - i0), nk = i0 + rows;  // ancestors come first: keys 0 .. nk-1
    float *sX = sm, *sA = sX + kTreeTok * D, *sB = sA + (size_t)T * m, *sY = sB + (size_t)TQ * m;
    const int ldy = D + 1 + T;
    float *sS = sY + (size_t)TQ * ldy, *sZ = sS + m, *sE = sZ + m, *sRed = sE + T, *sTop = sRed + 8 * 16;
    float *sC = sTop + 16;             // per row: e^(e_S - M), denominator
    int *sPar = (int *)(sC + TQ * 2);
    const size_t row0 = (size_t)bh * T * D;
    for (int i = tid; i < nk; i += kTreeThreads) sPar[i] = tree_parent(p.parents + (size_t)b * T, i);

    const float *S = p.state + (size_t)bh * ((size_t)D * m + 2 * m);
    const int r = tid;
    float zr = 0.f, Dr = 0.f, E = -INFINITY;
    if (r < m) {
        zr = S[(size_t)D * m + r];
        Dr = S[(size_t)D * m + m + r];
    }
    // key logits
    for (int j0 = 0; j0 < nk; j0 += kTreeTok) {
        const int nt = min(kTreeTok, nk - j0);
        __syncthreads();
        for (int i = tid; i < kTreeTok * D; i += kTreeThreads)
            sX[i] = i < nt * D ? ld_elem(p.k, p.bf16, row0 + (size_t)j0 * D + i) : 0.f;
        __syncthreads();
        for (int t = warp; t < nt; t += nw) {
            float s = 0.f;
            for (int c = lane; c < D; c += 32) s = fmaf(sX[t * D + c], sX[t * D + c], s);
            s = warp_sum(s);
            if (lane == 0) sE[j0 + t] = -0.5f * s;
        }
        if (r < m) {
            float acc[kTreeTok];
            feature_dots<D, kTreeTok>(p.W, p.bf16, r, sX, acc);
#pragma unroll
            for (int t = 0; t < kTreeTok; ++t)
                if (t < nt) {
                    sA[(size_t)(j0 + t) * m + r] = acc[t];
                    if (fabsf(acc[t]) < INFINITY) E = fmaxf(E, acc[t]);
                }
        }
    }
    if (E == -INFINITY) E = 0.f;  // no finite logit
    float ds = -INFINITY;
    if (r < m) {
        for (int j = 0; j < nk; ++j) sA[(size_t)j * m + r] = expf(sA[(size_t)j * m + r] - E);
        if (zr != 0.f) ds = Dr - E;
    }
    const float dw = warp_max(ds);
    if (lane == 0) sRed[warp] = dw;
    __syncthreads();
    float eS = sRed[0];
    for (int w = 1; w < nw; ++w) eS = fmaxf(eS, sRed[w]);
    if (r < m) {
        const float s = zr != 0.f ? expf(ds - eS) : 0.f;
        sS[r] = s;
        sZ[r] = s * zr;
    }
    // query features of the tile's rows
    for (int i = tid; i < TQ * D; i += kTreeThreads)
        sX[i] = i < rows * D ? ld_elem(p.q, p.bf16, row0 + (size_t)i0 * D + i) : 0.f;
    __syncthreads();
    float uq[TQ];
    if (r < m) {
        feature_dots<D, TQ>(p.W, p.bf16, r, sX, uq);
#pragma unroll
        for (int t = 0; t < TQ; ++t) uq[t] += E;
    } else {
#pragma unroll
        for (int t = 0; t < TQ; ++t) uq[t] = -INFINITY;
    }
#pragma unroll
    for (int t = 0; t < TQ; ++t) {
        const float mx = warp_max(uq[t]);
        if (lane == 0) sRed[warp * 16 + t] = mx;
    }
    __syncthreads();
    if (r < m) {
#pragma unroll
        for (int t = 0; t < TQ; ++t) {
            float f = sRed[t];
            for (int w = 1; w < nw; ++w) f = fmaxf(f, sRed[w * 16 + t]);
            sB[(size_t)t * m + r] = expf(uq[t] - f);
        }
    }
    __syncthreads();
    // products of every column over the features with all rows
    {
        const int kk = m >> 5;
        float breg[8][TQ];
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
            for (int t = 0; t < TQ; ++t) breg[k][t] = k < kk ? sB[(size_t)t * m + lane + 32 * k] : 0.f;
        // a column's entries; those of the next state column are asked for one column ahead
        auto state_col = [&](int col, float(&x)[8]) {
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = k < kk && col < D ? __ldg(S + (size_t)col * m + lane + 32 * k) : 0.f;
        };
        float ahead[8];
        state_col(warp, ahead);
        for (int col = warp; col < D + 1 + nk; col += nw) {
            float x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int f = lane + 32 * k;
                x[k] = k >= kk      ? 0.f
                       : col < D    ? ahead[k] * sS[f]
                       : col == D   ? sZ[f]
                                    : sA[(size_t)(col - D - 1) * m + f];
            }
            state_col(col + nw, ahead);
            float y[TQ];
#pragma unroll
            for (int t = 0; t < TQ; ++t) y[t] = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k)
#pragma unroll
                for (int t = 0; t < TQ; ++t) y[t] = fmaf(breg[k][t], x[k], y[t]);
            halving_sum<TQ>(y, lane);
            if (lane % (32 / TQ) == 0) sY[(size_t)(lane / (32 / TQ)) * ldy + col] = y[0];
        }
    }
    __syncthreads();
    // per row: the visible nodes' scales, the weights and the denominator
    for (int t = tid; t < rows; t += kTreeThreads) {
        float *y = sY + (size_t)t * ldy;
        float M = eS;
        for (int j = i0 + t; j >= 0; j = sPar[j]) M = fmaxf(M, sE[j]);
        const float cS = eS == -INFINITY ? 0.f : expf(eS - M);
        float den = cS == 0.f ? 0.f : cS * y[D];
        for (int j = i0 + t; j >= 0; j = sPar[j]) {
            const float w = expf(sE[j] - M) * y[D + 1 + j];
            y[D + 1 + j] = w;
            den += w;
        }
        sC[2 * t] = cS;
        sC[2 * t + 1] = den;
    }
    __syncthreads();
    for (int i = tid; i < rows * D; i += kTreeThreads) {
        const int t = i / D, c = i - t * D;
        const float *y = sY + (size_t)t * ldy;
        const float cS = sC[2 * t], den = sC[2 * t + 1];
        if (!(den >= kTreeDenMin)) continue;
        float num = cS == 0.f ? 0.f : cS * y[c];
        for (int j = i0 + t; j >= 0; j = sPar[j]) num = fmaf(y[D + 1 + j], ld_elem(p.v, p.bf16, row0 + (size_t)j * D + c), num);
        p.out[row0 + (size_t)(i0 + t) * D + c] = num / den;
    }
    for (int t = warp; t < rows; t += nw)
        if (!(sC[2 * t + 1] >= kTreeDenMin)) tree_row_exact<D>(p, bh, i0 + t, sPar);
}

// ---------------------------------------------------------------------------- few nodes (T <= 8)
//
// One CTA per (head, 64 value columns), one thread per feature, all nodes at once, fp32 throughout. The
// thread's 64 entries of S' are asked for before anything else and arrive under the projections; sums
// over features are halving exchanges inside each warp, then across warps through shared memory. Small
// trees are bound by the latency of that one chain: about 1 us for the loads and as much for the rest.

constexpr int kFewCols = 64;

// Sums of 64 per-lane values over the warp: on return lane l holds the sums of values 2 l, 2 l + 1.
__device__ __forceinline__ void halving_sum64(float (&v)[64], int lane) {
#pragma unroll
    for (int o = 16, n = 64; o > 0; o >>= 1, n >>= 1) {
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const float send = up ? v[i] : v[n / 2 + i];
            const float keep = up ? v[n / 2 + i] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
}

template <int D, int TT>
struct FewSmem {
    static constexpr int LD = kFewCols + TT + 1;  // a row's sums: value columns, keys, normaliser
    // floats: logits of keys and queries [m][17], values [TT][64], warps' sums [nw][TT][LD], sums [TT][LD], maxima, scales
    __host__ __device__ static size_t bytes(int m) {
        return 4 * ((size_t)m * 17 + TT * kFewCols + (size_t)(m / 32 + 1) * TT * LD + 8 * (TT + 1) + 4 * TT) + 8 * TT;
    }
};

template <int D, int TT>
__global__ void __launch_bounds__(256, 1) k_decode_tree_few(TreeParams p) {
    constexpr int LD = FewSmem<D, TT>::LD;
    extern __shared__ __align__(16) float sm[];
    const int bh = blockIdx.x, b = bh / p.H, m = p.m, T = p.T, c0 = blockIdx.y * kFewCols;
    const int r = threadIdx.x, warp = r >> 5, lane = r & 31, nw = m >> 5;
    const int n = tree_count(p.n_nodes, b, T);
    if (n == 0) return;
    float *sU = sm, *sV = sU + 17 * m, *sPart = sV + TT * kFewCols, *sY = sPart + (size_t)nw * TT * LD;
    float *sMax = sY + TT * LD, *sE = sMax + 8 * (TT + 1), *sC = sE + TT;  // sC: [TT][2], state's scale and denominator
    int *sPar = (int *)(sC + 3 * TT);
    uint32_t *sVis = (uint32_t *)(sPar + TT);
    const size_t row0 = (size_t)bh * T * D;

    const float *S = p.state + (size_t)bh * ((size_t)D * m + 2 * m);
    const float zr = S[(size_t)D * m + r], Dr = S[(size_t)D * m + m + r];
    float s[kFewCols];
#pragma unroll
    for (int c = 0; c < kFewCols; ++c) s[c] = __ldg(S + (size_t)(c0 + c) * m + r);
    for (int i = r; i < TT * kFewCols; i += m) {
        const int j = i / kFewCols, c = i % kFewCols;
        sV[i] = j < n ? ld_elem(p.v, p.bf16, row0 + (size_t)j * D + c0 + c) : 0.f;
    }
    if (r < n) sPar[r] = tree_parent(p.parents + (size_t)b * T, r);
    __syncthreads();
    if (r < n) {
        uint32_t x = 0;
        for (int j = r; j >= 0; j = sPar[j]) x |= 1u << j;
        sVis[r] = x;
    }
    {
        const size_t at = (row0 + (size_t)(lane >> 2) * D) * (p.bf16 ? 2 : 4);
        const void *xk = (lane >> 2) < n ? (const char *)p.k + at : nullptr, *xq = xk ? (const char *)p.q + at : nullptr;
        float sq;
        if (p.bf16) {
            sq = warp_logits<D, 17, 2, true>(p.W, m, 32 * warp, xk, sU + 32 * warp * 17, 0, lane);
            warp_logits<D, 17, 2, true>(p.W, m, 32 * warp, xq, sU + 32 * warp * 17, 8, lane);
        } else {
            sq = warp_logits<D, 17, 2, false>(p.W, m, 32 * warp, xk, sU + 32 * warp * 17, 0, lane);
            warp_logits<D, 17, 2, false>(p.W, m, 32 * warp, xq, sU + 32 * warp * 17, 8, lane);
        }
        if (warp == 0 && (lane & 3) == 0 && (lane >> 2) < TT) sE[lane >> 2] = -0.5f * sq;
    }
    __syncwarp();
    float u[2 * TT], E = -INFINITY;
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        u[t] = sU[r * 17 + t];
        u[TT + t] = sU[r * 17 + 8 + t];
    }
#pragma unroll
    for (int t = 0; t < TT; ++t)
        if (t < n && fabsf(u[t]) < INFINITY) E = fmaxf(E, u[t]);
    if (E == -INFINITY) E = 0.f;
    const float ds = zr != 0.f ? Dr - E : -INFINITY;
#pragma unroll
    for (int t = 0; t <= TT; ++t) {
        const float x = warp_max(t < TT ? u[TT + t] + E : ds);
        if (lane == 0) sMax[warp * (TT + 1) + t] = x;
    }
    __syncthreads();
    float eS = sMax[TT];
    for (int w = 1; w < nw; ++w) eS = fmaxf(eS, sMax[w * (TT + 1) + TT]);
    const float sr = zr != 0.f ? expf(ds - eS) : 0.f;
#pragma unroll
    for (int c = 0; c < kFewCols; ++c) s[c] = sr != 0.f ? s[c] * sr : 0.f;
#pragma unroll
    for (int t = 0; t < TT; ++t) u[t] = expf(u[t] - E);
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        if (t < n) {
            float f = sMax[t];
            for (int w = 1; w < nw; ++w) f = fmaxf(f, sMax[w * (TT + 1) + t]);
            const float bt = expf(u[TT + t] + E - f);
            float *part = sPart + (size_t)(warp * TT + t) * LD;
            float y[kFewCols], a[TT];
#pragma unroll
            for (int c = 0; c < kFewCols; ++c) y[c] = bt * s[c];
            halving_sum64(y, lane);
            part[2 * lane] = y[0];
            part[2 * lane + 1] = y[1];
#pragma unroll
            for (int j = 0; j < TT; ++j) a[j] = bt * u[j];
            halving_sum<TT>(a, lane);
            if (lane % (32 / TT) == 0) part[kFewCols + lane / (32 / TT)] = a[0];
            const float yz = warp_sum(bt * sr * zr);
            if (lane == 0) part[kFewCols + TT] = yz;
        }
    }
    __syncthreads();
    for (int i = r; i < n * LD; i += m) {
        float x = 0.f;
        for (int w = 0; w < nw; ++w) x += sPart[(size_t)w * TT * LD + i];
        sY[i] = x;
    }
    __syncthreads();
    if (r < n) {  // the visible nodes' weights and the denominator
        float *y = sY + r * LD, M = eS;
        for (uint32_t x = sVis[r]; x != 0; x &= x - 1) M = fmaxf(M, sE[__ffs(x) - 1]);
        const float cS = eS == -INFINITY ? 0.f : expf(eS - M);
        float den = cS == 0.f ? 0.f : cS * y[kFewCols + TT];
        for (uint32_t x = sVis[r]; x != 0; x &= x - 1) {
            const int j = __ffs(x) - 1;
            const float w = expf(sE[j] - M) * y[kFewCols + j];
            y[kFewCols + j] = w;
            den += w;
        }
        sC[2 * r] = cS;
        sC[2 * r + 1] = den;
    }
    __syncthreads();
    for (int i = r; i < n * kFewCols; i += m) {
        const int t = i / kFewCols, c = i % kFewCols;
        const float *y = sY + t * LD, cS = sC[2 * t], den = sC[2 * t + 1];
        if (!(den >= kTreeDenMin)) continue;
        float num = cS == 0.f ? 0.f : cS * y[c];
        for (uint32_t x = sVis[t]; x != 0; x &= x - 1) {
            const int j = __ffs(x) - 1;
            num = fmaf(y[kFewCols + j], sV[j * kFewCols + c], num);
        }
        p.out[row0 + (size_t)t * D + c0 + c] = num / den;
    }
    if (c0 == 0)
        for (int t = warp; t < n; t += nw)
            if (!(sC[2 * t + 1] >= kTreeDenMin)) tree_row_exact<D>(p, bh, t, sPar);
}

template <int D, int TT>
static cudaError_t launch_tree_few(const TreeParams &p, cudaStream_t st) {
    const size_t sm = FewSmem<D, TT>::bytes(p.m);
    if (sm > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(k_decode_tree_few<D, TT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm);
        if (e != cudaSuccess) return e;
    }
    k_decode_tree_few<D, TT><<<dim3(p.B * p.H, D / kFewCols), p.m, sm, st>>>(p);
    return cudaGetLastError();
}

template <int D, int TQ>
static cudaError_t launch_tree_rows(const TreeParams &p, cudaStream_t st) {
    const size_t sm = TreeSmem<D>::bytes(TQ, p.T, p.m);
    cudaError_t e = cudaFuncSetAttribute(k_decode_tree_rows<D, TQ>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm);
    if (e != cudaSuccess) return e;
    k_decode_tree_rows<D, TQ><<<dim3(p.B * p.H, (p.T + TQ - 1) / TQ), kTreeThreads, sm, st>>>(p);
    return cudaGetLastError();
}

template <int D>
static cudaError_t launch_decode_tree_d(const TreeParams &p, cudaStream_t st) {
    if (p.T == 1) return launch_tree_few<D, 1>(p, st);
    if (p.T <= 4) return launch_tree_few<D, 4>(p, st);
    if (p.T <= 8) return launch_tree_few<D, 8>(p, st);
    return launch_tree_rows<D, 16>(p, st);
}

cudaError_t launch_decode_tree(const TreeParams &p, int d, cudaStream_t st) {
    return d == 64 ? launch_decode_tree_d<64>(p, st) : launch_decode_tree_d<128>(p, st);
}

}  // namespace favor
