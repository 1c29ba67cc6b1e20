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
// (tree_row_exact, tree_row_exact_bf16); the same path takes nothing from nodes outside J(i), so NaN or infinities there
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

// w_r . x from global memory in fp32 (one thread; 16-byte loads).
template <int D>
__device__ float dot_global(const void *W, const void *x, int r, size_t x0) {
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    const float4 *w = (const float4 *)((const float *)W + (size_t)r * D), *y = (const float4 *)((const float *)x + x0);
#pragma unroll 4
    for (int i = 0; i < D / 4; ++i) {
        const float4 a = __ldg(w + i), c = __ldg(y + i);
        acc[0] = fmaf(a.x, c.x, acc[0]);
        acc[1] = fmaf(a.y, c.y, acc[1]);
        acc[2] = fmaf(a.z, c.z, acc[2]);
        acc[3] = fmaf(a.w, c.w, acc[3]);
    }
    return (acc[0] + acc[1]) + (acc[2] + acc[3]);
}

// One output row in log space over its own visible terms, fp32 (one warp; lanes over features, then over
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
        uq[k] = k < nk ? dot_global<D>(p.W, p.q, lane + 32 * k, row0 + (size_t)i * D) : -INFINITY;
        if (k < nk && z[lane + 32 * k] != 0.f) F = fmaxf(F, uq[k] + Dl[lane + 32 * k]);
    }
    auto half_norm = [&](int j) {
        float s = 0.f;
        for (int c = lane; c < D; c += 32) {
            const float x = ld_elem(p.k, 0, row0 + (size_t)j * D + c);
            s = fmaf(x, x, s);
        }
        return 0.5f * warp_sum(s);
    };
    for (int j = i; j >= 0; j = par[j]) {
        const float h = half_norm(j);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < nk)
                F = fmaxf(F, uq[k] + dot_global<D>(p.W, p.k, lane + 32 * k, row0 + (size_t)j * D) - h);
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
            if (k < nk) w += expf(uq[k] + dot_global<D>(p.W, p.k, lane + 32 * k, row0 + (size_t)j * D) - h);
        w = warp_sum(w);
        den += w;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            const float x = ld_elem(p.v, 0, row0 + (size_t)j * D + lane + 32 * c);
            num[c] = w == 0.f ? num[c] : fmaf(w, x, num[c]);
        }
    }
#pragma unroll
    for (int c = 0; c < D / 32; ++c) p.out[row0 + (size_t)i * D + lane + 32 * c] = num[c] / den;
}

// The same for bf16 by warp MMAs (exact products), q and 7 visible nodes at a time, 64 features after
// another with a running F, so that W is read once for 7 nodes and little is held: a lane has features
// 16 f + 8 h + g of rows 2 t and 2 t + 1 (row 0: q), g = lane / 4, t = lane % 4. At m = 256 a row of some 25
// nodes adds 40 us to a call at d = 64 and 75 at d = 128, 20 and 35 where four warps share it (one node at a
// time, each lane reading its features' rows of W, twice: 170 and 560).
// `parts` warps may share a row: groups of nodes and of features in turn; each then leaves its num, den and F
// in part_out [D + 2] for tree_row_join.
template <int D>
__device__ __noinline__ void tree_row_exact_bf16(const TreeParams &p, int bh, int i, const int *par, int part = 0,
                                                 int parts = 1, float *part_out = nullptr) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, m = p.m;
    const size_t row0 = (size_t)bh * p.T * D;
    const float *S = p.state + (size_t)bh * ((size_t)D * m + 2 * m), *z = S + (size_t)D * m, *Dl = z + m;
    auto over_g = [](float x) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        return x;
    };
    float num[D / 32], den = 0.f, dz = 0.f, F = -INFINITY;  // dz: the state's part of the denominator, this lane's features
#pragma unroll
    for (int k = 0; k < D / 32; ++k) num[k] = 0.f;
    bool first = true;  // the state is taken along
    for (int j = i, group = 0; j >= 0 || first; ++group) {
        int mine = -1;
#pragma unroll
        for (int k = 1; k < 8; ++k) {
            if (k == g) mine = j;
            j = j >= 0 ? par[j] : -1;
        }
        if (group % parts != part) {
            if (j >= 0 || !first) continue;
            mine = -1;  // no nodes for this part, but its features of the state
        }
        const uint16_t *x = (const uint16_t *)(g == 0 ? p.q : p.k) + row0 + (size_t)(g == 0 ? i : max(mine, 0)) * D + 8 * t;
        uint4 xb[D / 32];
        float sq = 0.f, h[2], w[2] = {0.f, 0.f};
        bool use[2];
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
            xb[k] = g == 0 || mine >= 0 ? __ldg((const uint4 *)(x + 32 * k)) : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t u[4] = {xb[k].x, xb[k].y, xb[k].z, xb[k].w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float lo = __uint_as_float(u[q] << 16), hi = __uint_as_float(u[q] & 0xFFFF0000u);
                sq = fmaf(lo, lo, sq);
                sq = fmaf(hi, hi, sq);
            }
        }
        sq += __shfl_xor_sync(0xffffffffu, sq, 1);
        sq += __shfl_xor_sync(0xffffffffu, sq, 2);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            h[q] = 0.5f * __shfl_sync(0xffffffffu, sq, 4 * (2 * t + q));
            use[q] = __shfl_sync(0xffffffffu, mine, 4 * (2 * t + q)) >= 0;
        }
#pragma unroll 1
        for (int f0 = 0; f0 < m; f0 += 64) {
            const bool state = first && (f0 >> 6) % parts == part;
            float u[4][4], e[8], top = -INFINITY;
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                const int r = f0 + 16 * f + g;
#pragma unroll
                for (int q = 0; q < 4; ++q) u[f][q] = 0.f;
                if (f0 + 16 * f < m) {
                    const uint16_t *W = (const uint16_t *)p.W + (size_t)r * D + 8 * t;
#pragma unroll
                    for (int k = 0; k < D / 32; ++k) {
                        const uint4 a = __ldg((const uint4 *)(W + 32 * k)), b = __ldg((const uint4 *)(W + 8 * D + 32 * k));
                        mma_bf16_16x8x16(u[f], a.x, b.x, a.y, b.y, xb[k].x, xb[k].y);
                        mma_bf16_16x8x16(u[f], a.z, b.z, a.w, b.w, xb[k].z, xb[k].w);
                    }
                }
                const bool in = f0 + 16 * f < m;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const float uq = __shfl_sync(0xffffffffu, u[f][2 * q], lane & 28);
                    e[2 * f + q] = state && in && z[r + 8 * q] != 0.f ? uq + Dl[r + 8 * q] : -INFINITY;
                    u[f][2 * q] = in && use[0] ? uq + u[f][2 * q] - h[0] : -INFINITY;
                    u[f][2 * q + 1] = in && use[1] ? uq + u[f][2 * q + 1] - h[1] : -INFINITY;
                    top = fmax3(top, e[2 * f + q], fmaxf(u[f][2 * q], u[f][2 * q + 1]));
                }
            }
            top = fmaxf(F, warp_max(top));
            if (top > F) {
                const float keep = expf(F - top);  // (0 at first)
                F = top;
                den *= keep;
                dz *= keep;
                w[0] *= keep;
                w[1] *= keep;
#pragma unroll
                for (int k = 0; k < D / 32; ++k) num[k] *= keep;
            }
#pragma unroll
            for (int f = 0; f < 4; ++f)
#pragma unroll
                for (int q = 0; q < 4; ++q) w[q & 1] += use[q & 1] && f0 + 16 * f < m ? expf(u[f][q] - F) : 0.f;
            if (state) {
#pragma unroll
                for (int f = 0; f < 8; ++f) {
                    e[f] = e[f] == -INFINITY ? 0.f : expf(e[f] - F);
                    if (e[f] != 0.f) dz = fmaf(e[f], z[f0 + 8 * f + g], dz);
                }
#pragma unroll
                for (int k = 0; k < D / 32; ++k)
#pragma unroll 4
                    for (int c = 0; c < 8; ++c) {  // columns 32 k + 4 c + t
                        const float *at = S + (size_t)(32 * k + 4 * c + t) * m + f0 + g;
                        float y = 0.f;
#pragma unroll
                        for (int f = 0; f < 8; ++f)
                            if (e[f] != 0.f) y = fmaf(e[f], at[8 * f], y);
                        y = over_g(y);
                        if (c == g) num[k] += y;
                    }
            }
        }
        w[0] = over_g(w[0]);
        w[1] = over_g(w[1]);
        float v[7][D / 32];
#pragma unroll
        for (int k = 1; k < 8; ++k) {
            const int at = __shfl_sync(0xffffffffu, mine, 4 * k);
#pragma unroll
            for (int c = 0; c < D / 32; ++c) v[k - 1][c] = at >= 0 ? ld_elem(p.v, 1, row0 + (size_t)at * D + lane + 32 * c) : 0.f;
        }
#pragma unroll
        for (int k = 1; k < 8; ++k) {
            const float y = __shfl_sync(0xffffffffu, w[k & 1], k >> 1);  // 0 where there is no node
            den += y;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) num[c] = y == 0.f ? num[c] : fmaf(y, v[k - 1][c], num[c]);
        }
        first = false;
    }
    den += over_g(dz);
    if (parts > 1) {
#pragma unroll
        for (int c = 0; c < D / 32; ++c) part_out[lane + 32 * c] = num[c];
        if (lane == 0) part_out[D] = den;
        if (lane == 0) part_out[D + 1] = F;
        return;
    }
#pragma unroll
    for (int c = 0; c < D / 32; ++c) p.out[row0 + (size_t)i * D + lane + 32 * c] = num[c] / den;
}

// Row i from its parts (one warp).
template <int D>
__device__ __forceinline__ void tree_row_join(const TreeParams &p, int bh, int i, int parts, const float *part_out) {
    const int lane = threadIdx.x & 31;
    float F = -INFINITY, num[D / 32], den = 0.f;
    for (int k = 0; k < parts; ++k) F = fmaxf(F, part_out[k * (D + 2) + D + 1]);
#pragma unroll
    for (int c = 0; c < D / 32; ++c) num[c] = 0.f;
    for (int k = 0; k < parts; ++k) {
        const float *x = part_out + k * (D + 2);
        const float w = x[D + 1] == -INFINITY ? 1.f : expf(x[D + 1] - F);  // (nothing in it, or no number)
        den = fmaf(w, x[D], den);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) num[c] = fmaf(w, x[lane + 32 * c], num[c]);
    }
#pragma unroll
    for (int c = 0; c < D / 32; ++c) p.out[((size_t)bh * p.T + i) * D + lane + 32 * c] = num[c] / den;
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

// ---------------------------------------------------------------------------- few nodes (T <= 4)
//
// One CTA per (head, 64 value columns), one thread per feature, all nodes at once, fp32 throughout. The
// thread's 64 entries of S' are asked for before anything else and arrive under the projections; sums
// over features are halving exchanges inside each warp, then across warps through shared memory. Small
// trees are bound by the latency of that one chain: 5.5 us for one node in 8 heads at d = 64, m = 256 (22 with
// the state's columns loaded where they are used).

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
            if (!(sC[2 * t + 1] >= kTreeDenMin)) {
                if (p.bf16)
                    tree_row_exact_bf16<D>(p, bh, t, sPar);
                else
                    tree_row_exact<D>(p, bh, t, sPar);
            }
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

// ------------------------------------------------------------------------- rows on warp MMAs
//
// One CTA per (head, tile of 16 rows, 64 value columns), 256 threads. Projections as warp MMAs with W's
// fragments in registers; the products over the features, [16 rows x m] [m x (64 state columns + keys)],
// as tf32 warp MMAs with both sides hi + lo (three products, 2^-22: fp32's precision), a group of 8
// columns a warp. A warp's state columns are asked for before anything else. fp32 trees of any size,
// and bf16 ones too small for whole tiles, where the latency of this chain (five barriers) is the bound: 17 us
// for fp32 trees of up to 33 nodes in 64 heads (34 as sums on CUDA cores).

constexpr int kRowsThreads = 256;
constexpr int kRowsTile = 16;
constexpr int kRowsCols = 64;

struct RowsSmem {
    // floats: a [T][m + 16], b and b s [16][m + 16] each, values [T][64], sums [16][64 + T rounded up to 8],
    // per feature E, D - E, z', per node e, parents and visible sets
    __host__ __device__ static int ldy(int T) { return kRowsCols + (T + 7) / 8 * 8; }
    __host__ __device__ static size_t floats(int T, int m) {
        return (size_t)(T + 2 * kRowsTile) * (m + 16) + (size_t)T * kRowsCols + (size_t)kRowsTile * ldy(T) + 3 * m + T + 8 + 4 * kRowsTile;
    }
    __host__ __device__ static size_t bytes(int T, int m) { return 4 * (floats(T, m) + T + 4 * kRowsTile); }
};

// o[token][f0 + f] = w . x for 16 NF features of a warp (f0 and on, 128 apart) and its tokens, in groups of
// 8: nk rows of k, then nq of q, o's rows on from each other's. W's fragments stay in registers; the next
// group's rows are asked for one group ahead.
template <int D, bool BF16, int NF>
__device__ __forceinline__ void rows_logits(const void *Wv, int f0, const void *k, int nk, float *ok, const void *q, int nq,
                                            float *oq, int ld, int lane) {
    const int g = lane >> 2, t = lane & 3;
    constexpr int NJ = BF16 ? D / 32 : D / 16;
    constexpr size_t es = BF16 ? 2 : 4;
    uint4 w[NF][2][NJ];
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                w[f][h][j] = __ldg((const uint4 *)((const char *)Wv + ((size_t)(f0 + 128 * f + g + 8 * h) * D + (16 / es) * t) * es + 64 * j));
    const int gk = (nk + 7) / 8, gq = (nq + 7) / 8;
    uint4 next[NJ];
    auto ask = [&](int i) {
        const bool key = i < gk;
        const int row = 8 * (key ? i : i - gk) + g;
        const bool in = i < gk + gq && row < (key ? nk : nq);
        const char *x = (const char *)(key ? k : q) + ((size_t)row * D + (16 / es) * t) * es;
#pragma unroll
        for (int j = 0; j < NJ; ++j) next[j] = in ? __ldg((const uint4 *)(x + 64 * j)) : make_uint4(0u, 0u, 0u, 0u);
    };
    ask(0);
    for (int i = 0; i < gk + gq; ++i) {
        const bool key = i < gk;
        const int t0 = 8 * (key ? i : i - gk), n = key ? nk : nq;
        float *o = key ? ok : oq;
        uint4 xb[NJ];
#pragma unroll
        for (int j = 0; j < NJ; ++j) xb[j] = next[j];
        ask(i + 1);
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            float d[4] = {0.f, 0.f, 0.f, 0.f}, d1[4] = {0.f, 0.f, 0.f, 0.f}, d2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const uint4 wa = w[f][0][j], wb = w[f][1][j];
                if constexpr (BF16) {
                    mma_bf16_16x8x16(d, wa.x, wb.x, wa.y, wb.y, xb[j].x, xb[j].y);
                    mma_bf16_16x8x16(d1, wa.z, wb.z, wa.w, wb.w, xb[j].z, xb[j].w);
                } else {
                    const uint32_t xs[4] = {xb[j].x, xb[j].y, xb[j].z, xb[j].w}, a0[4] = {wa.x, wa.y, wa.z, wa.w},
                                   a1[4] = {wb.x, wb.y, wb.z, wb.w};
                    uint32_t bh[4], bl[4], ah[2][4], al[2][4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        tf32_split(__uint_as_float(xs[e]), bh[e], bl[e]);
                        tf32_split(__uint_as_float(a0[e]), ah[0][e], al[0][e]);
                        tf32_split(__uint_as_float(a1[e]), ah[1][e], al[1][e]);
                    }
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        mma_tf32_16x8x8(d1, al[0][e], al[1][e], al[0][e + 1], al[1][e + 1], bh[e], bh[e + 1]);
                        mma_tf32_16x8x8(d2, ah[0][e], ah[1][e], ah[0][e + 1], ah[1][e + 1], bl[e], bl[e + 1]);
                        mma_tf32_16x8x8(d, ah[0][e], ah[1][e], ah[0][e + 1], ah[1][e + 1], bh[e], bh[e + 1]);
                    }
                }
            }
            float *at = o + (size_t)(t0 + 2 * t) * ld + f0 + 128 * f + g;
            if (t0 + 2 * t < n) {
                at[0] = d[0] + (d1[0] + d2[0]);
                at[8] = d[2] + (d1[2] + d2[2]);
            }
            if (t0 + 2 * t + 1 < n) {
                at[ld] = d[1] + (d1[1] + d2[1]);
                at[ld + 8] = d[3] + (d1[3] + d2[3]);
            }
        }
    }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kRowsThreads, 1) k_decode_tree_rows(TreeParams p) {
    extern __shared__ __align__(16) float sm[];
    const int bh = blockIdx.x, b = bh / p.H, m = p.m, T = p.T, i0 = blockIdx.y * kRowsTile, c0 = blockIdx.z * kRowsCols;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    constexpr int nw = kRowsThreads / 32;
    const int n = tree_count(p.n_nodes, b, T);
    if (i0 >= n) return;
    const int rows = min(kRowsTile, n - i0), nk = i0 + rows;  // ancestors come first: keys 0 .. nk-1
    const int ld = m + 16, ldy = RowsSmem::ldy(T);
    float *sA = sm, *sB = sA + (size_t)T * ld, *sBs = sB + kRowsTile * ld, *sV = sBs + kRowsTile * ld;
    float *sY = sV + (size_t)T * kRowsCols, *sEr = sY + (size_t)kRowsTile * ldy, *sDs = sEr + m, *sZ = sDs + m, *sE = sZ + m;
    float *sTop = sE + T, *sC = sTop + 8;  // warps' maxima; [16][4] y, state's scale, denominator
    int *sPar = (int *)(sC + 4 * kRowsTile);
    uint32_t *sVis = (uint32_t *)(sPar + T);  // [16][4]
    const size_t es = BF16 ? 2 : 4, row0 = (size_t)bh * T * D;

    // this warp's 8 state columns, as fragments
    const float *S = p.state + (size_t)bh * ((size_t)D * m + 2 * m);
    const float *col = S + (size_t)(c0 + 8 * warp + g) * m + 4 * t;
    float4 sf[16];
#pragma unroll
    for (int j = 0; j < 16; ++j)
        if (16 * j < m) sf[j] = __ldg((const float4 *)(col + 16 * j));
    float zr = 0.f, Dr = 0.f;
    if (tid < m) {
        zr = S[(size_t)D * m + tid];
        Dr = S[(size_t)D * m + m + tid];
    }
    for (int i = tid; i < nk; i += kRowsThreads) sPar[i] = tree_parent(p.parents + (size_t)b * T, i);
    for (int i = tid; i < nk * kRowsCols; i += kRowsThreads)
        sV[i] = ld_elem(p.v, BF16, row0 + (size_t)(i / kRowsCols) * D + c0 + i % kRowsCols);
    {
        const void *k = (const char *)p.k + row0 * es, *q = (const char *)p.q + (row0 + (size_t)i0 * D) * es;
        const int f = 16 * warp;
        if (f + 128 < m && (BF16 || D == 64)) {
            rows_logits<D, BF16, (BF16 || D == 64) ? 2 : 1>(p.W, f, k, nk, sA, q, rows, sB, ld, lane);
        } else {
            for (int f1 = f; f1 < m; f1 += 128) rows_logits<D, BF16, 1>(p.W, f1, k, nk, sA, q, rows, sB, ld, lane);
        }
    }
    for (int j = warp; j < nk; j += nw) {
        float x = 0.f;
#pragma unroll
        for (int c = lane; c < D; c += 32) {
            const float k = ld_elem(p.k, BF16, row0 + (size_t)j * D + c);
            x = fmaf(k, k, x);
        }
        x = warp_sum(x);
        if (lane == 0) sE[j] = -0.5f * x;
    }
    __syncthreads();
    // a: a feature a thread
    float ds = -INFINITY;
    if (tid < m) {
        float E = -INFINITY;
        for (int j = 0; j < nk; ++j) {
            const float x = sA[(size_t)j * ld + tid];
            if (fabsf(x) < INFINITY) E = fmaxf(E, x);
        }
        if (E == -INFINITY) E = 0.f;  // no finite logit
#pragma unroll 4
        for (int j = 0; j < nk; ++j) sA[(size_t)j * ld + tid] = expf(sA[(size_t)j * ld + tid] - E);
        if (zr != 0.f) ds = Dr - E;
        sEr[tid] = E;
        sDs[tid] = ds;
        sZ[tid] = zr;
    }
    if (tid >= kRowsThreads - 32 && lane < rows) {  // the rows' visible sets
        uint32_t x[4] = {0u, 0u, 0u, 0u};
        for (int j = i0 + lane; j >= 0; j = sPar[j]) {
#pragma unroll
            for (int w = 0; w < 4; ++w) x[w] |= (j >> 5) == w ? 1u << (j & 31) : 0u;
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) sVis[4 * lane + w] = x[w];
    }
    const float dw = warp_max(ds);
    if (lane == 0) sTop[warp] = dw;
    __syncthreads();
    float eS = sTop[0];
#pragma unroll
    for (int w = 1; w < nw; ++w) eS = fmaxf(eS, sTop[w]);
    // b and b s: a warp a row
    for (int i = warp; i < kRowsTile; i += nw) {
        float u[8], f = -INFINITY, y = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int r = lane + 32 * k;
            u[k] = r < m && i < rows ? sB[i * ld + r] + sEr[r] : -INFINITY;
            f = fmaxf(f, u[k]);
        }
        f = warp_max(f);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int r = lane + 32 * k;
            if (r < m) {
                const float x = i < rows ? expf(u[k] - f) : 0.f;
                const float s = sZ[r] != 0.f ? expf(sDs[r] - eS) : 0.f;
                sB[i * ld + r] = x;
                sBs[i * ld + r] = x * s;
                y = fmaf(x * s, sZ[r], y);
            }
        }
        y = warp_sum(y);
        if (lane == 0) sC[4 * i] = y;
    }
    __syncthreads();
    // products over the features, 8 columns a warp: the state's, then the keys'
    for (int nt = warp; nt < nw + (nk + 7) / 8; nt += nw) {
        const bool state = nt < nw;
        const int j0 = 8 * (nt - nw);
        const float *A = (state ? sBs : sB) + g * ld + 4 * t, *B = sA + (size_t)(j0 + g) * ld + 4 * t;
        const bool in = !state && j0 + g < nk;
        float d[4] = {0.f, 0.f, 0.f, 0.f}, d1[4] = {0.f, 0.f, 0.f, 0.f}, d2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            if (16 * j < m) {
                const float4 a0 = *(const float4 *)(A + 16 * j), a1 = *(const float4 *)(A + 8 * ld + 16 * j);
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                if (state)
                    x = sf[j];
                else if (in)
                    x = *(const float4 *)(B + 16 * j);
                const float xs[4] = {x.x, x.y, x.z, x.w}, as[2][4] = {{a0.x, a0.y, a0.z, a0.w}, {a1.x, a1.y, a1.z, a1.w}};
                uint32_t bh[4], bl[4], ah[2][4], al[2][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    tf32_split(xs[i], bh[i], bl[i]);
                    tf32_split(as[0][i], ah[0][i], al[0][i]);
                    tf32_split(as[1][i], ah[1][i], al[1][i]);
                }
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                    mma_tf32_16x8x8(d1, al[0][i], al[1][i], al[0][i + 1], al[1][i + 1], bh[i], bh[i + 1]);
                    mma_tf32_16x8x8(d2, ah[0][i], ah[1][i], ah[0][i + 1], ah[1][i + 1], bl[i], bl[i + 1]);
                    mma_tf32_16x8x8(d, ah[0][i], ah[1][i], ah[0][i + 1], ah[1][i + 1], bh[i], bh[i + 1]);
                }
            }
        }
        float *y = sY + (size_t)g * ldy + 8 * nt + 2 * t;
        y[0] = d[0] + (d1[0] + d2[0]);
        y[1] = d[1] + (d1[1] + d2[1]);
        y[8 * ldy] = d[2] + (d1[2] + d2[2]);
        y[8 * ldy + 1] = d[3] + (d1[3] + d2[3]);
    }
    __syncthreads();
    // per row: the visible nodes' scales, the weights and the denominator
    for (int i = warp; i < rows; i += nw) {
        float M = eS, w[4], den = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            w[k] = (sVis[4 * i + k] >> lane) & 1u ? sE[32 * k + lane] : -INFINITY;
            M = fmaxf(M, w[k]);
        }
        M = warp_max(M);
        const float cS = eS == -INFINITY ? 0.f : expf(eS - M);
        float *y = sY + (size_t)i * ldy + kRowsCols;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if ((sVis[4 * i + k] >> lane) & 1u) {
                const float x = expf(w[k] - M) * y[32 * k + lane];
                y[32 * k + lane] = x;
                den += x;
            }
        den = warp_sum(den);
        if (lane == 0) {
            sC[4 * i + 1] = cS;
            sC[4 * i + 2] = cS == 0.f ? den : fmaf(cS, sC[4 * i], den);
        }
    }
    __syncthreads();
    for (int i = tid; i < rows * kRowsCols; i += kRowsThreads) {
        const int r = i / kRowsCols, c = i % kRowsCols;
        const float *y = sY + (size_t)r * ldy, cS = sC[4 * r + 1], den = sC[4 * r + 2];
        if (!(den >= kTreeDenMin)) continue;
        float num = cS == 0.f ? 0.f : cS * y[c];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            for (uint32_t x = sVis[4 * r + k]; x != 0; x &= x - 1) {
                const int j = 32 * k + __ffs(x) - 1;
                num = fmaf(y[kRowsCols + j], sV[j * kRowsCols + c], num);
            }
        p.out[row0 + (size_t)(i0 + r) * D + c0 + c] = num / den;
    }
    if (c0 == 0)
        for (int i = warp; i < rows; i += nw)
            if (!(sC[4 * i + 2] >= kTreeDenMin)) {
                if constexpr (BF16)
                    tree_row_exact_bf16<D>(p, bh, i0 + i, sPar);
                else
                    tree_row_exact<D>(p, bh, i0 + i, sPar);
            }
}

template <int D, bool BF16>
static cudaError_t launch_tree_rows(const TreeParams &p, cudaStream_t st) {
    const size_t sm = RowsSmem::bytes(p.T, p.m);
    const cudaError_t e = cudaFuncSetAttribute(k_decode_tree_rows<D, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm);
    if (e != cudaSuccess) return e;
    const dim3 grid(p.B * p.H, (p.T + kRowsTile - 1) / kRowsTile, D / kRowsCols);
    k_decode_tree_rows<D, BF16><<<grid, kRowsThreads, sm, st>>>(p);
    return cudaGetLastError();
}

template <int D>
static cudaError_t launch_decode_tree_d(const TreeParams &p, cudaStream_t st) {
    if (p.T == 1) return launch_tree_few<D, 1>(p, st);
    if (p.T <= 4) return launch_tree_few<D, 4>(p, st);
    return p.bf16 ? launch_tree_rows<D, true>(p, st) : launch_tree_rows<D, false>(p, st);
}

cudaError_t launch_decode_tree(const TreeParams &p, int d, cudaStream_t st) {
    return d == 64 ? launch_decode_tree_d<64>(p, st) : launch_decode_tree_d<128>(p, st);
}

}  // namespace favor
