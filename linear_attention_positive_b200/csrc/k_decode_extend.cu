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

// ------------------------------------------------------------------------------- CUDA-core kernel
//
// One CTA per (head, run of tokens), one thread per feature with the feature's row of S' in
// registers; eight tokens at a time, so that W's row is streamed once per eight. With one run per
// head the state is read and written in place: for the few tokens of an accepted path that traffic,
// (m d + 2 m) * 8 bytes a head, is the bound. Longer inputs are split into runs whose partial states
// k_extend_combine adds.

constexpr int kExtTok = 8;

template <int D>
__global__ void __launch_bounds__(256) k_decode_extend_rows(ExtendParams p) {
    __shared__ __align__(16) float sK[kExtTok * D], sV[kExtTok * D];
    __shared__ float sN[kExtTok];
    __shared__ int sT[kExtTok];
    const int bh = blockIdx.y, b = bh / p.H, split = blockIdx.x, m = p.m, r = threadIdx.x;
    const int warp = r >> 5, lane = r & 31, nw = m >> 5;
    const int n = extend_count(p, b);
    const bool whole = p.n_split == 1;
    if (n == 0) return;  // the state stays as it is
    const size_t len = (size_t)D * m + 2 * m;
    float *S = whole ? p.state + (size_t)bh * len : p.part + ((size_t)bh * p.n_split + split) * len;
    float *z = S + (size_t)D * m, *Dl = z + m;
    const int t0 = split * p.tok_per_split, t1 = min(n, t0 + p.tok_per_split);
    if (t0 >= t1) {  // an empty run: nothing but its mark is read back
        z[r] = 0.f;
        return;
    }
    float s[D], zr = 0.f, Dr = -INFINITY;
    if (split == 0) {  // the first run starts from the carried state
        const float *S0 = p.state + (size_t)bh * len;
        zr = S0[(size_t)D * m + r];
        if (zr != 0.f) Dr = S0[(size_t)D * m + m + r];
#pragma unroll
        for (int c = 0; c < D; ++c) s[c] = zr != 0.f ? S0[(size_t)c * m + r] : 0.f;
    } else {
#pragma unroll
        for (int c = 0; c < D; ++c) s[c] = 0.f;
    }
    const size_t row0 = (size_t)bh * p.L;
    for (int t = t0; t < t1; t += kExtTok) {
        const int nt = min(kExtTok, t1 - t);
        __syncthreads();
        if (r < kExtTok) sT[r] = r < nt ? extend_token(p, b, t + r) : -1;
        __syncthreads();
        for (int i = r; i < kExtTok * D; i += m) {
            const int j = sT[i / D];
            const size_t at = (row0 + (j < 0 ? 0 : j)) * D + i % D;
            sK[i] = j < 0 ? 0.f : ld_elem(p.k, p.bf16, at);
            sV[i] = j < 0 ? 0.f : ld_elem(p.v, p.bf16, at);
        }
        __syncthreads();
        for (int i = warp; i < kExtTok; i += nw) {
            float x = 0.f;
            for (int c = lane; c < D; c += 32) x = fmaf(sK[i * D + c], sK[i * D + c], x);
            x = warp_sum(x);
            if (lane == 0) sN[i] = 0.5f * x;
        }
        float u[kExtTok];
        feature_dots<D, kExtTok>(p.W, p.bf16, r, sK, u);
        __syncthreads();
        float Dn = Dr;
#pragma unroll
        for (int i = 0; i < kExtTok; ++i) {
            u[i] = sT[i] < 0 ? -INFINITY : u[i] - sN[i];
            Dn = fmaxf(Dn, u[i]);
        }
        if (Dn > Dr) {
            const float sc = zr != 0.f ? expf(Dr - Dn) : 0.f;
            zr *= sc;
#pragma unroll
            for (int c = 0; c < D; ++c) s[c] *= sc;
            Dr = Dn;
        }
#pragma unroll
        for (int i = 0; i < kExtTok; ++i) {
            u[i] = u[i] == -INFINITY ? 0.f : expf(u[i] - Dr);
            zr += u[i];
        }
#pragma unroll
        for (int c = 0; c < D; c += 4) {
#pragma unroll
            for (int i = 0; i < kExtTok; ++i) {
                const float4 x = *(const float4 *)(sV + i * D + c);
                s[c] = fmaf(u[i], x.x, s[c]);
                s[c + 1] = fmaf(u[i], x.y, s[c + 1]);
                s[c + 2] = fmaf(u[i], x.z, s[c + 2]);
                s[c + 3] = fmaf(u[i], x.w, s[c + 3]);
            }
        }
    }
    if (zr == 0.f) {  // no token entered this feature
        if (!whole) z[r] = 0.f;
        return;
    }
#pragma unroll
    for (int c = 0; c < D; ++c) S[(size_t)c * m + r] = s[c];
    z[r] = zr;
    Dl[r] = Dr;
}

// ------------------------------------------------------------------------------- accepted paths
//
// Up to kExtPath tokens a head: one CTA per head, one thread per feature; all tokens' feature values
// are formed first (registers), then the state streams through, kExtCols value columns in flight at a
// time, each read, rescaled, added to and written once. Keeping S' out of the registers while the
// features are formed lets four CTAs share an SM, which is what its loads need to reach HBM's rate; the
// traffic, (m d + 2 m) * 8 bytes a head, is the bound.

constexpr int kExtPath = 16;
constexpr int kExtCols = 16;

template <int D>
__global__ void __launch_bounds__(256, 3) k_decode_extend_path(ExtendParams p) {
    __shared__ __align__(16) float sK[kExtPath * D], sV[kExtPath * D];
    __shared__ float sN[kExtPath];
    const int bh = blockIdx.x, b = bh / p.H, m = p.m, r = threadIdx.x, warp = r >> 5, lane = r & 31, nw = m >> 5;
    const int n = extend_count(p, b);
    if (n == 0) return;  // the state stays as it is
    float *S = p.state + (size_t)bh * ((size_t)D * m + 2 * m) + r;
    float *z = S + (size_t)D * m, *Dl = z + m;
    float zr = *z, Dr = *Dl, s[kExtCols];
#pragma unroll
    for (int c = 0; c < kExtCols; ++c) s[c] = S[(size_t)c * m];
    const size_t row0 = (size_t)bh * p.L;
    // a warp a token: gathered as fp32, half its squared norm with it (-1: not added)
    for (int t = warp; t < kExtPath; t += nw) {
        const int j = t < n ? extend_token(p, b, t) : -1;
        float x = 0.f;
        for (int c = lane; c < D; c += 32) {
            const float k = j < 0 ? 0.f : ld_elem(p.k, p.bf16, (row0 + j) * D + c);
            sK[t * D + c] = k;
            sV[t * D + c] = j < 0 ? 0.f : ld_elem(p.v, p.bf16, (row0 + j) * D + c);
            x = fmaf(k, k, x);
        }
        x = warp_sum(x);
        if (lane == 0) sN[t] = j < 0 ? -1.f : 0.5f * x;
    }
    __syncthreads();
    if (!(zr != 0.f)) Dr = -INFINITY;
    float u[kExtPath], Dn = Dr;
    {
        float v[8];
        feature_dots<D, 8>(p.W, p.bf16, r, sK, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = v[i], u[8 + i] = 0.f;
        if (n > 8) {
            feature_dots<D, 8>(p.W, p.bf16, r, sK + 8 * D, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) u[8 + i] = v[i];
        }
    }
#pragma unroll
    for (int i = 0; i < kExtPath; ++i) {
        u[i] = sN[i] < 0.f ? -INFINITY : u[i] - sN[i];
        Dn = fmaxf(Dn, u[i]);
    }
    const float keep = zr != 0.f ? expf(Dr - Dn) : 0.f;
    zr *= keep;
#pragma unroll
    for (int i = 0; i < kExtPath; ++i) {
        u[i] = u[i] == -INFINITY ? 0.f : expf(u[i] - Dn);
        zr += u[i];
    }
    if (zr != 0.f) {
        *z = zr;
        *Dl = Dn;
    }
#pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += kExtCols) {
        float x[kExtCols];
#pragma unroll
        for (int c = 0; c < kExtCols; ++c) {
            x[c] = keep != 0.f ? s[c] * keep : 0.f;
            if (c0 + kExtCols < D) s[c] = S[(size_t)(c0 + kExtCols + c) * m];
        }
#pragma unroll
        for (int i = 0; i < kExtPath; ++i) {
            if (i == 8 && n <= 8) break;
#pragma unroll
            for (int c = 0; c < kExtCols; c += 4) {
                const float4 v = *(const float4 *)(sV + i * D + c0 + c);
                ffma2(u[i], u[i], v.x, v.y, x[c], x[c + 1], x[c], x[c + 1]);
                ffma2(u[i], u[i], v.z, v.w, x[c + 2], x[c + 3], x[c + 2], x[c + 3]);
            }
        }
        if (zr != 0.f) {  // else no token entered this feature
#pragma unroll
            for (int c = 0; c < kExtCols; ++c) S[(size_t)(c0 + c) * m] = x[c];
        }
    }
}

// Adds the partial states of a head's runs (the first holds the carried state) into the state: one
// thread per feature, kCombCols value columns per CTA; the CTA of the first columns writes z' and D.
constexpr int kCombCols = 8;

__global__ void __launch_bounds__(256) k_extend_combine(ExtendParams p, int d) {
    const int bh = blockIdx.y, r = threadIdx.x, m = p.m, c0 = blockIdx.x * kCombCols;
    const size_t len = (size_t)d * m + 2 * m;
    if (extend_count(p, bh / p.H) == 0) return;
    const float *part = p.part + (size_t)bh * p.n_split * len + r;
    float *S = p.state + (size_t)bh * len + r;
    const size_t oz = (size_t)d * m, oD = oz + m;
    float D = -INFINITY;
    for (int s = 0; s < p.n_split; ++s)
        if (part[s * len + oz] != 0.f) D = fmaxf(D, part[s * len + oD]);
    float acc[kCombCols], z = 0.f;
#pragma unroll
    for (int c = 0; c < kCombCols; ++c) acc[c] = 0.f;
    for (int s = 0; s < p.n_split; ++s) {
        const float zs = part[s * len + oz];
        if (zs == 0.f) continue;
        const float w = expf(part[s * len + oD] - D);
        z = fmaf(w, zs, z);
#pragma unroll
        for (int c = 0; c < kCombCols; ++c) acc[c] = fmaf(w, part[s * len + (size_t)(c0 + c) * m], acc[c]);
    }
    if (z == 0.f) return;
#pragma unroll
    for (int c = 0; c < kCombCols; ++c) S[(size_t)(c0 + c) * m] = acc[c];
    if (c0 == 0) {
        S[oz] = z;
        S[oD] = D;
    }
}

cudaError_t launch_decode_extend(const ExtendParams &p, int d, cudaStream_t st) {
    const int BH = p.B * p.H;
    if (p.n_split == 1 && p.n_tok <= kExtPath) {
        if (d == 64)
            k_decode_extend_path<64><<<BH, p.m, 0, st>>>(p);
        else
            k_decode_extend_path<128><<<BH, p.m, 0, st>>>(p);
        return cudaGetLastError();
    }
    if (d == 64)
        k_decode_extend_rows<64><<<dim3(p.n_split, BH), p.m, 0, st>>>(p);
    else
        k_decode_extend_rows<128><<<dim3(p.n_split, BH), p.m, 0, st>>>(p);
    if (p.n_split > 1) k_extend_combine<<<dim3(d / kCombCols, BH), p.m, 0, st>>>(p, d);
    return cudaGetLastError();
}

}  // namespace favor
