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
    if (t0 >= t1) return;  // an empty run
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
    if (zr == 0.f && whole) return;  // no token entered this feature
#pragma unroll
    for (int c = 0; c < D; ++c) S[(size_t)c * m + r] = s[c];
    z[r] = zr;
    Dl[r] = Dr;
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

cudaError_t launch_decode_extend(const ExtendParams &p, int d, cudaStream_t st) {
    const int BH = p.B * p.H;
    if (p.n_tok <= kExtPath) return d == 64 ? launch_extend_path<64>(p, st) : launch_extend_path<128>(p, st);
    if (d == 64)
        k_decode_extend_rows<64><<<dim3(p.n_split, BH), p.m, 0, st>>>(p);
    else
        k_decode_extend_rows<128><<<dim3(p.n_split, BH), p.m, 0, st>>>(p);
    if (p.n_split > 1) k_extend_combine<<<dim3(d / kCombCols, BH), p.m, 0, st>>>(p, d);
    return cudaGetLastError();
}

}  // namespace favor
