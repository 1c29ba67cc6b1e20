// favor_decode_extend on tensor cores: bf16 tokens in order (no index), long enough to fill tiles.
//
// One CTA per (run of 128-token tiles, half of 128 features, head), two CTAs an SM, so that one CTA's
// MMAs and loads run under the other's exponentials. Per tile:
//   P^T = W_h K^T - |k|^2/2    tcgen05 (M = 128 features, N = 128 tokens), bf16 operands (exact
//                              products); the norm enters as a K = 16 step of three bf16 parts per key
//                              against ones columns of W (-inf for a key past the sequence's count);
//   phi' = 2^(P log2e - D_r)   one thread per feature; D_r, an integer, is set so that the first
//                              tile's largest exponent lands in (7, 8] and raised whenever a tile's
//                              passes 15 (fp16 holds 2^t below 2^16);
//   acc = phi'^T V'            tcgen05 (M = 128, N = d, K = 128), fp16 operands: phi' = hi + lo, two fp16
//                              values (22 bits), A from TMEM where they replace P chunk by chunk;
//                              V' = V 2^-b, exact in fp16 but for entries 2^-22 of the tile's largest;
//   S_r += 2^b acc             in fp32 registers, tile by tile: the tensor core's own accumulation
//                              truncates, and over a long run that bias would reach 1e-5.
// A single fp16 phi' would cost 1e-4 relative in S (the roundings do not average out against values of
// both signs); with hi + lo the state has fp32 precision and the MMA work is 1.5 times the least.
//
// Bound: 2^t on the MUFU (16 a cycle and SM): B H L m of them; next the tensor work, 6 L m d a head.
//
// Warps 0-3: exponentials, z_r, and value columns 64.. of S for d = 128. Warps 4-7: |k|^2 and norms'
// extension, V -> fp16, value columns 0..63 of S. Warp 8: TMA and MMA issue.

#include "common.cuh"

namespace favor {

template <int D_>
struct ExtTc {
    static constexpr int D = D_, NB = D / 64;
    static constexpr int NS = D == 64 ? 2 : 1;  // K and V stages each (227 KB for two CTAs)
    static constexpr uint32_t BLK = kTile * 128, KT = NB * BLK;
    static constexpr int THREADS = 288;
    static constexpr uint32_t T_P = 0, T_ACC = 128;  // TMEM columns
    static constexpr size_t OFF_K = KT, OFF_V = OFF_K + NS * KT, OFF_KX = OFF_V + NS * KT, OFF_WX = OFF_KX + NS * 4096,
                            OFF_D = OFF_WX + 4096, OFF_F = OFF_D + 2 * 128 * 4, OFF_MISC = OFF_F + 128 * 8,
                            OFF_BAR = OFF_MISC + 64, BYTES = OFF_BAR + 256 + 1024;
};

template <int D>
__global__ void __launch_bounds__(ExtTc<D>::THREADS, 2)
k_decode_extend_tc(const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                   const __grid_constant__ CUtensorMap mapW, ExtendParams p) {
    using C = ExtTc<D>;
    constexpr int NS = C::NS, NB = C::NB;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t *sW = smem, *sK = smem + C::OFF_K, *sV = smem + C::OFF_V, *sKx = smem + C::OFF_KX, *sWx = smem + C::OFF_WX;
    float *sD = (float *)(smem + C::OFF_D);      // [2 tile parities][128]: D_r of the tile
    float2 *sF = (float2 *)(smem + C::OFF_F);    // [128]: final factors of the run's and the old S'
    int *sShift = (int *)(smem + C::OFF_MISC);   // [4]: b of tile g
    uint32_t *sRed = (uint32_t *)(sShift + 4);   // [2][4]
    uint64_t *bars = (uint64_t *)(smem + C::OFF_BAR);
    uint64_t *w_full = bars, *k_full = bars + 1, *v_full = k_full + NS, *k_conv = v_full + NS, *v_conv = k_conv + NS;
    uint64_t *p_full = v_conv + NS, *phi_full = p_full + 1, *s_full = phi_full + 4, *acc_free = s_full + 1;
    uint64_t *d_full = acc_free + 1, *v_max = d_full + 2, *drain = v_max + 1;
    uint32_t *tmem_slot = (uint32_t *)(drain + 1);
    volatile int *abort_flag = (volatile int *)(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = blockIdx.x, half = blockIdx.y, bh = blockIdx.z;
    const int count = extend_count(p, bh / p.H);
    if (count == 0) return;  // the state stays as it is
    const int t0 = split * p.tok_per_split / kTile;  // tok_per_split is a multiple of the tile
    const int t1 = min((count - 1) / kTile + 1, t0 + p.tok_per_split / kTile);
    const int n = t1 - t0, m = p.m;
    const size_t len = (size_t)D * m + 2 * m;
    const bool whole = p.n_split == 1;
    float *dst = whole ? p.state + (size_t)bh * len : p.part + ((size_t)bh * p.n_split + split) * len;
    if (n <= 0) {  // an empty run: nothing but its mark is read back
        const int r = half * 128 + threadIdx.x;
        if (threadIdx.x < 128 && r < m) dst[(size_t)D * m + r] = 0.f;
        return;
    }

    if (threadIdx.x == 0) {
        mbar_init(w_full, 1);
        for (int s = 0; s < NS; ++s) {
            mbar_init(&k_full[s], 1);
            mbar_init(&v_full[s], 1);
            mbar_init(&k_conv[s], 128);
            mbar_init(&v_conv[s], 128);
        }
        mbar_init(p_full, 1);
        for (int c = 0; c < 4; ++c) mbar_init(&phi_full[c], 128);
        mbar_init(s_full, 1);
        mbar_init(acc_free, D == 64 ? 128 : 256);
        mbar_init(&d_full[0], 128);
        mbar_init(&d_full[1], 128);
        mbar_init(v_max, 128);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 8) {
        tmem_alloc(tmem_slot, 256);
        tmem_relinquish();
    }
    // extension rows (interleaved core matrices): W's three ones columns; the keys' second half is zero
    for (int i = threadIdx.x; i < 256; i += C::THREADS) {
        const int r = i >> 1, kc = i & 1;
        *(uint4 *)(sWx + (r >> 3) * 256 + kc * 128 + (r & 7) * 16) =
            kc == 0 ? make_uint4(0x3F803F80u, 0x00003F80u, 0u, 0u) : make_uint4(0u, 0u, 0u, 0u);
    }
    for (int i = threadIdx.x; i < NS * 128; i += C::THREADS)
        *(uint4 *)(sKx + (i >> 7) * 4096 + ((i & 127) >> 3) * 256 + 128 + (i & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 8) {
        auto load = [&](const CUtensorMap *map, uint8_t *buf, uint64_t *bar, int g) {
            if (elect_one()) {
                mbar_arrive_expect_tx(&bar[g % NS], C::KT);
                for (int nb = 0; nb < NB; ++nb)
                    tma_load_3d(buf + (size_t)(g % NS) * C::KT + nb * C::BLK, map, &bar[g % NS], 64 * nb, (t0 + g) * kTile, bh);
            }
            __syncwarp();
        };
        if (elect_one()) {
            mbar_arrive_expect_tx(w_full, C::KT);
            for (int nb = 0; nb < NB; ++nb) tma_load_2d(sW + nb * C::BLK, &mapW, w_full, 64 * nb, half * 128);
        }
        __syncwarp();
        int nk = 0, nv = 0;  // K and V tiles asked for
        for (; nk < min(NS, n); ++nk) load(&mapK, sK, k_full, nk);
        for (; nv < min(NS, n); ++nv) load(&mapV, sV, v_full, nv);
        const uint32_t idesc_p = make_idesc(128, 128, kFmtBF16, 0, 0), idesc_s = make_idesc(128, D, kFmtF16, 0, 1);
        const uint64_t dW = make_sdesc(smem_u32(sW), 16, 1024), dK = make_sdesc(smem_u32(sK), 16, 1024);
        const uint64_t dV = make_sdesc(smem_u32(sV), C::BLK, 1024);
        const uint64_t dWx = make_sdesc_interleaved(smem_u32(sWx), 128, 256);
        const uint64_t dKx = make_sdesc_interleaved(smem_u32(sKx), 128, 256);
        bool ok = mbar_wait_all(w_full, 0, abort_flag);
        for (int g = 0; ok && g < n; ++g) {
            const int s = g % NS;
            const uint32_t ph = (g / NS) & 1;
            // P's columns still hold phi'(g - 1) until the state MMA of tile g - 1 has read them
            if (g > 0) ok = mbar_wait_all(s_full, (g - 1) & 1, abort_flag);
            if (!ok) break;
            if (g > 0 && nv < n) load(&mapV, sV, v_full, nv++);
            ok = mbar_wait_all(&k_full[s], ph, abort_flag) && mbar_wait_all(&k_conv[s], ph, abort_flag);
            if (!ok) break;
            tc_fence_after();
            for (int nb = 0; nb < NB; ++nb)
                mma_ss_x4_w(tmem + C::T_P, dW + nb * (C::BLK / 16), dK + s * (C::KT / 16) + nb * (C::BLK / 16), idesc_p,
                            nb > 0, 2, 2);
            mma_f16_ss_w(tmem + C::T_P, dWx, dKx + s * (4096 / 16), idesc_p, 1u);
            mma_commit_w(p_full);
            ok = mbar_wait_all(p_full, g & 1, abort_flag);
            if (!ok) break;
            if (nk < n) load(&mapK, sK, k_full, nk++);
            ok = mbar_wait_all(&v_full[s], ph, abort_flag) && mbar_wait_all(&v_conv[s], ph, abort_flag);
            if (ok && g > 0) ok = mbar_wait_all(acc_free, (g - 1) & 1, abort_flag);
            const uint64_t dVs = dV + s * (C::KT / 16);
            for (int c = 0; ok && c < 4; ++c) {
                ok = mbar_wait_all(&phi_full[c], g & 1, abort_flag);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint64_t vd = dVs + (uint32_t)(32 * c + 16 * k) * 128 / 16;
                    mma_f16_ts_w(tmem + C::T_ACC, tmem + C::T_P + 32 * c + 8 * k, vd, idesc_s, c + k > 0);
                    mma_f16_ts_w(tmem + C::T_ACC, tmem + C::T_P + 32 * c + 16 + 8 * k, vd, idesc_s, 1u);
                }
            }
            if (ok) mma_commit_w(s_full);
        }
        // nothing of this CTA is in flight when it frees its memory
        mma_commit_w(drain);
        volatile int no_abort = 0;
        mbar_wait_all(drain, 0, &no_abort);
        mbar_wait_all(w_full, 0, &no_abort);
        for (int g = max(nk - NS, 0); g < nk; ++g) mbar_wait_all(&k_full[g % NS], (g / NS) & 1, &no_abort);
        for (int g = max(nv - NS, 0); g < nv; ++g) mbar_wait_all(&v_full[g % NS], (g / NS) & 1, &no_abort);
    } else {
        const int row = (warp & 3) * 32 + lane, r = half * 128 + row;
        const uint32_t tL = tmem + (((uint32_t)(warp & 3) * 32u) << 16);
        const float *old = p.state + (size_t)bh * len;
        constexpr int SC = 64;  // value columns of S a thread keeps
        float S[SC];
        float Dreg = 0.f;  // the units of S: 2^D
        // S <- S 2^(Dreg - D(g)) + 2^b acc, for columns c0 .. c0 + 63
        auto flush = [&](int g, int c0) {
            const float Dg = sD[(g & 1) * 128 + row];
            const float keep = exp2f(fminf(Dreg - Dg, 0.f));
            Dreg = Dg;
            const float up = __uint_as_float((uint32_t)(127 + sShift[g & 3]) << 23);
            float v[16];
#pragma unroll
            for (int q = 0; q < SC; q += 16) {
                tmem_ld16(tL + C::T_ACC + c0 + q, v);
#pragma unroll
                for (int c = 0; c < 16; c += 2) {
                    float a, b;
                    ffma2(v[c], v[c + 1], up, up, 0.f, 0.f, a, b);
                    ffma2(S[q + c], S[q + c + 1], keep, keep, a, b, S[q + c], S[q + c + 1]);
                }
            }
            tc_fence_before();
            mbar_arrive(acc_free);
        };
        // the run's S' columns c0 .. c0 + 63 in the state's units, joined with the carried ones
        auto finish = [&](int c0) {
            const float2 f = sF[row];
            if (r >= m || (f.x == 0.f && f.y == 0.f)) return;
#pragma unroll
            for (int c = 0; c < SC; ++c) {
                const size_t at = (size_t)(c0 + c) * m + r;
                float x = S[c] * f.x;
                if (f.y != 0.f) x = fmaf(old[at], f.y, x);
                dst[at] = x;
            }
        };
        bool ok = true;
        if (warp < 4) {
            float Dr = 0.f, z = 0.f, umax = -INFINITY;
            if (D == 128) {
#pragma unroll
                for (int c = 0; c < SC; ++c) S[c] = 0.f;
            }
            for (int g = 0; ok && g < n; ++g) {
                if (!(ok = mbar_wait_all(p_full, g & 1, abort_flag))) break;
                tc_fence_after();
                float va[32], vb[32];
                // the tile's largest u, then D_r
                tmem_ld32_nowait(tL + C::T_P, va);
                tmem_wait_ld32(va);
                tmem_ld32_nowait(tL + C::T_P + 32, vb);
                float um = chunk_vmax(va);
                tmem_wait_ld32(vb);
                tmem_ld32_nowait(tL + C::T_P + 64, va);
                um = fmaxf(um, chunk_vmax(vb));
                tmem_wait_ld32(va);
                tmem_ld32_nowait(tL + C::T_P + 96, vb);
                um = fmaxf(um, chunk_vmax(va));
                tmem_wait_ld32(vb);
                tmem_ld32_nowait(tL + C::T_P, va);
                um = fmaxf(um, chunk_vmax(vb));
                const float tm = um * kLog2e;
                if (tm > -INFINITY && (umax == -INFINITY || tm - Dr > 15.f)) {
                    const float Dn = ceilf(tm) - 8.f;
                    z = z == 0.f ? 0.f : z * exp2f(Dr - Dn);
                    Dr = Dn;
                }
                umax = fmaxf(umax, um);
                sD[(g & 1) * 128 + row] = Dr;
                mbar_arrive(&d_full[g & 1]);
                auto chunk = [&](float(&v)[32], int c) {
                    uint32_t hi[16], lo[16];
                    float s0 = 0.f, s1 = 0.f;
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        float a, b;
                        ffma2(v[e], v[e + 1], kLog2e, kLog2e, -Dr, -Dr, a, b);
                        a = ex2_approx(a);
                        b = ex2_approx(b);
                        ffma2(a, b, 1.f, 1.f, s0, s1, s0, s1);
                        // hi: the 11 leading bits (exact in fp16 from 2^-14 on), lo: the rest
                        const float ah = tf32_trunc(a), bh_ = tf32_trunc(b);
                        hi[e >> 1] = pack_f16x2(ah, bh_);
                        lo[e >> 1] = pack_f16x2(a - ah, b - bh_);
                    }
                    z += s0 + s1;
                    tmem_st16u(tL + C::T_P + 32 * c, hi);
                    tmem_st16u(tL + C::T_P + 32 * c + 16, lo);
                    tmem_wait_st();
                    tc_fence_before();
                    mbar_arrive(&phi_full[c]);
                };
                tmem_wait_ld32(va);
                tmem_ld32_nowait(tL + C::T_P + 32, vb);
                chunk(va, 0);
                tmem_wait_ld32(vb);
                tmem_ld32_nowait(tL + C::T_P + 64, va);
                chunk(vb, 1);
                tmem_wait_ld32(va);
                tmem_ld32_nowait(tL + C::T_P + 96, vb);
                chunk(va, 2);
                tmem_wait_ld32(vb);
                // b of this tile; seen before the last chunk is handed on, since V's next phase may follow then
                if (D == 128 && !(ok = mbar_wait_all(&v_conv[g % NS], (g / NS) & 1, abort_flag))) break;
                chunk(vb, 3);
                if (D == 128) {
                    if (!(ok = mbar_wait_all(s_full, g & 1, abort_flag))) break;
                    tc_fence_after();
                    flush(g, 64);
                }
            }
            // z', D and the factors that bring the run's S and the carried S' to D
            float2 f = make_float2(0.f, 0.f);
            if (ok && r < m) {
                float Dn = umax;
                if (z != 0.f) f.x = exp2f(-fmaf(umax, kLog2e, -Dr));
                if (split == 0) {
                    const float z_old = old[(size_t)D * m + r], D_old = old[(size_t)D * m + m + r];
                    if (z_old != 0.f) {
                        Dn = z != 0.f ? fmaxf(D_old, umax) : D_old;
                        f.y = expf(D_old - Dn);
                        if (z != 0.f) f.x *= expf(umax - Dn);
                        z = fmaf(z_old, f.y, z * f.x);
                    } else {
                        z *= f.x;
                    }
                } else {
                    z *= f.x;
                }
                if (z != 0.f) dst[(size_t)D * m + m + r] = Dn;
                if (z != 0.f || !whole) dst[(size_t)D * m + r] = z;
            }
            sF[row] = f;
            named_bar_sync(2, 256);
            if (D == 128 && ok) finish(64);
        } else {
            const int j = threadIdx.x - 128;  // token of the tile
#pragma unroll
            for (int c = 0; c < SC; ++c) S[c] = 0.f;
            // key row j of tile g: -|k|^2/2 in three bf16 parts (their sum has fp32's precision); keys past
            // the count become zero rows at -inf
            auto conv_k = [&](int g) -> bool {
                const int s = g % NS;
                if (!mbar_wait_all(&k_full[s], (g / NS) & 1, abort_flag)) return false;
                uint8_t *kt = sK + (size_t)s * C::KT;
                uint4 xb = make_uint4(0xFF80u, 0u, 0u, 0u);
                if ((t0 + g) * kTile + j < count) {
                    const float h = -0.5f * key_sq_norm<NB, kTile>(kt, j);
                    if (h >= -3e38f || h != h) {
                        const uint32_t hi = bf16_bits_rn(h);
                        const float r1 = h - __uint_as_float(hi << 16);
                        const uint32_t mid = bf16_bits_rn(r1);
                        xb = make_uint4(hi | (mid << 16), bf16_bits_rn(r1 - __uint_as_float(mid << 16)), 0u, 0u);
                    }
                } else {
                    for (int i = 0; i < 8 * NB; ++i)
                        *(uint4 *)(kt + (i >> 3) * C::BLK + j * 128 + (i & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
                *(uint4 *)(sKx + s * 4096 + (j >> 3) * 256 + (j & 7) * 16) = xb;
                fence_async_smem();
                mbar_arrive(&k_conv[s]);
                return true;
            };
            // V tile g to fp16, scaled by its largest finite magnitude (a power of two)
            auto conv_v = [&](int g) -> bool {
                const int s = g % NS;
                if (!mbar_wait_all(&v_full[s], (g / NS) & 1, abort_flag)) return false;
                uint8_t *vt = sV + (size_t)s * C::KT;
                const int valid = count - (t0 + g) * kTile;
                uint32_t mx = 0;
#pragma unroll 4
                for (int i = 0; i < 8 * NB; ++i) {
                    const int ch = j + 128 * i;  // 16-byte chunk: row (ch / 8) % 128
                    if ((ch >> 3) % kTile < valid) {
                        const uint4 x = *(const uint4 *)(vt + (size_t)ch * 16);
                        const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t a = u[k] & 0x7FFF7FFFu;
                            mx = __vmaxu2(mx, a & ~__vcmpgeu2(a, 0x7F807F80u));
                        }
                    }
                }
                mx = max(mx & 0xFFFFu, mx >> 16);
                for (int o = 16; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                if (lane == 0) sRed[(g & 1) * 4 + (warp & 3)] = mx;
                mbar_arrive(v_max);
                if (!mbar_wait_all(v_max, g & 1, abort_flag)) return false;
                mx = max(max(sRed[(g & 1) * 4], sRed[(g & 1) * 4 + 1]), max(sRed[(g & 1) * 4 + 2], sRed[(g & 1) * 4 + 3]));
                const int b = min(max((int)(mx >> 7) - 127 - 7, -100), 120);
                if (j == 0) sShift[g & 3] = b;
                const float scale = __uint_as_float((uint32_t)(127 - b) << 23);
#pragma unroll 4
                for (int i = 0; i < 8 * NB; ++i) {
                    const int ch = j + 128 * i;
                    uint4 *at = (uint4 *)(vt + (size_t)ch * 16);
                    uint4 x = make_uint4(0u, 0u, 0u, 0u);
                    if ((ch >> 3) % kTile < valid) {
                        x = *at;
                        uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            u[k] = pack_f16x2(__uint_as_float(u[k] << 16) * scale, __uint_as_float(u[k] & 0xFFFF0000u) * scale);
                        x = make_uint4(u[0], u[1], u[2], u[3]);
                    }
                    *at = x;
                }
                fence_async_smem();
                mbar_arrive(&v_conv[s]);
                return true;
            };
            ok = conv_k(0) && conv_v(0);
            for (int g = 0; ok && g < n; ++g) {
                // the next tile's keys first: its projection waits for them alone
                if (g + 1 < n) ok = conv_k(g + 1);
                if (ok && NS > 1 && g + 1 < n) ok = conv_v(g + 1);
                // (one barrier per parity: the exponent warps may be one tile ahead)
                if (ok) ok = mbar_wait_all(&d_full[g & 1], (g >> 1) & 1, abort_flag) && mbar_wait_all(s_full, g & 1, abort_flag);
                if (!ok) break;
                tc_fence_after();
                flush(g, 0);
                if (NS == 1 && g + 1 < n) ok = conv_v(g + 1);
            }
            named_bar_sync(2, 256);
            if (ok) finish(0);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) tmem_dealloc(tmem, 256);
}

template <int D>
static cudaError_t launch_extend_tc_t(const CUtensorMap &mK, const CUtensorMap &mV, const CUtensorMap &mW,
                                      const ExtendParams &p, cudaStream_t st) {
    using C = ExtTc<D>;
    const cudaError_t e =
        cudaFuncSetAttribute(k_decode_extend_tc<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::BYTES);
    if (e != cudaSuccess) return e;
    const int BH = p.B * p.H;
    k_decode_extend_tc<D><<<dim3(p.n_split, (p.m + 127) / 128, BH), C::THREADS, C::BYTES, st>>>(mK, mV, mW, p);
    if (p.n_split > 1) k_extend_combine<<<dim3(D / kCombCols, BH), p.m, 0, st>>>(p, D);
    return cudaGetLastError();
}

cudaError_t launch_decode_extend_tc(const CUtensorMap &mK, const CUtensorMap &mV, const CUtensorMap &mW,
                                    const ExtendParams &p, int d, cudaStream_t st) {
    return d == 64 ? launch_extend_tc_t<64>(mK, mV, mW, p, st) : launch_extend_tc_t<128>(mK, mV, mW, p, st);
}

}  // namespace favor
