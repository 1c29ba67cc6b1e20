// favor_decode_extend on tensor cores: bf16 tokens in order (no index), long enough to fill tiles.
//
// One CTA per (run of 64-token tiles, half of 128 features, head), two CTAs an SM. Per tile:
//   P^T = W_h K^T - |k|^2/2    tcgen05 (M = 128 features, N = 64 tokens), bf16 operands (exact
//                              products); the norm enters as a K = 16 step of three bf16 parts per key
//                              against ones columns of W (-inf for a key past the sequence's count);
//   phi' = 2^(P log2e - D_r)   one thread per feature; D_r, an integer, is set so that the first
//                              tile's largest exponent lands in (2, 3] and raised where a later one's
//                              passes 15 (fp16 holds 2^t below 2^16; its smallest step is 2^-24);
//   acc += phi'^T V'           tcgen05 (M = 128, N = d, K = 64), fp16 operands: phi' = hi + lo, two fp16
//                              values (22 bits), A from TMEM where they replace P; V' = V 2^-b, b per value
//                              column: exact in fp16 but for entries 2^-20 of the column's largest in this
//                              tile and below (off by 2^-21 of it);
//   S_r <- 2^(..) S_r + 2^b acc  in fp32, every kExtFlush tiles and before a tile that changes D_r or b:
//                              the tensor core's own accumulation truncates, up to 2^-23 of the sum at each
//                              of the 128 additions of 1024 tokens. Values of one sign come out 7e-6 low on
//                              average (1.6e-5 at most) and half that every 8 tiles, where 65536 tokens in 16
//                              heads take 213 us for 209 and 16384 at d = 128 127 for 118; values of both
//                              signs 1e-6 (d = 64) and 2e-6 (d = 128) off in all.
// A single fp16 phi' would cost 1e-4 relative in S (the roundings do not average out against values of
// both signs); with hi + lo the MMA work is 1.5 times the least.
//
// P is double-buffered: while the exponent warps work on one tile, the MMAs of the tile before (S) and
// the one after (P) run, so that the exponent warps do not wait for a round trip of the tensor core
// (with one buffer of 128 tokens they did: 283 us for 65536 tokens in 16 heads at d = 64, m = 256).
// Bound: the tensor work, 6 L m d a head (64 us for 65536 tokens in 16 heads), and 2^t on the MUFU (16 a cycle
// and SM), B H L m of them (60 us). What is measured (209 us) is issue, 4000 warp instructions a tile.
//
// Warps 0-3: exponentials and z_r. Warps 4, 5: |k|^2 and the norms' extension; 6, 7: V -> fp16 (one after
// the other in all four they held up the exponents: 4200 cycles a tile against 1550); 4-7: S. Warp 8: K
// and W copies, P; warp 9: V copies, the accumulator. Every barrier that a group waits on is at most one
// phase ahead of it, but d_full, which has four slots. What the tiles tell each other through shared memory
// (D_r, whether it changed, b) lies in rings of kExtRing tiles: the exponent warps may be five tiles ahead of
// warps 6, 7, each of which reads a tile's entries only after converting a later tile, and so may the
// other warp of the two (tests/test_extend_tile_protocol.py walks all these orderings).

#include "common.cuh"

namespace favor {

constexpr int kExtTile = 64;
constexpr int kExtFlush = 16;
constexpr int kExtRing = 8;

template <int D_>
struct ExtTc {
    static constexpr int D = D_, NB = D / 64;
    static constexpr int NS = D == 64 ? 4 : 2;  // K and V stages each (227 KB for two CTAs)
    static constexpr uint32_t WBLK = 128 * 128, WT = NB * WBLK, BLK = kExtTile * 128, KT = NB * BLK, KX = kExtTile * 32;
    static constexpr int THREADS = 320;
    static constexpr uint32_t T_P = 0, T_ACC = 128;  // TMEM columns: two tiles of P, the accumulator
    static constexpr size_t OFF_K = WT, OFF_V = OFF_K + NS * KT, OFF_KX = OFF_V + NS * KT, OFF_WX = OFF_KX + NS * KX,
                            OFF_D = OFF_WX + 4096, OFF_F = OFF_D + kExtRing * 128 * 4, OFF_MISC = OFF_F + 128 * 8,
                            OFF_B = OFF_MISC + 4 * 6 * kExtRing, OFF_BAR = OFF_B + kExtRing * D * 2, BYTES = OFF_BAR + 8 * (4 * NS + 2 + 2 + 2 + 4 + 5 + 4) + 8 + 1024;
};

// Per-column maxima of |entries| over a 64 x 64 block of V (a warp; `at`: the block's chunk of this lane).
// Chunk lane + 32 i is row lane / 8 + 4 i, columns 8 (L ^ 4 (i % 2)) and on, L = (lane % 8) ^ (lane / 8): the
// chunks of odd i change places between lanes of L and L ^ 4, then the lanes of one L come together. Returned
// are columns 8 L + 2 (lane / 8) and the next, as two bf16 patterns.
__device__ __forceinline__ void ext_swap(uint32_t (&mx)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) mx[k] = __shfl_xor_sync(0xffffffffu, mx[k], 4);
}
__device__ __forceinline__ uint32_t ext_reduce(const uint32_t (&mx)[4], int lane) {
    const bool h = (lane & 16) != 0, o = (lane & 8) != 0;
    const uint32_t s0 = __shfl_xor_sync(0xffffffffu, h ? mx[0] : mx[2], 18);
    const uint32_t s1 = __shfl_xor_sync(0xffffffffu, h ? mx[1] : mx[3], 18);
    const uint32_t a = __vmaxu2(h ? mx[2] : mx[0], s0), b = __vmaxu2(h ? mx[3] : mx[1], s1);
    return __vmaxu2(o ? b : a, __shfl_xor_sync(0xffffffffu, o ? a : b, 9));
}
__device__ __forceinline__ uint32_t ext_column_max(const uint8_t *at, int lane) {
    uint32_t mx[4] = {0u, 0u, 0u, 0u};
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {  // odd i, then even i
        if (q == 2) ext_swap(mx);
        const uint8_t *c = at + (8 * (q & 1) + (q < 2 ? 1 : 0)) * 512;
        uint4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *(const uint4 *)(c + i * 1024);
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            mx[0] = __vimax3_u16x2(mx[0], x[i].x & 0x7FFF7FFFu, x[i + 1].x & 0x7FFF7FFFu);
            mx[1] = __vimax3_u16x2(mx[1], x[i].y & 0x7FFF7FFFu, x[i + 1].y & 0x7FFF7FFFu);
            mx[2] = __vimax3_u16x2(mx[2], x[i].z & 0x7FFF7FFFu, x[i + 1].z & 0x7FFF7FFFu);
            mx[3] = __vimax3_u16x2(mx[3], x[i].w & 0x7FFF7FFFu, x[i + 1].w & 0x7FFF7FFFu);
        }
    }
    return ext_reduce(mx, lane);
}
// The same over the finite entries alone, and the conversion of a tile with others (rare; out of line, so
// that the instruction cache keeps the ordinary path).
__device__ __noinline__ uint32_t ext_column_max_finite(const uint8_t *at, int lane) {
    uint32_t mx[4] = {0u, 0u, 0u, 0u};
#pragma unroll 1
    for (int i = 0; i < 16; ++i) {
        if (i == 8) ext_swap(mx);
        const uint4 x = *(const uint4 *)(at + (i < 8 ? 2 * i + 1 : 2 * i - 16) * 512);
        const uint32_t u[4] = {x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu, x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu};
#pragma unroll
        for (int k = 0; k < 4; ++k) mx[k] = __vmaxu2(mx[k], u[k] & ~__vcmpgeu2(u[k], 0x7F807F80u));
    }
    return ext_reduce(mx, lane);
}
__device__ __noinline__ void ext_convert_odd(uint8_t *vt, const uint16_t *sb, int lane) {
    const int L = (lane & 7) ^ (lane >> 3);
#pragma unroll 1
    for (int i = 0; i < 16; ++i) {
        uint4 *at = (uint4 *)(vt + (lane + 32 * i) * 16);
        const uint4 x = *at, lw = *(const uint4 *)(sb + 8 * (L ^ (4 * (i & 1))));
        uint32_t u[4] = {x.x, x.y, x.z, x.w};
        const uint32_t low[4] = {lw.x, lw.y, lw.z, lw.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // an infinity or NaN stays one
            const uint32_t a = u[k] & 0x7FFF7FFFu, odd = __vcmpgeu2(a, 0x7F807F80u);
            const uint32_t h = ((__vmaxu2(a, low[k]) - low[k]) << 3) & ~odd;
            u[k] = h | (((a & 0x007F007Fu) << 3 | 0x7C007C00u) & odd) | (u[k] & 0x80008000u);
        }
        *at = make_uint4(u[0], u[1], u[2], u[3]);
    }
}

template <int D>
__global__ void __launch_bounds__(ExtTc<D>::THREADS, 2)
k_decode_extend_tc(const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                   const __grid_constant__ CUtensorMap mapW, ExtendParams p) {
    using C = ExtTc<D>;
    constexpr int NS = C::NS, NB = C::NB;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t *sW = smem, *sK = smem + C::OFF_K, *sV = smem + C::OFF_V, *sKx = smem + C::OFF_KX, *sWx = smem + C::OFF_WX;
    float *sD = (float *)(smem + C::OFF_D);       // [tile % kExtRing][128]: D_r
    float2 *sF = (float2 *)(smem + C::OFF_F);     // [128]: final factors of the run's and the old S'
    int *sRaise = (int *)(smem + C::OFF_MISC);    // [tile % kExtRing][warp]: some D_r of this warp's changes here
    int *sScale = sRaise + 4 * kExtRing;          // [tile % kExtRing][block]: some b of its 64 columns changes here
    uint16_t *sB = (uint16_t *)(smem + C::OFF_B); // [tile % kExtRing][D]: (112 + b) 2^7, as a bf16 exponent
    uint64_t *bars = (uint64_t *)(smem + C::OFF_BAR);
    uint64_t *k_full = bars, *v_full = k_full + NS, *k_conv = v_full + NS, *v_conv = k_conv + NS;
    uint64_t *p_full = v_conv + NS, *phi_full = p_full + 2, *s_done = phi_full + 2, *d_full = s_done + 2;
    uint64_t *w_full = d_full + 4, *acc_full = w_full + 1, *acc_free = w_full + 2, *drain = w_full + 3, *b_set = w_full + 5;
    uint32_t *tmem_slot = (uint32_t *)(b_set + 4);
    volatile int *abort_flag = (volatile int *)(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = blockIdx.x, half = blockIdx.y, bh = blockIdx.z;
    const int count = extend_count(p, bh / p.H);
    if (count == 0) return;  // the state stays as it is
    const int t0 = split * (p.tok_per_split / kExtTile);  // tok_per_split is a multiple of the tile
    const int t1 = min((count - 1) / kExtTile + 1, t0 + p.tok_per_split / kExtTile);
    const int n = t1 - t0, m = p.m;
    const size_t len = (size_t)D * m + 2 * m;
    const bool whole = p.n_split == 1 && D == 64;
    float *dst = whole ? p.state + (size_t)bh * len : p.part + ((size_t)bh * p.n_split + split) * len;
    if (n <= 0) return;  // an empty run

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&k_full[s], 1);
            mbar_init(&v_full[s], 1);
            mbar_init(&k_conv[s], 64);
            mbar_init(&v_conv[s], 32 * NB);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&p_full[s], 1);
            mbar_init(&phi_full[s], 128);
            mbar_init(&s_done[s], 1);
        }
        for (int s = 0; s < 4; ++s) {
            mbar_init(&d_full[s], 128 + 32 * NB);
            mbar_init(&b_set[s], 32);
        }
        mbar_init(w_full, 1);
        mbar_init(acc_full, 1);
        mbar_init(acc_free, 128);
        mbar_init(&drain[0], 1);
        mbar_init(&drain[1], 1);
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
    for (int i = threadIdx.x; i < NS * kExtTile; i += C::THREADS)
        *(uint4 *)(sKx + (i / kExtTile) * C::KX + ((i % kExtTile) >> 3) * 256 + 128 + (i & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // whether S takes the accumulator before tile g adds to it (read after tile g's d_full, or its phi_full
    // and v_conv)
    auto flush_before = [&](int g) {
        const int *r = sRaise + 4 * (g % kExtRing), *b = sScale + 2 * (g % kExtRing);
        return g > 0 && ((g % kExtFlush) == 0 || b[0] != 0 || (NB == 2 && b[1] != 0) || (r[0] | r[1] | r[2] | r[3]) != 0);
    };

    auto load = [&](const CUtensorMap *map, uint8_t *buf, uint64_t *bar, int g) {
        if (elect_one()) {
            mbar_arrive_expect_tx(&bar[g % NS], C::KT);
            for (int nb = 0; nb < NB; ++nb)
                tma_load_3d(buf + (size_t)(g % NS) * C::KT + nb * C::BLK, map, &bar[g % NS], 64 * nb, (t0 + g) * kExtTile, bh);
        }
        __syncwarp();
    };
    if (warp == 8) {  // K and W copies, P
        int nk = 0;  // K tiles asked for
        load(&mapK, sK, k_full, nk++);
        if (elect_one()) {
            mbar_arrive_expect_tx(w_full, C::WT);
            for (int nb = 0; nb < NB; ++nb) tma_load_2d(sW + nb * C::WBLK, &mapW, w_full, 64 * nb, half * 128);
        }
        __syncwarp();
        for (; nk < min(NS, n); ++nk) load(&mapK, sK, k_full, nk);
        const uint32_t idesc_p = make_idesc(128, kExtTile, kFmtBF16, 0, 0);
        const uint64_t dW = make_sdesc(smem_u32(sW), 16, 1024), dK = make_sdesc(smem_u32(sK), 16, 1024);
        const uint64_t dWx = make_sdesc_interleaved(smem_u32(sWx), 128, 256);
        const uint64_t dKx = make_sdesc_interleaved(smem_u32(sKx), 128, 256);
        bool ok = mbar_wait_all(w_full, 0, abort_flag);
        for (int i = 0; ok && i < n; ++i) {  // where phi' of tile i - 2 was
            const int s = i % NS;
            ok = mbar_wait_all(&k_conv[s], (i / NS) & 1, abort_flag) &&
                 (i < 2 || mbar_wait_all(&s_done[i & 1], ((i >> 1) - 1) & 1, abort_flag));
            if (!ok) break;
            tc_fence_after();
            const uint32_t P = tmem + C::T_P + kExtTile * (i & 1);
            for (int nb = 0; nb < NB; ++nb)
                mma_ss_x4_w(P, dW + nb * (C::WBLK / 16), dK + s * (C::KT / 16) + nb * (C::BLK / 16), idesc_p, nb > 0, 2, 2);
            mma_f16_ss_w(P, dWx, dKx + s * (C::KX / 16), idesc_p, 1u);
            mma_commit_w(&p_full[i & 1]);
            if (i >= 1 && nk < n) {  // the keys of the tile before are done with
                if (!(ok = mbar_wait_all(&p_full[(i - 1) & 1], ((i - 1) >> 1) & 1, abort_flag))) break;
                load(&mapK, sK, k_full, nk++);
            }
        }
        // nothing of this warp is in flight when the CTA frees its memory
        mma_commit_w(&drain[0]);
        volatile int no_abort = 0;
        mbar_wait_all(&drain[0], 0, &no_abort);
        mbar_wait_all(w_full, 0, &no_abort);
        for (int g = max(nk - NS, 0); g < nk; ++g) mbar_wait_all(&k_full[g % NS], (g / NS) & 1, &no_abort);
    } else if (warp == 9) {  // V copies, S
        int nv = 0, flushes = 0;  // V tiles asked for
        for (; nv < min(NS, n); ++nv) load(&mapV, sV, v_full, nv);
        const uint32_t idesc_s = make_idesc(128, D, kFmtF16, 0, 1);
        const uint64_t dV = make_sdesc(smem_u32(sV), C::BLK, 1024);
        bool ok = true;
        for (int j = 0; ok && j < n; ++j) {
            if (j >= 1 && nv < n) {  // the values of the tile before are done with
                if (!(ok = mbar_wait_all(&s_done[(j - 1) & 1], ((j - 1) >> 1) & 1, abort_flag))) break;
                load(&mapV, sV, v_full, nv++);
            }
            ok = mbar_wait_all(&v_conv[j % NS], (j / NS) & 1, abort_flag) &&
                 mbar_wait_all(&phi_full[j & 1], (j >> 1) & 1, abort_flag);
            if (!ok) break;
            tc_fence_after();
            const bool fresh = flush_before(j);
            if (fresh) {
                mma_commit_w(acc_full);
                if (!(ok = mbar_wait_all(acc_free, flushes++ & 1, abort_flag))) break;
                tc_fence_after();
            }
            const uint32_t phi = tmem + C::T_P + kExtTile * (j & 1);
            const uint64_t v = dV + (j % NS) * (C::KT / 16);
#pragma unroll
            for (int k = 0; k < kExtTile / 16; ++k) {
                mma_f16_ts_w(tmem + C::T_ACC, phi + 16 * k, v + k * (16 * 128 / 16), idesc_s, !(j == 0 || fresh) || k > 0);
                mma_f16_ts_w(tmem + C::T_ACC, phi + 16 * k + 8, v + k * (16 * 128 / 16), idesc_s, 1u);
            }
            mma_commit_w(&s_done[j & 1]);
        }
        if (ok) mma_commit_w(acc_full);
        mma_commit_w(&drain[1]);
        volatile int no_abort = 0;
        mbar_wait_all(&drain[1], 0, &no_abort);
        for (int g = max(nv - NS, 0); g < nv; ++g) mbar_wait_all(&v_full[g % NS], (g / NS) & 1, &no_abort);
    } else {
        const int row = (warp & 3) * 32 + lane, r = half * 128 + row;
        const uint32_t tL = tmem + (((uint32_t)(warp & 3) * 32u) << 16);
        const float *old = p.state + (size_t)bh * len;
        bool ok = true;
        if (warp < 4) {
            float Dr = 0.f, z = 0.f, umax = -INFINITY;
            for (int g = 0; ok && g < n; ++g) {
                if (!(ok = mbar_wait_all(&p_full[g & 1], (g >> 1) & 1, abort_flag))) break;
                tc_fence_after();
                const uint32_t P = tL + C::T_P + kExtTile * (g & 1);
                float va[32], vb[32];
                tmem_ld32_nowait(P, va);
                tmem_ld32_nowait(P + 32, vb);
                tmem_wait_ld32(va);
                tmem_wait_ld32(vb);
                // the tile's largest u, then D_r
                const float um = fmaxf(chunk_vmax(va), chunk_vmax(vb)), tm = um * kLog2e;
                bool raise = false;
                if (tm > -INFINITY && (umax == -INFINITY || tm - Dr > 15.f)) {
                    const float Dn = ceilf(tm) - 3.f;
                    z = z == 0.f ? 0.f : z * exp2f(Dr - Dn);
                    Dr = Dn;
                    raise = true;
                }
                umax = fmaxf(umax, um);
                sD[(g % kExtRing) * 128 + row] = Dr;
                raise = __any_sync(0xffffffffu, raise);
                if (lane == 0) sRaise[4 * (g % kExtRing) + warp] = raise;
                __syncwarp();
                mbar_arrive(&d_full[g & 3]);
                float s0 = 0.f, s1 = 0.f;
#pragma unroll 1
                for (int c = 0; c < kExtTile; c += 16) {  // 16 tokens: hi in 8 columns, lo in the next 8
                    float v[16];
                    tmem_ld16(P + c, v);
                    uint32_t hi[8], lo[8];
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        float a, b;
                        ffma2(v[e], v[e + 1], kLog2e, kLog2e, -Dr, -Dr, a, b);
                        a = ex2_approx(a);
                        b = ex2_approx(b);
                        ffma2(a, b, 1.f, 1.f, s0, s1, s0, s1);
                        // hi: the 11 leading bits (exact in fp16 from 2^-14 on), lo: the rest
                        const float ah = tf32_trunc(a), bh_ = tf32_trunc(b);
                        float al, bl;
                        ffma2(ah, bh_, -1.f, -1.f, a, b, al, bl);
                        hi[e >> 1] = pack_f16x2(ah, bh_);
                        lo[e >> 1] = pack_f16x2(al, bl);
                    }
                    tmem_st8u(P + c, hi);
                    tmem_st8u(P + c + 8, lo);
                }
                z += s0 + s1;
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&phi_full[g & 1]);
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
                if (z != 0.f || !whole) dst[(size_t)D * m + m + r] = Dn;
                if (z != 0.f || !whole) dst[(size_t)D * m + r] = z;
            }
            sF[row] = f;
            named_bar_sync(2, 256);
        } else {
            // Warps 4 and 5, key rows of tile g, one a thread: -|k|^2/2 in three bf16 parts (their sum has fp32's
            // precision); keys past the count become zero rows at -inf
            auto conv_k = [&](int g) -> bool {
                const int s = g % NS, j = threadIdx.x - 128;
                if (!mbar_wait_all(&k_full[s], (g / NS) & 1, abort_flag)) return false;
                uint8_t *kt = sK + (size_t)s * C::KT;
                uint4 xb = make_uint4(0xFF80u, 0u, 0u, 0u);
                if ((t0 + g) * kExtTile + j < count) {
                    const float h = -0.5f * key_sq_norm<NB, kExtTile>(kt, j);
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
                *(uint4 *)(sKx + s * C::KX + (j >> 3) * 256 + (j & 7) * 16) = xb;
                fence_async_smem();
                mbar_arrive(&k_conv[s]);
                return true;
            };
            // V tile g to fp16 at scale 2^-b, by warps 6 and 7 in turn or (d = 128) a block of 64 columns each: a
            // column's b follows its largest finite magnitude in the tile (which lands in [2^12, 2^13)), all of
            // a block where one would leave [2^6, 2^15). A bf16 value's fp16 form at that scale is integer
            // arithmetic on its bits, exact from 2^-14 on (smaller ones are off by 2^-15 at most); infinities and
            // NaN stay what they are.
            auto conv_v = [&](int g) -> bool {
                const int s = g % NS, blk = NB == 2 ? warp & 1 : 0, L = (lane & 7) ^ (lane >> 3);
                if (!mbar_wait_all(&v_full[s], (g / NS) & 1, abort_flag)) return false;
                uint8_t *vt = sV + (size_t)s * C::KT + blk * C::BLK;
                uint16_t *sb = sB + (g % kExtRing) * D + 64 * blk;
                const int valid = count - (t0 + g) * kExtTile;
                if (valid < kExtTile)
                    for (int c = lane; c < 512; c += 32)
                        if ((c >> 3) >= valid) *(uint4 *)(vt + (size_t)c * 16) = make_uint4(0u, 0u, 0u, 0u);
                uint32_t now = ext_column_max(vt + lane * 16, lane);  // of columns 8 L + 2 (lane / 8) and the next
                const bool odd = __any_sync(0xffffffffu, max(now & 0xFFFFu, now >> 16) >= 0x7F80u);
                if (odd) now = ext_column_max_finite(vt + lane * 16, lane);
                // b from the exponent, within -100 .. 114; 0 where the column is
                now = __vminu2(__vmaxu2(now & 0x7F807F80u, 0x13801380u) - 0x0D800D80u, 0x71007100u) & ~__vcmpeq2(now, 0u);
                if (NB == 1 && g > 0 && !mbar_wait_all(&b_set[(g - 1) & 3], ((g - 1) >> 2) & 1, abort_flag)) return false;
                {
                    const int at = 4 * L + (lane >> 3);
                    const uint32_t was = g > 0 ? ((const uint32_t *)(sB + ((g - 1) % kExtRing) * D + 64 * blk))[at] : 0x06000600u;
                    now |= was & __vcmpeq2(now, 0u);
                    const uint32_t by = now - was + 0x83008300u;  // b's change, from -6 to 2 or out of range
                    const bool changed = __any_sync(0xffffffffu, by != __vmaxu2(__vminu2(by, 0x84008400u), 0x80008000u)) || g == 0;
                    ((uint32_t *)sb)[at] = changed ? now : was;
                    if (lane == 0) sScale[2 * (g % kExtRing) + blk] = changed;
                }
                __syncwarp();
                if (NB == 1) mbar_arrive(&b_set[g & 3]);
                mbar_arrive(&d_full[g & 3]);
                if (!odd) {
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        uint8_t *at = vt + lane * 16 + (8 * (q & 1) + (q >> 1)) * 512;
                        const uint4 lw = *(const uint4 *)(sb + 8 * (L ^ (2 * (q & 2))));
                        const uint32_t low[4] = {lw.x, lw.y, lw.z, lw.w};
                        uint4 x[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[i] = *(const uint4 *)(at + i * 1024);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                u[k] = ((__vmaxu2(u[k] & 0x7FFF7FFFu, low[k]) - low[k]) << 3) | (u[k] & 0x80008000u);
                            *(uint4 *)(at + i * 1024) = make_uint4(u[0], u[1], u[2], u[3]);
                        }
                    }
                } else {
                    ext_convert_odd(vt, sb, lane);
                }
                fence_async_smem();
                mbar_arrive(&v_conv[s]);
                return true;
            };
            // S_r in units of 2^Dreg: registers at d = 64; at d = 128 the run's partial state in global
            // memory, 16 columns in flight at a time (128 more registers a thread are not to be had, and
            // as local memory they took 33,000 cycles a flush)
            constexpr int SR = D == 64 ? D : 1;
            float S[SR];
            float Dreg = 0.f, Dacc = 0.f;  // Dacc: the accumulator's D_r
            bool first = true;
#pragma unroll
            for (int c = 0; c < SR; ++c) S[c] = 0.f;
            auto flush = [&](int last) {  // the accumulator's last tile (its b is that of all of them)
                const float keep = exp2f(fminf(Dreg - Dacc, 0.f));
                const uint16_t *sb = sB + (last % kExtRing) * D;
                Dreg = Dacc;
                float v[16];
                // 16 columns times 2^b
                auto scaled = [&](int q) {
                    tmem_ld16(tL + C::T_ACC + q, v);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint4 x = *(const uint4 *)(sb + q + 8 * h);
                        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            v[8 * h + 2 * c] *= __uint_as_float((w[c] << 16) + 0x07800000u);
                            v[8 * h + 2 * c + 1] *= __uint_as_float((w[c] & 0xFFFF0000u) + 0x07800000u);
                        }
                    }
                };
                if constexpr (D == 64) {
                    // (in place and in a rolled loop: next to S there are no registers for the scales)
#pragma unroll 1
                    for (int q = 0; q < D; q += 16) {
                        scaled(q);
                        uint32_t u[16];
#pragma unroll
                        for (int c = 0; c < 16; ++c) u[c] = __float_as_uint(v[c]);
                        tmem_st16u(tL + C::T_ACC + q, u);
                    }
                    tmem_wait_st();
#pragma unroll
                    for (int q = 0; q < D; q += 16) {
                        tmem_ld16(tL + C::T_ACC + q, v);
#pragma unroll
                        for (int c = 0; c < 16; c += 2)
                            ffma2(S[q + c], S[q + c + 1], keep, keep, v[c], v[c + 1], S[q + c], S[q + c + 1]);
                    }
                } else {
                    float *at = dst + r, s[16];
#pragma unroll 1
                    for (int q = 0; q < D; q += 16, at += 16 * (size_t)m) {
#pragma unroll
                        for (int c = 0; c < 16; ++c) s[c] = first || r >= m ? 0.f : __ldcg(at + (size_t)c * m);
                        scaled(q);
                        if (r < m) {
#pragma unroll
                            for (int c = 0; c < 16; ++c) __stcg(at + (size_t)c * m, fmaf(s[c], keep, v[c]));
                        }
                    }
                    first = false;
                }
                tc_fence_before();
                mbar_arrive(acc_free);
            };
            const bool keys = warp < 6;
            int flushes = 0;
            // V is converted two tiles ahead where there are slots for it, by one of its warps a tile; where there
            // are not, that would be what everyone waits for (d = 128: 123 us for 16384 tokens in 16 heads, 118
            // with half a tile each)
            constexpr int lead = NS >= 4 ? 2 : 1;
            auto mine = [&](int g) { return NB == 2 || (g & 1) == (warp & 1); };
            ok = keys ? conv_k(0) && (n < 2 || conv_k(1)) : mine(0) ? conv_v(0) : lead == 1 || n < 2 || conv_v(1);
            for (int g = 0; ok && g < n; ++g) {
                if (keys)
                    ok = g + 2 >= n || conv_k(g + 2);
                else
                    ok = g + lead >= n || !mine(g + lead) || conv_v(g + lead);
                if (!ok || !(ok = mbar_wait_all(&d_full[g & 3], (g >> 2) & 1, abort_flag))) break;
                const bool take = flush_before(g);
                const float Dg = sD[(g % kExtRing) * 128 + row];  // (before the accumulator is given back)
                if (take) {
                    if (!(ok = mbar_wait_all(acc_full, flushes++ & 1, abort_flag))) break;
                    tc_fence_after();
                    flush(g - 1);
                }
                if (take || g == 0) Dacc = Dg;
            }
            if (ok && (ok = mbar_wait_all(acc_full, flushes & 1, abort_flag))) {
                tc_fence_after();
                flush(n - 1);
            }
            named_bar_sync(2, 256);
            // the run's S' in the state's units, joined with the carried one
            // (a partial state is written even where no token entered: the sum over runs reads it)
            const float2 f = sF[row];
            if (ok && r < m && (f.x != 0.f || f.y != 0.f || !whole)) {
#pragma unroll
                for (int q = 0; q < D; q += 16) {  // 16 columns' loads before their stores
                    float x[16], y[16];
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const size_t at = (size_t)(q + c) * m + r;
                        x[c] = D == 64 ? S[D == 64 ? q + c : 0] : __ldcg(dst + at);
                        y[c] = f.y != 0.f ? __ldcg(old + at) : 0.f;
                    }
#pragma unroll
                    for (int c = 0; c < 16; ++c)
                        dst[(size_t)(q + c) * m + r] = fmaf(y[c], f.y, f.x != 0.f ? x[c] * f.x : 0.f);
                }
            }
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
    if (p.n_split > 1 || D != 64) k_extend_combine<<<dim3(D / kCombCols, BH), p.m, 0, st>>>(p, D);
    return cudaGetLastError();
}

cudaError_t launch_decode_extend_tc(const CUtensorMap &mK, const CUtensorMap &mV, const CUtensorMap &mW,
                                    const ExtendParams &p, int d, cudaStream_t st) {
    return d == 64 ? launch_extend_tc_t<64>(mK, mV, mW, p, st) : launch_extend_tc_t<128>(mK, mV, mW, p, st);
}

}  // namespace favor
