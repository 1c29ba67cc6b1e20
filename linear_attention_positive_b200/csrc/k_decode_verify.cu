// Verification of a drafted tree against the target's probabilities with given random numbers, and
// the sample of the token that follows (speculative sampling: the accepted path and the last token
// are distributed as if each token had been sampled from the target).
//
// The walk: cur = node 0, w = p[cur], Z = 1. Each child c of cur, in ascending order, with token x:
// accepted iff u_c Z q(x) < w(x) (q = q[cur], or 1 for a draft of point masses), then cur = c,
// w = p[c], Z = 1; rejected: w <- max(w - Z q, 0), Z <- sum w (point masses: Z <- Z - w(x),
// w(x) <- 0). When no child is left the last token is the first y with sum_{y' <= y} w > r sum w.
//
// Since max(max(w - a, 0) - b, 0) = max(w - (a + b), 0), the residual of a node needs one number,
// R = the sum of its Z so far: w = max(p - R q, 0). The walk looks at single entries, gathered for
// all nodes at once before it starts; only a rejection (its Z) and the last token need a pass over a
// row. Sums are held in fp64: a border of the running sum then moves by about 1e-16 relative with
// the order of additions, so the sampled index does not depend on it in practice.
//
// One cluster of kVerCluster CTAs per sequence, every warp a contiguous part of the vocabulary: a pass
// reads each row once in 16-byte groups (the groups lie on 16-byte boundaries of memory, so rows of odd
// vocabularies are read element by element only at their ends), and the sums meet through distributed
// shared memory in a fixed order, so every CTA takes the same branch. 256 threads and 64 registers let
// all 512 CTAs of a batch of 64 be resident at once (512 threads a CTA left a second wave). The pass is
// bound by HBM latency and bandwidth on the rows it reads (64 sequences, V = 131072, fp32: 39 us, 59 element
// by element); the sample then re-reads one warp's part, shared among its CTA's warps.

#include <cooperative_groups.h>

#include "common.cuh"

namespace favor {

constexpr int kVerThreads = 256;
constexpr int kVerWarps = kVerThreads / 32;
constexpr int kVerCluster = 8;
constexpr int kVerNodes = FAVOR_TREE_MAX_NODES;

struct VerifyParams {
    int B, T, V;
    const int *parents, *tokens, *n_nodes;  // [B, T], [B, T], [B] or NULL
    const void *p, *q;                      // [B, T, V], q may be NULL
    const float *u, *r;                     // [B, T], [B]
    int *path, *n_path, *next;              // [B, T], [B], [B]
};

// The weight max(p - R q, 0); NaN counts as 0 (fmax drops it).
__device__ __forceinline__ double ver_weight(float p, float q, double R) {
    return fmax(fma(-R, (double)q, (double)p), 0.0);
}

template <bool BF16>
__device__ __forceinline__ float ver_elem(const void *a, size_t i) {
    return BF16 ? __uint_as_float((uint32_t)__ldg((const uint16_t *)a + i) << 16) : __ldg((const float *)a + i);
}

struct VerShared {
    int par[kVerNodes], tok[kVerNodes];
    float px[kVerNodes], qx[kVerNodes], u[kVerNodes];
    int lost[kVerNodes];       // point masses: tokens rejected at the current node
    double warp_sum[kVerWarps], sub_sum[kVerWarps];
    double cta_sum;            // read by the other CTAs of the cluster
    int win;                   // the warp whose part holds the sample, kVerWarps where none does
    int pick, last;            // the CTA's sampled index, V where it has none; its last index with weight
};

template <bool BF16, bool DENSE>
__global__ void __launch_bounds__(kVerThreads, 4) k_decode_verify(VerifyParams a) {
    namespace cg = cooperative_groups;
    cg::cluster_group cl = cg::this_cluster();
    __shared__ VerShared s;
    const int b = blockIdx.x / kVerCluster, rank = (int)cl.block_rank();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int T = a.T, V = a.V;
    int n = T;
    if (a.n_nodes != nullptr) {
        n = a.n_nodes[b];
        if ((n < 0 || n > T) && tid == 0) record_status(FAVOR_ERR_INVALID_ARG);
        n = min(max(n, 0), T);
    }
    const size_t base = (size_t)b * T;
    for (int i = tid; i < n; i += kVerThreads) {
        int par = a.parents[base + i];
        const int tok = a.tokens[base + i];
        if (par < -1 || par >= i) {
            record_status(FAVOR_ERR_INVALID_ARG);
            par = -1;
        }
        float px = 0.f, qx = 0.f;
        if (par >= 0 && tok >= 0 && tok < V) {
            px = ver_elem<BF16>(a.p, (base + par) * V + tok);
            qx = DENSE ? ver_elem<BF16>(a.q, (base + par) * V + tok) : 1.f;
        } else if (par >= 0) {
            record_status(FAVOR_ERR_INVALID_ARG);
            par = -1;  // a token outside the vocabulary: never reached
        }
        s.par[i] = par;
        s.tok[i] = tok;
        s.px[i] = px;
        s.qx[i] = qx;
        s.u[i] = a.u[base + i];
    }
    if (tid == 0) {
        s.pick = V;
        s.last = -1;
        s.win = kVerWarps;
    }
    __syncthreads();
    if (n == 0) {  // an empty row of a padded batch (the whole cluster leaves together)
        if (rank == 0) {
            for (int i = tid; i < T; i += kVerThreads) a.path[base + i] = -1;
            if (tid == 0) {
                a.n_path[b] = 0;
                a.next[b] = -1;
            }
        }
        return;
    }
    constexpr int VE = BF16 ? 8 : 4;  // entries of a 16-byte group

    int cur = 0, count = 1, n_lost = 0;
    double R = 0.0, Z = 1.0, total = 0.0;
    bool have = false;  // total and the warp sums belong to the current (cur, R)

    // Row cur in groups: group g holds entries g VE - off and on (those outside 0 .. V-1 weigh 0).
    size_t row = 0;
    int off = 0, groups = 0, per = 0;
    auto part_begin = [&](int w) { return (int)min((long long)groups, (long long)(rank * kVerWarps + w) * per); };
    auto set_row = [&]() {
        row = (base + cur) * (size_t)V;
        off = (int)(row % VE);
        groups = (V + off + VE - 1) / VE;
        per = (groups + kVerCluster * kVerWarps - 1) / (kVerCluster * kVerWarps);
    };
    auto load_group = [&](const void *t, int y0) -> uint4 {
        if (y0 >= 0 && y0 <= V - VE)
            return __ldg((const uint4 *)((const char *)t + (row + y0) * (BF16 ? 2 : 4)));
        uint32_t x[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int k = 0; k < VE; ++k)
            if (y0 + k >= 0 && y0 + k < V) {
                if (BF16)
                    x[k / 2] |= (uint32_t)__ldg((const uint16_t *)t + row + y0 + k) << (16 * (k & 1));
                else
                    x[k] = __ldg((const uint32_t *)t + row + y0 + k);
            }
        return make_uint4(x[0], x[1], x[2], x[3]);
    };
    auto entry = [&](const uint4 &g, int k) -> float {
        const uint32_t x[4] = {g.x, g.y, g.z, g.w};
        if (!BF16) return __uint_as_float(x[k]);
        return __uint_as_float((k & 1) ? x[k / 2] & 0xFFFF0000u : x[k / 2] << 16);
    };
    auto weights = [&](int y0, const uint4 &p, const uint4 &q, double (&w)[VE]) {
#pragma unroll
        for (int k = 0; k < VE; ++k) w[k] = DENSE ? ver_weight(entry(p, k), entry(q, k), R) : fmax((double)entry(p, k), 0.0);
        if (!DENSE)
            for (int i = 0; i < n_lost; ++i) {
                const int at = s.lost[i] - y0;
                if (at >= 0 && at < VE) {
#pragma unroll
                    for (int k = 0; k < VE; ++k) w[k] = at == k ? 0.0 : w[k];
                }
            }
    };
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    // Sum of the weights of groups g0 .. g1-1 over the warp.
    auto sum_groups = [&](int g0, int g1) -> double {
        double acc = 0.0;
        for (int g = g0 + lane; g < g1; g += 64) {
            const int y0 = g * VE - off, y1 = y0 + 32 * VE;
            const bool two = g + 32 < g1;
            const uint4 p0 = load_group(a.p, y0), p1 = two ? load_group(a.p, y1) : zero;
            uint4 q0 = zero, q1 = zero;
            if (DENSE && R > 0.0) {
                q0 = load_group(a.q, y0);
                if (two) q1 = load_group(a.q, y1);
            }
            double w[VE];
            weights(y0, p0, q0, w);
#pragma unroll
            for (int k = 0; k < VE; ++k) acc += w[k];
            if (two) {
                weights(y1, p1, q1, w);
#pragma unroll
                for (int k = 0; k < VE; ++k) acc += w[k];
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
        return acc;
    };
    // Sum of the weights over the row: per warp into s.warp_sum, over the cluster into total.
    auto pass = [&]() {
        set_row();
        const int lo = part_begin(warp);
        const double acc = sum_groups(lo, min(groups, lo + per));
        cl.sync();  // everyone has read the sums of the pass before
        if (lane == 0) s.warp_sum[warp] = acc;
        __syncthreads();
        if (tid == 0) {
            double t = 0.0;
            for (int w = 0; w < kVerWarps; ++w) t += s.warp_sum[w];
            s.cta_sum = t;
        }
        cl.sync();
        total = 0.0;
        for (int k = 0; k < kVerCluster; ++k) total += *cl.map_shared_rank(&s.cta_sum, k);
        have = true;
    };

    if (rank == 0 && tid == 0) a.path[base] = 0;
    for (int c = 1; c < n; ++c) {  // children come after their parent
        if (s.par[c] != cur) continue;
        const double q = DENSE ? (double)s.qx[c] : 1.0;
        double w = DENSE ? fmax(fma(-R, q, (double)s.px[c]), 0.0) : fmax((double)s.px[c], 0.0);
        if (!DENSE)
            for (int k = 0; k < n_lost; ++k) w = s.lost[k] == s.tok[c] ? 0.0 : w;
        if ((double)s.u[c] * (Z * q) < w) {
            cur = c;
            R = 0.0;
            Z = 1.0;
            n_lost = 0;
            have = false;
            if (rank == 0 && tid == 0) a.path[base + count] = c;
            ++count;
        } else if (DENSE) {
            R += Z;
            pass();
            Z = total;
        } else {
            Z -= w;
            __syncthreads();
            if (tid == 0) s.lost[n_lost] = s.tok[c];
            ++n_lost;
            __syncthreads();
        }
    }
    if (!have) pass();
    if (!(total > 0.0 && total < INFINITY)) {  // nothing is left over: from the target's row itself
        R = 0.0;
        n_lost = 0;
        pass();
    }
    const bool ok = total > 0.0 && total < INFINITY;
    if (ok) {
        // r in [0, 1); anything else is brought into it
        const double goal = fmin(fmax((double)a.r[b], 0.0) * total, total * (1.0 - 0x1p-53));
        double run_cta = 0.0;
        for (int k = 0; k < rank; ++k) run_cta += *cl.map_shared_rank(&s.cta_sum, k);
        const double next_cta = run_cta + s.cta_sum;
        double before = run_cta;
        bool tail = true;  // the CTA's last part with weight: it ends where the next CTA begins
        for (int w = 0; w < warp; ++w) before += s.warp_sum[w];
        for (int w = warp + 1; w < kVerWarps; ++w) tail = tail && !(s.warp_sum[w] > 0.0);
        // The parts' ranges of the running sum tile [0, total), so one of them holds the goal (two at
        // a border, where the order of additions decides; the lower index is taken).
        const double mine = s.warp_sum[warp];
        if (mine > 0.0 && goal >= before && goal < (tail ? next_cta : before + mine) && lane == 0) atomicMin(&s.win, warp);
        __syncthreads();
        const int win = s.win;
        if (win < kVerWarps) {  // the CTA's warps share that part: each sums a stretch, then scans it
            double run = run_cta;
            for (int w = 0; w < win; ++w) run += s.warp_sum[w];
            const int part0 = part_begin(win), part1 = min(groups, part0 + per);
            const int stretch = (part1 - part0 + kVerWarps - 1) / kVerWarps;
            const int g0 = min(part1, part0 + warp * stretch), g1 = min(part1, g0 + stretch);
            const double sub = sum_groups(g0, g1);
            if (lane == 0) s.sub_sum[warp] = sub;
            __syncthreads();
            for (int w = 0; w < warp; ++w) run += s.sub_sum[w];
            int pick = -1, last = -1;
            for (int g = g0; g < g1 && pick < 0; g += 32) {
                const int y0 = (g + lane) * VE - off;
                const bool in = g + lane < g1;
                const uint4 p0 = in ? load_group(a.p, y0) : zero;
                const uint4 q0 = DENSE && R > 0.0 && in ? load_group(a.q, y0) : zero;
                double w[VE], x = 0.0;
                weights(y0, p0, q0, w);
                int mine_last = -1;
#pragma unroll
                for (int k = 0; k < VE; ++k) {
                    x += w[k];
                    if (w[k] > 0.0) mine_last = y0 + k;
                }
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const double v = __shfl_up_sync(0xffffffffu, x, o);
                    if (lane >= o) x += v;
                }
                double r2 = __shfl_up_sync(0xffffffffu, x, 1);  // the sum before this lane's group
                r2 = run + (lane == 0 ? 0.0 : r2);
                const unsigned past = __ballot_sync(0xffffffffu, mine_last >= 0 && run + x > goal);
                const unsigned any = __ballot_sync(0xffffffffu, mine_last >= 0);
                int mine_pick = mine_last;
#pragma unroll
                for (int k = VE - 1; k >= 0; --k) {  // the first entry past the goal
                    double r3 = r2;
#pragma unroll
                    for (int i = 0; i <= k; ++i) r3 += w[i];
                    if (w[k] > 0.0 && r3 > goal) mine_pick = y0 + k;
                }
                if (past) pick = __shfl_sync(0xffffffffu, mine_pick, __ffs(past) - 1);
                if (any) last = __shfl_sync(0xffffffffu, mine_last, 31 - __clz(any));
                run += __shfl_sync(0xffffffffu, x, 31);
            }
            if (lane == 0 && pick >= 0) atomicMin(&s.pick, pick);
            if (lane == 0) atomicMax(&s.last, last);
            __syncthreads();
            if (tid == 0 && s.pick == V && s.last >= 0) s.pick = s.last;
        }
    }
    cl.sync();
    if (rank == 0 && tid == 0) {
        int pick = V;
        for (int k = 0; k < kVerCluster; ++k) pick = min(pick, *cl.map_shared_rank(&s.pick, k));
        if (!ok) record_status(FAVOR_ERR_INVALID_ARG);
        a.next[b] = ok && pick < V ? pick : -1;
        a.n_path[b] = count;
    }
    if (rank == 0)
        for (int i = count + tid; i < T; i += kVerThreads) a.path[base + i] = -1;
    cl.sync();  // no CTA leaves while another still reads its shared memory
}

template <bool BF16, bool DENSE>
static cudaError_t launch_verify_t(const VerifyParams &p, cudaStream_t st) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(p.B * kVerCluster);
    cfg.blockDim = dim3(kVerThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kVerCluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_decode_verify<BF16, DENSE>, p);
}

cudaError_t launch_decode_verify(const VerifyParams &p, bool bf16, cudaStream_t st) {
    if (bf16) return p.q ? launch_verify_t<true, true>(p, st) : launch_verify_t<true, false>(p, st);
    return p.q ? launch_verify_t<false, true>(p, st) : launch_verify_t<false, false>(p, st);
}

}  // namespace favor
