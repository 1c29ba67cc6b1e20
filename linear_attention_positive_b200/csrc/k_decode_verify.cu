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
// One cluster of kVerCluster CTAs per sequence, each holding a contiguous slice of the vocabulary,
// every warp a contiguous part of the slice: a pass reads each row once, coalesced, and the sums meet
// through distributed shared memory in a fixed order, so every CTA takes the same branch. The pass is
// bound by HBM latency and bandwidth on the rows it reads.

#include <cooperative_groups.h>

#include "common.cuh"

namespace favor {

constexpr int kVerThreads = 512;
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
    double warp_sum[kVerWarps];
    double cta_sum;            // read by the other CTAs of the cluster
    int pick;                  // the CTA's sampled index, V where it has none
};

template <bool BF16, bool DENSE>
__global__ void __launch_bounds__(kVerThreads) k_decode_verify(VerifyParams a) {
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
    if (tid == 0) s.pick = V;
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
    // this warp's entries of a row
    const int per = (V + kVerCluster * kVerWarps - 1) / (kVerCluster * kVerWarps);
    const int part = rank * kVerWarps + warp;
    const int lo = min(V, part * per), hi = min(V, lo + per);

    int cur = 0, count = 1, n_lost = 0;
    double R = 0.0, Z = 1.0, total = 0.0;
    bool have = false;  // total and the warp sums belong to the current (cur, R)

    auto weight = [&](size_t row, int y) -> double {
        const float p = ver_elem<BF16>(a.p, row + y);
        if (DENSE) return R > 0.0 ? ver_weight(p, ver_elem<BF16>(a.q, row + y), R) : fmax((double)p, 0.0);
        double w = fmax((double)p, 0.0);
        for (int k = 0; k < n_lost; ++k) w = s.lost[k] == y ? 0.0 : w;
        return w;
    };
    // Sum of the weights over the row: per warp into s.warp_sum, over the cluster into total.
    auto pass = [&]() {
        const size_t row = (base + cur) * (size_t)V;
        double acc = 0.0;
        for (int y = lo + lane; y < hi; y += 32) acc += weight(row, y);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
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
        double before = 0.0;
        for (int k = 0; k < rank; ++k) before += *cl.map_shared_rank(&s.cta_sum, k);
        const double next_cta = before + s.cta_sum;
        bool tail = true;  // the CTA's last part with weight: it ends where the next CTA begins
        for (int w = 0; w < warp; ++w) before += s.warp_sum[w];
        for (int w = warp + 1; w < kVerWarps; ++w) tail = tail && !(s.warp_sum[w] > 0.0);
        // The parts' ranges of the running sum tile [0, total), so one of them holds the goal (two at
        // a border, where the order of additions decides; the lower index is taken).
        const double mine = s.warp_sum[warp];
        if (mine > 0.0 && goal >= before && goal < (tail ? next_cta : before + mine)) {
            const size_t row = (base + cur) * (size_t)V;
            int last = -1, pick = -1;
            double run = before;
            for (int y0 = lo; y0 < hi && pick < 0; y0 += 32) {
                const int y = y0 + lane;
                const double w = y < hi ? weight(row, y) : 0.0;
                double x = w;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const double v = __shfl_up_sync(0xffffffffu, x, o);
                    if (lane >= o) x += v;
                }
                const unsigned any = __ballot_sync(0xffffffffu, w > 0.0);
                const unsigned past = __ballot_sync(0xffffffffu, w > 0.0 && run + x > goal);
                if (any) last = y0 + 31 - __clz(any);
                if (past) pick = y0 + __ffs(past) - 1;
                run += __shfl_sync(0xffffffffu, x, 31);
            }
            if (lane == 0) atomicMin(&s.pick, pick >= 0 ? pick : last);
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
