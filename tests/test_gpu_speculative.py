"""GPU parity of the drafted-tree calls (favor_decode_tree, favor_decode_extend, favor_decode_verify)
with the fp64 oracle.

Tolerance: the calls compute with fp32 precision for either input type, so the fp32 bound
1e-4 * RMS of favor_decode_step's tests applies to outputs. Where it comes from: the exponent u of a
feature is a sum of d products in fp32 and its absolute error is its features' relative error. With
|w| <= 16 and |x| <= 5 the d <= 128 products sum in magnitude to at most |w| |x| <= 80; each partial
sum is rounded by at most 80 2^-24, in all 128 * 80 * 6e-8 = 6e-4 at worst, and 1/sqrt(128) of that
(5e-5) with the roundings' signs mixed; outputs average features, which lowers it further. State
entries are compared per entry relative to the largest of their kind, with the same 1e-4."""

import numpy as np
import pytest
import torch

from linear_attention_positive_b200 import api
from oracle import speculative
from tests.helpers import features_for, rel_max_err, to_torch

pytestmark = pytest.mark.gpu

TOL = 1e-4


class Problem:
    """Seeded tokens, features and a carried state (after ``prior`` tokens) on both sides."""

    def __init__(self, B, H, T, d, m, dtype, device, prior=40, seed=0):
        g = np.random.default_rng(seed)
        self.B, self.H, self.T, self.d, self.m, self.dtype, self.device = B, H, T, d, m, dtype, device
        self.g = g
        self.Wr, self.W64 = features_for(3, m, d, dtype)
        self.W = to_torch(self.Wr, dtype, device)
        self.q, self.k, self.v = (self.tokens(T, d ** -0.25 if i < 2 else 1.0) for i in range(3))
        self.prior = [self.tokens(prior, d ** -0.25 if i < 2 else 1.0) for i in range(3)] if prior else None
        self.state = api.decode_state(B, H, d, m, device)
        for t in range(prior):
            api.decode_step(*(x[:, :, t].contiguous() for x in self.prior), self.W, self.state)

    def tokens(self, n, scale):
        return to_torch(self.g.standard_normal((self.B, self.H, n, self.d)) * scale, self.dtype, self.device)

    def head(self, x, b, h):
        return x[b, h].double().cpu().numpy()

    def oracle_state(self, b, h):
        S, z = np.zeros((self.m, self.d)), np.zeros(self.m)
        if self.prior is None:
            return S, z
        return speculative.decode_extend(S, z, self.head(self.prior[1], b, h), self.head(self.prior[2], b, h), self.W64)

    def gpu_state(self, state=None):
        """True sums S [B,H,m,d], z [B,H,m] of a device state, in the oracle's scale."""
        t = (self.state if state is None else state).double().cpu().numpy().reshape(self.B, self.H, self.d + 2, self.m)
        scale = np.where(t[:, :, self.d] != 0, np.exp(t[:, :, self.d + 1]), 0.0) / np.sqrt(self.m)
        return np.swapaxes(t[:, :, : self.d] * scale[:, :, None], 2, 3), t[:, :, self.d] * scale

    def oracle_tree(self, parents, n_nodes=None):
        out = np.full((self.B, self.H, self.T, self.d), np.nan)
        for b in range(self.B):
            n = self.T if n_nodes is None else n_nodes[b]
            for h in range(self.H):
                S, z = self.oracle_state(b, h)
                X = [self.head(x, b, h)[:n] for x in (self.q, self.k, self.v)]
                out[b, h, :n] = speculative.decode_tree(S, z, *X, self.W64, list(parents[b][:n]))
        return out


def i32(x, device):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=device)


def random_parents(B, T, seed=0, reach=12):
    g = np.random.default_rng(seed)
    return np.array([[-1 if i == 0 else int(g.integers(max(0, i - reach), i)) for i in range(T)] for _ in range(B)])


def status_ok():
    assert api.sync_status() == api.FAVOR_OK


# --------------------------------------------------------------------------------------------- tree

SHAPES = [(1, 1, 1, 64, 32), (2, 3, 1, 128, 256), (2, 2, 2, 64, 96), (1, 2, 4, 64, 256), (2, 2, 5, 128, 160),
          (2, 2, 16, 64, 128), (1, 3, 17, 64, 256), (2, 2, 33, 128, 96), (2, 2, 64, 64, 256), (1, 2, 65, 64, 224),
          (1, 2, 127, 128, 128), (1, 1, 128, 128, 256), (1, 2, 128, 64, 256), (3, 5, 40, 64, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("prior", [40, 0])
@pytest.mark.parametrize("B,H,T,d,m", SHAPES)
def test_tree_matches_oracle(cuda_device, dtype, prior, B, H, T, d, m):
    x = Problem(B, H, T, d, m, dtype, cuda_device, prior=prior, seed=T)
    parents = random_parents(B, T, seed=T)
    before = x.state.clone()
    out = api.decode_tree(x.q, x.k, x.v, x.W, x.state, i32(parents, cuda_device))
    status_ok()
    assert rel_max_err(out.double().cpu().numpy(), x.oracle_tree(parents)) <= TOL
    assert torch.equal(before, x.state)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["chain", "star", "forest"])
@pytest.mark.parametrize("T", [3, 48, 128])
def test_tree_shapes_at_the_extremes(cuda_device, dtype, kind, T):
    """A chain (every row sees all before it), a star (two nodes a row) and a forest of lone roots."""
    x = Problem(2, 2, T, 64, 256, dtype, cuda_device, seed=5)
    one = {"chain": np.arange(T) - 1, "star": np.where(np.arange(T) > 0, 0, -1), "forest": np.full(T, -1)}[kind]
    parents = np.stack([one] * 2)
    out = api.decode_tree(x.q, x.k, x.v, x.W, x.state, i32(parents, cuda_device))
    status_ok()
    assert rel_max_err(out.double().cpu().numpy(), x.oracle_tree(parents)) <= TOL


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tree_chain_is_repeated_steps(cuda_device, dtype):
    x = Problem(2, 3, 24, 64, 256, dtype, cuda_device, seed=9)
    parents = np.stack([np.arange(24) - 1] * 2)
    out = api.decode_tree(x.q, x.k, x.v, x.W, x.state, i32(parents, cuda_device))
    steps = [api.decode_step(*(y[:, :, t].contiguous() for y in (x.q, x.k, x.v)), x.W, x.state) for t in range(24)]
    status_ok()
    assert rel_max_err(out.double().cpu().numpy(), torch.stack(steps, 2).double().cpu().numpy()) <= TOL


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,T", [(64, 70), (128, 24)])
def test_tree_padding_is_neither_read_nor_written(cuda_device, dtype, d, T):
    x = Problem(4, 2, T, d, 128, dtype, cuda_device, seed=3)
    counts = [T, 0, 1, T // 2 + 1]
    parents = random_parents(4, T, seed=3)
    for b, n in enumerate(counts):
        for y in (x.q, x.k, x.v):
            y[b, :, n:] = float("nan")
        parents[b, n:] = 10**6
    out = torch.full((4, 2, T, d), 7.0, device=cuda_device)
    api.decode_tree(x.q, x.k, x.v, x.W, x.state, i32(parents, cuda_device), n_nodes=i32(counts, cuda_device), out=out)
    status_ok()
    ref = x.oracle_tree(parents, counts)
    got = out.double().cpu().numpy()
    for b, n in enumerate(counts):
        assert (got[b, :, n:] == 7.0).all()
        if n:
            assert rel_max_err(got[b, :, :n], ref[b, :, :n]) <= TOL


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["k", "v", "q"])
def test_tree_unseen_nodes_do_not_reach_a_row(cuda_device, dtype, bad, where):
    """Node 5 holds NaN or infinities; only the rows below it may show them."""
    T = 40
    x = Problem(1, 2, T, 64, 256, dtype, cuda_device, seed=4)
    parents = random_parents(1, T, seed=4)
    ref = x.oracle_tree(parents)
    getattr(x, where)[:, :, 5] = bad
    out = api.decode_tree(x.q, x.k, x.v, x.W, x.state, i32(parents, cuda_device))
    status_ok()
    got = out.double().cpu().numpy()
    sees = [5 in speculative.ancestors(list(parents[0]), i) if where != "q" else i == 5 for i in range(T)]
    clean = [i for i in range(T) if not sees[i]]
    assert rel_max_err(got[:, :, clean], ref[:, :, clean]) <= TOL
    if where == "v":  # what a row does see, it shows
        dirty = [i for i in range(T) if sees[i]]
        assert not np.isfinite(got[:, :, dirty]).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [4.0, 8.0])
@pytest.mark.parametrize("prior", [40, 0])
def test_tree_unseen_nodes_with_far_larger_logits(cuda_device, dtype, scale, prior):
    """Keys of very different norms and directions in one tree: features that unseen nodes dominate by
    hundreds of nats leave a row its own terms. The exponents reach |w| |x| ~ 16 * 40, so the
    tolerance grows with them: u's rounding error is 640 / 80 of the bound above."""
    T = 48
    x = Problem(1, 2, T, 64, 128, dtype, cuda_device, prior=prior, seed=6)
    parents = random_parents(1, T, seed=6, reach=30)
    x.k[:, :, 3::4] *= scale
    x.q[:, :, 1::3] *= -scale
    out = api.decode_tree(x.q, x.k, x.v, x.W, x.state, i32(parents, cuda_device))
    status_ok()
    got, ref = out.double().cpu().numpy(), x.oracle_tree(parents)
    assert np.isfinite(got).all()
    assert rel_max_err(got, ref) <= 8 * TOL


def tree_from_state(x, state, parents, n_nodes, heads):
    """Rows by the fp64 definition over the sums a device state holds, for some (b, h)."""
    S, z = x.gpu_state(state)
    return {(b, h): speculative.decode_tree(S[b, h], z[b, h], *(x.head(t, b, h)[: n_nodes[b]] for t in (x.q, x.k, x.v)),
                                            x.W64, list(parents[b][: n_nodes[b]])) for b, h in heads}


@pytest.mark.parametrize("T,d,m", [(64, 64, 256), (64, 128, 256), (100, 64, 256), (100, 128, 128), (17, 64, 96), (6, 64, 256)])
def test_tree_of_a_full_batch(cuda_device, T, d, m):
    """More heads than fit the device at once, sequences cut differently (some heads checked)."""
    B, H = 25, 16
    x = Problem(B, H, T, d, m, "bf16", cuda_device, prior=0, seed=T + d)
    state = api.decode_extend(x.tokens(70, d ** -0.25), x.tokens(70, 1.0), x.W, x.state)
    parents = random_parents(B, T, seed=T)
    counts = np.random.default_rng(T).integers(0, T + 1, B)
    counts[:4] = T, 0, 1, T - 1
    out = torch.full((B, H, T, d), 7.0, device=cuda_device)
    api.decode_tree(x.q, x.k, x.v, x.W, state, i32(parents, cuda_device), n_nodes=i32(counts, cuda_device), out=out)
    status_ok()
    got = out.double().cpu().numpy()
    heads = [(0, 0), (0, 15), (2, 5), (3, 1), (9, 9), (17, 3), (24, 15)]
    for (b, h), ref in tree_from_state(x, state, parents, counts, heads).items():
        assert rel_max_err(got[b, h, : counts[b]], ref) <= TOL if counts[b] else True
    for b in range(B):
        assert (got[b, :, counts[b]:] == 7.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("prior", [1, 3, 12])
@pytest.mark.parametrize("T,d", [(64, 64), (64, 128), (120, 64), (3, 64)])
def test_tree_behind_a_short_context(cuda_device, dtype, prior, T, d):
    """The tree's keys lie far above what a few tokens left in the state."""
    x = Problem(2, 3, T, d, 256, dtype, cuda_device, prior=prior, seed=prior + T)
    parents = random_parents(2, T, seed=T)
    out = api.decode_tree(x.q, x.k, x.v, x.W, x.state, i32(parents, cuda_device))
    status_ok()
    assert rel_max_err(out.double().cpu().numpy(), x.oracle_tree(parents)) <= TOL


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("factor", [2.0**40, 2.0**-40, 0.0])
def test_tree_over_features_of_very_different_sums(cuda_device, dtype, factor):
    """S' of the features from 64 on scaled away from the others' (also beyond what fp16 spans)."""
    x = Problem(1, 2, 40, 64, 192, dtype, cuda_device, seed=50)
    state = x.state.clone()
    state.view(2, 66, 192)[:, :64, 64:] *= factor
    parents = random_parents(1, 40, seed=50)
    out = api.decode_tree(x.q, x.k, x.v, x.W, state, i32(parents, cuda_device)).double().cpu().numpy()
    status_ok()
    for (b, h), ref in tree_from_state(x, state, parents, [40], [(0, 0), (0, 1)]).items():
        assert rel_max_err(out[b, h], ref) <= TOL


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,m", [(1, 64, 256), (2, 128, 96), (3, 64, 32), (4, 128, 256), (4, 64, 256)])
def test_tree_of_few_nodes_of_a_full_batch(cuda_device, dtype, T, d, m):
    """Up to four nodes in more heads than fit the device at once, counts cut differently (some heads checked)."""
    B, H = 25, 16
    x = Problem(B, H, T, d, m, dtype, cuda_device, prior=0, seed=T + d)
    state = api.decode_extend(x.tokens(70, d ** -0.25), x.tokens(70, 1.0), x.W, x.state)
    parents = random_parents(B, T, seed=T, reach=2)
    counts = np.random.default_rng(T).integers(0, T + 1, B)
    counts[:3] = T, 0, 1
    out = torch.full((B, H, T, d), 7.0, device=cuda_device)
    api.decode_tree(x.q, x.k, x.v, x.W, state, i32(parents, cuda_device), n_nodes=i32(counts, cuda_device), out=out)
    status_ok()
    got = out.double().cpu().numpy()
    for (b, h), ref in tree_from_state(x, state, parents, counts, [(0, 0), (0, 15), (2, 5), (9, 9), (24, 15)]).items():
        assert rel_max_err(got[b, h, : counts[b]], ref) <= TOL if counts[b] else True
    for b in range(B):
        assert (got[b, :, counts[b]:] == 7.0).all()


def column_scales(d, lowest, device):
    """Powers of two from 1 down to 2^lowest, one per value column, neighbours far apart (exact in any type)."""
    e = torch.round(torch.linspace(0, lowest, d))[torch.randperm(d, generator=torch.Generator().manual_seed(d))]
    return torch.exp2(e).to(device)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lowest", [-20, -60])
@pytest.mark.parametrize("B,H,T,d,m", [(1, 2, 40, 64, 256), (1, 2, 100, 128, 128), (25, 16, 64, 64, 256), (25, 16, 30, 128, 96),
                                       (25, 16, 100, 64, 128), (1, 2, 12, 64, 256), (1, 2, 4, 128, 64)])
def test_tree_value_columns_of_very_different_size(cuda_device, dtype, lowest, B, H, T, d, m):
    """Each output column to the tolerance of its own largest entry (some heads checked)."""
    x = Problem(B, H, T, d, m, dtype, cuda_device, prior=0, seed=T + d)
    scales = column_scales(d, lowest, cuda_device).to(x.v.dtype)
    x.v *= scales
    state = api.decode_extend(x.tokens(50, d ** -0.25), x.tokens(50, 1.0) * scales, x.W, x.state)
    parents = random_parents(B, T, seed=T)
    out = api.decode_tree(x.q, x.k, x.v, x.W, state, i32(parents, cuda_device)).double().cpu().numpy()
    status_ok()
    for (b, h), ref in tree_from_state(x, state, parents, [T] * B, [(0, 0), (0, 1), (B - 1, H - 1)]).items():
        assert (np.abs(out[b, h] - ref).max(0) <= TOL * np.abs(ref).max(0)).all()


@pytest.mark.parametrize("factor", [1.0, 2.0**-30, 2.0**30])
def test_tree_value_columns_that_only_later_features_hold(cuda_device, factor):
    """Columns of S' that are 0 in the first 64 features, whose size the column's scale comes from."""
    x = Problem(1, 2, 40, 64, 192, "bf16", cuda_device, seed=51)
    state = x.state.clone()
    state.view(2, 66, 192)[:, 3:9, :64] = 0
    state.view(2, 66, 192)[:, 3:9] *= factor
    x.v[:, :, :, 3:9] *= factor
    parents = random_parents(1, 40, seed=51)
    out = api.decode_tree(x.q, x.k, x.v, x.W, state, i32(parents, cuda_device)).double().cpu().numpy()
    status_ok()
    for (b, h), ref in tree_from_state(x, state, parents, [40], [(0, 0), (0, 1)]).items():
        assert (np.abs(out[b, h] - ref).max(0) <= TOL * np.abs(ref).max(0)).all()


@pytest.mark.parametrize("T,d,m,prior,scale", [(64, 64, 32, 2, 2.0), (64, 64, 32, 0, 3.0), (60, 128, 32, 1, 1.0), (100, 64, 32, 2, 2.0)])
def test_tree_rows_whose_terms_lie_below_the_scales_of_others(cuda_device, T, d, m, prior, scale):
    """Many roots over a short context, all heads: rows whose own terms are small next to what sets the features'
    scales. |w| |x| stays within the 80 of the bound above (|w| ~ 11, |x| ~ 7), so its tolerance applies."""
    B, H = 16, 8
    x = Problem(B, H, T, d, m, "bf16", cuda_device, prior=0, seed=m + T)
    x.q *= min(scale, 2.0)
    x.k *= scale
    state = x.state
    if prior:
        state = api.decode_extend(x.tokens(prior, scale * d ** -0.25), x.tokens(prior, 1.0), x.W, state)
    parents = random_parents(B, T, seed=T, reach=8)
    parents[:, ::3] = -1
    out = api.decode_tree(x.q, x.k, x.v, x.W, state, i32(parents, cuda_device)).double().cpu().numpy()
    status_ok()
    heads = [(b, h) for b in range(B) for h in range(H)]
    ref = tree_from_state(x, state, parents, [T] * B, heads)
    ref = np.stack([ref[at] for at in heads]).reshape(out.shape)
    assert rel_max_err(out, ref) <= TOL


@pytest.mark.parametrize("T,d,m", [(40, 64, 256), (64, 64, 160), (60, 128, 256), (100, 64, 256), (100, 128, 256), (40, 64, 64)])
def test_tree_equal_values_come_out_as_they_are(cuda_device, T, d, m):
    """Values of 1 everywhere give 1: numerator and denominator are the same sums. The tensor core's additions
    truncate, each by less than 2^-23 of the accumulator. Per 128 features eight of them see a full one (above 64
    nodes at d = 128, where 64 features are taken at a time, sixteen); the operands' parts add 2^-23 at most."""
    x = Problem(8, 8, T, d, m, "bf16", cuda_device, prior=0, seed=m + T)
    state = api.decode_extend(x.tokens(70, d ** -0.25), x.tokens(70, 1.0), x.W, x.state).view(64, d + 2, m)
    state[:, :d] = state[:, d:d + 1]
    x.v.fill_(1)
    out = api.decode_tree(x.q, x.k, x.v, x.W, state.view(-1), i32(random_parents(8, T, seed=T), cuda_device))
    status_ok()
    steps = 16 if T > 64 and d == 128 else 8
    assert abs(out.double().mean().item() - 1) <= (steps + 1) * 2.0**-23
    assert (out - 1).abs().max().item() <= TOL


def test_tree_bad_parents_and_counts_are_recorded(cuda_device):
    T = 20
    x = Problem(2, 2, T, 64, 128, "bf16", cuda_device, seed=8)
    parents = random_parents(2, T, seed=8)
    read = parents.copy()
    for i, p in ((3, 3), (7, 12), (9, -5), (11, 2**30)):
        parents[1, i], read[1, i] = p, -1
    out = api.decode_tree(x.q, x.k, x.v, x.W, x.state, i32(parents, cuda_device), n_nodes=i32([T, T], cuda_device))
    assert api.sync_status() == api.FAVOR_ERR_INVALID_ARG
    assert rel_max_err(out.double().cpu().numpy(), x.oracle_tree(read)) <= TOL
    out = api.decode_tree(x.q, x.k, x.v, x.W, x.state, i32(read, cuda_device), n_nodes=i32([T + 5, -1], cuda_device),
                          out=torch.zeros_like(out))
    assert api.sync_status() == api.FAVOR_ERR_INVALID_ARG
    assert rel_max_err(out[0].double().cpu().numpy(), x.oracle_tree(read)[0]) <= TOL and (out[1] == 0).all()
    status_ok()


# ------------------------------------------------------------------------------------------- extend

def check_state(x, state, chosen):
    """A device state against the oracle's after adding the chosen token positions of each sequence."""
    S, z = x.gpu_state(state)
    for b in range(x.B):
        for h in range(x.H):
            S0, z0 = x.oracle_state(b, h)
            Sr, zr = speculative.decode_extend(S0, z0, x.head(x.k, b, h), x.head(x.v, b, h), x.W64, chosen[b])
            assert np.abs(S[b, h] - Sr).max() <= TOL * np.abs(Sr).max()
            assert np.abs(z[b, h] - zr).max() <= TOL * np.abs(zr).max()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("prior", [40, 0])
@pytest.mark.parametrize("B,H,L,d,m", [(1, 1, 1, 64, 32), (2, 3, 7, 128, 256), (2, 2, 32, 64, 96), (2, 2, 33, 64, 256),
                                       (1, 3, 129, 128, 160), (2, 2, 500, 64, 128), (1, 2, 1500, 128, 256),
                                       (1, 2, 3001, 64, 256), (3, 1, 900, 64, 224)])
def test_extend_matches_oracle(cuda_device, dtype, prior, B, H, L, d, m):
    x = Problem(B, H, L, d, m, dtype, cuda_device, prior=prior, seed=L)
    old = x.state.clone()
    state = api.decode_extend(x.k, x.v, x.W, x.state)
    status_ok()
    assert state is x.state
    check_state(x, state, [None] * B)
    # D is the largest logit so far
    t = state.view(B, H, d + 2, m)[:, :, d + 1].double().cpu().numpy()
    for b in range(B):
        for h in range(H):
            k = np.concatenate([x.head(x.k, b, h)] + ([x.head(x.prior[1], b, h)] if prior else []))
            u = (k @ x.W64.T - 0.5 * (k * k).sum(1, keepdims=True)).max(0)
            assert np.abs(t[b, h] - u).max() <= TOL
    # the same bits again
    again = api.decode_extend(x.k, x.v, x.W, old)
    assert torch.equal(again, state)


@pytest.mark.parametrize("L,d,m", [(1300, 64, 256), (1300, 128, 256), (1153, 64, 96), (640, 128, 128), (257, 64, 128), (65, 64, 256), (128, 128, 256)])
def test_extend_runs_of_many_tiles(cuda_device, L, d, m):
    """Enough heads that each takes its tokens in one or two long runs (some heads checked)."""
    B, H = 20, 16
    x = Problem(B, H, L, d, m, "bf16", cuda_device, prior=0, seed=L)
    counts = np.random.default_rng(L).integers(0, L + 1, B)
    counts[:3] = L, 0, L - 1
    state = api.decode_extend(x.k, x.v, x.W, x.state, counts=i32(counts, cuda_device))
    status_ok()
    S, z = x.gpu_state(state)
    for b, h in [(0, 0), (0, 15), (1, 7), (2, 3), (3, 1), (11, 9), (19, 15)]:
        n = int(counts[b])
        Sr, zr = speculative.decode_extend(np.zeros((m, d)), np.zeros(m), x.head(x.k, b, h)[:n], x.head(x.v, b, h)[:n], x.W64)
        assert np.abs(S[b, h] - Sr).max() <= TOL * np.abs(Sr).max()
        assert np.abs(z[b, h] - zr).max() <= TOL * np.abs(zr).max()


@pytest.mark.parametrize("dtype,indexed", [("f32", False), ("f32", True), ("bf16", True)])
@pytest.mark.parametrize("L,d,m", [(100, 64, 256), (100, 128, 96), (33, 128, 256), (17, 64, 32)])
def test_extend_rows_of_a_full_batch(cuda_device, dtype, indexed, L, d, m):
    """More heads than fit the device at once, counts cut differently, fp32 or by index (some heads checked)."""
    B, H = 25, 16
    x = Problem(B, H, L, d, m, dtype, cuda_device, prior=0, seed=L + d)
    g = np.random.default_rng(L)
    counts = g.integers(0, L + 1, B)
    counts[:3] = L, 0, 1
    index = np.stack([g.permutation(L) for _ in range(B)])
    state = x.state
    for _ in range(2):  # into the empty state, then onto itself
        state = api.decode_extend(x.k, x.v, x.W, state, index=i32(index, cuda_device) if indexed else None,
                                  counts=i32(counts, cuda_device))
    status_ok()
    S, z = x.gpu_state(state)
    for b, h in [(0, 0), (0, 15), (1, 7), (2, 3), (8, 1), (16, 9), (24, 15)]:
        n = int(counts[b])
        at = index[b, :n] if indexed else np.arange(n)
        Sr, zr = np.zeros((m, d)), np.zeros(m)
        for _ in range(2):
            Sr, zr = speculative.decode_extend(Sr, zr, x.head(x.k, b, h)[at], x.head(x.v, b, h)[at], x.W64)
        assert np.abs(S[b, h] - Sr).max() <= TOL * np.abs(Sr).max()
        assert np.abs(z[b, h] - zr).max() <= TOL * np.abs(zr).max()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L,d,m", [(64, 64, 256), (64, 128, 96), (2000, 64, 256), (700, 128, 128)])
def test_extend_counts_and_padding(cuda_device, dtype, L, d, m):
    x = Problem(4, 2, L, d, m, dtype, cuda_device, seed=L + 1)
    counts = [L, 0, 1, L // 3]
    for b, n in enumerate(counts):
        x.k[b, :, n:] = float("nan")
        x.v[b, :, n:] = float("inf")
    old = x.state.clone()
    state = api.decode_extend(x.k, x.v, x.W, x.state, counts=i32(counts, cuda_device))
    status_ok()
    check_state(x, state, [list(range(n)) for n in counts])
    assert torch.equal(state.view(4, -1)[1], old.view(4, -1)[1])  # bit for bit


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [1, 9, 60])
def test_extend_by_index(cuda_device, dtype, N):
    """An accepted path, the same position twice, and positions in any order."""
    L = 64
    x = Problem(3, 2, L, 64, 256, dtype, cuda_device, seed=N)
    index = x.g.integers(0, L, (3, N))
    counts = [N, max(N - 2, 1), 0]
    state = api.decode_extend(x.k, x.v, x.W, x.state, index=i32(index, cuda_device), counts=i32(counts, cuda_device))
    status_ok()
    check_state(x, state, [index[b, :n].tolist() for b, n in enumerate(counts)])


def test_extend_bad_index_and_counts_are_recorded(cuda_device):
    L = 40
    x = Problem(2, 2, L, 64, 128, "bf16", cuda_device, seed=2)
    index = np.array([[3, L, 5, -1, 7], [L + 9, -3, 2**30, L, -1]])
    old = x.state.clone()
    state = api.decode_extend(x.k, x.v, x.W, x.state, index=i32(index, cuda_device))
    assert api.sync_status() == api.FAVOR_ERR_INVALID_ARG
    check_state(x, state, [[3, 5, 7], []])
    state = api.decode_extend(x.k, x.v, x.W, old, counts=i32([L + 1, -7], cuda_device))
    assert api.sync_status() == api.FAVOR_ERR_INVALID_ARG
    check_state(x, state, [list(range(L)), []])
    status_ok()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L", [20, 700])
def test_extend_keys_far_above_and_below_earlier_ones(cuda_device, dtype, L):
    """Keys whose logits jump by tens of nats over earlier ones (rescaling what was summed), and keys far
    below them (nothing may turn into NaN)."""
    x = Problem(1, 2, L, 64, 128, dtype, cuda_device, seed=1)
    x.k[:, :, L // 2] = (0.9 * x.W[0].float()).to(x.k.dtype)
    x.k[:, :, L - 3:] *= 12
    state = api.decode_extend(x.k, x.v, x.W, x.state)
    status_ok()
    t = state.view(2, 66, 128).double().cpu().numpy()
    assert np.isfinite(t).all()
    # per feature, relative to that feature's own sums: u reaches |w| |x| ~ 16 * 34, 7 times the bound above
    for h in range(2):
        S0, z0 = x.oracle_state(0, h)
        Sr, zr = speculative.decode_extend(S0, z0, x.head(x.k, 0, h), x.head(x.v, 0, h), x.W64)
        S, z = x.gpu_state(state)
        assert (np.abs(z[0, h] - zr) <= 7 * TOL * zr).all()
        assert (np.abs(S[0, h] - Sr) <= 7 * TOL * np.abs(Sr).max(1, keepdims=True)).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("at", [[500], [63, 64, 700], [200, 330, 460, 590, 720, 1000]])
def test_extend_keys_far_above_within_a_run_of_many_tiles(cuda_device, d, at):
    """Each head takes its tokens in one or two runs of many tiles; keys along a row of W raise D_r in the middle
    (some heads checked, per feature; u reaches |w| |x| ~ 16 * 16, 4 times the bound above)."""
    B, H, L, m = 20, 8, 1100, 256
    x = Problem(B, H, L, d, m, "bf16", cuda_device, prior=0, seed=d)
    for n, j in enumerate(at):
        x.k[:, :, j] = (0.9 * x.W[17 * n].float()).to(x.k.dtype)
    state = api.decode_extend(x.k, x.v, x.W, x.state)
    status_ok()
    S, z = x.gpu_state(state)
    for b, h in [(0, 0), (7, 3), (13, 7), (19, 7)]:
        Sr, zr = speculative.decode_extend(np.zeros((m, d)), np.zeros(m), x.head(x.k, b, h), x.head(x.v, b, h), x.W64)
        assert (np.abs(z[b, h] - zr) <= 4 * TOL * zr).all()
        assert (np.abs(S[b, h] - Sr) <= 4 * TOL * np.abs(Sr).max(1, keepdims=True)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("factor", [2.0**-40, 2.0**30])
def test_extend_values_of_any_size(cuda_device, dtype, factor):
    x = Problem(1, 2, 600, 64, 256, dtype, cuda_device, prior=0, seed=12)
    x.v *= factor
    state = api.decode_extend(x.k, x.v, x.W, x.state)
    status_ok()
    check_state(x, state, [None])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_extend_values_that_grow_along_the_sequence(cuda_device, dtype):
    """Value magnitudes 2^-30 .. 2^33 in one sequence, growing and falling."""
    L = 1100
    x = Problem(1, 2, L, 64, 128, dtype, cuda_device, prior=0, seed=13)
    e = torch.linspace(-30, 33, L // 2, device=cuda_device).floor()
    x.v *= torch.exp2(torch.cat([e, e.flip(0)]))[:, None].to(x.v.dtype)
    state = api.decode_extend(x.k, x.v, x.W, x.state)
    status_ok()
    check_state(x, state, [None])


@pytest.mark.parametrize("dtype,indexed", [("bf16", False), ("bf16", True), ("f32", False)])
@pytest.mark.parametrize("lowest", [-20, -60])
@pytest.mark.parametrize("L,d,m", [(64, 64, 256), (700, 64, 128), (700, 128, 128), (2500, 64, 96), (13, 128, 256)])
def test_extend_value_columns_of_very_different_size(cuda_device, dtype, indexed, lowest, L, d, m):
    """Each column of S' to the tolerance of its own largest entry."""
    x = Problem(1, 2, L, d, m, dtype, cuda_device, prior=0, seed=L + d)
    x.v *= column_scales(d, lowest, cuda_device).to(x.v.dtype)
    state = api.decode_extend(x.k, x.v, x.W, x.state, index=i32([np.arange(L)], cuda_device) if indexed else None)
    status_ok()
    S, z = x.gpu_state(state)
    for h in range(2):
        Sr, zr = speculative.decode_extend(np.zeros((m, d)), np.zeros(m), x.head(x.k, 0, h), x.head(x.v, 0, h), x.W64)
        assert (np.abs(S[0, h] - Sr).max(0) <= TOL * np.abs(Sr).max(0)).all()


@pytest.mark.parametrize("dtype,indexed", [("bf16", False), ("bf16", True), ("f32", False)])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("L,d,at", [(700, 64, 130), (700, 128, 699), (1300, 64, 0), (12, 64, 3)])
def test_extend_a_value_that_is_not_finite_stays_in_its_column(cuda_device, dtype, indexed, bad, L, d, at):
    """What the single-token step does: the other columns of S', z' and D are as ever."""
    x = Problem(1, 2, L, d, 128, dtype, cuda_device, prior=5, seed=L + at)
    x.v[:, :, at, 7] = bad
    state = api.decode_extend(x.k, x.v, x.W, x.state, index=i32([np.arange(L)], cuda_device) if indexed else None)
    status_ok()
    S, z = x.gpu_state(state)
    rest = [c for c in range(d) if c != 7]
    for h in range(2):
        S0, z0 = x.oracle_state(0, h)
        v = x.head(x.v, 0, h)
        v[at, 7] = 0.0
        Sr, zr = speculative.decode_extend(S0, z0, x.head(x.k, 0, h), v, x.W64)
        assert np.abs(S[0, h] - Sr)[:, rest].max() <= TOL * np.abs(Sr).max()
        assert np.abs(z[0, h] - zr).max() <= TOL * np.abs(zr).max()
        assert not np.isfinite(S[0, h][:, 7]).any()


def test_extend_then_step_continues_the_sequence(cuda_device):
    """A prompt through decode_extend, then single tokens: the rows of the causal forward."""
    from oracle import favor

    L, n = 300, 8
    x = Problem(1, 2, L + n, 64, 256, "f32", cuda_device, prior=0, seed=21)
    state = api.decode_extend(x.k[:, :, :L].contiguous(), x.v[:, :, :L].contiguous(), x.W, x.state)
    outs = [api.decode_step(*(y[:, :, t].contiguous() for y in (x.q, x.k, x.v)), x.W, state) for t in range(L, L + n)]
    status_ok()
    got = torch.stack(outs, 2).double().cpu().numpy()
    ref = favor.fwd(*(y.double().cpu().numpy() for y in (x.q, x.k, x.v)), x.W64, causal=True)[:, :, L:]
    assert rel_max_err(got, ref) <= TOL


# ------------------------------------------------------------------------------------------- verify

def draft(B, T, V, dtype, device, seed=0, spread=2.0):
    g = np.random.default_rng(seed)
    logits = g.standard_normal((B, T, V)) * spread
    other = logits + g.standard_normal((B, T, V)) * 0.7
    p, q = (torch.softmax(torch.tensor(a), -1).float() for a in (logits, other))
    if dtype == "bf16":
        p, q = p.to(torch.bfloat16), q.to(torch.bfloat16)
    parents = random_parents(B, T, seed=seed, reach=4)
    tokens = np.zeros((B, T), dtype=np.int64)
    for b in range(B):
        for c in range(1, T):
            w = q[b, parents[b, c]].double().numpy()
            tokens[b, c] = g.choice(V, p=w / w.sum())
    u, r = g.random((B, T)).astype(np.float32), g.random(B).astype(np.float32)
    return dict(parents=parents, tokens=tokens, p=p.to(device), q=q.to(device), u=u, r=r)


def run_verify(x, device, dense=True, n_nodes=None):
    got = api.decode_verify(i32(x["parents"], device), i32(x["tokens"], device), x["p"],
                            torch.tensor(x["u"], device=device), torch.tensor(x["r"], device=device),
                            q=x["q"] if dense else None,
                            n_nodes=None if n_nodes is None else i32(n_nodes, device))
    return [t.cpu().numpy() for t in got]


def check_verify(x, got, dense=True, n_nodes=None):
    path, count, token = got
    B, T = path.shape
    for b in range(B):
        n = T if n_nodes is None else n_nodes[b]
        if n == 0:
            assert count[b] == 0 and token[b] == -1 and (path[b] == -1).all()
            continue
        ref, nxt = speculative.verify(x["parents"][b][:n], x["tokens"][b], x["p"][b].double().cpu().numpy(),
                                      x["q"][b].double().cpu().numpy() if dense else None,
                                      x["u"][b].astype(np.float64), float(x["r"][b]))
        assert path[b].tolist() == ref + [-1] * (T - len(ref)) and count[b] == len(ref)
        assert token[b] == nxt


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dense", [True, False])
@pytest.mark.parametrize("B,T,V", [(1, 1, 1), (3, 2, 5), (2, 8, 31), (9, 16, 257), (1, 8, 32000), (4, 12, 5003),
                                   (24, 128, 1001), (2, 3, 131072), (70, 20, 640)])
def test_verify_matches_oracle(cuda_device, dtype, dense, B, T, V):
    x = draft(B, T, V, dtype, cuda_device, seed=B + T)
    got = run_verify(x, cuda_device, dense)
    status_ok()
    check_verify(x, got, dense)


@pytest.mark.parametrize("dense", [True, False])
def test_verify_ragged(cuda_device, dense):
    x = draft(12, 24, 999, "f32", cuda_device, seed=5)
    counts = [0, 1, 2, 24, 7, 0, 24, 12, 3, 23, 5, 1]
    for b, n in enumerate(counts):  # nothing behind a sequence's nodes is looked at
        x["parents"][b, n:], x["tokens"][b, n:], x["p"][b, n:] = 10**6, -(10**6), float("nan")
    got = run_verify(x, cuda_device, dense, counts)
    status_ok()
    check_verify(x, got, dense, counts)


@pytest.mark.parametrize("dense", [True, False])
def test_verify_all_siblings_and_chains(cuda_device, dense):
    """Many rejections at one node (repeated tokens among the siblings), and a chain accepted whole."""
    T, V = 60, 700
    x = draft(6, T, V, "f32", cuda_device, seed=6, spread=0.5)
    x["parents"][:3] = np.where(np.arange(T) > 0, 0, -1)
    x["u"][:3] = 0.9999
    x["tokens"][:3] %= 40
    x["parents"][3:] = np.arange(T) - 1
    x["u"][3:] = 0.0
    got = run_verify(x, cuda_device, dense)
    status_ok()
    check_verify(x, got, dense)
    assert (got[1][3:] == T).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_verify_sample_numbers_at_their_ends(cuda_device, dtype):
    x = draft(8, 1, 4000, dtype, cuda_device, seed=7)
    x["p"][:, :, :9] = 0
    x["p"][:, :, 3990:] = 0
    x["r"][:] = [0.0, 1 - 2.0**-24, 2.0**-30, 0.5, 0.999999, 1e-6, 0.25, 0.75]
    got = run_verify(x, cuda_device, False)
    status_ok()
    check_verify(x, got, False)
    assert got[2][0] == 9 and (got[2] >= 9).all() and (got[2] < 3990).all()


def test_verify_degenerate_rows(cuda_device):
    """A draft equal to the target leaves no residual: the target's own row is sampled. One-hot targets
    (greedy decoding). Rows without a positive sum answer -1 and are recorded."""
    x = draft(4, 3, 500, "f32", cuda_device, seed=8)
    x["q"] = x["p"].clone()
    x["u"][:] = 1.0  # a number outside [0, 1): rejects a draft equal to the target
    got = run_verify(x, cuda_device)
    status_ok()
    check_verify(x, got)
    hot = torch.zeros_like(x["p"])
    hot[:, :, 123] = 1
    x["p"], x["u"][:] = hot, 0.3
    x["tokens"][:, 1:] = 123
    for dense in (True, False):
        got = run_verify(x, cuda_device, dense)
        status_ok()
        check_verify(x, got, dense)
        assert (got[2] == 123).all() and (got[1] > 1).all()
    for bad in (0.0, float("nan"), float("inf"), -1.0):
        x["p"] = torch.full_like(hot, bad)
        x["parents"][:] = -1
        got = run_verify(x, cuda_device)
        assert api.sync_status() == api.FAVOR_ERR_INVALID_ARG
        assert (got[2] == -1).all() and (got[1] == 1).all()
    status_ok()


def test_verify_bad_parents_and_tokens_are_recorded(cuda_device):
    x = draft(3, 10, 300, "f32", cuda_device, seed=9)
    x["u"][:] = 0.0  # whatever can be accepted is
    ref = {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in x.items()}
    x["parents"][0, 1], ref["parents"][0, 1] = 5, -1
    x["tokens"][1, 1], ref["parents"][1, 1] = 300, -1
    x["tokens"][2, 2], ref["parents"][2, 2] = -4, -1
    got = run_verify(x, cuda_device)
    assert api.sync_status() == api.FAVOR_ERR_INVALID_ARG
    check_verify(ref, got)
    status_ok()


# ------------------------------------------------------------------------------------ used together

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_round_of_speculative_decoding(cuda_device, dtype):
    """Prompt into the state, a drafted tree answered over it, the walk, and the accepted path added --
    without a copy to the host. The state then holds the prompt and the path, and the accepted nodes'
    rows are those of single steps over them."""
    B, H, L, T, d, m, V = 3, 2, 90, 20, 64, 256, 400
    x = Problem(B, H, T, d, m, dtype, cuda_device, prior=L, seed=30)
    state = api.decode_extend(x.prior[1], x.prior[2], x.W, api.decode_state(B, H, d, m, cuda_device))
    y = draft(B, T, V, "f32", cuda_device, seed=31)
    parents, tokens = i32(y["parents"], cuda_device), i32(y["tokens"], cuda_device)
    u, r = (torch.tensor(y[k] * 0.6, device=cuda_device) for k in "ur")
    for _ in range(2):  # two rounds with the same drafts
        out = api.decode_tree(x.q, x.k, x.v, x.W, state, parents)
        path, n_path, token = api.decode_verify(parents, tokens, y["p"], u, r, q=y["q"])
        before = state.clone()
        api.decode_extend(x.k, x.v, x.W, state, index=path, counts=n_path)
        for b in range(B):
            cur = before.clone()
            nodes = path[b, : n_path[b]].tolist()
            for j in nodes:
                o = api.decode_step(*(t[:, :, j].contiguous() for t in (x.q, x.k, x.v)), x.W, cur)
                assert rel_max_err(out[b, :, j].double().cpu().numpy(), o[b].double().cpu().numpy()) <= TOL
            a, c = (s.view(B, H, d + 2, m)[b].double().cpu().numpy() for s in (state, cur))
            assert np.abs(a - c).max() <= TOL * np.abs(c).max()
    status_ok()
    assert int(n_path.max()) > 1


def test_another_stream_and_captured_graphs(cuda_device):
    """The calls on a side stream, and captured into two graphs that are replayed in turn: the same bits
    as eager calls."""
    B, H, T, V = 2, 3, 30, 3000
    x = Problem(B, H, T, 64, 256, "bf16", cuda_device, seed=40)
    long = Problem(1, 2, 1000, 64, 256, "bf16", cuda_device, seed=41)
    y = draft(B, T, V, "f32", cuda_device, seed=42)
    parents, tokens = i32(y["parents"], cuda_device), i32(y["tokens"], cuda_device)
    u, r = (torch.tensor(y[k], device=cuda_device) for k in "ur")
    base, base_long = x.state.clone(), long.state.clone()

    def decode():
        out = api.decode_tree(x.q, x.k, x.v, x.W, x.state, parents)
        path, n, token = api.decode_verify(parents, tokens, y["p"], u, r, q=y["q"])
        api.decode_extend(x.k, x.v, x.W, x.state, index=path, counts=n)
        return out, path, n, token, x.state

    def prompt():
        return (api.decode_extend(long.k, long.v, long.W, long.state),)

    def eager(f, state, start):
        state.copy_(start)
        return [t.clone() for t in f()]

    want = eager(decode, x.state, base), eager(prompt, long.state, base_long)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = eager(decode, x.state, base), eager(prompt, long.state, base_long)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(want, got):
        assert all(torch.equal(s, t) for s, t in zip(a, b))
    graphs, outs = [], []
    for f in (decode, prompt):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(f())
        graphs.append(g)
    for _ in range(2):
        x.state.copy_(base)
        long.state.copy_(base_long)
        for g in graphs:
            g.replay()
        for a, b in zip(want, outs):
            assert all(torch.equal(s, t) for s, t in zip(a, b))
    status_ok()


def test_calls_given_a_stream(cuda_device):
    """stream=: the same bits as on the current stream, though the current one keeps allocating and writing
    (what the call allocated for itself is not handed out while the other stream uses it)."""
    x = Problem(1, 4, 4000, 64, 256, "bf16", cuda_device, prior=0, seed=60)
    y = draft(4, 20, 20000, "f32", cuda_device, seed=61)
    parents, tokens = i32(y["parents"], cuda_device), i32(y["tokens"], cuda_device)
    u, r = (torch.tensor(y[k], device=cuda_device) for k in "ur")
    want_state = api.decode_extend(x.k, x.v, x.W, x.state.clone())
    want = api.decode_verify(parents, tokens, y["p"], u, r, q=y["q"])
    t = [z[:, :, :40].contiguous() for z in (x.q, x.k, x.v)]
    tree = i32(random_parents(1, 40), cuda_device)
    want_out = api.decode_tree(*t, x.W, want_state, tree)
    side = torch.cuda.Stream()
    n = api.library().favor_decode_extend_workspace_size(api.ctypes.byref(api.make_shape(1, 4, 4000, 64, 256, api.FAVOR_BF16)), 0)
    for _ in range(3):
        state = x.state.clone()
        side.wait_stream(torch.cuda.current_stream())
        for _ in range(4):  # the side stream is busy when the calls are made
            torch.cuda._sleep(200000)
            with torch.cuda.stream(side):
                torch.cuda._sleep(200000)
        api.decode_extend(x.k, x.v, x.W, state, stream=side)
        junk = [torch.full((n,), 255, dtype=torch.uint8, device=cuda_device) for _ in range(3)]
        got = api.decode_verify(parents, tokens, y["p"], u, r, q=y["q"], stream=side)
        out = api.decode_tree(*t, x.W, state, tree, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(state, want_state) and torch.equal(out, want_out)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del junk
    status_ok()


def test_calls_given_a_stream_leave_memory_in_use_alone(cuda_device):
    """A block freed on the current stream, whose queued work still reads or writes it, is not what a call on
    another stream takes for its workspace or results."""
    x = Problem(1, 4, 4000, 64, 256, "bf16", cuda_device, prior=0, seed=62)
    y = draft(4, 20, 20000, "f32", cuda_device, seed=63)
    parents, tokens = i32(y["parents"], cuda_device), i32(y["tokens"], cuda_device)
    u, r = (torch.tensor(y[k], device=cuda_device) for k in "ur")
    t = [z[:, :, :40].contiguous() for z in (x.q, x.k, x.v)]
    tree = i32(random_parents(1, 40), cuda_device)
    state = api.decode_extend(x.k, x.v, x.W, x.state.clone())
    n = api.library().favor_decode_extend_workspace_size(api.ctypes.byref(api.make_shape(1, 4, 4000, 64, 256, api.FAVOR_BF16)), 0)
    short = [z[:, :, :300].contiguous() for z in (x.q, x.k, x.v)]
    one = [z[:, :, 0].contiguous() for z in t]
    sizes = {"extend": n, "tree": 4 * t[0].numel(), "verify": 4 * parents.numel(), "fwd": 4 * short[0].numel(),
             "step": 4 * one[0].numel()}
    calls = {"extend": lambda s, st: (api.decode_extend(x.k, x.v, x.W, st, stream=s),),
             "tree": lambda s, st: (api.decode_tree(*t, x.W, st, tree, stream=s),),
             "verify": lambda s, st: api.decode_verify(parents, tokens, y["p"], u, r, q=y["q"], stream=s),
             "fwd": lambda s, st: (api.fwd(*short, x.W, stream=s),),
             "step": lambda s, st: (api.decode_step(*one, x.W, st, stream=s),)}
    side = torch.cuda.Stream()
    for name, call in calls.items():
        start = x.state if name == "extend" else state
        want = [z.clone() for z in call(None, start.clone())]
        for _ in range(2):
            mine = start.clone()
            torch.cuda.synchronize()
            block = torch.full((sizes[name],), 7, dtype=torch.uint8, device=cuda_device)
            torch.cuda.synchronize()
            torch.cuda._sleep(20000000)
            seen = block.clone()
            block.fill_(255)
            del block
            got = call(side, mine)
            side.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want)), name
            torch.cuda.synchronize()
            assert (seen == 7).all() and all(torch.equal(a, b) for a, b in zip(got, want)), name
    status_ok()


def test_binding_refuses_what_does_not_fit(cuda_device):
    x = Problem(2, 2, 6, 64, 128, "bf16", cuda_device, prior=0)
    parents = i32(random_parents(2, 6), cuda_device)
    p = torch.full((2, 6, 10), 0.1, device=cuda_device)
    u, r = torch.zeros(2, 6, device=cuda_device), torch.zeros(2, device=cuda_device)
    tree = [x.q, x.k, x.v, x.W, x.state, parents]

    def put(args, i, t):
        return args[:i] + [t] + args[i + 1:]

    calls = [lambda a=put(tree, i, t): api.decode_tree(*a) for i, t in
             [(1, x.k[:, :, :3].contiguous()), (2, x.v.float()), (3, x.W[:, :32].contiguous()), (4, x.state[:-1]),
              (4, x.state.half()), (5, parents.long()), (5, parents[:, :5].contiguous()), (5, parents.cpu()),
              (0, x.q.transpose(1, 2)), (5, parents.t().contiguous().t())]]
    calls += [lambda: api.decode_tree(*tree, n_nodes=parents), lambda: api.decode_tree(*tree, out=x.q),
              lambda: api.decode_extend(x.k, x.v, x.W, x.state, index=parents[0]),
              lambda: api.decode_extend(x.k, x.v, x.W, x.state, index=parents[:, :0]),
              lambda: api.decode_extend(x.k, x.v, x.W, x.state, counts=parents),
              lambda: api.decode_extend(x.k, x.v, x.W, x.state[2:]),
              lambda: api.decode_verify(parents, parents, p, u, r, q=p[:, :, :9].contiguous()),
              lambda: api.decode_verify(parents, parents, p, u, r, q=p.bfloat16()),
              lambda: api.decode_verify(parents, parents, p, u.double(), r),
              lambda: api.decode_verify(parents, parents, p, u, u),
              lambda: api.decode_verify(parents, parents, p.half(), u, r),
              lambda: api.decode_verify(parents, parents[:1], p, u, r)]
    for i, call in enumerate(calls):
        with pytest.raises(api.FavorError) as e:
            call()
        assert e.value.status == api.FAVOR_ERR_INVALID_ARG, i
    status_ok()


def test_binding_refuses_a_workspace_of_the_host(cuda_device):
    x = Problem(2, 2, 6, 64, 128, "bf16", cuda_device, prior=0)
    ws = torch.empty(1 << 24, dtype=torch.uint8)
    for call in (lambda: api.decode_extend(x.k, x.v, x.W, x.state, workspace=ws),
                 lambda: api.fwd(x.q, x.k, x.v, x.W, workspace=ws),
                 lambda: api.sp_state(x.k, x.v, x.W, workspace=ws)):
        with pytest.raises(api.FavorError) as e:
            call()
        assert e.value.status == api.FAVOR_ERR_INVALID_ARG
    status_ok()
