"""Cases that measure the operators of speculative decoding over the carried FAVOR+ state.

Three operators make one decoding round of a model with FAVOR+ attention:

* ``tree``   attention of a tree of drafted tokens over the carried state: with u_r(x) = w_r.x - |x|^2/2
             and J(i) the ancestors of node i and itself,
             out_i = [sum_r e^(w_r.q_i) (S_r + sum_{j in J(i)} e^(u_r(k_j)) v_j)]
                     / [sum_r e^(w_r.q_i) (z_r + sum_{j in J(i)} e^(u_r(k_j)))];
* ``verify`` the walk down the drafted tree against the target's probabilities with given random numbers:
             accepts children or rejects them with the residual max(w - Z q, 0), then samples one more token;
* ``extend`` tokens (a prompt's, or those on the accepted path) added to the carried state:
             S_r += sum_j e^(u_r(k_j)) v_j, z_r += sum_j e^(u_r(k_j)), each feature held relative to e^(D_r)
             with D_r the largest u_r so far.

The state of one head is fp32 [d m + 2 m]: S'[c][r], z'[r], D[r] with S_r[c] = e^(D_r) S'[c][r] and
z_r = e^(D_r) z'[r]; a feature with z'[r] = 0 is empty.

``own = False``: plain torch forms; ``own = True``: the library's calls.
"""

import math

import torch

own = False

DEVICE = "cuda"

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # One request on a small model, one drafted token: an ordinary decoding step that leaves the
        # state alone (latency).
        tree("tree-one-token", 1, 8, 1, 64, 256, "bf16"),
        # A few requests with a small tree each: interactive serving (latency).
        tree("tree-16-nodes", 4, 8, 16, 64, 256, "bf16"),
        # fp32 inputs, an odd number of nodes, sequences with fewer nodes than the buffer holds.
        tree("tree-f32-33-ragged", 8, 8, 33, 64, 128, "f32", ragged=True),
        # Wide heads, trees of 60 nodes cut differently per request: a mid-size batch.
        tree("tree-d128-60-ragged", 16, 16, 60, 128, 256, "bf16", ragged=True),
        # A full serving batch, 64 nodes a request.
        tree("tree-batch-64", 64, 16, 64, 64, 256, "bf16"),
        # The accepted paths of a full serving batch (1 to 9 of the 64 nodes each) enter the state.
        extend("extend-paths", 64, 16, 64, 64, 256, "bf16", paths=9),
        # fp32 prompts of different lengths, padded to 500 tokens.
        extend("extend-f32-prompts", 4, 8, 500, 64, 128, "f32", ragged=True),
        # Prompts of a model with wide heads (the training workload's shape).
        extend("extend-d128-L16384", 2, 8, 16384, 128, 256, "bf16"),
        # One long prompt (the long causal workload's shape).
        extend("extend-L65536", 1, 16, 65536, 64, 256, "bf16"),
        # One request whose draft is deterministic (point masses), 32,000 tokens of vocabulary (latency).
        verify("verify-one-point", 1, 8, 32000, "f32", "point"),
        # A mid-size batch with bf16 probabilities and an odd vocabulary, so that rows are unaligned.
        verify("verify-bf16-V50257", 16, 16, 50257, "bf16", "dense", ragged=True),
        # A full serving batch with a large vocabulary and a sampling draft.
        verify("verify-batch-V131072", 64, 32, 131072, "f32", "dense"),
    ]


def tree(name, B, H, T, d, m, dtype, ragged=False):
    return {"name": name, "op": "tree", "B": B, "H": H, "T": T, "d": d, "m": m, "dtype": dtype, "ragged": ragged}


def extend(name, B, H, L, d, m, dtype, ragged=False, paths=0):
    return {"name": name, "op": "extend", "B": B, "H": H, "L": L, "d": d, "m": m, "dtype": dtype, "ragged": ragged,
            "paths": paths}


def verify(name, B, T, V, dtype, draft, ragged=False):
    return {"name": name, "op": "verify", "B": B, "T": T, "V": V, "dtype": dtype, "draft": draft, "ragged": ragged}


def draw(rng):
    def spread(lo, hi):
        return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))

    op = rng.choice(["tree", "extend", "verify"])
    dtype, ragged = rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.5
    d, m = rng.choice([64, 128]), rng.choice([32, 96, 128, 160, 256, 256])
    B = spread(1, 64)
    if op == "tree":  # up to the full batch's work
        H = min(spread(1, 16), max(1, 1024 * 64 // (B * d)))
        T = min(spread(1, 128), max(1, 1024 * 64 * 64 // (B * H * d)))
        case = tree("", B, H, T, d, m, dtype, ragged)
    elif op == "extend":  # short, ordinary and long prompts, or accepted paths
        H = min(spread(1, 16), max(1, 1024 * 64 // (B * d)))
        if rng.random() < 0.4:
            T = spread(1, 128)
            case = extend("", B, H, T, d, m, dtype, paths=min(T, rng.randint(1, 16)))
        else:
            case = extend("", B, H, min(spread(1, 65536), (1 << 20) * 64 // (B * H * d)), d, m, dtype, ragged)
    else:
        V = spread(1000, 131072)
        T = min(spread(1, 64), max(1, (1 << 28) // (B * V)))
        case = verify("", B, T, V, dtype, rng.choice(["point", "dense"]), ragged)
    del case["name"]
    return case


# ------------------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return {"tree": _prepare_tree, "extend": _prepare_extend, "verify": _prepare_verify}[case["op"]](case, g)


def _features(m, d, dtype, g):
    """Block-orthogonal Gaussian rows with chi(d) norms, as the library draws them."""
    n = -(-m // d)
    q, _ = torch.linalg.qr(torch.randn(n, d, d, generator=g, device=DEVICE, dtype=torch.float64))
    norms = torch.randn(n, d, d, generator=g, device=DEVICE, dtype=torch.float64).square().sum(-1).sqrt()
    return (q * norms[..., None]).reshape(n * d, d)[:m].to(dtype).contiguous()


def _tokens(B, H, L, d, dtype, g):
    """Queries and keys (scaled by d^-1/4) and values of L tokens."""
    rows = [torch.randn(B, H, L, d, generator=g, device=DEVICE) for _ in range(3)]
    s = d ** -0.25
    return (rows[0] * s).to(dtype), (rows[1] * s).to(dtype), rows[2].to(dtype)


def _carried(B, H, d, W, dtype, g):
    """The carried state after 96 tokens."""
    _, k, v = _tokens(B, H, 96, d, dtype, g)
    u = _logits(k.float(), W.float())
    D = u.amax(2)
    phi = torch.exp(u - D[:, :, None])
    S = v.float().mT @ phi
    return torch.cat([S.flatten(2), phi.sum(2), D], 2).reshape(-1).contiguous()


def _parents(B, T, g):
    """Random trees in topological order, a root first: a node's parent is one of the nodes before it,
    the near ones more often."""
    i = torch.arange(T, device=DEVICE)
    back = (torch.rand(B, T, generator=g, device=DEVICE).square() * i.clamp(max=12)).long() + 1
    return (i - back).clamp(min=0).masked_fill(i == 0, -1).to(torch.int32)


def _lengths(B, L, g, lo=1):
    return (torch.rand(B, generator=g, device=DEVICE) * (L + 1 - lo)).long().add(lo).clamp(max=L).to(torch.int32)


def _prepare_tree(c, g):
    B, H, T, d, dtype = c["B"], c["H"], c["T"], c["d"], DTYPES[c["dtype"]]
    W = _features(c["m"], d, dtype, g)
    q, k, v = _tokens(B, H, T, d, dtype, g)
    return {"op": "tree", "q": q, "k": k, "v": v, "W": W, "state": _carried(B, H, d, W, dtype, g),
            "parents": _parents(B, T, g), "n_nodes": _lengths(B, T, g) if c["ragged"] else None,
            "out": torch.zeros(B, H, T, d, device=DEVICE)}


def _prepare_extend(c, g):
    B, H, L, d, dtype = c["B"], c["H"], c["L"], c["d"], DTYPES[c["dtype"]]
    W = _features(c["m"], d, dtype, g)
    _, k, v = _tokens(B, H, L, d, dtype, g)
    s = {"op": "extend", "k": k, "v": v, "W": W, "index": None, "counts": None}
    if c["paths"]:  # the state of a request under way
        s["state"] = _carried(B, H, d, W, dtype, g)
        order = torch.rand(B, L, generator=g, device=DEVICE).argsort(1)[:, :c["paths"]]
        s["index"] = order.sort(1).values.to(torch.int32).contiguous()
        s["counts"] = _lengths(B, c["paths"], g)
    else:  # a new request: the empty state
        s["state"] = torch.zeros(B * H * (d + 2) * c["m"], device=DEVICE)
        if c["ragged"]:
            s["counts"] = _lengths(B, L, g)
    return s


def _prepare_verify(c, g):
    B, T, V, dtype = c["B"], c["T"], c["V"], DTYPES[c["dtype"]]
    logits = torch.randn(B, T, V, generator=g, device=DEVICE) * 3
    p = torch.softmax(logits, -1).to(dtype)
    logits += torch.randn(B, T, V, generator=g, device=DEVICE) * 0.7
    q = torch.softmax(logits, -1).to(dtype)
    del logits
    parents = _parents(B, T, g)
    # each node's token is a sample of the draft's distribution behind its parent
    rows = q[torch.arange(B, device=DEVICE)[:, None], parents.long().clamp(min=0)].float()
    tokens = (rows / torch.empty_like(rows).exponential_(generator=g).clamp_(min=1e-30)).argmax(-1).to(torch.int32)
    del rows
    return {"op": "verify", "parents": parents, "tokens": tokens, "p": p, "q": q if c["draft"] == "dense" else None,
            "u": torch.rand(B, T, generator=g, device=DEVICE), "r": torch.rand(B, generator=g, device=DEVICE),
            "n_nodes": _lengths(B, T, g) if c["ragged"] else None}


# --------------------------------------------------------------------------------------------- run

def run(s):
    if own:
        from linear_attention_positive_b200 import api

        if s["op"] == "tree":
            return api.decode_tree(s["q"], s["k"], s["v"], s["W"], s["state"], s["parents"], n_nodes=s["n_nodes"],
                                   out=s["out"])
        if s["op"] == "extend":
            return api.decode_extend(s["k"], s["v"], s["W"], s["state"], index=s["index"], counts=s["counts"])
        return api.decode_verify(s["parents"], s["tokens"], s["p"], s["u"], s["r"], q=s["q"], n_nodes=s["n_nodes"])
    return {"tree": _plain_tree, "extend": _plain_extend, "verify": _plain_verify}[s["op"]](s)


def _logits(x, W):
    return x @ W.T - 0.5 * x.square().sum(-1, keepdim=True)


def _views(state, B, H, d, m):
    rows = state.view(B, H, (d + 2) * m)
    return rows[..., : d * m].view(B, H, d, m), rows[..., d * m: (d + 1) * m], rows[..., (d + 1) * m:]


def _plain_tree(s):
    q, k, v, W = s["q"].float(), s["k"].float(), s["v"].float(), s["W"].float()
    B, H, T, d = q.shape
    S, z, D = _views(s["state"], B, H, d, W.shape[0])
    # ancestors and self: powers of the parent relation by squaring
    node = torch.arange(T, device=q.device)
    reach = ((s["parents"].long()[..., None] == node) | (node[:, None] == node)).float()
    for _ in range(max(1, (T - 1).bit_length())):
        reach = (reach @ reach > 0).float()
    uk = _logits(k, W)
    D = torch.where(z > 0, D, -math.inf)
    top = torch.maximum(D, uk.amax(2))
    uq = q @ W.T + top[:, :, None]
    fq = torch.exp(uq - uq.amax(-1, keepdim=True))
    fk = torch.exp(uk - top[:, :, None])
    carried = torch.exp(D - top)
    a = (fq @ fk.mT) * reach[:, None]
    num = a @ v + (fq * carried[:, :, None]) @ S.mT
    den = a.sum(-1) + (fq * (carried * z)[:, :, None]).sum(-1)
    out = num / den[..., None]
    if s["n_nodes"] is not None:
        out = torch.where((node < s["n_nodes"][:, None])[:, None, :, None], out, s["out"])
    return s["out"].copy_(out)


def _plain_extend(s):
    k, v, W, counts = s["k"], s["v"], s["W"].float(), s["counts"]
    B, H, _, d = k.shape
    if s["index"] is not None:
        at = s["index"].long()[:, None, :, None].expand(-1, H, -1, d)
        k, v = k.gather(2, at), v.gather(2, at)
    S, z, D = _views(s["state"], B, H, d, W.shape[0])
    u = _logits(k.float(), W)
    if counts is not None:
        off = torch.arange(k.shape[2], device=k.device) >= counts[:, None]
        u = u.masked_fill(off[:, None, :, None], -math.inf)
    D_old = torch.where(z > 0, D, -math.inf)
    D_new = torch.maximum(D_old, u.amax(2))
    phi = torch.exp(u.sub_(D_new[:, :, None]))
    keep = torch.exp(D_old - D_new)
    S.copy_(S * keep[:, :, None] + v.float().mT @ phi)
    z.copy_(z * keep + phi.sum(2))
    D.copy_(D_new)
    return s["state"]


def _plain_verify(s):
    parents, tokens, p, q = s["parents"], s["tokens"].long(), s["p"], s["q"]
    B, T, V = p.shape
    b = torch.arange(B, device=p.device)
    n = s["n_nodes"].long() if s["n_nodes"] is not None else torch.full((B,), T, device=p.device)
    cur, w, Z = torch.zeros_like(b), p[:, 0].double(), torch.ones(B, device=p.device, dtype=torch.float64)
    path = torch.full((B, T), -1, device=p.device, dtype=torch.int32)
    path[:, 0] = 0
    length = torch.ones_like(b)
    # The walk is a recurrence over the nodes: in topological order, each looks at what the ones before
    # it left of the current node's distribution.
    for c in range(1, T):
        asked = (parents[:, c] == cur) & (c < n)
        x = tokens[:, c]
        wx = w[b, x]
        qx = q[b, cur, x].double() if q is not None else 1.0
        taken = asked & (s["u"][:, c].double() * (Z * qx) < wx)
        lost = asked & ~taken
        if q is not None:
            rest = (w - Z[:, None] * q[b, cur].double()).clamp(min=0)
            w = torch.where(lost[:, None], rest, w)
            Z = torch.where(lost, w.sum(1), Z)
        else:
            w[b, x] = torch.where(lost, 0.0, wx)
            Z = torch.where(lost, Z - wx, Z)
        w = torch.where(taken[:, None], p[:, c].double(), w)
        Z = torch.where(taken, 1.0, Z)
        cur = torch.where(taken, c, cur)
        path[b, length.clamp(max=T - 1)] = torch.where(taken, c, path[b, length.clamp(max=T - 1)])
        length += taken
    # an empty residual (drafts that cover the target exactly) falls back to the target's own row
    w = torch.where(w.sum(1, keepdim=True) > 0, w, p[b, cur].double())
    sums = w.cumsum(1)
    token = (sums <= s["r"].double()[:, None] * sums[:, -1:]).sum(1).clamp(max=V - 1)
    return path, length.to(torch.int32), token.to(torch.int32)


# -------------------------------------------------------------------------------------------- work

def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    B = case["B"]
    if case["op"] == "verify":
        # the last node's row of the target, and of the draft where one is given (counted as if its
        # residual were always needed); the walk itself looks at single entries
        rows = 2 if case["draft"] == "dense" else 1
        return {"bytes": B * (case["V"] * rows * size + 24 * case["T"]), "flops": 4 * B * case["V"]}
    H, d, m = case["H"], case["d"], case["m"]
    BH, state = B * H, (d + 2) * m * 4
    if case["op"] == "tree":
        T = case["T"] * (0.5 if case["ragged"] else 1)
        return {"bytes": BH * (state + T * d * (3 * size + 4)) + m * d * size + 8 * B,
                "flops": BH * T * (6 * m * d + (m + d) * T)}
    n = (case["paths"] + 1) / 2 if case["paths"] else case["L"] * (0.5 if case["ragged"] else 1)
    return {"bytes": BH * (2 * state + n * d * 2 * size) + m * d * size, "flops": BH * n * 4 * m * d}


# ------------------------------------------------------------------------------------------- exact

def exact(case, seed):
    s = prepare(case, seed)
    return {"tree": _exact_tree, "extend": _exact_extend, "verify": _exact_verify}[s["op"]](s)


def _exact_state(state, B, H, d, m):
    """The state's true sums S [B, H, d, m], z [B, H, m]."""
    t = state.double().view(B * H, d + 2, m)
    scale = torch.where(t[:, d] > 0, torch.exp(t[:, d + 1]), 0.0)
    return (t[:, :d] * scale[:, None]).view(B, H, d, m), (t[:, d] * scale).view(B, H, m)


def _exact_tree(s):
    q, k, v, W = (s[x].double() for x in ("q", "k", "v", "W"))
    B, H, T, d = q.shape
    S, z = _exact_state(s["state"], B, H, d, W.shape[0])
    parents, out = s["parents"].tolist(), s["out"].double().clone()
    lengths = s["n_nodes"].tolist() if s["n_nodes"] is not None else [T] * B
    for b in range(B):
        mask = torch.zeros(T, T, dtype=torch.float64)
        for i in range(T):
            j = i
            while j >= 0:
                mask[i, j] = 1
                j = parents[b][j]
        fq = torch.exp(q[b] @ W.T)
        fk = torch.exp(k[b] @ W.T) * torch.exp(-0.5 * (k[b] ** 2).sum(-1, keepdim=True))
        a = torch.einsum("hir,hjr->hij", fq, fk) * mask.to(q.device)
        num = torch.einsum("hij,hjc->hic", a, v[b]) + torch.einsum("hir,hcr->hic", fq, S[b])
        den = a.sum(-1) + torch.einsum("hir,hr->hi", fq, z[b])
        n = lengths[b]
        out[b, :, :n] = (num / den[..., None])[:, :n]
    return out


def _exact_extend(s):
    W, counts = s["W"].double(), s["counts"]
    B, H, L, d = s["k"].shape
    m = W.shape[0]
    S, z = _exact_state(s["state"], B, H, d, m)
    old = s["state"].double().view(B, H, d + 2, m)
    out = torch.empty_like(old)
    for b in range(B):
        n = int(counts[b]) if counts is not None else (L if s["index"] is None else s["index"].shape[1])
        at = s["index"][b, :n].long() if s["index"] is not None else slice(0, n)
        for h in range(H):
            k, v = s["k"][b, h, at].double(), s["v"][b, h, at].double()
            u = k @ W.T - (k * k).sum(1, keepdim=True) / 2
            f = torch.exp(u)
            D = torch.where(old[b, h, d] > 0, torch.maximum(old[b, h, d + 1], u.amax(0)), u.amax(0))
            out[b, h, :d] = (S[b, h] + v.T @ f) * torch.exp(-D)
            out[b, h, d] = (z[b, h] + f.sum(0)) * torch.exp(-D)
            out[b, h, d + 1] = D
    return out.reshape(-1)


def _exact_verify(s):
    """One sequence after another, each walked child by child."""
    parents, tokens = s["parents"].tolist(), s["tokens"].tolist()
    u, r = s["u"].double().tolist(), s["r"].double().tolist()
    B, T, V = s["p"].shape
    lengths = s["n_nodes"].tolist() if s["n_nodes"] is not None else [T] * B
    paths, counts, samples = [], [], []
    for b in range(B):
        node, path = 0, [0]
        while node is not None:
            w, Z, accepted = s["p"][b, node].double().clone(), 1.0, None
            for c in [c for c in range(node + 1, lengths[b]) if parents[b][c] == node]:
                x = tokens[b][c]
                draft = 1.0 if s["q"] is None else float(s["q"][b, node, x])
                if u[b][c] * draft * Z < float(w[x]):
                    accepted = c
                    break
                if s["q"] is None:
                    Z -= float(w[x])
                    w[x] = 0
                else:
                    w = torch.relu(w - s["q"][b, node].double() * Z)
                    Z = float(w.sum())
            if accepted is not None:
                path.append(accepted)
                node = accepted
                continue
            if not float(w.sum()) > 0:
                w = s["p"][b, node].double()
            sums = torch.cumsum(w, 0)
            hit = torch.nonzero(sums > r[b] * sums[-1])
            samples.append(int(hit[0]) if len(hit) else int(torch.nonzero(w)[-1]))
            node = None
        paths.append(path + [-1] * (T - len(path)))
        counts.append(len(path))
    return tuple(torch.tensor(t, dtype=torch.int32) for t in (paths, counts, samples))
