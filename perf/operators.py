"""Measured operators of the recurrent layers: the scan over whole sequences that
leaves the dense state a conversion starts from, its backward pass, and the tree of
drafted tokens read against the stored (sink plus low-rank) state.

The three forms, per head, state S (d_k x d_v), a token's k, q (d_k), v (d_v):

    S' = Diag(a) S            (a: one decay per head for GDN and Mamba-2, one per channel for KDA)
    w  = beta (v - S'^T k)    (Mamba-2, which has no erase: w = beta v)
    S+ = S' + k w^T,   o = S+^T q

`run` computes them in plain torch where `own` is false (chunks of 64 tokens, products
and exponentials in float32, sums of log decays and triangular inverses in float64), and
through rank_recurrent_state_b200.seed where it is true.  `exact` steps token by token
in float64.
"""

import torch

own = False

GDN, KDA, MAMBA2 = "gdn", "kda", "mamba2"
FORMS = {GDN: 0, KDA: 1, MAMBA2: 2}
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
CHUNK = 64
DIMS = [(16, 16), (32, 32), (64, 64), (128, 128), (128, 64), (64, 128)]
MOST_TOKEN_HEADS = 8192 * 32      # of a scan: the long prompt's


# ------------------------------------------------------------------ cases

def _scan(name, form, typ, seqs, lo, hi, heads, k_heads, d_k, d_v, train=False, state=True):
    """seqs sequences of lo..hi tokens (one of exactly hi), heads value heads that share
    k_heads key heads; state: an initial state comes in and the final one goes out."""
    return {"name": name, "op": "train" if train else "scan", "form": form, "type": typ, "seqs": seqs, "lo": lo,
            "hi": hi, "heads": heads, "k_heads": k_heads, "d_k": d_k, "d_v": d_v, "state": state}


def _tree(name, form, typ, batch, nodes, heads, d_k, d_v, R, W, chain):
    """batch requests with up to `nodes` drafted tokens each; chain: how often (percent) a
    node continues its predecessor instead of branching off an earlier one."""
    return {"name": name, "op": "tree", "form": form, "type": typ, "batch": batch, "nodes": nodes, "heads": heads,
            "d_k": d_k, "d_v": d_v, "R": R, "W": W, "chain": chain}


def listed():
    return [
        # one token per request through a GDN layer's dense states: the decode step of a
        # model served without the shallow form, bound by the states' bytes and latency
        _scan("scan gdn one token", GDN, "bf16", 16, 1, 1, 48, 16, 128, 128),
        # short ragged prompts of a small layer: chat turns appended to a live state
        _scan("scan kda short ragged", KDA, "f32", 12, 1, 90, 4, 4, 64, 64),
        # one 4096-token prompt of a GDN layer, three value heads to a key head: time to
        # first token, one long chain of chunks per head
        _scan("scan gdn prompt", GDN, "bf16", 1, 4096, 4096, 48, 16, 128, 128),
        # a prefill batch of ragged prompts, the throughput case
        _scan("scan gdn batch", GDN, "bf16", 8, 700, 1024, 48, 48, 128, 128),
        # Mamba-2 heads that share one B and C, float32 activations
        _scan("scan mamba2 prompt", MAMBA2, "f32", 2, 2048, 2048, 64, 1, 128, 64),
        # a long Kimi Delta Attention prompt with its per-channel decays
        _scan("scan kda prompt", KDA, "bf16", 1, 8192, 8192, 32, 32, 128, 128),
        # training: forward and backward over packed documents
        _scan("train gdn packed", GDN, "bf16", 6, 300, 1500, 16, 8, 128, 128, train=True, state=False),
        _scan("train mamba2", MAMBA2, "f32", 2, 1024, 1024, 32, 4, 128, 64, train=True, state=False),
        # the same with a state carried across segments of one long document
        _scan("train kda carried state", KDA, "f16", 1, 2048, 2048, 16, 16, 128, 128, train=True, state=True),
        # a single user's draft of a small tree: latency
        _tree("tree gdn one request", GDN, "f32", 1, 8, 48, 128, 128, 16, 16, 60),
        # a serving batch, trees of 16 tokens, at the GDN layer workload's batch
        _tree("tree gdn batch", GDN, "f32", 64, 16, 48, 128, 128, 16, 16, 60),
        # wider trees over 16-bit factors with per-channel decays
        _tree("tree kda wide", KDA, "bf16", 32, 32, 32, 128, 128, 16, 32, 40),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    form = rng.choice([GDN, KDA, MAMBA2])
    op = rng.choice(["scan", "scan", "train", "tree"])
    d_k, d_v = rng.choice(DIMS[:3] + 2 * DIMS[3:])
    typ = rng.choice(["f32", "f16", "bf16"])
    if op == "tree":
        m = min(d_k, d_v)
        R = rng.randint(1, min(16, m // 2))
        nodes = _spread(rng, 1, 48)
        W = rng.randint(1, min(m, 64) - R)
        heads = rng.randint(1, 48)
        batch = _spread(rng, 1, 64)
        while batch * heads * nodes * (d_k + d_v) > 64 * 48 * 16 * 256:
            batch = max(1, batch // 2)
            heads = heads if batch > 1 else max(1, heads // 2)
        c = _tree("", form, typ, batch, nodes, heads, d_k, d_v, R, W, rng.randint(20, 95))
    else:
        k_heads = rng.randint(1, 16)
        heads = k_heads * rng.choice([1, 1, 2, 3, 4])
        most = MOST_TOKEN_HEADS // (8 if op == "train" else 1)
        seqs = _spread(rng, 1, 40)
        hi = _spread(rng, 1, 8192) if op == "scan" else _spread(rng, 24, 2048)
        while seqs * hi * heads > most:
            if seqs > 1:
                seqs -= max(1, seqs // 4)
            else:
                hi = most // heads
        lo = rng.choice([0, 1, max(1, hi // 2), hi])
        c = _scan("", form, typ, seqs, lo, hi, heads, k_heads, d_k, d_v, train=op == "train", state=rng.random() < 0.5)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def _token_values(c, shape, h_k, h, g, vbar):
    """q, k, v, alpha, beta of tokens in `shape`, with the synthetic workloads' values: GDN and
    KDA unit keys and queries, v = 3 vbar + 0.3 z, beta = sigmoid(z), GDN decay
    exp(-softplus(-3 + z/2)), KDA decays 0.85 + 0.15 u; Mamba-2 keys and queries
    z / sqrt(d_k), v = vbar + z/2, beta = softplus(-2 + z/2), alpha = exp(-beta A), A = 1 + 15 u."""
    randn = lambda *s: torch.randn(*shape, *s, generator=g, device="cuda")  # noqa: E731
    k, q = randn(h_k, c["d_k"]), randn(h_k, c["d_k"])
    if c["form"] == MAMBA2:
        k, q = k / c["d_k"] ** 0.5, q / c["d_k"] ** 0.5
        v = vbar + 0.5 * randn(h, c["d_v"])
        beta = torch.log1p(torch.exp(-2 + 0.5 * randn(h)))
        alpha = torch.exp(-beta * (1 + 15 * torch.rand(h, generator=g, device="cuda")))
    else:
        k, q = (x / x.square().sum(-1, keepdim=True).sqrt() for x in (k, q))
        v = 3 * vbar + 0.3 * randn(h, c["d_v"])
        beta = torch.sigmoid(randn(h))
        if c["form"] == GDN:
            alpha = torch.exp(-torch.log1p(torch.exp(-3 + 0.5 * randn(h))))
        else:
            alpha = 0.85 + 0.15 * torch.rand(*shape, h, c["d_k"], generator=g, device="cuda")
    return q, k, v, alpha, beta


def _vbar(c, g):
    x = torch.randn(c["heads"], c["d_v"], generator=g, device="cuda")
    norm = 1 + 3 * torch.rand(c["heads"], 1, generator=g, device="cuda")
    return x / x.square().sum(-1, keepdim=True).sqrt() * norm


def _lengths(c):
    """The sequences' lengths, by the case alone: every seed packs the same shapes."""
    g = torch.Generator().manual_seed(c["seqs"] * 10007 + c["hi"])
    n = torch.randint(c["lo"], c["hi"] + 1, (c["seqs"],), generator=g)
    n[int(torch.randint(0, c["seqs"], (1,), generator=g))] = c["hi"]
    return n.tolist()


def _prepare_scan(c, g):
    lengths = _lengths(c)
    tokens = sum(lengths)
    t = TYPES[c["type"]]
    q, k, v, alpha, beta = _token_values(c, (tokens,), c["k_heads"], c["heads"], g, _vbar(c, g))
    s = {"case": c, "lengths": lengths, "tokens": tokens,
         "offsets": torch.tensor([0] + torch.tensor(lengths).cumsum(0).tolist(), dtype=torch.int32, device="cuda"),
         "q": q.to(t), "k": k.to(t), "v": v.to(t), "alpha": alpha, "beta": beta, "S0": None, "dS": None}
    mat = (c["seqs"], c["heads"], c["d_k"], c["d_v"])
    if c["state"]:
        s["S0"] = torch.randn(mat, generator=g, device="cuda") * 0.2
    if c["op"] == "train":
        s["do"] = torch.randn(tokens, c["heads"], c["d_v"], generator=g, device="cuda").to(t)
        if c["state"]:
            s["dS"] = torch.randn(mat, generator=g, device="cuda") * 0.2
    if own:
        from rank_recurrent_state_b200 import seed as S
        s["dims"] = S.ScanDims(FORMS[c["form"]], c["seqs"], tokens, c["heads"], c["k_heads"], c["d_k"], c["d_v"],
                               max(lengths), S.FACTOR_NAMES[c["type"]])
        s["ws"] = S.ScanWorkspace(s["dims"], backward=c["op"] == "train")
    return s


def _prepare_tree(c, seed, g):
    B, N, H, dk, dv, R, W = (c[x] for x in ("batch", "nodes", "heads", "d_k", "d_v", "R", "W"))
    m = R + W
    vbar = _vbar(c, g)
    cpu = torch.Generator().manual_seed(2000 + seed)
    parent = torch.full((B, N), -2, dtype=torch.int32)
    leaf = torch.full((B,), -1, dtype=torch.int32)
    ncols = torch.zeros(B, dtype=torch.int32)
    for b in range(B):
        n = int(torch.randint(max(1, N // 2), N + 1, (1,), generator=cpu))
        cont = torch.randint(0, 100, (n,), generator=cpu) < c["chain"]
        back = torch.rand(n, generator=cpu)
        depth = []
        for t in range(n):
            p = t - 1 if cont[t] else int(back[t] * (t + 1)) - 1
            parent[b, t] = p
            depth.append(1 + (depth[p] if p >= 0 else 0))
        fits = [t for t in range(n) if depth[t] <= W] + [-1]        # the deepest commit the window has room for
        leaf[b] = fits[int(torch.randint(0, len(fits), (1,), generator=cpu))]
        used = depth[leaf[b]] if leaf[b] >= 0 else 0
        ncols[b] = int(torch.randint(R, m - used + 1, (1,), generator=cpu)) if m - used >= R else R
    q, k, v, alpha, beta = _token_values(c, (B, N), H, H, g, vbar)
    t = TYPES[c["type"]]
    randn = lambda *x: torch.randn(*x, generator=g, device="cuda")  # noqa: E731
    U = randn(B, 1, H, m, dk) / dk ** 0.5
    V = randn(B, 1, H, m, dv) / dv ** 0.5
    V = 3 * (V - (V * vbar[:, None]).sum(-1, keepdim=True) * vbar[:, None] / vbar[:, None].square().sum(-1, keepdim=True))
    scale = 0.3 + 0.7 * torch.rand(B, 1, H, dk if c["form"] == KDA else (m + 3) // 4 * 4, generator=g, device="cuda")
    s = {"case": c, "parent": parent.cuda(), "leaf": leaf.cuda(), "q": q, "k": k, "v": v, "alpha": alpha, "beta": beta,
         "vbar": vbar[None].contiguous(), "U": U.to(t), "V": V.to(t), "a0": randn(B, 1, H, dk), "scale0": scale,
         "ncols0": ncols.cuda()[:, None, None].expand(B, 1, H).contiguous()}
    s["a"], s["scale"], s["ncols"] = s["a0"].clone(), s["scale0"].clone(), s["ncols0"].clone()
    if own:
        from rank_recurrent_state_b200 import seed as S
        s["dims"] = S.Dims(FORMS[c["form"]], B, 1, H, dk, dv, R, W, S.FACTOR_NAMES[c["type"]])
        s["stored"] = S.State(s["a"], s["U"], s["V"], s["scale"], s["ncols"], s["vbar"])
        s["ws"] = S.Workspace(s["dims"])
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return _prepare_tree(case, seed, g) if case["op"] == "tree" else _prepare_scan(case, g)


# ------------------------------------------------------------------ plain form

def _inverse(A):
    """(I + A)^-1 of strictly lower triangular A, by products in float64: the two halves'
    inverses by repeated squaring of the nilpotent part, joined block by block."""
    n = A.shape[-1]
    A = A.double()
    if n > 32:
        h = n // 2
        a, d = _inverse(A[..., :h, :h]), _inverse(A[..., h:, h:])
        low = -d @ A[..., h:, :h] @ a
        return torch.cat([torch.cat([a, torch.zeros_like(low).transpose(-1, -2)], -1), torch.cat([low, d], -1)], -2)
    eye = torch.eye(n, dtype=A.dtype, device=A.device)
    T, P, p = eye - A, A @ A, 2
    while p < n:
        T = T + T @ P
        P, p = P @ P, 2 * p
    return T


def _plain_scan(c, s, q, k, v, la, beta, S0):
    """o (packed, float32) and the final states; la: log decays in float64."""
    B, L, H, dk, dv = c["seqs"], max(s["lengths"]), c["heads"], c["d_k"], c["d_v"]
    n = max(1, -(-L // CHUNK))
    at = torch.arange(n * CHUNK, device="cuda")[None] + s["offsets"][:-1, None]
    valid = at < s["offsets"][1:, None]
    at = torch.where(valid, at, 0).long()

    def chunks(x):      # [tokens][H][d] -> [B][H][n][CHUNK][d], zero behind each sequence
        if x.shape[0] == 0:
            return x.new_zeros(B, x.shape[1], n, CHUNK, x.shape[2])
        y = torch.where(valid[..., None, None], x[at], 0)
        return y.view(B, n, CHUNK, x.shape[1], x.shape[2]).permute(0, 3, 1, 2, 4)

    q, k = (chunks(x.repeat_interleave(H // c["k_heads"], 1)) for x in (q, k))
    v, beta = chunks(v), chunks(beta[..., None])
    G = chunks(la if c["form"] == KDA else la[..., None]).cumsum(-2)         # float64
    low = torch.ones(CHUNK, CHUNK, device="cuda").tril()
    B0 = torch.exp(G).float()                                               # decay since the chunk's start
    BC = torch.exp(G[..., -1:, :] - G).float()                              # decay to its end
    if c["form"] == KDA:
        ki = k * torch.exp(-G).float()
        kk, P = (k * B0) @ ki.transpose(-1, -2), ((q * B0) @ ki.transpose(-1, -2)) * low
    else:
        D = torch.exp((G - G.transpose(-1, -2)).masked_fill(low == 0, float("-inf"))).float()
        kk, P = (k @ k.transpose(-1, -2)) * D, (q @ k.transpose(-1, -2)) * D
    qs, ks, ke = q * B0, k * B0, k * BC
    erase = c["form"] != MAMBA2
    if erase:
        T = _inverse(beta * kk.tril(-1)).float()
    St = torch.zeros(B, H, dk, dv, device="cuda") if S0 is None else S0
    o = []
    for i in range(n):
        w = T[:, :, i] @ (beta[:, :, i] * (v[:, :, i] - ks[:, :, i] @ St)) if erase else beta[:, :, i] * v[:, :, i]
        o.append(qs[:, :, i] @ St + P[:, :, i] @ w)
        St = B0[:, :, i, -1, :, None] * St + ke[:, :, i].transpose(-1, -2) @ w
    o = torch.stack(o, 2).permute(0, 2, 3, 1, 4).reshape(B, n * CHUNK, H, dv)
    return o[valid], St


def _run_plain_scan(s):
    c = s["case"]
    t = TYPES[c["type"]]
    q, k, v, beta = (s[x].float() for x in ("q", "k", "v", "beta"))
    la = torch.log(s["alpha"].double())
    if c["op"] == "scan":
        o, S = _plain_scan(c, s, q, k, v, la, beta, s["S0"])
        return {"o": o.to(t), "S": S} if c["state"] else {"o": o.to(t)}
    leaves = [x.detach().clone().requires_grad_() for x in (q, k, v, la, beta)]
    S0 = None if s["S0"] is None else s["S0"].clone().requires_grad_()
    o, S = _plain_scan(c, s, *leaves, S0)
    loss = (o * s["do"].float()).sum() + (0 if s["dS"] is None else (S * s["dS"]).sum())
    grads = torch.autograd.grad(loss, leaves + ([S0] if c["state"] else []))
    out = dict(zip(["dq", "dk", "dv", "dlog_alpha", "dbeta"], [x.to(t) for x in grads[:3]] + [x.float() for x in grads[3:5]]))
    out["o"] = o.detach().to(t)
    if c["state"]:
        out["S"], out["dS0"] = S.detach(), grads[5]
    return out


def _run_plain_tree(s):
    c = s["case"]
    N, dv, kda = c["nodes"], c["d_v"], c["form"] == KDA
    for x in ("a", "scale", "ncols"):
        s[x].copy_(s[x + "0"])
    heads = lambda x: x.transpose(1, 2)  # noqa: E731       [B][N][H].. -> [B][H][N]..
    q, k, v, beta = heads(s["q"]), heads(s["k"]), heads(s["v"]), heads(s["beta"])[..., None]
    used = s["parent"] >= -1
    la = heads(torch.log(s["alpha"].double()))
    la = la if kda else la[..., None]
    # M[b][t][j]: j is t or an ancestor of t
    step = torch.arange(N, device="cuda") == s["parent"][..., None]
    M = (step | torch.eye(N, dtype=torch.bool, device="cuda")).float()
    for _ in range(max(1, N - 1).bit_length()):
        M = ((M @ M) > 0).float()
    M = (M * used[:, :, None])[:, None]
    G = M.double() @ la
    Bt = torch.exp(G).float()
    if kda:
        ki = k * torch.exp(-G).float()
        kk, P = (k * Bt) @ ki.transpose(-1, -2) * M, (q * Bt) @ ki.transpose(-1, -2) * M
    else:
        D = torch.exp((G - G.transpose(-1, -2)).masked_fill(M == 0, float("-inf"))).float()
        kk, P = (k @ k.transpose(-1, -2)) * D, (q @ k.transpose(-1, -2)) * D
    cols = torch.arange(c["R"] + c["W"], device="cuda")
    held = (cols < s["ncols"][:, 0, :, None])[..., None].float()              # [B][H][m][1]
    sc = s["scale"][:, 0]
    U = s["U"][:, 0].float() * held * (sc[:, :, None, :] if kda else sc[..., : cols.numel(), None])
    V = torch.where(held > 0, s["V"][:, 0].float(), 0)
    a, vb = s["a"][:, 0], s["vbar"][0]
    read = lambda x: (x @ a[..., None]) * vb[:, None] + (x @ U.transpose(-1, -2)) @ V  # noqa: E731     x^T S
    # with the values' coordinate along vbar beside them, whose write goes to the sink alone
    v = torch.cat([v, (v * vb[:, None]).sum(-1, keepdim=True) / vb.square().sum(-1)[:, None, None]], -1)
    if c["form"] == MAMBA2:
        w = beta * v
    else:
        kt = k * Bt
        w = _inverse(beta * kk.tril(-1)).float() @ (beta * (v - torch.cat([read(kt), kt @ a[..., None]], -1)))
    on = used[:, None, :, None]
    w, sw = torch.where(on, w[..., :-1], 0), w[..., -1:]
    o = torch.where(on, read(q * Bt) + P @ w, 0)
    # the accepted path's column pairs, in the order of its nodes
    path = torch.where(s["leaf"][:, None] >= 0, M[:, 0].gather(1, s["leaf"].clamp(min=0).long()[:, None, None].expand(-1, 1, N))[:, 0], 0)
    has = path[:, None, :, None] > 0
    Gl = (path[:, None, :, None].double() * la).sum(2, keepdim=True)         # log decay of the whole path
    col = w - sw * vb[:, None]
    after = torch.exp(Gl - G).float()                                        # decay behind each node of the path
    a_new = torch.exp(Gl[:, :, 0]).float() * a + (torch.where(has, after * sw * k, 0)).sum(2)
    slot = s["ncols"][:, 0, :, None] + (path.cumsum(-1) - 1).long()[:, None]
    bi, hi, ti = torch.nonzero(has[..., 0].expand(-1, c["heads"], -1), as_tuple=True)
    at = slot[bi, hi, ti]
    if kda:
        P_new = sc[:, :, None] * torch.exp(G).float()                        # decays up to each node, stored factors'
        s["U"][bi, 0, hi, at] = (k / P_new)[bi, hi, ti].to(s["U"].dtype)
        s["scale"][:, 0] = sc * torch.exp(Gl[:, :, 0]).float()
    else:
        s["U"][bi, 0, hi, at] = k[bi, hi, ti].to(s["U"].dtype)
        was = (torch.arange(sc.shape[-1], device="cuda") < s["ncols"][:, 0, :, None])
        s["scale"][:, 0] = torch.where(was, sc * torch.exp(Gl[:, :, 0]).float(), sc)
        s["scale"][bi, 0, hi, at] = after[bi, hi, ti, 0]
    s["V"][bi, 0, hi, at] = col[bi, hi, ti].to(s["V"].dtype)
    s["a"][:, 0] = a_new
    s["ncols"] += path.sum(-1).int()[:, None, None]
    return {"o": o.transpose(1, 2), "w": w.transpose(1, 2),
            "a": s["a"], "U": s["U"], "V": s["V"], "scale": s["scale"], "ncols": s["ncols"]}


# ------------------------------------------------------------------ the framework's kernels

def _run_own_scan(s):
    from rank_recurrent_state_b200 import seed as S
    c, d = s["case"], s["dims"]
    o = torch.empty_like(s["v"])
    S_out = torch.empty(c["seqs"], c["heads"], c["d_k"], c["d_v"], device="cuda") if c["state"] else None
    S.seed_dense_scan(d, s["offsets"], s["q"], s["k"], s["v"], s["alpha"], s["beta"], o, s["ws"], S0=s["S0"], S_out=S_out)
    out = {"o": o}
    if c["op"] == "train":
        out["dq"], out["dk"], out["dv"] = (torch.empty_like(s[x]) for x in ("q", "k", "v"))
        out["dlog_alpha"], out["dbeta"] = torch.empty_like(s["alpha"]), torch.empty_like(s["beta"])
        dS0 = torch.empty_like(s["S0"]) if c["state"] else None
        S.seed_dense_scan_backward(d, s["offsets"], s["q"], s["k"], s["v"], s["alpha"], s["beta"], s["do"], out["dq"],
                                   out["dk"], out["dv"], out["dlog_alpha"], out["dbeta"], s["ws"], S0=s["S0"],
                                   dS_out=s["dS"], dS0=dS0)
        if c["state"]:
            out["dS0"] = dS0
    if c["state"]:
        out["S"] = S_out
    return out


def _run_own_tree(s):
    from rank_recurrent_state_b200 import seed as S
    for x in ("a", "scale", "ncols"):         # the state of before the draft
        s[x].copy_(s[x + "0"])
    d, st = s["dims"], s["stored"]
    o, w = torch.empty_like(s["v"]), torch.empty_like(s["v"])
    S.seed_decode_tree(d, st, 0, s["parent"], s["q"], s["k"], s["v"], s["alpha"], s["beta"], o, w, s["ws"])
    S.seed_decode_tree_commit(d, st, 0, s["parent"], s["leaf"], s["k"], s["v"], s["alpha"], s["beta"], w, s["ws"])
    return {"o": o, "w": w, "a": st.a, "U": st.U, "V": st.V, "scale": st.scale, "ncols": st.ncols}


def run(state):
    tree = state["case"]["op"] == "tree"
    if own:
        return _run_own_tree(state) if tree else _run_own_scan(state)
    return _run_plain_tree(state) if tree else _run_plain_scan(state)


# ------------------------------------------------------------------ work

def work(case):
    c = case
    kda = c["form"] == KDA
    products = 2 if c["form"] == MAMBA2 else 3              # S^T k (not Mamba-2), k w^T, S^T q
    if c["op"] == "tree":
        es = TYPES[c["type"]].itemsize
        units = c["batch"] * c["heads"]
        cols, nodes = c["R"] + c["W"] / 2, 0.75 * c["nodes"]
        state = 4 * c["d_k"] * (2 + kda) + es * cols * (c["d_k"] + c["d_v"])
        token = 4 * (2 * c["d_k"] + 3 * c["d_v"] + (c["d_k"] if kda else 1) + 1)
        flops = 2 * nodes * (cols * (c["d_k"] + c["d_v"]) + c["d_k"] + c["d_v"]) * (products - 1) \
            + nodes * nodes * (c["d_k"] + c["d_v"]) * (products - 1)
        return {"bytes": units * (state + nodes * token), "flops": units * flops}
    es = TYPES[c["type"]].itemsize
    tokens = c["hi"] + (c["seqs"] - 1) * (c["lo"] + c["hi"]) / 2
    mats = 4 * c["seqs"] * c["heads"] * c["d_k"] * c["d_v"] if c["state"] else 0
    qk, v = es * tokens * c["k_heads"] * c["d_k"] * 2, es * tokens * c["heads"] * c["d_v"]
    gates = 4 * tokens * c["heads"] * ((c["d_k"] if kda else 1) + 1)
    one = {"bytes": qk + 2 * v + gates + 2 * mats, "flops": 2 * products * tokens * c["heads"] * c["d_k"] * c["d_v"]}
    if c["op"] == "train":      # and backward: inputs, do and dS in, every gradient out; two products for each of the forward's
        one = {"bytes": one["bytes"] + 2 * qk + 3 * v + 2 * gates + 3 * mats, "flops": 3 * one["flops"]}
    return one


# ------------------------------------------------------------------ float64, token by token

def _exact_step(c, S, a, k, v, beta):
    """(S', v - S'^T k, w, S+) of one token; S [n][d_k][d_v], a [n][d_k or 1], beta [n][1]."""
    Sd = a[..., :, None] * S
    r = v if c["form"] == MAMBA2 else v - (k[..., None, :] @ Sd)[..., 0, :]
    w = beta * r
    return Sd, r, w, Sd + k[..., :, None] * w[..., None, :]


def _exact_scan(c, s):
    B, H, rep = c["seqs"], c["heads"], c["heads"] // c["k_heads"]
    L = max(s["lengths"])
    pick, mask = torch.zeros(L, B, dtype=torch.long), torch.zeros(L, B, dtype=torch.bool)
    first = 0
    for b, n in enumerate(s["lengths"]):
        pick[:n, b] = torch.arange(first, first + n)
        mask[:n, b] = True
        first += n
    pick, mask = pick.cuda(), mask.cuda()

    def steps(x, share, behind):        # packed -> [L][B][H][d], `behind` where a sequence has ended
        x = x.double()
        if L == 0:
            return x.new_zeros(0, B, H, x.shape[-1])
        y = x[pick].repeat_interleave(share, 2)
        y[~mask] = behind
        return y

    q, k, v = steps(s["q"], rep, 0), steps(s["k"], rep, 0), steps(s["v"], 1, 0)
    a = steps(s["alpha"] if c["form"] == KDA else s["alpha"][..., None], 1, 1)
    beta = steps(s["beta"][..., None], 1, 0)
    S = torch.zeros(B, H, c["d_k"], c["d_v"], dtype=torch.float64, device="cuda")
    if s["S0"] is not None:
        S = S + s["S0"].double()
    o, kept = torch.zeros_like(v), []
    for t in range(L):
        if c["op"] == "train" and t % 48 == 0:
            kept.append(S)
        S = _exact_step(c, S, a[t], k[t], v[t], beta[t])[3]
        o[t] = (q[t][..., None, :] @ S)[..., 0, :]

    def packed(y):
        out = y.new_zeros((s["tokens"],) + y.shape[2:])
        out[pick[mask]] = y[mask]
        return out

    out = {"o": packed(o)}
    if c["op"] == "train":
        do = steps(s["do"], 1, 0)
        grads = {n: torch.zeros_like(x) for n, x in (("dq", q), ("dk", k), ("dv", v), ("dlog_alpha", a), ("dbeta", beta))}
        G = torch.zeros_like(S)
        if s["dS"] is not None:
            G = G + s["dS"].double()
        for t0 in reversed(range(0, L, 48)):
            seg, x = [], kept.pop()
            for t in range(t0, min(L, t0 + 48)):
                seg.append((t, _exact_step(c, x, a[t], k[t], v[t], beta[t])))
                x = seg[-1][1][3]
            for t, (Sd, r, w, Sn) in reversed(seg):
                grads["dq"][t] = (Sn @ do[t][..., None])[..., 0]
                G = G + q[t][..., :, None] * do[t][..., None, :]
                dw = (k[t][..., None, :] @ G)[..., 0, :]
                grads["dk"][t] = (G @ w[..., None])[..., 0]
                grads["dv"][t] = beta[t] * dw
                grads["dbeta"][t] = (r * dw).sum(-1, keepdim=True)
                if c["form"] != MAMBA2:
                    grads["dk"][t] -= (Sd @ (beta[t] * dw)[..., None])[..., 0]
                    G = G - k[t][..., :, None] * (beta[t] * dw)[..., None, :]
                dl = (G * Sd).sum(-1)
                grads["dlog_alpha"][t] = dl if c["form"] == KDA else dl.sum(-1, keepdim=True)
                G = a[t][..., :, None] * G
        for n in ("dq", "dk"):
            grads[n] = grads[n].view(L, B, c["k_heads"], rep, c["d_k"]).sum(3)
        for n, y in grads.items():
            y = packed(y)
            out[n] = y[..., 0] if n == "dbeta" or (n == "dlog_alpha" and c["form"] != KDA) else y
        if c["state"]:
            out["dS0"] = G
    if c["state"]:
        out["S"] = S
    return out


def _exact_tree(c, s):
    """Every node's dense state from its parent's, the sink coefficient (the same recurrence
    on the values' coordinate along vbar) as one more column; of the stored state after the
    commit, the sink and the count have values of their own."""
    B, H, m = c["batch"], c["heads"], c["R"] + c["W"]
    vb = s["vbar"][0].double()
    n = s["ncols0"][:, 0].long()
    U, V = s["U"][:, 0].double(), s["V"][:, 0].double()
    sc = s["scale0"][:, 0].double()
    U = U * (sc[:, :, None, :] if c["form"] == KDA else sc[..., :m, None])
    gone = torch.arange(m, device="cuda")[None, None, :] >= n[..., None]
    U[gone], V[gone] = 0, 0
    a0 = s["a0"][:, 0].double()[..., :, None]
    root = torch.cat([a0 * vb[..., None, :] + U.transpose(-1, -2) @ V, a0], -1)
    v = s["v"].double()
    v = torch.cat([v, (v * vb).sum(-1, keepdim=True) / vb.square().sum(-1, keepdim=True)], -1)
    a = s["alpha"].double() if c["form"] == KDA else s["alpha"].double()[..., None]
    o = torch.zeros(s["v"].shape, dtype=torch.float64, device="cuda")
    w = torch.zeros_like(o)
    at = [root]
    ends, deep = root.clone(), [torch.zeros(B, dtype=torch.int32, device="cuda")]
    rows = torch.arange(B, device="cuda")
    for t in range(c["nodes"]):
        p = s["parent"][:, t].long()
        S = torch.zeros_like(root)
        d = torch.zeros_like(deep[0])
        for j in range(t + 1):
            hit = p == j - 1
            S[hit], d[hit] = at[j][hit], deep[j][hit]
        _, _, wt, Sn = _exact_step(c, S, a[:, t], s["k"][:, t].double(), v[:, t], s["beta"][:, t].double()[..., None])
        on = p >= -1
        w[:, t] = torch.where(on[:, None, None], wt[..., :-1], 0)
        o[:, t] = torch.where(on[:, None, None], (s["q"][:, t].double()[..., None, :] @ Sn)[..., 0, :-1], 0)
        at.append(Sn)
        deep.append(d + 1)
        end = rows[s["leaf"] == t]
        ends[end] = Sn[end]
    count = s["ncols0"].clone()
    for t in range(c["nodes"]):
        hit = s["leaf"] == t
        count[hit] += deep[t + 1][hit][:, None, None]
    return {"o": o, "w": w, "a": ends[:, None, ..., -1], "U": None, "V": None, "scale": None, "ncols": count}


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        if case["op"] == "tree":
            if case["batch"] * case["heads"] * case["nodes"] * case["d_k"] * case["d_v"] * 8 > 60e9:
                return None
            return _exact_tree(case, s)
        return _exact_scan(case, s)
