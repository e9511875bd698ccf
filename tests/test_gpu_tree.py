"""seed_decode_tree and its commit against the float64 oracle and the decode step."""

import numpy as np
import pytest
import torch

from oracle import sequence
from parity_util import ensure_lib
from sequence_util import FORMS, TYPES, close, device, token_values

pytestmark = pytest.mark.gpu
FACTORS = {"f32": 0, "f16": 1, "bf16": 2}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def random_tree(B, N, rng, unused=0.2):
    parent = np.full((B, N), -2, dtype=np.int32)
    for b in range(B):
        ok = []
        for t in range(N):
            if t and rng.random() < unused:
                continue
            parent[b, t] = rng.choice([-1] + ok[-6:])
            ok.append(t)
    return parent


class Problem:
    def __init__(self, form, B, N, H, dk, dv, R, W, c, factors="f32", seed=0, layers=2, layer=1, parent=None):
        from rank_recurrent_state_b200 import seed as S
        self.S, self.form, self.layer = S, FORMS[form], layer
        rng = np.random.default_rng(seed)
        self.rng = rng
        self.parent = random_tree(B, N, rng) if parent is None else np.asarray(parent, dtype=np.int32)
        vals = token_values(self.form, (B, N), H, H, dk, dv, rng)
        self.x, self.r = {}, {}
        for name, val in zip(["q", "k", "v", "alpha", "beta"], vals):
            self.x[name], self.r[name] = device(val)
        m = R + W
        self.dims = S.Dims(self.form, B, layers, H, dk, dv, R, W, FACTORS[factors])
        vbar, self.vbar = device(rng.normal(size=(layers, H, dv)))
        st = S.State.allocate(self.dims, vbar)
        t = TYPES[factors]
        U, self.U = device(rng.normal(size=st.U.shape) / dk ** 0.5, t)
        V, self.V = device(rng.normal(size=st.V.shape), t)
        a, self.a = device(rng.normal(size=st.a.shape))
        sc, self.sc = device(rng.uniform(0.3, 1.0, size=st.scale.shape))
        st.U.copy_(U), st.V.copy_(V), st.a.copy_(a), st.scale.copy_(sc)
        self.c = np.broadcast_to(np.asarray(c).reshape(-1, 1), (B, H))
        st.ncols.copy_(torch.from_numpy(np.ascontiguousarray(np.broadcast_to(self.c[:, None], st.ncols.shape))))
        self.st, self.ws = st, S.Workspace(self.dims)
        self.par = torch.from_numpy(self.parent).cuda()

    def dense(self, b):
        """The layer's stored states of request b (H, d_k, d_v), float64."""
        l, out = self.layer, []
        for h in range(self.dims.heads):
            c = int(self.c[b, h])
            U, V, sc = self.U[b, l, h, :c], self.V[b, l, h, :c], self.sc[b, l, h]
            U = U * (sc if self.form == FORMS["kda"] else sc[:c, None])
            out.append(np.outer(self.a[b, l, h], self.vbar[l, h]) + U.T @ V)
        return np.array(out)

    def read(self, fill=float("nan")):
        o, w = torch.full_like(self.x["v"], fill), torch.full_like(self.x["v"], fill)
        x = self.x
        self.S.seed_decode_tree(self.dims, self.st, self.layer, self.par, x["q"], x["k"], x["v"], x["alpha"],
                                x["beta"], o, w, self.ws)
        return o, w

    def commit(self, leaf, w):
        x = self.x
        self.S.seed_decode_tree_commit(self.dims, self.st, self.layer, self.par,
                                       torch.tensor(leaf, dtype=torch.int32, device="cuda"), x["k"], x["v"],
                                       x["alpha"], x["beta"], w, self.ws)

    def oracle(self, b):
        r = {n: v[b] for n, v in self.r.items()}
        return sequence.tree(self.form, self.dense(b), self.parent[b].tolist(), r["q"], r["k"], r["v"], r["alpha"],
                             r["beta"])

    def device_dense(self):
        d = self.dims
        out = torch.empty(d.batch, d.heads, d.d_k, d.d_v, device="cuda")
        self.S.seed_state_to_dense(d, self.st, self.layer, out, self.ws)
        return out


DIMS = [(16, 16), (32, 32), (64, 64), (128, 128), (128, 64), (64, 128)]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("factors", FACTORS)
def test_tree_and_commit(form, dk, dv, factors):
    N, B = 11, 5
    p = Problem(form, B, N, 3, dk, dv, 4, 12, [4, 5, 6, 4, 8], factors, seed=dk + dv)
    before = {n: getattr(p.st, n).clone() for n in ("a", "U", "V", "scale", "ncols")}
    o, w = p.read()
    for n, t in before.items():
        assert torch.equal(t, getattr(p.st, n)), n          # reads only
    refs = [p.oracle(b) for b in range(B)]
    close(o, np.array([r[0] for r in refs]), "o")
    close(w, np.array([r[1] for r in refs]), "w")
    leaf = []
    for b in range(B):
        fits = [t for t in range(N) if refs[b][2][t] is not None
                and len(sequence.path(p.parent[b], t)) <= 16 - p.c[b, 0]]
        leaf.append(int(p.rng.choice(fits)) if b != 2 else -1)
    p.commit(leaf, w)
    assert p.S.seed_get_status(p.ws) == 0
    want = np.array([p.dense(b) if leaf[b] < 0 else refs[b][2][leaf[b]] for b in range(B)])
    got = p.device_dense()
    if factors == "f32":
        close(got, want, "state")
    else:      # the appended pairs are rounded: half a step of each k and column
        eps = torch.finfo(TYPES[factors]).eps
        assert np.linalg.norm(got.cpu().numpy() - want) <= (eps + 2e-5) * np.linalg.norm(want)
    n = p.st.ncols[:, p.layer].cpu().numpy()
    for b in range(B):
        assert (n[b] == p.c[b] + (len(sequence.path(p.parent[b], leaf[b])) if leaf[b] >= 0 else 0)).all()
    assert torch.equal(p.st.U[:, 0], before["U"][:, 0]) and torch.equal(p.st.a[:, 0], before["a"][:, 0])


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("N", [1, 2, 7, 8, 9, 33, 64])
def test_node_counts_and_column_counts(form, N):
    """From one node to the most, over states of no columns up to full ones."""
    p = Problem(form, 4, N, 2, 128, 128, 32, 64, [0, 1, 64, 96], "f32", seed=N)
    o, w = p.read()
    assert p.S.seed_get_status(p.ws) == 0
    refs = [p.oracle(b) for b in range(4)]
    close(o, np.array([r[0] for r in refs]), "o")
    close(w, np.array([r[1] for r in refs]), "w")


@pytest.mark.parametrize("form", FORMS)
def test_a_chain_is_decode_steps(form):
    """A chain committed whole leaves what as many decode steps leave, and the compression
    that follows takes it the same way."""
    N = 12
    p = Problem(form, 3, N, 2, 128, 128, 16, 16, [20, 20, 20], "f32", seed=3, parent=[list(range(-1, N - 1))] * 3)
    S, d, st = p.S, p.dims, p.st
    twin = S.State.allocate(d, st.vbar)
    twin.load_state_dict(st.state_dict())
    o, w = p.read()
    p.commit([N - 1] * 3, w)
    for t in range(N):
        x = {n: p.x[n][:, t].contiguous() for n in p.x}
        ot = torch.empty_like(x["v"])
        S.seed_decode_step(d, twin, p.layer, x["q"], x["k"], x["v"], x["alpha"], x["beta"], ot, p.ws)
        close(o[:, t], ot.double().cpu().numpy(), f"o {t}")
    for n in ("a", "U", "V", "scale"):
        close(getattr(st, n)[:, p.layer], getattr(twin, n)[:, p.layer].double().cpu().numpy(), n)
    assert torch.equal(st.ncols, twin.ncols)
    S.seed_compress(d, st, p.layer, p.ws)
    assert S.seed_get_status(p.ws) == 0 and (st.ncols[:, p.layer] == 16).all()


@pytest.mark.parametrize("form", FORMS)
def test_branches_do_not_meet(form):
    """NaN, infinities and a zero decay in one branch stay in it."""
    parent = [[-1, 0, 0, 1, 2, -1]]
    p = Problem(form, 1, 6, 2, 64, 64, 8, 8, [8], "f32", seed=5, parent=parent)
    p.x["v"][:, 1] = float("nan")
    p.x["k"][:, 3] = float("inf")
    p.x["alpha"][:, 4] = 0.0
    p.r["alpha"][:, 4] = 0.0
    o, w = p.read()
    assert p.S.seed_get_status(p.ws) == p.S.FLAG_NONFINITE
    ref = p.oracle(0)
    good = [0, 2, 4, 5]
    close(o[:, good], ref[0][None][:, good], "o")
    close(w[:, good], ref[1][None][:, good], "w")


def test_refusals_on_the_device():
    p = Problem("gdn", 6, 4, 2, 64, 64, 4, 4, [4, 7, 9, 4, 4, 4], "f32", seed=6,
                parent=[[-1, 0, 1, 2]] * 3 + [[-1, 1, 1, 0], [-1, 0, -7, 2], [0, 0, 1, 2]])
    S = p.S
    o, w = p.read(fill=5.0)
    assert S.seed_get_status(p.ws) == S.FLAG_BADINDEX | S.FLAG_BADCOLS
    assert (o[2] == 5).all() and (w[2] == 5).all()                       # a bad column count
    assert not o[3, 1:3].any() and o[3, 3].any()                         # its own parent, and below it
    assert not o[4, 2:].any() and not o[5].any()
    before = {n: getattr(p.st, n).clone() for n in ("a", "U", "V", "scale", "ncols")}
    same = lambda b: all(torch.equal(t[b], getattr(p.st, n)[b]) for n, t in before.items())  # noqa: E731
    for leaf, flag in (([-1, 3, -1, -1, -1, -1], S.FLAG_FULL), ([-1, -1, 0, -1, -1, -1], S.FLAG_BADCOLS),
                       ([-1, -1, -1, 2, -1, -1], S.FLAG_BADINDEX), ([-1, -1, -1, -1, 2, -1], S.FLAG_BADINDEX),
                       ([4, -1, -1, -1, -1, -1], S.FLAG_BADINDEX), ([-1, -1, -1, -1, -1, 3], S.FLAG_BADINDEX),
                       ([-3] * 6, 0)):
        p.commit(leaf, w)
        assert S.seed_get_status(p.ws) == flag, leaf
        assert all(same(b) for b in range(6)), leaf
    p.st.vbar.zero_()
    p.commit([0] + [-1] * 5, w)
    assert S.seed_get_status(p.ws) == S.FLAG_ZERO_VBAR and same(0)


def test_captured_and_replayed():
    p = Problem("kda", 4, 9, 3, 128, 128, 8, 24, [8, 9, 10, 11], "bf16", seed=7)
    want = p.read()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g, out = torch.cuda.CUDAGraph(), [torch.empty_like(x) for x in want]
    x = p.x
    with torch.cuda.graph(g, stream=st):
        p.S.seed_decode_tree(p.dims, p.st, p.layer, p.par, x["q"], x["k"], x["v"], x["alpha"], x["beta"], *out, p.ws)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, out))


@pytest.mark.parametrize("form", FORMS)
def test_prefill_convert_draft_commit(form):
    """As they are used together: a scan leaves the dense states, the conversion stores
    them, a draft is read and its path committed, a decode step follows."""
    from rank_recurrent_state_b200 import seed as S
    B, H, d, R, W, N = 3, 2, 64, 16, 8, 6
    f = FORMS[form]
    rng = np.random.default_rng(8)
    lens = [40, 7, 90]
    x = token_values(f, (sum(lens),), H, H, d, d, rng)
    (q, qr), (k, kr), (v, vr), (al, ar), (be, br) = (device(t) for t in x)
    sd = S.ScanDims(f, B, sum(lens), H, H, d, d, max(lens))
    off = torch.tensor([0, 40, 47, 137], dtype=torch.int32, device="cuda")
    S_out, o = torch.empty(B, H, d, d, device="cuda"), torch.empty_like(v)
    S.seed_dense_scan(sd, off, q, k, v, al, be, o, S.ScanWorkspace(sd), S_out=S_out)
    p = Problem(form, B, N, H, d, d, R, W, [R] * B, "f32", seed=9, layers=1, layer=0,
                parent=[[-1, 0, 1, 0, 3, 4]] * B)
    S.seed_state_init_from_dense(p.dims, p.st, 0, S_out, p.ws)
    root = p.device_dense().double().cpu().numpy()
    o, w = p.read()
    p.commit([5, 2, -1], w)
    assert S.seed_get_status(p.ws) == 0
    dense = p.device_dense()
    for b, leaf in enumerate([5, 2, -1]):
        r = {n: t[b] for n, t in p.r.items()}
        ro, rw, states = sequence.tree(p.form, root[b], p.parent[b].tolist(), r["q"], r["k"], r["v"], r["alpha"], r["beta"])
        close(o[b], ro, "o")
        close(dense[b], states[leaf] if leaf >= 0 else root[b], "state")
    y = S.alloc_step_inputs(p.dims)
    for n in ("q", "k", "v", "alpha", "beta"):
        y[n].copy_(p.x[n][:, 0])
    S.seed_decode_step(p.dims, p.st, 0, y["q"], y["k"], y["v"], y["alpha"], y["beta"], y["o"], p.ws)
    assert S.seed_get_status(p.ws) == 0
    assert p.st.ncols[:, 0, 0].tolist() == [R + 5, R + 4, R + 1]
