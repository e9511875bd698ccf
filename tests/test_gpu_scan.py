"""seed_dense_scan and its backward pass against the float64 token-by-token oracle."""

import numpy as np
import pytest
import torch

from oracle import sequence
from parity_util import ensure_lib
from sequence_util import F32, FORMS, TYPES, close, device, token_values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


class Problem:
    """One packed problem on the device and, for the oracle, in float64."""

    def __init__(self, form, lens, h, h_k, dk, dv, typ="f32", state=True, seed=0, lead=0, tail=0, edit=None):
        from rank_recurrent_state_b200 import seed as S
        self.S, self.form, self.lens, self.h, self.h_k = S, FORMS[form], lens, h, h_k
        rng = np.random.default_rng(seed)
        self.off = np.concatenate([[0], np.cumsum(lens)]) + lead
        n = int(self.off[-1]) + tail
        vals = dict(zip(["q", "k", "v", "alpha", "beta"], token_values(self.form, (n,), h_k, h, dk, dv, rng)))
        vals["do"] = rng.normal(size=(n, h, dv))
        if edit:
            edit(vals)
        t = TYPES[typ]
        self.x, self.r = {}, {}
        for name, val in vals.items():
            self.x[name], self.r[name] = device(val, torch.float32 if name in ("alpha", "beta") else t)
        mat = (len(lens), h, dk, dv)
        self.S0, self.r0 = device(rng.normal(size=mat) * 0.3) if state else (None, np.zeros(mat))
        self.dS, self.rd = device(rng.normal(size=mat) * 0.3) if state else (None, np.zeros(mat))
        self.dims = S.ScanDims(self.form, len(lens), n, h, h_k, dk, dv, max(lens), S.FACTOR_NAMES[typ])
        self.offsets = torch.tensor(self.off.tolist(), dtype=torch.int32, device="cuda")
        self.ws = S.ScanWorkspace(self.dims, backward=True)

    def outputs(self, fill=float("nan")):
        x = self.x
        full = lambda y, dtype=None: torch.full_like(y, fill, dtype=dtype)  # noqa: E731
        mat = (len(self.lens), self.h, self.dims.d_k, self.dims.d_v)
        return {"o": full(x["v"]), "S": torch.full(mat, fill, device="cuda"), "dq": full(x["q"]), "dk": full(x["k"]),
                "dv": full(x["v"]), "dla": full(x["alpha"]), "dbeta": full(x["beta"]),
                "dS0": torch.full(mat, fill, device="cuda")}

    def forward(self, out, stream=None):
        x = self.x
        self.S.seed_dense_scan(self.dims, self.offsets, x["q"], x["k"], x["v"], x["alpha"], x["beta"], out["o"],
                               self.ws, S0=self.S0, S_out=out["S"], stream=stream)

    def backward(self, out, stream=None):
        x = self.x
        self.S.seed_dense_scan_backward(self.dims, self.offsets, x["q"], x["k"], x["v"], x["alpha"], x["beta"],
                                        x["do"], out["dq"], out["dk"], out["dv"], out["dla"], out["dbeta"], self.ws,
                                        S0=self.S0, dS_out=self.dS, dS0=out["dS0"], stream=stream)

    def reference(self, s, backward):
        """The oracle's answers for sequence s (dq, dk summed over shared heads)."""
        rows = slice(int(self.off[s]), int(self.off[s + 1]))
        rep = self.h // self.h_k
        q, k = (np.repeat(self.r[n][rows], rep, axis=1) for n in ("q", "k"))
        v, al, be, do = (self.r[n][rows] for n in ("v", "alpha", "beta", "do"))
        o, S = sequence.scan(self.form, q, k, v, al, be, self.r0[s])
        ref = {"o": o, "S": S}
        if backward:
            g = sequence.scan_backward(self.form, q, k, v, al, be, self.r0[s], do, self.rd[s])
            share = lambda y: y.reshape(y.shape[0], self.h_k, rep, y.shape[2]).sum(2)  # noqa: E731
            ref.update(dq=share(g[0]), dk=share(g[1]), dv=g[2], dla=g[3], dbeta=g[4], dS0=g[5])
        return ref

    def check(self, out, backward=True, skip=()):
        """Every output over all sequences that are not in `skip`."""
        refs = {s: self.reference(s, backward) for s in range(len(self.lens)) if s not in skip}
        for name in ("o", "S") + (("dq", "dk", "dv", "dla", "dbeta", "dS0") if backward else ()):
            per_seq = name in ("S", "dS0")
            got = [out[name][s] if per_seq else out[name][int(self.off[s]):int(self.off[s + 1])] for s in refs]
            ref = [refs[s][name] for s in refs]
            close(torch.cat([g.reshape(-1) for g in got]), np.concatenate([r.reshape(-1) for r in ref]), name)


DIMS = [(16, 16), (32, 32), (64, 64), (128, 128), (128, 64), (64, 128)]
LENS = [0, 1, 63, 64, 65, 130, 17]      # empty, one token, around a chunk, ragged


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("typ", TYPES)
def test_every_output(form, dk, dv, typ):
    p = Problem(form, LENS, 4, 2, dk, dv, typ, seed=dk + dv)
    out = p.outputs()
    p.forward(out)
    p.backward(out)
    assert p.S.seed_get_status(p.ws) == 0
    p.check(out)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("lens", [[1], [2, 1, 1], [5], [33], [64], [128, 128], [700]])
def test_lengths_without_states(form, lens):
    p = Problem(form, lens, 3, 3, 64, 64, "f32", state=False, seed=sum(lens))
    out = p.outputs()
    p.forward(out)
    p.backward(out)
    assert p.S.seed_get_status(p.ws) == 0
    p.check(out)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("h,h_k", [(6, 1), (6, 3), (5, 5)])
def test_shared_key_heads(form, h, h_k):
    p = Problem(form, [90, 40], h, h_k, 128, 64, "bf16", seed=h)
    out = p.outputs()
    p.forward(out)
    p.backward(out)
    p.check(out)


@pytest.mark.parametrize("form", FORMS)
def test_zero_and_tiny_decays(form):
    """Resets (alpha = 0) and decays whose product underflows: finite, and exact."""
    def edit(v):
        v["alpha"][5] = 0.0
        v["alpha"][64:70] = 1e-30
        v["alpha"][100, 0] = 0.0
    p = Problem(form, [150], 3, 3, 128, 128, "f32", seed=4, edit=edit)
    out = p.outputs()
    p.forward(out)
    p.backward(out)
    assert p.S.seed_get_status(p.ws) == 0
    p.check(out)
    assert not out["dla"][5].any()


@pytest.mark.parametrize("form", ["gdn", "kda"])
def test_repeated_keys_and_full_writes(form):
    """The same key at every token, beta = 1, no decay: the triangular system's worst
    entries.  Every token then overwrites the last value, so o = (q . k) v."""
    def edit(v):
        v["k"][:] = v["k"][:1]
        v["beta"][:] = 1.0
        v["alpha"][:] = 1.0
    p = Problem(form, [200], 2, 2, 128, 128, "f32", state=False, seed=5, edit=edit)
    out = p.outputs()
    p.forward(out)
    p.backward(out)
    if form == "gdn":
        # The erase leaves G' without the component along k, the only one S' has: their
        # product summed over the head, dlog alpha, is an exact zero, summed from terms of the
        # size of q dq and k dk.  Each is rounded to float32, so what stands there is bounded
        # by F32 of those terms.
        ref = p.reference(0, True)
        terms = np.linalg.norm(p.r["q"] * ref["dq"]) + np.linalg.norm(p.r["k"] * ref["dk"])
        assert np.linalg.norm(ref["dla"]) < 1e-9 * terms
        assert float(out["dla"].double().norm()) <= F32 * terms * 64 ** 0.5      # one chunk's suffix sums
        out["dla"].copy_(torch.from_numpy(ref["dla"]))
    p.check(out)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("scale", [1e-12, 1e8])
def test_scales_far_from_one(form, scale):
    """Values, states and output gradients scaled alike: every result scales with them."""
    def edit(v):
        v["v"] *= scale
        v["do"] *= scale
    p = Problem(form, [100, 70], 2, 2, 128, 128, "f32", seed=6, edit=edit)
    p.S0.mul_(scale), p.dS.mul_(scale)
    p.r0, p.rd = p.S0.double().cpu().numpy(), p.dS.double().cpu().numpy()
    out = p.outputs()
    p.forward(out)
    p.backward(out)
    p.check(out)


def test_rows_outside_the_sequences_stay():
    p = Problem("gdn", [70, 3], 2, 1, 128, 128, "bf16", seed=7, lead=5, tail=9)
    for n in ("q", "k", "v", "alpha", "beta", "do"):       # never read either
        p.x[n][:5] = float("nan")
        p.x[n][-9:] = float("nan")
    out = p.outputs(fill=-3.0)
    p.forward(out)
    p.backward(out)
    assert p.S.seed_get_status(p.ws) == 0
    p.check(out)
    for n in ("o", "dq", "dk", "dv", "dla", "dbeta"):
        assert (out[n][:5] == -3).all() and (out[n][-9:] == -3).all(), n


@pytest.mark.parametrize("form", FORMS)
def test_a_bad_sequence_leaves_its_neighbours(form):
    """NaN and infinite tokens of one sequence reach no other one and raise the flag."""
    def edit(v):
        v["v"][75] = np.nan
        v["k"][80] = np.inf
        v["q"][74] = np.inf
    p = Problem(form, [70, 30, 64, 40], 2, 2, 128, 128, "f32", seed=8, edit=edit)
    out = p.outputs()
    p.forward(out)
    p.backward(out)
    assert p.S.seed_get_status(p.ws) == p.S.FLAG_NONFINITE
    p.check(out, skip=[1])


def test_states_in_place_and_split_runs():
    """A sequence in two calls through an in-place state equals one call."""
    p = Problem("gdn", [200], 4, 2, 128, 128, "f32", seed=9)
    out = p.outputs()
    p.forward(out)
    S = p.S0.clone()
    o = torch.empty_like(out["o"])
    for a, b in ((0, 77), (77, 200)):
        d = p.S.ScanDims(p.form, 1, b - a, 4, 2, 128, 128, b - a)
        x = {n: t[a:b].contiguous() for n, t in p.x.items()}
        oo = torch.empty_like(x["v"])
        off = torch.tensor([0, b - a], dtype=torch.int32, device="cuda")
        p.S.seed_dense_scan(d, off, x["q"], x["k"], x["v"], x["alpha"], x["beta"], oo, p.S.ScanWorkspace(d), S0=S, S_out=S)
        o[a:b] = oo
    close(o, out["o"].double().cpu().numpy(), "o")
    close(S, out["S"].double().cpu().numpy(), "S")


def test_scan_equals_the_dense_step():
    p = Problem("kda", [1, 1, 1], 4, 4, 128, 128, "f32", seed=10)
    out = p.outputs()
    p.forward(out)
    S = p.S
    d = S.Dims(p.form, 3, 1, 4, 128, 128, 16, 16)
    st, o = p.S0.clone(), torch.empty_like(out["o"])
    S.seed_dense_step(d, st, 0, p.x["q"], p.x["k"], p.x["v"], p.x["alpha"], p.x["beta"], o, S.Workspace(d))
    close(out["o"], o.double().cpu().numpy(), "o")
    close(out["S"], st.double().cpu().numpy(), "S")


def test_no_tokens_and_no_backward_state():
    from rank_recurrent_state_b200 import seed as S
    d = S.ScanDims(0, 2, 0, 2, 2, 64, 64, 0)
    ws = S.ScanWorkspace(d, backward=True)
    e = torch.empty(0, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    S0 = torch.randn(2, 2, 64, 64, device="cuda")
    S_out, dS0 = torch.empty_like(S0), torch.empty_like(S0)
    S.seed_dense_scan(d, off, e, e, e, e, e, e, ws, S0=S0, S_out=S_out)
    S.seed_dense_scan_backward(d, off, e, e, e, e, e, e, e, e, e, e, e, ws, S0=S0, dS_out=S0, dS0=dS0)
    assert torch.equal(S_out, S0) and torch.equal(dS0, S0)
    S.seed_dense_scan(d, off, e, e, e, e, e, e, ws, S_out=S_out)
    assert not S_out.any() and S.seed_get_status(ws) == 0


def test_bad_offsets_are_flagged():
    """Offsets outside the arrays: a flag, empty sequences, no access outside."""
    p = Problem("gdn", [64, 64, 64], 2, 2, 128, 128, "f32", seed=11)
    for off in ([0, 64, 300, 400], [0, 128, 64, 192], [-5, 64, 128, 192], [0, 64, 128, 2 ** 31 - 1]):
        p.offsets.copy_(torch.tensor(off, dtype=torch.int32))
        out = p.outputs(fill=0.0)
        p.forward(out)
        p.backward(out)
        assert p.S.seed_get_status(p.ws) & p.S.FLAG_BADINDEX


@pytest.mark.parametrize("lens", [[150, 64], [1, 1]])
def test_streams_graphs_and_repeats(lens):
    """Side stream, captured and replayed on new inputs; two runs give the same bits."""
    p = Problem("kda", lens, 4, 2, 128, 128, "bf16", seed=12)
    want, out = p.outputs(), p.outputs()
    p.forward(want), p.backward(want)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        p.forward(out), p.backward(out)
    st.synchronize()
    for n in want:
        assert torch.equal(want[n], out[n]), n
    g, out2 = torch.cuda.CUDAGraph(), p.outputs()
    with torch.cuda.graph(g):
        p.forward(out2), p.backward(out2)
    p.x["v"].mul_(0.5)
    p.r["v"] = p.x["v"].double().cpu().numpy()
    g.replay()
    torch.cuda.synchronize()
    p.check(out2)


def test_two_graphs_share_a_workspace():
    a = Problem("gdn", [130], 4, 4, 128, 128, "f32", seed=13)
    b = Problem("gdn", [130], 4, 4, 128, 128, "f32", seed=14)
    b.ws = a.ws
    graphs = []
    for p in (a, b):
        p.forward(p.outputs()), p.backward(p.outputs())
        out, g = p.outputs(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            p.forward(out), p.backward(out)
        graphs.append((p, out, g))
    for _ in range(2):
        for _, _, g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for p, out, _ in graphs:
        p.check(out)


def test_gradients_match_differences():
    """A directional difference of the device's own forward, float64 sums of its outputs:
    step h, error h^2 of the third derivative plus 2^-23 of the loss's terms / h."""
    p = Problem("kda", [70], 2, 1, 64, 64, "f32", seed=15)
    out = p.outputs()
    p.backward(out)
    rng = np.random.default_rng(3)

    def loss():
        y = p.outputs()
        p.forward(y)
        return float((y["o"].double() * p.x["do"].double()).sum() + (y["S"].double() * p.dS.double()).sum())

    h = 2e-3
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("beta", "dbeta"), ("alpha", "dla")):
        x = p.x[name]
        was = x.clone()
        d = torch.from_numpy(rng.normal(size=tuple(x.shape))).cuda().float()
        terms = float((out[grad].double() * d.double()).square().sum().sqrt())
        vals = []
        for s in (h, -h):
            x.copy_(was * torch.exp(s * d) if name == "alpha" else was + s * d)
            vals.append(loss())
        x.copy_(was)
        num, ana = (vals[0] - vals[1]) / (2 * h), float((out[grad].double() * d.double()).sum())
        assert abs(num - ana) <= 2e-2 * terms + 2e-3 * abs(ana), (name, num, ana, terms)


def test_float32_results_are_float32_accurate():
    """A long sequence keeps the per-chunk error: the norm bound holds at every chunk."""
    p = Problem("gdn", [1500], 2, 1, 128, 128, "bf16", seed=16)
    out = p.outputs()
    p.forward(out)
    ref = p.reference(0, False)
    close(out["S"][0], ref["S"], "S")
    eps = torch.finfo(torch.bfloat16).eps / 2
    o = out["o"].double().cpu().numpy()
    for t in range(0, 1500, 64):
        r = ref["o"][t:t + 64]
        assert np.linalg.norm(o[t:t + 64] - r) <= (F32 + eps) * np.linalg.norm(r), t


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("hint", [1, 2, 20, 1000])
def test_max_len_decides_speed_alone(form, hint):
    """Sequences longer and shorter than the hint: every kernel takes every length."""
    from dataclasses import replace
    p = Problem(form, [3, 70, 0, 130, 1], 4, 2, 128, 64, "f16", seed=17)
    p.dims = replace(p.dims, max_len=hint)
    p.ws = p.S.ScanWorkspace(p.dims, backward=True)
    out = p.outputs()
    p.forward(out)
    p.backward(out)
    assert p.S.seed_get_status(p.ws) == 0
    p.check(out)


@pytest.mark.parametrize("form", FORMS)
def test_many_sequences_and_heads(form):
    """More (sequence, head) pairs than SMs, more sequences than one probe of the chunk
    look-up, lengths around the switch between the kernels."""
    rng = np.random.default_rng(18)
    lens = rng.integers(0, 30, size=70).tolist()
    p = Problem(form, lens, 6, 3, 64, 64, "bf16", seed=18)
    out = p.outputs()
    p.forward(out)
    p.backward(out)
    assert p.S.seed_get_status(p.ws) == 0
    p.check(out)


def test_arrays_beyond_32_bit_elements():
    """v and o of more than 2^31 elements: the last sequence equals a call of its own."""
    from rank_recurrent_state_b200 import seed as S
    h, d, n, tail = 64, 128, 262400, 150
    g = torch.Generator(device="cuda").manual_seed(19)
    k = torch.randn(n, 1, d, generator=g, device="cuda")
    k = (k / k.norm(dim=-1, keepdim=True)).bfloat16()
    v = torch.empty(n, h, d, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    alpha = torch.rand(n, h, generator=g, device="cuda") * 0.1 + 0.9
    beta = torch.rand(n, h, generator=g, device="cuda")
    assert v.numel() > 2 ** 31
    o = torch.empty_like(v)
    off = torch.tensor([0, n - tail, n], dtype=torch.int32, device="cuda")
    dims = S.ScanDims(S.SEED_GDN, 2, n, h, 1, d, d, n, S.SEED_FACTORS_BF16)
    ws = S.ScanWorkspace(dims)
    S_out = torch.empty(2, h, d, d, device="cuda")
    S.seed_dense_scan(dims, off, k, k, v, alpha, beta, o, ws, S_out=S_out)
    assert S.seed_get_status(ws) == 0
    one = S.ScanDims(S.SEED_GDN, 1, tail, h, 1, d, d, tail, S.SEED_FACTORS_BF16)
    x = [t[n - tail:].contiguous() for t in (k, k, v, alpha, beta)]
    o1, S1 = torch.empty_like(x[2]), torch.empty(1, h, d, d, device="cuda")
    S.seed_dense_scan(one, torch.tensor([0, tail], dtype=torch.int32, device="cuda"), *x, o1, S.ScanWorkspace(one), S_out=S1)
    assert torch.equal(o[n - tail:], o1) and torch.equal(S_out[1], S1[0])


def test_the_binding_refuses_strided_and_foreign_arrays():
    p = Problem("gdn", [20], 2, 2, 64, 64, "f32", seed=20)
    out = p.outputs()
    p.x["v"] = torch.stack([p.x["v"], p.x["v"]], -1)[..., 0]
    with pytest.raises(ValueError, match="contiguous"):
        p.forward(out)
    p.x["v"] = p.x["v"].contiguous().cpu()
    with pytest.raises(ValueError, match="v: on cpu"):
        p.forward(out)
    assert torch.isnan(out["o"]).all()
