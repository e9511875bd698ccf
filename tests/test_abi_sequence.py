"""Host-side refusals of the scan and tree entry points (no GPU)."""

import ctypes

import pytest
import torch

from rank_recurrent_state_b200 import _lib, build
from rank_recurrent_state_b200 import seed as S

A, MIS, BIG = 0x10000, 0x10004, 1 << 40


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def _scan(**kw):
    base = dict(form=0, seqs=2, heads=4, k_heads=2, d_k=128, d_v=128, max_len=100, elem=2, tokens=150)
    base.update(kw)
    return _lib.seed_scan_dims(**base)


BAD = [(dict(form=3), -1), (dict(elem=3), -1), (dict(elem=-1), -1), (dict(seqs=0), -1), (dict(heads=0), -1),
       (dict(k_heads=0), -1), (dict(k_heads=3), -2), (dict(tokens=-1), -1), (dict(max_len=-1), -1),
       (dict(d_k=48), -2), (dict(d_k=64, d_v=32), -2), (dict(tokens=2 ** 31), -2),
       (dict(seqs=2 ** 30, heads=64, k_heads=64), -2)]


@pytest.mark.parametrize("kw,code", BAD)
def test_scan_rejects_dims(lib, kw, code):
    d = ctypes.byref(_scan(**kw))
    assert lib.seed_dense_scan(d, *[A] * 10, BIG, None) == code
    assert lib.seed_dense_scan_backward(d, *[A] * 16, BIG, None) == code
    assert lib.seed_scan_workspace_bytes(d, 0) == 0 and lib.seed_scan_workspace_bytes(d, 1) == 0
    assert lib.seed_dense_scan(None, *[A] * 10, BIG, None) == -1


def test_scan_rejects_pointers_and_workspaces(lib):
    d = ctypes.byref(_scan())
    fwd, bwd = lib.seed_scan_workspace_bytes(d, 0), lib.seed_scan_workspace_bytes(d, 1)
    assert 256 <= fwd <= bwd
    optional = {6: "S0", 8: "S_out"}
    for i in range(9):            # offsets q k v alpha beta S0 o S_out
        args = [A] * 10
        if i not in optional:
            args[i] = None
            assert lib.seed_dense_scan(d, *args, BIG, None) == -1
        args[i] = MIS
        assert lib.seed_dense_scan(d, *args, BIG, None) == -3
    optional = {7: "S0", 8: "dS_out", 14: "dS0"}
    for i in range(15):
        args = [A] * 16
        if i not in optional:
            args[i] = None
            assert lib.seed_dense_scan_backward(d, *args, BIG, None) == -1
        args[i] = MIS
        assert lib.seed_dense_scan_backward(d, *args, BIG, None) == -3
    assert lib.seed_dense_scan(d, *[A] * 9, None, BIG, None) == -5
    assert lib.seed_dense_scan(d, *[A] * 10, fwd - 1, None) == -5
    assert lib.seed_dense_scan_backward(d, *[A] * 16, bwd - 1, None) == -5


def test_tree_rejects(lib):
    d = _lib.seed_dims(form=0, batch=2, layers=3, heads=4, d_k=128, d_v=128, R=16, W=16)
    s = _lib.seed_state(a=A, U=A, V=A, scale=A, ncols=A, vbar=A)
    read = lambda layer=0, n=8, args=(), ws=A, b=256: lib.seed_decode_tree(  # noqa: E731
        ctypes.byref(d), ctypes.byref(s), layer, n, *(args or [A] * 8), ws, b, None)
    commit = lambda layer=0, n=8, args=(), ws=A, b=256: lib.seed_decode_tree_commit(  # noqa: E731
        ctypes.byref(d), ctypes.byref(s), layer, n, *(args or [A] * 7), ws, b, None)
    for call, count in ((read, 8), (commit, 7)):
        assert call(layer=3) == -1 and call(layer=-1) == -1
        assert call(n=0) == -1 and call(n=65) == -2
        assert call(ws=None) == -5 and call(b=8) == -5
        for i in range(count):
            assert call(args=[A] * i + [None] + [A] * (count - 1 - i)) == -1
            assert call(args=[A] * i + [MIS] + [A] * (count - 1 - i)) == -3
    bad = _lib.seed_dims(form=0, batch=2, layers=3, heads=4, d_k=48, d_v=128, R=16, W=16)
    assert lib.seed_decode_tree(ctypes.byref(bad), ctypes.byref(s), 0, 8, *[A] * 8, A, 256, None) == -2


def test_binding_checks_arrays():
    """Types, sizes and devices that the C ABI cannot see are refused before any call."""
    d = S.ScanDims(S.SEED_KDA, 1, 10, 2, 1, 64, 64, 10, S.SEED_FACTORS_BF16)

    class Ws:
        buf = torch.empty(16, dtype=torch.uint8)
        ptr, nbytes = 0, 16

    bf, f = torch.bfloat16, torch.float32
    good = dict(offsets=torch.zeros(2, dtype=torch.int32), q=torch.zeros(10, 1, 64, dtype=bf),
                k=torch.zeros(10, 1, 64, dtype=bf), v=torch.zeros(10, 2, 64, dtype=bf), alpha=torch.zeros(10, 2, 64),
                beta=torch.zeros(10, 2), o=torch.zeros(10, 2, 64, dtype=bf))
    for name, bad in (("offsets", torch.zeros(2, dtype=torch.int64)), ("q", torch.zeros(10, 1, 64)),
                      ("k", torch.zeros(10, 2, 64, dtype=bf)), ("alpha", torch.zeros(10, 2)),
                      ("beta", torch.zeros(10, 2, dtype=bf)), ("o", torch.zeros(9, 2, 64, dtype=bf))):
        with pytest.raises(ValueError, match=name):
            S.seed_dense_scan(d, *{**good, name: bad}.values(), Ws)
    with pytest.raises(ValueError, match="S_out"):
        S.seed_dense_scan(d, *good.values(), Ws, S_out=torch.zeros(1, 2, 64, 32))
    with pytest.raises(ValueError, match="dlog_alpha"):
        S.seed_dense_scan_backward(d, *list(good.values())[:6], good["o"], good["q"], good["k"], good["v"],
                                   torch.zeros(10, 2, dtype=f), good["beta"], Ws)
    with pytest.raises(ValueError, match="unsupported dims"):
        S.ScanWorkspace(S.ScanDims(0, 1, 10, 2, 1, 48, 64, 10), device="cpu")
    t = S.Dims(S.SEED_GDN, 2, 1, 2, 64, 64, 8, 8)
    st = S.State.allocate(t, torch.ones(1, 2, 64), device="cpu")
    k, v, g = torch.zeros(2, 3, 2, 64), torch.zeros(2, 3, 2, 64), torch.zeros(2, 3, 2)
    with pytest.raises(ValueError, match="parent"):
        S.seed_decode_tree(t, st, 0, torch.zeros(3, 3, dtype=torch.int32), k, k, v, g, g, v, v, Ws)
    with pytest.raises(ValueError, match="leaf"):
        S.seed_decode_tree_commit(t, st, 0, torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2), k, v, g, g, v, Ws)
