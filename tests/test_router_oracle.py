"""The fp64 oracle of the router, the gate gradient and the clip against
something other than itself: central differences of the losses, the values the
balance loss takes at uniform load and at collapse, brute-force products, and
the host checks of the entry points that need no GPU."""

import ctypes

import numpy as np
import pytest

import oracle as O
from backward_token_expert_gb300 import build as B
from backward_token_expert_gb300 import lrm as L


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load_library()


def test_balance_loss_is_one_at_uniform_load_and_E_at_collapse():
    E = 8
    cyc = np.zeros((E, E))
    for t in range(E):
        cyc[t, t] = 1e-12  # each expert once, equal probabilities
    r = O.router_forward(cyc, 1, True, 1.0, 0.0)
    assert np.array_equal(r["counts"], np.ones(E)) and abs(r["aux"] - 1.0) < 1e-9
    hot = np.full((5, E), -800.0)
    hot[:, 3] = 0.0
    r = O.router_forward(hot, 1, True, 1.0, 0.0)
    assert r["counts"][3] == 5 and abs(r["aux"] - E) < 1e-9


def test_order_ties_nan_and_uncounted_rows():
    n = np.nan
    x = np.array([[1.0, 3.0, 3.0, -np.inf], [n, -np.inf, 2.0, n], [-np.inf] * 4, [0.0, -0.0, 0.0, -1.0]])
    r = O.router_forward(x, 3, True, 1.0, 1.0, valid=np.array([1, 0, 1, 1]))
    assert r["expert_idx"].tolist() == [[1, 2, 0], [2, 1, 0], [0, 1, 2], [0, 1, 2]]
    assert r["tokens"] == 2 and r["counts"].tolist() == [2, 2, 2, 0]
    assert np.all(r["alpha"][[1, 2]] == 0) and np.isfinite(r["loss"])


@pytest.mark.parametrize("renorm", [True, False])
def test_router_gradient_against_central_differences(renorm):
    rng = np.random.default_rng(5)
    T, E, k = 7, 9, 3
    l = rng.standard_normal((T, E)) * 1.5
    l[2, 4] = -40.0
    valid = np.ones(T)
    valid[5] = 0
    w = rng.standard_normal((T, k))  # the upstream gradient of the gates
    base = O.router_forward(l, k, renorm, 0.3, 0.2, valid)
    f0, ids0 = base["f"], base["expert_idx"]

    def total(x):
        # f held at its value, as the gradient's definition says
        r = O.router_forward(x, k, renorm, 0.0, 0.2, valid)
        assert np.array_equal(r["expert_idx"], ids0)
        return 0.3 * E * float((f0 * r["P"]).sum()) + r["loss"] + float((w * r["alpha"]).sum())

    g = O.router_backward(l, ids0, base["alpha"], f0, base["tokens"], base["alpha"] * w, renorm, 0.3, 0.2,
                          base["counted"])
    h = 1e-6
    for t in range(T):
        for e in range(E):
            up, dn = l.copy(), l.copy()
            up[t, e] += h
            dn[t, e] -= h
            # central difference: truncation ~h^2, rounding ~1e-16 * |total| / h
            assert abs((total(up) - total(dn)) / (2 * h) - g[t, e]) < 1e-8, (t, e)
    assert np.all(g[5] == 0)


def test_gate_gradient_against_central_differences():
    rng = np.random.default_rng(6)
    T, k, h, I, E = 4, 2, 6, 5, 3
    W = rng.standard_normal((E, h, I))
    phi = rng.standard_normal((T * k, I))
    g = rng.standard_normal((T, h))
    alpha = rng.random(T * k)
    ids = np.stack([rng.choice(E, k, replace=False) for _ in range(T)]).reshape(-1)

    def loss(a):
        y = np.zeros((T, h))
        for u in range(T * k):
            y[u // k] += a[u] * (W[ids[u]] @ phi[u])
        return float((y * g).sum())

    sel = np.array([1, 2, 5, 7])
    rows = np.stack([(alpha[u] * g[u // k]) @ W[ids[u]] for u in sel])
    got = O.gate_grad(rows, phi[sel], sel, T * k)
    for u in range(T * k):
        up, dn = alpha.copy(), alpha.copy()
        up[u] += 1e-5
        dn[u] -= 1e-5
        want = alpha[u] * (loss(up) - loss(dn)) / 2e-5 if u in sel else 0.0
        assert abs(got[u] - want) < 1e-8


def test_clip_oracle():
    norm, coef, out = O.clip([np.array([3.0]), np.array([[4.0]])], 1.0)
    assert norm == 5.0 and coef == 0.2 and abs(np.hypot(out[0][0], out[1][0]) - 1.0) < 1e-15
    assert O.clip([np.array([3e200]), np.array([4e200])], np.inf)[0] == pytest.approx(5e200)
    assert O.clip([np.zeros(3)], 0.0)[:2] == (0.0, 1.0)


def test_null_context_is_rejected_without_device_work(lib):
    d = L.dims_of(16, 4, 2, 64, 32)
    bad = L.LRM_ERR_INVALID_ARG
    assert lib.lrm_router_forward(None, 16, 0, None, d, 1, 0.0, 0.0, 16, 16, 16, 16, 16, 16, 16, 256, 9, None) == bad
    assert lib.lrm_router_backward(None, 16, 0, 16, 16, 16, None, 16, 16, d, 1, 0.0, 0.0, 16, 0, None) == bad
    assert lib.lrm_gate_grad(None, 16, 16, 16, 16, d, 4, 16, None) == bad
    assert lib.lrm_grad_norm(None, None, 16, None) == bad
    assert lib.lrm_grad_clip(None, None, 1.0, 16, None) == bad
    assert lib.lrm_grad_list_destroy(None) == L.LRM_OK
    out = ctypes.c_void_p()
    assert lib.lrm_grad_list_create(None, None, 0, 256, 1 << 20, None, ctypes.byref(out)) == bad
    assert out.value is None


def test_grad_table_size(lib):
    def size(entries):
        return L.lrm_grad_table_size(L.tensor_array(entries), len(entries))

    empty = size([])
    assert size([(0, 0, 0, L.DTYPE_F32)]) == empty
    one = size([(256, 256, 1, L.DTYPE_F32)]) - empty
    assert one > 0
    # off a 16-byte boundary: a short first run, whole vectors, a tail
    assert size([(260, 260, 3 + 8 + 1, L.DTYPE_F32)]) - empty == 3 * one
    assert size([(256, 256, 8, L.DTYPE_BF16), (1024, 0, 8, L.DTYPE_F32)]) - empty == 2 * one
    for entries, code in [([(256, 256, -1, 0)], L.LRM_ERR_INVALID_ARG), ([(256, 256, 1, 7)], L.LRM_ERR_INVALID_ARG),
                          ([(0, 256, 1, 0)], L.LRM_ERR_INVALID_ARG), ([(258, 256, 1, 0)], L.LRM_ERR_ALIGN),
                          ([(256, 257, 1, 1)], L.LRM_ERR_ALIGN), ([(256, 256, 1 << 50, 0)], L.LRM_ERR_SHAPE)]:
        with pytest.raises(L.LrmError) as ei:
            size(entries)
        assert ei.value.code == code
    assert lib.lrm_grad_table_size(None, 1, ctypes.byref(ctypes.c_size_t())) == L.LRM_ERR_INVALID_ARG
    assert lib.lrm_grad_table_size(None, 0, None) == L.LRM_ERR_INVALID_ARG
