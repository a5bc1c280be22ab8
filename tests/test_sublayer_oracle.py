"""The fp64 oracle of the experts' forward and backward, layer norm and dropout
against something other than itself: central differences, published vectors of
the generator, and the host checks of the entry points that need no GPU."""

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


@pytest.mark.parametrize("counter,key,want", [
    # the generator's published known answers
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_philox_known_answers(counter, key, want):
    assert tuple(int(w) for w in O.philox4x32_10([counter], key)[0]) == want


def test_dropout_mask_rate_and_words():
    n, p = 1 << 18, 0.3
    kept = O.dropout_kept(n, p, 12345, 7)
    assert abs(kept.mean() - (1 - p)) < 5 * np.sqrt(p * (1 - p) / n)
    assert np.array_equal(O.dropout_kept(1000, p, 12345, 7, first=777), kept[777:1777])
    assert O.dropout_kept(64, 0.0, 1, 1).all() and not O.dropout_kept(64, 1.0, 1, 1).any()
    assert (O.dropout_kept(n, p, 12345, 8) != kept).any()


def test_block_gradients_are_those_of_the_forward():
    rng = np.random.default_rng(0)
    T, E, k, h, I = 6, 3, 2, 5, 4
    x, W1, W = rng.normal(size=(T, h)), rng.normal(size=(E, 2 * I, h)), rng.normal(size=(E, h, I))
    experts = np.argsort(rng.normal(size=(T, E)), 1)[:, :k].reshape(-1)
    ids = np.argsort(experts, kind="stable")
    offsets = np.searchsorted(experts[ids], np.arange(E + 1))
    alpha, g = rng.random(T * k), rng.normal(size=(T, h))

    def loss(x, W1, alpha):
        ab, phi_r = O.ffn_up(x, W1, offsets, ids, k)
        phi = np.zeros((T * k, I))
        phi[ids] = phi_r
        rows = np.zeros((T * k, h))
        rows[ids] = O.ffn_down(phi, W, offsets, ids)
        return (O.ffn_combine(rows, alpha, k) * g).sum(), ab

    _, ab_r = loss(x, W1, alpha)
    ab = np.zeros((T * k, 2 * I))
    ab[ids] = ab_r
    delta = alpha[ids][:, None] * g[ids // k]
    dh1, dgate = O.ffn_backward(delta, W, ab, offsets, ids, T * k)
    dW1, dx = np.zeros_like(W1), np.zeros_like(x)
    for e in range(E):
        seg = slice(offsets[e], offsets[e + 1])
        dW1[e] = dh1[seg].T @ x[ids[seg] // k]
        np.add.at(dx, ids[seg] // k, dh1[seg] @ W1[e])
    eps = 1e-6
    for _ in range(20):
        for arr, grad in ((x, dx), (W1, dW1)):
            at = tuple(rng.integers(0, s) for s in arr.shape)
            keep = arr[at]
            arr[at] = keep + eps
            up = loss(x, W1, alpha)[0]
            arr[at] = keep - eps
            dn = loss(x, W1, alpha)[0]
            arr[at] = keep
            assert abs(grad[at] - (up - dn) / (2 * eps)) < 1e-6
        u = rng.integers(0, T * k)
        up, dn = alpha.copy(), alpha.copy()
        up[u] += eps
        dn[u] -= eps
        assert abs(dgate[u] - alpha[u] * (loss(x, W1, up)[0] - loss(x, W1, dn)[0]) / (2 * eps)) < 1e-6


def test_layer_norm_gradients_are_those_of_the_forward():
    rng = np.random.default_rng(1)
    rows, width, eps = 5, 7, 1e-3
    x, gamma, beta = rng.normal(size=(rows, width)), rng.normal(size=width), rng.normal(size=width)
    valid, g = np.array([1, 1, 0, 1, 1]), rng.normal(size=(rows, width))
    loss = lambda: (O.layer_norm(x, gamma, beta, eps, valid)[0] * g).sum()  # noqa: E731
    _, stats = O.layer_norm(x, gamma, beta, eps, valid)
    grads = O.layer_norm_backward(x, g, gamma, stats, valid)
    for arr, grad in zip((x, gamma, beta), grads):
        for at in np.ndindex(arr.shape):
            keep = arr[at]
            arr[at] = keep + 1e-6
            up = loss()
            arr[at] = keep - 1e-6
            dn = loss()
            arr[at] = keep
            assert abs(grad[at] - (up - dn) / 2e-6) < 1e-6
    dres = rng.normal(size=(rows, width))
    dx = O.layer_norm_backward(x, g, gamma, stats, valid, dres)[0]
    assert np.all(dx[2] == 0) and np.allclose(dx[valid != 0], (grads[0] + dres)[valid != 0])


def test_null_context_is_rejected_without_device_work(lib):
    d = L.dims_of(16, 4, 2, 64, 32)
    bad, n = L.LRM_ERR_INVALID_ARG, ctypes.c_size_t()
    assert lib.lrm_ffn_up(None, 16, 16, 16, 16, d, 4, 16, 16, None) == bad
    assert lib.lrm_ffn_down(None, 16, 16, 16, 16, d, 4, 16, None) == bad
    assert lib.lrm_ffn_combine(None, 16, 16, d, 16, None) == bad
    assert lib.lrm_ffn_backward(None, 16, 16, 16, 16, 16, d, 4, 16, 16, 16, 1 << 20, None) == bad
    assert lib.lrm_ffn_backward_workspace(None, d, 4, ctypes.byref(n)) == bad
    assert lib.lrm_layer_norm(None, 16, 0, 16, 16, None, 4, 8, 1e-5, 16, 16, None) == bad
    assert lib.lrm_layer_norm_workspace(None, 4, 8, ctypes.byref(n)) == bad
    assert lib.lrm_layer_norm_backward(None, 16, 0, 16, 16, 16, None, None, 4, 8, 16, 16, 16, 16, 1 << 20, None) == bad
    assert lib.lrm_dropout_add(None, 16, None, 0, 4, 0.5, 1, 1, None, 16, None) == bad
