"""The experts' forward at the sizes where the kernel for few pairs hands over to
the tiles, by the pairs' number and by the bytes of the weights that pairs share:
every pair on one expert, spread, and out of order, against the fp64 oracle with
the tolerances of the other tests of these calls."""

import numpy as np
import pytest
import torch

import oracle as O
from gpu_common import built_library, need_gpu
from test_gpu_ffn import BF, _bf, _np, _steps

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    from backward_token_expert_gb300 import lrm as L

    need_gpu()
    built_library()
    c = L.lrm_create(0)
    yield c
    L.lrm_destroy(c)


@pytest.mark.parametrize("pairs,E,h,I", [
    (15, 1, 2048, 768), (16, 1, 2048, 768), (17, 1, 2048, 768), (32, 32, 264, 136), (33, 32, 264, 136),
    (6, 1, 5120, 1536), (7, 1, 5120, 1536), (16, 1, 5120, 1536), (7, 2, 5120, 1536), (8, 2, 5120, 1536), (1, 1, 5120, 1536)])
@pytest.mark.parametrize("spread", [True, False])
def test_both_sides_of_the_rule(ctx, pairs, E, h, I, spread):
    from backward_token_expert_gb300 import lrm as L

    rng = np.random.default_rng(pairs + h)
    N = pairs + 3
    ids = rng.permutation(N)[:pairs]
    who = np.sort(rng.integers(0, E, pairs)) if spread else np.full(pairs, E - 1)
    offsets = np.searchsorted(who, np.arange(E + 1))
    x, W1 = _bf(rng, N, h), _bf(rng, E, 2 * I, h, scale=h ** -0.5)
    W = _bf(rng, E, h, I, scale=I ** -0.5)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    ab, phi, rows = torch.full((N, 2 * I), 7.0, **bf), torch.full((N, I), 7.0, **bf), torch.full((N, h), 7.0, **bf)
    dids = torch.from_numpy(ids.astype(np.int32)).cuda()
    off = torch.from_numpy(offsets.astype(np.int32)).cuda()
    dims = L.dims_of(N, E, 1, h, I)
    L.lrm_ffn_up(ctx, x.cuda(), W1.cuda(), off, dids, dims, pairs, ab, phi)
    L.lrm_ffn_down(ctx, phi, W.cuda(), off, dids, dims, pairs, rows)
    torch.cuda.synchronize()
    assert L.lrm_get_device_status(ctx) == 0
    xn, W1n, Wn = _np(x), _np(W1), _np(W)
    ref, phi_ref = O.ffn_up(xn, W1n, offsets, ids, 1)
    S, _ = O.ffn_up(np.abs(xn), np.abs(W1n), offsets, ids, 1)
    tol = S * _steps(h)
    assert np.all(np.abs(_np(ab)[ids] - ref) <= BF * (np.abs(ref) + tol) + tol + 2.0 ** -133)
    a, b, ta, tb = ref[:, :I], ref[:, I:], tol[:, :I], tol[:, I:]
    tp = 1.1 * ta * (np.abs(b) + tb) + np.abs(a) * tb + np.abs(a * b) * (2 + np.abs(a)) * 2.0 ** -20
    got = _np(phi)
    assert np.all(np.abs(got[ids] - phi_ref) <= BF * (np.abs(phi_ref) + tp) + tp + 2.0 ** -133)
    ref = O.ffn_down(got, Wn, offsets, ids)
    tol = O.ffn_down(np.abs(got), np.abs(Wn), offsets, ids) * _steps(I)
    assert np.all(np.abs(_np(rows)[ids] - ref) <= BF * (np.abs(ref) + tol) + tol + 2.0 ** -133)
    others = np.setdiff1d(np.arange(N), ids)
    for t in (ab, phi, rows):
        assert bool((t[others] == 7.0).all())
