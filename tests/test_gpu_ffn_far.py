"""The experts' second product and the gated sum past 2^31 elements of a tensor:
the last pairs of a batch against the fp64 oracle, per value, with the tolerances of
the other tests of these calls."""

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


@pytest.mark.parametrize("pairs", [24, 200])  # of the kernel for few pairs, and of the tiles
def test_down_and_combine_beyond_32_bits(ctx, pairs):
    from backward_token_expert_gb300 import lrm as L

    k, E, h, I = 2, 32, 2048, 1024
    T = (1 << 31) // (I * k) + 100  # phi and rows pass 2^31 elements
    N = T * k
    rng = np.random.default_rng(pairs)
    phi = torch.zeros(N, I, dtype=torch.bfloat16, device="cuda")
    phi[-pairs:] = _bf(rng, pairs, I).cuda()
    rows = torch.zeros(N, h, dtype=torch.bfloat16, device="cuda")
    W = _bf(rng, E, h, I, scale=I ** -0.5).cuda()
    ids = torch.arange(N - pairs, N, dtype=torch.int32, device="cuda")
    cuts = np.sort(rng.integers(0, pairs + 1, E - 1))
    offsets = np.concatenate([[0], cuts, [pairs]])
    alpha = torch.zeros(N, device="cuda")
    alpha[-pairs:] = torch.rand(pairs, device="cuda")
    out = torch.full((T, h), 7.0, dtype=torch.bfloat16, device="cuda")
    dims = L.dims_of(T, E, k, h, I)
    L.lrm_ffn_down(ctx, phi, W, torch.from_numpy(offsets.astype(np.int32)).cuda(), ids, dims, pairs, rows)
    L.lrm_ffn_combine(ctx, rows, alpha, dims, out)
    torch.cuda.synchronize()
    assert L.lrm_get_device_status(ctx) == 0
    local = np.arange(pairs)
    p, w, got = _np(phi[-pairs:]), _np(W), _np(rows[-pairs:])
    ref = O.ffn_down(p, w, offsets, local)
    tol = O.ffn_down(np.abs(p), np.abs(w), offsets, local) * _steps(I)
    assert np.all(np.abs(got - ref) <= BF * (np.abs(ref) + tol) + tol + 2.0 ** -133)
    assert not rows[:-pairs].any()
    a = alpha[-pairs:].double().cpu().numpy()
    ref = O.ffn_combine(got, a, k)
    tol = O.ffn_combine(np.abs(got), a, k) * (k + 1) * 2.0 ** -24
    assert np.all(np.abs(_np(out[-pairs // k:]) - ref) <= BF * (np.abs(ref) + tol) + tol + 2.0 ** -133)
    assert not out[: -pairs // k].any()
