"""Gradient norm and clipping against the fp64 oracle.

A batch of at most 64 squares is summed in fp32 in four chains: at most 19
roundings of 2^-24 on the squares, half of that on the norm, and the norm's own
rounding: 1e-6 relative.  The clipped values are exactly the fp32 product of
the value and the reported coefficient, rounded once to the type."""

import math

import numpy as np
import pytest
import torch

import oracle as O
from gpu_common import built_library, need_gpu

pytestmark = pytest.mark.gpu

REL = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _setup():
    need_gpu()
    built_library()


def _ref(grads, max_norm):
    """The oracle's values for the limit the call takes (fp32), the norm in the
    type it is reported in (fp32: its subnormals are coarse)."""
    norm, coef, out = O.clip([g.double().cpu().numpy() for g in grads], float(np.float32(max_norm)))
    with np.errstate(over="ignore"):  # a norm above fp32's largest is reported as infinity
        return float(np.float32(norm)), coef, out


def _expect(g, coef):
    return (g.float() * coef).to(g.dtype)


def check(grads, max_norm, in_place=False, outs=None):
    from backward_token_expert_gb300.pipeline import GradClip

    norm, coef, _ = _ref(grads, max_norm)
    before = [g.clone() for g in grads]
    if not in_place and outs is None:
        outs = [torch.full_like(g, 7.0) for g in grads]
    c = GradClip(grads, None if in_place else outs)
    c.clip(max_norm)
    torch.cuda.synchronize()
    got = float(c.norm.item())
    assert got == norm or abs(got - norm) <= REL * norm, (got, norm)
    assert abs(float(c.coef.item()) - coef) <= 1.2 * REL * coef
    assert int(c.nonfinite.item()) == 0
    for b, o, g in zip(before, grads if in_place else outs, grads):
        assert torch.equal(o, _expect(b, c.coef))
        if not in_place:
            assert torch.equal(g, b)
    if not in_place:
        c.measure()
        assert float(c.norm.item()) == got and float(c.coef.item()) == 1.0
    return c


def _tensors(sizes, dtype, seed, scale=0.01):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * scale).to(dtype) for n in sizes]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sizes", [[1], [2, 3], [7, 8, 9, 1, 16, 17], [31, 4095, 4096, 4097], [8191, 8192, 8193, 1],
                                   [100003], [1 << 20, 5, 300001], [1] * 1500, list(range(1, 400))])
def test_sizes(sizes, dtype):
    grads = _tensors(sizes, dtype, len(sizes))
    full = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    check(grads, 0.5 * full)
    check(grads, 2.0 * full)


# one cluster takes up to 128 chunks: blocks that fill unevenly, the last chunk short, and one chunk more
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("count", [8, 9, 15, 17, 32, 33, 57, 63, 65, 121, 127, 128, 129])
@pytest.mark.parametrize("each", [1, 37, 128])
def test_chunks_of_a_cluster(count, each, dtype):
    grads = _tensors([each] * (count - 1) + [1], dtype, count)
    full = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    check(grads, 0.5 * full)
    check(grads, 0.5 * full, in_place=True)


@pytest.mark.parametrize("words", [32 * 1024 - 4, 32 * 1024, 32 * 1024 + 4, 128 * 1024 - 1, 128 * 1024, 128 * 1024 + 1])
def test_sizes_around_a_cluster(words):
    grads = _tensors([words], torch.float32, words)
    full = math.sqrt(float(grads[0].double().square().sum()))
    check(grads, 0.5 * full)
    check(grads, 2.0 * full)


def test_mixed_types_in_place():
    grads = _tensors([1000, 33], torch.float32, 1) + _tensors([70001, 3], torch.bfloat16, 2)
    check(grads, 0.1, in_place=True)
    kept = [g.clone() for g in grads]
    check(grads, 1e9, in_place=True)
    assert all(torch.equal(a, b) for a, b in zip(kept, grads))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("so,do", [(1, 1), (3, 0), (0, 5), (7, 2), (2, 10)])
def test_offsets_inside_buffers(dtype, so, do):
    src = _tensors([20000], dtype, 3)[0]
    dst = torch.zeros(20000, dtype=dtype, device="cuda")
    grads = [src[so:so + 9001], src[10000 + so:10000 + so + 5]]
    outs = [dst[do:do + 9001], dst[10000 + do:10000 + do + 5]]
    check(grads, 0.05, outs=outs)
    written = torch.zeros(20000, dtype=torch.bool, device="cuda")
    written[do:do + 9001] = True
    written[10000 + do:10000 + do + 5] = True
    assert not dst[~written].any()


def test_empty_and_zero_gradients():
    c = check(_tensors([0, 5, 0], torch.float32, 4), 0.001)
    assert c.outs[0].numel() == 0
    z = [torch.zeros(3000, device="cuda"), torch.zeros(10, dtype=torch.bfloat16, device="cuda")]
    c = check(z, 0.0)
    assert float(c.norm.item()) == 0.0 and float(c.coef.item()) == 1.0
    check(_tensors([0], torch.float32, 5), 1.0)
    check(_tensors([100], torch.float32, 5), 0.0)  # everything to zero


def test_dimension_orders():
    g = torch.Generator(device="cuda").manual_seed(6)
    a = torch.randn(6, 5, 7, generator=g, device="cuda")
    check([a.permute(2, 0, 1), torch.randn(8, 3, generator=g, device="cuda").t()], 0.7,
          outs=[torch.empty_like(a).permute(2, 0, 1), torch.empty(8, 3, device="cuda").t()])


@pytest.mark.parametrize("scale", [1e-44, 1e-38, 1e-30, 1e-20, 1e-15, 1e15, 1e19, 1e30, 3e37])
def test_magnitudes_whose_squares_leave_fp32(scale):
    x = torch.linspace(-1, 1, 30001, device="cuda") * scale
    full = float(_ref([x], 1.0)[0])
    check([x], 0.25 * full if full * 0.25 > 1e-45 else 1.0)
    y = (torch.linspace(-1, 1, 3001, device="cuda") * scale).to(torch.bfloat16)
    check([y, torch.ones(5, device="cuda") * scale], 1.0)


def test_mixed_magnitudes():
    x = torch.full((10000,), 1e-25, device="cuda")
    x[::97] = 1e22
    x[5] = 1.0
    check([x, torch.full((4000,), 1e-3, device="cuda")], 1.0)


def test_norm_beyond_fp32_still_scales():
    # every value is finite and the norm is above fp32's largest: reported as infinity, clipped all the same
    from backward_token_expert_gb300.pipeline import GradClip

    x = torch.full((1 << 16,), 3e38, device="cuda")
    out = torch.empty_like(x)
    c = GradClip([x], [out])
    c.clip(1.0)
    assert math.isinf(float(c.norm.item())) and int(c.nonfinite.item()) == 0
    # the coefficient is a subnormal of fp32: rounded to a multiple of 2^-149
    coef = 1.0 / (3e38 * 256)
    assert abs(float(c.coef.item()) - coef) <= 2.0 ** -149
    assert torch.equal(out, x * c.coef)


@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_nonfinite_gradients_are_reported_and_left_alone(value, dtype):
    from backward_token_expert_gb300.pipeline import GradClip

    for n, at in ((1, 0), (37, 36), (50000, 31234)):
        grads = _tensors([200, n], dtype, 7)
        grads[1][at] = value
        before = [g.clone() for g in grads]
        outs = [torch.zeros_like(g) for g in grads]
        c = GradClip(grads, outs)
        c.clip(0.001)
        assert int(c.nonfinite.item()) == 1 and float(c.coef.item()) == 1.0
        assert not math.isfinite(float(c.norm.item())) and math.isnan(float(c.norm.item())) == math.isnan(value)
        c.measure()
        assert int(c.nonfinite.item()) == 1
        d = GradClip(grads)
        d.clip(0.001)
        for a, b, o in zip(before, grads, outs):
            assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num())
            assert torch.equal(a.isnan(), o.isnan()) and torch.equal(a.nan_to_num(), o.nan_to_num())


def test_infinite_limit_copies():
    check(_tensors([5000, 3], torch.bfloat16, 8), float("inf"))


def test_same_bits_graph_and_streams():
    from backward_token_expert_gb300.pipeline import GradClip

    grads = _tensors([300000, 77, 1 << 18], torch.float32, 9)
    outs = [torch.empty_like(g) for g in grads]
    c = GradClip(grads, outs)
    c.clip(0.3)
    torch.cuda.synchronize()
    want = [o.clone() for o in outs] + [c._stats.clone()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    [o.zero_() for o in outs]
    torch.cuda.synchronize()
    c.clip(0.3, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs + [c._stats]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        c.clip(0.3)
    [g.mul_(2.0) for g in grads]
    graph.replay()
    torch.cuda.synchronize()
    assert abs(float(c.norm.item()) - 2.0 * float(want[-1][0])) <= 4e-7 * float(c.norm.item())
    for g, o in zip(grads, outs):
        assert torch.equal(o, g * c.coef)


def test_refusals():
    from backward_token_expert_gb300 import lrm as L
    from backward_token_expert_gb300.pipeline import GradClip

    a, b = _tensors([64, 64], torch.float32, 10)
    for grads, outs in [([], None), ([a.half()], None), ([a.cpu()], None), ([a], [b, a]), ([a], [b.bfloat16()]),
                        ([a], [b[:32]]), ([a[::2]], None), ([a.view(8, 8)], [b.view(8, 8).t()]), ([a, a], None),
                        ([a[:40], a[32:]], None), ([a, b], [b, a]), ([a], [torch.empty(65, device="cuda")[1:][:64].cpu()]),
                        ([a.expand(3, 64)], None)]:
        with pytest.raises(ValueError):
            GradClip(grads, outs)
    c = GradClip([a], [b])
    stats = torch.zeros(3, device="cuda")
    inv = L.LRM_ERR_INVALID_ARG
    for call, code in [(lambda: L.lrm_grad_clip(c.ctx, c.list, -1.0, stats), inv),
                       (lambda: L.lrm_grad_clip(c.ctx, c.list, float("nan"), stats), inv),
                       (lambda: L.lrm_grad_clip(c.ctx, c.list, 1.0, None), inv),
                       (lambda: L.lrm_grad_clip(c.ctx, None, 1.0, stats), inv),
                       (lambda: L.lrm_grad_norm(c.ctx, c.list, None), inv),
                       (lambda: L.lrm_grad_norm(c.ctx, c.list, stats.data_ptr() + 1), L.LRM_ERR_ALIGN)]:
        with pytest.raises(L.LrmError) as ei:
            call()
        assert ei.value.code == code
    arr = L.tensor_array([(a, None, 64, L.DTYPE_F32)])
    need = L.lrm_grad_table_size(arr, 1)
    table = torch.empty(need, dtype=torch.uint8, device="cuda")
    for t, n, code in [(None, need, L.LRM_ERR_WORKSPACE), (table, need - 1, L.LRM_ERR_WORKSPACE),
                       (table.data_ptr() + 16, need, L.LRM_ERR_ALIGN)]:
        with pytest.raises(L.LrmError) as ei:
            L.lrm_grad_list_create(c.ctx, arr, 1, t, n)
        assert ei.value.code == code
    only_norm = L.lrm_grad_list_create(c.ctx, arr, 1, table, need)
    L.lrm_grad_norm(c.ctx, only_norm, stats)
    assert abs(float(stats[0]) - float(a.double().norm())) <= REL * float(stats[0])
    with pytest.raises(L.LrmError) as ei:
        L.lrm_grad_clip(c.ctx, only_norm, 1.0, stats)
    assert ei.value.code == inv
    L.lrm_grad_list_destroy(only_norm)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        with pytest.raises(L.LrmError) as ei:  # a list is made before capturing
            L.lrm_grad_list_create(c.ctx, arr, 1, table, need, s)
        a.add_(0.0)
    assert ei.value.code == inv


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_lists_beyond_the_l2(dtype):
    # above 128 MB: whole runs, short ones, tensors off the 16-byte grid (src, dst, both), single elements
    n = 40_000_000 if dtype == torch.float32 else 80_000_000
    g = torch.Generator(device="cuda").manual_seed(20)
    src = (torch.randn(n, generator=g, device="cuda") * 0.01).to(dtype)
    dst = torch.full_like(src, 3.0)
    cuts = [(0, 1), (8, 8191), (8208, 8192), (16400 + 3, 50001), (70000, 7), (70016, 4096 * 5 + 1), (100003, 12_000_000),
            (12_200_000, n - 12_200_000 - 5)]
    grads = [src[a:a + m] for a, m in cuts]
    outs = [dst[a + (1 if i == 2 else 0):a + (1 if i == 2 else 0) + m] for i, (a, m) in enumerate(cuts)]
    from backward_token_expert_gb300.pipeline import GradClip

    norm = math.sqrt(sum(float(t.double().square().sum()) for t in grads))
    kept = src.clone()
    for limit in (0.3 * norm, 2.0 * norm):
        c = GradClip(grads, outs)
        c.clip(limit)
        assert abs(float(c.norm) - norm) <= REL * norm
        assert abs(float(c.coef) - min(1.0, limit / norm)) <= 1.2 * REL
        for a, b in zip(grads, outs):
            assert torch.equal(b, _expect(a, c.coef))
    assert torch.equal(src, kept)
    written = torch.zeros(n, dtype=torch.bool, device="cuda")
    for i, (a, m) in enumerate(cuts):
        written[a + (1 if i == 2 else 0):a + (1 if i == 2 else 0) + m] = True
    assert bool((dst[~written] == 3.0).all())
    c = GradClip(grads)
    c.clip(2.0 * norm)  # in place, nothing to do
    assert torch.equal(src, kept)
    c.clip(0.3 * norm)
    inside = torch.zeros(n, dtype=torch.bool, device="cuda")
    for a, m in cuts:
        inside[a:a + m] = True
    assert torch.equal(src, torch.where(inside, _expect(kept, c.coef), kept))


def test_more_elements_than_32_bits():
    from backward_token_expert_gb300.pipeline import GradClip

    n = (1 << 31) + 4099
    x = torch.full((n,), 0.25, dtype=torch.bfloat16, device="cuda")
    x[-1] = 64.0
    c = GradClip([x])
    norm = math.sqrt((n - 1) * 0.0625 + 4096.0)
    c.clip(norm / 2)
    assert abs(float(c.norm.item()) - norm) <= REL * norm
    assert x[0] == 0.125 and x[-2] == 0.125 and x[-1] == 32.0
    assert int((x == 0.125).sum()) == n - 1


def test_two_lists_at_once():
    # lists that each fill the GPU, clipped on two streams at the same time, beside other work on a third
    from backward_token_expert_gb300 import lrm as L
    from backward_token_expert_gb300.pipeline import GradClip

    ctx = L.lrm_create(0)
    try:
        grads = [_tensors([3_000_000 + 7 * i, 77], torch.float32, 30 + i) for i in range(2)]
        outs = [[torch.empty_like(t) for t in g] for g in grads]
        clips = [GradClip(g, o, ctx=ctx) for g, o in zip(grads, outs)]
        streams = [torch.cuda.Stream() for _ in range(3)]
        work = torch.randn(2048, 2048, device="cuda")
        torch.cuda.synchronize()
        for _ in range(60):
            for c, s in zip(clips, streams):
                c.clip(0.5, stream=s)
            with torch.cuda.stream(streams[2]):
                work = torch.tanh(work @ work)
        torch.cuda.synchronize()
        assert L.lrm_get_device_status(ctx) == 0
        for g, o, c in zip(grads, outs, clips):
            norm = math.sqrt(sum(float(t.double().square().sum()) for t in g))
            assert abs(float(c.norm) - norm) <= REL * norm
            for a, b in zip(g, o):
                assert torch.equal(b, _expect(a, c.coef))
        for c in clips:
            c.close()
    finally:
        L.lrm_destroy(ctx)


@pytest.mark.parametrize("n", [1 << 20, 50_000_000])
def test_a_wait_that_runs_out_is_reported_and_the_list_stays_usable(n):
    # no time at all for the waits on copies and on the other blocks
    from backward_token_expert_gb300 import lrm as L
    from backward_token_expert_gb300.pipeline import GradClip

    ctx = L.lrm_create(0)
    try:
        x = torch.full((n,), 0.5, device="cuda")
        out = torch.zeros_like(x)
        c = GradClip([x], [out], ctx=ctx)
        L.lrm_set_wait_budget(ctx, 0)
        for _ in range(3):
            c.clip(1.0)
        assert L.lrm_get_device_status(ctx) in (0, 1 << L.LRM_ERR_TIMEOUT)
        L.lrm_set_wait_budget(ctx, 2_000_000_000)
        for _ in range(3):
            out.zero_()
            c.clip(1.0)
            assert L.lrm_get_device_status(ctx) == 0
            assert abs(float(c.norm.item()) - 0.5 * math.sqrt(n)) <= REL * 0.5 * math.sqrt(n)
            assert torch.equal(out, x * c.coef)
        c.close()
    finally:
        L.lrm_destroy(ctx)


def test_large_tensor():
    n = (1 << 27) + 12345
    x = torch.full((n,), 0.5, device="cuda")
    from backward_token_expert_gb300.pipeline import GradClip

    c = GradClip([x])
    c.clip(1.0)
    assert abs(float(c.norm.item()) - 0.5 * math.sqrt(n)) <= REL * 0.5 * math.sqrt(n)
    assert torch.all(x == 0.5 * c.coef)


@pytest.mark.parametrize("in_place", [False, True])
def test_no_time_for_the_other_blocks_writes_nothing_and_says_so(in_place):
    # no time at all: no block can wait for the others, so the wait runs out in every call
    from backward_token_expert_gb300 import lrm as L
    from backward_token_expert_gb300.pipeline import GradClip

    ctx = L.lrm_create(0)
    try:
        x = torch.linspace(-1.0, 1.0, 1 << 20, device="cuda")
        kept, norm = x.clone(), math.sqrt(float(x.double().square().sum()))
        out = x if in_place else torch.full_like(x, 7.0)
        before = out.clone()
        c = GradClip([x], None if in_place else [out], ctx=ctx)
        for calls in (1, 2, 3):  # an odd and an even number of calls in a row that gave up
            c.clip(2.0 * norm)
            assert abs(float(c.norm) - norm) <= REL * norm and int(c.nonfinite) == 0
            out.copy_(before)
            L.lrm_set_wait_budget(ctx, 0)
            for i in range(calls):
                c.clip(0.25 * norm) if i != 1 else c.measure()
                assert L.lrm_get_device_status(ctx) == 1 << L.LRM_ERR_TIMEOUT
                assert math.isnan(float(c.norm)) and float(c.coef) == 1.0 and int(c.nonfinite) == 1
                assert torch.equal(out, before) and torch.equal(x, kept)
            L.lrm_set_wait_budget(ctx, 2_000_000_000)
        c.clip(0.25 * norm)
        assert L.lrm_get_device_status(ctx) == 0 and int(c.nonfinite) == 0
        assert abs(float(c.norm) - norm) <= REL * norm and torch.equal(out, kept * c.coef)
        c.close()
    finally:
        L.lrm_destroy(ctx)


def test_a_long_list_whose_copies_ran_out_of_time_says_so():
    # beyond 128 MB: the copies may come in time all the same, and then everything is written
    from backward_token_expert_gb300 import lrm as L
    from backward_token_expert_gb300.pipeline import GradClip

    ctx = L.lrm_create(0)
    try:
        x = torch.full((50_000_000,), 0.5, device="cuda")
        out, norm = torch.empty_like(x), 0.5 * math.sqrt(50_000_000)
        c = GradClip([x], [out], ctx=ctx)
        L.lrm_set_wait_budget(ctx, 0)
        for _ in range(5):
            out.zero_()
            c.clip(1.0)
            late = L.lrm_get_device_status(ctx)
            assert late in (0, 1 << L.LRM_ERR_TIMEOUT)
            assert int(c.nonfinite) == (1 if late else 0)
            if late:
                assert math.isnan(float(c.norm)) and bool(((out == 0) | (out == x * c.coef)).all())
            else:
                assert abs(float(c.norm) - norm) <= REL * norm and torch.equal(out, x * c.coef)
        c.close()
    finally:
        L.lrm_destroy(ctx)


def test_lists_without_a_context_report_their_own_timeouts():
    from backward_token_expert_gb300 import lrm as L
    from backward_token_expert_gb300.pipeline import GradClip

    x = torch.full((1 << 20,), 0.5, device="cuda")
    late, other, short, empty = (GradClip([t]) for t in (x, x.clone(), x[:100].clone(), x[:0]))
    assert [c.device_status() for c in (late, other, short, empty)] == [0] * 4
    L.lrm_set_wait_budget(late.ctx, 0)  # their common context's
    try:
        late.clip(1.0)
        late.clip(1.0)
    finally:
        L.lrm_set_wait_budget(late.ctx, 2_000_000_000)
    for c in (other, short, empty):
        c.clip(1.0)
        assert c.device_status() == 0
    assert late.device_status() == 1 << L.LRM_ERR_TIMEOUT
    assert late.device_status() == 0  # cleared by the read
    late.clip(1.0)
    assert late.device_status() == 0 and float(late.norm) == 512.0
    L.lrm_get_device_status(late.ctx)  # the common word


def test_status_refusals():
    from backward_token_expert_gb300 import lrm as L
    from backward_token_expert_gb300.pipeline import GradClip

    c = GradClip([torch.ones(3, device="cuda")])
    for ctx, lst in ((None, c.list), (c.ctx, None)):
        with pytest.raises(L.LrmError) as ei:
            L.lrm_grad_list_status(ctx, lst)
        assert ei.value.code == L.LRM_ERR_INVALID_ARG
    assert L.load_library().lrm_grad_list_status(c.ctx, c.list, None, None) == L.LRM_ERR_INVALID_ARG


def test_a_list_made_while_the_current_stream_is_busy():
    # what the constructor fills on the current stream is there before another stream clips
    from backward_token_expert_gb300.pipeline import GradClip

    for n in (300, 300000):
        x = torch.full((n,), 0.5, device="cuda")
        out, s = torch.zeros_like(x), torch.cuda.Stream()
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)
        c = GradClip([x], [out], stream=s)
        c.clip(1.0, stream=s)
        torch.cuda.synchronize()
        assert abs(float(c.norm) - 0.5 * math.sqrt(n)) <= REL * 0.5 * math.sqrt(n)
        assert int(c.nonfinite) == 0 and torch.equal(out, x * c.coef)


def test_memory_of_a_dropped_list_stays_until_its_stream_is_done():
    from backward_token_expert_gb300.pipeline import GradClip

    x = torch.full((300000,), 0.5, device="cuda")
    out, s = torch.zeros_like(x), torch.cuda.Stream()
    c = GradClip([x], [out])
    size, table, stats = c.table.numel(), c.table.data_ptr(), c._stats.data_ptr()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)
    c.clip(1.0, stream=s)
    del c
    others = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(64)]
    others += [torch.empty(3, device="cuda") for _ in range(64)]
    spans = [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in others]
    assert not s.query()  # still asleep, the clip behind it
    for at in (table, stats):
        assert not any(a <= at < b for a, b in spans)
    s.synchronize()
    assert abs(float(out[0]) * 0.5 * math.sqrt(300000) - 0.5) <= 2 * REL


def test_strides_of_dimensions_of_one_element():
    # a column or a row cut out of a larger buffer: its stride in the dimension of one element is the buffer's
    g = torch.linspace(-1.0, 1.0, 40, device="cuda")
    whole = torch.full((3, 40), 7.0, device="cuda")
    check([g.view(1, 40), g.clone().view(40, 1), g.clone().view(1, 8, 1, 5)], 0.5,
          outs=[whole[1:2], torch.empty(40, device="cuda").as_strided((40, 1), (1, 40)),
                torch.empty(40, device="cuda").as_strided((1, 8, 1, 5), (999, 5, 7, 1))])
    assert bool((whole[0] == 7.0).all()) and bool((whole[2] == 7.0).all())
    check([whole[1:2]], 0.1, outs=[torch.empty(1, 40, device="cuda")])
