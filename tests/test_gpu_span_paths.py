"""Every span kernel on the calls that it serves.  Which kernel a call goes to follows from its sizes, so
each test here says which ones it is for and looks at what was launched."""
import pytest
import torch

import grouped_query_attention_decode_b200 as gqa
import test_gpu_cross as cross
import test_gpu_shared as shared
from span_kernels import kernels_of
from span_ref import attend64

pytestmark = pytest.mark.gpu
NAMES = {torch.bfloat16: "bf16", torch.float32: "f32"}
TYPES = pytest.mark.parametrize("dtype", list(NAMES), ids=NAMES.values())


def launched(fn, *kernels):
    """fn(), which launches these span kernels and no others.  The profiler drops a record now and then, so
    what is missing is looked for again; what is too much counts at once."""
    seen, recorded = set(), False
    for _ in range(5):
        result, names = kernels_of(fn)
        if names is not None:
            recorded = True
            seen |= names
            assert seen <= set(kernels)
            if seen == set(kernels):
                return result
    assert not recorded, (seen, kernels)
    return result


def kernel(dtype, d, paged, few):
    if dtype == torch.float32:
        return f"span_f32<{d}, {16 if few else 64} rows>"
    return f"{'span_few' if few else 'span_tc'}<{d}, {'paged' if paged else 'dense'}>"


# (group starts, shared rows, own rows, heads, tokens): the shared rows under many query rows, the own rows
# under few; both under many (whatever the type); both under few
MANY_FEW = [([0, 9, 17], [512, 768], [40, 1, 300, 77, 0, 129, 16, 15, 17] + [i * 11 for i in range(8)] + [33], (64, 8, 128), 1),
            ([1, 34], [256], [1 + i * 7 % 50 for i in range(35)], (12, 4, 64), 1)]
MANY = [([0, 3, 5], [512, 256], [40, 5, 300, 77, 133, 129], (64, 8, 128), 5),
        ([0, 2, 5], [256, 768], [40, 1, 300, 77, 0, 129], (24, 1, 64), 1),
        ([1, 4], [512], [140, 12, 300, 19], (12, 4, 64), 12),
        ([0, 3], [256], [1, 128, 260], (40, 1, 128), 1)]
FEW = [([0, 2], [256], [40, 1, 130], (16, 4, 64), 1), ([0, 2], [256], [40, 1, 130], (16, 4, 128), 1)]


@TYPES
@pytest.mark.parametrize("page_size", [0, 8, 16, 64, 128, 256])  # 0: contiguous caches
@pytest.mark.parametrize("case", MANY_FEW + MANY + FEW, ids=lambda c: "%d_%d_%d" % c[3] + "_%d_%d" % (c[4], len(c[2])))
def test_rows(case, page_size, dtype):
    starts, prefix, own, heads, Q = case
    x = shared.make(starts, prefix, own, len(own), Q, heads, dtype)
    d, scale = heads[2], heads[2] ** -0.5
    run = (lambda: shared.run_paged(x, page_size, scale)) if page_size else (lambda: shared.run(x, scale))
    want = {kernel(dtype, d, page_size, case in FEW), kernel(dtype, d, page_size, case not in MANY)}
    out, status = launched(run, *want)
    assert status == 0
    shared.close(out, shared.expect(x, scale), shared.tol(x, scale))


@TYPES
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.5, -1e-30])
@pytest.mark.parametrize("case", [MANY_FEW[0], MANY[0], MANY[1], FEW[0]], ids=["many and few", "many", "many, d 64", "few"])
def test_scales(case, scale, dtype):
    starts, prefix, own, heads, Q = case
    x = shared.make(starts, prefix, own, len(own), Q, heads, dtype)
    out, status = launched(lambda: shared.run_paged(x, 16, scale), kernel(dtype, heads[2], True, case in FEW), kernel(dtype, heads[2], True, case not in MANY))
    assert status == 0
    shared.close(out, shared.expect(x, scale), shared.tol(x, scale))


@TYPES
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.5, -1e-30])
@pytest.mark.parametrize("heads", [(16, 4, 64), (16, 4, 128)], ids=["64", "128"])
@pytest.mark.parametrize("tokens", [[1, 3], [40, 130]], ids=["few", "many"])
def test_scales_of_cross_attention(tokens, heads, scale, dtype):
    x = cross.make(tokens, [300, 129], heads, dtype)
    out, status = launched(lambda: cross.run(x, scale), kernel(dtype, heads[2], False, tokens == [1, 3]))
    assert status == 0
    cross.check(x, out, scale)


@pytest.mark.parametrize("case", [([0, 9], [1504], [300] * 9, (64, 8, 128), 1), ([0, 2], [1504], [300] * 2, (24, 1, 64), 1)], ids=["128", "64"])
def test_growing_scores_are_rescaled(case):
    # scores that grow along the rows, so that every tile raises the running maximum
    starts, prefix, own, heads, Q = case
    x = shared.make(starts, prefix, own, len(own), Q, heads, torch.bfloat16)
    x["q"][:] = 1.0
    x["k_prefix"][0, :1504] = (torch.arange(1504) / 100).to(torch.bfloat16)[:, None, None]
    x["k_cache"][:, :300] = (20 + torch.arange(300) / 50).to(torch.bfloat16)[:, None, None]
    scale = 8 / heads[2]
    few = {kernel(torch.bfloat16, heads[2], True, True)} if heads[2] == 128 else set()
    out, status = launched(lambda: shared.run_paged(x, 16, scale), kernel(torch.bfloat16, heads[2], True, False), *few)
    assert status == 0
    shared.close(out, shared.expect(x, scale), shared.tol(x, scale))


@pytest.mark.parametrize("heads", [(64, 8, 128), (24, 1, 64)], ids=["two launches", "one"])
def test_same_as_decode_paged(heads):
    x = shared.make([0, 9], [512], [40, 1, 300, 77, 5, 16, 17, 130, 9], 9, 1, heads, torch.bfloat16)
    kp, vp, table, lens = (t.cuda() for t in shared.paged(x, 16))
    whole = gqa.decode_paged(x["q"].cuda(), kp, vp, table, lens, 0.09)
    out, _ = shared.run_paged(x, 16, 0.09)
    assert float((out - whole).abs().max()) <= 2 * shared.tol(x, 0.09)


@TYPES
@pytest.mark.parametrize("case", [MANY_FEW[0], MANY[0]], ids=["two launches", "one"])
def test_captured_and_replayed(case, dtype):
    """A paged call in a graph, replayed, also with other lengths, and eagerly on another stream."""
    starts, prefix, own, heads, Q = case
    x = shared.make(starts, prefix, own, len(own), Q, heads, dtype)
    want, _ = shared.run_paged(x, 16, 0.1)
    kp, vp, table, lens = (t.cuda() for t in shared.paged(x, 16))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    args = (x["q"].cuda(), kp, vp, table, lens, i32(starts), i32(prefix), 0.1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gqa.decode_shared_paged(*args)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    got = gqa.decode_shared_paged(*args, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    shorter = [max(Q, n // 2) if n else 0 for n in own]  # lengths are read on the device
    group = [shared.group(starts, b) for b in range(len(own))]
    lens.copy_(i32([n + (prefix[g] if g >= 0 else 0) for n, g in zip(shorter, group)]))
    graph.replay()
    torch.cuda.synchronize()
    y = dict(x, own=shorter)
    shared.close(out, shared.expect(y, 0.1), shared.tol(y, 0.1))


@TYPES
@pytest.mark.parametrize("few", [True, False], ids=["few", "many"])
def test_a_bad_page_of_the_shared_rows(few, dtype):
    """Reported, read as page 0, and nothing of it reaches a sequence outside the group."""
    starts, prefix, own, heads, Q = FEW[1] if few else MANY_FEW[0]
    x = shared.make(starts, prefix, own, len(own), Q, heads, dtype)
    kp, vp, table, lens = (t.cuda() for t in shared.paged(x, 16))
    table[:starts[1], 3] = 10 ** 6
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    status = i32([0])
    out = gqa.decode_shared_paged(x["q"].cuda(), kp, vp, table, lens, i32(starts), i32(prefix), 0.1, status=status)
    assert int(status) == gqa.STATUS_PAGE_RANGE
    ref = shared.expect(x, 0.1)
    for b in range(starts[1], len(own)):
        assert float((out[b].double() - ref[b]).abs().max()) <= shared.tol(x, 0.1)
