"""GPU parity of cross attention (gqa_cross_attend) against float64.  States past every length hold
NaN."""
import pytest
import torch

import grouped_query_attention_decode_b200 as gqa
from span_ref import attend64, normal, tolerance

pytestmark = pytest.mark.gpu


def make(tokens, states, heads, dtype, before=0, behind=0, seed=7, S_max=None):
    H_q, H_kv, d = heads
    g = torch.Generator().manual_seed(seed)
    starts = [before + sum(tokens[:i]) for i in range(len(tokens) + 1)]
    S = S_max or max(1, max(states)) + 3
    x = {"q": normal((starts[-1] + behind, H_q, d), g, dtype), "starts": starts, "states": states}
    for n in ("k", "v"):
        x[n] = normal((len(tokens), S, H_kv, d), g, dtype)
        for e, m in enumerate(states):
            x[n][e, max(0, m):] = float("nan")
    return x


def run(x, scale, out=None, **kw):
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = gqa.cross_attend(x["q"].cuda(), x["k"].cuda(), x["v"].cuda(), i32(x["states"]), i32(x["starts"]), scale, out=out,
                           status=status, **kw)
    torch.cuda.synchronize()
    return out, int(status.item())


def check(x, out, scale):
    bound = tolerance(x["q"], [x["k"]], [x["v"]], scale, max(x["states"]))
    for e, n in enumerate(x["states"]):
        k, v = x["k"][e, :n].cuda(), x["v"][e, :n].cuda()
        for i in range(x["starts"][e], x["starts"][e + 1]):
            ref = attend64(x["q"][i].cuda(), k, v, scale)
            err = float((out[i].double() - ref).abs().max())
            assert err <= bound, (e, i, err, bound)  # NaN fails too


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("heads", [(8, 2, 64), (64, 8, 128), (7, 7, 64), (24, 2, 128), (160, 1, 64), (5, 1, 128)], ids=lambda h: "%d_%d_%d" % h)
def test_heads(heads, dtype):
    x = make([1, 4, 70], [200, 129, 333], heads, dtype)
    scale = heads[2] ** -0.5
    out, status = run(x, scale)
    assert status == 0
    check(x, out, scale)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", [
    ([1], [1]),
    ([1, 1, 1], [0, 127, 128]),
    ([0, 5, 0], [64, 65, 66]),      # encoder sequences that no token attends
    ([33, 64, 65], [0, 256, 255]),  # tokens whose encoder sequence has no states
    ([200], [3000]),                # cut over many CTAs
    ([3] * 40, list(range(1, 401, 10))),
], ids=["one", "none", "idle", "empty", "cut", "many"])
def test_lengths(case, dtype):
    x = make(*case, (16, 4, 64), dtype)
    out, status = run(x, 0.125)
    assert status == 0
    check(x, out, 0.125)


def test_tokens_outside_are_left():
    x = make([2, 3], [100, 0], (8, 2, 64), torch.bfloat16, before=2, behind=3)
    out, status = run(x, 0.1, out=torch.full((10, 8, 64), 7.0, device="cuda"))
    assert status == 0
    check(x, out, 0.1)
    assert (out[:2] == 7).all() and (out[7:] == 7).all() and not out[4:7].any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_out_of_range_is_reported(dtype):
    x = make([2, 3, 2], [100, 90, 80], (8, 2, 64), dtype)
    good, _ = run(x, 0.1)
    for bad in (-1, 1000):
        out, status = run(dict(x, states=[100, bad, 80]), 0.1)
        assert status == gqa.STATUS_SEQLEN_RANGE
        assert torch.equal(out[:2], good[:2]) and torch.equal(out[5:], good[5:]) and not out[2:5].any()
    out, status = run(dict(x, starts=[0, 2, 5, 8]), 0.1, out=torch.full((7, 8, 64), 7.0, device="cuda"))
    assert status == gqa.STATUS_GROUP_RANGE
    assert torch.equal(out[:5], good[:5]) and (out[5:] == 7).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_captured_and_replayed(dtype):
    x = make([5, 70], [400, 333], (64, 8, 128), dtype)
    want, _ = run(x, 0.1)
    q, k, v = x["q"].cuda(), x["k"].cuda(), x["v"].cuda()
    states = torch.tensor(x["states"], dtype=torch.int32, device="cuda")
    starts = torch.tensor(x["starts"], dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gqa.cross_attend(q, k, v, states, starts, 0.1)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_far_rows():
    """States whose offsets pass 32 bits."""
    E, S, H_kv, d = 33, 65536, 8, 128  # 33 * 65536 * 1024 elements: over 2^31
    k = torch.zeros((E, S, H_kv, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    g = torch.Generator(device="cuda").manual_seed(1)
    k[-1, -200:].normal_(generator=g)
    v[-1, -200:].normal_(generator=g)
    q = torch.empty((3, 8, d), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    states = torch.zeros(E, dtype=torch.int32, device="cuda")
    states[-1] = S
    starts = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    starts[-1] = 3
    out = gqa.cross_attend(q, k, v, states, starts, 0.3)
    bound = tolerance(q, [k[-1, -200:]], [v[-1, -200:]], 0.3, S)
    for i in range(3):
        assert float((out[i].double() - attend64(q[i], k[-1], v[-1], 0.3)).abs().max()) <= bound


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("heads", [(8, 8, 64), (8, 2, 64), (64, 2, 128), (12, 4, 128), (24, 1, 64)], ids=lambda h: "%d_%d_%d" % h)
@pytest.mark.parametrize("tokens", [[1, 1, 1], [2, 0, 1, 3], [1, 0, 0, 0, 0, 0, 0, 40], [4] * 9], ids=str)
def test_few_tokens(tokens, heads, dtype):
    """One token, a beam or two per encoder sequence, and one sequence with many more than the mean."""
    states = [(i * 211) % 700 for i in range(len(tokens))]  # the first has none
    x = make(tokens, states, heads, dtype, before=1, behind=2)
    out, status = run(x, 0.1, out=torch.full(x["q"].shape, 7.0, device="cuda"))
    assert status == 0
    check(x, out, 0.1)
    assert (out[0] == 7).all() and (out[-2:] == 7).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_few_tokens_out_of_range(dtype):
    x = make([1, 1, 1], [100, 90, 80], (8, 8, 64), dtype)
    good, _ = run(x, 0.1)
    out, status = run(dict(x, states=[100, -1, 80]), 0.1)
    assert status == gqa.STATUS_SEQLEN_RANGE and torch.equal(out[::2], good[::2]) and not out[1].any()
    out, status = run(dict(x, starts=[0, 1, 0, 3]), 0.1)
    # sequence 2 is now [0, 3), so token 0 is no longer sequence 0's alone
    assert status == gqa.STATUS_GROUP_RANGE


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("tokens", [[1], [3, 0, 1], [40]], ids=str)
@pytest.mark.parametrize("heads", [(8, 1, 128), (12, 4, 64)], ids=lambda h: "%d_%d_%d" % h)
def test_many_pieces(heads, tokens, dtype):
    """Spans cut into far more pieces than there are query rows, one of them among empty ones."""
    x = make(tokens, [20001, 5, 0][:len(tokens)], heads, dtype, behind=1)
    ws = torch.full((gqa.cross_workspace_size(len(tokens), x["q"].shape[0], *heads, dtype),), 255, dtype=torch.uint8, device="cuda")
    out, status = run(x, 0.1, workspace=ws)
    assert status == 0
    check(x, out, 0.1)
    again, _ = run(x, 0.1, workspace=ws)
    n = x["starts"][-1]
    assert torch.equal(out[:n], again[:n])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_few_tokens_repeat(dtype):
    # the workspace's counters are set anew by each call
    x = make([1] * 5, [700, 3, 2000, 129, 0], (16, 4, 128), dtype)
    ws = torch.full((gqa.cross_workspace_size(5, 5, 16, 4, 128, dtype),), 255, dtype=torch.uint8, device="cuda")
    first, _ = run(x, 0.1, workspace=ws)
    again, _ = run(x, 0.1, workspace=ws)
    assert torch.equal(first, again)
    check(x, first, 0.1)


@pytest.mark.parametrize("tokens", [[1, 2, 1], [5, 70, 300]], ids=["few", "many"])
def test_wait_timeout_is_reported_and_the_context_recovers(tokens):
    x = make(tokens, [700, 333, 2000], (16, 4, 128), torch.bfloat16)
    gqa.set_wait_timeout_ns(1)
    try:
        _, status = run(x, 0.1)
    finally:
        gqa.set_wait_timeout_ns(0)
    # a warp of the kernel for few tokens waits for copies alone, which may be in before it looks twice
    assert status & gqa.STATUS_WAIT_TIMEOUT or (status == 0 and sum(tokens) < 10)
    out, status = run(x, 0.1)
    assert status == 0
    check(x, out, 0.1)


@pytest.mark.parametrize("tokens", [[2, 3], [40, 90]], ids=["few", "many"])
def test_out_at_sixteen_bytes(tokens):
    """out need not be aligned to more than 16 bytes, and nothing around it is written."""
    x = make(tokens, [200, 130], (8, 2, 64), torch.bfloat16)
    want, _ = run(x, 0.1)
    n = want.numel()
    room = torch.full((n + 8,), 7.0, device="cuda")
    out = room[4:4 + n].view(want.shape)
    assert out.data_ptr() % 32 == 16
    got, status = run(x, 0.1, out=out)
    assert status == 0 and torch.equal(got, want)
    assert (room[:4] == 7).all() and (room[4 + n:] == 7).all()


def test_values_that_differ_by_much():
    # one state outweighs all others, far into the span; huge and tiny scores beside each other
    x = make([3, 140], [3000, 500], (8, 2, 64), torch.bfloat16)
    x["q"] *= 20
    x["k"][0, 2500] *= 8
    out, status = run(x, 1.0)
    assert status == 0
    check(x, out, 1.0)


def test_one_state_is_returned():
    # The weight is 2^(x - m) with x - m what rounding m left, not exactly 1; it enters the product as
    # two bf16 parts, 2^-8 * 2^-8 off at most, is divided by itself (2^-23) and multiplied (2^-24).
    for tokens in ([1, 1], [30, 40]):
        x = make(tokens, [1, 1], (8, 2, 64), torch.bfloat16)
        out, _ = run(x, 0.7)
        for e in range(2):
            v = x["v"][e, 0].float().repeat_interleave(4, 0).cuda()
            assert ((out[x["starts"][e]:x["starts"][e + 1]] - v).abs() <= v.abs() * (2.0 ** -16 + 2.0 ** -22)).all()


def test_refusals():
    x = make([2, 3], [100, 90], (8, 2, 64), torch.bfloat16)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    args = [x["q"].cuda(), x["k"].cuda(), x["v"].cuda(), i32(x["states"]), i32(x["starts"])]
    for i, bad in [(0, x["q"].cuda().half()), (1, args[1].float()), (2, args[2][:, :50]), (3, i32([1])), (4, i32([0, 2])),
                   (3, torch.tensor(x["states"], dtype=torch.int32))]:
        with pytest.raises(ValueError):
            gqa.cross_attend(*args[:i], bad, *args[i + 1:], 0.1)
    with pytest.raises(gqa.GQAError):
        gqa.cross_attend(*args, float("inf"))
    with pytest.raises(gqa.GQAError):
        gqa.cross_attend(args[0][:, :7].contiguous(), *args[1:], 0.1)  # 7 heads over 2
