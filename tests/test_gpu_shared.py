"""GPU parity of the decode over shared rows (gqa_decode_shared, gqa_decode_shared_paged) against
float64.  Rows past every length, and unused pages, hold NaN."""
import pytest
import torch

import grouped_query_attention_decode_b200 as gqa
from span_ref import attend64, normal, tolerance

pytestmark = pytest.mark.gpu
NAN = float("nan")
HEADS = [(8, 2, 64), (64, 8, 128), (12, 4, 64), (6, 1, 128), (7, 7, 64), (40, 1, 128), (160, 1, 64), (144, 1, 128)]


def make(starts, prefix, own, B, Q, heads, dtype, seed=5, capacity=None):
    H_q, H_kv, d = heads
    g = torch.Generator().manual_seed(seed)
    P = len(prefix)
    Lp, Lo = max(1, max(prefix)) + 3, max(1, max(own)) + 5
    x = {"q": normal((B, H_q, d) if Q == 1 else (B, Q, H_q, d), g, dtype), "prefix": prefix, "own": own, "starts": starts}
    for n in ("k_prefix", "v_prefix"):
        x[n] = normal((P, Lp, H_kv, d), g, dtype)
        for i, n_ in enumerate(prefix):
            x[n][i, max(0, n_):] = NAN
    for n in ("k_cache", "v_cache"):
        x[n] = normal((B, Lo, H_kv, d), g, dtype)
        for i, n_ in enumerate(own):
            x[n][i, max(0, n_):] = NAN
    return x


def group(starts, b):
    return next((g for g in range(len(starts) - 1) if starts[g] <= b < starts[g + 1]), -1)


def expect(x, scale, dev="cuda"):
    q = x["q"].to(dev)
    B, H_q, d = q.shape[0], q.shape[-2], q.shape[-1]
    q = q.view(B, -1, H_q, d)
    Q = q.shape[1]
    out = torch.zeros(q.shape, dtype=torch.float64, device=dev)
    for b in range(B):
        g, n = group(x["starts"], b), x["own"][b]
        h = x["prefix"][g] if g >= 0 else 0
        k = torch.cat([x["k_prefix"][max(g, 0), :h], x["k_cache"][b, :n]]).to(dev)
        v = torch.cat([x["v_prefix"][max(g, 0), :h], x["v_cache"][b, :n]]).to(dev)
        for j in range(Q):
            out[b, j] = attend64(q[b, j], k[:h + n - Q + 1 + j], v[:h + n - Q + 1 + j], scale)
    return out.view(x["q"].shape)


def tol(x, scale):
    return tolerance(x["q"], [x["k_prefix"], x["k_cache"]], [x["v_prefix"], x["v_cache"]], scale, max(x["prefix"]) + max(x["own"]))


def run(x, scale, **kw):
    c = {n: x[n].cuda() for n in ("q", "k_prefix", "v_prefix", "k_cache", "v_cache")}
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = gqa.decode_shared(c["q"], c["k_prefix"], c["v_prefix"], i32(x["prefix"]), i32(x["starts"]), c["k_cache"], c["v_cache"],
                            i32(x["own"]), scale, status=status, **kw)
    torch.cuda.synchronize()
    return out, int(status.item())


def paged(x, page_size, seed=3):
    """The same rows as a pool of pages in random order: a group's shared rows once."""
    B, H_kv, d = x["q"].shape[0], *x["k_prefix"].shape[2:]
    dtype = x["q"].dtype
    rows = [(x["prefix"][max(0, group(x["starts"], b))] if group(x["starts"], b) >= 0 else 0) + x["own"][b] for b in range(B)]
    max_pages = max(1, max(-(-r // page_size) for r in rows)) + 1
    need = sum(p // page_size for p in x["prefix"]) + sum(-(-n // page_size) for n in x["own"]) + 4
    perm = torch.randperm(need, generator=torch.Generator().manual_seed(seed)).tolist()
    pools = {n: torch.full((need, page_size, H_kv, d), NAN, dtype=dtype) for n in ("k", "v")}
    table = torch.full((B, max_pages), -1, dtype=torch.int32)

    def put(name, i, n):
        pages = [perm.pop() for _ in range(-(-n // page_size))]
        for kv in ("k", "v"):
            for j, pg in enumerate(pages):
                m = min(page_size, n - j * page_size)
                pools[kv][pg, :m] = x[f"{kv}_{name}"][i, j * page_size:j * page_size + m]
        return torch.tensor(pages, dtype=torch.int32)

    shared = [put("prefix", g, n) for g, n in enumerate(x["prefix"])]
    for b in range(B):
        g = group(x["starts"], b)
        both = torch.cat([shared[g] if g >= 0 else torch.empty(0, dtype=torch.int32), put("cache", b, x["own"][b])])
        table[b, :len(both)] = both
    return pools["k"], pools["v"], table, torch.tensor(rows, dtype=torch.int32)


def run_paged(x, page_size, scale, **kw):
    kp, vp, table, lens = paged(x, page_size)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = gqa.decode_shared_paged(x["q"].cuda(), kp.cuda(), vp.cuda(), table.cuda(), lens.cuda(), i32(x["starts"]), i32(x["prefix"]),
                                  scale, status=status, **kw)
    torch.cuda.synchronize()
    return out, int(status.item())


def close(out, ref, bound):
    assert torch.isfinite(out).all()
    err = float((out.double() - ref).abs().max())
    assert err <= bound, (err, bound)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("heads", HEADS, ids=lambda h: "%d_%d_%d" % h)
def test_heads(heads, dtype):
    x = make([0, 3, 5], [300, 129], [40, 1, 130, 77, 128, 5], 6, 1, heads, dtype)
    scale = heads[2] ** -0.5
    out, status = run(x, scale)
    assert status == 0
    close(out, expect(x, scale), tol(x, scale))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", [
    # (group starts, prefix lengths, own lengths)
    ([0, 2], [0], [3, 0]),                        # no prefix rows; a sequence of none at all
    ([0, 2], [1], [0, 1]),
    ([0, 1, 1, 4], [127, 50, 128], [0, 0, 129, 1]),  # an empty group between two
    ([1, 3], [255], [0, 5, 64, 256]),             # sequences before and behind the groups
    ([0, 17], [513], [i * 7 for i in range(17)]),  # more than one row tile
    ([0, 40], [2048], [0] * 40),                  # shared rows alone, cut over many CTAs
    ([0, 1], [5000], [3]),
    ([2, 2], [64], [33, 34]),                     # nobody shares
], ids=str)
def test_lengths(case, dtype):
    starts, prefix, own = case
    x = make(starts, prefix, own, len(own), 1, (32, 4, 128), dtype)
    out, status = run(x, 0.09)
    assert status == 0
    close(out, expect(x, 0.09), tol(x, 0.09))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("Q", [2, 5, 32])
@pytest.mark.parametrize("heads", [(8, 2, 64), (40, 1, 128)], ids=lambda h: "%d_%d_%d" % h)
def test_drafted_tokens(Q, heads, dtype):
    x = make([0, 3, 4], [200, 128], [Q, Q + 1, 128 + Q, 64, 100], 5, Q, heads, dtype)
    out, status = run(x, 0.1)
    assert status == 0
    close(out, expect(x, 0.1), tol(x, 0.1))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("page_size", [8, 16, 64, 128, 256])
def test_paged(page_size, dtype):
    x = make([0, 3, 5], [2 * 256, 256], [40, 1, 300, 77, 0, 129], 6, 1, (64, 8, 128), dtype)
    out, status = run_paged(x, page_size, 0.09)
    assert status == 0
    close(out, expect(x, 0.09), tol(x, 0.09))
    x = make([1, 3], [768], [100, 5, 300, 32], 4, 3, (12, 4, 64), dtype)
    out, status = run_paged(x, page_size, 0.1)
    assert status == 0
    close(out, expect(x, 0.1), tol(x, 0.1))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.5])
def test_scales(scale, dtype):
    x = make([0, 3], [200], [40, 1, 130], 3, 1, (8, 2, 64), dtype)
    out, status = run(x, scale)
    assert status == 0
    close(out, expect(x, scale), tol(x, scale))


def test_growing_scores_are_rescaled():
    # scores that grow along the rows, so that every tile raises the running maximum
    x = make([0, 5], [1500], [300] * 5, 5, 1, (8, 2, 64), torch.bfloat16)
    x["q"][:] = 1.0
    x["k_prefix"][0, :1500] = (torch.arange(1500) / 100).to(torch.bfloat16)[:, None, None]
    x["k_cache"][:, :300] = (20 + torch.arange(300) / 50).to(torch.bfloat16)[:, None, None]
    out, status = run(x, 0.125)
    close(out, expect(x, 0.125), tol(x, 0.125))


def test_same_as_decode_paged():
    x = make([0, 4], [512], [40, 1, 300, 77], 4, 1, (64, 8, 128), torch.bfloat16)
    kp, vp, table, lens = (t.cuda() for t in paged(x, 16))
    whole = gqa.decode_paged(x["q"].cuda(), kp, vp, table, lens, 0.09)
    out, _ = run_paged(x, 16, 0.09)
    assert float((out - whole).abs().max()) <= 2 * tol(x, 0.09)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_lengths_out_of_range_are_reported(dtype):
    x = make([0, 2, 4], [64, 64], [9, 8, 7, 6, 5], 5, 1, (8, 2, 64), dtype)
    good, _ = run(x, 0.1)
    y = dict(x, own=[9, -1, 7, 1000, 5])
    out, status = run(y, 0.1)
    assert status == gqa.STATUS_SEQLEN_RANGE
    assert torch.equal(out[[0, 2, 4]], good[[0, 2, 4]]) and not out[[1, 3]].any()
    y = dict(x, prefix=[64, 70])
    out, status = run(y, 0.1)
    assert status == gqa.STATUS_SEQLEN_RANGE
    assert torch.equal(out[[0, 1, 4]], good[[0, 1, 4]]) and not out[2:4].any()
    out, status = run(dict(x, starts=[0, 3, 2]), 0.1)
    assert status == gqa.STATUS_GROUP_RANGE
    out, status = run(dict(x, starts=[0, 2, 6]), 0.1)
    assert status == gqa.STATUS_GROUP_RANGE and torch.equal(out[[0, 1]], good[[0, 1]])


def test_shared_rows_must_be_whole_pages():
    x = make([0, 2], [64], [9, 8], 2, 1, (8, 2, 64), torch.bfloat16)
    kp, vp, table, lens = (t.cuda() for t in paged(x, 16))
    for rows in (8, 80, -16):  # half a page; past a sequence's rows; negative
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = gqa.decode_shared_paged(x["q"].cuda(), kp, vp, table, lens, torch.tensor([0, 2], dtype=torch.int32, device="cuda"),
                                      torch.tensor([rows], dtype=torch.int32, device="cuda"), 0.1, status=status)
        assert int(status.item()) == gqa.STATUS_SEQLEN_RANGE and not out.any()


def test_empty_sequences_of_a_group():
    # sequences that have been freed stay in their group: zeros, and no complaint
    x = make([0, 4], [512], [40, 1, 300, 77], 4, 1, (64, 8, 128), torch.bfloat16)
    kp, vp, table, lens = (t.cuda() for t in paged(x, 16))
    args = (x["q"].cuda(), kp, vp, table, lens, torch.tensor([0, 4], dtype=torch.int32, device="cuda"),
            torch.tensor([512], dtype=torch.int32, device="cuda"), 0.1)
    whole = gqa.decode_shared_paged(*args)
    lens[2] = 0
    table[2] = -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = gqa.decode_shared_paged(*args, status=status)
    assert int(status) == 0 and not out[2].any()
    bound = tol(x, 0.1)  # the line of tiles is cut elsewhere
    assert float((out[[0, 1, 3]] - whole[[0, 1, 3]]).abs().max()) <= 2 * bound


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_bad_page_is_reported(dtype):
    x = make([0, 2], [64], [9, 8], 2, 1, (8, 2, 64), dtype)
    kp, vp, table, lens = (t.cuda() for t in paged(x, 16))
    table[1, 4] = 10_000
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = gqa.decode_shared_paged(x["q"].cuda(), kp, vp, table, lens, torch.tensor([0, 2], dtype=torch.int32, device="cuda"),
                                  torch.tensor([64], dtype=torch.int32, device="cuda"), 0.1, status=status)
    assert int(status.item()) & gqa.STATUS_PAGE_RANGE
    assert float((out[0].double() - expect(x, 0.1)[0]).abs().max()) <= tol(x, 0.1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_repeats_and_workspace_reuse(dtype):
    # the same bits again, with a workspace that another call with other sizes has used
    x = make([0, 17, 20], [1000, 77], [i * 9 for i in range(20)], 20, 1, (32, 4, 128), dtype)
    ws = torch.full((gqa.shared_workspace_size(20, 1, 2, 32, 4, 128, dtype) + 4096,), 255, dtype=torch.uint8, device="cuda")
    first, _ = run(x, 0.1, workspace=ws)
    run(make([0, 1], [40], [3, 2], 2, 1, (8, 2, 64), dtype), 0.1, workspace=ws)
    again, _ = run(x, 0.1, workspace=ws)
    assert torch.equal(first, again)
    close(first, expect(x, 0.1), tol(x, 0.1))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_captured_and_replayed(dtype):
    x = make([0, 3], [500], [40, 1, 130], 3, 1, (64, 8, 128), dtype)
    c = {n: x[n].cuda() for n in ("q", "k_prefix", "v_prefix", "k_cache", "v_cache")}
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    prefix, starts, own = i32(x["prefix"]), i32(x["starts"]), i32(x["own"])
    want, _ = run(x, 0.1)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = gqa.decode_shared(c["q"], c["k_prefix"], c["v_prefix"], prefix, starts, c["k_cache"], c["v_cache"], own, 0.1)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    own.copy_(i32([40, 0, 100]))  # lengths are read on the device
    graph.replay()
    torch.cuda.synchronize()
    y = dict(x, own=[40, 0, 100])
    close(out, expect(y, 0.1), tol(y, 0.1))


def test_on_another_stream():
    x = make([0, 3], [500], [40, 1, 130], 3, 1, (64, 8, 128), torch.bfloat16)
    want, _ = run(x, 0.1)
    side = torch.cuda.Stream()
    got, _ = run(x, 0.1, stream=side)
    assert torch.equal(got, want)


@pytest.mark.parametrize("Q", [1, 32])  # own rows in a launch of their own, and beside the shared ones
def test_wait_timeout_is_reported_and_the_context_recovers(Q):
    x = make([0, 17, 20], [1000, 77], [Q + i * 9 for i in range(20)], 20, Q, (32, 4, 128), torch.bfloat16)
    gqa.set_wait_timeout_ns(1)
    try:
        _, status = run(x, 0.1)
    finally:
        gqa.set_wait_timeout_ns(0)
    assert status & gqa.STATUS_WAIT_TIMEOUT
    out, status = run(x, 0.1)
    assert status == 0
    close(out, expect(x, 0.1), tol(x, 0.1))


@pytest.mark.parametrize("case", [
    # enough spans that a thread (and a warp) has several to look at; many empty ones among them
    (list(range(0, 700)), [(i * 37) % 150 * (i % 3 > 0) for i in range(699)], [(i * 13) % 40 * (i % 5 > 0) for i in range(700)]),
    ([0] + [3] * 399 + [4], [8] * 400, [i % 7 for i in range(4)]),
], ids=["many", "empty groups"])
def test_many_groups(case):
    starts, prefix, own = case
    x = make(starts, prefix, own, len(own), 1, (8, 2, 64), torch.bfloat16)
    out, status = run(x, 0.125)
    assert status == 0
    close(out, expect(x, 0.125), tol(x, 0.125))


def test_calls_on_two_streams_at_once():
    x = make([0, 17, 20], [3000, 77], [i * 9 for i in range(20)], 20, 1, (32, 4, 128), torch.bfloat16)
    y = make([0, 5], [1500], [300] * 5, 5, 1, (8, 2, 64), torch.bfloat16)
    want = [run(v, 0.1)[0] for v in (x, y)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    args = []
    for v in (x, y):
        c = {n: v[n].cuda() for n in ("q", "k_prefix", "v_prefix", "k_cache", "v_cache")}
        args.append((c["q"], c["k_prefix"], c["v_prefix"], i32(v["prefix"]), i32(v["starts"]), c["k_cache"], c["v_cache"], i32(v["own"])))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            got[i].append(gqa.decode_shared(*args[i], 0.1, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])


def test_refusals():
    x = make([0, 2], [64], [9, 8], 2, 1, (8, 2, 64), torch.bfloat16)
    c = {n: x[n].cuda() for n in ("q", "k_prefix", "v_prefix", "k_cache", "v_cache")}
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    args = [c["q"], c["k_prefix"], c["v_prefix"], i32([64]), i32([0, 2]), c["k_cache"], c["v_cache"], i32([9, 8])]

    def refused(kind, i, value, **kw):
        with pytest.raises(kind):
            gqa.decode_shared(*args[:i], value, *args[i + 1:], 0.1, **kw)

    refused(ValueError, 0, c["q"].cpu())
    refused(ValueError, 0, c["q"].half())
    refused(ValueError, 0, c["q"].float())                    # the caches are bf16
    refused(ValueError, 1, c["k_prefix"].transpose(1, 2))     # not dense
    refused(ValueError, 3, i32([64]).long())
    refused(ValueError, 4, i32([0, 1, 2]))
    refused(ValueError, 7, i32([9, 8, 7]))
    refused(ValueError, 7, args[7], out=torch.empty(2, 8, 64, dtype=torch.bfloat16, device="cuda"))
    refused(gqa.GQAError, 7, args[7], workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(gqa.GQAError):
        gqa.decode_shared(*args, float("nan"))
    with pytest.raises(gqa.GQAError):  # 33 query tokens
        gqa.decode_shared(c["q"].unsqueeze(1).repeat(1, 33, 1, 1).contiguous(), *args[1:], 0.1)
