"""Sequences that have ended but stay in the batch: members of a group of gqa_decode_shared_paged that
hold none of its rows any more, the first of them among the others."""
import pytest
import torch

import grouped_query_attention_decode_b200 as gqa
from span_ref import attend64, normal, tolerance
from test_gpu_shared import expect, make, paged, tol

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def decode(x, ended, change, page_size=16, scale=0.1):
    """The call after ``change(table, lens, b)`` for every ended sequence b: out and the status word."""
    kp, vp, table, lens = paged(x, page_size)
    for b in ended:
        change(table, lens, b)
    status = i32([0])
    out = gqa.decode_shared_paged(x["q"].cuda(), kp.cuda(), vp.cuda(), table.cuda(), lens.cuda(), i32(x["starts"]), i32(x["prefix"]),
                                  scale, status=status)
    return out, int(status)


def freed(table, lens, b):
    table[b], lens[b] = -1, 0


def one_row(table, lens, b):
    """As gqa_pages_free, gqa_pages_reserve and an append leave it: one row, in a page of its own."""
    page = int(table[b, (int(lens[b]) - 1) // 16])  # its last page is its own
    table[b], lens[b] = -1, 1
    table[b, 0] = page


def check(x, out, ended, scale=0.1):
    live = [b for b in range(len(x["own"])) if b not in ended]
    assert not out[list(ended)].any()
    err = float((out[live].double() - expect(x, scale)[live]).abs().max()) if live else 0.0
    assert err <= tol(x, scale), err  # NaN fails too


# (group starts, shared rows, own rows, heads): own and shared rows in one launch for few query rows; in
# two; in one for many
GROUPS = {
    "one launch": ([0, 4], [512], [40, 1, 300, 77], (16, 4, 64)),
    "two launches": ([0, 9, 11], [512, 64], [40, 1, 300, 77, 5, 16, 17, 9, 2, 33, 8], (64, 8, 128)),
    "many rows": ([1, 6], [384], [40, 1, 300, 77, 5, 16], (24, 1, 128)),
}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("ended", [[0], [0, 1], [1, 2, 3], [3]], ids=str)
@pytest.mark.parametrize("case", GROUPS, ids=str)
def test_ended_members_are_passed_over(case, ended, dtype):
    starts, prefix, own, heads = GROUPS[case]
    x = make(starts, prefix, own, len(own), 1, heads, dtype)
    out, status = decode(x, ended, freed)
    assert status == 0
    check(x, out, ended)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", GROUPS, ids=str)
def test_a_group_that_has_ended_reads_nothing(case, dtype):
    starts, prefix, own, heads = GROUPS[case]
    x = make(starts, prefix, own, len(own), 1, heads, dtype)
    ended = list(range(starts[0], starts[1]))
    out, status = decode(x, ended, freed)
    assert status == 0
    check(x, out, ended)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", GROUPS, ids=str)
def test_a_first_member_with_a_row_of_its_own(case, dtype):
    # shorter than what its group shares: reported, zeros, and no other output depends on its table
    starts, prefix, own, heads = GROUPS[case]
    x = make(starts, prefix, own, len(own), 1, heads, dtype)
    ended = [starts[0], starts[0] + 1]
    out, status = decode(x, ended, one_row)
    assert status == gqa.STATUS_SEQLEN_RANGE
    check(x, out, ended)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_drafts_of_the_members_that_are_left(dtype):
    # with several tokens a sequence an empty one is reported; a length that leaves less than Q own rows too
    x = make([0, 40], [64], [3 + b % 19 for b in range(40)], 40, 3, (12, 4, 64), dtype)
    ended = list(range(33))
    out, status = decode(x, ended, freed)
    assert status == gqa.STATUS_SEQLEN_RANGE
    check(x, out, ended)
    out, status = decode(x, [0], lambda table, lens, b: lens.__setitem__(b, 64 + 2))
    assert status == gqa.STATUS_SEQLEN_RANGE
    check(x, out, [0])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_beams_that_end(dtype):
    """Beams of two prompts that fork and end, the first of a prompt among them: fork, reserve, copy,
    append, free the ended ones, decode; each live beam against float64 over its own rows."""
    H_q, H_kv, d, ps, n_pages, max_pages, B, scale = 16, 2, 64, 8, 120, 12, 10, 0.2
    g = torch.Generator().manual_seed(4)
    k_pool = torch.full((n_pages, ps, H_kv, d), float("nan"), dtype=dtype, device="cuda")
    v_pool = k_pool.clone()
    state = [(torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda"), i32([0] * B)) for _ in range(2)]
    refs, status = i32([0] * n_pages), i32([0])
    rows = [([], []) for _ in range(B)]
    starts, shared = i32([0, 5, 10]), i32([32, 40])
    # beams 0 and 5 are the prompts at first; from step 45 on every second step forks and ends beams
    ended, forks = [], {45: [0] * 5 + [5] * 5, 47: [-1, 2, 1, 2, 1, 6, 6, -1, 9, 5], 49: [-1, -1, 3, 4, 4, -1, 5, -1, 8, 6],
                        51: [-1] * 5 + [6, -1, -1, 8, 9]}
    for t in range(55):
        if t in forks:
            (table, lens), (table2, lens2) = state
            gqa.pages_fork(i32(forks[t]), table, lens, table2, lens2, refs, status=status)
            state.reverse()
            ended = [b for b, p in enumerate(forks[t]) if p < 0]
            rows = [([], []) if p < 0 else (list(rows[p][0]), list(rows[p][1])) for p in forks[t]]
        table, lens = state[0]
        gqa.pages_copy(k_pool, v_pool, gqa.pages_reserve(table, lens, refs, 1, ps, status=status))
        kn, vn = normal((B, H_kv, d), g, dtype), normal((B, H_kv, d), g, dtype)
        gqa.kv_append_paged(kn.cuda(), vn.cuda(), k_pool, v_pool, table, lens, status=status)
        for b in range(B):
            rows[b][0].append(kn[b])
            rows[b][1].append(vn[b])
        if ended:
            gqa.pages_free(i32(ended), table, lens, refs, status=status)
        if t >= 45:
            q = normal((B, H_q, d), g, dtype)
            out = gqa.decode_shared_paged(q.cuda(), k_pool, v_pool, table, lens, starts, shared, scale, status=status)
            assert int(status) == 0
            for b in range(B):
                if b in ended:
                    assert not out[b].any() and not int(lens[b])
                    continue
                k, v = torch.stack(rows[b][0]).cuda(), torch.stack(rows[b][1]).cuda()
                assert int(lens[b]) == len(k)
                err = float((out[b].double() - attend64(q[b].cuda(), k, v, scale)).abs().max())
                assert err <= tolerance(q, [k], [v], scale, len(k)), (t, b, err)
    want = torch.bincount(state[0][0][state[0][0] >= 0].long(), minlength=n_pages)
    assert torch.equal(want.int(), refs)
