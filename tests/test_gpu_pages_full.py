"""Page calls at the ends: a pool that runs out while sequences that share a partly filled page are
given pages of their own (what the first call has handed out is copied, pages are freed, the second
call serves the rest, and every sequence's rows are what it appended), and lists of nothing."""
import pytest
import torch

import grouped_query_attention_decode_b200 as gqa
from span_ref import normal

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("layers", [1, 2])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_rows_survive_a_full_pool(dtype, layers):
    B, ps, H_kv, d, n_pages, filled = 4, 8, 2, 64, 5, 5
    g = torch.Generator().manual_seed(2)
    pools = [[torch.full((n_pages, ps, H_kv, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2)] for _ in range(layers)]
    rows = [[[normal((filled, H_kv, d), g, dtype) for _ in range(2)] for _ in range(layers)] for _ in range(B)]
    table = torch.full((B, 2), -1, dtype=torch.int32, device="cuda")
    # sequences 0..2 hold page 0, sequence 3 two pages of its own; page 3 is free
    table[:3, 0] = 0
    table[3] = i32([1, 2])
    lens, refs = i32([filled] * 3 + [16]), i32([3, 1, 1, 0, 1])
    for layer in range(layers):
        for kv in range(2):
            for b in range(3):
                rows[b][layer][kv] = rows[0][layer][kv]
            pools[layer][kv][0, :filled] = rows[0][layer][kv].cuda()

    def reserve():
        status = i32([0])
        copies = gqa.pages_reserve(table, lens, refs, 1, ps, status=status)
        for k, v in pools:  # whatever the status
            gqa.pages_copy(k, v, copies)
        return copies.cpu().tolist(), int(status)

    # sequences 0 and 1 need a page (2 keeps page 0), one is free; sequence 3 has no room in its table
    copies, status = reserve()
    assert status == gqa.STATUS_POOL_FULL | gqa.STATUS_APPEND_OVERFLOW
    assert copies == [[0, 3], [-1, -1], [-1, -1], [-1, -1]]
    gqa.pages_free(i32([3]), table, lens, refs)
    copies, status = reserve()
    assert status == 0
    # sequence 1 gets page 1, 2 keeps page 0, 3 begins anew; sequence 0's pair is not given again
    assert copies == [[-1, -1], [0, 1], [-1, -1], [-1, -1]]
    assert table[:, 0].cpu().tolist() == [3, 1, 0, 2] and refs.cpu().tolist() == [1, 1, 1, 1, 1]
    new = [[normal((B, H_kv, d), g, dtype) for _ in range(2)] for _ in range(layers)]
    for layer, (k, v) in enumerate(pools):
        after = lens.clone()
        gqa.kv_append_paged(new[layer][0].cuda(), new[layer][1].cuda(), k, v, table, after)
        assert after.cpu().tolist() == [filled + 1] * 3 + [1]
        for b in range(3):
            for kv, pool in enumerate((k, v)):
                have = pool[table[b, 0].long(), :filled + 1].cpu()
                assert torch.equal(have, torch.cat([rows[b][layer][kv], new[layer][kv][b:b + 1]]))


def test_empty_lists():
    """A step in which nothing has ended and nothing moves."""
    table, lens, refs = i32([[0, -1], [1, -1]]), i32([5, 3]), i32([1, 1, 0, 0])
    pool = torch.ones((4, 8, 2, 64), dtype=torch.bfloat16, device="cuda")
    gqa.pages_free(i32([]), table, lens, refs)
    gqa.pages_copy(pool, pool.clone(), torch.empty((0, 2), dtype=torch.int32, device="cuda"))
    assert refs.tolist() == [1, 1, 0, 0] and lens.tolist() == [5, 3] and table.tolist() == [[0, -1], [1, -1]]
    with pytest.raises(ValueError):  # checked all the same
        gqa.pages_free(i32([]), table, lens, refs.long())
