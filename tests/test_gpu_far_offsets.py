"""Offsets past 32 bits that a product of 32-bit numbers would lose: 2^32 16-byte vectors into a pool that is
copied, and 2^32 float32 elements into what the float32 kernels read.  Past 2^32, not 2^31, so that the place
such a product leads to is another one of the same tensor."""
import pytest
import torch

import grouped_query_attention_decode_b200 as gqa
from span_ref import attend64, tolerance

pytestmark = pytest.mark.gpu
H_KV, D = 8, 128


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.fixture(autouse=True)
def memory():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def test_copy_past_64_gib():
    ps, far = 64, 524_288  # pages of 128 KiB, 2^13 vectors: page 524288 starts at vector 2^32
    if torch.cuda.mem_get_info()[0] < 72 << 30:
        pytest.skip("needs 69 GB")
    pool = torch.empty((far + 8, ps, H_KV, D), dtype=torch.bfloat16, device="cuda")
    assert far * ps * H_KV * D // 8 == 2 ** 32
    g = torch.Generator(device="cuda").manual_seed(1)
    pool[far:].normal_(generator=g)
    pool[:8].normal_(generator=g)
    before = {p: pool[p].clone() for p in [*range(8), *range(far, far + 8)]}
    pairs = [[far + 7, 2], [1, far + 6], [far + 5, far + 4]]
    status = i32([0])
    gqa.pages_copy(pool, pool, i32(pairs), status=status)  # K and V alike: both write the same
    assert int(status) == 0
    for a, b in pairs:
        before[b] = before[a]
    for p, want in before.items():
        assert torch.equal(pool[p], want), p


def test_float32_states():
    E, S = 65, 65536  # 64 * 65536 * 1024 elements before the last
    k, v = (torch.empty((E, S, H_KV, D), device="cuda") for _ in range(2))
    assert (E - 1) * S * H_KV * D == 2 ** 32
    g = torch.Generator(device="cuda").manual_seed(1)
    for t in (k, v):
        t[-1].normal_(generator=g)
        t[0, :2000] = float("nan")  # where 32 bits would lead
    for tokens in (1, 9):  # units of 16 rows and of 64
        q = torch.empty((tokens, 4 * H_KV, D), device="cuda").normal_(generator=g)
        out = gqa.cross_attend(q, k, v, i32([0] * (E - 1) + [2000]), i32([0] * E + [tokens]), 0.1)
        bound = tolerance(q, [k[-1, :2000]], [v[-1, :2000]], 0.1, 2000)
        for i in range(tokens):
            assert float((out[i].double() - attend64(q[i], k[-1, :2000], v[-1, :2000], 0.1)).abs().max()) <= bound


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("Q", [1, 6], ids=["few", "many"])
def test_far_pages(Q, dtype):
    ps, n_pages, B = 64, 65_800, 4  # of 2^16 elements: page 65536 starts at element 2^32
    pools = [torch.empty((n_pages, ps, H_KV, D), dtype=dtype, device="cuda") for _ in range(2)]
    first = n_pages - 3 * B - 4
    assert first * ps * H_KV * D >= 2 ** 32
    g = torch.Generator(device="cuda").manual_seed(1)
    for t in pools:
        t[first:].normal_(generator=g)
        t[first - 65_536:n_pages - 65_536] = float("nan")  # where 32 bits would lead
    table = torch.full((B, 8), -1, dtype=torch.int32, device="cuda")
    table[:, :4] = torch.arange(first, first + 4)
    table[:, 4:7] = torch.arange(first + 4, n_pages).view(B, 3)
    lens = [256 + n for n in (Q, 64, 150, 192)]
    q = torch.empty((B, Q, 8 * H_KV, D), device="cuda").normal_(generator=g).to(dtype)
    status = i32([0])
    out = gqa.decode_shared_paged(q, *pools, table, i32(lens), i32([0, B]), i32([256]), 0.1, status=status)
    assert int(status) == 0
    for b, n in enumerate(lens):
        k, v = (t[table[b, :7].long()].flatten(0, 1) for t in pools)
        bound = tolerance(q, [k[:n]], [v[:n]], 0.1, n)
        for j in range(Q):
            m = n - Q + 1 + j
            assert float((out[b, j].double() - attend64(q[b, j], k[:m], v[:m], 0.1)).abs().max()) <= bound
