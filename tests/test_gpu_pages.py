"""The page calls (gqa_pages_*) against a sequential model of them on the host, and a run of them with
the appends and decodes they serve."""
import numpy as np
import pytest
import torch

import grouped_query_attention_decode_b200 as gqa
from span_ref import attend64, normal, tolerance

pytestmark = pytest.mark.gpu


class Pages:
    """The state on the host, changed one sequence at a time."""

    def __init__(self, B, max_pages, n_pages, page_size):
        self.table = np.full((B, max_pages), -1, np.int32)
        self.lens = np.zeros(B, np.int32)
        self.refs = np.zeros(n_pages, np.int32)
        self.ps = page_size

    def fork(self, parents):
        out, lens = np.full((len(parents), self.table.shape[1]), -1, np.int32), np.zeros(len(parents), np.int32)
        for i, p in enumerate(parents):
            if 0 <= p < len(self.lens):
                out[i], lens[i] = self.table[p], self.lens[p]
        self.table, self.lens = out, lens
        self.refs = np.bincount(out[out >= 0], minlength=len(self.refs)).astype(np.int32)

    def free(self, seqs):
        for s in seqs:
            if 0 <= s < len(self.lens):
                for p in self.table[s][self.table[s] >= 0]:
                    self.refs[p] -= 1
                self.table[s], self.lens[s] = -1, 0

    def reserve(self, rows):
        """(copies, refused or not served)"""
        copies, full = np.full((len(self.lens), 2), -1, np.int32), 0
        for b, n in enumerate(self.lens):
            if n < 0 or n + rows > self.table.shape[1] * self.ps:
                full |= gqa.STATUS_APPEND_OVERFLOW
                continue
            slots = range(n // self.ps, (n + rows - 1) // self.ps + 1)
            need = [j for j in slots if self.table[b, j] < 0 or self.refs[self.table[b, j]] > 1]
            free = np.flatnonzero(self.refs == 0)
            if full & gqa.STATUS_POOL_FULL or len(need) > len(free):
                full |= gqa.STATUS_POOL_FULL
                continue
            for j, page in zip(need, free):
                old = self.table[b, j]
                if old >= 0:
                    self.refs[old] -= 1
                    if j == n // self.ps and n % self.ps:
                        copies[b] = old, page
                self.table[b, j], self.refs[page] = page, 1
        return copies, full

    def compact(self):
        n = int((self.refs > 0).sum())
        pairs = list(zip([i for i in range(n, len(self.refs)) if self.refs[i] > 0], [i for i in range(n) if self.refs[i] <= 0]))
        for a, b in pairs:
            self.table[self.table == a] = b
            self.refs[b], self.refs[a] = self.refs[a], 0
        copies = np.full((max(1, len(self.refs) // 2), 2), -1, np.int32)
        copies[:len(pairs)] = np.array(pairs, np.int32).reshape(-1, 2)
        return copies, n

    def gpu(self):
        return [torch.from_numpy(a.copy()).cuda() for a in (self.table, self.lens, self.refs)]

    def same(self, table, lens, refs):
        for want, got in zip((self.table, self.lens, self.refs), (table, lens, refs)):
            assert np.array_equal(want, got.cpu().numpy())


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def random_state(rng, B, max_pages, n_pages, ps, seed):
    """Prompts, some forked, some freed."""
    m = Pages(B, max_pages, n_pages, ps)
    for b in range(B):
        m.lens[b] = rng.integers(0, max_pages * ps + 1)
    keep = m.lens.copy()
    m.lens[:] = 0
    for b in range(B):  # reserve for one after another, as far as the pool goes
        one = Pages(1, max_pages, n_pages, ps)
        one.refs = m.refs
        if keep[b] and not one.reserve(int(keep[b]))[1]:
            m.table[b], m.lens[b] = one.table[0], keep[b]
    m.fork([int(x) for x in rng.integers(-1, B, B)])
    # pages spread over the pool, whatever the order they came in
    place = rng.permutation(n_pages).astype(np.int32)
    m.table[m.table >= 0] = place[m.table[m.table >= 0]]
    refs = np.zeros_like(m.refs)
    refs[place] = m.refs
    m.refs = refs
    return m


SIZES = [  # sequences, table width, pages, page size
    (1, 1, 1, 8), (2, 3, 5, 8), (7, 9, 40, 16), (64, 33, 1500, 16), (130, 20, 2050, 8), (1500, 3, 5000, 8), (40, 700, 21001, 8)]


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_fork(size):
    B, max_pages, n_pages, ps = size
    rng = np.random.default_rng(B)
    m = random_state(rng, B, max_pages, n_pages, ps, 1)
    table, lens, refs = m.gpu()
    B_out = max(1, B + int(rng.integers(-3, 4)))
    parents = [int(x) for x in rng.integers(-1, B, B_out)]
    out, lens_out, status = torch.full((B_out, max_pages), 77, dtype=torch.int32, device="cuda"), i32([5] * B_out), word()
    gqa.pages_fork(i32(parents), table, lens, out, lens_out, refs, status=status)
    m.fork(parents)
    m.same(out, lens_out, refs)
    assert int(status) == 0


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_free(size):
    B, max_pages, n_pages, ps = size
    rng = np.random.default_rng(B)
    m = random_state(rng, B, max_pages, n_pages, ps, 1)
    table, lens, refs = m.gpu()
    seqs = [int(x) for x in rng.integers(0, B, max(1, B // 2))]  # some twice
    status = word()
    gqa.pages_free(i32(seqs), table, lens, refs, status=status)
    m.free(seqs)
    m.same(table, lens, refs)
    assert int(status) == 0


@pytest.mark.parametrize("rows", [1, 3, 16, 17, 200])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_reserve(size, rows):
    B, max_pages, n_pages, ps = size
    rng = np.random.default_rng(B + rows)
    m = random_state(rng, B, max_pages, n_pages, ps, 1)
    m.lens = np.minimum(m.lens, np.maximum(0, max_pages * ps - rows)).astype(np.int32)
    if B > 2:
        m.lens[1] = max_pages * ps  # no room for another row
    table, lens, refs = m.gpu()
    for _ in range(2):  # again: nothing more is needed, unless the pool was too small
        status = word()
        copies = gqa.pages_reserve(table, lens, refs, rows, ps, status=status)
        want, bits = m.reserve(rows)
        m.same(table, lens, refs)
        assert np.array_equal(copies.cpu().numpy(), want)
        assert int(status) == bits


def test_last_holder_keeps_its_page():
    m = Pages(4, 4, 10, 8)
    m.lens[0] = 4
    m.reserve(1)
    m.fork([0, 0, 0, -1])
    table, lens, refs = m.gpu()
    copies = gqa.pages_reserve(table, lens, refs, 1, 8)
    assert copies.cpu().tolist() == [[0, 1], [0, 2], [-1, -1], [-1, -1]]
    assert table[:, 0].cpu().tolist() == [1, 2, 0, 3] and refs.cpu().tolist() == [1] * 4 + [0] * 6


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_compact(size):
    B, max_pages, n_pages, ps = size
    rng = np.random.default_rng(B)
    m = random_state(rng, B, max_pages, n_pages, ps, 1)
    m.free(range(0, B, 3))
    table, lens, refs = m.gpu()
    for _ in range(2):  # the second time nothing moves
        status = word()
        copies, live = gqa.pages_compact(table, refs, status=status)
        want, n = m.compact()
        m.same(table, lens, refs)
        assert np.array_equal(copies.cpu().numpy(), want) and int(live) == n and int(status) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.uint8, torch.float8_e4m3fn], ids=str)
@pytest.mark.parametrize("page", [(8, 1, 64), (16, 8, 128), (256, 3, 64)], ids=str)
def test_copy(page, dtype):
    n_pages = 50
    g = torch.Generator().manual_seed(1)
    pools = [torch.randint(0, 255, (n_pages, *page), generator=g, dtype=torch.uint8) for _ in range(2)]
    pools = [p.cuda() if dtype == torch.uint8 else p.view(dtype).cuda() if dtype == torch.float8_e4m3fn else p.to(dtype).cuda() for p in pools]
    before = [p.clone() for p in pools]
    pairs = [[3, 40], [-1, -1], [7, 1], [3, 0], [49, 2]]
    status = word()
    gqa.pages_copy(*pools, i32(pairs), status=status)
    for b in before:
        for x, y in pairs:
            if x >= 0:
                b[y] = b[x]
    raw = lambda t: t.contiguous().view(torch.uint8)  # noqa: E731
    assert all(torch.equal(raw(p), raw(b)) for p, b in zip(pools, before)) and int(status) == 0
    gqa.pages_copy(*pools, i32([[0, 50], [-1, 3], [-2, -2]]), status=status)
    assert all(torch.equal(raw(p), raw(b)) for p, b in zip(pools, before)) and int(status) == gqa.STATUS_INDEX_RANGE


def test_bad_numbers_are_reported():
    m = Pages(3, 4, 10, 8)
    m.lens[:] = 20, 9, 0
    for b in range(3):
        n = m.lens[b]
        m.table[b, :-(-n // 8)] = np.arange(-(-n // 8)) + 3 * b
    m.refs = np.bincount(m.table[m.table >= 0], minlength=10).astype(np.int32)
    table, lens, refs = m.gpu()
    out, lens_out, status = torch.empty_like(table), torch.empty_like(lens), word()
    gqa.pages_fork(i32([0, 3, -2]), table, lens, out, lens_out, refs.clone(), status=status)
    assert int(status) == gqa.STATUS_INDEX_RANGE and (out[1:] == -1).all() and not lens_out[1:].any()
    status = word()
    gqa.pages_free(i32([1, 5, -1]), table, lens, refs, status=status)
    m.free([1])
    m.same(table, lens, refs)
    assert int(status) == gqa.STATUS_INDEX_RANGE
    table[0, 1] = 10  # no such page
    status = word()
    gqa.pages_free(i32([0]), table, lens, refs, status=status)
    assert int(status) == gqa.STATUS_PAGE_RANGE
    table[2, 0] = 9   # held, but counted as free
    status = word()
    gqa.pages_free(i32([2]), table, lens, refs, status=status)
    assert int(status) == gqa.STATUS_PAGE_REFS


def test_no_free_page():
    m = Pages(3, 2, 2, 8)
    table, lens, refs = m.gpu()
    status = word()
    copies = gqa.pages_reserve(table, lens, refs, 1, 8, status=status)
    assert int(status) == gqa.STATUS_POOL_FULL and (copies == -1).all()
    assert table[:, 0].cpu().tolist() == [0, 1, -1] and refs.cpu().tolist() == [1, 1]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_samples_of_two_prompts(dtype):
    """Two prompts, forked into samples that decode on, lose some of their number, move to the front
    of the pool and decode on: every step against float64 over each sequence's own rows."""
    H_q, H_kv, d, ps, n_pages, max_pages, B = 16, 2, 64, 16, 200, 24, 9
    g = torch.Generator().manual_seed(11)
    k_pool = torch.full((n_pages, ps, H_kv, d), float("nan"), dtype=dtype, device="cuda")
    v_pool = k_pool.clone()
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
    lens, refs, status = i32([0] * B), i32([0] * n_pages), word()
    rows = [([], []) for _ in range(B)]  # what each sequence has appended, on the host
    live = list(range(B))

    def step():
        gqa.pages_copy(k_pool, v_pool, gqa.pages_reserve(table, lens, refs, 1, ps, status=status))
        kn, vn = normal((B, H_kv, d), g, dtype), normal((B, H_kv, d), g, dtype)
        gqa.kv_append_paged(kn.cuda(), vn.cuda(), k_pool, v_pool, table, lens, status=status)
        for b in range(B):
            rows[b][0].append(kn[b])
            rows[b][1].append(vn[b])

    for _ in range(70):
        step()
    # samples 0..5 of prompt 0, 6..8 of prompt 1 (which is sequence 3)
    parents = [0] * 6 + [3] * 3
    table2, lens2 = torch.empty_like(table), torch.empty_like(lens)
    gqa.pages_fork(i32(parents), table, lens, table2, lens2, refs, status=status)
    table, lens = table2, lens2
    rows = [(list(rows[p][0]), list(rows[p][1])) for p in parents]
    starts, shared = i32([0, 6, 9]), i32([64, 64])
    for t in range(20):
        step()
        if t >= 10:  # two samples have ended; they still take part in every append
            gqa.pages_free(i32([1, 4]), table, lens, refs, status=status)
            live = [b for b in live if b not in (1, 4)]
        if t == 10:
            pairs, n = gqa.pages_compact(table, refs, status=status)
            gqa.pages_copy(k_pool, v_pool, pairs)
            used = torch.unique(table[table >= 0])
            assert int(n) == len(used) and int(used.max()) == int(n) - 1
        if t % 5 == 1:
            q = normal((B, H_q, d), g, dtype)
            out = gqa.decode_shared_paged(q.cuda(), k_pool, v_pool, table, lens, starts, shared, 0.2, status=status)
            whole = gqa.decode_paged(q.cuda(), k_pool, v_pool, table, lens, 0.2, status=status)
            for b in live:
                k, v = torch.stack(rows[b][0]).cuda(), torch.stack(rows[b][1]).cuda()
                assert int(lens[b]) == len(rows[b][0])
                bound = tolerance(q, [k], [v], 0.2, len(k))
                ref = attend64(q[b].cuda(), k, v, 0.2)
                assert float((out[b].double() - ref).abs().max()) <= bound
                assert float((whole[b].double() - ref).abs().max()) <= bound
    assert int(status) == 0
    want = torch.bincount(table[table >= 0].long(), minlength=n_pages)
    assert torch.equal(want.int(), refs)
    gqa.pages_free(i32(list(range(B))), table, lens, refs, status=status)
    assert not refs.any() and (table == -1).all() and not lens.any()


def test_captured_step():
    """Reserve, copy and append in one graph, replayed."""
    B, H_kv, d, ps, n_pages = 6, 2, 64, 8, 64
    k_pool = torch.zeros((n_pages, ps, H_kv, d), dtype=torch.bfloat16, device="cuda")
    v_pool = torch.zeros_like(k_pool)
    m = Pages(B, 6, n_pages, ps)
    m.lens[0] = 12
    m.table[0, :2] = 5, 9
    m.refs[[5, 9]] = 1
    m.fork([0] * 4 + [-1] * 2)
    table, lens, refs = m.gpu()
    kn = torch.ones((B, H_kv, d), dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        copies = gqa.pages_reserve(table, lens, refs, 1, ps)
        gqa.pages_copy(k_pool, v_pool, copies)
        gqa.kv_append_paged(kn, kn, k_pool, v_pool, table, lens)
    for t in range(20):
        graph.replay()
        m.reserve(1)
        m.lens += 1
    torch.cuda.synchronize()
    m.same(table, lens, refs)


def test_refusals():
    m = Pages(3, 4, 16, 8)
    table, lens, refs = m.gpu()
    out, lens_out = torch.empty_like(table), torch.empty_like(lens)
    with pytest.raises(gqa.GQAError):  # the tables overlap
        gqa.pages_fork(i32([0, 1, 2]), table, lens, table, lens_out, refs)
    with pytest.raises(gqa.GQAError):
        gqa.pages_fork(i32([0, 1, 2]), table, lens, out, lens, refs)
    with pytest.raises(ValueError):
        gqa.pages_fork(i32([0, 1]), table, lens, out, lens_out, refs)
    with pytest.raises(ValueError):
        gqa.pages_free(i32([0]), table.long(), lens, refs)
    with pytest.raises(gqa.GQAError):
        gqa.pages_reserve(table, lens, refs, 0, 8)
    with pytest.raises(gqa.GQAError):
        gqa.pages_reserve(table, lens, refs, 1, 8, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(gqa.GQAError):
        gqa.pages_compact(table, torch.zeros(17, dtype=torch.int32, device="cuda")[1:])  # counts not 16-byte aligned
    pool = torch.zeros((16, 8, 2, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        gqa.pages_copy(pool, pool[:8], i32([[0, 1]]))
    with pytest.raises(ValueError):
        gqa.pages_copy(pool, pool, i32([0, 1]))
    with pytest.raises(gqa.GQAError):
        gqa.pages_copy(torch.zeros((4, 8, 2, 96), dtype=torch.bfloat16, device="cuda"),
                       torch.zeros((4, 8, 2, 96), dtype=torch.bfloat16, device="cuda"), i32([[0, 1]]))


def test_copy_far_pages():
    """Pages whose offsets pass 32 bits (of 16-byte vectors: 2^31 is 32 GiB in; of bytes here)."""
    n_pages = 140_000  # of 32 KiB: 4.6 GB a pool
    k = torch.zeros((n_pages, 16, 8, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    k[n_pages - 1] = 3
    v[n_pages - 2] = 5
    gqa.pages_copy(k, v, i32([[n_pages - 1, 2], [n_pages - 2, n_pages - 3], [0, 1]]))
    assert (k[2] == 3).all() and (v[n_pages - 3] == 5).all() and not k[3].any() and not v[2].any()
