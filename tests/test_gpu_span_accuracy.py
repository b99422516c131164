"""The accuracy that the span kernels are built for: every output within the bound of span_bounds.py, and, over
pieces of many tiles, outputs that do not lean towards zero."""
import pytest
import torch

import grouped_query_attention_decode_b200 as gqa
import test_gpu_cross as cross
import test_gpu_shared as shared
from span_bounds import attend_and_bound, lean, lean_bound
from test_gpu_span_paths import FEW, MANY, MANY_FEW, TYPES, kernel, launched

pytestmark = pytest.mark.gpu


def within(out, q, k, v, scale):
    """out, q [T, H_q, d] over all rows of k, v [n, H_kv, d], head by head."""
    T, H_q, d = q.shape
    r = H_q // k.shape[1]
    for h in range(k.shape[1]):
        rows = q[:, h * r:(h + 1) * r].reshape(T * r, d)
        ref, bound = attend_and_bound(rows, k[:, h], v[:, h], scale, q.dtype == torch.bfloat16)
        over = ((out[:, h * r:(h + 1) * r].reshape(T * r, d).double() - ref).abs() / bound).max()
        assert float(over) <= 1, (h, float(over))  # NaN fails too


@TYPES
@pytest.mark.parametrize("scale", [0.5, 1.0, -1.5], ids=lambda s: "scale %.1f" % s)  # times d ** -0.5
@pytest.mark.parametrize("states", [[1, 17], [300, 129], [5000, 4097]], ids=str)
@pytest.mark.parametrize("heads", [(16, 4, 64), (16, 4, 128), (64, 8, 64), (64, 8, 128)], ids=lambda h: "%d_%d_%d" % h)
@pytest.mark.parametrize("tokens", [[1, 2], [40, 70]], ids=["few", "many"])
def test_cross_attention(tokens, heads, states, scale, dtype):
    x = cross.make(tokens, states, heads, dtype)
    scale *= heads[2] ** -0.5
    out, status = launched(lambda: cross.run(x, scale), kernel(dtype, heads[2], False, tokens == [1, 2]))
    assert status == 0
    for e, n in enumerate(states):
        i = slice(x["starts"][e], x["starts"][e + 1])
        within(out[i], x["q"][i].cuda(), x["k"][e, :n].cuda(), x["v"][e, :n].cuda(), scale)


@TYPES
@pytest.mark.parametrize("page_size", [0, 16, 128])
@pytest.mark.parametrize("case", MANY_FEW + MANY + FEW + [([0, 2, 12], [4096, 6400], [700 + i * 50 for i in range(12)], (64, 8, 128), 1)],
                         ids=lambda c: "%d_%d_%d" % c[3] + "_%d_%d" % (c[4], len(c[2])))
def test_shared_rows(case, page_size, dtype):
    starts, prefix, own, heads, Q = case
    x = shared.make(starts, prefix, own, len(own), Q, heads, dtype)
    scale = heads[2] ** -0.5
    out, status = shared.run_paged(x, page_size, scale) if page_size else shared.run(x, scale)
    assert status == 0
    out, q = (t.cuda().view(len(own), Q, *heads[::2]) for t in (out, x["q"]))
    for b, n in enumerate(own):
        g = shared.group(starts, b)
        h = prefix[g] if g >= 0 else 0
        k, v = (torch.cat([x[f"{t}_prefix"][max(g, 0), :h], x[f"{t}_cache"][b, :n]]).cuda() for t in "kv")
        for j in range(Q):
            rows = h + n - Q + 1 + j
            if rows > 0:
                within(out[b, j:j + 1], q[b, j:j + 1], k[:rows], v[:rows], scale)
            else:
                assert not out[b, j].any()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("few", [True, False], ids=["few", "many"])
def test_long_pieces_do_not_lean(few, d):
    """Pieces of 40 tiles of 128 rows a CTA, or of 256 of 16 rows a warp: sums that were kept over a piece's
    tiles by additions towards zero would be 1e-5 of their size too small."""
    E, tokens, S, H_q, H_kv = (19 * 128 // d, 4, 4096, 64, 64) if few else (19, 32, 5120, 64, 8)
    g = torch.Generator(device="cuda").manual_seed(d)
    q, k, v = (torch.empty(s, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
               for s in ((E * tokens, H_q, d), (E, S, H_kv, d), (E, S, H_kv, d)))
    i32 = lambda t: torch.tensor(t, dtype=torch.int32, device="cuda")  # noqa: E731
    scale, r = d ** -0.5, H_q // H_kv
    out = launched(lambda: gqa.cross_attend(q, k, v, i32([S] * E), i32([tokens * e for e in range(E + 1)]), scale),
                   kernel(torch.bfloat16, d, False, few))
    ref = torch.empty(out.shape, dtype=torch.float64, device="cuda")
    for e in range(E):
        i = slice(tokens * e, tokens * (e + 1))
        rows = q[i].double().view(tokens, H_kv, r, d).permute(1, 0, 2, 3).reshape(H_kv, tokens * r, d)
        w = torch.softmax(rows @ k[e].double().permute(1, 2, 0) * scale, -1)
        ref[i] = (w @ v[e].double().permute(1, 0, 2)).view(H_kv, tokens, r, d).permute(1, 0, 2, 3).reshape(tokens, H_q, d)
    assert abs(lean(out, ref)) <= lean_bound(d), lean(out, ref)
