"""The bounds of span_bounds.py against the kernels' arithmetic done on the CPU: they hold for what the kernels
are built to do, and fail with one bf16 part for the weights, with sums kept over many tiles by additions that
round towards zero, and with scores of TF32."""
import numpy as np
import pytest
import torch

from span_bounds import attend_and_bound, lean, lean_bound


def towards_zero(x):
    """float64 to float32, towards zero."""
    y = x.astype(np.float32)
    return np.where(np.abs(y.astype(np.float64)) > np.abs(x), np.nextafter(y, np.float32(0)), y).astype(np.float32)


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).float().numpy()


def tf32(x):
    return (x.view(np.uint32) & np.uint32(0xFFFFE000)).view(np.float32)


def emulate(q, k, v, scale, parts=2, restart=True, T=128, score_type=None):
    """out [R, d] of one piece: tiles of T rows, products of 16, as span_tc.cu adds them."""
    q, k, v = (t.float().numpy() for t in (q, k, v))
    if score_type is not None:
        q, k = score_type(q), score_type(k)
    s = np.zeros((q.shape[0], k.shape[0]), np.float32)
    for i in range(0, q.shape[1], 16):
        s = towards_zero(s + q[:, i:i + 16].astype(np.float64) @ k[:, i:i + 16].astype(np.float64).T)
    y = s * np.float32(scale * 1.4426950408889634)
    w = np.exp2(y - y.max(-1, keepdims=True)).astype(np.float32)
    hi = bf16(w) if parts else w
    lo = bf16(w - hi) if parts == 2 else np.zeros_like(w)
    total = np.zeros((q.shape[0], v.shape[1]), np.float32)
    run = np.zeros_like(total)
    for t in range(0, k.shape[0], T):
        if restart:
            run = np.zeros_like(total)
        for part in (hi, lo):
            for i in range(t, min(t + T, k.shape[0]), 16):
                run = towards_zero(run + part[:, i:i + 16].astype(np.float64) @ v[i:i + 16].astype(np.float64))
        if restart:
            total = total + run
    out = total if restart else run
    return torch.from_numpy(out / w.sum(-1, keepdims=True, dtype=np.float32))


def case(n, d, dtype, R=24):
    g = torch.Generator().manual_seed(n + d)
    return [torch.randn(s, generator=g).to(dtype) for s in ((R, d), (n, d), (n, d))] + [d ** -0.5]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 17, 300, 5000])
def test_bounds_hold(n, d):
    for dtype, parts in ((torch.bfloat16, 2), (torch.float32, 0)):
        q, k, v, scale = case(n, d, dtype)
        ref, bound = attend_and_bound(q, k, v, scale, parts == 2)
        out = emulate(q, k, v, scale, parts=parts)
        assert ((out.double() - ref).abs() <= bound).all()
        if n == 5000:
            assert abs(lean(out, ref)) <= lean_bound(d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [17, 300, 5000])
def test_one_part_does_not_pass(n, d):
    q, k, v, scale = case(n, d, torch.bfloat16)
    ref, bound = attend_and_bound(q, k, v, scale, True)
    over = (emulate(q, k, v, scale, parts=1).double() - ref).abs() / bound
    assert float(over.max()) > 3


@pytest.mark.parametrize("d", [64, 128])
def test_sums_over_many_tiles_do_not_pass(d):
    q, k, v, scale = case(5000, d, torch.bfloat16)
    ref, _ = attend_and_bound(q, k, v, scale, True)
    assert abs(lean(emulate(q, k, v, scale, restart=False), ref)) > 2 * lean_bound(d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [17, 300, 5000])
def test_tf32_scores_do_not_pass(n, d):
    q, k, v, scale = case(n, d, torch.float32)
    ref, bound = attend_and_bound(q, k, v, scale, False)
    over = (emulate(q, k, v, scale, parts=0, score_type=tf32).double() - ref).abs() / bound
    assert float(over.max()) > 2
