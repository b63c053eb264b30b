"""sage_rope against the FP64 rotation: both layouts, rotated widths that do
and do not split into vectors, strided and in-place views, far positions, the
transpose, streams and graphs."""
import numpy as np
import pytest

import cache_util as cu

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def sage():
    import fp8_quantized_exact_b200 as s
    from fp8_quantized_exact_b200 import build
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    return s


DEV = "cuda:0"


def rand(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).to(DEV)


def check(got, x, positions, f, m, half, rot, inverse=False):
    """One BF16 rounding (2^-8 of the value; the smallest step below the normal
    range), and cos and sin off by 2^-21 each: the turn's FP32 rounding is
    2 pi 2^-25 of an angle below half a turn, sincospi and the products a few 2^-24."""
    want = cu.rope(x, positions, f, m, half, rot, inverse)
    a = x.double().abs()
    i0 = torch.arange(rot // 2) if half else torch.arange(0, rot, 2)
    i1 = i0 + (rot // 2 if half else 1)
    size = torch.zeros_like(want)
    size[..., i0] = size[..., i1] = (a[..., i0] + a[..., i1]) * m
    tol = 2.0 ** -8 * want.abs() + 2.0 ** -21 * size + 2.0 ** -134
    bad = (got.double() - want).abs() > tol
    assert not bad.any(), torch.nonzero(bad)[:4].tolist()
    assert torch.equal(got[..., rot:], x[..., rot:])


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 64), (128, 112), (128, 2), (128, 30), (64, 64), (64, 48), (64, 8),
                                   (64, 34), (64, 62)])
@pytest.mark.parametrize("B,N,Hq,Hk", [(1, 1, 1, 1), (2, 3, 7, 1), (1, 130, 4, 2), (5, 1, 56, 8)])
def test_rope_shapes(sage, half, D, rot, B, N, Hq, Hk):
    q, k = rand(B, N, Hq, D, seed=N + rot), rand(B, N, Hk, D, seed=rot)
    pos = torch.randint(0, 200000, (B, N), generator=torch.Generator().manual_seed(rot), dtype=torch.int32)
    f, m = sage.sage_rope_freqs(rot, scaling=sage.SAGE_ROPE_YARN, factor=3.0)
    layout = sage.SAGE_ROPE_HALF if half else sage.SAGE_ROPE_INTERLEAVED
    for inverse in (False, True):
        qo, ko = torch.full_like(q, 7), torch.full_like(k, 7)
        sage.sage_rope(q, k, qo, ko, pos.to(DEV), f, m, layout, rot, inverse)
        check(qo, q, pos, f.cpu(), m, half, rot, inverse)
        check(ko, k, pos, f.cpu(), m, half, rot, inverse)


def test_rope_far_and_negative_positions(sage):
    """Positions to 2^31: the angle's FP64 product is off by 2^-53 of 2^31
    radians, 2^-22, which the check's 2^-21 covers."""
    q = rand(1, 6, 2, 128, seed=3)
    pos = torch.tensor([[0, 1, 1000003, 2**30 + 7, -5, -999999]], dtype=torch.int32)
    f, m = sage.sage_rope_freqs(128)
    out = torch.empty_like(q)
    sage.sage_rope(q, None, out, None, pos.to(DEV), f, m)
    check(out, q, pos, f.cpu(), m, True, 128)
    assert torch.equal(out[0, 0], q[0, 0])  # position 0 turns nothing


def test_rope_default_and_shared_positions(sage):
    q = rand(3, 40, 2, 64, seed=4)
    f, m = sage.sage_rope_freqs(64)
    a, b = torch.empty_like(q), torch.empty_like(q)
    sage.sage_rope(q, None, a, None, None, f, m)
    sage.sage_rope(q, None, b, None, torch.arange(40, dtype=torch.int32, device=DEV), f, m)
    assert torch.equal(a, b)
    check(a, q, torch.arange(40).expand(3, 40), f.cpu(), m, True, 64)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("rot", [128, 32, 20])
def test_rope_strided_and_in_place(sage, half, rot):
    """Column ranges of one projection buffer, in place: V's columns and the
    channels behind the rotated ones stay as they were."""
    buf = rand(2, 37, 12 * 128, seed=5)
    old = buf.clone()
    view = lambda t, h0, h: t[..., h0 * 128:(h0 + h) * 128].unflatten(-1, (h, 128))
    pos = torch.randint(0, 5000, (2, 37), dtype=torch.int32, device=DEV)
    f, m = sage.sage_rope_freqs(rot, base=500000.0)
    layout = sage.SAGE_ROPE_HALF if half else sage.SAGE_ROPE_INTERLEAVED
    q, k = view(buf, 0, 6), view(buf, 6, 3)
    sage.sage_rope(q, k, q, k, pos, f, m, layout, rot)
    check(q, view(old, 0, 6), pos.cpu(), f.cpu(), m, half, rot)
    check(k, view(old, 6, 3), pos.cpu(), f.cpu(), m, half, rot)
    assert torch.equal(view(buf, 9, 3), view(old, 9, 3))
    # q in place, k to another tensor: the untouched channels are still copied
    buf2, ko = old.clone(), torch.full((2, 37, 3, 128), 9, dtype=torch.bfloat16, device=DEV)
    sage.sage_rope(view(buf2, 0, 6), view(buf2, 6, 3), view(buf2, 0, 6), ko, pos, f, m, layout, rot)
    assert torch.equal(view(buf2, 0, 6), q) and torch.equal(ko, k)


def test_rope_broadcast_input(sage):
    x = rand(1, 5, 1, 64, seed=6).expand(4, 5, 3, 64)
    f, m = sage.sage_rope_freqs(64)
    out = torch.empty(4, 5, 3, 64, dtype=torch.bfloat16, device=DEV)
    pos = torch.arange(20, dtype=torch.int32).view(4, 5)
    sage.sage_rope(x, None, out, None, pos.to(DEV), f, m)
    check(out, x, pos, f.cpu(), m, True, 64)


@pytest.mark.parametrize("half", [True, False])
def test_rope_gradient(sage, half):
    """<g, J x> = <J^T g, x>, J^T by the inverse call, and by differences of
    the FP64 map along each input channel."""
    x, g = rand(1, 9, 2, 64, seed=7), rand(1, 9, 2, 64, seed=8)
    pos = torch.arange(100, 109, dtype=torch.int32)[None]
    f, m = sage.sage_rope_freqs(48, scaling=sage.SAGE_ROPE_YARN, factor=2.0)
    layout = sage.SAGE_ROPE_HALF if half else sage.SAGE_ROPE_INTERLEAVED
    dx = torch.empty_like(g)
    sage.sage_rope(g, None, dx, None, pos.to(DEV), f, m, layout, 48, True)
    xx = x.cpu().double().requires_grad_(True)
    (cu.rope(xx, pos, f.cpu(), m, half, 48) * g.cpu().double()).sum().backward()
    want = xx.grad
    assert ((dx.cpu().double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -19 * 4).all()
    base = x.cpu().double()
    for d in (0, 1, 23, 24, 47, 48, 63):
        e = torch.zeros(64, dtype=torch.float64)
        e[d] = 0.5
        diff = ((cu.rope(base + e, pos, f.cpu(), m, half, 48) - cu.rope(base - e, pos, f.cpu(), m, half, 48)) *
                g.cpu().double()).sum(-1)
        assert ((dx.cpu().double()[..., d] - diff).abs() <= 2.0 ** -8 * diff.abs() + 2.0 ** -17).all(), d


def test_rope_stream_and_graph(sage):
    q = rand(2, 8, 4, 128, seed=9)
    f, m = sage.sage_rope_freqs(128)
    pos = torch.arange(16, dtype=torch.int32, device=DEV).view(2, 8)
    out = torch.zeros_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    sage.sage_rope(q, None, out, None, pos, f, m, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    check(out, q, pos.cpu(), f.cpu(), m, True, 128)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sage.sage_rope(q, None, out, None, pos, f, m)
    pos += 1000
    q.copy_(rand(2, 8, 4, 128, seed=10))
    graph.replay()
    torch.cuda.synchronize()
    check(out, q, pos.cpu(), f.cpu(), m, True, 128)


def test_rope_non_finite_values_stay_in_their_pair(sage):
    q = rand(1, 2, 1, 64, seed=11)
    q[0, 0, 0, 3] = float("inf")
    q[0, 1, 0, 40] = float("nan")
    f, m = sage.sage_rope_freqs(64)
    out = torch.empty_like(q)
    sage.sage_rope(q, None, out, None, torch.tensor([5, 6], dtype=torch.int32, device=DEV), f, m)
    bad = ~torch.isfinite(out)
    assert set(torch.nonzero(bad[0, 0, 0]).flatten().tolist()) == {3, 35}
    assert set(torch.nonzero(bad[0, 1, 0]).flatten().tolist()) == {8, 40}


def test_rope_refusals(sage):
    q = rand(1, 2, 1, 64)
    f, m = sage.sage_rope_freqs(64)
    with pytest.raises(ValueError):
        sage.sage_rope(q, None, q[:, :1], None, None, f, m)
    with pytest.raises(ValueError):
        sage.sage_rope(q, None, q, None, torch.zeros(1, 2, dtype=torch.int64, device=DEV), f, m)
    with pytest.raises(ValueError):
        sage.sage_rope(q, None, q, None, None, f, m, rot_dim=32)
    with pytest.raises(ValueError):
        sage.sage_rope(q.float(), None, q, None, None, f, m)
