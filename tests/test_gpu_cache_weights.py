"""Attention over the quantised cache where small weights carry the output: a first key that takes nearly all of the
probability and has next to no value, a key of huge value and no probability, and V scales over many orders.  The
error is judged by the row's own sum of p |v|, whatever the largest value or probability is."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
INT8, E4M3 = 0, 1
PAGE = 128


@pytest.fixture(scope="module")
def sage():
    import fp8_quantized_exact_b200 as s
    from fp8_quantized_exact_b200 import build
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    return s


def problem(sage, n, T, G, D, vf, score, vscale, seed):
    """One sequence of n context tokens and T drafted ones: the context's scores (natural units) and V scales are given
    [H, n], the drafted tokens' are 30 below the smallest and the smallest.  V codes have a mean, so the small weights add up.  All
    channels of K are +-127 times its scale and Q's are a power of two, so a score is exact but for its scale."""
    H = score.shape[0]
    g = torch.Generator().manual_seed(seed)
    pages = -(-(n + T) // PAGE)
    cache = sage.cache_buffers(pages, H, PAGE, D, INT8, vf)
    u = torch.where(torch.rand(D, generator=g) < 0.5, -1, 1)
    s = torch.cat((score.double(), torch.full((H, T), float(score.min()) - 30.0, dtype=torch.float64)), 1)
    vs = torch.cat((vscale.double(), torch.full((H, T), float(vscale.min()), dtype=torch.float64)), 1).float()
    q = (u * 0.5).bfloat16().to(DEV).expand(1, T, H * G, D).contiguous()
    # score = 0.5 * D * 127 * scale / sqrt(D)
    ks = (s.abs() / (63.5 * math.sqrt(D))).float()
    kc = (127 * torch.where(s < 0, -1, 1)[..., None] * u).to(torch.int8)
    if vf == INT8:
        vc = torch.randint(-20, 128, (H, n + T, D), generator=g).to(torch.int8)
    else:
        vc = (torch.rand(H, n + T, D, generator=g) * 500 - 60).clamp(-448, 448).to(torch.float8_e4m3fn)

    def lay(x):  # [H, n + T, ...] -> [pages, H, PAGE, ...]
        y = torch.zeros((H, pages * PAGE) + x.shape[2:], dtype=torch.float32)
        y[:, :n + T] = x.float()
        return y.view((H, pages, PAGE) + x.shape[2:]).transpose(0, 1)

    for to, x in zip(cache, (kc, ks, vc, vs)):
        to.copy_(lay(x).to(to.dtype))
    return q, cache, torch.arange(pages, dtype=torch.int32, device=DEV)[None], kc, ks, vc, vs


def check(sage, n, T, G, D, vf, score, vscale, B, seed, left_out=()):
    """B sequences share the pages, so that there are enough units (sequence and head) for each to lie in one stretch of
    the work list, or few enough that each is cut; all give the same rows but for where they are cut.  left_out: pages
    whose table entry names none."""
    q, cache, table, kc, ks, vc, vs = problem(sage, n, T, G, D, vf, score, vscale, seed)
    keep = torch.ones(n, dtype=torch.bool)
    for page in left_out:
        table[0, page] = -1
        keep[page * PAGE:(page + 1) * PAGE] = False
    H = ks.shape[0]
    ws = sage.workspace(sage.SAGE_OP_CACHE_ATTN, 1, 1, 1, D)
    out = torch.full((B, T, H * G, D), 5.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((B, T, H * G), 5.0, device=DEV)
    sage.sage_cache_attn(q.expand(B, -1, -1, -1), cache, table.expand(B, -1).contiguous(),
                         torch.full((B,), n, dtype=torch.int32, device=DEV), None, None, out, lse, 0.0, ws)
    torch.cuda.synchronize()
    assert sage.sage_read_device_status(ws) == (sage.SAGE_ERR_DEVICE if left_out else sage.SAGE_OK)
    kc, ks, vc, vs = (x[:, :n][:, keep] for x in (kc, ks, vc, vs))
    kk = kc.double().to(DEV) * ks[..., None].double().to(DEV)
    s = (kk @ q[0, 0, 0].double()) * D ** -0.5  # [H, n]; the drafted tokens' share is below e^-30 of the smallest
    p = torch.softmax(s, -1)
    v = vc.double().to(DEV) * vs[..., None].double().to(DEV)
    want = torch.einsum("hn,hnd->hd", p, v)
    spread = torch.einsum("hn,hnd->hd", p, v.abs())
    # a score is an FP32 sum of D products of one sign and three more roundings: (D + 4) 2^-24 of itself, which moves p and
    # the denominator by that; a weight is rounded to FP16 (2^-11); exp2 and the FP32 steps 2^-19; sums over n keys n 2^-24;
    # the result to BF16 (2^-8)
    ds = (s.abs().amax(-1) * (D + 4) * 2.0 ** -24)[:, None]
    tol = spread * (2.0 ** -11 + 2 * ds + 2.0 ** -19 + n * 2.0 ** -24) + 2.0 ** -8 * want.abs()
    got = out.double().view(B, T, H, G, D)
    err = (got - want[None, None, :, None]).abs()
    worst = float((err / tol[None, None, :, None]).max())
    assert worst <= 1.0, (worst, float((err.norm(dim=-1) / want.norm(dim=-1)[None, None, :, None]).max()))
    wl = torch.logsumexp(s, -1)
    el = (lse.double().view(B, T, H, G) - wl[None, None, :, None]).abs()
    assert (el <= (ds[:, 0] + 2.0 ** -22 * (wl.abs() + 1) + n * 2.0 ** -24)[None, None, :, None]).all(), float(el.max())


# rows per head 4 and 8 (one group of rows), 16 (two), 52 and 128 (the tcgen05 variant)
SHAPES = [(1, 4, 128), (1, 8, 64), (2, 8, 128), (2, 8, 64), (16, 8, 128), (13, 4, 64)]
# sequences times 8 heads: more units than warps of all CTAs, and so few that every unit is cut
WHOLE, CUT = 190, 3


def noise(H, n, sigma, seed):
    return torch.randn(H, n, generator=torch.Generator().manual_seed(seed), dtype=torch.float64) * sigma


def count(T, G, D, B):
    """A CTA of the tcgen05 variant has one stretch, not one per warp."""
    return -(-B // 10) if T * G > (32 if D == 128 else 48) and B > CUT else B


@pytest.mark.parametrize("T,G,D", SHAPES)
@pytest.mark.parametrize("B", [WHOLE, CUT])
@pytest.mark.parametrize("n,mass,small", [(8192, 0.9, 1e-3), (8192, 0.999, 1e-3), (32768, 0.997, 1e-3), (32768, 0.999, 0.0),
                                          (151241, 0.985, 1e-3), (151241, 0.996, 1e-3), (8192, 1 - 1e-9, 0.0)])
def test_key_of_nearly_all_the_probability_and_no_value(sage, n, mass, small, B, T, G, D):
    H = 8
    s = noise(H, n, 1.0, n)
    s -= torch.logsumexp(s, -1, keepdim=True)  # the tail's sum is 1
    at = [0, 5, n // 2, n - 1, 1, 40, 700, 64]  # where the key is, by head
    vs = torch.exp(0.3 * noise(H, n, 1.0, n + 1))
    for h, a in enumerate(at):
        s[h, a] = math.log(mass / (1 - mass))
        vs[h, a] = small
    check(sage, n, T, G, D, INT8 if D == 64 else E4M3, s, vs, count(T, G, D, B), seed=n)


@pytest.mark.parametrize("T,G,D", SHAPES)
@pytest.mark.parametrize("B", [WHOLE, CUT])
@pytest.mark.parametrize("n", [100, 1000, 8192])
@pytest.mark.parametrize("power", [6, 12, 18, 30])
def test_key_of_huge_value_and_no_probability(sage, power, n, B, T, G, D):
    H = 8
    s = noise(H, n, 2.0, power)
    vs = torch.exp(0.3 * noise(H, n, 1.0, n + 1))
    for h, a in enumerate([0, 5, n // 2, n - 1, 1, 40, 70, 64]):
        s[h, a] = float(torch.logsumexp(s[h], -1)) - 60.0
        vs[h, a] = 2.0 ** power
    check(sage, n, T, G, D, E4M3 if D == 64 else INT8, s, vs, count(T, G, D, B), seed=n)


@pytest.mark.parametrize("T,G,D", SHAPES)
@pytest.mark.parametrize("B", [WHOLE, CUT])
@pytest.mark.parametrize("kind", ["rising", "falling", "wild", "against", "tiny", "large", "largest"])
def test_value_scales_over_many_orders(sage, kind, B, T, G, D):
    """V scales that rise or fall by 2^60 along the context with scores that undo most of it, that are wild, that are the
    inverse of the probability (every key gives the same share), that are all tiny or large, and that put V at the largest
    BF16 values."""
    H, n = 8, 4096
    s = noise(H, n, 2.0, 5)
    vs = torch.exp(0.3 * noise(H, n, 1.0, 6))
    ramp = torch.linspace(0.0, 60.0, n, dtype=torch.float64)
    if kind in ("rising", "falling"):
        e = ramp if kind == "rising" else ramp.flip(0)
        vs = vs * torch.exp2(e - 30.0)
        s = s - 0.9 * e * math.log(2.0)
    elif kind == "wild":
        vs = torch.exp(4.0 * noise(H, n, 1.0, 7))
    elif kind == "against":
        s = noise(H, n, 8.0, 8)
        vs = torch.exp(-s)
    elif kind == "largest":
        vs = torch.full((H, n), 3.38e38 / (127 if D == 64 else 448), dtype=torch.float64)
    else:
        vs = vs * (1e-34 if kind == "tiny" else 1e30)
    check(sage, n, T, G, D, INT8 if D == 64 else E4M3, s, vs, count(T, G, D, B), seed=1)


@pytest.mark.parametrize("T,G,D", SHAPES)
@pytest.mark.parametrize("kind", ["equal", "steps"])
def test_scores_that_do_not_differ_and_that_climb(sage, kind, T, G, D):
    """All weights alike, at the top of their range; and scores that climb by a little in every tile."""
    H, n = 8, 5000
    s = torch.zeros(H, n, dtype=torch.float64) + 1.0
    if kind == "steps":
        s = s + torch.arange(n, dtype=torch.float64) // 32 * 0.7
    check(sage, n, T, G, D, E4M3, s, torch.ones(H, n, dtype=torch.float64), count(T, G, D, WHOLE), seed=2)


@pytest.mark.parametrize("T,G,D", SHAPES)
@pytest.mark.parametrize("B", [WHOLE, CUT])
@pytest.mark.parametrize("kind", ["rising", "wild"])
def test_pages_left_out_between_value_scales(sage, kind, B, T, G, D):
    """Pages left out in the middle of a context (tiles that not every group of keys has), with V scales that grow before,
    on and behind them."""
    H, n = 8, 4000
    s = noise(H, n, 2.0, 9)
    vs = torch.exp(4.0 * noise(H, n, 1.0, 10)) if kind == "wild" else torch.exp2(torch.linspace(-20.0, 20.0, n, dtype=torch.float64)).expand(H, n)
    check(sage, n, T, G, D, INT8 if D == 64 else E4M3, s, vs, count(T, G, D, B), seed=3, left_out=(0, 7, 8, 19, 30))


@pytest.mark.parametrize("T,G,D", SHAPES)
@pytest.mark.parametrize("poison", [math.inf, -math.inf, math.nan])
def test_poison_in_q_spoils_its_row_and_no_other(sage, poison, T, G, D):
    """An infinity or a NaN in a Q row, on a channel where all keys have one sign: every score of the row is that infinity
    or NaN, and so the row is NaN, also where all are -infinity; a row that sees nothing stays 0 and -infinity, and the
    other rows keep their bits."""
    B, H, n, page = 2, 2, 150, 16
    g = torch.Generator().manual_seed(T + D)
    context = torch.tensor([n, 0], dtype=torch.int32, device=DEV)
    pages = -(-(n + T) // page)
    cache = sage.cache_buffers(B * pages, H, page, D)
    table = torch.arange(B * pages, dtype=torch.int32, device=DEV).view(B, pages)
    x = torch.randn(B, n + T, H, D, generator=g)
    x[..., 3] = x[..., 3].abs() + 0.1
    ws = sage.workspace(sage.SAGE_OP_CACHE_ATTN, 1, 1, 1, D)
    sage.sage_cache_append(cache, x.bfloat16().to(DEV), x.bfloat16().to(DEV), table, None, None, ws)
    q = torch.randn(B, T, H * G, D, generator=g).bfloat16().to(DEV)
    mask = torch.zeros(B, T, -(-T // 32), dtype=torch.int32, device=DEV)
    mask[:, 1:, 0] = 1  # the rows of token 0 of the second sequence see nothing, the others the first drafted token

    def run(q):
        out, lse = torch.full_like(q, 5.0), torch.full((B, T, H * G), 5.0, device=DEV)
        sage.sage_cache_attn(q, cache, table, context, None, mask, out, lse, 0.0, ws)
        torch.cuda.synchronize()
        assert sage.sage_read_device_status(ws) == sage.SAGE_OK
        return out, lse

    want, wl = run(q)
    assert torch.isfinite(want).all() and (want[1, 0] == 0).all() and (wl[1, 0] == -math.inf).all()
    bad = q.clone()
    spoiled = torch.zeros(B, T, H * G, dtype=torch.bool, device=DEV)
    for t, h in ((0, 0), (T - 1, 1), (T // 2, H * G - 1)):
        bad[:, t, h, 3] = poison
        spoiled[:, t, h] = True
    spoiled[1, 0] = False
    out, lse = run(bad)
    assert torch.isnan(out[spoiled]).all() and torch.isnan(lse[spoiled]).all()
    assert torch.equal(out[~spoiled].view(torch.int16), want[~spoiled].view(torch.int16))
    assert torch.equal(lse[~spoiled], wl[~spoiled])
