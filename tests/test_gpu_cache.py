"""The quantised paged cache against plain FP64 forms: append (codes and
scales exact), read (exact), attention of new and drafted tokens within the
derived bound, over formats, pages, lengths from zero on, masks, ragged counts,
shared heads, bad pages, streams and graphs; and the whole step together."""
import math

import pytest

import cache_util as cu

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DEV = "cuda:0"
INT8, E4M3 = 0, 1


@pytest.fixture(scope="module")
def sage():
    import fp8_quantized_exact_b200 as s
    from fp8_quantized_exact_b200 import build
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    return s


@pytest.fixture()
def ws(sage):
    w = sage.workspace(sage.SAGE_OP_CACHE_ATTN, 1, 1, 1, 64)
    yield w


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rand(*shape, seed=0):
    return torch.randn(*shape, generator=gen(seed)).to(torch.bfloat16).to(DEV)


def empty_cache(sage, pages, H, page, D, kf, vf):
    """Unwritten slots hold codes of every kind (E4M3 NaN among them) and NaN scales."""
    c = sage.cache_buffers(pages, H, page, D, kf, vf)
    for t in c[::2]:
        t.view(torch.uint8).copy_(torch.randint(0, 256, t.shape, generator=gen(99), dtype=torch.uint8))
    for t in c[1::2]:
        t.fill_(math.nan)
    return c


def make_table(B, per, pages, lens, page, seed=0):
    """Random distinct pages for the pages that the lengths reach; -1 behind them."""
    order = torch.randperm(pages, generator=gen(seed))
    table = torch.full((B, per), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lens):
        m = -(-n // page)
        table[b, :m] = order[at:at + m].int()
        at += m
    assert at <= pages
    return table.to(DEV)


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def status(sage, ws):
    torch.cuda.synchronize()
    return sage.sage_read_device_status(ws)


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kf,vf", [(INT8, E4M3), (E4M3, INT8)])
def test_append_and_read_exact(sage, ws, page, D, kf, vf):
    H, start, count = 3, [0, 5, 100, 17], [70, 0, 1, 33]
    lens = [s + c for s, c in zip(start, count)]
    per = -(-max(lens) // page) + 1
    pages = sum(-(-n // page) for n in lens) + 2
    cache = empty_cache(sage, pages, H, page, D, kf, vf)
    before = [t.clone() for t in cache]
    table = make_table(4, per, pages, lens, page, seed=page)
    N = 75
    x = [rand(4, N, H, D, seed=s) * torch.exp(2 * torch.randn(4, N, H, 1, generator=gen(s))).to(DEV) for s in (1, 2)]
    k, v = (t.to(torch.bfloat16) for t in x)
    sage.sage_cache_append(cache, k, v, table, i32(*start), i32(*count), ws)
    assert status(sage, ws) == 0
    want = [t.clone() for t in before]
    for i, t in enumerate((k, v)):
        dt = cache[2 * i].dtype
        code, scale = cu.quantise(t, dt)
        for b in range(4):
            s = torch.arange(count[b], device=DEV)
            at = (table[b].long()[(start[b] + s) // page], slice(None), (start[b] + s) % page)
            want[2 * i][at] = code[b, :count[b]].to(dt)
            want[2 * i + 1][at] = scale[b, :count[b]]
    for got, w in zip(cache, want):
        assert torch.equal(got.view(torch.uint8 if got.element_size() == 1 else torch.int32),
                           w.view(torch.uint8 if w.element_size() == 1 else torch.int32))
    ko, vo = (torch.full((4, N, H, D), 3.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    sage.sage_cache_read(cache, table, i32(*start), i32(*count), ko, vo, ws)
    for out, i in ((ko, 0), (vo, 2)):
        for b in range(4):
            s = start[b] + torch.arange(count[b], device=DEV)
            at = (table[b].long()[s // page], slice(None), s % page)
            assert torch.equal(out[b, :count[b]], (cache[i][at].float() * cache[i + 1][at][..., None]).to(torch.bfloat16))
            assert (out[b, count[b]:] == 3.0).all()
    only = torch.full_like(ko, 4.0)
    sage.sage_cache_read(cache, table, i32(*start), i32(*count), None, only, ws)
    assert torch.equal(only[0, :70], vo[0, :70])
    assert status(sage, ws) == 0


@pytest.mark.parametrize("fmt", [INT8, E4M3])
def test_append_ties_and_extremes(sage, ws, fmt):
    """Every BF16 value of eight binades against every 8-bit maximum: all half-way
    cases; zeros, subnormals, the largest values; infinities and NaN."""
    D, dt = 128, (torch.int8, torch.float8_e4m3fn)[fmt]
    mant = torch.arange(128, 256, dtype=torch.float64)
    rows = []
    for e in range(0, 12):  # 128 maxima x 12 binades of 127 values below the maximum
        body = (mant[None, 1:] * 2.0 ** -e).expand(128, 127).clone()
        body[body > mant[:, None]] = 1.0
        rows.append(torch.cat((mant[:, None], body * torch.where(torch.arange(127) % 2 == 0, 1.0, -1.0)), 1))
    x = torch.cat(rows)
    special = torch.zeros(8, D, dtype=torch.float64)
    special[1, 5] = 2.0 ** -133
    special[1, 6] = -(2.0 ** -133)
    special[2] = torch.linspace(-1, 1, D, dtype=torch.float64) * 2.0 ** -126
    special[3] = torch.linspace(-1, 1, D, dtype=torch.float64) * 3.3e38
    special[4, 0], special[4, 1] = math.inf, 1.0
    special[5, 0], special[5, 1] = math.nan, 1.0
    special[6, 127] = -math.inf
    special[7, 64] = -0.0
    x = torch.cat((x, x * 2.0 ** -120, special))
    x = x.to(torch.bfloat16)[None, :, None].to(DEV)
    n = x.shape[1]
    cache = empty_cache(sage, -(-n // 64), 1, 64, D, fmt, fmt)
    table = torch.arange(-(-n // 64), dtype=torch.int32, device=DEV)[None]
    sage.sage_cache_append(cache, x, x, table, None, None, ws)
    assert status(sage, ws) == 0
    code, scale = cu.quantise(x[0, :, 0], dt)
    got = cache[0].double().permute(0, 2, 1, 3).reshape(-1, D)[:n]
    assert torch.equal(got, code), torch.nonzero(got != code)[:4].tolist()
    gs = cache[1].permute(0, 2, 1).reshape(-1)[:n]
    assert torch.equal(torch.nan_to_num(gs, nan=-1.0), torch.nan_to_num(scale, nan=-1.0))
    assert torch.isnan(gs[-4:-1]).all()
    assert torch.equal(cache[0].view(torch.uint8), cache[2].view(torch.uint8))
    out = torch.empty_like(x)
    sage.sage_cache_read(cache, table, None, None, out, None, ws)
    assert torch.isnan(out[0, -4:-1]).all() and torch.isfinite(out[0, :-4]).all()


def test_append_strided_default_arguments_and_one_token(sage, ws):
    buf = rand(2, 33, 3 * 4 * 64, seed=3)
    k = buf[..., 4 * 64:8 * 64].unflatten(-1, (4, 64))
    v = buf[..., 8 * 64:].unflatten(-1, (4, 64))
    cache = empty_cache(sage, 12, 4, 16, 64, INT8, INT8)
    table = make_table(2, 4, 12, [48, 48], 16)
    sage.sage_cache_append(cache, k, v, table, None, None, ws)
    one = rand(2, 1, 4, 64, seed=4)
    sage.sage_cache_append(cache, one, one, table, i32(33, 47), None, ws)
    out = torch.zeros(2, 48, 4, 64, dtype=torch.bfloat16, device=DEV)
    sage.sage_cache_read(cache, table, None, None, out, None, ws)
    assert status(sage, ws) == 0
    for b in range(2):
        for x, s, n in ((k[b], 0, 33), (one[b], (33, 47)[b], 1)):
            code, scale = cu.quantise(x, torch.int8)
            want = (code.float() * scale[..., None]).to(torch.bfloat16)
            assert torch.equal(out[b, s:s + n], want)


def test_append_and_read_bad_pages(sage, ws):
    """Tokens on entries that name no page are skipped and reported; the others are written."""
    cache = empty_cache(sage, 4, 1, 16, 64, INT8, INT8)
    before = [t.clone() for t in cache]
    x = rand(1, 80, 1, 64, seed=5)
    for table, start, count, good in (([0, -1, 2, 4], 0, 64, [0, 2]), ([1, 3, 2, 0], 0, 80, [1, 3, 2, 0]),
                                      ([1, 0, 2, 3], -16, 32, [1]), ([1, 0, 2, 3], 2**31 - 8, 16, []),
                                      ([1, 0, 2, 3], 0, -3, []), ([-2**31, 2**31 - 1, 0, 1], 0, 64, [0, 1])):
        for t, o in zip(cache, before):
            t.copy_(o)
        sage.sage_clear_device_status(ws)
        assert status(sage, ws) == 0
        tb = i32(*table)[None]
        sage.sage_cache_append(cache, x, x, tb, i32(start), i32(count), ws)
        assert status(sage, ws) == sage.SAGE_ERR_DEVICE
        changed = [p for p in range(4) if not torch.equal(cache[0][p], before[0][p])]
        assert changed == sorted(good), (table, start, count)
        sage.sage_clear_device_status(ws)
        out = torch.full((1, 80, 1, 64), 2.0, dtype=torch.bfloat16, device=DEV)
        sage.sage_cache_read(cache, tb, i32(start), i32(count), out, None, ws)
        assert status(sage, ws) == sage.SAGE_ERR_DEVICE
        rows = [i for i in range(80) if not (out[0, i] == 2.0).all()]
        assert rows == [i for i in range(min(max(count, 0), 80)) if 0 <= (start + i) // 16 < 4 and
                        0 <= table[(start + i) // 16] < 4]
    # a count above N is taken as N
    sage.sage_clear_device_status(ws)
    sage.sage_cache_append(cache, x[:, :16], x[:, :16], i32(0, 1, 2, 3)[None], None, i32(17), ws)
    assert status(sage, ws) == sage.SAGE_ERR_DEVICE
    # the first error stays over later good calls
    sage.sage_cache_append(cache, x[:, :16], x[:, :16], i32(0, 1, 2, 3)[None], None, None, ws)
    assert status(sage, ws) == sage.SAGE_ERR_DEVICE


# --------------------------------------------------------------- attention
def filled(sage, lens, H, page, D, kf, vf, seed, spread=1.0):
    """A cache with lens[b] tokens per sequence (unwritten slots hold garbage)."""
    per = max(1, -(-max(max(lens), 1) // page))
    pages = sum(-(-n // page) for n in lens) + 2
    cache = empty_cache(sage, pages, H, page, D, kf, vf)
    table = make_table(len(lens), per, pages, lens, page, seed)
    w = sage.workspace(sage.SAGE_OP_CACHE, 1, 1, 1, D)
    N = max(max(lens), 1)
    k, v = rand(len(lens), N, H, D, seed=seed + 1), rand(len(lens), N, H, D, seed=seed + 2)
    v = (v * torch.exp(spread * torch.randn(len(lens), N, H, 1, generator=gen(seed + 3))).to(DEV)).to(torch.bfloat16)
    sage.sage_cache_append(cache, k, v, table, None, i32(*lens), w)
    assert status(sage, w) == 0
    return cache, table


def run_attn(sage, ws, q, cache, table, context, count, mask, scale=0.0):
    B, T, Hq, D = q.shape
    out = torch.full((B, T, Hq, D), 5.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((B, T, Hq), 5.0, device=DEV)
    sage.sage_cache_attn(q, cache, table, context, count, mask, out, lse, scale, ws)
    return out, lse


def check_attn(q, cache, table, context, count, mask, out, lse, scale=None):
    T = q.shape[1]
    want, wl, tol, tl = cu.attention(q, cache, table, context, count, mask, scale)
    for b in range(q.shape[0]):
        n = T if count is None else int(count[b])
        err = (out[b, :n].double() - want[b, :n]).abs()
        assert (err <= tol[b, :n]).all(), (b, float((err - tol[b, :n]).max()), float((err / tol[b, :n]).nan_to_num().max()))
        el = lse[b, :n].double()
        none = torch.isinf(wl[b, :n])
        assert torch.equal(none, torch.isinf(el)) and (el[none] < 0).all()
        assert ((el - wl[b, :n]).abs()[~none] <= tl[b, :n][~none]).all()
        assert (out[b, n:] == 5.0).all() and (lse[b, n:] == 5.0).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("kf,vf", [(INT8, E4M3), (E4M3, INT8), (INT8, INT8), (E4M3, E4M3)])
@pytest.mark.parametrize("T,G", [(1, 1), (1, 7), (4, 4), (9, 8)])
def test_attn_lengths(sage, ws, D, page, kf, vf, T, G):
    context = [0, 1, 15, 16, 63, 64, 65, 127, 128, 129, 300]
    cache, table = filled(sage, [n + T for n in context], 2, page, D, kf, vf, seed=page + T)
    q = rand(len(context), T, 2 * G, D, seed=T)
    ctx = i32(*context)
    out, lse = run_attn(sage, ws, q, cache, table, ctx, None, None)
    assert status(sage, ws) == 0
    check_attn(q, cache, table, ctx, None, None, out, lse)


@pytest.mark.parametrize("T,G,H", [(13, 4, 2), (21, 4, 1), (33, 2, 2), (64, 8, 1), (64, 1, 3), (100, 5, 1), (256, 1, 1),
                                   (129, 2, 1), (16, 16, 1), (2, 8, 4)])
@pytest.mark.parametrize("D,kf,vf", [(128, INT8, E4M3), (64, E4M3, INT8)])
def test_attn_trees(sage, ws, T, G, H, D, kf, vf):
    context = [0, 50, 200]
    cache, table = filled(sage, [n + T for n in context], H, 32, D, kf, vf, seed=T)
    r = gen(T)
    parents = [[int(torch.randint(-1, i, (1,), generator=r)) if i else -1 for i in range(T)] for _ in context]
    mask = cu.tree_mask(parents, DEV)
    q = rand(3, T, H * G, D, seed=T + 1)
    count = i32(T, max(T - 3, 0), 1)
    for cnt in (None, count):
        out, lse = run_attn(sage, ws, q, cache, table, i32(*context), cnt, mask)
        assert status(sage, ws) == 0
        check_attn(q, cache, table, i32(*context), cnt, mask, out, lse)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("D,kf,vf", [(128, E4M3, INT8), (128, INT8, INT8), (64, INT8, E4M3), (64, E4M3, E4M3)])
@pytest.mark.parametrize("T,G", [(2, 4), (3, 3), (2, 8), (17, 1), (4, 8), (11, 3), (6, 8), (7, 7), (16, 8), (43, 3)])
def test_attn_rows_per_head(sage, ws, T, G, D, kf, vf, page):
    """8, 9, 16, 17, 32, 33, 48, 49, 128 and 129 rows per head: each side of every choice by rows."""
    context = [0, 47, 64, 65, 230]
    cache, table = filled(sage, [n + T for n in context], 2, page, D, kf, vf, seed=T)
    r = gen(T + page)
    mask = cu.tree_mask([[int(torch.randint(-1, i, (1,), generator=r)) if i else -1 for i in range(T)] for _ in context], DEV)
    q = rand(len(context), T, 2 * G, D, seed=T + 1)
    out, lse = run_attn(sage, ws, q, cache, table, i32(*context), None, mask)
    assert status(sage, ws) == 0
    check_attn(q, cache, table, i32(*context), None, mask, out, lse)


@pytest.mark.parametrize("T,G,D", [(1, 2, 64), (3, 4, 128), (20, 4, 128)])
def test_attn_many_sequences(sage, ws, T, G, D):
    """More sequences than a warp counts at once, some without rows, of lengths from zero on."""
    B = 75
    context = [(7 * b * b) % 91 for b in range(B)]
    count = [b % (T + 1) for b in range(B)]
    cache, table = filled(sage, [n + T for n in context], 1, 16, D, INT8, E4M3, seed=T)
    q = rand(B, T, G, D, seed=T)
    out, lse = run_attn(sage, ws, q, cache, table, i32(*context), i32(*count), None)
    assert status(sage, ws) == 0
    check_attn(q, cache, table, i32(*context), i32(*count), None, out, lse)


@pytest.mark.parametrize("T,G,D", [(64, 2, 128), (50, 1, 64)])
def test_attn_many_rows_long(sage, ws, T, G, D):
    """The variant for many rows over contexts that several CTAs share, scores that rise along the
    context (so that offsets are raised often), and V scales that grow."""
    context = [5000, 3, 1700]
    cache, table = filled(sage, [n + T for n in context], 1, 64, D, INT8, E4M3, seed=T)
    grow = torch.linspace(0.01, 6.0, 64, device=DEV)
    for b, n in enumerate(context):
        pages = table[b, :(n + T + 63) // 64].long()
        for j, pg in enumerate(pages.tolist()):
            cache[1][pg] *= float(0.05 + 3.0 * j / max(len(pages), 1))
            cache[3][pg] *= grow * 2.0 ** (j % 9 - 4)
    q = rand(3, T, G, D, seed=T) * 2
    out, lse = run_attn(sage, ws, q, cache, table, i32(*context), None, None)
    check_attn(q, cache, table, i32(*context), None, None, out, lse)
    again, lse2 = run_attn(sage, ws, q, cache, table, i32(*context), None, None)
    assert torch.equal(again, out) and torch.equal(lse2, lse) and status(sage, ws) == 0


@pytest.mark.parametrize("T,G", [(1, 4), (8, 2), (40, 4)])
def test_attn_empty_rows(sage, ws, T, G):
    """Rows whose mask leaves nothing (no context, no bits), whole empty
    batches, counts of zero, and masks with bits behind the count and T."""
    context = [0, 0, 3]
    cache, table = filled(sage, [n + T for n in context], 1, 16, 64, INT8, E4M3, seed=7)
    words = -(-T // 32)
    mask = torch.zeros(3, T, words, dtype=torch.int32, device=DEV)
    mask[1, T - 1, 0] = 1
    q = rand(3, T, G, 64, seed=8)
    ctx = i32(*context)
    out, lse = run_attn(sage, ws, q, cache, table, ctx, None, mask)
    check_attn(q, cache, table, ctx, None, mask, out, lse)
    assert (out[0] == 0).all() and torch.isinf(lse[0]).all()
    mask[:] = -1
    count = i32(0, T // 2, T)
    out, lse = run_attn(sage, ws, q, cache, table, ctx, count, mask)
    assert status(sage, ws) == 0
    check_attn(q, cache, table, ctx, count, mask, out, lse)


@pytest.mark.parametrize("T,G,D", [(1, 4, 128), (1, 8, 64), (16, 8, 128)])
def test_attn_long_ragged(sage, ws, T, G, D):
    """Contexts long enough that the work of one sequence is split."""
    context = [9000, 0, 1, 4097, 70, 2500]
    cache, table = filled(sage, [n + T for n in context], 2, 64, D, INT8, E4M3, seed=T)
    q = rand(len(context), T, 2 * G, D, seed=T) * 2
    ctx = i32(*context)
    out, lse = run_attn(sage, ws, q, cache, table, ctx, None, None)
    assert status(sage, ws) == 0
    check_attn(q, cache, table, ctx, None, None, out, lse)
    again, lse2 = run_attn(sage, ws, q, cache, table, ctx, None, None)
    assert torch.equal(again, out) and torch.equal(lse2, lse)


@pytest.mark.parametrize("T,G", [(1, 4), (12, 8)])
def test_attn_score_range(sage, ws, T, G):
    """Scores far apart (one key takes all, others underflow), large and tiny Q, V scales over many
    orders and tokens of zero V, and a scale of its own."""
    context = [700, 64, 1]
    for seed, amp, scale in ((1, 30.0, 0.0), (2, 1e-3, 0.0), (3, 1.0, 1.7), (4, 2.0 ** 60, 2.0 ** -62), (5, 2.0 ** -60, 2.0 ** 58)):
        cache, table = filled(sage, [n + T for n in context], 1, 16, 64, INT8, E4M3, seed=seed, spread=4.0)
        cache[2].view(torch.uint8)[::3, :, 5] = 0
        cache[3][::3, :, 5] = 0.0
        q = (rand(3, T, G, 64, seed=seed).float() * amp).to(torch.bfloat16)
        out, lse = run_attn(sage, ws, q, cache, table, i32(*context), None, None, scale)
        check_attn(q, cache, table, i32(*context), None, None, out, lse, scale if scale > 0 else None)
    assert status(sage, ws) == 0


def test_attn_tiny_v_scales(sage, ws):
    """V of small and large magnitudes, alone and beside each other."""
    context = [40] * 5
    cache, table = filled(sage, [n + 1 for n in context], 1, 16, 64, INT8, INT8, seed=3)
    vs = cache[3]
    for b, (lo, hi) in enumerate(((1e-18, 1e-18), (3e22, 3e22), (1e-12, 1e12), (1e-36, 1e-36), (1e34, 1e-34))):
        for s in range(41):
            vs[int(table[b, s // 16]), 0, s % 16] = lo if s % 2 else hi
    q = rand(5, 1, 4, 64, seed=4)
    out, lse = run_attn(sage, ws, q, cache, table, i32(*context), None, None)
    check_attn(q, cache, table, i32(*context), None, None, out, lse)


@pytest.mark.parametrize("T,G", [(1, 4), (20, 8)])
def test_attn_hidden_draft_of_huge_values(sage, ws, T, G):
    """A drafted token that a row does not see may hold any V: the row keeps its precision."""
    T += 1
    context = [70]
    cache, table = filled(sage, [70 + T], 1, 16, 64, INT8, E4M3, seed=31)
    big = rand(1, 1, 1, 64, seed=32) * 2.0 ** 100
    sage.sage_cache_append(cache, big, big, table, i32(70 + T - 1), None, ws)
    mask = cu.tree_mask([[i - 1 for i in range(T - 1)] + [-1]], DEV)
    q = rand(1, T, G, 64, seed=33)
    out, lse = run_attn(sage, ws, q, cache, table, i32(*context), None, mask)
    check_attn(q[:, :T - 1], cache, table, i32(*context), None, cu.tree_mask([[i - 1 for i in range(T - 1)]], DEV),
               out[:, :T - 1], lse[:, :T - 1])


@pytest.mark.parametrize("T,G", [(1, 4), (24, 8)])
def test_attn_nan_token_spoils_only_what_sees_it(sage, ws, T, G):
    context = [100, 100]
    cache, table = filled(sage, [n + T for n in context], 1, 32, 128, INT8, E4M3, seed=5)
    x = rand(1, 1, 1, 128, seed=6)
    x[..., 3] = math.nan
    parents = [[i - 1 if i != T // 2 else -1 for i in range(T)] for _ in context]
    mask = cu.tree_mask(parents, DEV)
    # a poisoned drafted token T-1 of sequence 0, and a poisoned context token of sequence 1
    sage.sage_cache_append(cache, x, x, table[:1].contiguous(), i32(100 + T - 1), None, ws)
    sage.sage_cache_append(cache, x, x, table[1:].contiguous(), i32(50), None, ws)
    q = rand(2, T, G, 128, seed=7)
    out, lse = run_attn(sage, ws, q, cache, table, i32(*context), None, mask)
    assert status(sage, ws) == 0
    assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
    assert torch.isnan(out[0, T - 1]).all()
    assert torch.isfinite(out[0, :T - 1]).all() and torch.isfinite(lse[0, :T - 1]).all()


def test_attn_bad_pages_are_left_out(sage, ws):
    """Keys on entries that name no page, or behind the table, count as unseen and are reported."""
    for T, G in ((1, 2), (20, 8)):
        cache, table = filled(sage, [200 + T], 1, 16, 64, INT8, E4M3, seed=9)
        q = rand(1, T, G, 64, seed=10)
        bad = table.clone()
        bad[0, 3], bad[0, 7] = -1, cache[0].shape[0]
        keep = [i for i in range(13) if i not in (3, 7)]
        good = torch.cat((table[:, keep], table[:, [12, 13]]), 1) if T > 8 else table[:, keep]
        sage.sage_clear_device_status(ws)
        out, lse = run_attn(sage, ws, q, cache, bad, i32(200), None, None)
        assert status(sage, ws) == sage.SAGE_ERR_DEVICE
        short = table[:, [i for i in range(table.shape[1]) if i not in (3, 7)]].contiguous()
        check_attn(q, cache, short, i32(200 - 32), None, None, out, lse)
        # a context longer than the table
        sage.sage_clear_device_status(ws)
        out, lse = run_attn(sage, ws, q, cache, table[:, :4].contiguous(), i32(200), None, None)
        assert status(sage, ws) == sage.SAGE_ERR_DEVICE
        k, v = cu.rows(cache, table, 0, torch.arange(64, device=DEV))
        s = torch.einsum("thd,jd->thj", q[0].double(), k[:, 0]) / 8
        want = torch.softmax(s, -1) @ v[:, 0]
        assert ((out[0].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -10 * v.abs().max()).all()
    # a negative context is none, a negative count no row, a count above T is T
    cache, table = filled(sage, [4], 1, 16, 64, INT8, E4M3, seed=11)
    q = rand(1, 4, 2, 64, seed=12)
    for ctx, cnt, as_ctx, as_cnt in ((-5, 4, 0, 4), (0, -1, 0, 0), (0, 9, 0, 4)):
        sage.sage_clear_device_status(ws)
        out, lse = run_attn(sage, ws, q, cache, table, i32(ctx), i32(cnt), None)
        assert status(sage, ws) == sage.SAGE_ERR_DEVICE
        check_attn(q, cache, table, i32(as_ctx), i32(as_cnt), None, out, lse)


def test_attn_strided_views_and_no_lse(sage, ws):
    cache, table = filled(sage, [60, 33], 2, 16, 128, E4M3, E4M3, seed=13)
    buf = rand(2, 3, 20 * 128, seed=14)
    q = buf[..., 4 * 128:12 * 128].unflatten(-1, (8, 128))
    big = torch.full((2, 8, 3, 128), 5.0, dtype=torch.bfloat16, device=DEV)  # head-major output
    ctx = i32(57, 30)
    sage.sage_cache_attn(q, cache, table, ctx, None, None, big.permute(0, 2, 1, 3), None, 0.0, ws)
    out, lse = run_attn(sage, ws, q, cache, table, ctx, None, None)
    assert torch.equal(big.permute(0, 2, 1, 3), out)
    check_attn(q, cache, table, ctx, None, None, out, lse)


def test_attn_shared_prefix_pages(sage, ws):
    """Two sequences whose tables name the same pages."""
    cache, table = filled(sage, [100], 1, 16, 64, INT8, INT8, seed=15)
    both = table.expand(2, -1).contiguous()
    q = rand(1, 1, 4, 64, seed=16).expand(2, 1, 4, 64)
    out, lse = run_attn(sage, ws, q, cache, both, i32(99, 99), None, None)
    assert torch.equal(out[0], out[1])
    check_attn(q, cache, both, i32(99, 99), None, None, out, lse)


@pytest.mark.parametrize("T,G", [(1, 4), (24, 8)])
def test_attn_pages_beyond_32_bit_offsets(sage, ws, T, G):
    """Rows of a pool whose codes take more than 4 GiB."""
    H, page, D, n = 8, 128, 128, 400
    pages = (1 << 32) // (H * page * D) + 64
    cache = sage.cache_buffers(pages, H, page, D, INT8, E4M3)
    used = [pages - 1, 3, pages - 2, pages // 2]
    table = i32(*used)[None]
    k, v = rand(1, n + T, H, D, seed=17), rand(1, n + T, H, D, seed=18)
    sage.sage_cache_append(cache, k, v, table, None, None, ws)
    q = rand(1, T, H * G, D, seed=19)
    out, lse = run_attn(sage, ws, q, cache, table, i32(n), None, None)
    assert status(sage, ws) == 0
    check_attn(q, cache, table, i32(n), None, None, out, lse)
    back = torch.zeros_like(k)
    sage.sage_cache_read(cache, table, None, None, back, None, ws)
    code, scale = cu.quantise(k, torch.int8)
    assert torch.equal(back, (code.float() * scale[..., None]).to(torch.bfloat16))


@pytest.mark.parametrize("T,G", [(1, 4), (16, 8)])
def test_attn_streams_and_graphs(sage, T, G):
    """Two streams at once with a workspace each, and two captured graphs that
    share one workspace, replayed in turn after lengths and values changed."""
    context = [3000, 100]
    sets = []
    for seed in (20, 30):
        cache, table = filled(sage, [n + T + 8 for n in context], 2, 64, 128, INT8, E4M3, seed=seed)
        q = rand(2, T, 2 * G, 128, seed=seed + 5)
        sets.append((q, cache, table, i32(*context)))
    torch.cuda.synchronize()
    spaces = [sage.workspace(sage.SAGE_OP_CACHE_ATTN, 1, 1, 1, 64) for _ in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    outs = [(torch.full_like(s[0], 5.0), torch.full(s[0].shape[:3], 5.0, device=DEV)) for s in sets]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, w, st, (o, l) in zip(sets, spaces, streams, outs):
            sage.sage_cache_attn(s[0], s[1], s[2], s[3], None, None, o, l, 0.0, w, stream=st)
    torch.cuda.synchronize()
    for s, (o, l) in zip(sets, outs):
        check_attn(s[0], s[1], s[2], s[3], None, None, o, l)
    w = spaces[0]
    graphs = []
    for s, (o, l) in zip(sets, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sage.sage_cache_attn(s[0], s[1], s[2], s[3], None, None, o, l, 0.0, w)
        graphs.append(g)
    for s in sets:
        s[3].copy_(i32(17, 101))
        s[0].mul_(0.5)
    for g in graphs + graphs[::-1]:
        g.replay()
    torch.cuda.synchronize()
    for s, (o, l) in zip(sets, outs):
        check_attn(s[0], s[1], s[2], s[3], None, None, o, l)
    assert sage.sage_read_device_status(w) == 0


@pytest.mark.parametrize("T,G", [(1, 4), (16, 8)])
def test_attn_withheld_tile_times_out_and_context_survives(sage, ws, T, G):
    """Producers that withhold their first tile: the bounded waits behind it run out (about 1 ms each), the
    status word says so, the kernel returns, and the next call is right."""
    context = [20000]
    cache, table = filled(sage, [20000 + T], 2, 64, 128, INT8, E4M3, seed=50)
    q = rand(1, T, 2 * G, 128, seed=51)
    try:
        sage.sage_debug_set_stall(0, 2_000_000)
        run_attn(sage, ws, q, cache, table, i32(*context), None, None)
        assert status(sage, ws) == sage.SAGE_ERR_TIMEOUT
    finally:
        sage.sage_debug_set_stall(-1, 0)
    sage.sage_clear_device_status(ws)
    out, lse = run_attn(sage, ws, q, cache, table, i32(*context), None, None)
    assert status(sage, ws) == 0
    check_attn(q, cache, table, i32(*context), None, None, out, lse)


def test_step_together(sage, ws):
    """A serving loop: prompts rotated and appended, single-token steps, then a
    drafted tree over the cache, against FP64 attention on the dequantised rows, captured as a graph."""
    B, Hq, H, D, page = 2, 8, 2, 128, 16
    prompt, N = [37, 20], 37
    f, m = sage.sage_rope_freqs(64, scaling=sage.SAGE_ROPE_YARN, factor=2.0)
    cache = empty_cache(sage, 16, H, page, D, INT8, E4M3)
    table = make_table(B, 6, 16, [90, 90], page)
    q, k, v = rand(B, N, Hq, D, seed=40), rand(B, N, H, D, seed=41), rand(B, N, H, D, seed=42)
    sage.sage_rope(q, k, q, k, None, f, m, sage.SAGE_ROPE_HALF, 64)
    sage.sage_cache_append(cache, k, v, table, None, i32(*prompt), ws)
    # the prompt's cached K through the read is the rotated K to the format's precision
    back = torch.zeros_like(k)
    sage.sage_cache_read(cache, table, None, i32(*prompt), back, None, ws)
    amax = k[1, :20].float().abs().amax(-1, keepdim=True)
    assert ((back[1, :20].float() - k[1, :20].float()).abs() <= amax / 254 * 1.01 + 2.0 ** -8 * amax).all()
    lens = i32(*prompt)
    for step in range(3):
        q1, k1, v1 = rand(B, 1, Hq, D, seed=50 + step), rand(B, 1, H, D, seed=60 + step), rand(B, 1, H, D, seed=70 + step)
        sage.sage_rope(q1, k1, q1, k1, lens[:, None], f, m, sage.SAGE_ROPE_HALF, 64)
        sage.sage_cache_append(cache, k1, v1, table, lens, None, ws)
        out, lse = run_attn(sage, ws, q1, cache, table, lens, None, None)
        check_attn(q1, cache, table, lens, None, None, out, lse)
        lens += 1
    T = 7
    parents = [[-1, 0, 0, 1, 1, 3, 2], [-1, -1, 0, 1, 2, 2, 5]]
    depth = [[0] * T for _ in range(B)]
    for b in range(B):
        for i, p in enumerate(parents[b]):
            depth[b][i] = 0 if p < 0 else depth[b][p] + 1
    mask = cu.tree_mask(parents, DEV)
    qt, kt, vt = rand(B, T, Hq, D, seed=80), rand(B, T, H, D, seed=81), rand(B, T, H, D, seed=82)
    pos = torch.empty(B, T, dtype=torch.int32, device=DEV)
    out, lse = torch.full_like(qt, 5.0), torch.full((B, T, Hq), 5.0, device=DEV)
    qr, kr = torch.empty_like(qt), torch.empty_like(kt)
    d = torch.tensor(depth, dtype=torch.int32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        torch.add(lens[:, None], d, out=pos)
        sage.sage_rope(qt, kt, qr, kr, pos, f, m, sage.SAGE_ROPE_HALF, 64)
        sage.sage_cache_append(cache, kr, vt, table, lens, None, ws)
        sage.sage_cache_attn(qr, cache, table, lens, None, mask, out, lse, 0.0, ws)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        check_attn(qr, cache, table, lens, None, mask, out, lse)
        qt.copy_(rand(B, T, Hq, D, seed=90))
        lens += 2
    assert status(sage, ws) == 0


def test_read_feeds_the_full_attention(sage, ws):
    """A cached context read back and attended to by sage_attn_fwd is the same
    as sage_attn_fwd on the dequantised tensors."""
    n, H, D = 150, 2, 128
    cache, table = filled(sage, [n], H, 32, D, INT8, E4M3, seed=43)
    k, v = (torch.zeros(1, n, H, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    sage.sage_cache_read(cache, table, None, None, k, v, ws)
    q = rand(1, n, H, D, seed=44)
    kd, vd = cu.rows(cache, table, 0, torch.arange(n, device=DEV))
    want = sage.attention(q, kd.float().to(torch.bfloat16)[None], vd.float().to(torch.bfloat16)[None])
    got = sage.attention(q, k, v)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_binding_refusals(sage, ws):
    cache, table = filled(sage, [20], 2, 16, 64, INT8, E4M3, seed=45)
    q, x, c = rand(1, 1, 4, 64), rand(1, 1, 2, 64), i32(19)
    out, lse = torch.empty_like(q), torch.empty(1, 1, 4, device=DEV)
    bad = [lambda: sage.sage_cache_attn(q, cache, table.long(), c, None, None, out, lse, 0.0, ws),
           lambda: sage.sage_cache_attn(q, cache, table, None, None, None, out, lse, 0.0, ws),
           lambda: sage.sage_cache_attn(q, cache, table, c.long(), None, None, out, lse, 0.0, ws),
           lambda: sage.sage_cache_attn(q, cache, table, c, None, torch.zeros(1, 1, 2, dtype=torch.int32, device=DEV), out, lse, 0.0, ws),
           lambda: sage.sage_cache_attn(q, cache, table, c, None, None, out, lse.double(), 0.0, ws),
           lambda: sage.sage_cache_attn(q[:, :, :3], cache, table, c, None, None, out[:, :, :3], None, 0.0, ws),
           lambda: sage.sage_cache_attn(q, (cache[0].view(torch.uint8),) + cache[1:], table, c, None, None, out, lse, 0.0, ws),
           lambda: sage.sage_cache_attn(q, (cache[0], cache[1].half()) + cache[2:], table, c, None, None, out, lse, 0.0, ws),
           lambda: sage.sage_cache_append(cache, x.float(), x, table, c, None, ws),
           lambda: sage.sage_cache_append(cache, q, q, table, c, None, ws),
           lambda: sage.sage_cache_append(cache, x, x, table.expand(2, -1), c, None, ws),
           lambda: sage.sage_cache_read(cache, table, c, None, None, None, ws),
           lambda: sage.sage_cache_read(cache, table, c, None, q, None, ws)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(sage.SageError):
        sage.sage_cache_attn(q, cache, table, c, None, None, out, lse, 0.0, ws[:512])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,G", [(1, 4), (2, 8), (24, 8)])
@pytest.mark.parametrize("power", [4, 20, 28, 32, 36, 44, 60, 100])
def test_attn_scores_of_any_size(sage, ws, power, T, G, D):
    """Scores of +-D^0.5 2^power: two equal keys of the largest score share the row, however large it is.  The others are
    at most half of it, below by 2^power D^0.5 / 2 >= 64, and leave nothing (e^-64).  w has 2^-11, exp2 and the sums 2^-19,
    the result 2^-8; lse the score's (D + 4) 2^-24, relative here since every product has the sign of the sum."""
    B, H, page, ctx = 2, 2, 32, 1500
    n = ctx + T
    per = -(-n // page)
    cache = empty_cache(sage, B * per, H, page, D, INT8, E4M3)
    table = make_table(B, per, B * per, [n] * B, page, seed=power)
    rng = gen(power + T)
    u = torch.where(torch.rand(D, generator=rng) < 0.5, -1.0, 1.0).to(DEV)
    r = (torch.rand(B, n, H, generator=rng) * 1.5 - 1.0).to(DEV)  # below 0.5
    top = [[5, ctx - 3], [40, 777]]
    for b in range(B):
        r[b, top[b]] = 1.0
    a = power // 2
    k = (r[..., None] * u * 2.0 ** (power - a)).bfloat16()
    v = rand(B, n, H, D, seed=power)
    q = (u * 2.0 ** a).bfloat16().expand(B, T, H * G, D).contiguous()
    sage.sage_cache_append(cache, k, v, table, None, None, ws)
    out = torch.empty_like(q)
    lse = torch.empty(B, T, H * G, device=DEV)
    sage.sage_cache_attn(q, cache, table, i32(*[ctx] * B), None, None, out, lse, 0.0, ws)
    assert status(sage, ws) == sage.SAGE_OK
    for b in range(B):
        kk, vv = cu.rows(cache, table, b, torch.tensor(top[b], device=DEV))
        want = vv.mean(0).repeat_interleave(G, 0).expand(T, H * G, D)
        spread = vv.abs().mean(0).repeat_interleave(G, 0).expand(T, H * G, D)
        err = (out[b].double() - want).abs()
        assert (err <= spread * (2.0 ** -11 + 2.0 ** -18) + 2.0 ** -8 * want.abs()).all(), float(err.max())
        s = (q[b, 0, ::G].double() * kk[0]).sum(-1) * D ** -0.5 + math.log(2.0)
        got = lse[b].double().view(T, H, G)
        assert ((got - s[None, :, None]).abs() <= s.abs()[None, :, None] * (D + 8) * 2.0 ** -24).all()


@pytest.mark.parametrize("T,G,D", [(1, 4, 128), (1, 8, 64), (2, 8, 64), (4, 4, 128), (40, 4, 128), (33, 2, 64)])
@pytest.mark.parametrize("n", [300, 2100, 20011])
def test_attn_one_head_cut_into_many_parts(sage, ws, T, G, D, n):
    """One sequence and one head: every CTA has a part of the same unit, or of the same few."""
    cache, table = filled(sage, [n + T], 1, 16, D, INT8, E4M3, seed=n + T)
    q = rand(1, T, G, D, seed=n)
    out, lse = run_attn(sage, ws, q, cache, table, i32(n), None, None)
    assert status(sage, ws) == sage.SAGE_OK
    check_attn(q, cache, table, i32(n), None, None, out, lse)
