"""The serving calls where their inputs change under way: lengths written right in front of a call, forks of streams, and
the append's largest values."""
import pytest

import cache_util as cu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

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


def problem(sage, B, T, G, H, D, n, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    page = 64
    per = -(-(n + T) // page)
    cache = sage.cache_buffers(B * per, H, page, D)
    table = torch.randperm(B * per, device=DEV, generator=g).to(torch.int32).view(B, per).contiguous()
    ws = sage.workspace(sage.SAGE_OP_CACHE_ATTN, 1, 1, 1, D)
    x = torch.randn(2, B, n + T, H, D, device=DEV, generator=g).bfloat16()
    sage.sage_cache_append(cache, x[0], x[1], table, None, None, ws)
    q = torch.randn(B, T, H * G, D, device=DEV, generator=g).bfloat16()
    return cache, table, ws, q


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("B,T,G,H,D", [(1, 1, 4, 8, 128), (3, 2, 8, 2, 64), (40, 1, 7, 2, 128), (5, 16, 8, 2, 128), (2, 64, 1, 1, 64)])
def test_lengths_written_right_in_front_of_each_call(sage, B, T, G, H, D, captured):
    """Calls whose lengths, and with them which units are cut and into how many parts, jump from one to the next, written by
    the kernel in front: the bits of calls on an idle device."""
    n, calls = 6000, 24
    cache, table, ws, q = problem(sage, B, T, G, H, D, n, seed=B + T)
    g = torch.Generator("cuda").manual_seed(7)
    lengths = torch.randint(0, n + 1, (calls, B), device=DEV, generator=g, dtype=torch.int32)
    lengths[::3] //= 50
    counts = torch.randint(0, T + 1, (calls, B), device=DEV, generator=g, dtype=torch.int32)
    ctx, cnt = torch.zeros(B, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
    out = torch.full((2, calls) + tuple(q.shape), 5.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((2, calls, B, T, H * G), 5.0, device=DEV)

    def call(k, i):
        torch.add(lengths[i], 0, out=ctx)
        torch.add(counts[i], 0, out=cnt)
        sage.sage_cache_attn(q, cache, table, ctx, cnt, None, out[k, i], lse[k, i], 0.0, ws)

    for i in range(calls):
        call(0, i)
        torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for i in range(calls):
                call(1, i)
        graph.replay()
    else:
        for i in range(calls):
            call(1, i)
    torch.cuda.synchronize()
    assert sage.sage_read_device_status(ws) == sage.SAGE_OK
    assert torch.equal(out[0].view(torch.int16), out[1].view(torch.int16)) and torch.equal(lse[0], lse[1])
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("power", [104, 111, 115, 119, 120])
def test_append_ties_of_the_largest_values(sage, fmt, power):
    """All half-way cases (BF16 values of twelve binades against every 8-bit maximum) where the quotient's second term is
    subnormal: the codes are those of the exact quotient."""
    D, dt = 128, (torch.int8, torch.float8_e4m3fn)[fmt]
    mant = torch.arange(128, 256, dtype=torch.float64)
    rows = []
    for e in range(12):
        body = (mant[None, 1:] * 2.0 ** -e).expand(128, 127).clone()
        body[body > mant[:, None]] = 1.0
        rows.append(torch.cat((mant[:, None], body * torch.where(torch.arange(127) % 2 == 0, 1.0, -1.0)), 1))
    x = (torch.cat(rows) * 2.0 ** power).to(torch.bfloat16)[None, :, None].to(DEV)
    assert torch.isfinite(x).all()
    n = x.shape[1]
    ws = sage.workspace(sage.SAGE_OP_CACHE, 1, 1, 1, D)
    cache = sage.cache_buffers(-(-n // 64), 1, 64, D, fmt, fmt)
    table = torch.arange(-(-n // 64), dtype=torch.int32, device=DEV)[None]
    sage.sage_cache_append(cache, x, x, table, None, None, ws)
    torch.cuda.synchronize()
    assert sage.sage_read_device_status(ws) == sage.SAGE_OK
    code, scale = cu.quantise(x[0, :, 0], dt)
    assert torch.equal(cache[0].double().permute(0, 2, 1, 3).reshape(-1, D)[:n], code)
    assert torch.equal(cache[1].permute(0, 2, 1).reshape(-1)[:n], scale)


@pytest.mark.parametrize("B,T,G,H,D", [(1, 1, 4, 8, 128), (3, 21, 4, 2, 64)])
def test_calls_behind_an_eager_fork_of_streams(sage, B, T, G, H, D):
    """A loop whose append runs on a second stream, forked from and joined to the first by events, while the first stream
    rotates Q: the bits of the same loop on an idle device."""
    n, steps = 1500, 16
    results = []
    for idle in (True, False):
        cache, table, ws, q = problem(sage, B, T, G, H, D, n + steps * T, seed=3)
        ws2 = sage.workspace(sage.SAGE_OP_CACHE, 1, 1, 1, D)
        f, m = sage.sage_rope_freqs(D)
        ctx = torch.full((B,), n, dtype=torch.int32, device=DEV)
        out, k = torch.empty_like(q), torch.empty(B, T, H, D, dtype=torch.bfloat16, device=DEV)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        wait = torch.cuda.synchronize if idle else (lambda: None)
        for _ in range(steps):
            k.copy_(q[:, :, ::G])
            wait()
            side.wait_stream(torch.cuda.current_stream())
            sage.sage_cache_append(cache, k, k, table, ctx, None, ws2, stream=side)
            wait()
            sage.sage_rope(q, None, q, None, None, f, m)
            wait()
            torch.cuda.current_stream().wait_stream(side)
            sage.sage_cache_attn(q, cache, table, ctx, None, None, out, None, 0.0, ws)
            wait()
            q.copy_(out).mul_(8.0)
            ctx.add_(T)
            wait()
        torch.cuda.synchronize()
        assert sage.sage_read_device_status(ws) == sage.sage_read_device_status(ws2) == sage.SAGE_OK
        back = torch.empty(B, n + steps * T, H, D, dtype=torch.bfloat16, device=DEV)  # the slots that were written
        sage.sage_cache_read(cache, table, None, None, back, None, ws)
        results.append((q, back))
    assert all(torch.isfinite(t).all() for t in results[0])
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_a_sequence_without_rows_does_not_slow_the_others(sage):
    """A long context that has no drafted token in this call takes no part in how the others are cut."""
    B, T, G, D, n = 9, 64, 2, 128, 4096
    cache, table, ws, q = problem(sage, B, T, G, 1, D, 150000 // 32, seed=5)
    table = torch.cat((table, torch.full((B, 150000 // 64), -1, dtype=torch.int32, device=DEV)), 1).contiguous()
    count = torch.tensor([0] + [T] * (B - 1), dtype=torch.int32, device=DEV)
    out = torch.empty_like(q)
    times = {}
    for first in (0, 150000, 0, 150000):
        ctx = torch.tensor([first] + [n] * (B - 1), dtype=torch.int32, device=DEV)
        for _ in range(3):
            sage.sage_cache_attn(q, cache, table, ctx, count, None, out, None, 0.0, ws)
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(50):
            sage.sage_cache_attn(q, cache, table, ctx, count, None, out, None, 0.0, ws)
        b.record()
        torch.cuda.synchronize()
        times[first] = min(times.get(first, 1e9), a.elapsed_time(b) / 50)
    assert sage.sage_read_device_status(ws) == sage.SAGE_OK
    assert times[150000] <= 1.5 * times[0], times
