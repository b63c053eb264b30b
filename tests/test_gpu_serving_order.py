"""Order among the serving calls, whose kernels start before the ones in front of them have drained: chains in
which every call reads what the call before wrote give the same bits as with the device idle between calls,
eager, captured, with foreign kernels, copies and memsets in between, and behind a fork and join of streams."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sage():
    import fp8_quantized_exact_b200 as s
    from fp8_quantized_exact_b200 import build
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    return s


class Loop:
    """Steps that feed on one another: the output of a step is the next one's Q, K and V."""

    def __init__(self, sage, B, T, G, H, D, page, context):
        g = torch.Generator("cuda").manual_seed(B * 1000 + T * 100 + D)
        self.sage, self.T, self.H, self.G = sage, T, H, G
        per = (context + 64 * T) // page + 1
        self.cache = sage.cache_buffers(B * per, H, page, D)
        for i, t in enumerate(self.cache):
            t.view(torch.uint8).zero_() if i % 2 == 0 else t.zero_()
        self.table = torch.randperm(B * per, device="cuda", generator=g).to(torch.int32).view(B, per).contiguous()
        self.ws = sage.workspace(sage.SAGE_OP_CACHE_ATTN, 1, 1, 1, D)
        first = torch.randn(2, B, context, H, D, device="cuda", generator=g).bfloat16()
        sage.sage_cache_append(self.cache, first[0], first[1], self.table, None, None, self.ws)
        self.context = torch.full((B,), context, dtype=torch.int32, device="cuda")
        self.positions = (context + torch.arange(T, dtype=torch.int32, device="cuda")).repeat(B, 1).contiguous()
        self.freq, self.mscale = sage.sage_rope_freqs(D)
        self.q = torch.randn(B, T, H * G, D, device="cuda", generator=g).bfloat16()
        self.out = torch.empty_like(self.q)
        self.k = torch.empty(B, T, H, D, device="cuda", dtype=torch.bfloat16)
        self.v = torch.empty_like(self.k)
        self.back = torch.zeros(2, B, T, H, D, device="cuda", dtype=torch.bfloat16)

    def step(self, between):
        s = self.sage
        self.k.copy_(self.q[:, :, :: self.G])
        self.v.copy_(self.q[:, :, self.G - 1 :: self.G])
        between()
        s.sage_rope(self.q, self.k, self.q, self.k, self.positions, self.freq, self.mscale)
        between()
        s.sage_cache_append(self.cache, self.k, self.v, self.table, self.context, None, self.ws)
        between()
        s.sage_cache_attn(self.q, self.cache, self.table, self.context, None, None, self.out, None, 0.0, self.ws)
        between()
        # the next call reads the output of this one at once, and writes what this one read
        s.sage_rope(self.out, self.k, self.q, self.k, self.positions, self.freq, self.mscale, inverse=True)
        between()
        s.sage_cache_read(self.cache, self.table, self.context, None, self.back[0], self.back[1], self.ws)
        between()
        s.sage_cache_attn(self.q, self.cache, self.table, self.context, None, None, self.out, None, 0.0, self.ws)
        s.sage_cache_attn(self.out, self.cache, self.table, self.context, None, None, self.q, None, 0.0, self.ws)
        between()
        self.q.mul_(8.0).add_(self.back[1].repeat_interleave(self.G, dim=2))
        self.context.add_(self.T)
        self.positions.add_(self.T)

    def state(self):
        torch.cuda.synchronize()
        assert self.sage.sage_read_device_status(self.ws) == self.sage.SAGE_OK
        return [t.clone() for t in (self.q, self.out, self.k, self.back, self.cache[1], self.cache[3],
                                    self.cache[0].view(torch.uint8), self.cache[2].view(torch.uint8))]


SHAPES = [(1, 1, 4, 8, 128, 64, 1000), (3, 1, 1, 2, 64, 16, 333), (5, 9, 2, 3, 64, 32, 700), (4, 21, 4, 4, 128, 128, 900),
          (64, 1, 7, 2, 128, 64, 200)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("how", ["eager", "copies", "graph", "fork"])
def test_chained_calls_keep_their_order(sage, shape, how):
    steps = 12
    ref = Loop(sage, *shape)
    torch.cuda.synchronize()
    for _ in range(steps):
        ref.step(torch.cuda.synchronize)
    want = ref.state()
    assert all(torch.isfinite(t).all() for t in want[:4])
    got = Loop(sage, *shape)
    torch.cuda.synchronize()
    noise = torch.zeros(1 << 16, device="cuda")
    host = torch.zeros(4, pin_memory=True)
    side = torch.cuda.Stream()

    def copies():
        noise.zero_()
        noise[:4].copy_(host, non_blocking=True)

    def fork():
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            noise.add_(1.0)
        noise.view(torch.uint8)[1 << 17 :].zero_()
        torch.cuda.current_stream().wait_stream(side)

    between = {"eager": lambda: None, "graph": lambda: None, "copies": copies, "fork": fork}[how]
    if how in ("eager", "copies"):
        for _ in range(steps):
            got.step(between)
    else:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.step(between)
        for _ in range(steps):
            graph.replay()
    for a, b in zip(got.state(), want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_first_call_of_a_process_may_be_captured(sage, tmp_path):
    """No call has loaded a kernel before: capture sets the attributes and loads them."""
    import os
    import subprocess
    import sys
    src = tmp_path / "first.py"
    src.write_text(
        "import sys, torch\n"
        f"sys.path.insert(0, {os.path.dirname(os.path.dirname(os.path.abspath(sage.__file__)))!r})\n"
        "import fp8_quantized_exact_b200 as s\n"
        "c = s.cache_buffers(4, 2, 16, 64)\n"
        "ws = s.workspace(s.SAGE_OP_CACHE_ATTN, 1, 1, 1, 64)\n"
        "x = torch.ones(1, 1, 2, 64, device='cuda', dtype=torch.bfloat16)\n"
        "q = torch.ones(1, 1, 4, 64, device='cuda', dtype=torch.bfloat16)\n"
        "out = torch.zeros_like(q)\n"
        "table = torch.tensor([[2, 1]], dtype=torch.int32, device='cuda')\n"
        "ctx = torch.zeros(1, dtype=torch.int32, device='cuda')\n"
        "f, m = s.sage_rope_freqs(64)\n"
        "torch.cuda.synchronize()\n"
        "g = torch.cuda.CUDAGraph()\n"
        "with torch.cuda.graph(g):\n"
        "    s.sage_rope(q, x, q, x, None, f, m)\n"
        "    s.sage_cache_append(c, x, x, table, ctx, None, ws)\n"
        "    s.sage_cache_attn(q, c, table, ctx, None, None, out, None, 0.0, ws)\n"
        "g.replay()\n"
        "torch.cuda.synchronize()\n"
        "assert (out == 1).all() and s.sage_read_device_status(ws) == 0\n")
    subprocess.run([sys.executable, str(src)], check=True, timeout=300)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("N,H,D", [(150, 2, 128), (700, 4, 64), (2000, 3, 128)])
def test_chain_with_the_full_attention(sage, N, H, D, captured):
    """Cache and rotary calls between full attentions, whose own kernels start early too: each reads what the one in
    front wrote, and the rotary call and the read write what it has just read."""
    g = torch.Generator("cuda").manual_seed(N)
    first = torch.randn(3, 1, N, H, D, device="cuda", generator=g).bfloat16()
    pages = -(-N // 32)
    table = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)[None].contiguous()
    freq, mscale = sage.sage_rope_freqs(D)
    ws = sage.workspace(sage.SAGE_OP_CACHE, 1, 1, 1, D)
    full_ws = sage.workspace(sage.SAGE_OP_ATTN_FWD, 1, N, H, D)

    def chain(between, x, cache, out):
        q, k, v = x
        sage.sage_rope(q, k, q, k, None, freq, mscale)
        between()
        sage.sage_cache_append(cache, k, v, table, None, None, ws)
        between()
        sage.sage_cache_read(cache, table, None, None, k, v, ws)
        between()
        sage.sage_attn_fwd(q, k, v, out, 0.0, full_ws)
        between()
        sage.sage_rope(out, k, q, k, None, freq, mscale, inverse=True)
        between()
        sage.sage_attn_fwd(q, k, v, out, 0.0, full_ws)
        between()
        sage.sage_cache_append(cache, out, k, table, None, None, ws)
        between()
        sage.sage_cache_read(cache, table, None, None, v, q, ws)
        between()

    results = []
    for sync in (True, False):
        x, out = [t.clone() for t in first], torch.empty_like(first[0])
        cache = sage.cache_buffers(pages, H, 32, D)
        between = torch.cuda.synchronize if sync else lambda: None
        torch.cuda.synchronize()
        if captured and not sync:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                chain(between, x, cache, out)
            for _ in range(8):
                graph.replay()
        else:
            for _ in range(8):
                chain(between, x, cache, out)
        torch.cuda.synchronize()
        assert sage.sage_read_device_status(ws) == sage.SAGE_OK
        results.append([t.clone() for t in (*x, out)])
    assert all(torch.isfinite(t).all() for t in results[0])
    assert all(torch.equal(a, b) for a, b in zip(*results))
