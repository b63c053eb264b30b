"""Host-side checks of the rotary positions and of the paged cache that need
no GPU: frequencies, workspace sizes, refusals of bad arguments before the
device is touched, and the binding's own checks."""
import ctypes
import math

import numpy as np
import pytest

import cache_util as cu
import fp8_quantized_exact_b200 as sage

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    from fp8_quantized_exact_b200 import build
    build.build()
    return sage.lib()


@pytest.mark.parametrize("rot", [2, 6, 32, 64, 96, 128])
@pytest.mark.parametrize("scaling,factor", [(0, 1.0), (1, 1.0), (1, 4.0), (2, 2.0), (3, 1.0), (3, 8.5), (3, 40.0)])
def test_rope_frequencies(lib, rot, scaling, factor):
    if scaling == 2 and rot == 2:
        with pytest.raises(sage.SageError):
            sage.sage_rope_freqs(rot, scaling=scaling, factor=factor, device="cpu")
        return
    for base in (10000.0, 500000.0):
        f, m = sage.sage_rope_freqs(rot, base, scaling, factor, device="cpu")
        want, wm = cu.frequencies(rot, base, scaling, factor)
        # pow's last bits, and (1 - r) + r / factor against f / factor r + f (1 - r)
        np.testing.assert_allclose(f.numpy(), want, rtol=1e-13, atol=0)
        assert m == np.float32(wm)


def test_rope_frequencies_refusals(lib):
    out, m = (ctypes.c_double * 64)(), ctypes.c_float()
    addr = ctypes.addressof(out)

    def call(rot=64, scaling=3, base=1e4, factor=2.0, trained=4096.0, fast=32.0, slow=1.0, to=addr):
        c = sage.sage_rope_config(scaling, rot, base, factor, trained, fast, slow)
        return lib.sage_rope_freqs(ctypes.byref(c), to, ctypes.byref(m))
    assert call() == sage.SAGE_OK
    for rot in (0, 1, 63, 130, -2):
        assert call(rot=rot) == sage.SAGE_ERR_UNSUPPORTED
    for bad in (dict(scaling=4), dict(scaling=-1), dict(base=1.0), dict(base=math.nan), dict(base=math.inf),
                dict(factor=0.5), dict(factor=math.nan), dict(factor=math.inf), dict(trained=0.0), dict(fast=1.0),
                dict(slow=0.0), dict(fast=math.nan), dict(to=None)):
        assert call(**bad) == sage.SAGE_ERR_INVALID_ARG, bad
    assert call(scaling=0, factor=0.5) == sage.SAGE_OK  # unused


def test_workspace(lib):
    n = sage.sage_workspace_bytes
    assert n(sage.SAGE_OP_CACHE, 3, 5, 2, 64) >= sage.SAGE_STATUS_BYTES
    one = n(sage.SAGE_OP_CACHE_ATTN, 1, 1, 1, 64)
    assert one == n(sage.SAGE_OP_CACHE_ATTN, 64, 256, 56, 128) and one <= 64 << 20
    assert one >= n(sage.SAGE_OP_CACHE, 64, 256, 56, 128)


NULL = sage.sage_view_bf16(None, 0, 0, 0)
GOOD = sage.sage_view_bf16(4096, 1024, 256, 128)
ODD = sage.sage_view_bf16(4098, 1024, 256, 128)
STRIDE = sage.sage_view_bf16(4096, 1024, 252, 128)
NEG = sage.sage_view_bf16(4096, -1024, 256, 128)


def test_rope_refusals(lib):
    def call(q=GOOD, Hq=2, qo=4096, k=GOOD, Hk=2, ko=4096, pos=4096, ps=4, f=4096, m=1.0, layout=0, rot=64, B=1, N=4,
             D=128, so=128):
        return lib.sage_rope(q, Hq, qo, 1024, 256, so, k, Hk, ko, 1024, 256, 128, pos, ps, f, m, layout, rot, 0, B, N, D,
                             None)
    I, U = sage.SAGE_ERR_INVALID_ARG, sage.SAGE_ERR_UNSUPPORTED
    for bad, code in ((dict(q=NULL), I), (dict(q=NEG), I), (dict(q=ODD), U), (dict(k=STRIDE), U), (dict(qo=None), I),
                      (dict(ko=None), I), (dict(ko=4098), U), (dict(so=-8), I), (dict(so=4), U), (dict(f=None), I),
                      (dict(f=4100), U), (dict(pos=4097), U), (dict(ps=-1), I), (dict(m=math.nan), I),
                      (dict(m=math.inf), I), (dict(layout=2), I), (dict(rot=0), U), (dict(rot=63), U),
                      (dict(rot=130), U), (dict(D=96), U), (dict(Hq=-1), I), (dict(B=-1), I), (dict(Hk=70000), U),
                      (dict(B=65535, N=1 << 20), U)):
        assert call(**bad) == code, bad
    assert call(B=0) == call(N=0) == call(Hq=0, Hk=0) == sage.SAGE_OK


def cache_struct(**kw):
    c = sage.sage_cache(4096, 4096, 4096, 4096, 0, 1, 10, 16, 2, 128)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


CACHE_BAD = [(dict(k_codes=None), 1), (dict(v_scale=None), 1), (dict(k_codes=4100), 2), (dict(k_scale=4100), 2),
             (dict(k_format=2), 1), (dict(v_format=-1), 1), (dict(page_size=24), 2), (dict(page_size=256), 2),
             (dict(page_size=8), 2), (dict(D=96), 2), (dict(pages=-1), 1), (dict(pages=0), 1), (dict(H=-1), 1),
             (dict(pages=1 << 20, H=2, page_size=128), 0), (dict(pages=1 << 23, H=2, page_size=128), 2)]


def test_append_and_read_refusals(lib):
    def append(c=None, k=GOOD, v=GOOD, table=4096, per=4, start=4096, count=4096, B=1, N=4, ws=4096, n=1024):
        return lib.sage_cache_append(ctypes.addressof(c or cache_struct()), k, v, table, per, start, count, B, N, ws, n, None)

    def read(c=None, table=4096, per=4, start=4096, count=4096, ko=4096, vo=4096, so=128, B=1, N=4, ws=4096, n=1024):
        return lib.sage_cache_read(ctypes.addressof(c or cache_struct()), table, per, start, count, ko, 1024, 256, so, vo,
                                   1024, 256, 128, B, N, ws, n, None)
    for call in (append, read):
        for bad, code in CACHE_BAD:
            if code:
                assert call(c=cache_struct(**bad)) == code, bad
        for bad, code in ((dict(table=None), 1), (dict(per=0), 1), (dict(per=(1 << 24) + 1), 2), (dict(table=4098), 2), (dict(start=4098), 2),
                          (dict(count=4098), 2), (dict(ws=None), 3), (dict(ws=4112), 3), (dict(n=100), 3),
                          (dict(B=-1), 1), (dict(N=-1), 1), (dict(B=70000), 2)):
            assert call(**bad) == code, bad
        assert call(B=0) == call(N=0) == call(c=cache_struct(H=0)) == sage.SAGE_OK
        # a token grid beyond the launch extents
        assert call(c=cache_struct(H=65535, pages=1), N=1 << 28) == 2
    for bad, code in ((dict(k=NULL), 1), (dict(v=ODD), 2), (dict(k=STRIDE), 2)):
        assert append(**bad) == code
    for bad, code in ((dict(ko=None, vo=None), 1), (dict(ko=4098), 2), (dict(vo=4098), 2), (dict(so=4), 2)):
        assert read(**bad) == code
    assert lib.sage_cache_append(None, GOOD, GOOD, 4096, 4, None, None, 1, 4, 4096, 1024, None) == 1


def test_attention_refusals(lib):
    need = sage.sage_workspace_bytes(sage.SAGE_OP_CACHE_ATTN, 1, 1, 1, 128)

    def call(q=GOOD, c=None, table=4096, per=4, ctx=4096, count=None, mask=None, out=4096, so=128, lse=None, B=1, T=4, Hq=4,
             ws=4096, n=need):
        return lib.sage_cache_attn(q, ctypes.addressof(c or cache_struct()), table, per, ctx, count, mask, out, 1024, 256, so,
                                   lse, B, T, Hq, 0.0, ws, n, None)
    for bad, code in CACHE_BAD:
        if code:
            assert call(c=cache_struct(**bad)) == code, bad
    for bad, code in ((dict(q=NULL), 1), (dict(q=ODD), 2), (dict(q=STRIDE), 2), (dict(table=None), 1), (dict(per=0), 1),
                      (dict(per=(1 << 24) + 1), 2), (dict(ctx=None), 1), (dict(ctx=4098), 2), (dict(count=4098), 2), (dict(mask=4098), 2),
                      (dict(lse=4098), 2), (dict(out=None), 1), (dict(out=4104), 2), (dict(so=-8), 1), (dict(Hq=3), 1),
                      (dict(Hq=-2), 1), (dict(T=257), 2), (dict(T=-1), 1), (dict(ws=None), 3), (dict(ws=4112), 3),
                      (dict(n=need - 1), 3), (dict(B=70000), 2), (dict(c=cache_struct(H=0)), 1)):
        assert call(**bad) == code, bad
    assert call(B=0) == call(T=0) == call(Hq=0) == sage.SAGE_OK


def test_clear_status_refusal(lib):
    assert lib.sage_clear_device_status(None, None) == sage.SAGE_ERR_INVALID_ARG


def test_binding_refuses_host_tensors_and_wrong_shapes(lib):
    c = sage.cache_buffers(4, 2, 16, 64, device="cpu")
    assert [t.dtype for t in c] == [torch.int8, torch.float32, torch.float8_e4m3fn, torch.float32]
    x = torch.zeros(1, 3, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, 4, dtype=torch.int32)
    ws = torch.zeros(1024, dtype=torch.uint8)
    with pytest.raises(ValueError):
        sage.sage_cache_append(c, x, x, i, None, None, ws)
    with pytest.raises(ValueError):
        sage.sage_cache_read(c, i, None, None, x, x, ws)
    with pytest.raises(ValueError):
        sage.sage_cache_attn(x, c, i, i[:, 0], None, None, x, None, 0.0, ws)
    with pytest.raises(ValueError):
        sage.sage_rope(x, None, x, None, None, torch.zeros(32, dtype=torch.float64))
