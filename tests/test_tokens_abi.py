"""Refusals of the token operators that need no GPU: the C ABI checks its
arguments on the host before any HIP call, the binding before the library."""
import ctypes

import pytest
import torch

import depth_weighted_scatter_amd as dws
from depth_weighted_scatter_amd import tokens

F32, F16, E4M3, BF16 = dws.F32, dws.F16, dws.FP8_E4M3, dws.BF16
FAKE = 1 << 40          # never dereferenced: validation fails first
INVALID, UNSUPPORTED, OVERFLOW, WORKSPACE = -1, -2, -3, -4

# Fake device pointers: where a GPU is visible a gap in the host checks would
# launch a kernel on them, so these run only where none is.
no_gpu_only = pytest.mark.skipif(torch.cuda.is_available(), reason="fake device pointers")


@pytest.fixture(scope="module")
def lib():
    return tokens._lib()


def sections(*v):
    return (ctypes.c_int32 * max(len(v), 1))(*v)


ROPE = dict(qw=FAKE, kw=FAKE, wdt=BF16, eps=1e-6, pos=FAKE, axes=3, sec=sections(16, 24, 24),
            freq=FAKE, layout=0)
PAGED = dict(kc=FAKE, vc=FAKE, cdt=BF16, ks=1.0, vs=1.0, pages=10, page=16)
BATCH = dict(off=FAKE, len=FAKE, seqs=3, table=FAKE, width=4)


def rope_call(lib, **kw):
    a = dict(q=FAKE, qs=1024, k=FAKE, ks_=256, dt=BF16, n=10, hq=8, hk=2, d=128, **ROPE, qo=FAKE,
             qos=1024, ko=FAKE, kos=256, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.bevpool_qk_norm_rope(*a.values())


def grad_call(lib, **kw):
    a = dict(dqo=FAKE, dqos=1024, dko=FAKE, dkos=256, q=FAKE, qs=1024, k=FAKE, ks_=256, dt=BF16,
             n=10, hq=8, hk=2, d=128, **ROPE, dq=FAKE, dqs=1024, dk=FAKE, dks=256, dqw=FAKE,
             dkw=FAKE, ws=FAKE, wsb=1 << 30, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.bevpool_qk_norm_rope_backward(*a.values())


def append_call(lib, **kw):
    a = dict(q=FAKE, qs=1024, k=FAKE, ks_=256, v=FAKE, vs_=256, dt=BF16, n=10, hq=8, hk=2, d=128,
             **ROPE, qo=FAKE, qos=1024, **PAGED, **BATCH, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.bevpool_kv_append(*a.values())


def attend_call(lib, **kw):
    a = dict(q=FAKE, qs=1024, dt=BF16, n=10, hq=8, hk=2, d=128, **PAGED, **BATCH, scale=0.1,
             causal=1, window=0, out=FAKE, os=1024, ws=FAKE, wsb=1 << 40, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.bevpool_paged_attention(*a.values())


ROPE_BAD = [
    (dict(d=0), INVALID), (dict(n=-1), INVALID), (dict(hk=-1), INVALID),
    (dict(d=120), UNSUPPORTED), (dict(d=272), UNSUPPORTED),
    (dict(wdt=F16), UNSUPPORTED), (dict(wdt=E4M3), UNSUPPORTED),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(axes=5), INVALID), (dict(axes=-1), INVALID), (dict(sec=None), INVALID),
    (dict(sec=sections(16, -8, 24)), INVALID),
    (dict(sec=sections(16, 24, 25)), UNSUPPORTED),        # more than head_dim turns
    (dict(sec=sections(16, 24, 20)), UNSUPPORTED),        # R not a multiple of 16
    (dict(sec=sections(2 ** 31 - 1, 2 ** 31 - 1, 2)), UNSUPPORTED),
    (dict(pos=None), INVALID), (dict(freq=None), INVALID), (dict(freq=FAKE + 2), INVALID),
    (dict(layout=2), INVALID), (dict(layout=-1), INVALID),
    (dict(qw=FAKE + 1), INVALID),
    (dict(n=2 ** 31), OVERFLOW), (dict(n=2 ** 28), OVERFLOW), (dict(n=2 ** 62), OVERFLOW),
]
SIDES_BAD = [
    (dict(hq=0), INVALID), (dict(dt=E4M3), UNSUPPORTED), (dict(dt=9), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(q=FAKE + 8), INVALID), (dict(qs=1016), INVALID),
    (dict(qs=1025), INVALID), (dict(k=None), INVALID), (dict(ks_=248), INVALID),
    (dict(qs=2 ** 31 + 8), OVERFLOW),
]


@no_gpu_only
@pytest.mark.parametrize("kw,code", ROPE_BAD + SIDES_BAD + [
    (dict(qo=None), INVALID), (dict(ko=None), INVALID), (dict(qos=1000), INVALID),
    (dict(ko=FAKE + 4), INVALID)])
def test_norm_rope_rejects(lib, kw, code):
    assert rope_call(lib, **kw) == code


@no_gpu_only
@pytest.mark.parametrize("kw,code", ROPE_BAD + SIDES_BAD + [
    (dict(dqo=None), INVALID), (dict(dko=None), INVALID), (dict(dq=None), INVALID),
    (dict(dk=FAKE + 2), INVALID), (dict(dqw=None), INVALID), (dict(dkw=FAKE + 2), INVALID),
    (dict(ws=None), INVALID), (dict(ws=FAKE + 128), WORKSPACE), (dict(wsb=100), WORKSPACE)])
def test_norm_rope_backward_rejects(lib, kw, code):
    assert grad_call(lib, **kw) == code


PAGED_BAD = [
    (dict(dt=F32), UNSUPPORTED), (dict(cdt=F16), UNSUPPORTED), (dict(cdt=F32), UNSUPPORTED),
    (dict(page=8), UNSUPPORTED), (dict(page=512), UNSUPPORTED), (dict(page=48), UNSUPPORTED),
    (dict(page=0), UNSUPPORTED), (dict(hk=0), INVALID), (dict(seqs=-1), INVALID),
    (dict(width=-1), INVALID), (dict(pages=0), INVALID), (dict(pages=-4), INVALID),
    (dict(pages=2 ** 31), OVERFLOW), (dict(pages=2 ** 27), OVERFLOW), (dict(width=2 ** 27), OVERFLOW),
    (dict(seqs=2 ** 24 + 1), OVERFLOW), (dict(seqs=2 ** 20, width=2 ** 12), OVERFLOW),
    (dict(kc=None), INVALID), (dict(vc=FAKE + 8), INVALID), (dict(off=None), INVALID),
    (dict(len=None), INVALID), (dict(table=None), INVALID), (dict(table=FAKE + 2), INVALID),
    (dict(cdt=E4M3, ks=0.0), INVALID), (dict(cdt=E4M3, vs=-1.0), INVALID),
    (dict(cdt=E4M3, ks=float("nan")), INVALID), (dict(cdt=E4M3, vs=1e30), INVALID),
    (dict(n=2 ** 31), OVERFLOW), (dict(n=2 ** 29, hq=2), OVERFLOW),
    (dict(d=24), UNSUPPORTED), (dict(n=-1), INVALID),
]


@no_gpu_only
@pytest.mark.parametrize("kw,code", [b for b in ROPE_BAD if "hk" not in b[0]] + PAGED_BAD + [
    (dict(q=None), INVALID), (dict(qo=None), INVALID), (dict(qos=1016), INVALID),
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(vs_=255), INVALID),
    (dict(k=FAKE + 8), INVALID)])
def test_append_rejects(lib, kw, code):
    assert append_call(lib, **kw) == code


@no_gpu_only
@pytest.mark.parametrize("kw,code", PAGED_BAD + [
    (dict(hq=0), INVALID), (dict(hq=9), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=-1.0), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(cdt=E4M3, ks=2.0 ** 60, scale=2.0 ** 100), INVALID),
    (dict(scale=1e-38), INVALID), (dict(scale=2.0 ** -97), INVALID), (dict(scale=2.0 ** 97), INVALID),
    (dict(cdt=E4M3, ks=2.0 ** -60, scale=2.0 ** -40), INVALID),
    (dict(window=-1), INVALID), (dict(causal=2), INVALID), (dict(q=None), INVALID),
    (dict(out=None), INVALID), (dict(out=FAKE + 4), INVALID), (dict(os=1000), INVALID),
    (dict(ws=None), INVALID), (dict(ws=FAKE + 64), WORKSPACE), (dict(wsb=0), WORKSPACE)])
def test_attention_rejects(lib, kw, code):
    assert attend_call(lib, **kw) == code


def test_nothing_to_do(lib):
    """No tokens, or no sequences: OK without touching the GPU."""
    assert rope_call(lib, n=0, q=None, qo=None, k=None, ko=None) == 0
    assert append_call(lib, n=0, k=None, v=None, kc=None) == 0
    assert append_call(lib, seqs=0, off=None) == 0
    assert attend_call(lib, n=0, q=None, ws=None) == 0
    assert attend_call(lib, seqs=0, out=None) == 0


def test_workspace_sizes(lib):
    size = dws.bevpool_qk_norm_rope_backward_workspace_size
    assert size(0, 1, 0, 16) > 0 and size(10 ** 6, 16, 4, 128) > 0
    for bad in ((-1, 1, 0, 16), (1, 0, 0, 16), (1, 1, 0, 24), (1, 1, -1, 16), (2 ** 31, 1, 0, 16)):
        assert size(*bad) == 0
    size = dws.bevpool_paged_attention_workspace_size
    assert size(0, 0, 1, 1, 16, 16, 0) > 0 and size(64, 64, 32, 8, 128, 16, 513) > 0
    for bad in ((-1, 1, 8, 2, 64, 16, 4), (1, -1, 8, 2, 64, 16, 4), (1, 1, 8, 3, 64, 16, 4),
                (1, 1, 8, 0, 64, 16, 4), (1, 1, 8, 2, 65, 16, 4), (1, 1, 8, 2, 64, 17, 4),
                (1, 1, 8, 2, 64, 16, -1), (1, 1, 8, 2, 64, 16, 2 ** 28),
                (1, 2 ** 24 + 1, 8, 2, 64, 16, 4)):
        assert size(*bad) == 0, bad


def test_attention_launch_fits(lib):
    """Blocks of 512 threads, 2^32 threads a launch: up to 2^23 - 1 blocks."""
    size = dws.bevpool_paged_attention_workspace_size
    assert size(2, 2 ** 22 - 1, 2, 2, 16, 16, 1) > 0 and size(2, 2 ** 22, 2, 2, 16, 16, 1) == 0
    assert attend_call(lib, seqs=2 ** 22, hq=2, hk=2) == OVERFLOW
    assert size(2 ** 27, 1, 8, 1, 16, 16, 1) == 0            # 2^30 rows: 2^23 tiles
    assert size(2 ** 27 - 256, 1, 8, 1, 16, 16, 1) > 0


def test_binding_wants_gpu_tensors():
    q = torch.zeros(4, 2, 64)
    with pytest.raises(TypeError):
        dws.bevpool_qk_norm_rope(q, None, None, None)
    with pytest.raises(TypeError):
        dws.bevpool_kv_append(q, q, None, None, None, None)
    with pytest.raises(TypeError):
        dws.bevpool_paged_attention(q, None, None)
    with pytest.raises(TypeError):
        dws.bevpool_qk_norm_rope_backward(q, None, None, None, None, None)
    with pytest.raises(TypeError):
        dws.PagedCache(q, q)
    with pytest.raises(TypeError):
        dws.PagedBatch(q, q, q)
    with pytest.raises(TypeError):
        dws.Rope(torch.ones(8), (8,))


def test_rope_refusals():
    assert dws.Rope(None).sections == ()
    with pytest.raises(ValueError):
        dws.Rope(None, (1, 2, 3, 4, 5))
    with pytest.raises(ValueError):
        dws.Rope(None, (-8,))
    with pytest.raises(ValueError):
        dws.Rope(None, (), 3)
    with pytest.raises(ValueError):
        dws.Rope(torch.ones(8))


def test_header_limits():
    import os
    import re
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                        "bevpool.h")
    with open(path) as f:
        text = f.read()
    for name, want in (("MAX_HEAD_DIM", dws.MAX_HEAD_DIM), ("MAX_ROPE_AXES", dws.MAX_ROPE_AXES)):
        assert int(re.search(rf"#define BEVPOOL_{name} (\d+)", text).group(1)) == want
