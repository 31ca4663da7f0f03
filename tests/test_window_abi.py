"""Refusals of the window entry points, answered on the host before any
launch."""
import ctypes

import pytest

from paged_kv_cache_481_b200 import binding, build

OK, INVALID, UNSUPPORTED, WORKSPACE = (binding.PA_OK, binding.PA_ERR_INVALID_ARG,
                                       binding.PA_ERR_UNSUPPORTED, binding.PA_ERR_WORKSPACE)
NULL = ctypes.c_void_p(None)
P = ctypes.c_void_p(0x10000)        # never dereferenced: every call here is refused
ODD = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def _rope(lib, eight=False, **change):
    a = dict(q_out=P, qo=256, q=P, qs=256, k=P, ks=128, v=P, vs=128, kc=P, vc=P, scales=P, table=P,
             rotary=64, maxp=10, inter=0, pos=P, slots=P, n=1, h=4, kvh=2, d=64, bs=16, nb=4,
             dtype=0, kind=0, stream=NULL)
    a.update(change)
    if not eight:
        del a["scales"], a["kind"]
    f = lib.pa_rope_and_cache_q8 if eight else lib.pa_rope_and_cache
    return f(*a.values())


@pytest.mark.parametrize("eight", [False, True])
def test_rope_refuses(lib, eight):
    r = lambda **c: _rope(lib, eight, **c)
    assert r(n=0, q=NULL) == OK
    for c in (dict(n=-1), dict(nb=0), dict(maxp=-1), dict(dtype=2), dict(dtype=-1), dict(h=3),
              dict(kvh=0), dict(h=0), dict(h=512, kvh=2), dict(q=NULL), dict(q_out=NULL),
              dict(k=NULL), dict(v=NULL), dict(kc=NULL), dict(vc=NULL), dict(slots=NULL),
              dict(table=NULL), dict(pos=NULL), dict(maxp=0), dict(q=ODD), dict(kc=ODD), dict(table=ODD),
              dict(qs=248), dict(ks=120), dict(vs=0), dict(qo=260), dict(ks=-128),
              dict(qs=264)):           # q in place with another stride
        assert r(**c) == INVALID, c
    for c in (dict(d=96), dict(bs=24), dict(rotary=24), dict(rotary=80), dict(rotary=-16)):
        assert r(**c) == UNSUPPORTED, c
    if eight:
        for c in (dict(kind=2), dict(scales=NULL), dict(scales=ODD)):
            assert r(**c) == INVALID, c


def _decode(lib, eight=False, **change):
    a = dict(out=P, q=P, k=P, v=P, scales=P, tables=P, mb=4, lens=P, maxlen=64, window=16, sinks=0,
             b=1, h=4, kvh=2, d=64, bs=16, nb=4, dtype=0, kind=0, scale=1.0, ws=P, wsb=1 << 30,
             stream=NULL)
    a.update(change)
    if not eight:
        del a["scales"], a["kind"]
    return (lib.pa_decode_q8 if eight else lib.pa_decode_window)(*a.values())


@pytest.mark.parametrize("eight", [False, True])
def test_decode_refuses(lib, eight):
    r = lambda **c: _decode(lib, eight, **c)
    assert r(b=0, q=NULL) == OK
    for c in (dict(b=-1), dict(b=70000), dict(nb=0), dict(maxlen=-1), dict(mb=-1), dict(window=0),
              dict(window=-3), dict(sinks=-1), dict(dtype=2), dict(h=5), dict(h=512, kvh=2),
              dict(scale=float("nan")), dict(scale=float("inf")), dict(maxlen=65),
              dict(maxlen=2 ** 30 + 1, mb=2 ** 30), dict(out=NULL), dict(q=NULL), dict(k=NULL),
              dict(v=NULL), dict(tables=NULL), dict(lens=NULL), dict(out=ODD), dict(v=ODD),
              dict(ws=ODD), dict(tables=ctypes.c_void_p(0x10002))):
        assert r(**c) == INVALID, c
    for c in (dict(d=96), dict(bs=12), dict(d=256)):
        assert r(**c) == UNSUPPORTED, c
    need = lib.pa_decode_window_workspace_size(1, 4, 2, 64)
    for c in (dict(ws=NULL), dict(wsb=0), dict(wsb=need - 1)):
        assert r(**c) == WORKSPACE, c
    if eight:
        for c in (dict(kind=2), dict(kind=-1), dict(scales=NULL), dict(scales=ODD)):
            assert r(**c) == INVALID, c


def test_workspace_size(lib):
    size = binding.pa_decode_window_workspace_size
    assert size(0, 1, 1, 64) > 0 and size(-1, 3, 2, 0) > 0
    # one size for every head_dim, so that calls may share a workspace
    assert size(8, 32, 8, 64) == size(8, 32, 8, 128)
    # a counter per (sequence, K/V head, 16 query heads)
    assert size(1000, 32, 1, 64) - size(0, 1, 1, 64) >= 2 * 1000 * 4 - 256


def _prefill(lib, **change):
    a = dict(out=P, q=P, k=P, v=P, tables=P, mb=4, lens=P, maxlen=64, starts=P, n=8, maxnew=8,
             window=16, sinks=0, b=1, h=4, kvh=2, d=64, bs=16, nb=4, dtype=0, scale=1.0, stream=NULL)
    a.update(change)
    return lib.pa_prefill_window(*a.values())


def test_prefill_refuses(lib):
    r = lambda **c: _prefill(lib, **c)
    for c in (dict(b=0), dict(n=0), dict(maxnew=0)):
        assert r(q=NULL, **c) == OK
    for c in (dict(b=-1), dict(b=70000), dict(n=-1), dict(maxnew=-1), dict(nb=0), dict(maxlen=-1),
              dict(mb=-1), dict(window=0), dict(sinks=-1), dict(dtype=2), dict(h=5),
              dict(h=512, kvh=2), dict(scale=float("nan")), dict(scale=0.0), dict(scale=-1.0),
              dict(maxlen=65), dict(maxnew=65), dict(maxlen=2 ** 30 + 1, mb=2 ** 30),
              dict(nb=2 ** 30), dict(out=NULL), dict(q=NULL), dict(k=NULL), dict(v=NULL),
              dict(tables=NULL), dict(lens=NULL), dict(starts=NULL), dict(out=ODD), dict(q=ODD),
              dict(k=ODD), dict(starts=ctypes.c_void_p(0x10002))):
        assert r(**c) == INVALID, c
    for c in (dict(d=96), dict(bs=12), dict(d=256)):
        assert r(**c) == UNSUPPORTED, c
