"""Refusals of the rotary and 8-bit cache entry points on the CPU: bad
arguments are rejected on the host before anything touches CUDA."""

import ctypes
import math
import os

import pytest
import torch

P = ctypes.c_void_p
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 4


@pytest.fixture(scope="module")
def lib():
    from head_scaled_dot_gb300 import mha
    if not os.path.exists(mha.LIB_PATH):
        from head_scaled_dot_gb300 import build
        build.build()
    return mha.load()


def _sections(*v):
    return (ctypes.c_int32 * len(v))(*v)


def _steps(lib, sections, base=10000.0, per_axis=0, n=None):
    out = (ctypes.c_uint64 * 256)()
    st = lib.mha_rotary_steps(_sections(*sections), len(sections) if n is None else n, base,
                              per_axis, out)
    return st, list(out[:sum(max(0, s) for s in sections)])


def test_rotary_steps_are_the_fractions_of_a_turn(lib):
    for sections, per_axis in [((64,), 0), ((16, 24, 24), 0), ((16, 24, 24), 1), ((0, 3), 1)]:
        st, got = _steps(lib, sections, 10000.0, per_axis)
        assert st == OK
        pairs = sum(sections)
        w = [10000.0 ** -(j / m) for m in sections for j in range(m)] if per_axis else \
            [10000.0 ** -(i / pairs) for i in range(pairs)]
        for s, x in zip(got, w):
            # double precision: a few units of 2^-53 of the value
            assert abs(s / 2.0 ** 64 - x / (2 * math.pi)) <= 8 * 2.0 ** -53 * x


def test_rotary_steps_refusals(lib):
    assert _steps(lib, (4,), base=0.0)[0] == INVALID
    assert _steps(lib, (4,), base=math.inf)[0] == INVALID
    assert _steps(lib, (4,), base=math.nan)[0] == INVALID
    assert _steps(lib, (4, -1))[0] == INVALID
    assert _steps(lib, (0, 0))[0] == INVALID
    assert _steps(lib, (1, 1, 1, 1, 1))[0] == UNSUPPORTED
    assert _steps(lib, (100, 29))[0] == UNSUPPORTED
    assert lib.mha_rotary_steps(None, 1, 10.0, 0, (ctypes.c_uint64 * 4)()) == INVALID
    assert lib.mha_rotary_steps(_sections(4), 1, 10.0, 0, None) == INVALID


def _rotary(lib, **kw):
    a = dict(Q=4096, K=8192, pos=12288, steps=16384, sections=(16, 16), Qo=4096, Ko=8192, B=2,
             T=3, h=4, h_kv=2, d=64, inter=0, inv=0, dt=1)
    a.update(kw)
    return lib.mha_rotary(P(a["Q"]), P(a["K"]), P(a["pos"]), P(a["steps"]),
                          _sections(*a["sections"]) if a["sections"] else None,
                          a.get("axes", len(a["sections"] or ())), P(a["Qo"]), P(a["Ko"]),
                          a["B"], a["T"], a["h"], a["h_kv"], a["d"], a["inter"], a["inv"],
                          a["dt"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(Q=None), INVALID), (dict(Qo=None), INVALID), (dict(pos=None), INVALID),
    (dict(steps=None), INVALID), (dict(sections=None, axes=2), INVALID),
    (dict(K=None), INVALID), (dict(Ko=None), INVALID),
    (dict(B=0), INVALID), (dict(T=-1), INVALID), (dict(h=0), INVALID), (dict(h_kv=0), INVALID),
    (dict(d=0), INVALID), (dict(dt=2), INVALID), (dict(axes=0), INVALID),
    (dict(sections=(16, 17)), INVALID), (dict(sections=(-1, 2)), INVALID),
    (dict(sections=(0, 0)), INVALID),
    (dict(sections=(1, 1, 1, 1, 1)), UNSUPPORTED), (dict(d=65), UNSUPPORTED),
    (dict(d=258), UNSUPPORTED), (dict(h=60000, h_kv=6000), UNSUPPORTED),
    (dict(Q=4104), UNSUPPORTED), (dict(Ko=8200), UNSUPPORTED),
])
def test_rotary_refusals(lib, kw, code):
    assert _rotary(lib, **kw) == code


def _reserve(lib, release=False, **kw):
    a = dict(cached=4096, new=8192, free=12288, n_free=16384, table=20480, slots=24576,
             total=28672, n_out=32768, B=4, n=5, n_blocks=100, max_blocks=10, bt=16)
    a.update(kw)
    head = [P(a["cached"]), P(a["new"]), P(a["free"]), P(a["n_free"]), P(a["table"])]
    if release:
        return lib.mha_cache_release(*head, P(a["total"]), P(a["n_out"]), a["B"], a["n_blocks"],
                                     a["max_blocks"], a["bt"], None, None)
    return lib.mha_cache_reserve(*head, P(a["slots"]), P(a["total"]), P(a["n_out"]), a["B"],
                                 a["n"], a["n_blocks"], a["max_blocks"], a["bt"], None, None)


@pytest.mark.parametrize("release", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(cached=None), INVALID), (dict(new=None), INVALID), (dict(free=None), INVALID),
    (dict(n_free=None), INVALID), (dict(table=None), INVALID), (dict(total=None), INVALID),
    (dict(n_out=None), INVALID), (dict(B=0), INVALID), (dict(n_blocks=0), INVALID),
    (dict(max_blocks=-1), INVALID), (dict(bt=0), INVALID),
    (dict(n_out=16384), INVALID), (dict(total=4096), INVALID), (dict(total=8192), INVALID),
    (dict(B=1025), UNSUPPORTED), (dict(bt=1025), UNSUPPORTED),
    (dict(max_blocks=1 << 28, bt=16), UNSUPPORTED),
    (dict(max_blocks=1 << 22, bt=16, B=1024), UNSUPPORTED),
])
def test_pool_refusals(lib, release, kw, code):
    assert _reserve(lib, release, **kw) == code


def test_reserve_needs_slots(lib):
    assert _reserve(lib, slots=None) == INVALID
    assert _reserve(lib, n=0) == INVALID


def _append(lib, **kw):
    a = dict(K=4096, V=8192, slots=12288, Kc=16384, Vc=20480, Ks=24576, Vs=28672, B=2, n=3, h=4,
             d_h=64, d_vh=128, n_blocks=10, bt=16, dt=1)
    a.update(kw)
    return lib.mha_cache_append(*[P(a[k]) for k in ("K", "V", "slots", "Kc", "Vc", "Ks", "Vs")],
                                *[a[k] for k in ("B", "n", "h", "d_h", "d_vh", "n_blocks", "bt",
                                                 "dt")], None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(K=None), INVALID), (dict(V=None), INVALID), (dict(slots=None), INVALID),
    (dict(Kc=None), INVALID), (dict(Vc=None), INVALID), (dict(Ks=None), INVALID),
    (dict(Vs=None), INVALID), (dict(B=0), INVALID), (dict(n=0), INVALID), (dict(h=-1), INVALID),
    (dict(d_h=0), INVALID), (dict(n_blocks=0), INVALID), (dict(bt=0), INVALID),
    (dict(dt=7), INVALID), (dict(d_h=72), UNSUPPORTED), (dict(d_vh=272), UNSUPPORTED),
    (dict(bt=24), UNSUPPORTED), (dict(bt=1040), UNSUPPORTED), (dict(B=32768), UNSUPPORTED),
    (dict(K=4104), UNSUPPORTED), (dict(Vc=20481), UNSUPPORTED),
    (dict(n=(1 << 31) - 100), UNSUPPORTED),
])
def test_append_refusals(lib, kw, code):
    assert _append(lib, **kw) == code


def _attend(lib, **kw):
    a = dict(Q=4096, Kc=8192, Vc=12288, Ks=16384, Vs=20480, table=24576, total=28672, new=32768,
             Z=36864, B=2, n_q=3, h=8, h_kv=2, d_h=64, d_vh=128, n_blocks=10, max_blocks=5, bt=16,
             c=0.125, tail=1, dt=1, ws=1 << 20, ws_bytes=1 << 30)
    a.update(kw)
    return lib.mha_attention_cache(
        *[P(a[k]) for k in ("Q", "Kc", "Vc", "Ks", "Vs", "table", "total", "new", "Z")],
        *[a[k] for k in ("B", "n_q", "h", "h_kv", "d_h", "d_vh", "n_blocks", "max_blocks", "bt",
                         "c", "tail", "dt")], P(a["ws"]), a["ws_bytes"], None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(Q=None), INVALID), (dict(Kc=None), INVALID), (dict(Vc=None), INVALID),
    (dict(Ks=None), INVALID), (dict(Vs=None), INVALID), (dict(table=None), INVALID),
    (dict(total=None), INVALID), (dict(Z=None), INVALID), (dict(B=0), INVALID),
    (dict(n_q=0), INVALID), (dict(h=0), INVALID), (dict(h_kv=0), INVALID),
    (dict(h_kv=3), INVALID), (dict(d_h=0), INVALID), (dict(d_vh=-16), INVALID),
    (dict(n_blocks=0), INVALID), (dict(max_blocks=0), INVALID), (dict(bt=-16), INVALID),
    (dict(c=math.nan), INVALID), (dict(c=math.inf), INVALID), (dict(dt=2), INVALID),
    (dict(d_h=24), UNSUPPORTED), (dict(d_vh=272), UNSUPPORTED), (dict(bt=8), UNSUPPORTED),
    (dict(bt=2048), UNSUPPORTED), (dict(B=1025), UNSUPPORTED),
    (dict(max_blocks=1 << 28), UNSUPPORTED), (dict(B=1000, max_blocks=1 << 22), UNSUPPORTED),
    (dict(B=1, h=1, h_kv=1, max_blocks=1, n_q=(1 << 31) - 100), UNSUPPORTED),
    (dict(n_q=1 << 28), UNSUPPORTED), (dict(Q=4104), UNSUPPORTED), (dict(Z=36872), UNSUPPORTED),
    (dict(ws=None), WORKSPACE), (dict(ws=(1 << 20) + 16), WORKSPACE), (dict(ws_bytes=4096), WORKSPACE),
])
def test_attention_refusals(lib, kw, code):
    assert _attend(lib, **kw) == code


def test_attention_workspace_size(lib):
    from head_scaled_dot_gb300 import mha
    size = mha.attention_cache_workspace_size
    assert size(0, 1, 8, 8, 64, 64) == 0 and size(1, 1, 8, 3, 64, 64) == 0
    assert size(1, 1, 8, 8, 128, 128) == size(1000, 1, 8, 8, 128, 128) > 0
    # at most 256 rows share a summary slot: more need no more
    assert size(1, 4, 32, 8, 128, 128) < size(1, 64, 32, 8, 128, 128) == size(1, 4000, 32, 8, 128, 128)


def test_binding_refuses_cpu_tensors_and_wrong_types(lib):
    from head_scaled_dot_gb300 import mha
    Q = torch.zeros((1, 2, 1, 64), dtype=torch.bfloat16)
    steps = torch.zeros(32, dtype=torch.int64)
    pos = torch.zeros((1, 1, 1), dtype=torch.int32)
    with pytest.raises(ValueError):
        mha.rotary(Q, None, pos, steps, [32])
    with pytest.raises(ValueError):
        mha.rotary(Q.half(), None, pos, steps, [32])
    with pytest.raises(ValueError):
        mha.rotary(Q.transpose(1, 3), None, pos, steps, [32])
    for dtype, shape in [(torch.float32, Q.shape), (torch.bfloat16, (1, 2, 1, 32)),
                         (torch.bfloat16, Q.shape)]:  # the last is on the CPU
        with pytest.raises(ValueError):
            mha._cuda("x", Q, dtype, shape, 0)
    with pytest.raises(ValueError):
        mha._cache_type(Q)
