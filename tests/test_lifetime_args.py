"""Host-side checks of the cache-lifetime operators (no GPU): refusals at the
C ABI before any CUDA call, RotaryAxes, workspace sizes, and the references
the GPU tests use."""
import ctypes

import numpy as np
import pytest

import lifetime_ref as ref
from paged_kv_cache_48_gb300 import RotaryAxes, _native, build

ARG, SHAPE, WORKSPACE = 1, 3, 7


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _native.lib()


def _cache(**kw):
    c = _native.PkvCache(4096, 8192, 4, 16, 2, 128, 0, 1.0, 1.0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _rope_call(lib, q=1 << 20, qs=256, k=1 << 21, ks=256, v=1 << 22, vs=256, pos=16, axs=10,
               slots=16, T=10, heads=2, rope=None, cache=None, out=1 << 23, os=256):
    rope = rope if rope is not None else RotaryAxes(128, [64]).c_struct()
    return lib.paged_kv_rope_write(q, qs, k, ks, v, vs, pos, axs, slots, T, heads,
                                   ctypes.byref(rope) if rope else None,
                                   ctypes.byref(cache if cache is not None else _cache()), out,
                                   os, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rope=False), ARG),
    (dict(T=-1), ARG),
    (dict(heads=-1), ARG),
    (dict(heads=65536, qs=1 << 24, os=1 << 24), ARG),
    (dict(k=None), ARG),
    (dict(v=None), ARG),
    (dict(q=None), ARG),
    (dict(out=None), ARG),
    (dict(pos=None), ARG),
    (dict(slots=None), ARG),
    (dict(k=(1 << 21) + 8), ARG),          # not 16-byte aligned
    (dict(out=(1 << 23) + 2), ARG),
    (dict(ks=248), ARG),                   # shorter than a row
    (dict(qs=260), ARG),                   # not a multiple of 8
    (dict(os=248), ARG),
    (dict(axs=-1), ARG),
    (dict(T=1 << 31), ARG),
    (dict(ks=1 << 31), ARG),
    (dict(out=(1 << 20) + 16), ARG),       # q_out shifted over q
    (dict(out=1 << 20, os=512), ARG),      # q_out over q with another stride
    (dict(out=1 << 21), ARG),              # q_out over k
    (dict(out=(1 << 22) + 512 * 4), ARG),  # q_out over v's later rows
    (dict(cache=_cache(head_dim=96)), SHAPE),
    (dict(cache=_cache(dtype=1, k_scale=0.0)), ARG),
    (dict(T=0), 0),
    (dict(T=0, q=None, k=None, v=None), 0),
])
def test_rope_write_refusals(lib, kw, status):
    assert _rope_call(lib, **kw) == status


def test_rope_descriptor_refusals(lib):
    def call(**kw):
        r = RotaryAxes(64, [32])
        s = r.c_struct()
        for k, v in kw.items():
            setattr(s, k, v)
        return _rope_call(lib, rope=s)
    for R in (0, 8, 24, 136, 144, -16):
        assert call(rotary_dim=R) == SHAPE, R
    assert _rope_call(lib, rope=RotaryAxes(128, [64]).c_struct(),
                      cache=_cache(head_dim=64)) == SHAPE  # past head_dim
    assert call(num_axes=0) == SHAPE and call(num_axes=5) == SHAPE
    assert call(frequencies=None) == ARG and call(axis=None) == ARG
    for f in (np.nan, np.inf, 1025.0):
        r = RotaryAxes(16, [8], frequencies=[f] * 8)
        assert _rope_call(lib, rope=r.c_struct()) == ARG
    r = RotaryAxes(16, [4, 4])
    r.axis[3] = 2  # an axis past num_axes
    assert _rope_call(lib, rope=r.c_struct()) == ARG


def test_rotary_axes():
    r = RotaryAxes(128, [16, 24, 24], base=1e6)
    assert r.axis.tolist() == [0] * 16 + [1] * 24 + [2] * 24
    assert np.allclose(r.frequencies, 1e6 ** (-np.arange(64) / 64.0), rtol=1e-15)
    r = RotaryAxes(128, [24, 20, 20], interleave_axes=True)
    assert r.axis[:60].tolist() == [0, 1, 2] * 20 and r.axis[60:].tolist() == [0] * 4
    assert RotaryAxes(32, [8, 8]).num_axes == 2
    for bad in (dict(rotary_dim=24, sections=[12]), dict(rotary_dim=8, sections=[4]),
                dict(rotary_dim=144, sections=[72]), dict(rotary_dim=32, sections=[8]),
                dict(rotary_dim=32, sections=[]), dict(rotary_dim=32, sections=[17, -1]),
                dict(rotary_dim=32, sections=[4, 3, 3, 3, 3]),
                dict(rotary_dim=32, sections=[4, 12], interleave_axes=True),
                dict(rotary_dim=32, sections=[16], frequencies=[1.0] * 15)):
        with pytest.raises(ValueError):
            RotaryAxes(**bad)


def _weights_call(lib, batch=2, heads=4, weights=1 << 20, stride=128, decay=1.0, k=None, v=None,
                  nsl=None, n_new=0, max_len=128, pt=0, ws=None, ws_bytes=0, cache=None, q=16):
    c = cache if cache is not None else _cache()
    return lib.paged_attention_decode_weights(q, k, v, nsl, n_new, ctypes.byref(c), 16, 8, 16,
                                              batch, heads, 0.1, 16, weights, stride, decay,
                                              max_len, pt, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(weights=None), ARG),
    (dict(weights=(1 << 20) + 2), ARG),
    (dict(stride=127), ARG),
    (dict(decay=float("nan")), ARG),
    (dict(decay=float("inf")), ARG),
    (dict(k=16), ARG),                      # k_new without v_new
    (dict(k=16, v=16, n_new=3), ARG),       # one row per sequence
    (dict(k=24, v=16, n_new=2), ARG),
    (dict(nsl=16, n_new=-1), ARG),
    (dict(heads=3), SHAPE),
    (dict(pt=24), ARG),
    (dict(batch=65536), ARG),
    (dict(batch=-1), ARG),
    (dict(), WORKSPACE),
    (dict(ws=1 << 20, ws_bytes=64), WORKSPACE),
    (dict(ws=(1 << 20) + 16, ws_bytes=1 << 30), WORKSPACE),
    (dict(q=24), ARG),
    (dict(batch=0), 0),
    (dict(batch=0, weights=None), 0),
    (dict(cache=_cache(dtype=7)), 2),
])
def test_decode_weights_refusals(lib, kw, status):
    assert _weights_call(lib, **kw) == status


def test_workspace_sizes(lib):
    f = lib.paged_attention_decode_weights_workspace_bytes
    # short sequences: no partials, but statistics and scores
    assert f(4, 8, 8, 64, 64, 0) >= 4 * 8 * (8 + 4 * 64)
    # groups of 5 keep 6 scores a token; 12 keep 2 sub-groups of 8
    assert f(2, 40, 8, 128, 160, 160) >= 2 * 8 * 160 * 6 * 4
    assert f(2, 24, 2, 128, 160, 160) >= 2 * 2 * 2 * 160 * 8 * 4
    # past 32-bit byte counts
    assert f(128, 64, 8, 128, 131072, 0) > 128 * 64 * 131072 * 4 > 1 << 31
    assert f(0, 8, 8, 64, 64, 0) == 0 and f(4, 7, 2, 64, 64, 0) == 0
    e = lib.paged_kv_evict_workspace_bytes
    assert e(4, 8, 1000, 100) >= 4 * 8 * 100 * 4 + 4 * 8
    assert e(0, 8, 1000, 100) == 0 and e(4, 8, 1000, -1) == 0


def _evict_call(lib, cache=None, max_blocks=8, lens=1 << 16, w=1 << 20, stride=128, keep=1 << 17,
                batch=2, max_keep=32, sink=1, recent=2, dst=None, dmb=0, dw=None, dstride=0,
                new=1 << 18, kept=None, ws=1 << 24, ws_bytes=1 << 20, tables=1 << 19):
    c = cache if cache is not None else _cache()
    return lib.paged_kv_evict(ctypes.byref(c), tables, max_blocks, lens, w, stride, keep, batch,
                              max_keep, sink, recent, 1, dst, dmb, dw, dstride, new, kept, ws,
                              ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(tables=None), ARG),
    (dict(lens=None), ARG),
    (dict(w=None), ARG),
    (dict(keep=None), ARG),
    (dict(new=None), ARG),
    (dict(batch=-1), ARG),
    (dict(batch=65536), ARG),
    (dict(max_keep=-1), ARG),
    (dict(sink=-1), ARG),
    (dict(recent=-1), ARG),
    (dict(stride=-1), ARG),
    (dict(stride=1 << 31), ARG),
    (dict(max_keep=(1 << 30) + 1), ARG),
    (dict(max_blocks=0), ARG),
    (dict(dst=1 << 21, dmb=0), ARG),
    (dict(dw=(1 << 20) + 64, dstride=64), ARG),   # over the weights still to be read
    (dict(new=(1 << 16) + 4), ARG),               # shifted over seq_lens
    (dict(new=1 << 17), ARG),                     # over keep
    (dict(ws=None), WORKSPACE),
    (dict(ws=(1 << 24) + 16), WORKSPACE),
    (dict(ws_bytes=100), WORKSPACE),
    (dict(cache=_cache(block_size=8)), SHAPE),
    (dict(batch=0), 0),
])
def test_evict_refusals(lib, kw, status):
    assert _evict_call(lib, **kw) == status


def test_reference_rotation_turns_and_keeps_lengths():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 3, 64))
    r = RotaryAxes(32, [10, 6], interleave_pairs=True)
    pos = rng.integers(-1000, 1000, (2, 5))
    y, _ = ref.rotate(x, pos, r.frequencies, r.axis, 32, True)
    assert np.allclose(np.linalg.norm(x, axis=-1), np.linalg.norm(y, axis=-1))
    assert np.array_equal(x[:, :, 32:], y[:, :, 32:])
    back, _ = ref.rotate(y, -pos, r.frequencies, r.axis, 32, True)
    assert np.allclose(back, x)
    # a quarter turn per position: (x, y) -> (-y, x)
    q = RotaryAxes(16, [8], frequencies=[np.pi / 2] * 8)
    z, _ = ref.rotate(x[:, :, :16], np.ones((1, 5), int), q.frequencies, q.axis, 16, False)
    assert np.allclose(z[:, :, :8], -x[:, :, 8:16]) and np.allclose(z[:, :, 8:], x[:, :, :8])


def test_reference_eviction_order():
    nan, inf = float("nan"), float("inf")
    w = np.array([0, 5, 1, 5, nan, -inf, inf, 0.0, -0.0, 2], dtype=np.float32)
    assert ref.evict_choice(w, 10, 3, 0, 0) == [1, 3, 6]
    assert ref.evict_choice(w, 10, 2, 0, 0) == [1, 6]          # ties: the lower position
    assert ref.evict_choice(w, 10, 4, 1, 2) == [0, 6, 8, 9]
    assert ref.evict_choice(w, 10, 9, 0, 0) == [0, 1, 2, 3, 5, 6, 7, 8, 9]  # NaN goes first
    assert ref.evict_choice(w, 10, 6, 0, 0) == [0, 1, 2, 3, 6, 9]  # -0 ties with 0
    assert ref.evict_choice(w, 10, 2, 5, 5) == [8, 9]          # recent before sink
    assert ref.evict_choice(w, 10, 0, 5, 5) == []
    assert ref.evict_choice(w, 3, 7, 1, 1) == [0, 1, 2]
