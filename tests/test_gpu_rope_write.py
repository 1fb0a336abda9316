"""paged_kv_rope_write against the 64-bit rotation (angles in extended
precision) and the oracle's slot-mapped write.

Tolerances, per element with pair (x, y): cosine and sine are off by at most
2^-22 (the angle by 2^-26 turns, 2 pi 2^-26 < 2^-23, and the functions by
2^-23), the two products and their sum by 2^-22 (|x| + |y|) more, so the
binary32 result by (|x| + |y|) 2^-21; then one rounding: 2^-8 of the value
for bf16, 2^-4 of the value or half the smallest E4M3 step (2^-10) for E4M3.
"""
import numpy as np
import pytest
import torch

import lifetime_ref as ref
import oracle
from paged_kv_cache_48_gb300 import (PagedKVCache, PagedKVError, RotaryAxes,
                                     paged_kv_rope_write, paged_kv_write, pkv_check)

pytestmark = pytest.mark.gpu
INT_MAX = 2 ** 31 - 1


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _bf16(rng, shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16)


def _make(T, Hq, Hkv, D, kv_dtype="bf16", fused=False, seed=0, blocks=None):
    rng = np.random.default_rng(seed)
    blocks = blocks or max(2, (T + 15) // 16 + 2)
    if fused:
        x = _bf16(rng, (T, (Hq + 2 * Hkv) * D)).cuda()
        q = x[:, :Hq * D].view(T, Hq, D)
        k = x[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
        v = x[:, (Hq + Hkv) * D:].view(T, Hkv, D)
    else:
        q, k, v = (_bf16(rng, (T, h, D)).cuda() for h in (Hq, Hkv, Hkv))
    elt = torch.bfloat16 if kv_dtype == "bf16" else torch.uint8
    shape = (blocks, 16, Hkv, D)
    kc, vc = (torch.empty(shape, dtype=elt, device="cuda") for _ in range(2))
    kc.view(torch.uint8).fill_(0xFF)
    vc.view(torch.uint8).fill_(0xFF)
    cache = PagedKVCache(kc, vc, kv_dtype, *((4.5 / 448, 5.0 / 448) if kv_dtype != "bf16"
                                             else (1.0, 1.0)))
    slots = torch.from_numpy(rng.permutation(blocks * 16)[:T].astype(np.int64)).cuda()
    return rng, q, k, v, cache, slots


def _check(q, k, v, qo, cache, slots, pos, rope, q_in=None, k_in=None):
    """qo and the cache against the references; rows no slot names keep 0xFF."""
    T, Hkv, D = k.shape
    p = pos.cpu().numpy().reshape(rope.num_axes, T)
    args = (p, rope.frequencies, rope.axis, rope.rotary_dim, rope.interleave_pairs)
    R = rope.rotary_dim
    if qo is not None:
        src = q_in if q_in is not None else q
        want, mag = ref.rotate(_f64(src), *args)
        got = _f64(qo)
        err = np.abs(got - want) - (2.0 ** -8 * np.abs(want) + mag * 2.0 ** -21)
        assert err[:, :, :R].max(initial=-1) <= 0
        assert torch.equal(qo[:, :, R:].contiguous().view(torch.int16),
                           src[:, :, R:].contiguous().view(torch.int16))
    want, mag = ref.rotate(_f64(k if k_in is None else k_in), *args)
    s = slots.cpu().numpy()
    live = (s >= 0) & (s < cache.num_blocks * 16)
    raw = [c.view(torch.uint8).cpu().numpy().reshape(cache.num_blocks * 16, -1)
           for c in (cache.key_cache, cache.value_cache)]
    rest = np.setdiff1d(np.arange(cache.num_blocks * 16), s[live])
    for r in raw:
        assert (r[rest] == 0xFF).all()
    # v: the oracle's slot-mapped write, bit for bit
    o = oracle.load()
    dt = oracle.DTYPE_BF16 if cache.kv_dtype == "bf16" else oracle.DTYPE_FP8_E4M3
    ok, ov = (np.full(raw[0].size, 0xFF, np.uint8) for _ in range(2))
    bits = v.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
    o.kv_write(ok, ov, dt, 16, Hkv, D, cache.k_scale, cache.v_scale, bits, bits,
               np.where(live, s, -1))
    assert np.array_equal(raw[1].reshape(-1), ov)
    if cache.kv_dtype == "bf16":
        got = _f64(cache.key_cache).reshape(-1, Hkv, D)[s[live]]
        tol = 2.0 ** -8 * np.abs(want) + mag * 2.0 ** -21
        assert (np.abs(got - want[live]) <= tol[live]).all()
        same = cache.key_cache.view(torch.int16).cpu().numpy().reshape(-1, Hkv, D)[s[live]]
        kb = k.contiguous().view(torch.int16).cpu().numpy()[live]
        assert np.array_equal(same[:, :, R:], kb[:, :, R:])
    else:
        got = ref.E4M3[raw[0].reshape(-1, Hkv, D)[s[live]]]
        scale = float(np.float32(cache.k_scale))
        t = np.clip(want / scale, -448, 448)
        tol = np.maximum(2.0 ** -4 * np.abs(t), 2.0 ** -10) + mag / scale * 2.0 ** -20
        assert (np.abs(got - t[live]) <= tol[live]).all()
        if R < D:  # not turned: exactly the slot-mapped write's codes
            kb = k.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
            o.kv_write(ok, ov, dt, 16, Hkv, D, cache.k_scale, cache.v_scale, kb, kb,
                       np.where(live, s, -1))
            assert np.array_equal(raw[0].reshape(-1, Hkv, D)[s[live]][:, :, R:],
                                  ok.reshape(-1, Hkv, D)[s[live]][:, :, R:])


CASES = [
    # T, Hq, Hkv, D, R, sections, dealt, adjacent, fused
    (1, 1, 1, 64, 64, [32], False, False, False),
    (1, 32, 8, 128, 128, [16, 24, 24], False, False, True),
    (2, 8, 8, 64, 16, [8], False, True, False),
    (3, 7, 1, 128, 48, [8, 8, 8], True, False, True),
    (17, 40, 8, 128, 128, [24, 20, 20], True, False, False),
    (33, 6, 3, 64, 32, [4, 4, 4, 4], False, True, True),
    (64, 5, 5, 128, 96, [20, 0, 28], False, True, True),
    (257, 9, 3, 64, 64, [16, 16], True, True, False),
    (1111, 4, 2, 64, 48, [9, 15], False, False, True),
]


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "T%d_q%d_kv%d_d%d_r%d" % c[:5])
def test_matches_reference(case, kv_dtype):
    T, Hq, Hkv, D, R, sections, dealt, adjacent, fused = case
    rng, q, k, v, cache, slots = _make(T, Hq, Hkv, D, kv_dtype, fused, seed=T)
    rope = RotaryAxes(R, sections, base=5e5, interleave_axes=dealt, interleave_pairs=adjacent)
    pos = torch.from_numpy(rng.integers(0, 100000, (len(sections), T)).astype(np.int32)).cuda()
    qo = paged_kv_rope_write(q, k, v, pos, slots, cache, rope)
    assert pkv_check()[0] == 0
    _check(q, k, v, qo, cache, slots, pos, rope)


@pytest.mark.parametrize("adjacent", [False, True])
def test_extreme_positions(adjacent):
    """Negative positions, zero, and the ends of int32, where a binary32
    angle would keep no digit of the turn."""
    T = 12
    rng, q, k, v, cache, slots = _make(T, 4, 2, 128, seed=5)
    rope = RotaryAxes(128, [32, 32], base=1e4, interleave_pairs=adjacent)
    p = [[0, 1, -1, INT_MAX, -INT_MAX - 1, INT_MAX - 7, 1 << 24, (1 << 24) + 1, -(1 << 30), 12345,
          -99999, 3], [INT_MAX, 0, -5, -INT_MAX, 77, 1, 1 << 30, 2, 3, -4, 5, 999999999]]
    pos = torch.tensor(p, dtype=torch.int32, device="cuda")
    qo = paged_kv_rope_write(q, k, v, pos, slots, cache, rope)
    _check(q, k, v, qo, cache, slots, pos, rope)


def test_given_frequencies():
    """Any frequency up to the limit, negative, zero and a half turn."""
    T = 9
    rng, q, k, v, cache, slots = _make(T, 2, 2, 64, seed=6)
    f = [0.0, -0.5, np.pi, -np.pi, 2 * np.pi, 1024.0, -1024.0, 1e-12] + \
        list(rng.uniform(-100, 100, 24))
    rope = RotaryAxes(64, [32], frequencies=f)
    pos = torch.from_numpy(rng.integers(-5000, 5000, T).astype(np.int32)).cuda()  # 1-D: one axis
    qo = paged_kv_rope_write(q, k, v, pos, slots, cache, rope)
    _check(q, k, v, qo, cache, slots, pos, rope)


def test_zero_positions_leave_the_bits():
    T = 40
    _, q, k, v, cache, slots = _make(T, 8, 4, 128, fused=True, seed=7)
    rope = RotaryAxes(128, [64])
    qo = paged_kv_rope_write(q, k, v, torch.zeros(T, dtype=torch.int32, device="cuda"), slots,
                             cache, rope)
    assert torch.equal(qo, q)
    other = PagedKVCache.empty(cache.num_blocks, 4, 128)
    other.key_cache.copy_(cache.key_cache)
    paged_kv_write(k.contiguous(), v.contiguous(), slots, other)
    assert torch.equal(other.key_cache.view(torch.int16), cache.key_cache.view(torch.int16))


@pytest.mark.parametrize("T", [1, 45])
def test_in_place_and_slices(T):
    """q turned in place inside a fused projection; q_out and positions with
    row strides of their own; bytes around them untouched."""
    rng, q, k, v, cache, slots = _make(T, 8, 2, 64, fused=True, seed=8)
    rope = RotaryAxes(64, [12, 20], interleave_axes=False)
    wide = torch.from_numpy(rng.integers(0, 9999, (2, T + 13)).astype(np.int32)).cuda()
    pos = wide[:, :T]
    q_in, k_in, v_in = q.clone(), k.clone(), v.clone()
    buf = torch.full((T, 8 * 64 + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    qo = buf[:, 8:8 + 512].view(T, 8, 64)
    paged_kv_rope_write(q, k, v, pos, slots, cache, rope, q_out=qo)
    assert (buf[:, :8] == 7.0).all() and (buf[:, 520:] == 7.0).all()
    _check(q, k, v, qo, cache, slots, pos, rope)
    r = paged_kv_rope_write(q, k, v, pos, slots, cache, rope, q_out=q)
    assert r is q and torch.equal(q, qo)
    assert torch.equal(k, k_in) and torch.equal(v, v_in)
    _check(q, k, v, q, cache, slots, pos, rope, q_in=q_in)


def test_one_row_of_positions_for_every_axis():
    """Text only: positions expanded over the axes (stride 0)."""
    T = 19
    rng, q, k, v, cache, slots = _make(T, 4, 2, 64, seed=14)
    rope = RotaryAxes(64, [12, 10, 10])
    pos = torch.from_numpy(rng.integers(0, 9999, T).astype(np.int32)).cuda()
    qo = paged_kv_rope_write(q, k, v, pos.expand(3, T), slots, cache, rope)
    _check(q, k, v, qo, cache, slots, torch.stack([pos, pos, pos]), rope)


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8_e4m3"])
def test_padding_and_bad_slots(kv_dtype):
    T = 21
    _, q, k, v, cache, slots = _make(T, 4, 2, 128, kv_dtype, seed=9)
    slots[3] = -1
    slots[7] = -(2 ** 62)
    rope = RotaryAxes(128, [64])
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    qo = paged_kv_rope_write(q, k, v, pos, slots, cache, rope)
    assert pkv_check()[0] == 0
    _check(q, k, v, qo, cache, slots, pos, rope)  # padding: q turned, nothing written
    cache.key_cache.view(torch.uint8).fill_(0xFF)
    cache.value_cache.view(torch.uint8).fill_(0xFF)
    slots[11] = cache.num_blocks * 16  # one past the pool
    slots[12] = 2 ** 62
    qo = paged_kv_rope_write(q, k, v, pos, slots, cache, rope)
    st, detail = pkv_check()
    assert st == 5 and detail in (11, 12)
    _check(q, k, v, qo, cache, slots, pos, rope)
    assert pkv_check()[0] == 0


def test_without_q_and_empty():
    T = 10
    _, q, k, v, cache, slots = _make(T, 4, 2, 64, seed=10)
    rope = RotaryAxes(32, [16])
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    assert paged_kv_rope_write(None, k, v, pos, slots, cache, rope) is None
    _check(q, k, v, None, cache, slots, pos, rope)
    out = paged_kv_rope_write(q[:0], k[:0], v[:0], pos[:0], slots[:0], cache, rope)
    assert out.shape == (0, 4, 64)


def test_non_finite_values_stay_in_their_pair():
    T = 4
    _, q, k, v, cache, slots = _make(T, 2, 1, 64, seed=11)
    q[1, 0, 5] = float("nan")
    q[2, 1, 40] = float("inf")
    rope = RotaryAxes(64, [32])
    pos = torch.arange(1, T + 1, dtype=torch.int32, device="cuda")
    qo = paged_kv_rope_write(q, k, v, pos, slots, cache, rope)
    bad = ~torch.isfinite(qo.float())
    want = torch.zeros_like(bad)
    want[1, 0, 5] = want[1, 0, 37] = want[2, 1, 40] = want[2, 1, 8] = True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("T,Hq,Hkv,D,kv_dtype", [
    (20011, 2, 1, 64, "bf16"), (2431, 4, 2, 128, "bf16"), (2433, 4, 2, 128, "fp8_e4m3"),
    (1300, 20, 5, 128, "bf16"), (1217, 17, 8, 64, "fp8_e4m3"), (4000, 1, 1, 128, "bf16")])
def test_many_tokens_take_every_unit(T, Hq, Hkv, D, kv_dtype):
    """Warps with runs of several units, tokens cut between two warps, last
    units of a token partly empty."""
    rng, q, k, v, cache, slots = _make(T, Hq, Hkv, D, kv_dtype, seed=12)
    slots[T // 2] = -1
    slots[T - 1] = -1
    rope = RotaryAxes(D, [D // 4, D // 4])
    pos = torch.from_numpy(rng.integers(0, 1 << 20, (2, T)).astype(np.int32)).cuda()
    qo = paged_kv_rope_write(q, k, v, pos, slots, cache, rope)
    _check(q, k, v, qo, cache, slots, pos, rope)


def test_binding_refusals():
    T = 6
    _, q, k, v, cache, slots = _make(T, 4, 2, 64, seed=13)
    rope = RotaryAxes(64, [32])
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    ok = dict(q=q, k=k, v=v, positions=pos, slot_mapping=slots, cache=cache, rope=rope)

    def bad(exc, **kw):
        with pytest.raises(exc):
            paged_kv_rope_write(**{**ok, **kw})
    bad(TypeError, q=q.float())
    bad(TypeError, positions=pos.long())
    bad(TypeError, slot_mapping=slots.int())
    bad(TypeError, rope=64)
    bad(ValueError, positions=pos[:5])
    bad(ValueError, positions=torch.stack([pos, pos]))
    bad(ValueError, positions=torch.stack([pos, pos], 1)[:, 0])   # strided
    bad(ValueError, q=q.transpose(0, 1).contiguous().transpose(0, 1))
    bad(ValueError, k=k[:, :, :32])
    bad(ValueError, v=v[:5])
    bad(ValueError, slot_mapping=slots[:5])
    bad(ValueError, q=None, q_out=q)
    bad(ValueError, q=q.cpu())
    bad(ValueError, q_out=q[:5])
    with pytest.raises(PagedKVError):
        paged_kv_rope_write(**{**ok, "rope": RotaryAxes(128, [64])})   # past head_dim
    both = torch.empty(T, 8, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(PagedKVError):  # overlapping rows
        paged_kv_rope_write(**{**ok, "q": both[:, :4], "q_out": both[:, 2:6]})
    paged_kv_rope_write(**{**ok, "q": both[:, :4], "q_out": both[:, 4:]})  # apart: fine
    assert pkv_check()[0] == 0
