"""The cache-lifetime operators together, as a serving loop uses them: prompts
written with rotary positions and attended by the chunked prefill, decode
steps that write, attend and keep weights, evictions in place, further steps
whose positions go on while their slots moved up.  A plain model of every
(sequence, kv head)'s tokens is kept beside it.  Also: replay from CUDA
graphs, other streams, large pools, and guard rows."""
import numpy as np
import pytest
import torch

import harness
import lifetime_ref as ref
from paged_kv_cache_48_gb300 import (PagedKVCache, RotaryAxes,
                                     paged_attention_decode_weights,
                                     paged_attention_decode_weights_workspace_bytes,
                                     paged_attention_prefill, paged_kv_evict,
                                     paged_kv_evict_workspace_bytes,
                                     paged_kv_rope_write, paged_prepare_inputs, pkv_check)
from paged_kv_cache_48_gb300 import workload as wl

pytestmark = pytest.mark.gpu


def _dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def _cached(cache, slots):
    """What the cache holds at these slots: (K, V) [n, Hkv, D] float64, as
    attention reads it (scales applied), and the raw bytes."""
    raw = [c.view(torch.uint8).reshape(cache.num_blocks * 16, -1)[_dev(slots)].cpu().numpy()
           for c in (cache.key_cache, cache.value_cache)]
    vals = []
    for r, s in zip(raw, (cache.k_scale, cache.v_scale)):
        if cache.kv_dtype == "bf16":
            u = r.view(np.uint16).astype(np.uint32) << 16
            vals.append(u.view(np.float32).astype(np.float64))
        else:
            vals.append(ref.E4M3[r] * float(np.float32(s)))
    D = cache.head_dim
    return [v.reshape(len(slots), -1, D) for v in vals], raw


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("per_head", [True, False])
def test_serving_loop(kv_dtype, per_head):
    rng = np.random.default_rng(3)
    B, Hq, Hkv, D, S = 3, 8, 2, 64, 160
    group, scale = Hq // Hkv, 1.0 / 8.0
    cache = PagedKVCache.empty(64, Hkv, D, kv_dtype,
                               *((4.5 / 448, 4.5 / 448) if kv_dtype != "bf16" else ()))
    for c in (cache.key_cache, cache.value_cache):
        c.view(torch.uint8).fill_(0xFF)  # NaN: stale bits must never matter
    tables = rng.permutation(64)[:B * (S // 16)].astype(np.int32).reshape(B, -1)
    gt = _dev(tables)
    rope = RotaryAxes(D, [8, 12, 12], base=1e4)
    weights = torch.zeros(B, Hkv, S, device="cuda")
    slot = lambda b, t: int(tables[b, t // 16]) * 16 + t % 16

    def bf16(*shape):
        return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).bfloat16().cuda()

    # prompts: q, k and v slices of one projection, text and grid positions
    lens = np.array([37, 64, 90], np.int32)
    pos = lens.astype(np.int64).copy()  # a sequence's next position
    T = int(lens.sum())
    qkv = bf16(T, (Hq + 2 * Hkv) * D)
    q, k, v = (x.view(T, -1, D) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], dim=1))
    p0 = np.concatenate([np.arange(n) for n in lens])
    p3 = np.stack([p0, p0 + p0 % 7, p0 + p0 % 5]).astype(np.int32)
    slots = np.array([slot(b, t) for b in range(B) for t in range(lens[b])])
    qsl = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    qr = paged_kv_rope_write(q, k, v, _dev(p3), _dev(slots), cache, rope)
    out = paged_attention_prefill(qr, cache, gt, _dev(lens), _dev(qsl), scale, int(lens.max()))
    assert pkv_check()[0] == 0
    turned, _ = ref.rotate(q.float().cpu().numpy().astype(np.float64), p3, rope.frequencies,
                           rope.axis, D, False)
    (K, V), _ = _cached(cache, slots)
    got = out.float().cpu().numpy()
    want = np.zeros_like(got)
    for b in range(B):
        for i in range(lens[b]):
            r = qsl[b] + i
            for h in range(Hkv):
                o, _, _ = ref.attention_weights(turned[r, h * group:(h + 1) * group],
                                                K[qsl[b]:r + 1, h], V[qsl[b]:r + 1, h], scale)
                want[r, h * group:(h + 1) * group] = o
    harness.assert_close(got, want, kv_dtype)
    # the model: raw rows of every (sequence, head)'s tokens, in order
    _, raw = _cached(cache, slots)
    e = D * cache.key_cache.element_size()
    rows = [[[[raw[c][qsl[b] + t, h * e:(h + 1) * e].copy() for t in range(lens[b])]
              for h in range(Hkv)] for c in (0, 1)] for b in range(B)]
    gl = _dev(lens)
    for step in range(24):
        # one new token each: position from the stream, slot from the length
        new = np.array([slot(b, int(lens[b])) for b in range(B)])
        p3 = np.stack([pos, pos + 1, pos + 2]).astype(np.int32)
        lens += 1
        pos += 1
        gl += 1
        q, k, v = bf16(B, Hq, D), bf16(B, Hkv, D), bf16(B, Hkv, D)
        qr = paged_kv_rope_write(q, k, v, _dev(p3), _dev(new), cache, rope)
        old = weights.cpu().numpy().astype(np.float64)
        decay = 1.0 if step % 2 else 0.9
        out = paged_attention_decode_weights(qr, cache, gt, gl, scale, S, weights, decay=decay)
        assert pkv_check()[0] == 0
        q64 = qr.float().cpu().numpy().astype(np.float64)
        _, raw = _cached(cache, new)
        for b in range(B):
            L = int(lens[b])
            for c in (0, 1):
                for h in range(Hkv):
                    rows[b][c][h].append(raw[c][b, h * e:(h + 1) * e].copy())
            sl = np.array([slot(b, t) for t in range(L)])
            (K, V), now = _cached(cache, sl)
            for h in range(Hkv):
                for c in (0, 1):  # the cache is the model, byte for byte
                    assert np.array_equal(now[c][:, h * e:(h + 1) * e], np.array(rows[b][c][h]))
                o, p, bound = ref.attention_weights(q64[b, h * group:(h + 1) * group], K[:, h],
                                                    V[:, h], scale)
                tol = ref.weights_tolerance(D, L, group, bound)
                w = weights[b, h].cpu().numpy().astype(np.float64)
                base = float(np.float32(decay)) * old[b, h, :L]
                lim = tol * p + 2.0 ** -23 * (np.abs(base) + p)
                assert (np.abs(w[:L] - base - p) <= lim).all()
                assert (w[L:] == 0).all()  # positions not reached yet, or given up
                harness.assert_close(out[b, h * group:(h + 1) * group].float().cpu().numpy(), o,
                                     kv_dtype)
        if step % 5 == 4:
            keep = np.array([30, 70 - step, 45], np.int32)
            w = weights.cpu().numpy()
            paged_kv_evict(cache, gt, gl, weights, _dev(keep), 70, sink=2, recent=8,
                           per_head=per_head, new_seq_lens=gl)
            assert pkv_check()[0] == 0
            for b in range(B):
                L = int(lens[b])
                for h in range(Hkv):
                    rank = w[b, h] if per_head else ref.heads_sum(w[b])
                    at = ref.evict_choice(rank, L, int(keep[b]), 2, 8)
                    for c in (0, 1):
                        rows[b][c][h] = [rows[b][c][h][t] for t in at]
                lens[b] = min(L, int(keep[b]))
            assert np.array_equal(gl.cpu().numpy(), lens)


def test_prepared_inputs_feed_the_rotary_write():
    """paged_prepare_inputs' positions (one axis) and slots go straight in."""
    rng = np.random.default_rng(5)
    R, MB, B, Hkv, D = 10, 8, 4, 2, 64
    sbt = rng.permutation(R * MB).astype(np.int32).reshape(R, MB)
    done = np.array([0, 5, 17, 60, 33, 2, 9, 100, 64, 31], np.int32)
    idx, n = np.array([7, 2, 0, 8], np.int32), np.array([3, 1, 20, 16], np.int32)
    T = int(n.sum())
    o = paged_prepare_inputs(_dev(idx), _dev(n), _dev(sbt), _dev(done),
                             _dev(np.zeros((R, 128), np.int32)), T)
    cache = PagedKVCache.empty(R * MB, Hkv, D)
    k, v, q = (torch.randn(T, h, D, device="cuda").bfloat16() for h in (Hkv, Hkv, 4))
    rope = RotaryAxes(D, [D // 2])
    qo = paged_kv_rope_write(q, k, v, o["positions"], o["slot_mapping"], cache, rope)
    assert pkv_check()[0] == 0
    pos = np.concatenate([done[i] + np.arange(c) for i, c in zip(idx, n)])
    want, mag = ref.rotate(q.float().cpu().numpy().astype(np.float64), pos[None],
                           rope.frequencies, rope.axis, D, False)
    got = qo.float().cpu().numpy().astype(np.float64)
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + mag * 2.0 ** -21).all()
    t = np.concatenate([np.arange(done[i], done[i] + c) for i, c in zip(idx, n)])
    row = np.repeat(idx, n)
    slots = sbt[row, t // 16].astype(np.int64) * 16 + t % 16
    assert torch.equal(cache.value_cache.view(-1, Hkv, D)[_dev(slots)], v)


def _loop_state(seed=0, B=5, Hq=8, Hkv=2, D=64, S=200, kv_dtype="bf16"):
    rng = np.random.default_rng(seed)
    lens = rng.integers(20, S, B).astype(np.int32)
    nb = (S + 15) // 16
    order = rng.permutation(2 * B * nb).astype(np.int32)
    s = dict(lens=_dev(lens), tables=_dev(order[:B * nb].reshape(B, nb)),
             dst=_dev(order[B * nb:].reshape(B, nb)), max_len=S, B=B, Hkv=Hkv, S=S)
    cache = PagedKVCache.empty(2 * B * nb, Hkv, D, kv_dtype)
    cache.key_cache.copy_(torch.randn(cache.key_cache.shape, device="cuda"))
    cache.value_cache.copy_(torch.randn(cache.key_cache.shape, device="cuda"))
    s["cache"] = cache
    s["q"] = torch.randn(B, Hq, D, device="cuda").bfloat16()
    s["k"] = torch.randn(B, Hkv, D, device="cuda").bfloat16()
    s["v"] = torch.randn(B, Hkv, D, device="cuda").bfloat16()
    s["pos"] = _dev(rng.integers(0, 5000, (3, B)).astype(np.int32))
    last = lens - 1
    s["slots"] = _dev(order[:B * nb].reshape(B, nb)[np.arange(B), last // 16].astype(np.int64) * 16
                      + last % 16)
    s["rope"] = RotaryAxes(D, [12, 10, 10])
    s["weights"] = torch.rand(B, Hkv, S, device="cuda")
    s["keep"] = _dev(np.minimum(lens, rng.integers(1, 100, B)).astype(np.int32))
    s["dst_w"] = torch.zeros(B, Hkv, S, device="cuda")
    s["new"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    s["kept"] = torch.zeros(B, Hkv, 100, dtype=torch.int32, device="cuda")
    s["qr"], s["out"] = torch.zeros_like(s["q"]), torch.zeros_like(s["q"])
    need = max(paged_attention_decode_weights_workspace_bytes(B, Hq, Hkv, D, S, 64),
               paged_kv_evict_workspace_bytes(B, Hkv, S, 100))
    s["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    return s


def _loop_step(s, stream=None, ws=None):
    ws = s["ws"] if ws is None else ws
    paged_kv_rope_write(s["q"], s["k"], s["v"], s["pos"], s["slots"], s["cache"], s["rope"],
                        q_out=s["qr"], stream=stream)
    paged_attention_decode_weights(s["qr"], s["cache"], s["tables"], s["lens"], 0.125,
                                   s["max_len"], s["weights"], decay=0.5, out=s["out"],
                                   partition_tokens=64, workspace=ws, stream=stream)
    paged_kv_evict(s["cache"], s["tables"], s["lens"], s["weights"], s["keep"], 100, sink=1,
                   recent=3, dst_tables=s["dst"], dst_weights=s["dst_w"], new_seq_lens=s["new"],
                   kept=s["kept"], workspace=ws, stream=stream)


_OUTS = ("qr", "out", "weights", "dst_w", "new", "kept")


def _result(s):
    torch.cuda.synchronize()
    return [s[n].clone() for n in _OUTS] + [s["cache"].key_cache.clone(),
                                           s["cache"].value_cache.clone()]


def _same(a, b):
    bits = lambda t: t.view(torch.int16) if t.dtype == torch.bfloat16 else t
    return all(torch.equal(bits(x), bits(y)) for x, y in zip(a, b))


def test_replayed_from_graphs_that_share_a_workspace():
    """Two captured steps over different states and one workspace, replayed
    in turn, give what the eager steps give (weights accumulate on every
    replay)."""
    A, B = _loop_state(1), _loop_state(2)
    big = max(A["ws"].numel(), B["ws"].numel())
    ws = torch.full((big,), 0xA5, dtype=torch.uint8, device="cuda")
    EA, EB = _loop_state(1), _loop_state(2)
    for n in ("weights", "q", "k", "v"):
        EA[n].copy_(A[n])
        EB[n].copy_(B[n])
    for X, E in ((A, EA), (B, EB)):
        E["cache"].key_cache.copy_(X["cache"].key_cache)
        E["cache"].value_cache.copy_(X["cache"].value_cache)
    w0 = {id(X): X["weights"].clone() for X in (A, B)}
    graphs = []
    for X in (A, B):
        _loop_step(X, ws=ws)  # warm
        torch.cuda.synchronize()
        X["weights"].copy_(w0[id(X)])
        g = torch.cuda.CUDAGraph()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            with torch.cuda.graph(g, stream=s):
                _loop_step(X, ws=ws)
        torch.cuda.current_stream().wait_stream(s)
        graphs.append(g)
    for _ in range(3):
        for g, E in zip(graphs, (EA, EB)):
            g.replay()
            _loop_step(E)
    ra, rb, ea, eb = (_result(x) for x in (A, B, EA, EB))
    assert _same(ra, ea) and _same(rb, eb)
    assert pkv_check()[0] == 0


def test_two_streams_at_once():
    """The same calls on two streams, each with its own workspace, and calls
    that allocate their outputs and workspaces themselves on a side stream."""
    states = [_loop_state(3), _loop_state(4)]
    alone = [_loop_state(3), _loop_state(4)]
    for X, E in zip(states, alone):
        for n in ("weights", "q", "k", "v"):
            E[n].copy_(X[n])
        E["cache"].key_cache.copy_(X["cache"].key_cache)
        E["cache"].value_cache.copy_(X["cache"].value_cache)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for X, s in zip(states, streams):
            _loop_step(X, stream=s)
    for _ in range(20):
        for E in alone:
            _loop_step(E)
    got, want = [_result(x) for x in states], [_result(x) for x in alone]
    for g, w in zip(got, want):
        assert _same(g, w)
    # outputs and workspaces allocated by the call, while the current stream
    # keeps reusing freed memory
    X = states[0]
    ref_out = paged_attention_decode_weights(X["qr"], X["cache"], X["tables"], X["lens"], 0.125,
                                             X["max_len"], X["weights"].clone())
    torch.cuda.synchronize()
    s = streams[1]
    for _ in range(30):
        o = paged_attention_decode_weights(X["qr"], X["cache"], X["tables"], X["lens"], 0.125,
                                           X["max_len"], X["dst_w"], stream=s)
        junk = torch.full((1 << 20,), 0xFF, dtype=torch.uint8, device="cuda")
        q = paged_kv_rope_write(X["q"], X["k"], X["v"], X["pos"], X["slots"], X["cache"],
                                X["rope"], stream=s)
        n = paged_kv_evict(X["cache"], X["tables"], X["lens"], X["weights"], X["keep"], 100,
                           dst_tables=X["dst"], dst_weights=X["dst_w"], stream=s)
        junk2 = torch.full((1 << 16,), 0xFF, dtype=torch.uint8, device="cuda")
        s.synchronize()
        assert torch.equal(o.view(torch.int16), ref_out.view(torch.int16))
        assert torch.equal(q.view(torch.int16), X["qr"].view(torch.int16))
        assert torch.equal(n, X["keep"])
    del junk, junk2
    assert pkv_check()[0] == 0


def test_calls_repeat_to_the_bit():
    a = _loop_state(7, B=9, S=700)
    b = _loop_state(7, B=9, S=700)
    for n in ("weights", "q", "k", "v"):
        b[n].copy_(a[n])
    b["cache"].key_cache.copy_(a["cache"].key_cache)
    b["cache"].value_cache.copy_(a["cache"].value_cache)
    for _ in range(5):
        _loop_step(a)
        _loop_step(b)
    assert _same(_result(a), _result(b))


def test_pools_past_four_gigabytes():
    """Blocks whose byte offsets pass 2^32 (and element offsets 2^31): the
    write, the attention, the weights and the moves land there."""
    Hkv, D, Hq = 8, 128, 16
    nb = (1 << 32) // (16 * Hkv * D * 2) + 64  # blocks of 32 KiB
    cache = PagedKVCache.empty(nb, Hkv, D)
    rng = np.random.default_rng(9)
    L = 40
    tables = np.array([[nb - 1, nb - 33, nb - 7], [3, nb - 2, 11]], np.int32)
    dst = np.array([[nb - 3, 7], [nb - 50, nb - 51]], np.int32)
    slots = np.array([int(tables[b, t // 16]) * 16 + t % 16 for b in range(2) for t in range(L)])
    k, v = (torch.randn(2 * L, Hkv, D, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(2, Hq, D, device="cuda").bfloat16()
    rope = RotaryAxes(D, [64])
    pos = torch.arange(2 * L, dtype=torch.int32, device="cuda")
    paged_kv_rope_write(None, k, v, pos, _dev(slots), cache, rope)
    lens = torch.tensor([L, L], dtype=torch.int32, device="cuda")
    w = torch.zeros(2, Hkv, 48, device="cuda")
    out = paged_attention_decode_weights(q, cache, _dev(tables), lens, 0.09, 48, w)
    kept = torch.zeros(2, Hkv, 20, dtype=torch.int32, device="cuda")
    dw = torch.zeros(2, Hkv, 48, device="cuda")
    paged_kv_evict(cache, _dev(tables), lens, w, _dev(np.array([20, 20], np.int32)), 20,
                   dst_tables=_dev(dst), dst_weights=dw, kept=kept)
    assert pkv_check()[0] == 0
    small = PagedKVCache.empty(6, Hkv, D)  # the same at small block ids
    st = np.arange(6, dtype=np.int32).reshape(2, 3)
    ss = np.array([int(st[b, t // 16]) * 16 + t % 16 for b in range(2) for t in range(L)])
    paged_kv_rope_write(None, k, v, pos, _dev(ss), small, rope)
    w2 = torch.zeros_like(w)
    o2 = paged_attention_decode_weights(q, small, _dev(st), lens, 0.09, 48, w2)
    assert torch.equal(out.view(torch.int16), o2.view(torch.int16)) and torch.equal(w, w2)
    kv = small.key_cache.view(-1, Hkv, D)
    big = cache.key_cache.view(-1, Hkv, D)
    at = kept.cpu().numpy()
    for b in range(2):
        for h in (0, 7):
            want = ref.evict_choice(w2[b, h].cpu().numpy(), L, 20, 0, 0)
            assert at[b, h].tolist() == want
            s = np.array([int(st[b, t // 16]) * 16 + t % 16 for t in want])
            d = np.array([int(dst[b, i // 16]) * 16 + i % 16 for i in range(20)])
            assert torch.equal(big[_dev(d), h], kv[_dev(s), h])


def test_workspace_past_two_gigabytes():
    """A host bound of 131072 tokens for 80 sequences: the last sequence's
    scores lie past 2^31 bytes of the workspace."""
    B, Hq, Hkv, D, bound = 80, 64, 8, 128, 131072
    need = paged_attention_decode_weights_workspace_bytes(B, Hq, Hkv, D, bound, 0)
    assert need > 1 << 31
    rng = np.random.default_rng(10)
    lens = np.zeros(B, np.int32)
    lens[0], lens[-1], lens[40] = 70, 333, 16
    cache = PagedKVCache.empty(64, Hkv, D)
    cache.key_cache.copy_(torch.randn(cache.key_cache.shape, device="cuda"))
    cache.value_cache.copy_(torch.randn(cache.key_cache.shape, device="cuda"))
    tables = np.zeros((B, bound // 16), np.int32)
    tables[:, :30] = rng.integers(0, 64, (B, 30))
    q = torch.randn(B, Hq, D, device="cuda").bfloat16()
    w = torch.zeros(B, Hkv, bound, device="cuda")
    out = paged_attention_decode_weights(q, cache, _dev(tables), _dev(lens), 0.09, bound, w)
    idx = _dev(np.array([0, 40, B - 1]))
    w2 = torch.zeros(3, Hkv, 336, device="cuda")
    o2 = paged_attention_decode_weights(q[idx].contiguous(), cache,
                                        _dev(tables[[0, 40, B - 1], :30]),
                                        _dev(lens[[0, 40, B - 1]]), 0.09, 336, w2)
    assert pkv_check()[0] == 0
    # another bound, another partition length: equal up to the sums' order
    assert torch.allclose(w[idx][:, :, :336], w2, rtol=1e-5, atol=0)
    assert torch.allclose(out[idx].float(), o2.float(), rtol=2e-2, atol=2e-3)
    assert not bool(w[:, :, 336:].any()) and not bool(w[1:40].any())


def test_largest_batch():
    """65535 sequences, the grid's limit, of 1 to 20 tokens."""
    B, D = 65535, 64
    lens = (np.arange(B) % 20 + 1).astype(np.int32)
    order = torch.randperm(2 * B, device="cuda").to(torch.int32).view(B, 2)
    cache = PagedKVCache.empty(2 * B, 1, D)
    cache.key_cache.normal_()
    cache.value_cache.normal_()
    gl = _dev(lens)
    q = torch.randn(B, 1, D, device="cuda").bfloat16()
    w = torch.zeros(B, 1, 20, device="cuda")
    out = paged_attention_decode_weights(q, cache, order, gl, 0.125, 20, w)
    t = torch.arange(20, device="cuda")
    slots = order.long()[:, t // 16] * 16 + t % 16
    k = cache.key_cache.view(-1, D)[slots].double()
    v = cache.value_cache.view(-1, D)[slots].double()
    s = torch.einsum("bd,btd->bt", q[:, 0].double(), k) * 0.125
    s[t >= gl[:, None]] = float("-inf")
    p = torch.softmax(s, -1)
    bound = float((torch.einsum("bd,btd->bt", q[:, 0].double().abs(), k.abs()) * 0.125).max())
    tol = ref.weights_tolerance(D, 20, 1, bound)
    assert bool(((w[:, 0].double() - p).abs() <= tol * p + 1e-37).all())
    ref_out = torch.einsum("bt,btd->bd", p, torch.where((t < gl[:, None])[:, :, None], v, 0.0))
    assert bool(((out[:, 0].double() - ref_out).abs() <= 1e-2 + 1e-2 * ref_out.abs()).all())
    keep = torch.full((B,), 7, dtype=torch.int32, device="cuda")
    old = w.clone()
    before = cache.key_cache.view(-1, D)[slots].clone()
    kept = torch.empty(B, 1, 7, dtype=torch.int32, device="cuda")
    new = paged_kv_evict(cache, order, gl, w, keep, 7, sink=1, recent=2, kept=kept)
    assert pkv_check()[0] == 0
    assert torch.equal(new, torch.clamp(gl, max=7))
    at = kept[:, 0].long()
    live = at >= 0
    assert torch.equal(live.sum(-1).int(), new)
    got = cache.key_cache.view(-1, D)[slots[:, :7]]
    want = torch.gather(before, 1, at.clamp(min=0)[:, :, None].expand(-1, -1, D))
    assert torch.equal(got[live].view(torch.int16), want[live].view(torch.int16))
    assert torch.equal(w[:, 0, :7][live], torch.gather(old[:, 0], 1, at.clamp(min=0))[live])
    for b in (0, 6, 7, 8, 19, 65534):
        assert at[b][live[b]].tolist() == ref.evict_choice(old[b, 0].cpu().numpy(), int(lens[b]), 7,
                                                           1, 2)


@pytest.mark.parametrize("per_head", [True, False])
def test_many_kv_heads(per_head):
    """300 kv heads with a query head each."""
    H, D, L = 300, 64, 90
    cache = PagedKVCache.empty(12, H, D)
    rng = np.random.default_rng(2)
    tables = rng.permutation(12).astype(np.int32).reshape(2, 6)
    slots = np.array([int(tables[b, t // 16]) * 16 + t % 16 for b in range(2) for t in range(L)])
    q, k, v = (torch.randn(2 * L, H, D, device="cuda").bfloat16() for _ in range(3))
    pos = torch.arange(2 * L, dtype=torch.int32, device="cuda")
    rope = RotaryAxes(D, [32])
    qr = paged_kv_rope_write(q, k, v, pos, _dev(slots), cache, rope)
    want, mag = ref.rotate(q[:3].float().cpu().numpy().astype(np.float64), np.arange(3)[None],
                           rope.frequencies, rope.axis, D, False)
    got = qr[:3].float().cpu().numpy()
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + mag * 2.0 ** -21).all()
    lens = torch.tensor([L, L], dtype=torch.int32, device="cuda")
    w = torch.zeros(2, H, L, device="cuda")
    paged_attention_decode_weights(qr[:2].contiguous(), cache, _dev(tables), lens, 0.125, L, w)
    old = w.cpu().numpy()
    for b in range(2):
        kk = cache.key_cache.view(-1, H, D)[_dev(slots[b * L:(b + 1) * L])].double()
        p = torch.softmax(torch.einsum("hd,thd->ht", qr[b].double(), kk) * 0.125, -1)
        bound = float((torch.einsum("hd,thd->ht", qr[b].double().abs(), kk.abs()) * 0.125).max())
        tol = ref.weights_tolerance(D, L, 1, bound)
        assert bool(((w[b].double() - p).abs() <= tol * p + 1e-37).all())
    kept = torch.empty(2, H if per_head else 1, 33, dtype=torch.int32, device="cuda")
    paged_kv_evict(cache, _dev(tables), lens, w, _dev(np.array([33, 20], np.int32)), 33, sink=3,
                   recent=5, per_head=per_head, kept=kept)
    assert pkv_check()[0] == 0
    for b, n in ((0, 33), (1, 20)):
        for h in (0, 1, 150, 299):
            rank = old[b, h] if per_head else ref.heads_sum(old[b])
            at = ref.evict_choice(rank, L, n, 3, 5)
            assert kept[b, h if per_head else 0, :n].tolist() == at
            d = np.array([int(tables[b, i // 16]) * 16 + i % 16 for i in range(n)])
            assert torch.equal(cache.value_cache.view(-1, H, D)[_dev(d), h],
                               v[b * L:(b + 1) * L, h][_dev(np.array(at))])


def test_host_threads_call_at_once():
    """Four host threads, a stream and a state each."""
    import threading
    states, alone = [_loop_state(10 + i) for i in range(4)], [_loop_state(10 + i) for i in range(4)]
    for X, E in zip(states, alone):
        for n in ("weights", "q", "k", "v"):
            E[n].copy_(X[n])
        E["cache"].key_cache.copy_(X["cache"].key_cache)
        E["cache"].value_cache.copy_(X["cache"].value_cache)
    torch.cuda.synchronize()
    failed = []

    def work(X):
        try:
            s = torch.cuda.Stream()
            for _ in range(25):
                _loop_step(X, stream=s)
            s.synchronize()
        except Exception as e:  # noqa: BLE001 (reported below)
            failed.append(e)
    threads = [threading.Thread(target=work, args=(X,)) for X in states]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for _ in range(25):
        for E in alone:
            _loop_step(E)
    for X, E in zip(states, alone):
        assert _same(_result(X), _result(E))
    assert pkv_check()[0] == 0
