"""paged_attention_decode_weights: the output and the caches bit for bit
those of paged_attention_decode / paged_attention_decode_step, the weights
against a 64-bit softmax over what the cache holds (tolerance derived in
lifetime_ref.weights_tolerance)."""
import numpy as np
import pytest
import torch

import harness
import lifetime_ref as ref
from paged_kv_cache_48_gb300 import _native
from paged_kv_cache_48_gb300 import (PagedKVCache, PagedKVError, paged_attention_decode,
                                     paged_attention_decode_step,
                                     paged_attention_decode_weights,
                                     paged_attention_decode_weights_workspace_bytes,
                                     pkv_check)
from paged_kv_cache_48_gb300 import workload as wl

pytestmark = pytest.mark.gpu


def _values(cache):
    """(K, V) float64 of the pool, scales applied."""
    if cache.kv_dtype == "bf16":
        return (cache.key_cache.float().cpu().numpy().astype(np.float64),
                cache.value_cache.float().cpu().numpy().astype(np.float64))
    return (ref.E4M3[cache.key_cache.cpu().numpy()] * float(np.float32(cache.k_scale)),
            ref.E4M3[cache.value_cache.cpu().numpy()] * float(np.float32(cache.v_scale)))


def _expect(W, G, lens, tables, scale):
    """Per (b, kv head): summed weights, tolerance (relative)."""
    K, _ = _values(G.cache)
    q = G.q.float().cpu().numpy().astype(np.float64)
    group = W.num_heads // W.num_kv_heads
    res = {}
    for b, L in enumerate(lens):
        L = int(L)
        t = np.arange(L)
        blk = tables[b][t // 16]
        ok = (blk >= 0) & (blk < G.cache.num_blocks)
        for h in range(W.num_kv_heads):
            k = K[np.where(ok, blk, 0), t % 16, h]
            w = np.zeros(L)
            _, p, bound = ref.attention_weights(q[b, h * group:(h + 1) * group], k[ok], k[ok],
                                                scale)
            w[ok] = p
            res[b, h] = (w, ref.weights_tolerance(W.head_dim, L, group, bound))
    return res


def _check(W, G, weights, old, lens, tables, decay, fresh=None, scale=None):
    """weights against decay * old + the step's (fresh[b]: first position
    that starts from 0)."""
    got = weights.cpu().numpy().astype(np.float64)
    old = old.cpu().numpy()
    exp = _expect(W, G, lens, tables, W.scale if scale is None else scale)
    for b, L in enumerate(lens):
        L = int(L)
        assert np.array_equal(weights[b, :, L:].cpu().numpy(), old[b, :, L:], equal_nan=True)
        for h in range(W.num_kv_heads):
            w, tol = exp[b, h]
            base = np.zeros(L) if decay == 0 else \
                float(np.float32(decay)) * old[b, h, :L].astype(np.float64)
            if fresh is not None:
                base[fresh[b]:] = 0.0
            err = np.abs(got[b, h, :L] - (base + w))
            lim = tol * w + 2.0 ** -23 * (np.abs(base) + w) + 1e-37
            assert (err <= lim).all(), (b, h, float((err - lim).max()))


def _old(W, width, seed=1):
    g = torch.Generator().manual_seed(seed)
    return torch.rand(W.batch, W.num_kv_heads, width, generator=g).cuda()


CASES = {
    "tiny": (lambda: wl.tiny_mha(), 0),
    "gqa": (lambda: wl.llama8b_gqa(small=True), 0),
    "gqa_warp": (lambda: wl.llama8b_gqa(small=True), 64),
    "fp8": (lambda: wl.fp8_recycle(small=True), 0),
    "fp8_warp": (lambda: wl.fp8_recycle(small=True), 32),
    "long": (lambda: wl.long_context(small=True), 0),
    "long_512": (lambda: wl.long_context(small=True), 512),
    "g16_d64": (lambda: wl.make_workload("g16", 3, 32, 2, 64, 1, 300, 31), 0),
    "g16_fp8_d64": (lambda: wl.make_workload("g16", 3, 32, 2, 64, 1, 300, 31,
                                             kv_dtype="fp8_e4m3"), 48),
    "g3": (lambda: wl.make_workload("g3", 5, 9, 3, 128, 0, 0, 32,
                                    seq_lens=[0, 1, 16, 17, 1025]), 0),
    "g11_split": (lambda: wl.make_workload("g11", 2, 22, 2, 128, 0, 0, 33,
                                           seq_lens=[2100, 3]), 1024),
    "unsplit": (lambda: wl.make_workload("unsplit", 3, 8, 2, 128, 0, 0, 36,
                                         seq_lens=[700, 256, 257]), 704),
    "g136": (lambda: wl.make_workload("g136", 2, 136, 1, 64, 0, 0, 35, seq_lens=[37, 130]), 0),
    "one_long": (lambda: wl.make_workload("one", 1, 8, 1, 128, 0, 0, 34, seq_lens=[6001]), 0),
}


@pytest.mark.parametrize("decay", [1.0, 0.5, 0.0])
@pytest.mark.parametrize("name", list(CASES))
def test_weights_and_output(name, decay):
    make, pt = CASES[name]
    W = make()
    G = harness.upload(W)
    ref_out = harness.gpu_step(W, G, partition_tokens=pt)
    old = _old(W, W.max_seq_len + 5)
    weights = old.clone()
    if decay == 0.0:
        weights[:] = float("nan")  # never read
        old = weights.clone()
    out = paged_attention_decode_weights(G.q, G.cache, G.tables, G.seq_lens, W.scale,
                                         W.max_seq_len, weights, decay=decay,
                                         partition_tokens=pt)
    assert pkv_check()[0] == 0
    assert torch.equal(out.view(torch.int16), ref_out.view(torch.int16))
    _check(W, G, weights, old, W.seq_lens, W.block_tables, decay)


@pytest.mark.parametrize("pt", [0, 64])
@pytest.mark.parametrize("make", [lambda: wl.llama8b_gqa(small=True),
                                  lambda: wl.make_workload(
                                      "fp8", 6, 10, 2, 64, 0, 0, 11, kv_dtype="fp8_e4m3",
                                      seq_lens=[1, 0, 17, 33, 200, 64])], ids=["bf16", "fp8"])
def test_with_new_tokens(make, pt):
    """The new token's write as in the decode step; its weight starts from 0
    although the row holds NaN there."""
    W = make()
    A, B = harness.upload(W), harness.upload(W)
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(W.batch, W.num_kv_heads, W.head_dim, generator=g).bfloat16().cuda()
            for _ in range(2))
    a = paged_attention_decode_step(A.q, k, v, A.cache, A.tables, A.seq_lens, W.scale,
                                    W.max_seq_len, partition_tokens=pt)
    old = _old(W, W.max_seq_len)
    fresh = [max(0, int(L) - 1) for L in W.seq_lens]
    for b, f in enumerate(fresh):
        old[b, :, f] = float("nan")
    weights = old.clone()
    b = paged_attention_decode_weights(B.q, B.cache, B.tables, B.seq_lens, W.scale, W.max_seq_len,
                                       weights, k_new=k, v_new=v, partition_tokens=pt)
    assert pkv_check()[0] == 0
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    for n in ("key_cache", "value_cache"):
        assert torch.equal(getattr(A.cache, n).view(torch.uint8),
                           getattr(B.cache, n).view(torch.uint8))
    # (rows stay as set up where the step's other writes would be: the
    # reference reads the cache as it is)
    _check(W, B, weights, old, W.seq_lens, W.block_tables, 1.0, fresh)


def test_several_new_tokens():
    W = wl.make_workload("tails", 4, 8, 2, 128, 0, 0, 12, seq_lens=[40, 33, 16, 5])
    A, B = harness.upload(W), harness.upload(W)
    for G in (A, B):  # sequence 2 brings no new token: its last one is written before
        harness.gpu_step(W, G)
    start = torch.tensor([0, 3, 20, 20, 25], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(4)
    k, v = (torch.randn(25, 2, 128, generator=g).bfloat16().cuda() for _ in range(2))
    a = paged_attention_decode_step(A.q, k, v, A.cache, A.tables, A.seq_lens, W.scale,
                                    W.max_seq_len, new_start_loc=start)
    old = _old(W, W.max_seq_len)
    weights = old.clone()
    b = paged_attention_decode_weights(B.q, B.cache, B.tables, B.seq_lens, W.scale, W.max_seq_len,
                                       weights, k_new=k, v_new=v, new_start_loc=start)
    assert pkv_check()[0] == 0
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    _check(W, B, weights, old, W.seq_lens, W.block_tables, 1.0, [37, 16, 16, 0])
    # a tail longer than its sequence: reported, its weights accumulate
    start2 = torch.tensor([0, 3, 20, 19, 25], dtype=torch.int32, device="cuda")
    weights = old.clone()
    paged_attention_decode_weights(B.q, B.cache, B.tables, B.seq_lens, W.scale, W.max_seq_len,
                                   weights, k_new=k, v_new=v, new_start_loc=start2)
    assert pkv_check()[0] == 5
    _check(W, B, weights, old, W.seq_lens, W.block_tables, 1.0, [37, 16, 16, 5])


def test_weights_sum_to_the_heads():
    """Each query head's weights sum to one, so a kv head's to its group."""
    W = wl.llama8b_gqa(small=True)
    G = harness.upload(W)
    harness.gpu_step(W, G)
    w = torch.empty(W.batch, W.num_kv_heads, W.max_seq_len, device="cuda")
    paged_attention_decode_weights(G.q, G.cache, G.tables, G.seq_lens, W.scale, W.max_seq_len, w,
                                   decay=0.0)
    valid = torch.arange(W.max_seq_len, device="cuda") < G.seq_lens[:, None]
    s = torch.where(valid[:, None], w, 0.0).double().sum(-1)
    # lifetime_ref.weights_tolerance with |q| . |k| scale below 24 (128 products
    # of N(0, 1) values average 7.2) and 400 tokens: 7.7e-4, below 2^-10
    assert ((s - W.group_size).abs() <= W.group_size * 2.0 ** -10).all()


@pytest.mark.parametrize("scale", [0.0, -0.3, 20.0])
def test_score_scales(scale):
    """Uniform weights, a reversed order, and peaks where most weights
    underflow to 0."""
    W = wl.make_workload("scales", 3, 8, 2, 64, 0, 0, 13, seq_lens=[70, 16, 1])
    G = harness.upload(W)
    harness.gpu_step(W, G)
    old = torch.zeros(3, 2, W.max_seq_len, device="cuda")
    weights = old.clone()
    paged_attention_decode_weights(G.q, G.cache, G.tables, G.seq_lens, scale, W.max_seq_len,
                                   weights, decay=0.0)
    got = weights.cpu().numpy().astype(np.float64)
    exp = _expect(W, G, W.seq_lens, W.block_tables, scale)
    for (b, h), (w, tol) in exp.items():
        tol = abs(tol)
        lim = (np.expm1(min(tol, 5.0))) * w + 1e-30
        assert (np.abs(got[b, h, :w.size] - w) <= lim + 2.0 ** -22 * w).all()
    assert pkv_check()[0] == 0


def test_bad_blocks_and_lengths():
    """Tokens of a block outside the pool gain nothing; a length above the
    host bound is clamped; both are reported, the rest stays right."""
    W = wl.make_workload("bad", 4, 8, 2, 128, 0, 0, 14, seq_lens=[64, 100, 30, 40])
    G = harness.upload(W)
    harness.gpu_step(W, G)
    tables = W.block_tables.copy()
    tables[0, 2] = 10 ** 6
    tables[2, 0] = -1
    old = _old(W, W.max_seq_len)
    for pt in (0, 16):
        weights = old.clone()
        paged_attention_decode_weights(G.q, G.cache, torch.from_numpy(tables).cuda(), G.seq_lens,
                                       W.scale, W.max_seq_len, weights, partition_tokens=pt)
        assert pkv_check()[0] == 5
        _check(W, G, weights, old, W.seq_lens, tables, 1.0)
    weights = old.clone()
    lens = np.array([64, 80, 30, 40], np.int32)  # sequence 1 clamped to 80
    paged_attention_decode_weights(G.q, G.cache, G.tables, G.seq_lens, W.scale, 80, weights)
    assert pkv_check() == (5, 1)
    _check(W, G, weights, old, lens, W.block_tables, 1.0)


def test_stale_rows_never_reach_the_weights():
    """Every slot outside the sequences holds NaN (the fixture's 0xFF)."""
    W = wl.make_workload("stale", 3, 8, 8, 64, 0, 0, 15, seq_lens=[1, 18, 47])
    G = harness.upload(W)
    harness.gpu_step(W, G)
    w = torch.zeros(3, 8, W.max_seq_len, device="cuda")
    paged_attention_decode_weights(G.q, G.cache, G.tables, G.seq_lens, W.scale, W.max_seq_len, w)
    assert bool(torch.isfinite(w).all())


@pytest.mark.parametrize("pt", [0, 16, 64])
@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8_e4m3"])
def test_nan_inside_a_sequence_is_not_hidden(kv_dtype, pt):
    """NaN in a cached key, in q, and in a cached value: NaN exactly where
    the formula has it."""
    W = wl.make_workload("nan", 4, 8, 2, 64, 0, 0, 17, kv_dtype=kv_dtype,
                         seq_lens=[40, 150, 90, 33])
    G = harness.upload(W)
    harness.gpu_step(W, G)
    ref_w = torch.zeros(4, 2, W.max_seq_len, device="cuda")
    ref_out = paged_attention_decode_weights(G.q, G.cache, G.tables, G.seq_lens, W.scale,
                                             W.max_seq_len, ref_w, partition_tokens=pt)
    nan = float("nan") if kv_dtype == "bf16" else 0x7F
    G.cache.key_cache[int(W.block_tables[0, 1]), 3, 1, 5] = nan     # sequence 0, head 1, token 19
    G.cache.value_cache[int(W.block_tables[1, 8]), 2, 0, 7] = nan   # sequence 1, head 0, token 130
    G.q[2, 6, 0] = float("nan")                                     # sequence 2, query head 6
    if kv_dtype == "bf16":  # an infinite key: +inf or -inf by the sign of q
        G.cache.key_cache[int(W.block_tables[3, 2]), 0, 0, 9] = float("inf")  # token 32
    w = torch.zeros_like(ref_w)
    out = paged_attention_decode_weights(G.q, G.cache, G.tables, G.seq_lens, W.scale,
                                         W.max_seq_len, w, partition_tokens=pt)
    assert pkv_check()[0] == 0
    bad = torch.zeros_like(ref_out, dtype=torch.bool)
    bad[0, 4:] = True
    bad[1, :4, 7] = True
    bad[2, 6] = True
    up = (G.q[3, :4, 9] > 0) if kv_dtype == "bf16" else torch.zeros(4, dtype=torch.bool).cuda()
    bad[3, :4] = up[:, None]
    assert torch.equal(torch.isnan(out), bad)
    same = ~bad
    same[3, :4] = same[3, :4] & (kv_dtype != "bf16")  # (rows that lost a token to -inf differ)
    assert torch.equal(out[same], ref_out[same])
    badw = torch.zeros_like(ref_w, dtype=torch.bool)
    badw[0, 1, :40] = True
    badw[2, 1, :90] = True
    badw[3, 0, :33] = bool(up.any())
    assert torch.equal(torch.isnan(w), badw)
    same = ~badw
    same[3, 0, :33] = same[3, 0, :33] & (kv_dtype != "bf16")
    assert torch.equal(w[same], ref_w[same])


def test_timeout_gives_no_weight():
    """The test hook stops sequence 1's warps: its weights are left without
    the stopped warps' tokens, the others are right."""
    W = wl.make_workload("timeout", 3, 8, 2, 128, 0, 0, 16, seq_lens=[50, 200, 90])
    G = harness.upload(W)
    harness.gpu_step(W, G)
    old = _old(W, W.max_seq_len)
    weights = old.clone()
    _native.lib().pkv_testing_fail_decode_sequence(1)
    try:
        out = paged_attention_decode_weights(G.q, G.cache, G.tables, G.seq_lens, W.scale,
                                             W.max_seq_len, weights)
        assert pkv_check() == (6, 1)
    finally:
        _native.lib().pkv_testing_fail_decode_sequence(-1)
    assert bool((out[1] == 0).all())
    assert torch.equal(weights[1], old[1])
    w2, o2 = weights.clone(), old.clone()
    lens = W.seq_lens.copy()
    lens[1] = 0
    _check(W, G, w2, o2, lens, W.block_tables, 1.0)


def test_empty_batch_and_zero_bound():
    W = wl.tiny_mha()
    G = harness.upload(W)
    harness.gpu_step(W, G)
    w = torch.full((W.batch, W.num_kv_heads, 4), 3.0, device="cuda")
    out = paged_attention_decode_weights(G.q[:0], G.cache, G.tables[:0], G.seq_lens[:0], W.scale,
                                         64, torch.empty(0, W.num_kv_heads, 64, device="cuda"))
    assert out.shape[0] == 0
    zero = torch.zeros_like(G.seq_lens)
    out = paged_attention_decode_weights(G.q, G.cache, G.tables, zero, W.scale, 0, w)
    assert pkv_check()[0] == 0
    assert bool((out == 0).all()) and bool((w == 3.0).all())


def test_workspace_contents_and_guards():
    """The result does not depend on what the workspace held; nothing past
    its declared size, and no weight row's end, is written."""
    W = wl.llama8b_gqa(small=True)
    G = harness.upload(W)
    harness.gpu_step(W, G)
    need = paged_attention_decode_weights_workspace_bytes(
        W.batch, W.num_heads, W.num_kv_heads, W.head_dim, W.max_seq_len, 64)
    res = []
    for fill in (0x00, 0xFF, 0xA5):
        ws = torch.full((need + 4096,), fill, dtype=torch.uint8, device="cuda")
        w = torch.zeros(W.batch, W.num_kv_heads, W.max_seq_len, device="cuda")
        out = paged_attention_decode_weights(G.q, G.cache, G.tables, G.seq_lens, W.scale,
                                             W.max_seq_len, w, partition_tokens=64,
                                             workspace=ws[:need])
        assert bool((ws[need:] == fill).all())
        res.append((out.clone(), w))
    for out, w in res[1:]:
        assert torch.equal(out, res[0][0]) and torch.equal(w, res[0][1])


def test_binding_refusals():
    W = wl.tiny_mha()
    G = harness.upload(W)
    w = torch.zeros(W.batch, W.num_kv_heads, W.max_seq_len, device="cuda")
    ok = dict(q=G.q, cache=G.cache, block_tables=G.tables, seq_lens=G.seq_lens, scale=W.scale,
              max_seq_len=W.max_seq_len, weights=w)

    def bad(exc, **kw):
        with pytest.raises(exc):
            paged_attention_decode_weights(**{**ok, **kw})
    k = torch.zeros(W.batch, W.num_kv_heads, W.head_dim, dtype=torch.bfloat16, device="cuda")
    bad(TypeError, weights=w.double())
    bad(ValueError, weights=w[:, :, :-1].contiguous())
    bad(ValueError, weights=w[:, :1].contiguous())
    bad(ValueError, weights=w[:, :, ::2])
    bad(ValueError, max_seq_len=W.max_seq_len + 1)
    bad(TypeError, k_new=k)
    bad(ValueError, k_new=k[1:], v_new=k[1:])
    bad(ValueError, out=G.q[:1])
    bad(PagedKVError, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    bad(PagedKVError, decay=float("nan"))
    assert bool((w == 0).all())


def _many(B, Hq, Hkv, D, lens, kv_dtype="bf16", seed=0):
    """Inputs of a large batch, made on the GPU: (cache, q, tables, lens)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    nb = [(int(n) + 15) // 16 for n in lens]
    total = sum(nb) + 3
    shape = (total, 16, Hkv, D)
    x = [torch.empty(shape, device="cuda").normal_(generator=g) for _ in range(2)]
    if kv_dtype == "bf16":
        cache = PagedKVCache(x[0].bfloat16(), x[1].bfloat16())
    else:
        s = 8.0 / 448
        c = [(v / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) for v in x]
        cache = PagedKVCache(c[0], c[1], kv_dtype, s, s)
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32).cpu().numpy()
    tables = np.full((B, max(1, max(nb))), -1, np.int32)
    at = 0
    for b, n in enumerate(nb):
        tables[b, :n] = order[at:at + n]
        at += n
    q = torch.empty(B, Hq, D, device="cuda").normal_(generator=g).bfloat16()
    return cache, q, tables, np.asarray(lens, np.int32)


def _exact_weights(cache, q, tables, lens, scale):
    """(summed weights [B, Hkv, S] float64, relative tolerance), on the GPU."""
    B, Hq, D = q.shape
    Hkv, S = cache.num_kv_heads, int(max(lens))
    kc = cache.key_cache.double() if cache.kv_dtype == "bf16" else \
        cache.key_cache.view(torch.float8_e4m3fn).double() * float(np.float32(cache.k_scale))
    w = torch.zeros(B, Hkv, S, dtype=torch.float64, device="cuda")
    bound = 0.0
    for b, L in enumerate(lens):
        L = int(L)
        if L == 0:
            continue
        t = torch.from_numpy(tables[b, :(L + 15) // 16].astype(np.int64)).cuda()
        k = kc[t].flatten(0, 1)[:L]
        for h in range(Hkv):
            qh = q[b, h * (Hq // Hkv):(h + 1) * (Hq // Hkv)].double()
            w[b, h, :L] = torch.softmax(scale * qh @ k[:, h].t(), -1).sum(0)
            bound = max(bound, float((scale * qh.abs() @ k[:, h].abs().t()).max()))
    return w, ref.weights_tolerance(D, int(max(lens)), Hq // Hkv, bound)


LARGE = {
    # batch, q heads, kv heads, head_dim, longest, partition, cache
    "g4": (80, 32, 8, 128, 2500, 1024, "bf16"),
    "g8_ragged": (70, 64, 8, 64, 2000, 528, "bf16"),
    "g5_fp8": (90, 40, 8, 64, 1800, 640, "fp8_e4m3"),
    "g1_auto": (130, 8, 8, 64, 2100, 0, "bf16"),
    "g2_two_heads": (300, 4, 2, 64, 1700, 544, "bf16"),
}


@pytest.mark.parametrize("name", list(LARGE))
def test_large_batches(name):
    """Many waves of CTAs, several partitions a sequence, runs of several
    chunks: every token's weight is right, none is added twice or left out,
    whatever the workspace held, and calls repeat to the bit."""
    B, Hq, Hkv, D, longest, pt, kv_dtype = LARGE[name]
    rng = np.random.default_rng(B)
    lens = rng.integers(0, longest + 1, B)
    lens[0], lens[3], lens[-1] = 0, longest, longest
    cache, q, tables, lens = _many(B, Hq, Hkv, D, lens, kv_dtype)
    gt, gl = torch.from_numpy(tables).cuda(), torch.from_numpy(lens).cuda()
    scale = D ** -0.5
    w64, tol = _exact_weights(cache, q, tables, lens, scale)
    S = longest + 7
    need = paged_attention_decode_weights_workspace_bytes(B, Hq, Hkv, D, longest, pt)
    plain = paged_attention_decode(q, cache, gt, gl, scale, longest, partition_tokens=pt)
    first = None
    for fill in (0, 0xFF, 0x5A, None, None):
        if fill is not None:
            ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        w = torch.ones(B, Hkv, S, device="cuda")
        out = paged_attention_decode_weights(q, cache, gt, gl, scale, longest, w, decay=0.5,
                                             partition_tokens=pt, workspace=ws)
        assert pkv_check()[0] == 0
        assert torch.equal(out.view(torch.int16), plain.view(torch.int16))
        if first is None:
            first = w
            t = torch.arange(S, device="cuda")
            valid = (t < gl[:, None])[:, None].expand_as(w)
            assert bool((w[~valid] == 1.0).all())
            got = w[:, :, :w64.shape[2]].double()
            want = torch.where(valid[:, :, :w64.shape[2]], w64 + 0.5, 1.0)
            lim = tol * w64 + 2.0 ** -23 * want
            assert bool(((got - want).abs() <= lim).all())
        assert torch.equal(w, first)


def test_replayed_with_other_queries_and_lengths():
    """One graph replayed with other queries and lengths in its inputs: nothing
    of an earlier replay is left in the result."""
    B, Hq, Hkv, D, longest, pt = 80, 32, 8, 64, 2200, 1024
    rng = np.random.default_rng(77)
    cache, q, tables, lens = _many(B, Hq, Hkv, D, np.full(B, longest), seed=5)
    gt = torch.from_numpy(tables).cuda()
    gl = torch.from_numpy(lens).cuda()
    need = paged_attention_decode_weights_workspace_bytes(B, Hq, Hkv, D, longest, pt)
    ws = torch.full((need,), 0xA5, dtype=torch.uint8, device="cuda")
    w, out = torch.zeros(B, Hkv, longest, device="cuda"), torch.empty_like(q)

    def step():
        paged_attention_decode_weights(q, cache, gt, gl, 0.125, longest, w, decay=0.0, out=out,
                                       partition_tokens=pt, workspace=ws)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            step()
    torch.cuda.synchronize()
    for _ in range(4):
        q.normal_()
        new = rng.integers(1, longest + 1, B).astype(np.int32)
        gl.copy_(torch.from_numpy(new))
        w.fill_(-1.0)
        g.replay()
        got, o = w.clone(), out.clone()
        w2 = torch.full_like(w, -1.0)
        o2 = paged_attention_decode_weights(q, cache, gt, gl, 0.125, longest, w2, decay=0.0,
                                            partition_tokens=pt)
        torch.cuda.synchronize()
        assert torch.equal(got, w2) and torch.equal(o.view(torch.int16), o2.view(torch.int16))
    assert pkv_check()[0] == 0


@pytest.mark.parametrize("Hq,D,kv_dtype", [(64, 128, "bf16"), (40, 64, "fp8_e4m3"),
                                           (24, 128, "bf16"), (88, 64, "bf16")])
def test_the_bound_does_not_change_the_weights(Hq, D, kv_dtype):
    """The same sequences under a bound that lets their scores fit in L2 and
    under one that does not: weights bit for bit, and the workspace is used
    again by the next call."""
    B, Hkv, longest, pt = 64, 8, 1100, 1024
    lens = [1, 0, 16, 17, 1024, 1025, 1099] + list(range(40, 40 + 18 * (B - 8), 18)) + [longest]
    cache, q, tables, lens = _many(B, Hq, Hkv, D, lens, kv_dtype, seed=9)
    gt, gl = torch.from_numpy(tables).cuda(), torch.from_numpy(lens).cuda()
    group = Hq // Hkv
    units = (group + 7) // 8
    heads = (min(8, group) + 1) // 2 * 2
    results = []
    for megabytes in (0, 100):
        tokens = max(longest, (megabytes << 20) // (B * Hkv * units * heads * 4) + 1)
        need = paged_attention_decode_weights_workspace_bytes(B, Hq, Hkv, D, tokens, pt)
        ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
        w = torch.zeros(B, Hkv, tokens, device="cuda")
        for _ in range(3):
            out = paged_attention_decode_weights(q, cache, gt, gl, 0.125, tokens, w, decay=0.5,
                                                 partition_tokens=pt, workspace=ws)
        plain = paged_attention_decode(q, cache, gt, gl, 0.125, max_seq_len=tokens,
                                       partition_tokens=pt)
        assert torch.equal(out.view(torch.int16), plain.view(torch.int16))
        assert not bool(w[:, :, longest:].any())
        results.append(w[:, :, :longest].clone())
    assert torch.equal(results[0], results[1])
    sums = results[0].double().sum(-1).cpu().numpy()
    # 1 + 1/2 + 1/4 of a softmax a query head; statistics and weights come from
    # the same scores, so what is left is the binary32 sum of at most 1100
    # terms (1100 * 2^-24 < 2^-13) and a few roundings and exponentials a term
    want = 1.75 * group * (lens > 0)
    assert np.abs(sums - want[:, None]).max() <= 1.75 * group * 2.0 ** -10
    assert pkv_check()[0] == 0
