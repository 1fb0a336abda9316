"""paged_kv_evict against a plain per-sequence choice and copy: kept
positions, moved bytes, weights and lengths are all exact."""
import numpy as np
import pytest
import torch

import lifetime_ref as ref
from paged_kv_cache_48_gb300 import (PagedKVCache, PagedKVError, paged_kv_evict,
                                     paged_kv_evict_workspace_bytes, pkv_check)

pytestmark = pytest.mark.gpu


class State:
    """A pool of random bytes with shuffled tables, random weights."""

    def __init__(self, lens, Hkv=2, D=64, kv_dtype="bf16", seed=0, dst_lens=None, width=None,
                 spare=3):
        rng = np.random.default_rng(seed)
        self.lens = np.asarray(lens, np.int32)
        B = self.lens.size
        nb = [(max(0, int(n)) + 15) // 16 for n in lens]
        db = [(int(n) + 15) // 16 for n in (dst_lens if dst_lens is not None else [])]
        total = sum(nb) + sum(db) + spare
        order = rng.permutation(total).astype(np.int32)

        def table(counts, at):
            t = np.full((B, max(1, max(counts, default=1))), -1, np.int32)
            for b, n in enumerate(counts):
                t[b, :n] = order[at:at + n]
                at += n
            return t
        self.tables = table(nb, 0)
        self.dst = table(db, sum(nb)) if db else None
        e = 2 if kv_dtype == "bf16" else 1
        self.pool = [rng.integers(0, 256, (total, 16, Hkv, D * e), dtype=np.uint8)
                     for _ in range(2)]
        elt = torch.bfloat16 if kv_dtype == "bf16" else torch.uint8
        dev = [torch.from_numpy(p).view(elt).cuda() for p in self.pool]
        self.cache = PagedKVCache(dev[0], dev[1], kv_dtype, 0.5 if e == 1 else 1.0,
                                  0.5 if e == 1 else 1.0)
        S = width if width is not None else max(1, int(self.lens.max(initial=1)))
        self.w = np.exp(1.5 * rng.standard_normal((B, Hkv, S))).astype(np.float32)
        self.rng, self.B, self.Hkv, self.S = rng, B, Hkv, S

    def expect(self, keep, sink, recent, per_head, in_place, dst_w, bad=()):
        pools = [p.copy() for p in self.pool]
        old = [p.copy() for p in self.pool]
        dst = self.tables if in_place else self.dst
        w = self.w.copy() if dst_w is None else dst_w.copy()
        lens = self.lens.copy()
        kept = [[[] for _ in range(self.Hkv if per_head else 1)] for _ in range(self.B)]
        for b in range(self.B):
            if b in bad:
                continue
            L, n = int(self.lens[b]), min(int(self.lens[b]), int(keep[b]))
            lens[b] = n
            w[b, :, n:min(L, w.shape[2])] = 0.0
            for h in range(self.Hkv):
                rank = self.w[b, h] if per_head else ref.heads_sum(self.w[b])
                at = ref.evict_choice(rank, L, n, sink, recent)
                kept[b][h if per_head else 0] = at
                w[b, h, :n] = self.w[b, h, at]
                for i, t in enumerate(at):
                    s, d = self.tables[b, t // 16], dst[b, i // 16]
                    ok = 0 <= s < pools[0].shape[0] and 0 <= d < pools[0].shape[0]
                    for p, o in zip(pools, old):
                        if ok:
                            p[d, i % 16, h] = o[s, t % 16, h]
        return pools, w, lens, kept

    def run(self, keep, sink=0, recent=0, per_head=True, in_place=True, dst_w=None, bad=(),
            max_keep=None, alias=False, status=0, stream=None):
        keep = np.asarray(keep, np.int32)
        max_keep = int(max(0, keep.max(initial=0))) if max_keep is None else max_keep
        pools, w, lens, kept = self.expect(keep, sink, recent, per_head, in_place, dst_w, bad)
        c = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
        gw, gl = c(self.w), c(self.lens)
        gd = None if dst_w is None else c(dst_w)
        gk = torch.full((self.B, self.Hkv if per_head else 1, max_keep), 77, dtype=torch.int32,
                        device="cuda")
        need = paged_kv_evict_workspace_bytes(self.B, self.Hkv, self.S, max_keep)
        ws = torch.full((need + 1024,), 0xA5, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        new = paged_kv_evict(self.cache, c(self.tables), gl, gw, c(keep), max_keep, sink=sink,
                             recent=recent, per_head=per_head,
                             dst_tables=None if in_place else c(self.dst), dst_weights=gd,
                             new_seq_lens=gl if alias else None, kept=gk, workspace=ws[:need],
                             stream=stream)
        st = pkv_check(stream)
        assert st[0] == status, st
        assert new is gl if alias else torch.equal(gl, c(self.lens))
        assert np.array_equal(new.cpu().numpy(), lens)
        assert bool((ws[need:] == 0xA5).all())
        got = gk.cpu().numpy()
        for b in range(self.B):
            for h in range(got.shape[1]):
                row = np.full(max_keep, -1)
                row[:len(kept[b][h])] = kept[b][h]
                assert np.array_equal(got[b, h], row), (b, h)
        gw2 = gw if gd is None else gd
        assert np.array_equal(gw2.cpu().numpy().view(np.uint32), w.view(np.uint32))
        if gd is not None:
            assert np.array_equal(gw.cpu().numpy().view(np.uint32), self.w.view(np.uint32))
        for p, t in zip(pools, (self.cache.key_cache, self.cache.value_cache)):
            assert np.array_equal(t.view(torch.uint8).cpu().numpy().reshape(p.shape), p)
        return st


LENS = [0, 1, 15, 16, 17, 100, 333, 64]
KEEP = [5, 1, 16, 9, 17, 33, 100, 0]


# new_seq_lens being seq_lens takes the two-launch form at every size; with
# few tokens kept and lengths of their own, one launch does it all.
ALIAS = pytest.mark.parametrize("alias", [False, True], ids=["one_launch", "two_launches"])


@ALIAS
@pytest.mark.parametrize("per_head", [True, False])
@pytest.mark.parametrize("kv_dtype,D", [("bf16", 64), ("bf16", 128), ("fp8_e4m3", 64),
                                        ("fp8_e4m3", 128)])
@pytest.mark.parametrize("in_place", [True, False])
def test_ragged(in_place, kv_dtype, D, per_head, alias):
    n = np.minimum(LENS, KEEP)
    s = State(LENS, 3, D, kv_dtype, seed=D, dst_lens=None if in_place else n)
    s.run(KEEP, sink=2, recent=5, per_head=per_head, in_place=in_place, alias=alias)


@ALIAS
@pytest.mark.parametrize("sink,recent", [(0, 0), (1000, 0), (0, 1000), (20, 30), (3, 47), (50, 50)])
def test_protected_tokens(sink, recent, alias):
    s = State([50, 200, 51, 49], seed=sink + recent)
    s.run([50, 50, 50, 50], sink=sink, recent=recent, alias=alias)


@ALIAS
@pytest.mark.parametrize("in_place", [True, False])
def test_separate_weights(in_place, alias):
    lens, keep = [90, 20, 300, 7], [40, 30, 123, 7]
    s = State(lens, seed=3, dst_lens=None if in_place else np.minimum(lens, keep))
    g = np.random.default_rng(1).random((4, 2, 130)).astype(np.float32)  # narrower than weights
    s.run(keep, sink=1, recent=2, in_place=in_place, dst_w=g, alias=alias)
    s = State(lens, seed=3, dst_lens=None if in_place else np.minimum(lens, keep))
    g = np.random.default_rng(1).random((4, 2, 500)).astype(np.float32)  # wider
    s.run(keep, sink=1, recent=2, in_place=in_place, dst_w=g, alias=alias)


@ALIAS
@pytest.mark.parametrize("per_head", [True, False])
def test_ties_zeros_and_special_values(per_head, alias):
    """Equal weights go by position; NaN below -inf below all; -0 ties 0;
    subnormals are ordered."""
    s = State([400, 400, 400, 400, 64], 4, seed=5)
    s.w[0] = 0.25
    s.w[1] = np.float32(0.0)
    s.w[1, :, ::3] = np.float32(-0.0)
    s.w[2, :, ::2] = np.nan
    s.w[2, :, 5::7] = np.inf
    s.w[2, :, 4::9] = -np.inf
    s.w[3] = s.rng.integers(0, 6, s.w[3].shape).astype(np.float32)
    s.w[4, :, :64] = (s.rng.integers(0, 4, (4, 64)) * 2.0 ** -149).astype(np.float32)
    s.run([100, 101, 250, 77, 20], sink=4, recent=9, per_head=per_head, alias=alias)


@pytest.mark.parametrize("per_head", [True, False])
def test_negative_weights(per_head):
    s = State([300, 40], 2, seed=6)
    s.w = (s.rng.standard_normal(s.w.shape) * 3).astype(np.float32)
    s.run([90, 39], per_head=per_head)


@pytest.mark.parametrize("L,keep", [(5000, 4999), (5000, 1), (20000, 7777), (70001, 2049),
                                    (131072, 60000), (150001, 20000)])
@pytest.mark.parametrize("per_head", [True, False])
def test_long(L, keep, per_head):
    s = State([L, L // 3], 2, 64, "fp8_e4m3", seed=L, dst_lens=[keep, min(keep, L // 3)])
    s.run([keep, keep], sink=4, recent=min(64, keep // 2), per_head=per_head, in_place=False)


@pytest.mark.parametrize("kv_dtype,D", [("bf16", 128), ("fp8_e4m3", 64)])
@pytest.mark.parametrize("B,Hkv", [(6, 4), (2, 3)])
def test_in_place_by_clusters(B, Hkv, kv_dtype, D):
    """Planes walked by clusters of CTAs: few of them, and a middle count;
    chunks where nothing, something and everything moves."""
    lens = [5000 - 311 * b for b in range(B)]
    s = State(lens, Hkv, D, kv_dtype, seed=B)
    s.w[0, :, :1500] += 1e6  # a long run that stays where it is
    s.run([4000 - 500 * b for b in range(B)], sink=1, recent=7)


@pytest.mark.parametrize("Hkv", [8, 9])
@pytest.mark.parametrize("in_place", [True, False])
def test_borders_of_the_one_launch_form(in_place, Hkv):
    """256 and 257 tokens kept, rows of 4096 and 4097 keys, one choice for all
    heads: either side of the rule gives the same."""
    for L, keep in ((4096, 256), (4097, 256), (1000, 257), (256, 256), (257, 255)):
        n = [keep, min(keep, 300)]
        s = State([L, 300], Hkv, 64, seed=L + keep, dst_lens=None if in_place else n)
        s.run(n, sink=3, recent=11, per_head=Hkv == 8, in_place=in_place)
    s = State([4096, 300], 2, 128, seed=31, dst_lens=None if in_place else [256, 256])
    s.run([256, 256], sink=3, recent=11, in_place=in_place)


def test_long_in_place():
    s = State([30000, 9000], 2, 128, seed=8)
    s.run([12345, 8999], sink=4, recent=100)


def test_more_keys_than_a_cluster_holds():
    """150001 tokens: the keys past 8 x 16384 are read again in every round,
    ties among them included."""
    s = State([150001], 1, 64, "fp8_e4m3", seed=30, dst_lens=[70000])
    s.w = (s.rng.integers(0, 9, s.w.shape) / 8.0).astype(np.float32)
    s.run([70000], sink=1, recent=2, in_place=False)


def test_clustered_weights():
    """Keys that share their leading 24 bits, and one bin holding nearly all."""
    s = State([6000], 1, seed=9)
    s.w[0, 0] = (1.0 + s.rng.integers(0, 200, 6000) * 2.0 ** -23).astype(np.float32)
    s.w[0, 0, ::50] = 3.0
    s.run([2500], recent=10)


def test_new_lens_may_be_the_lens():
    s = State([100, 50, 10], seed=10)
    s.run([30, 60, 10], alias=True)


def test_shared_prefix_into_own_blocks():
    """Two sequences sharing their first blocks are cut into blocks of their
    own; the shared blocks stay as they were."""
    s = State([80, 96], seed=11, dst_lens=[33, 40])
    s.tables[1, :3] = s.tables[0, :3]
    s.run([33, 40], sink=2, recent=4, in_place=False)


def test_max_keep_above_and_kept_zero():
    s = State([40, 3], seed=12)
    s.run([10, 10], max_keep=64)
    s = State([40, 3], seed=13)
    s.run([0, 0], max_keep=0)


@ALIAS
def test_range_errors_leave_the_sequence_alone(alias):
    lens = [40, 60, 50, 30, 20]
    s = State(lens, seed=14)
    s.run([10, -1, 20, 30, 20], bad=(1,), status=5, alias=alias)    # negative keep
    s = State(lens, seed=15)
    s.run([10, 45, 20, 30, 20], max_keep=40, bad=(1,), status=5, alias=alias)    # n past max_keep
    s = State(lens, seed=16, width=55)                              # past the weights row
    s.run([10, 20, 20, 30, 20], bad=(1,), status=5, alias=alias)
    s = State(lens, seed=17)
    s.lens[2] = -3
    s.run([10, 20, 20, 30, 20], bad=(2,), status=5, alias=alias)
    s = State(lens, seed=18)
    s.lens[0] = 16 * s.tables.shape[1] + 1                          # past the table
    s.w = np.pad(s.w, ((0, 0), (0, 0), (0, 20)))
    s.S = s.w.shape[2]
    s.run([10, 20, 20, 30, 20], bad=(0,), status=5, alias=alias)
    s = State([40, 60], seed=19, dst_lens=[16, 16])                 # past dst_tables
    s.run([10, 17], in_place=False, bad=(1,), status=5, alias=alias)
    s = State([40, 60], seed=20)                                    # past dst_weights
    s.run([10, 17], dst_w=np.ones((2, 2, 16), np.float32), bad=(1,), status=5, alias=alias)


@ALIAS
def test_bad_blocks_are_skipped(alias):
    s = State([100, 80], seed=21)
    s.tables[0, 3] = 10 ** 6
    s.tables[1, 0] = -1
    s.run([40, 30], recent=20, status=5, alias=alias)
    s = State([100, 80], seed=22, dst_lens=[40, 30])
    s.tables[0, 6] = -5
    s.dst[1, 1] = 10 ** 6
    s.run([40, 30], recent=20, in_place=False, status=5, alias=alias)


def test_deterministic():
    outs = []
    for _ in range(2):
        s = State([3000, 2000], 4, 128, seed=23)
        s.w[:] = s.rng.integers(0, 5, s.w.shape)
        s.run([900, 901], sink=3, recent=50)
        outs.append(s.cache.key_cache.clone())
    assert torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16))


def test_binding_refusals():
    s = State([40, 20], seed=24)
    c = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    ok = dict(cache=s.cache, block_tables=c(s.tables), seq_lens=c(s.lens), weights=c(s.w),
              keep=c(np.array([10, 10], np.int32)), max_keep=10)

    def bad(exc, **kw):
        with pytest.raises(exc):
            paged_kv_evict(**{**ok, **kw})
    bad(TypeError, keep=[10, 10])
    bad(TypeError, keep=ok["keep"].long())
    bad(TypeError, weights=ok["weights"].half())
    bad(ValueError, weights=ok["weights"][:, :1].contiguous())
    bad(ValueError, weights=ok["weights"][:, :, ::2])
    bad(ValueError, keep=ok["keep"][:1])
    bad(ValueError, dst_tables=ok["block_tables"][:1])
    bad(ValueError, dst_tables=ok["block_tables"][:, :0].contiguous())
    bad(ValueError, dst_weights=ok["weights"][:, :, :0].contiguous())
    bad(ValueError, kept=torch.zeros(2, 1, 10, dtype=torch.int32, device="cuda"))
    bad(ValueError, new_seq_lens=torch.zeros(3, dtype=torch.int32, device="cuda"))
    bad(PagedKVError, dst_weights=ok["weights"])      # over the weights still to be read
    bad(PagedKVError, new_seq_lens=ok["keep"])
    bad(PagedKVError, sink=-1)
    bad(PagedKVError, max_keep=-1)
    bad(PagedKVError, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert torch.equal(ok["weights"], c(s.w))
