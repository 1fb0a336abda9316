"""Cases of the cache-lifetime operators: the rotary write, decode attention
with running attention weights, and eviction by those weights.

Each operator has a plain form in elementary torch operations (32-bit
arithmetic, one rounding at the end) and the framework's own call; `exact`
computes the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

BLOCK = 16
F8 = torch.float8_e4m3fn


def listed():
    return [
        # one token of one sequence: the latency of the write in a decode step
        dict(name="rope_one_token", op="rope", tokens=1, heads=32, kv_heads=8, dim=128,
             rotary=128, sections="64", dealt=False, adjacent=False, fp8=False, fused=True,
             base=500000.0, start=40000),
        # a decode step of 128 sequences into an E4M3 cache
        dict(name="rope_step_fp8", op="rope", tokens=128, heads=40, kv_heads=8, dim=128,
             rotary=128, sections="24,20,20", dealt=True, adjacent=False, fp8=True, fused=True,
             base=1000000.0, start=100000),
        # an odd chunk of a small model: half of each head rotates, in
        # adjacent pairs, by image coordinates
        dict(name="rope_chunk_odd", op="rope", tokens=1237, heads=8, kv_heads=8, dim=64,
             rotary=32, sections="8,8", dealt=False, adjacent=True, fp8=False, fused=False,
             base=10000.0, start=0),
        # an 8K prompt chunk of text and image tokens, time / height / width
        dict(name="rope_chunk_8k", op="rope", tokens=8192, heads=32, kv_heads=8, dim=128,
             rotary=128, sections="16,24,24", dealt=False, adjacent=False, fp8=False, fused=True,
             base=1000000.0, start=6000),
        # a few short sequences: the latency of a step
        dict(name="weights_short", op="weights", batch=4, heads=8, kv_heads=8, dim=64, lo=1,
             hi=64, fp8=False, append=True, decay=1.0),
        # a decode step of 64 sequences, grouped queries
        dict(name="weights_batch64", op="weights", batch=64, heads=32, kv_heads=8, dim=128,
             lo=512, hi=4096, fp8=False, append=True, decay=1.0),
        # a decode step over an E4M3 cache, groups of five, decayed totals
        dict(name="weights_fp8", op="weights", batch=128, heads=40, kv_heads=8, dim=128, lo=1024,
             hi=8192, fp8=True, append=False, decay=0.98),
        # few long contexts, split over their length
        dict(name="weights_long", op="weights", batch=8, heads=64, kv_heads=8, dim=128, lo=32768,
             hi=131072, fp8=False, append=False, decay=1.0),
        # a few short sequences, some of them below their budget
        dict(name="evict_short", op="evict", batch=4, kv_heads=8, dim=64, lo=1, hi=100, fp8=False,
             keep=48, sink=4, recent=16, per_head=True),
        # a batch of 64 cut to 1024 tokens, each kv head keeping its own
        dict(name="evict_batch64", op="evict", batch=64, kv_heads=8, dim=128, lo=512, hi=4096,
             fp8=False, keep=1024, sink=4, recent=256, per_head=True),
        # an E4M3 cache, one choice for all heads of a sequence
        dict(name="evict_fp8_shared", op="evict", batch=128, kv_heads=8, dim=128, lo=1024,
             hi=8192, fp8=True, keep=2000, sink=16, recent=501, per_head=False),
        # few long contexts cut to an eighth of the longest
        dict(name="evict_long", op="evict", batch=8, kv_heads=8, dim=128, lo=32768, hi=131072,
             fp8=False, keep=16384, sink=64, recent=1024, per_head=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "weights", "evict"))
    kv, group = rng.choice((1, 2, 3, 8, 8)), rng.choice((1, 2, 3, 4, 5, 7, 8, 12))
    dim = rng.choice((64, 128))
    if op == "rope":
        rotary = 16 * rng.randint(1, dim // 16)
        axes = rng.randint(1, 4)
        dealt = axes > 1 and rng.random() < 0.5
        pairs = rotary // 2
        if dealt:  # every axis but the first gets at most its share of the turns
            rest = [rng.randint(1, max(1, pairs // axes)) for _ in range(axes - 1)]
        else:
            rest = [rng.randint(0, pairs // axes) for _ in range(axes - 1)]
        sections = [pairs - sum(rest)] + rest
        return dict(op=op, tokens=_log(rng, 1, 8192), heads=kv * group, kv_heads=kv, dim=dim,
                    rotary=rotary, sections=",".join(map(str, sections)), dealt=dealt,
                    adjacent=rng.random() < 0.5, fp8=rng.random() < 0.5, fused=rng.random() < 0.5,
                    base=rng.choice((10000.0, 500000.0, 1000000.0)),
                    start=_log(rng, 1, 1000000))
    hi = _log(rng, 16, 100000)
    lo = rng.randint(max(1, hi // 8), hi)
    batch = max(1, min(_log(rng, 1, 128), 500000 // hi))
    if op == "weights":
        return dict(op=op, batch=batch, heads=kv * group, kv_heads=kv, dim=dim, lo=lo, hi=hi,
                    fp8=rng.random() < 0.5, append=rng.random() < 0.5,
                    decay=rng.choice((0.0, 0.9, 1.0)))
    keep = rng.randint(1, hi)
    return dict(op=op, batch=batch, kv_heads=kv, dim=dim, lo=lo, hi=hi, fp8=rng.random() < 0.5,
                keep=keep, sink=rng.randint(0, 8), recent=rng.randint(0, keep),
                per_head=rng.random() < 0.6)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _lens(case):
    """Lengths spread evenly over [lo, hi]; their order comes from the seed."""
    n, lo, hi = case["batch"], case["lo"], case["hi"]
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _keep(case):
    """The sequences' budgets, in the order of _lens: not all alike."""
    n = case["keep"]
    return [n if i % 4 else max(1, n - i) for i in range(case["batch"])]


def _values(gen, shape, fp8, scale):
    """Cache contents: N(0, 1) in bf16, or its E4M3 codes under `scale`."""
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    return (x / scale).to(F8).view(torch.uint8) if fp8 else x


def _sections(case):
    return [int(s) for s in case["sections"].split(",")]


def _prepare_rope(case, gen, s):
    T, H, K, D = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
    A = len(_sections(case))
    if case["fused"]:  # views of one projection's output
        qkv = torch.empty(T, (H + 2 * K) * D, dtype=torch.bfloat16, device="cuda")
        qkv.normal_(generator=gen)
        s["q"] = qkv[:, :H * D].view(T, H, D)
        s["k"] = qkv[:, H * D:(H + K) * D].view(T, K, D)
        s["v"] = qkv[:, (H + K) * D:].view(T, K, D)
    else:
        for n, h in (("q", H), ("k", K), ("v", K)):
            s[n] = torch.empty(T, h, D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    # text tokens advance every axis together; every second run of 256 tokens
    # is a 16 x 16 grid at one time
    t = torch.arange(T, device="cuda")
    run, i = t // 256, t % 256
    text = run % 2 == 0
    at = case["start"] + torch.where(text, t, run * 256)
    axes = [at, torch.where(text, at, at + i // 16), torch.where(text, at, at + i % 16), at]
    s["positions"] = torch.stack(axes[:A]).to(torch.int32).contiguous()
    blocks = max(4, (T * 6 // 5 + BLOCK - 1) // BLOCK)
    s["slots"] = torch.randperm(blocks * BLOCK, generator=gen, device="cuda")[:T]
    s["kc"] = _values(gen, (blocks, BLOCK, K, D), case["fp8"], s["k_scale"])
    s["vc"] = _values(gen, (blocks, BLOCK, K, D), case["fp8"], s["v_scale"])
    s["q_out"] = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda")


def _tables(gen, lens, first, spare):
    """Shuffled blocks from `first` on for sequences of these lengths; returns
    the table and the number of blocks taken (with `spare` unused ones)."""
    need = [(n + BLOCK - 1) // BLOCK for n in lens]
    total = sum(need) + spare
    order = (torch.randperm(total, generator=gen, device="cuda") + first).to(torch.int32)
    width = max(1, max(need))
    at = torch.tensor([sum(need[:i]) for i in range(len(need))], device="cuda")[:, None]
    j = torch.arange(width, device="cuda")[None]
    count = torch.tensor(need, device="cuda")[:, None]
    return torch.where(j < count, order[(at + j).clamp(max=total - 1)], -1).contiguous(), total


def _prepare_cached(case, gen, s):
    B, K, D = case["batch"], case["kv_heads"], case["dim"]
    order = torch.randperm(B, generator=gen, device="cuda").tolist()
    lens = [_lens(case)[i] for i in order]
    s["lens_host"] = lens
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["tables"], blocks = _tables(gen, lens, 0, max(1, sum(lens) // (8 * BLOCK)))
    s["weights"] = torch.empty(B, K, max(lens), device="cuda").normal_(generator=gen)
    # running totals of some steps: few large, many small
    s["weights"].mul_(1.5).exp_().mul_(8.0 / max(lens))
    if case["op"] == "weights":
        H = case["heads"]
        s["q"] = torch.empty(B, H, D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
        s["k_new"] = torch.empty(B, K, D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
        s["v_new"] = torch.empty(B, K, D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
        s["out"] = torch.empty_like(s["q"])
    else:
        keep = [_keep(case)[i] for i in order]
        s["keep"] = torch.tensor(keep, dtype=torch.int32, device="cuda")
        new = [min(a, b) for a, b in zip(lens, keep)]
        s["first"] = blocks
        s["dst"], more = _tables(gen, new, blocks, 0)
        blocks += more
        # tokens that no query has attended yet: equal totals of zero
        s["weights"][torch.rand(s["weights"].shape, generator=gen, device="cuda") < 0.02] = 0.0
        s["dst_weights"] = torch.zeros(B, K, max(lens), device="cuda")
        s["new_lens"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        heads = K if case["per_head"] else 1
        s["kept"] = torch.empty(B, heads, case["keep"], dtype=torch.int32, device="cuda")
    s["kc"] = _values(gen, (blocks, BLOCK, K, D), case["fp8"], s["k_scale"])
    s["vc"] = _values(gen, (blocks, BLOCK, K, D), case["fp8"], s["v_scale"])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=case, k_scale=1.0, v_scale=1.0)
    if case["fp8"]:
        s["k_scale"], s["v_scale"] = 5.5 / 448.0, 6.0 / 448.0
    for n in ("k", "v"):  # on the GPU, where dividing by it is one IEEE division
        s[n + "_scale_gpu"] = torch.tensor(s[n + "_scale"], device="cuda")
    (_prepare_rope if case["op"] == "rope" else _prepare_cached)(case, gen, s)
    if own:  # the handles that a serving program keeps
        import paged_kv_cache_48_gb300 as pk
        s["pk"] = pk
        s["cache"] = pk.PagedKVCache(s["kc"], s["vc"], "fp8_e4m3" if case["fp8"] else "bf16",
                                     s["k_scale"], s["v_scale"])
        if case["op"] == "rope":
            s["rope"] = pk.RotaryAxes(case["rotary"], _sections(case), base=case["base"],
                                      interleave_axes=case["dealt"],
                                      interleave_pairs=case["adjacent"])
        elif case["op"] == "weights":
            n = pk.paged_attention_decode_weights_workspace_bytes(
                case["batch"], case["heads"], case["kv_heads"], case["dim"],
                max(s["lens_host"]))
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        else:
            n = pk.paged_kv_evict_workspace_bytes(case["batch"], case["kv_heads"],
                                                  s["weights"].shape[2], case["keep"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return {"rope": _run_rope, "weights": _run_weights, "evict": _run_evict}[s["case"]["op"]](s)


def _seen(s, cache, first=0):
    """A cache as the values it holds (from block `first` on)."""
    c = cache[first:]
    return c.view(F8) if s["case"]["fp8"] else c


def _axis_of_pair(case):
    sections = _sections(case)
    A, n = len(sections), case["rotary"] // 2
    if case["dealt"]:
        return [i % A if i < A * sections[i % A] else 0 for i in range(n)]
    return [a for a in range(A) for _ in range(sections[a])]


def _rotate(x, cos, sin, case):
    R = case["rotary"]
    if case["adjacent"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
    return torch.cat((y, x[..., R:]), dim=-1)


def _encode(x, scale, fp8):
    return (x / scale).clamp(-448.0, 448.0).to(F8).view(torch.uint8) if fp8 else x.bfloat16()


def _run_rope(s):
    case = s["case"]
    if own:
        s["pk"].paged_kv_rope_write(s["q"], s["k"], s["v"], s["positions"], s["slots"],
                                    s["cache"], s["rope"], q_out=s["q_out"])
        return dict(q=s["q_out"], k=_seen(s, s["kc"]), v=_seen(s, s["vc"]))
    pair = torch.arange(case["rotary"] // 2, device="cuda", dtype=torch.float64)
    freq = case["base"] ** (-2.0 * pair / case["rotary"])
    axis = torch.tensor(_axis_of_pair(case), device="cuda")
    angle = s["positions"][axis].double().t() * freq
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    s["q_out"].copy_(_rotate(s["q"].float(), cos, sin, case))
    k = _rotate(s["k"].float(), cos, sin, case)
    K, D = case["kv_heads"], case["dim"]
    s["kc"].view(-1, K, D)[s["slots"]] = _encode(k, s["k_scale_gpu"], case["fp8"])
    s["vc"].view(-1, K, D)[s["slots"]] = _encode(s["v"].float(), s["v_scale_gpu"], case["fp8"])
    return dict(q=s["q_out"], k=_seen(s, s["kc"]), v=_seen(s, s["vc"]))


def _run_weights(s):
    case = s["case"]
    B, H, K, D = case["batch"], case["heads"], case["kv_heads"], case["dim"]
    scale = 1.0 / math.sqrt(D)
    if own:
        new = dict(k_new=s["k_new"], v_new=s["v_new"]) if case["append"] else {}
        s["pk"].paged_attention_decode_weights(
            s["q"], s["cache"], s["tables"], s["lens"], scale, max(s["lens_host"]), s["weights"],
            decay=case["decay"], out=s["out"], workspace=s["workspace"], **new)
        r = dict(out=s["out"], weights=s["weights"])
        return dict(r, k=_seen(s, s["kc"]), v=_seen(s, s["vc"])) if case["append"] else r
    L = s["lens"].long()
    S = s["weights"].shape[2]
    t = torch.arange(S, device="cuda")
    b = torch.arange(B, device="cuda")
    valid = t < L[:, None]
    old = s["weights"] * case["decay"] if case["decay"] else torch.zeros_like(s["weights"])
    if case["append"]:
        last = L - 1
        block, row = s["tables"][b, last // BLOCK].long(), last % BLOCK
        below = (torch.arange(BLOCK, device="cuda") > row[:, None]) & (row == 0)[:, None]
        for c, x, cs in ((s["kc"], s["k_new"], s["k_scale_gpu"]),
                         (s["vc"], s["v_new"], s["v_scale_gpu"])):
            c[block, row] = _encode(x.float(), cs, case["fp8"])
            # a block that the token opens starts out zero
            c[block] = torch.where(below[:, :, None, None], torch.zeros_like(c[:1, :1]), c[block])
        old = torch.where((t == last[:, None])[:, None], torch.zeros_like(old), old)
    blocks = s["tables"].long().clamp(min=0)

    def gathered(c, cs):
        x = c.view(F8)[blocks] if case["fp8"] else c[blocks]
        return x.flatten(1, 2)[:, :S].float() * cs
    q = s["q"].float().view(B, K, H // K, D)
    score = torch.einsum("bkgd,btkd->bkgt", q, gathered(s["kc"], s["k_scale"])) * scale
    score = torch.where(valid[:, None, None], score, float("-inf"))
    e = (score - score.amax(-1, keepdim=True)).exp()
    del score
    p = e / e.sum(-1, keepdim=True)
    s["out"].copy_(torch.einsum("bkgt,btkd->bkgd", p, gathered(s["vc"], s["v_scale"])).view(B, H, D))
    s["weights"].copy_(torch.where(valid[:, None], old + p.sum(2), s["weights"]))
    r = dict(out=s["out"], weights=s["weights"])
    return dict(r, k=_seen(s, s["kc"]), v=_seen(s, s["vc"])) if case["append"] else r


def _run_evict(s):
    case = s["case"]
    B, K, D = case["batch"], case["kv_heads"], case["dim"]
    if own:
        s["pk"].paged_kv_evict(
            s["cache"], s["tables"], s["lens"], s["weights"], s["keep"], case["keep"],
            sink=case["sink"], recent=case["recent"], per_head=case["per_head"],
            dst_tables=s["dst"], dst_weights=s["dst_weights"], new_seq_lens=s["new_lens"],
            kept=s["kept"], workspace=s["workspace"])
    else:
        M, S = case["keep"], s["weights"].shape[2]
        L, keep = s["lens"].long(), s["keep"].long()
        n = torch.minimum(L, keep)
        recent = n.clamp(max=case["recent"])
        sink = (n - recent).clamp(max=case["sink"])
        t = torch.arange(S, device="cuda")
        w = s["weights"] if case["per_head"] else s["weights"].double().sum(1, keepdim=True).float()
        held = (t < sink[:, None]) | (t >= (L - recent)[:, None])
        key = torch.where(held[:, None], float("inf"), w)
        key = torch.where((t < L[:, None])[:, None], key, float("-inf"))
        order = key.argsort(dim=-1, descending=True, stable=True)[:, :, :M]
        i = torch.arange(order.shape[2], device="cuda")
        live = (i < n[:, None])[:, None].expand_as(order)
        at = torch.where(live, order, S).sort(dim=-1).values  # positions ascending, S past n
        s["kept"].fill_(-1)
        s["kept"][:, :, :at.shape[2]] = torch.where(live, at, -1)
        s["new_lens"].copy_(n)
        at, live = at.expand(B, K, -1), live.expand(B, K, -1)
        head = torch.arange(K, device="cuda")[None, :, None].expand_as(at)[live]
        row = torch.arange(B, device="cuda")[:, None, None].expand_as(at)[live]
        i, at = i.expand(B, K, -1)[live], at[live]
        src = s["tables"][row, at // BLOCK].long(), at % BLOCK, head
        dst = s["dst"][row, i // BLOCK].long(), i % BLOCK, head
        for c in (s["kc"], s["vc"]):
            c[dst] = c[src]
        gone = (t >= n[:, None]) & (t < L[:, None])
        s["dst_weights"].masked_fill_(gone[:, None], 0.0)
        s["dst_weights"][row, head, i] = s["weights"][row, head, at]
    return dict(k=_seen(s, s["kc"], s["first"]), v=_seen(s, s["vc"], s["first"]),
                weights=s["dst_weights"], lens=s["new_lens"], kept=s["kept"])


# ---------------------------------------------------------------------------
# 64 bits, and what a pass cannot do without
# ---------------------------------------------------------------------------
def _held(s, c):
    """What a cache's elements stand for, without its scale."""
    return (c.view(F8) if s["case"]["fp8"] else c).double()


def exact(case, seed):
    s = prepare(case, seed)
    B, K, D = case.get("batch"), case["kv_heads"], case["dim"]
    if case["op"] == "rope":
        R = case["rotary"]
        q, k = s["q"].double(), s["k"].double()
        for i, a in enumerate(_axis_of_pair(case)):
            x, y = (2 * i, 2 * i + 1) if case["adjacent"] else (i, i + R // 2)
            angle = s["positions"][a].double() * math.exp(-2.0 * i / R * math.log(case["base"]))
            c, d = angle.cos()[:, None], angle.sin()[:, None]
            for z in (q, k):
                u, w = z[:, :, x].clone(), z[:, :, y].clone()
                z[:, :, x], z[:, :, y] = u * c - w * d, w * c + u * d
        r = dict(q=q)
        for n, z in (("k", k), ("v", s["v"].double())):
            c = _held(s, s[n + "c"]).view(-1, K, D)
            z = (z / s[n + "_scale"]).clamp(-448, 448) if case["fp8"] else z
            c[s["slots"]] = z
            r[n] = c.view(s[n + "c"].shape)
        return r
    if case["op"] == "weights":
        H, G = case["heads"], case["heads"] // K
        weights, out = s["weights"].double(), torch.empty(B, H, D, dtype=torch.float64, device="cuda")
        kc, vc = s["kc"], s["vc"]
        for b, n in enumerate(s["lens_host"]):
            blocks = s["tables"][b, :(n + BLOCK - 1) // BLOCK].long()
            k, v = (_held(s, c[blocks]).flatten(0, 1)[:n] for c in (kc, vc))
            if case["append"]:
                for x, z, cs in ((k, s["k_new"], s["k_scale_gpu"]),
                                 (v, s["v_new"], s["v_scale_gpu"])):
                    x[n - 1] = (z[b].float() / cs).clamp(-448, 448).to(F8).double() if case["fp8"] \
                        else z[b].double()
                weights[b, :, n - 1] = 0
            weights[b, :, :n] *= case["decay"]
            for h in range(K):
                score = s["q"][b, h * G:(h + 1) * G].double() @ k[:, h].t()
                p = torch.softmax(score * s["k_scale"] / math.sqrt(D), dim=-1)
                out[b, h * G:(h + 1) * G] = p @ v[:, h] * s["v_scale"]
                weights[b, h, :n] += p.sum(0)
        return dict(out=out, weights=weights, k=None, v=None)
    kept = torch.full_like(s["kept"], -1)
    new_lens, weights = torch.zeros_like(s["new_lens"]), torch.zeros_like(s["dst_weights"]).double()
    for b, n in enumerate(s["lens_host"]):
        m = min(n, int(s["keep"][b]))
        new_lens[b] = m
        r = min(m, case["recent"])
        f = min(m - r, case["sink"])
        w = s["weights"][b, :, :n].double()
        if not case["per_head"]:
            w = w.sum(0, keepdim=True).float().double()
        middle = torch.sort(w[:, f:n - r], dim=-1, descending=True, stable=True).indices
        middle = middle[:, :m - r - f].sort(dim=-1).values + f
        t = torch.arange(n, device="cuda").expand(middle.shape[0], n)
        at = torch.cat((t[:, :f], middle, t[:, n - r:]), dim=-1)
        kept[b, :, :m] = at
        weights[b, :, :m] = s["weights"][b].double().gather(1, at.expand(K, m))
    return dict(k=None, v=None, weights=weights, lens=new_lens, kept=kept)


def work(case):
    K, D = case["kv_heads"], case["dim"]
    e = 1 if case["fp8"] else 2
    if case["op"] == "rope":
        T, H = case["tokens"], case["heads"]
        rows = T * D * (2 * 2 * H + (2 + e) * 2 * K)
        return dict(bytes=rows + 4 * T * len(_sections(case)) + 8 * T,
                    flops=3 * T * case["rotary"] * (H + K))
    lens = _lens(case)
    if case["op"] == "weights":
        B, H = case["batch"], case["heads"]
        new = B * K * D * 2 * (2 + e) if case["append"] else 0
        weights = K * sum(lens) * (8 if case["decay"] else 4)
        return dict(bytes=2 * K * D * e * sum(lens) + weights + 2 * 2 * B * H * D + new,
                    flops=4 * H * D * sum(lens))
    kept = sum(map(min, lens, _keep(case)))
    return dict(bytes=4 * K * sum(lens) + kept * K * (2 * 2 * D * e + 4)
                + 4 * kept * (K if case["per_head"] else 1), flops=K * sum(lens))
