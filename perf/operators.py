"""Measured cases of the view-cache operators.

A reconstruction that runs frame by frame keeps the keys and values of the frames it has
seen in a cache.  Three operators serve it:

* ``attend``:  a batch of views attends to the cache (the prefix that all views share) and
  to its own tokens (``prefix_attn``);
* ``weights``: how much attention every cached and every new token received, added to a
  running account (``key_weights``);
* ``evict``:   the cache shrinks to the tokens with the largest account (``cache_evict``).

``run`` computes them in plain 32-bit torch operations, or calls the package where ``own``
is true.  Heads are 64 wide; the sizes are those of this repository's workloads (16 heads,
frames of 5 special and 37 x 37 patch tokens = 1374) and generic ones around them.
"""

import random

import numpy as np
import torch

own = False

D = 64
FRAME = 5 + 37 * 37


def _case(name, op, **kw):
    c = {"name": name, "op": op}
    if op == "evict":
        c.update(heads=16, n=0, keep=0, recent=0)
    else:
        c.update(heads=16, kv_heads=16, views=1, q_min=1, q_max=1, own_min=0, own_max=0, prefix=0, causal=False, lens=1)
    c.update(kw)
    return c


def listed():
    one = dict(q_min=1, q_max=1, own_min=1, own_max=1)
    frame = dict(q_min=FRAME, q_max=FRAME, own_min=FRAME, own_max=FRAME)
    pose = dict(views=64, q_min=1, q_max=5, own_min=0, own_max=100)
    return [
        # one camera token asks a cache that holds one frame: the latency of a call
        _case("attend token", "attend", prefix=FRAME, **one),
        # one camera token asks a cache of 100 frames: a read of the whole cache
        _case("attend token long", "attend", prefix=100 * FRAME, **one),
        # the camera and register tokens of 64 views against the 30 frames that all share
        _case("attend poses", "attend", prefix=30 * FRAME, **pose),
        # the next frame of a stream, with ten frames behind it
        _case("attend frame", "attend", prefix=10 * FRAME, **frame),
        # views of unequal size that share three frames; four query heads a key head, later tokens of a view hidden
        _case("attend ragged", "attend", heads=16, kv_heads=4, views=7, q_min=301, q_max=1111, own_min=301, own_max=1500,
              prefix=3 * FRAME + 77, causal=True, lens=3),
        # four frames at a time against 30 frames: the largest
        _case("attend frames", "attend", prefix=30 * FRAME, views=4, **frame),
        # the account after a single token
        _case("weights token", "weights", prefix=FRAME, **one),
        # the account after 64 views' camera and register tokens
        _case("weights poses", "weights", prefix=30 * FRAME, **pose),
        # the account after four frames against 30
        _case("weights frames", "weights", prefix=30 * FRAME, views=4, **frame),
        # a small cache makes room for one more view's patches
        _case("evict small", "evict", n=FRAME + 331, keep=FRAME, recent=331),
        # a cache of 30 frames after the next one has been appended
        _case("evict frame", "evict", n=31 * FRAME, keep=30 * FRAME, recent=FRAME),
        # 200 frames shrink to 100
        _case("evict half", "evict", n=200 * FRAME, keep=100 * FRAME, recent=2 * FRAME),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(("attend", "weights", "evict"))
    if op == "evict":
        n = _log(rng, 100, 200 * FRAME)
        keep = max(1, int(n * rng.uniform(0.3, 0.99)))
        return {"op": op, "heads": rng.choice((2, 4, 8, 16)), "n": n, "keep": keep, "recent": rng.randint(0, min(keep, 2 * FRAME))}
    heads, kv = rng.choice(((16, 16), (16, 16), (16, 4), (8, 8), (12, 4), (2, 2), (8, 1)))
    c = {"op": op, "heads": heads, "kv_heads": kv, "views": _log(rng, 1, 64), "q_max": _log(rng, 1, FRAME), "prefix": _log(rng, 1, 30 * FRAME),
         "causal": rng.random() < 0.3, "lens": rng.randint(1, 10 ** 6)}
    while c["views"] > 1 and c["views"] * c["q_max"] > 4 * FRAME:
        c["views"] -= 1
    c["q_min"] = rng.randint(1, c["q_max"])
    c["own_max"] = min(FRAME, rng.choice((0, c["q_max"], c["q_max"] + rng.randint(0, 100))))
    c["own_min"] = rng.randint(0, c["own_max"])
    return c


def _lengths(case):
    """The views' numbers of queries and of own tokens: the same for every seed."""
    r = random.Random(case["lens"])
    q = [r.randint(case["q_min"], case["q_max"]) for _ in range(case["views"])]
    t = [r.randint(case["own_min"], case["own_max"]) for _ in range(case["views"])]
    return q, t


def _offsets(lens):
    at = [0]
    for x in lens:
        at.append(at[-1] + x)
    return at


def _make(case, seed):
    """Inputs from the seed: queries share a direction in each head, and one key in 50 lies along it (the tokens that gather attention)."""
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    if case["op"] == "evict":
        H, n = case["heads"], case["n"]
        s = {"k": normal(n, H, D).bfloat16(), "v": normal(n, H, D).bfloat16()}
        acc = torch.exp(1.5 * normal(H, n))
        # an eighth of the tokens has been looked at equally little, one in 200 is to stay for good
        u = torch.rand(H, n, generator=g, device="cuda")
        acc = torch.where(u < 0.125, torch.full_like(acc, 0.25), acc)
        s["acc"] = torch.where(u > 0.995, torch.full_like(acc, float("inf")), acc)
        # token numbers: slots are in no order, but for the newest at the end
        order = torch.rand(H, n, generator=g, device="cuda")
        order[:, n - case["recent"]:] += torch.arange(1, case["recent"] + 1, device="cuda")
        s["ids"] = torch.argsort(torch.argsort(order, 1), 1).int()
        return s
    H, Hk, P = case["heads"], case["kv_heads"], case["prefix"]
    ql, tl = _lengths(case)
    nq, nt = sum(ql), sum(tl)
    mu = 0.5 * normal(Hk, D)
    sink = (torch.rand(P + nt, Hk, 1, generator=g, device="cuda") < 0.02).float()
    k = (normal(P + nt, Hk, D) + 2 * sink * mu).bfloat16()
    s = {"q": (normal(nq, H, D) + mu.repeat_interleave(H // Hk, 0)).bfloat16(), "k_prefix": k[:P].clone(), "k_own": k[P:].clone(),
         "q_off": torch.tensor(_offsets(ql), dtype=torch.int32, device="cuda"), "own_off": torch.tensor(_offsets(tl), dtype=torch.int32, device="cuda")}
    if case["op"] == "attend":
        v = normal(P + nt, Hk, D).bfloat16()
        s.update(v_prefix=v[:P].clone(), v_own=v[P:].clone())
    else:
        s["acc"] = torch.exp(normal(Hk, P))
        s["decay"] = 0.875
    return s


def prepare(case, seed):
    s = _make(case, seed)
    s["case"] = case
    if case["op"] != "evict":
        ql, tl = _lengths(case)
        s.update(max_q=max(ql), max_own=max(tl))
    if case["op"] == "weights":
        # the attention over the same keys came before: its log-sum-exps are at hand
        s["lse"] = torch.logsumexp(_scores(s), 2).transpose(0, 1).contiguous()
    return s


def _scores(s):
    """Scaled logits [heads][queries][prefix + own], -inf where a query does not see an own token."""
    c = s["case"]
    P, G = c["prefix"], c["heads"] // c["kv_heads"]
    k = torch.cat((s["k_prefix"], s["k_own"])).float().repeat_interleave(G, 1)
    x = torch.matmul(s["q"].float().transpose(0, 1), k.permute(1, 2, 0)).mul_(D ** -0.5)
    nq, nt = s["q"].shape[0], s["k_own"].shape[0]
    if nt:
        i, j = torch.arange(nq, device="cuda")[:, None], torch.arange(nt, device="cuda")[None]
        qo, to = s["q_off"].long(), s["own_off"].long()
        view = torch.searchsorted(qo, i, right=True) - 1
        sees = (j >= to[view]) & (j < to[view + 1])
        if c["causal"]:
            sees &= j - to[view + 1] <= i - qo[view + 1]
        x[:, :, P:].masked_fill_(~sees, float("-inf"))
    return x


def _attend(s):
    x = _scores(s)
    G = s["case"]["heads"] // s["case"]["kv_heads"]
    v = torch.cat((s["v_prefix"], s["v_own"])).float().repeat_interleave(G, 1)
    top = x.amax(2, keepdim=True)
    p = x.sub_(top).exp_()
    total = p.sum(2, keepdim=True)
    out = torch.matmul(p, v.transpose(0, 1)) / total
    return {"out": out.transpose(0, 1).contiguous().bfloat16(), "lse": (top + total.log())[:, :, 0].transpose(0, 1).contiguous()}


def _weights(s):
    c = s["case"]
    p = _scores(s).sub_(s["lse"].transpose(0, 1)[:, :, None]).exp_()
    w = p.sum(1).view(c["kv_heads"], -1, p.shape[2]).sum(1)
    w[:, :c["prefix"]] += s["decay"] * s["acc"]
    return {"acc": w}


def _evict(s):
    c = s["case"]
    H, n, keep = c["heads"], c["n"], c["keep"]
    key = torch.where(s["ids"] >= n - c["recent"], torch.full_like(s["acc"], float("inf")), s["acc"])
    kept = torch.zeros(H, n, dtype=torch.bool, device="cuda")
    kept.scatter_(1, torch.sort(key, dim=1, descending=True, stable=True)[1][:, :keep], True)
    slot = torch.arange(n, device="cuda").expand(H, n)
    # the i-th kept token behind `keep` moves into the i-th free slot before it
    movers = torch.where(kept & (slot >= keep), 0, 1).sort(dim=1, stable=True)[1]
    free = (~kept[:, :keep]).long().cumsum(1) - 1
    source = torch.where(kept[:, :keep], slot[:, :keep], torch.gather(movers, 1, free.clamp(min=0)))
    rows = source.transpose(0, 1)[:, :, None].expand(keep, H, D)
    return {"k": torch.gather(s["k"], 0, rows), "v": torch.gather(s["v"], 0, rows), "acc": torch.gather(s["acc"], 1, source), "ids": torch.gather(s["ids"], 1, source)}


def _own(s):
    import sparse_global_attention_view_b200 as G

    c = s["case"]
    if c["op"] == "evict":
        if "ws" not in s:
            s["ws"] = G.new_cache_workspace(c["heads"], c["n"], c["keep"], "cuda")
            s["acc_out"], s["ids_out"] = torch.empty_like(s["acc"]), torch.empty_like(s["ids"])
        G.cache_evict(c["n"], c["keep"], c["n"] - c["recent"], s["k"], s["v"], s["acc"], s["ids"], s["acc_out"], s["ids_out"], s["ws"])
        return {"k": s["k"][:c["keep"]], "v": s["v"][:c["keep"]], "acc": s["acc_out"][:, :c["keep"]], "ids": s["ids_out"][:, :c["keep"]]}
    nq, nt, P = s["q"].shape[0], s["k_own"].shape[0], c["prefix"]
    if "ws" not in s:
        s["batch"] = G.ViewBatch(n_views=c["views"], n_q=nq, n_own=nt, n_prefix=P, n_heads=c["heads"], n_kv_heads=c["kv_heads"],
                                 max_q=s["max_q"], max_own=s["max_own"], causal=c["causal"])
        s["ws"] = G.new_view_workspace(s["batch"], "cuda")
        if c["op"] == "attend":
            s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty(nq, c["heads"], device="cuda")
        else:
            s["acc_out"] = torch.empty(c["kv_heads"], P + nt, device="cuda")
    if c["op"] == "attend":
        G.prefix_attn(s["batch"], s["q"], s["k_prefix"], s["v_prefix"], s["k_own"], s["v_own"], s["q_off"], s["own_off"], s["out"], s["lse"], s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    G.key_weights(s["batch"], s["q"], s["k_prefix"], s["k_own"], s["q_off"], s["own_off"], s["lse"], s["acc"], s["acc_out"], s["decay"], s["ws"])
    return {"acc": s["acc_out"]}


def run(s):
    if own:
        return _own(s)
    return {"attend": _attend, "weights": _weights, "evict": _evict}[s["case"]["op"]](s)


def _moves(case):
    """Tokens that have to move, a head: about the share of evicted ones among the first `keep` slots (the newest, at the end, all stay)."""
    n, keep, recent = case["n"], case["keep"], case["recent"]
    old = n - recent
    return min(keep, old) * (n - keep) / max(1, old)


def _pairs(case):
    """(query, key) pairs that a head looks at."""
    pairs = 0
    for q, t in zip(*_lengths(case)):
        pairs += q * (case["prefix"] + t)
        if case["causal"]:
            # the last query sees every own token, each one before it one token less
            h = min(q - 1, t)
            pairs -= h * (h + 1) // 2 + (q - 1 - h) * t
    return pairs


def work(case):
    if case["op"] == "evict":
        H = case["heads"]
        # the account and the token numbers in and out, and the moved rows of K and V, read and written
        return {"bytes": H * (8 * case["n"] + 8 * case["keep"] + _moves(case) * 2 * 2 * 2 * D), "flops": 0}
    ql, tl = _lengths(case)
    H, Hk, nq, keys = case["heads"], case["kv_heads"], sum(ql), case["prefix"] + sum(tl)
    if case["op"] == "attend":
        return {"bytes": 2 * D * (2 * nq * H + 2 * keys * Hk) + 4 * nq * H, "flops": 4 * D * H * _pairs(case)}
    return {"bytes": 2 * D * (nq * H + keys * Hk) + 4 * nq * H + 4 * Hk * (keys + case["prefix"]), "flops": 2 * D * H * _pairs(case)}


def exact(case, seed):
    """The definitions in 64 bits: every view by itself, one head after the other."""
    s = _make(case, seed)
    if case["op"] == "evict":
        return _exact_evict(case, s)
    H, Hk, P = case["heads"], case["kv_heads"], case["prefix"]
    ql, tl = _lengths(case)
    q0, t0 = _offsets(ql), _offsets(tl)
    out = torch.zeros(q0[-1], H, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(q0[-1], H, dtype=torch.float64, device="cuda")
    acc = torch.zeros(Hk, P + t0[-1], dtype=torch.float64, device="cuda")
    for h in range(H):
        hk = h // (H // Hk)
        for b in range(case["views"]):
            if not ql[b]:
                continue
            rows, cols = slice(q0[b], q0[b + 1]), slice(t0[b], t0[b + 1])
            k = torch.cat((s["k_prefix"][:, hk], s["k_own"][cols, hk])).double()
            x = s["q"][rows, h].double() @ k.T / 8.0
            if case["causal"]:
                # the last query sees every own token, each one before it one token less
                hidden = torch.ones(ql[b], tl[b], dtype=torch.bool, device="cuda").triu(tl[b] - ql[b] + 1)
                x[:, P:][hidden] = float("-inf")
            z = torch.logsumexp(x, 1)
            lse[rows, h] = z
            x -= z[:, None]
            x.exp_()
            if case["op"] == "attend":
                out[rows, h] = x @ torch.cat((s["v_prefix"][:, hk], s["v_own"][cols, hk])).double()
            else:
                acc[hk, :P] += x[:, :P].sum(0)
                acc[hk, P + t0[b]:P + t0[b + 1]] += x[:, P:].sum(0)
    if case["op"] == "attend":
        return {"out": out, "lse": lse}
    acc[:, :P] += s["decay"] * s["acc"].double()
    return {"acc": acc}


def _exact_evict(case, s):
    n, keep = case["n"], case["keep"]
    sources = []
    for h in range(case["heads"]):
        a, ids = s["acc"][h].cpu().numpy().astype(np.float64), s["ids"][h].cpu().numpy()
        a[ids >= n - case["recent"]] = np.inf
        chosen = np.lexsort((np.arange(n), -a))[:keep]
        stays = np.zeros(n, bool)
        stays[chosen] = True
        src = np.arange(keep)
        src[~stays[:keep]] = np.sort(chosen[chosen >= keep])
        sources.append(src)
    at = torch.from_numpy(np.stack(sources)).cuda()
    heads = torch.arange(case["heads"], device="cuda")
    return {"k": s["k"][at.T, heads].double(), "v": s["v"][at.T, heads].double(), "acc": s["acc"][heads[:, None], at].double(), "ids": None}
