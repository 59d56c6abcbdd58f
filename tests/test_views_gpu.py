"""The view-cache operators on a B200 against their formulas in 64 bits."""

import pytest
import torch

import views_ref as R

pytestmark = pytest.mark.gpu

DEV = "cuda"


def G():
    import sparse_global_attention_view_b200 as g
    return g


def offsets(lens):
    at = [0]
    for x in lens:
        at.append(at[-1] + x)
    return at


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def make(H, Hk, ql, tl, prefix, seed=0, strength=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda n, h: torch.randn(n, h, 64, generator=g, device=DEV).bfloat16()  # noqa: E731
    nq, nt = sum(ql), sum(tl)
    return dict(q=(r(nq, H) * strength).bfloat16(), kp=r(prefix, Hk), vp=r(prefix, Hk), ko=r(nt, Hk), vo=r(nt, Hk),
                q_off=offsets(ql), own_off=offsets(tl))


def batch_of(x, causal=False, **kw):
    ql = [b - a for a, b in zip(x["q_off"], x["q_off"][1:])]
    tl = [b - a for a, b in zip(x["own_off"], x["own_off"][1:])]
    kw = dict(max_q=max(ql), max_own=max(tl), causal=causal) | kw
    return G().ViewBatch(n_views=len(ql), n_q=x["q"].shape[0], n_own=x["ko"].shape[0], n_prefix=x["kp"].shape[0],
                         n_heads=x["q"].shape[1], n_kv_heads=x["kp"].shape[1], **kw)


def attend(x, batch, out=None, lse=None, ws=None, stream=None):
    ws = G().new_view_workspace(batch) if ws is None else ws
    out = torch.full(x["q"].shape, 7.0, dtype=torch.bfloat16, device=DEV) if out is None else out
    lse = torch.full(x["q"].shape[:2], 7.0, device=DEV) if lse is None else lse
    G().prefix_attn(batch, x["q"], x["kp"], x["vp"], x["ko"], x["vo"], ints(x["q_off"]), ints(x["own_off"]), out, lse, ws,
                    stream)
    G().check_device_error(ws)
    return out, lse


def assert_attend(x, out, lse, causal=False, scale=0.125):
    o, z, to, tz = R.attend(x["q"], x["kp"], x["vp"], x["ko"], x["vo"], x["q_off"], x["own_off"], causal, scale)
    rows = slice(x["q_off"][0], x["q_off"][-1])
    o, z, to, tz = o[rows], z[rows], to[rows], tz[rows]
    out, lse = out[rows].double(), lse[rows].double()
    empty = z == R.NEG
    assert torch.equal(lse == R.NEG, empty)
    assert (out[empty] == 0).all()
    over = ((out - o).abs() - to).max() if out.numel() else torch.tensor(0.0)
    assert over <= 0, f"out: {over.item():.3e} over its bound, {((out - o).abs() / to.clamp(min=1e-30)).max().item():.2f} of it"
    dz = torch.where(empty, torch.zeros_like(z), (lse - z).abs())
    assert (dz <= tz).all(), f"lse: {dz.max().item():.3e}, bound {tz.max().item():.3e}"


# heads, key heads, queries of the views, own tokens of the views, prefix
SIZES = {
    "one token": (2, 2, [1], [1], 5),
    "one token, no prefix": (2, 2, [1], [1], 0),
    "one token, no own": (4, 2, [1], [0], 1374),
    "three rows": (3, 1, [1], [7], 1300),
    "three rows, long": (3, 1, [1], [700], 20000),
    "four tokens, long": (2, 2, [1, 0, 2, 1], [7, 3, 0, 130], 17000),
    "four tokens, many own": (2, 2, [2, 1, 1], [300, 0, 1300], 100),
    "four tokens": (2, 2, [1, 2, 1], [7, 0, 130], 1300),
    "five tokens": (2, 2, [1, 3, 1], [7, 0, 130], 300),
    "no keys": (2, 2, [3, 130], [0, 0], 0),
    "views without keys": (2, 2, [3, 2, 0, 1], [0, 5, 4, 0], 0),
    "long token": (16, 16, [1], [1], 13740),
    "poses": (4, 4, [1, 5, 3, 2, 5, 1, 4, 4], [0, 100, 31, 7, 1, 0, 64, 13], 700),
    "poses, groups of 4": (16, 4, [1, 4, 3, 2], [9, 100, 31, 7], 1000),
    "groups of 3": (6, 2, [50, 7, 100], [33, 129, 100], 257),
    "groups of 3, short": (6, 2, [5, 1, 2], [33, 129, 100], 130),
    "one key head of 128": (128, 1, [1, 2, 3], [4, 5, 6], 129),
    "tile edges": (1, 1, [128, 127, 129, 1], [127, 128, 129, 1], 128),
    "prefix of one": (2, 2, [300], [300], 1),
    "prefix 127": (2, 2, [256], [128], 127),
    "prefix 129": (2, 2, [257], [0], 129),
    "no prefix": (2, 2, [300, 20, 511], [300, 25, 500], 0),
    "long views": (2, 2, [700, 650], [700, 650], 900),
    "mixed views": (2, 1, [1, 600, 2, 90, 1, 1], [50, 600, 700, 90, 1, 0], 1000),
    "few rows, long own": (2, 2, [1], [9000], 0),
    "many single tokens": (2, 2, [1] * 300, [3] * 300, 400),
    "split rows": (2, 2, [300], [10], 6000),
}


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("name", list(SIZES))
def test_attend(name, causal):
    x = make(*SIZES[name], seed=len(name))
    out, lse = attend(x, batch_of(x, causal))
    assert_attend(x, out, lse, causal)


def weigh(x, batch, lse, acc, decay, acc_out=None, ws=None, stream=None):
    ws = G().new_view_workspace(batch) if ws is None else ws
    Hk, n = x["kp"].shape[1], x["kp"].shape[0] + x["ko"].shape[0]
    acc_out = torch.full((Hk, n), 7.0, device=DEV) if acc_out is None else acc_out
    G().key_weights(batch, x["q"], x["kp"], x["ko"], ints(x["q_off"]), ints(x["own_off"]), lse, acc, acc_out, decay, ws,
                    stream)
    G().check_device_error(ws)
    return acc_out


def exact_lse(x, causal=False):
    z = R.attend(x["q"], x["kp"], x["vp"], x["ko"], x["vo"], x["q_off"], x["own_off"], causal)[1]
    return z.nan_to_num(0.0, neginf=R.NEG).float()


def assert_weights(x, got, lse, acc, decay, causal=False):
    w, tol = R.weights(x["q"], x["kp"], x["ko"], x["q_off"], x["own_off"], lse, acc, decay, causal)
    there = ~w.isnan()
    d = (got[:, :w.shape[1]].double() - w).abs()[there]
    assert (d <= tol[there]).all(), f"{d.max().item():.3e}: {(d / tol[there]).max().item():.2f} of the bound"
    assert (got[:, :w.shape[1]][~there] == 7).all()


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("name", list(SIZES))
def test_weights(name, causal):
    x = make(*SIZES[name], seed=len(name))
    lse = exact_lse(x, causal)
    acc = torch.rand(x["kp"].shape[1], x["kp"].shape[0], device=DEV)
    got = weigh(x, batch_of(x, causal), lse, acc, 0.75)
    assert_weights(x, got, lse, acc, 0.75, causal)


@pytest.mark.parametrize("n_q", [1, 3, 8, 9, 300])
def test_weights_sum_to_the_queries(n_q):
    x = make(4, 4, [n_q], [40], 3000)
    batch = batch_of(x)
    _, lse = attend(x, batch)
    got = weigh(x, batch, lse, None, 1.0)
    # each query's weights sum to 1, up to the errors of its lse (1e-5) and of the sums
    assert (got.double().sum(1) / n_q - 1).abs().max() < 4e-5


def cache(heads, n, seed, ties=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    k = torch.randn(n, heads, 64, generator=g, device=DEV).bfloat16()
    v = torch.randn(n, heads, 64, generator=g, device=DEV).bfloat16()
    acc = torch.rand(heads, n, generator=g, device=DEV)
    if ties:
        acc = (acc * 4).floor() / 4
    ids = torch.argsort(torch.rand(heads, n, generator=g, device=DEV), 1).int()
    return k, v, acc, ids


def assert_evicted(k, v, acc, ids, keep, recent_from, k2, v2, acc2, ids2):
    n, heads = k.shape[:2]
    src = R.evict(acc.cpu(), ids.cpu(), keep, recent_from).to(DEV)
    h = torch.arange(heads, device=DEV)
    assert torch.equal(ids2[:, :keep], ids[h[:, None], src])
    assert torch.equal(acc2[:, :keep].view(torch.int32), acc[h[:, None], src].view(torch.int32))
    for a, b in ((k, k2), (v, v2)):
        assert torch.equal(b[:keep].view(torch.int16), a[src.T, h].view(torch.int16))
        assert torch.equal(b[keep:].view(torch.int16), a[keep:].view(torch.int16))


def evict(k, v, acc, ids, keep, recent_from, n=None):
    n = k.shape[0] if n is None else n
    k2, v2 = k.clone(), v.clone()
    acc2, ids2 = torch.full_like(acc, 7.0), torch.full_like(ids, 7)
    ws = G().new_cache_workspace(k.shape[1], n, keep)
    G().cache_evict(n, keep, recent_from, k2, v2, acc, ids, acc2, ids2, ws)
    G().check_device_error(ws)
    assert (acc2[:, keep:] == 7).all() and (ids2[:, keep:] == 7).all()
    return k2, v2, acc2, ids2


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("heads,n,keep", [(1, 1, 1), (2, 2, 1), (1, 31, 7), (3, 33, 32), (2, 257, 256), (16, 1705, 1374),
                                          (2, 5000, 1), (2, 5000, 4999), (2, 5000, 5000), (4, 8191, 4096), (1, 40000, 20001), (2, 4097, 3000), (1, 65537, 30000),
                                          (3, 4096, 7)])
def test_evict(heads, n, keep, ties):
    k, v, acc, ids = cache(heads, n, n + keep, ties)
    for recent in (0, min(keep, 5), keep, n):
        assert_evicted(k, v, acc, ids, keep, n - recent, *evict(k, v, acc, ids, keep, n - recent))


def test_evict_of_special_values():
    k, v, acc, ids = cache(2, 3000, 1)
    inf, nan = float("inf"), float("nan")
    for i, x in enumerate((inf, -inf, nan, 0.0, -0.0, 1e-45, -1e-45, 3e38, -3e38)):
        acc[:, i::23] = x
    for keep in (1, 200, 300, 1500, 2900, 2999):
        assert_evicted(k, v, acc, ids, keep, 3000, *evict(k, v, acc, ids, keep, 3000))
    acc[:] = nan
    assert_evicted(k, v, acc, ids, 1000, 3000, *evict(k, v, acc, ids, 1000, 3000))


def test_evict_beyond_shared_memory():
    # a slice of a head's slots that does not fit a CTA's shared memory
    k, v, acc, ids = cache(1, 8 * 96 * 1024 + 1000, 5, True)
    assert_evicted(k, v, acc, ids, 200_000, 800_000, *evict(k, v, acc, ids, 200_000, 800_000))


def test_evict_twice_is_evict_once():
    k, v, acc, ids = cache(2, 3000, 2)
    k2, v2, acc2, ids2 = evict(k, v, acc, ids, 1700, 2900)
    assert_evicted(k, v, acc, ids, 1700, 2900, *evict(k2, v2, acc, ids, 1700, 2900))


# ---------------------------------------------------------------------------------------------------------------
# how users hold their tensors

# a shape for each way a call is cut up: one row, few rows, packed rows with the own keys apart, long views
WAYS = {
    "one token": (2, 2, [1], [9], 700),
    "poses": (4, 2, [1, 5, 3, 2], [0, 100, 31, 7], 700),
    "mixed views": (2, 2, [1, 300, 2], [50, 300, 200], 300),
    "long views": (2, 2, [300, 280], [300, 280], 300),
}


def everything(x, causal=False, decay=0.75, **kw):
    """attend and weigh, against their formulas."""
    batch = batch_of(x, causal, **kw)
    out, lse = attend(x, batch)
    assert_attend(x, out, lse, causal)
    lse = exact_lse(x, causal)
    acc = torch.rand(x["kp"].shape[1], x["kp"].shape[0], device=DEV)
    assert_weights(x, weigh(x, batch, lse, acc, decay), lse, acc, decay, causal)


@pytest.mark.parametrize("name", list(WAYS))
def test_slices_of_larger_tensors(name):
    x = make(*WAYS[name])
    H, Hk = x["q"].shape[1], x["kp"].shape[1]
    nq, nt, P = x["q"].shape[0], x["ko"].shape[0], x["kp"].shape[0]
    fused = torch.full((nq, H + 2, 64), float("nan"), dtype=torch.bfloat16, device=DEV)
    fused[:, 1:1 + H] = x["q"]
    kv = torch.full((P + 100, 2, Hk, 64), float("nan"), dtype=torch.bfloat16, device=DEV)
    kv[:P, 0], kv[:P, 1] = x["kp"], x["vp"]
    own = torch.full((nt, 3 * Hk, 64), float("nan"), dtype=torch.bfloat16, device=DEV)
    own[:, Hk:2 * Hk], own[:, 2 * Hk:] = x["ko"], x["vo"]
    x.update(q=fused[:, 1:1 + H], kp=kv[:P, 0], vp=kv[:P, 1], ko=own[:, Hk:2 * Hk], vo=own[:, 2 * Hk:])
    everything(x)
    # an output of a larger tensor: what lies around it stays
    room = torch.full((nq, H + 1, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    out, lse = attend(x, batch_of(x), room[:, :H])
    assert_attend(x, out, lse)
    assert (room[:, H] == 7).all()
    # an account with longer rows, in place
    acc = torch.full((Hk, P + nt + 13), 7.0, device=DEV)
    acc[:, :P] = torch.rand(Hk, P, device=DEV)
    before, z = acc.clone(), exact_lse(x)
    weigh(x, batch_of(x), z, acc, 0.5, acc)
    assert_weights(x, acc, z, before, 0.5)
    assert (acc[:, P + nt:] == 7).all()


@pytest.mark.parametrize("name", list(WAYS))
def test_rows_of_no_view(name):
    x = make(*WAYS[name])
    nan = float("nan")

    def padded(t, front, back):
        pad = lambda n: torch.full((n, *t.shape[1:]), nan, dtype=t.dtype, device=DEV)  # noqa: E731
        return torch.cat((pad(front), t, pad(back)))

    nq, nt = x["q"].shape[0], x["ko"].shape[0]
    x.update(q=padded(x["q"], 3, 150), ko=padded(x["ko"], 5, 140), vo=padded(x["vo"], 5, 140),
             q_off=[3 + a for a in x["q_off"]], own_off=[5 + a for a in x["own_off"]])
    batch = batch_of(x)
    out, lse = attend(x, batch)
    assert_attend(x, out, lse)
    z = exact_lse(x)
    got = weigh(x, batch, z, None, 1.0)
    assert_weights(x, got, z, None, 1.0)
    for rows in (slice(0, 3), slice(3 + nq, None)):
        assert (out[rows] == 7).all() and (lse[rows] == 7).all()
    P = x["kp"].shape[0]
    assert (got[:, P:P + 5] == 7).all() and (got[:, P + 5 + nt:] == 7).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("name", ["poses", "mixed views", "long views"])
def test_bad_values_stay_in_their_view(name, bad):
    x = make(*WAYS[name])
    batch, z = batch_of(x), exact_lse(x)
    good = attend(x, batch)
    w = weigh(x, batch, z, None, 1.0)
    x["ko"], x["vo"] = x["ko"].clone(), x["vo"].clone()
    rows, cols = slice(x["q_off"][1], x["q_off"][2]), slice(x["own_off"][1], x["own_off"][2])
    x["ko"][cols], x["vo"][cols] = bad, bad
    out, lse = attend(x, batch)
    # view 1 sees keys without a finite score: a score of +inf or NaN leaves no number (one of -inf would, but the
    # queries' signs give both)
    assert out[rows].isnan().all() and lse[rows].isnan().all()
    keep = torch.ones(out.shape[0], dtype=torch.bool)
    keep[rows] = False
    assert torch.equal(out[keep], good[0][keep]) and torch.equal(lse[keep], good[1][keep])
    w2 = weigh(x, batch, z, None, 1.0)
    P = x["kp"].shape[0]
    keep = torch.ones(w.shape[1], dtype=torch.bool)
    keep[P + cols.start:P + cols.stop] = False
    assert torch.equal(w2[:, keep], w[:, keep])


@pytest.mark.parametrize("name", list(WAYS))
def test_a_nan_that_is_seen_shows(name):
    for j in (0, 77, 299):
        x = make(*WAYS[name])
        x["kp"][j, 0] = float("nan")
        out, lse = attend(x, batch_of(x))
        G_ = x["q"].shape[1] // x["kp"].shape[1]
        assert out[:, :G_].isnan().all() and lse[:, :G_].isnan().all()
        assert not out[:, G_:].isnan().any()


@pytest.mark.parametrize("what", ["query", "lse"])
@pytest.mark.parametrize("name", list(WAYS))
def test_a_nan_that_is_seen_shows_in_the_account(name, what):
    # every place of a row in a chunk of scores, in each view
    x = make(*WAYS[name])
    batch, z = batch_of(x), exact_lse(x)
    w = weigh(x, batch, z, None, 1.0)
    P = x["kp"].shape[0]
    for b, rows, cols in R.views(x["q_off"], x["own_off"]):
        for i in range(rows.start, min(rows.stop, rows.start + 16)):
            y, zz = x | dict(q=x["q"].clone()), z.clone()
            if what == "query":
                y["q"][i, 0] = float("nan")
            else:
                zz[i, 0] = float("nan")
            got = weigh(y, batch, zz, None, 1.0)
            nan = torch.zeros_like(w, dtype=torch.bool)
            nan[0, :P] = True
            nan[0, P + cols.start:P + cols.stop] = True
            assert torch.equal(got.isnan(), nan), (b, i)
            assert torch.equal(got[~nan], w[~nan]), (b, i)


# the ways, and rows of a tile that are no token's: groups that do not divide 128, tokens that do not fill the tile
ACCOUNTS = WAYS | {"groups of 3": (6, 2, [50, 7, 100], [33, 129, 100], 257), "groups of 5, short": (5, 1, [1, 2, 1], [33, 129, 100], 257)}


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("name", list(ACCOUNTS))
def test_queries_without_a_log_sum_count_for_nothing(name, bad):
    x = make(*ACCOUNTS[name])
    for b, rows, cols in R.views(x["q_off"], x["own_off"]):
        for i in range(rows.start, min(rows.stop, rows.start + 16)):
            z = exact_lse(x)
            z[i] = R.NEG
            y = x | dict(q=x["q"].clone())
            y["q"][i] = bad
            batch = batch_of(x)
            got = weigh(y, batch, z, None, 1.0)
            # finite in the place of what counts for nothing: the same bits
            assert not got.isnan().any() and torch.equal(got, weigh(x, batch, z, None, 1.0)), (b, i)
    # nobody counts at all
    y, z = x | dict(q=torch.full_like(x["q"], bad)), torch.full_like(z, R.NEG)
    assert (weigh(y, batch, z, None, 1.0) == 0).all()


@pytest.mark.parametrize("name", list(ACCOUNTS))
def test_queries_that_do_not_see_a_key_leave_its_account(name):
    # causal: the first query of a view holds NaN, in its values or its log sum
    x = make(*ACCOUNTS[name])
    batch, z0 = batch_of(x, True), exact_lse(x, True)
    good = weigh(x, batch, z0, None, 1.0)
    P = x["kp"].shape[0]
    for b, rows, cols in R.views(x["q_off"], x["own_off"]):
        see = R.seen(rows.stop - rows.start, cols.stop - cols.start, True, DEV)[0]
        for y, z in ((x | dict(q=x["q"].clone()), z0), (x, z0.clone())):
            (z if y is x else y["q"])[rows.start] = float("nan")
            got = weigh(y, batch, z, None, 1.0)
            nan = torch.zeros_like(got, dtype=torch.bool)
            nan[:, :P] = True
            nan[:, P + cols.start:P + cols.stop] = see
            assert torch.equal(got.isnan(), nan), b
            assert torch.equal(got[~nan], good[~nan]), b


@pytest.mark.parametrize("name", list(ACCOUNTS))
def test_an_infinite_key_that_nobody_looks_at(name):
    # every score with it is -infinity: a weight of 0, whatever lies in a tile's other rows
    x = make(*ACCOUNTS[name])
    x["q"] = x["q"].abs()
    P = x["kp"].shape[0]
    cols = [0, 100, P - 1]
    for t, at in ((x["kp"], cols), (x["ko"], [0, x["ko"].shape[0] - 1])):
        t[at] = float("-inf")
    z = exact_lse(x)
    assert z.isfinite().all()
    got = weigh(x, batch_of(x), z, None, 1.0)
    assert (got[:, cols + [P, -1]] == 0).all()
    assert_weights(x, got, z, None, 1.0)


@pytest.mark.parametrize("name", ["poses", "mixed views", "long views"])
def test_hidden_values_weigh_nothing(name):
    # the largest finite values, behind what the causal mask lets a query see
    x = make(*WAYS[name])
    batch = batch_of(x, True)
    good = attend(x, batch)
    for b, rows, cols in R.views(x["q_off"], x["own_off"]):
        hidden = min(rows.stop - rows.start - 1, cols.stop - cols.start)  # the first query does not see so many
        y = x | dict(vo=x["vo"].clone())
        for n in range(1, min(hidden, 20) + 1):
            y["vo"][cols.stop - n] = 3.3e38
        out, lse = attend(y, batch)
        keep = torch.ones(out.shape[0], dtype=torch.bool)
        keep[rows.stop - min(hidden, 20):rows.stop] = False
        assert torch.equal(out[keep], good[0][keep]), b
        assert torch.equal(lse, good[1])


@pytest.mark.parametrize("strength", [0.0, 30.0, 3000.0])
@pytest.mark.parametrize("name", list(WAYS))
def test_flat_and_steep_scores(name, strength):
    x = make(*WAYS[name], strength=strength)
    out, lse = attend(x, batch_of(x))
    assert_attend(x, out, lse)
    if strength <= 30:
        z = exact_lse(x)
        assert_weights(x, weigh(x, batch_of(x), z, None, 1.0), z, None, 1.0)


@pytest.mark.parametrize("name", list(WAYS))
def test_scale(name):
    x = make(*WAYS[name])
    out, lse = attend(x, batch_of(x, scale=0.5))
    assert_attend(x, out, lse, scale=0.5)


@pytest.mark.parametrize("name", list(WAYS))
def test_rising_scores_rescale(name):
    # every key tile raises the maximum by far
    x = make(*WAYS[name])
    n = x["kp"].shape[0]
    ramp = torch.linspace(0.1, 40, n, device=DEV)[:, None, None]
    x["q"] = x["q"].abs()
    x["kp"] = (x["kp"].abs() * ramp).bfloat16()
    out, lse = attend(x, batch_of(x))
    assert_attend(x, out, lse)


def test_a_cache_beyond_4_gigabytes():
    # token strides that take offsets past 2^32 bytes
    n, stride = 40_000, 1 << 16
    room = torch.empty(n * stride, dtype=torch.bfloat16, device=DEV)
    for ql in ([1], [1, 2, 3, 4], [300]):
        x = make(2, 2, ql, [3] * len(ql), 8)
        g = torch.Generator(device=DEV).manual_seed(1)
        k = room.as_strided((n, 2, 64), (stride, 64, 1))
        v = room.as_strided((n, 2, 64), (stride, 64, 1), 128)
        k.copy_(torch.randn(n, 2, 64, generator=g, device=DEV))
        v.copy_(torch.randn(n, 2, 64, generator=g, device=DEV))
        x.update(kp=k, vp=v)
        out, lse = attend(x, batch_of(x))
        assert_attend(x, out, lse)
        z = exact_lse(x)
        assert_weights(x, weigh(x, batch_of(x), z, None, 1.0), z, None, 1.0)
    _, _, acc, ids = cache(2, n, 3)
    k0, v0 = k.clone(), v.clone()
    acc2, ids2 = torch.empty_like(acc), torch.empty_like(ids)
    G().cache_evict(n, 30_000, n, k, v, acc, ids, acc2, ids2, G().new_cache_workspace(2, n, 30_000))
    assert_evicted(k0, v0, acc, ids, 30_000, n, k, v, acc2, ids2)


@pytest.mark.parametrize("n", [1705, 6000])
def test_evict_slices_of_larger_tensors(n):
    k, v, acc, ids = cache(3, n, 8)
    kv = torch.full((n + 9, 2, 3, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    kv[:n, 0], kv[:n, 1] = k, v
    wide = [torch.full((3, n + 77), 7, dtype=t.dtype, device=DEV) for t in (acc, ids, acc, ids)]
    wide[0][:, :n], wide[1][:, :n] = acc, ids
    keep, recent_from = n - 400, n - 100
    G().cache_evict(n, keep, recent_from, kv[:, 0], kv[:, 1], *wide, G().new_cache_workspace(3, n, keep))
    assert_evicted(k, v, acc, ids, keep, recent_from, kv[:n, 0], kv[:n, 1], wide[2], wide[3])
    assert (kv[n:] == 7).all() and (wide[2][:, keep:] == 7).all() and (wide[3][:, keep:] == 7).all()


@pytest.mark.parametrize("n", [1000, 9000])
def test_evict_nothing_and_everything(n):
    k, v, acc, ids = cache(2, n, 4)
    assert_evicted(k, v, acc, ids, n, n, *evict(k, v, acc, ids, n, n))
    k2, v2, acc2, ids2 = evict(k, v, acc, ids, 0, n)
    assert torch.equal(k2, k) and torch.equal(v2, v)


def test_account_of_special_values():
    x = make(2, 2, [20], [20], 300)
    z = exact_lse(x)
    w = weigh(x, batch_of(x), z, None, 1.0)
    acc = torch.full((2, 300), float("nan"), device=DEV)
    assert torch.equal(weigh(x, batch_of(x), z, acc, 0.0), w)  # not read
    acc[:] = float("inf")
    got = weigh(x, batch_of(x), z, acc, 0.5)
    assert (got[:, :300] == float("inf")).all() and torch.equal(got[:, 300:], w[:, 300:])
    z[3] = float("-inf")  # a query that counts for nothing
    y = dict(x, q=x["q"].clone())
    y["q"][3] = 0
    z2 = z.clone()
    z2[3] = 1000.0
    assert torch.allclose(weigh(x, batch_of(x), z, None, 1.0), weigh(y, batch_of(y), z2, None, 1.0), rtol=1e-6)


@pytest.mark.parametrize("H,Hk", [(2, 1), (4, 2)])
@pytest.mark.parametrize("ql,tl", [([1], [9]), ([300, 280], [300, 280]), ([5, 3], [100, 50])])
def test_an_account_in_place_by_its_slice(H, Hk, ql, tl):
    x = make(H, Hk, ql, tl, 700)
    z = exact_lse(x)
    acc = torch.full((Hk, 1200 + sum(tl)), 7.0, device=DEV)
    acc[:, :700] = torch.rand(Hk, 700, device=DEV)
    before = acc[:, :700].clone()
    weigh(x, batch_of(x), z, acc[:, :700], 0.5, acc)
    assert_weights(x, acc, z, before, 0.5)
    assert (acc[:, 700 + sum(tl):] == 7).all()


@pytest.mark.parametrize("name", list(ACCOUNTS))
def test_log_sums_may_be_any_number(name):
    # far below the scores: large weights, and infinity beyond fp32; far above: nothing
    x = make(*ACCOUNTS[name])
    batch, z0 = batch_of(x), exact_lse(x)
    P = x["kp"].shape[0]
    for by in (-60.0, 40.0):
        assert_weights(x, weigh(x, batch, z0 + by, None, 1.0), z0 + by, None, 1.0)
    for b, rows, cols in R.views(x["q_off"], x["own_off"]):
        for i in range(rows.start, min(rows.stop, rows.start + 16)):
            for by, inf in ((-150.0, True), (-1e30, True), (R.NEG + 0, False), (1e30, False)):
                z = z0.clone()
                z[i] += by
                got = weigh(x, batch, z, None, 1.0)
                want = torch.zeros_like(got, dtype=torch.bool)
                want[:, :P] = inf
                want[:, P + cols.start:P + cols.stop] = inf
                assert torch.equal(got == float("inf"), want) and not got.isnan().any(), (b, i, by)


# ---------------------------------------------------------------------------------------------------------------
# streams, graphs, errors


@pytest.mark.parametrize("name", list(WAYS) + ["split rows"])
def test_equal_calls_give_equal_bits(name):
    x = make(*(WAYS | SIZES)[name])
    batch = batch_of(x)
    a, b = attend(x, batch), attend(x, batch)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    z = exact_lse(x)
    assert torch.equal(weigh(x, batch, z, None, 1.0), weigh(x, batch, z, None, 1.0))


def test_another_stream():
    side = torch.cuda.Stream()
    x = make(*WAYS["mixed views"])
    k, v, acc, ids = cache(2, 5000, 6)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)  # what runs on the wrong stream would be early
        y = {n: (t.clone() if isinstance(t, torch.Tensor) else t) for n, t in x.items()}
        batch = batch_of(y)
        out, lse = attend(y, batch)
        w = weigh(y, batch, lse, None, 1.0)
        moved = evict(k, v, acc, ids, 3000, 4900)
    side.synchronize()
    # the stream as an argument
    ws = G().new_view_workspace(batch, stream=side)
    out2 = torch.zeros_like(out)
    lse2 = torch.zeros_like(lse)
    torch.cuda.synchronize()
    G().prefix_attn(batch, y["q"], y["kp"], y["vp"], y["ko"], y["vo"], ints(y["q_off"]), ints(y["own_off"]), out2, lse2, ws,
                    side)
    side.synchronize()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    assert_attend(x, out, lse)
    assert_weights(x, w, lse, None, 1.0)
    assert_evicted(k, v, acc, ids, 3000, 4900, *moved)


def test_a_workspace_belongs_to_its_stream():
    # freed memory that the current stream still writes is not handed to another stream
    x = make(2, 2, [300], [10], 6000)
    batch, side = batch_of(x), torch.cuda.Stream()
    n = G().view_workspace_size(batch)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    busy = torch.empty(n, dtype=torch.uint8, device=DEV)
    torch.cuda._sleep(50_000_000)
    busy.fill_(255)
    del busy
    ws = G().new_view_workspace(batch, stream=side)
    cache_ws = G().new_cache_workspace(2, 100, 50, stream=side)
    torch.cuda.synchronize()
    assert not ws[:256].any() and not cache_ws[:256].any()
    G().check_device_error(ws, side)


@pytest.mark.parametrize("name", list(WAYS))
def test_captured_calls(name):
    x = make(*WAYS[name])
    batch = batch_of(x, max_q=x["q"].shape[0], max_own=x["ko"].shape[0])
    P, nt = x["kp"].shape[0], x["ko"].shape[0]
    Hk = x["kp"].shape[1]
    ws, q_off, own_off = G().new_view_workspace(batch), ints(x["q_off"]), ints(x["own_off"])
    out = torch.full(x["q"].shape, 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full(x["q"].shape[:2], 7.0, device=DEV)
    acc, acc_out = torch.rand(Hk, P + nt, device=DEV), torch.full((Hk, P + nt), 7.0, device=DEV)
    k, v, ids = x["kp"].clone(), x["vp"].clone(), torch.arange(P, dtype=torch.int32, device=DEV).repeat(Hk, 1)
    keep, wide = P - 100, torch.full((Hk, P), 7.0, device=DEV)
    ids2, evict_ws = torch.zeros_like(ids), G().new_cache_workspace(Hk, P, P - 100)

    def calls():
        G().prefix_attn(batch, x["q"], x["kp"], x["vp"], x["ko"], x["vo"], q_off, own_off, out, lse, ws)
        G().key_weights(batch, x["q"], x["kp"], x["ko"], q_off, own_off, lse, acc, acc_out, 0.5, ws)
        G().cache_evict(P, keep, P, k, v, acc_out[:, :P].clone(), ids, wide, ids2, evict_ws)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        calls()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    # other inputs, and other views in the same buffers
    y = make(*WAYS[name], seed=9)
    if len(y["q_off"]) > 2:
        y["q_off"][1] -= min(1, y["q_off"][1])
        y["own_off"][-1] -= 3
    for n in ("q", "kp", "vp", "ko", "vo"):
        x[n].copy_(y[n])
    q_off.copy_(ints(y["q_off"]))
    own_off.copy_(ints(y["own_off"]))
    k.copy_(y["kp"])
    v.copy_(y["vp"])
    out.fill_(7)
    lse.fill_(7)
    acc_out.fill_(7)
    graph.replay()
    torch.cuda.synchronize()
    G().check_device_error(ws)
    assert_attend(y, out, lse)
    assert_weights(y, acc_out, lse, acc[:, :P], 0.5)
    assert_evicted(y["kp"], y["vp"], acc_out[:, :P], ids, keep, P, k, v, wide, ids2)


@pytest.mark.parametrize("name", list(WAYS))
def test_bad_offsets_are_reported(name):
    x = make(*WAYS[name])
    batch = batch_of(x)
    good = attend(x, batch)
    z = exact_lse(x)
    nq, nt, B = x["q"].shape[0], x["ko"].shape[0], len(x["q_off"]) - 1
    cases = [dict(own_off=x["own_off"][:-1] + [nt + 1]), dict(own_off=[-1] + x["own_off"][1:]),
             dict(q_off=x["q_off"][:-1] + [nq + 7])]
    if B > 1:
        cases += [dict(q_off=[0, nq] + [0] * (B - 1)), dict(own_off=[0] * B + [nt])]
    for case in cases:
        for call in (lambda y: attend(y, batch), lambda y: weigh(y, batch, z, None, 1.0)):
            with pytest.raises(G().GsaError) as e:
                call(x | case)
            assert e.value.status == 6, case
    again = attend(x, batch)
    assert torch.equal(again[0], good[0]) and torch.equal(again[1], good[1])


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("H,Hk,ql,tl,prefix", [
    (2, 2, [1] * 9, [4000, 0, 1, 255, 256, 257, 31, 4096, 2], 700),   # blocks of 16 warps, one row
    (2, 2, [3, 1, 4, 2, 0, 3], [4000, 3, 4096, 0, 300, 65], 0),       # two rows, an odd number of them
    (4, 1, [1, 4, 3, 2], [2000, 511, 513, 4096], 300),                # rows of a key head's group
    (5, 1, [3, 2, 1], [1030, 17, 700], 300),
    (64, 64, [1] * 40, [300 - i for i in range(40)], 130),            # blocks of four warps
    (32, 32, [2] * 40, [300 + 7 * i for i in range(40)], 130),
    (2, 2, [1] * 70, [i % 3 for i in range(70)], 300),                # keys of several views and of none, side by side
])
def test_few_rows_over_many_own_keys(H, Hk, ql, tl, prefix, causal):
    everything(make(H, Hk, ql, tl, prefix), causal)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("name", list(WAYS))
def test_offsets_may_be_any_number(name, causal):
    # products and differences of these leave 32 bits
    x = make(*WAYS[name])
    batch = batch_of(x, causal)
    z = exact_lse(x, causal)
    good = attend(x, batch)
    weights = weigh(x, batch, z, None, 1.0)
    B = len(x["q_off"]) - 1
    for wild in (-(2**31), -(2**30) - 1, 2**30, 2**30 + 2**29, 2**31 - 1):
        for field in ("q_off", "own_off"):
            for i in range(B + 1):
                y = x | {field: x[field][:i] + [wild] + x[field][i + 1 :]}
                for call in (lambda: attend(y, batch), lambda: weigh(y, batch, z, None, 1.0)):
                    with pytest.raises(G().GsaError) as e:
                        call()
                    assert e.value.status == 6, (field, i, wild)
    again = attend(x, batch)
    assert torch.equal(again[0], good[0]) and torch.equal(again[1], good[1])
    assert torch.equal(weigh(x, batch, z, None, 1.0), weights)


@pytest.mark.parametrize("H,ql,prefix", [(2, [1], 300), (2, [1], 20000), (2, [20], 300), (2, [300], 300), (2, [300], 6000),
                                         (2, [4], 0), (2, [300], 0)])
def test_offsets_are_looked_at_where_no_own_key_is_expected(H, ql, prefix):
    x = make(H, H, ql, [40], prefix)
    z = exact_lse(x)
    none, no_queries = batch_of(x, max_own=0), batch_of(x, max_q=0)
    for batch in (none, no_queries):
        for call in (lambda b: attend(x, b), lambda b: weigh(x, b, z, None, 1.0)):
            with pytest.raises(G().GsaError) as e:
                call(batch)
            assert e.value.status == 6
    y = x | dict(own_off=[0, 0])
    out, lse = attend(y, none)
    assert_attend(y, out, lse)
    assert_weights(y, weigh(y, none, exact_lse(y), None, 1.0), exact_lse(y), None, 1.0)
    y = x | dict(q_off=[0, 0])
    out, lse = attend(y, no_queries)
    assert (out == 7).all() and (lse == 7).all()
    w = weigh(y, no_queries, z, None, 1.0)
    assert (w == 0).all()  # nobody looked


def test_offsets_written_by_the_kernel_before():
    # a batch without any key is one kernel; its offsets are what the call before leaves: log sums of 0 are the number 0
    n = 200_000
    x = make(1, 1, [n], [0], 1)
    x["q"] = torch.zeros_like(x["q"])
    batch, ws = batch_of(x), G().new_view_workspace(batch_of(x))
    off, out, lse = ints([0, n]), torch.empty_like(x["q"]), torch.empty(n, 1, device=DEV)
    none = G().ViewBatch(n_views=1, n_q=300, n_own=0, n_prefix=0, n_heads=1)
    ws2, out2, lse2 = G().new_view_workspace(none), torch.full((300, 1, 64), 7.0, device=DEV).bfloat16(), torch.full((300, 1), 7.0, device=DEV)
    for _ in range(20):
        lse.view(torch.int32).fill_(1 << 30)
        G().prefix_attn(batch, x["q"], x["kp"], x["vp"], None, None, off, ints([0, 0]), out, lse, ws)
        late = lse.view(torch.int32).flatten()[-2:]
        G().prefix_attn(none, x["q"][:300], None, None, None, None, late, ints([0, 0]), out2, lse2, ws2)
        G().check_device_error(ws2)
        assert (late == 0).all() and (out2 == 7).all() and (lse2 == 7).all()
    off2 = ints([0, 300])
    G().prefix_attn(none, x["q"][:300], None, None, None, None, off2, ints([0, 0]), out2, lse2, ws2)
    assert (out2 == 0).all() and (lse2 == R.NEG).all()


@pytest.mark.parametrize("prefix", [1, 100, 6000])
def test_offsets_are_looked_at_behind_a_padded_front(prefix):
    # the first tiles hold no view's rows
    x = make(2, 2, [300, 40], [0, 0], prefix)
    x["q"] = torch.cat((torch.full((700, 2, 64), float("nan"), dtype=torch.bfloat16, device=DEV), x["q"]))
    x["q_off"] = [700 + a for a in x["q_off"]]
    batch = batch_of(x)
    out, lse = attend(x, batch)
    assert_attend(x, out, lse)
    for case in (dict(own_off=[0, 0, 40]), dict(q_off=[700, 650, 1040]), dict(q_off=[1040, 1040, 700]), dict(q_off=[0, -1, -5])):
        for call in (lambda y: attend(y, batch), lambda y: weigh(y, batch, lse, None, 1.0)):
            with pytest.raises(G().GsaError) as e:
                call(x | case)
            assert e.value.status == 6, case


def test_many_views_of_unknown_length():
    # the default sizes: every view may hold all tokens
    x = make(1, 1, [10 - i % 3 for i in range(2000)], [11 - i % 4 for i in range(2000)], 300)
    batch = batch_of(x, max_q=-1, max_own=-1)
    assert batch.c().max_q == x["q"].shape[0]
    out, lse = attend(x, batch)
    assert_attend(x, out, lse)
    z = exact_lse(x)
    assert_weights(x, weigh(x, batch, z, None, 1.0), z, None, 1.0)


def test_more_views_than_a_short_number():
    n, P = 140_000, 40
    x = make(1, 1, [1] * n, [1] * n, P)
    batch = batch_of(x)
    out, lse = attend(x, batch)
    q, kp, vp, ko, vo = (x[t][:, 0].double() for t in ("q", "kp", "vp", "ko", "vo"))
    s = torch.cat((q @ kp.T, (q * ko).sum(1, keepdim=True)), 1) * 0.125
    z = torch.logsumexp(s, 1)
    p = (s - z[:, None]).exp()
    v = torch.cat((vp, vo[:1] * 0))  # own values apart: one for each query
    o = p @ v + p[:, P:] * vo
    # roundings of the weights and the result to bf16; sums, logits and exponentials of 41 terms are within 2e-5
    size = p[:, :P] @ vp.abs() + p[:, P:] * vo.abs()
    assert ((out[:, 0].double() - o).abs() <= (R.U16 + 2e-5) * 1.01 * size + R.U16 * 1.01 * o.abs()).all()
    assert ((lse[:, 0].double() - z).abs() <= 2e-5 * (1 + z.abs())).all()
    w = weigh(x, batch, lse, None, 1.0)[0].double()
    assert ((w[P:] - p[:, P]).abs() <= 1e-4 * p[:, P]).all()
    # 140000 terms: at most n / 64 + 64 roundings of a sum on the way
    assert ((w[:P] - p[:, :P].sum(0)).abs() <= (1e-4 + (n / 64 + 64) * R.U32) * p[:, :P].sum(0)).all()


def test_waits_that_run_out():
    # the hardware itself holds a waiting thread for a microsecond or so before the limit is looked at, so this takes
    # waits that are longer: the copies' on a full ring of key or query tiles
    x = make(2, 2, [3000], [10], 6000)
    batch, z = batch_of(x), exact_lse(x)
    short = batch_of(x, wait_limit_ns=1)
    for call in (lambda b: attend(x, b), lambda b: weigh(x, b, z, None, 1.0)):
        with pytest.raises(G().GsaError) as e:
            call(short)
        assert e.value.status == 5
    out, lse = attend(x, batch)
    assert_attend(x, out, lse)
    assert_weights(x, weigh(x, batch, z, None, 1.0), z, None, 1.0)


def test_python_refusals():
    x = make(2, 2, [5], [5], 300)
    batch = batch_of(x)
    ws, off = G().new_view_workspace(batch), ints([0, 5])
    out, lse = torch.empty_like(x["q"]), torch.empty(5, 2, device=DEV)
    args = [x["q"], x["kp"], x["vp"], x["ko"], x["vo"], off, off, out, lse, ws]
    for i, bad in ((0, x["q"].float()), (0, x["q"][:4]), (0, x["q"].cpu()), (0, None), (1, x["kp"][:, :, ::2]), (2, x["vp"][:, :1]),
                   (3, x["ko"].transpose(0, 1)), (5, off.long()), (5, ints([0, 5, 5])), (8, lse[:, :1]), (8, lse.double()),
                   (9, ws[:100]), (9, ws.cpu())):
        with pytest.raises(ValueError):
            G().prefix_attn(batch, *args[:i], bad, *args[i + 1:])
    with pytest.raises(G().GsaError) as e:  # two bytes off
        G().prefix_attn(batch, torch.empty(5 * 128 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(5, 2, 64), *args[1:])
    assert e.value.status == 1
    big = batch_of(make(2, 2, [300], [10], 6000))
    y = make(2, 2, [300], [10], 6000)
    with pytest.raises(G().GsaError) as e:
        G().prefix_attn(big, y["q"], y["kp"], y["vp"], y["ko"], y["vo"], ints([0, 300]), ints([0, 10]), torch.empty_like(y["q"]),
                        None, G().new_workspace(None))
    assert e.value.status == 3
    k, v, acc, ids = cache(2, 100, 1)
    evict_ws = G().new_cache_workspace(2, 100, 50)
    for bad in ((k, v, acc, ids, acc, torch.empty_like(ids)), (k, v, acc, ids, torch.empty_like(acc), ids)):
        with pytest.raises(G().GsaError):
            G().cache_evict(100, 50, 100, *bad, evict_ws)
    with pytest.raises(ValueError):
        G().cache_evict(101, 50, 100, k, v, acc, ids, torch.empty_like(acc), torch.empty_like(ids), evict_ws)


def test_a_token_number_that_does_not_fit_is_refused():
    k, v, acc, ids = cache(2, 100, 1)
    before = k.clone()
    for keep, recent_from in ((50, 2 ** 31), (2 ** 32 + 50, 100), (50, -2 ** 31 - 1)):
        with pytest.raises(ValueError, match="32 bits"):
            G().cache_evict(100, keep, recent_from, k, v, acc, ids, acc.clone(), ids.clone(), G().new_cache_workspace(2, 100, 50))
    assert torch.equal(k, before)
    assert_evicted(k, v, acc, ids, 50, 2 ** 31 - 1, *evict(k, v, acc, ids, 50, 2 ** 31 - 1))


def test_expanded_tensors_are_refused():
    x = make(2, 2, [5], [5], 300)
    batch = batch_of(x)
    ws, off = G().new_view_workspace(batch), ints([0, 5])
    out, lse = torch.empty_like(x["q"]), torch.empty(5, 2, device=DEV)
    args = [x["q"], x["kp"], x["vp"], x["ko"], x["vo"], off, off, out, lse, ws]
    shared = lambda t: t[:1].expand_as(t)  # noqa: E731
    for i in (0, 1, 2, 3, 4, 7):
        with pytest.raises(ValueError):
            G().prefix_attn(batch, *args[:i], shared(args[i]), *args[i + 1:])
    args = [x["q"], x["kp"], x["ko"], off, off, lse, None, torch.empty(2, 305, device=DEV), 1.0, ws]
    for i in (0, 1, 2):
        with pytest.raises(ValueError):
            G().key_weights(batch, *args[:i], shared(args[i]), *args[i + 1:])
    k, v, acc, ids = cache(2, 100, 1)
    for kv in ((shared(k), v), (k, shared(v))):
        with pytest.raises(ValueError):
            G().cache_evict(90, 50, 100, *kv, acc, ids, acc.clone(), ids.clone(), G().new_cache_workspace(2, 100, 50))


# ---------------------------------------------------------------------------------------------------------------
# a stream of views


@pytest.mark.parametrize("H,Hk", [(4, 4), (6, 2)])
def test_a_stream_of_views(H, Hk):
    c = G().ViewCache(700, H, Hk)
    g = torch.Generator(device=DEV).manual_seed(2)
    seen_k, seen_v = [], []  # every token ever appended
    acc = torch.zeros(Hk, 0, dtype=torch.float64, device=DEV)
    heads = torch.arange(Hk, device=DEV)
    for step, lens in enumerate(([60], [1], [40, 3, 120], [130], [2, 2], [200], [90])):
        n = sum(lens)
        q, k, v = (torch.randn(n, h, 64, generator=g, device=DEV).bfloat16() for h in (H, Hk, Hk))
        kp, vp, ids = c.k[:c.n].clone(), c.v[:c.n].clone(), c.ids[:, :c.n].clone()
        if c.n:
            # the cache holds the tokens that its numbers say
            assert torch.equal(kp, torch.cat(seen_k)[ids.T.long(), heads]) and torch.equal(vp, torch.cat(seen_v)[ids.T.long(), heads])
        before = c.acc[:, :c.n].clone()
        out = c.step(q, k, v, lens, decay=0.5)
        c.check_device_error()
        off = offsets(lens)
        o, z, to, _ = R.attend(q, kp, vp, k, v, off, off)
        assert ((out.double() - o).abs() <= to).all(), step
        w, tol = R.weights(q, kp, k, off, off, z.float(), before, 0.5)
        # the account goes by the kernel's own log sums: their error comes on top
        assert ((c.acc[:, :c.n].double() - w).abs() <= tol + 2e-5 * w).all(), step
        seen_k.append(k)
        seen_v.append(v)
        assert c.n == kp.shape[0] + n and torch.equal(c.ids[:, c.n - n:c.n], c.ids[:1, c.n - n:c.n].expand(Hk, n))
        if c.n > 300:
            ids, acc, full = c.ids[:, :c.n].clone(), c.acc[:, :c.n].clone(), c.next_id
            c.evict(300, recent=50)
            src = R.evict(acc.cpu(), ids.cpu(), 300, full - 50).to(DEV)
            assert c.n == 300 and torch.equal(c.ids[:, :300], ids[heads[:, None], src])
            assert all((c.ids[:, :300] == i).any(1).all() for i in range(full - 50, full))
    with pytest.raises(ValueError):
        c.step(*(torch.zeros(500, h, 64, dtype=torch.bfloat16, device=DEV) for h in (H, Hk, Hk)))


def test_errors_outlive_a_workspace():
    c = G().ViewCache(20_000, 2)
    g = torch.Generator(device=DEV).manual_seed(4)
    step = lambda n: c.step(*(torch.randn(n, 2, 64, generator=g, device=DEV).bfloat16() for _ in range(3)))  # noqa: E731
    step(40)
    small = c._ws.numel()
    c._ws[:4].view(torch.int32)[0] = 2  # what a kernel leaves whose check failed
    step(6000)
    assert c._ws.numel() > small
    step(300)
    with pytest.raises(G().GsaError) as e:
        c.check_device_error()
    assert e.value.status == 6
    step(3)
    c.check_device_error()  # reported once


def test_the_last_token_numbers():
    c = G().ViewCache(100, 2)
    g = torch.Generator(device=DEV).manual_seed(5)
    step = lambda n: c.step(*(torch.randn(n, 2, 64, generator=g, device=DEV).bfloat16() for _ in range(3)))  # noqa: E731
    c.next_id = 2 ** 31 - 51
    step(20)
    step(30)
    assert c.next_id == 2 ** 31 - 1 and c.ids[:, :50].tolist() == [list(range(2 ** 31 - 51, 2 ** 31 - 1))] * 2
    n, acc, k = c.n, c.acc.clone(), c.k.clone()
    with pytest.raises(ValueError):
        step(1)
    assert c.n == n and torch.equal(c.acc, acc) and torch.equal(c.k[:n], k[:n])
    # none of them is recent; then some; then more than there ever were
    for keep, recent in ((40, 0), (30, 10), (20, 2 ** 40)):
        ids, acc, last = c.ids[:, :c.n].clone(), c.acc[:, :c.n].clone(), 2 ** 31 - 1 - min(recent, 2 ** 31 - 1)
        c.evict(keep, recent)
        src = R.evict(acc.cpu(), ids.cpu(), keep, last).to(DEV)
        assert torch.equal(c.ids[:, :keep], ids.gather(1, src))


def test_a_cache_keeps_no_graph():
    c = G().ViewCache(100, 2)
    for _ in range(2):
        q, k, v = (torch.randn(20, 2, 64, device=DEV).bfloat16().requires_grad_() for _ in range(3))
        out = c.step(q, k * 1, v * 1)
        assert not any(t.requires_grad for t in (out, c.k, c.v, c.acc))
    c.evict(15)
    assert c.n == 15 and not c.k.requires_grad
