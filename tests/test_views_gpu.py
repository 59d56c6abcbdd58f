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
                                          (2, 5000, 1), (2, 5000, 4999), (2, 5000, 5000), (4, 8191, 4096), (1, 40000, 20001), (2, 4097, 3000),
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
