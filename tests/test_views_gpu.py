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
