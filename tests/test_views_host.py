"""The view-cache operators on the host: sizes, and arguments that are refused before anything is launched (every call
below fails validation, so no CUDA work is attempted)."""

import ctypes

import pytest
import torch

FAKE = 0x10000  # aligned, never dereferenced
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    from sparse_global_attention_view_b200 import build
    build.build()
    from sparse_global_attention_view_b200 import _lib
    return _lib.load()


def batch(**kw):
    from sparse_global_attention_view_b200 import _lib
    base = dict(n_views=3, n_heads=16, n_kv_heads=4, head_dim=64, n_q=300, n_own=200, n_prefix=1000, max_q=200, max_own=100,
                causal=0, scale=0.0, wait_limit_ns=0, q_stride=0, k_prefix_stride=0, v_prefix_stride=0, k_own_stride=0,
                v_own_stride=0, out_stride=0)
    base.update(kw)
    return _lib.GsaViewBatch(**base)


def cache(**kw):
    from sparse_global_attention_view_b200 import _lib
    base = dict(n_kv_heads=4, head_dim=64, n_tokens=1000, n_keep=700, recent_from=900, k_stride=0, v_stride=0, w_stride=1000)
    base.update(kw)
    return _lib.GsaCache(**base)


def size(lib, b):
    n = ctypes.c_size_t()
    return lib.view_workspace_size(ctypes.byref(b), ctypes.byref(n)), n.value


BAD_BATCHES = [
    (dict(n_views=0), 1), (dict(n_heads=0), 1), (dict(n_kv_heads=0), 1), (dict(n_kv_heads=3), 1), (dict(n_kv_heads=32), 1),
    (dict(head_dim=32), 2), (dict(head_dim=0), 1), (dict(n_heads=256, n_kv_heads=2), 2), (dict(n_q=-1, max_q=0), 1),
    (dict(n_own=-1, max_own=0), 1), (dict(n_prefix=-1), 1), (dict(max_q=301), 1), (dict(max_q=-1), 1), (dict(max_own=201), 1),
    (dict(max_own=-1), 1), (dict(causal=2), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(wait_limit_ns=-1), 1), (dict(n_prefix=2 ** 31 - 1000), 1), (dict(n_q=2 ** 30), 1),
    (dict(q_stride=1016), 1), (dict(q_stride=1028), 1), (dict(out_stride=64), 1), (dict(k_own_stride=248), 1),
    (dict(v_prefix_stride=-256), 1), (dict(k_prefix_stride=1 << 39), 1), (dict(n_views=2 ** 24), 1),
]


@pytest.mark.parametrize("kw,status", BAD_BATCHES)
def test_bad_batches_are_refused(lib, kw, status):
    b = batch(**kw)
    assert size(lib, b)[0] == status
    assert lib.prefix_attn(ctypes.byref(b), *[FAKE] * 10, BIG, None) == status
    assert lib.key_weights(ctypes.byref(b), *[FAKE] * 7, BIG >> 4, FAKE << 20, BIG >> 4, 1.0, FAKE, BIG, None) == status


def test_batches_that_are_fine(lib):
    for kw in (dict(), dict(n_kv_heads=16), dict(n_kv_heads=1), dict(n_heads=128, n_kv_heads=1), dict(n_q=0, max_q=0),
               dict(n_own=0, max_own=0), dict(n_prefix=0), dict(n_prefix=0, n_own=0, max_own=0), dict(max_own=0), dict(max_q=0),
               dict(q_stride=3 * 16 * 64, k_own_stride=512), dict(n_prefix=2 ** 30), dict(n_views=10000)):
        st, n = size(lib, batch(**kw))
        assert st == 0 and n >= 256 and n % 256 == 0, kw


def test_null_and_misaligned_pointers_are_refused(lib):
    b = ctypes.byref(batch())
    good = [FAKE] * 10  # q kp vp ko vo q_off own_off out lse ws
    assert lib.prefix_attn(None, *good, BIG, None) == 1
    for i in (0, 1, 2, 3, 4, 5, 6, 7, 9):
        assert lib.prefix_attn(b, *good[:i], None, *good[i + 1:], BIG, None) == 1, i
    for i in range(10):
        off = 2 if i in (5, 6, 8) else 8
        assert lib.prefix_attn(b, *good[:i], FAKE + off, *good[i + 1:], BIG, None) == 1, i
    assert lib.prefix_attn(b, *good, 255, None) == 3
    out = FAKE << 20
    good = [FAKE] * 7 + [1000, out, 1200, 1.0, FAKE, BIG]  # q kp ko q_off own_off lse acc stride out stride decay ws
    assert lib.key_weights(None, *good, None) == 1
    for i in (0, 1, 2, 3, 4, 5, 8, 11):
        assert lib.key_weights(b, *good[:i], None, *good[i + 1:], None) == 1, i
    for i, x in ((7, 999), (9, 1199), (10, -0.5), (10, float("nan")), (10, float("inf")), (6, FAKE + 2), (8, out + 2)):
        assert lib.key_weights(b, *good[:i], x, *good[i + 1:], None) == 1, (i, x)
    assert lib.key_weights(b, *good[:12], 255, None) == 3


def test_accounts_that_overlap_are_refused(lib):
    b = ctypes.byref(batch())
    for acc, acc_stride, out, out_stride in ((FAKE, 1200, FAKE + 4, 1200), (FAKE, 1200, FAKE, 1300), (FAKE + 4 * 1000, 1200, FAKE, 1200)):
        assert lib.key_weights(b, *[FAKE] * 6, acc, acc_stride, out, out_stride, 1.0, FAKE, BIG, None) == 1
    c = ctypes.byref(cache())
    span = 4 * 4 * 1000
    places = [FAKE + (i << 24) for i in range(4)]  # acc ids acc_out ids_out
    for i, j in ((0, 2), (1, 3), (0, 3), (1, 2), (2, 3)):
        p = list(places)
        p[j] = p[i] + span - 4
        assert lib.cache_evict(c, FAKE << 20, FAKE << 20, *p, FAKE, BIG, None) == 1, (i, j)


@pytest.mark.parametrize("kw,status", [
    (dict(n_kv_heads=0), 1), (dict(head_dim=0), 1), (dict(head_dim=128), 2), (dict(n_kv_heads=129), 2), (dict(n_tokens=-1), 1),
    (dict(n_keep=-1), 1), (dict(n_keep=1001), 1), (dict(w_stride=999), 1), (dict(k_stride=255), 1), (dict(k_stride=260), 1),
    (dict(v_stride=-1), 1), (dict(n_tokens=2 ** 31 - 1, w_stride=2 ** 31), 1)])
def test_bad_caches_are_refused(lib, kw, status):
    c = cache(**kw)
    n = ctypes.c_size_t()
    assert lib.cache_workspace_size(ctypes.byref(c), ctypes.byref(n)) == status
    p = [FAKE + (i << 44) for i in range(6)]
    assert lib.cache_evict(ctypes.byref(c), *p, FAKE, BIG, None) == status


def test_cache_pointers_are_refused(lib):
    c = ctypes.byref(cache())
    p = [FAKE + (i << 24) for i in range(7)]  # k v acc ids acc_out ids_out ws
    assert lib.cache_evict(None, *p, BIG, None) == 1
    for i in range(7):
        assert lib.cache_evict(c, *p[:i], None, *p[i + 1:], BIG, None) == 1, i
        assert lib.cache_evict(c, *p[:i], p[i] + (2 if 2 <= i < 6 else 8), *p[i + 1:], BIG, None) == 1, i
    assert lib.cache_evict(c, *p, 256, None) == 3
    n = ctypes.c_size_t()
    assert lib.cache_workspace_size(c, None) == 1 and lib.cache_workspace_size(c, ctypes.byref(n)) == 0
    assert n.value >= 256 + 4 * 4 * 2 * 300


def test_python_refuses_tensors_off_the_gpu(lib):
    import sparse_global_attention_view_b200 as G
    b = G.ViewBatch(n_views=1, n_q=2, n_own=2, n_prefix=2, n_heads=1)
    x, off = torch.zeros(2, 1, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="workspace"):
        G.prefix_attn(b, x, x, x, x, x, off, off, x, None, torch.zeros(4096, dtype=torch.uint8))
    with pytest.raises(ValueError, match="workspace"):
        G.key_weights(b, x, x, x, off, off, torch.zeros(2, 1), None, torch.zeros(1, 4), 1.0, torch.zeros(4096, dtype=torch.uint8))
    with pytest.raises(ValueError, match="workspace"):
        G.cache_evict(2, 1, 2, x, x, *[torch.zeros(1, 2)] * 4, torch.zeros(4096, dtype=torch.uint8))


def test_batch_defaults(lib):
    import sparse_global_attention_view_b200 as G
    b = G.ViewBatch(n_views=1, n_q=5, n_own=7, n_prefix=3, n_heads=8)
    c = b.copy_c()
    assert (c.n_kv_heads, c.max_q, c.max_own, c.causal, c.head_dim) == (8, 5, 7, 0, 64)
    c.q_stride = 4096
    assert b.copy_c().q_stride == 0  # each call has its own


def test_tokens_that_share_memory_are_refused(lib):
    # `_rows` takes host tensors for device -1, that of theirs: nothing is launched
    from sparse_global_attention_view_b200 import views
    x = torch.zeros(40, 2, 64, dtype=torch.bfloat16)
    one = x[:1]
    assert views._rows(x, 40, 2, -1, "x")[1] == 0 and views._rows(x[::2], 20, 2, -1, "x")[1] == 256
    assert views._rows(one, 1, 2, -1, "x")[1] == 0 and views._rows(one.expand(1, 2, 64), 1, 2, -1, "x")[1] == 0
    flat = x.flatten()
    for bad in (one.expand(40, 2, 64), flat.as_strided((40, 2, 64), (64, 64, 1)), flat[:64].view(1, 1, 64).expand(40, 2, 64),
                flat.as_strided((40, 2, 64), (120, 64, 1))):
        for exact in (True, False):
            with pytest.raises(ValueError):
                views._rows(bad, 40, 2, -1, "x", exact)
    for n in (40, 39):  # one head, a cache with room
        with pytest.raises(ValueError):
            views._rows(x[:1, :1].expand(40, 1, 64), n, 1, -1, "x", False)


def test_many_views_are_fine(lib):
    frame = 1374
    for kw in (dict(n_views=200, n_q=200 * frame, n_own=200 * frame, max_q=200 * frame, max_own=200 * frame),  # the defaults
               dict(n_views=1000, n_q=1000 * frame, n_own=1000 * frame, max_q=1000 * frame, max_own=1000 * frame, n_kv_heads=16),
               dict(n_views=131072, max_q=1), dict(n_views=5_000_000, n_q=5_000_000, max_q=1, n_own=5_000_000, max_own=1),
               dict(n_views=2 ** 25 - 1, max_q=64, max_own=0), dict(n_views=2 ** 24 - 1, max_q=65, max_own=0)):
        st, n = size(lib, batch(**kw))
        assert st == 0 and n >= 256, kw
    for kw in (dict(n_views=2 ** 25, max_q=64), dict(n_views=2 ** 24, max_q=65), dict(n_views=2 ** 25, max_q=0),
               dict(n_views=2 ** 24, n_heads=128, n_kv_heads=1, max_q=3)):
        assert size(lib, batch(**kw))[0] == 1, kw


def test_accounts_of_too_many_views_are_refused(lib):
    # views, heads and items of 512 own tokens: more of them than 32 bits count
    args = [FAKE] * 6 + [None, 0, FAKE << 20, BIG >> 4, 1.0, FAKE, 1 << 62, None]
    for kw in (dict(n_views=2 ** 27 // 16, n_kv_heads=16, n_own=20 * 512, max_own=16 * 512), dict(n_views=2 ** 24, max_q=64, max_own=100, n_kv_heads=128, n_heads=128)):
        b = batch(**kw)
        assert size(lib, b)[0] == 0, kw
        assert lib.key_weights(ctypes.byref(b), *args) == 1, kw


def test_numbers_beyond_32_bits_are_refused(lib):
    import sparse_global_attention_view_b200 as G
    from sparse_global_attention_view_b200 import views
    base = dict(n_views=1, n_q=5, n_own=7, n_prefix=3, n_heads=8)
    for name in ("n_views", "n_q", "n_own", "n_prefix", "n_heads", "n_kv_heads", "max_q", "max_own", "wait_limit_ns"):
        for x in (2 ** 32 + base.get(name, 5), -2 ** 32 + 5):
            with pytest.raises(ValueError, match="32 bits"):
                G.view_workspace_size(G.ViewBatch(**base | {name: x}))
    assert G.view_workspace_size(G.ViewBatch(**base)) >= 256
    # n_keep of 2^32 + 5 is not 5, and recent_from of 2^31 (no token is so recent) not -2^31 (all are)
    for args in ((4, 100, 2 ** 32 + 5, 0), (4, 100, 50, 2 ** 31), (4, 100, 50, -2 ** 31 - 1), (4, 2 ** 32 + 100, 50, 0), (2 ** 32 + 4, 100, 50, 0)):
        with pytest.raises(ValueError, match="32 bits"):
            views._cache(*args, 0, 0, 100)
    with pytest.raises(ValueError, match="32 bits"):
        G.cache_workspace_size(4, 100, 2 ** 32 + 5)
    assert views._cache(4, 100, 50, 2 ** 31 - 1, 0, 0, 100).recent_from == 2 ** 31 - 1


def test_a_cache_refuses_steps_before_it_changes(lib):
    import sparse_global_attention_view_b200 as G
    x = torch.zeros(6, 2, 64, dtype=torch.bfloat16)
    c = G.ViewCache(100, 2, device="cpu")  # nothing below gets as far as a kernel
    for lens in ([7, -1], [5], [], [6, 1]):
        with pytest.raises(ValueError, match="views of"):
            c.step(x, x, x, lens)
    with pytest.raises(ValueError, match="do not fit a cache"):
        c.step(*[torch.zeros(101, 2, 64, dtype=torch.bfloat16)] * 3)
    c.next_id = 2 ** 31 - 6
    with pytest.raises(ValueError, match="have no number"):
        c.step(x, x, x)
    assert c.n == 0 and c.next_id == 2 ** 31 - 6 and not c.ids.any()


def test_one_row_of_an_account_has_no_stride(lib):
    # in place, as a slice of acc_out: refused for its small workspace alone
    for kw, status in ((dict(n_kv_heads=1), 3), (dict(n_kv_heads=2), 1)):
        b = batch(**kw)
        assert lib.key_weights(ctypes.byref(b), *[FAKE] * 6, FAKE, 1000, FAKE, 1200, 1.0, FAKE, 255, None) == status
    b = batch(n_kv_heads=1)
    assert lib.key_weights(ctypes.byref(b), *[FAKE] * 6, FAKE + 4, 1000, FAKE, 1200, 1.0, FAKE, 255, None) == 1
