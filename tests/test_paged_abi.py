"""Host-only checks of the rotary and paged calls: workspace sizes, and every refusal that needs no
GPU (the pointers are never dereferenced), of the C ABI and of the binding."""
import ctypes

import pytest
import torch

from sparse_long_context_cca_gb300 import api
from sparse_long_context_cca_gb300 import build as cbuild

BAD, UNSUP = api.CCA_ERR_INVALID_ARG, api.CCA_ERR_UNSUPPORTED
P = [0x100000 * (k + 1) for k in range(16)]


@pytest.fixture(scope="module")
def lib():
    cbuild.build()
    return api.load_library()


def rope_params(*v):
    return ctypes.byref(api.CcaRopeParams(*v))


def rope_tensors(*each):
    """x, y, H, three strides of x, three of y; one or more tensors."""
    return (api.CcaRopeTensor * len(each))(*[api.CcaRopeTensor(*e[:3], (ctypes.c_int64 * 3)(*e[3:6]), (ctypes.c_int64 * 3)(*e[6:9]))
                                             for e in each])


def rope_call(lib, x=None, y=None, n=1, xs=(8192, 4096, 64), ys=None, H=2, second=None, **kw):
    prm = dict(B=1, N=64, d=64, rot=64, layout=0, dtype=api.CCA_F32, inverse=0, factor=1.0, inv_freq=P[8], positions=0,
               pos_stride=0, start=0)
    prm.update(kw)
    first = (P[0] if x is None else x, P[1] if y is None else y, H, *xs, *(ys or xs))
    t = rope_tensors(first, *([second] if second is not None else []))
    return lib.cca_rope(t, n, rope_params(*prm.values()), None)


@pytest.mark.parametrize("kw", [
    dict(B=0), dict(N=0), dict(rot=63), dict(rot=-2), dict(rot=66), dict(layout=2), dict(dtype=7), dict(inverse=2),
    dict(factor=float("nan")), dict(inv_freq=0), dict(inv_freq=P[8] + 4), dict(positions=P[9] + 2), dict(pos_stride=-1),
    dict(x=0), dict(y=0), dict(x=P[0] + 8), dict(y=P[1] + 4), dict(xs=(8192, 4096, 63)), dict(xs=(8192, 4096, 2 ** 60)),
    dict(H=0), dict(n=0), dict(n=3), dict(y=P[0], ys=(8192, 64, 128)),      # over itself with other strides
    dict(y=P[0] + 4096),                                                    # half over itself
    dict(ys=(8192, 32, 64)), dict(ys=(8192, 0, 64)), dict(ys=(8192, 4096, -64)),   # rows that share memory
])
def test_rope_refuses(lib, kw):
    assert rope_call(lib, **kw) == BAD


def test_rope_refuses_two_tensors_that_meet(lib):
    s = (8192, 4096, 64)
    assert rope_call(lib, n=2, second=(P[2], P[1], 2, *s, *s)) == BAD            # one output for both
    assert rope_call(lib, n=2, second=(P[1], P[2], 2, *s, *s)) == BAD            # the second reads the first's output
    assert rope_call(lib, y=P[0], n=2, second=(P[0], P[0], 2, *s, *s)) == BAD    # the same tensor twice in place
    assert rope_call(lib, d=96, rot=64) == UNSUP
    assert lib.cca_rope(None, 1, rope_params(1, 64, 64, 64, 0, 1, 0, 1.0, P[8], 0, 0, 0), None) == BAD
    assert lib.cca_rope(rope_tensors((P[0], P[1], 2, *s, *s)), 1, None, None) == BAD


def append_call(lib, q=True, kv=None, pages=None, lens=P[4], parents=0, counts=0, status=0, **kw):
    prm = dict(B=2, N=4, d=64, rot=64, layout=0, dtype=api.CCA_F32, inverse=0, factor=1.0, inv_freq=P[8], positions=0,
               pos_stride=0, start=0)
    prm.update(kw)
    s = (4 * 64 * 2, 4 * 64, 64)
    t = lambda x, y: rope_tensors((x, y, 2, *s, *s))  # noqa: E731
    k, v = kv or (P[2], P[3])
    pg = dict(K=P[5], V=P[6], table=P[7], n_pages=4, rows=16, cols=2, layers=1)
    pg.update(pages or {})
    return lib.cca_rope_append(t(P[0], P[1]) if q else None, t(k, 0), t(v, 0), ctypes.byref(api.CcaPages(*pg.values())),
                               lens or None, parents or None, counts or None, status or None, rope_params(*prm.values()), None)


@pytest.mark.parametrize("kw", [
    dict(positions=P[9]), dict(start=3), dict(inverse=1), dict(lens=0), dict(lens=P[4] + 2), dict(parents=P[4] + 1),
    dict(counts=P[4] + 2), dict(status=P[4] + 1), dict(B=65536), dict(pages=dict(K=0)), dict(pages=dict(V=P[6] + 8)),
    dict(pages=dict(table=0)), dict(pages=dict(n_pages=0)), dict(pages=dict(rows=0)), dict(pages=dict(cols=0)),
    dict(pages=dict(layers=2)), dict(pages=dict(V=P[5] + 64)), dict(kv=(P[5] + 4096, P[3])), dict(kv=(P[1] + 1024, P[3])),
    dict(kv=(0, P[3])),
])
def test_append_refuses(lib, kw):
    assert append_call(lib, **kw) == BAD


def test_append_tree_limit(lib):
    assert append_call(lib, N=257, parents=P[9], q=False) == UNSUP


def params(**kw):
    p = dict(B=2, Hq=4, Hkv=2, N=0, d=128, g=16, w=64, dtype=api.CCA_BF16, scale=0.0, status=0, window_mode=0, pool_mode=0)
    p.update(kw)
    return ctypes.pointer(api.CcaParams(*p.values()))


def pages(**kw):
    p = dict(K=P[0], V=P[1], table=P[2], n_pages=4, rows=16, cols=8, layers=1)
    p.update(kw)
    return ctypes.pointer(api.CcaPages(*p.values()))


CORE = dict(K=P[3], V=P[4], table=P[5], rows=4)


def tree_call(lib, T=4, raw=None, core=None, lens=P[6], parents=0, Q=P[7], O=P[8], L=P[9], ws=P[10], ws_bytes=None, prm=None):
    prm = params() if prm is None else prm
    need = lib.cca_tree_workspace_size(prm, T)
    return lib.cca_tree_fwd(Q or None, pages(**(raw or {})), pages(**{**CORE, **(core or {})}), lens or None, parents or None, T,
                            O or None, L or None, prm, ws or None, need if ws_bytes is None else ws_bytes, None)


@pytest.mark.parametrize("kw", [
    dict(T=0), dict(Q=0), dict(O=0), dict(L=0), dict(ws=0), dict(Q=P[7] + 8), dict(ws=P[10] + 4), dict(lens=0), dict(lens=P[6] + 1),
    dict(parents=P[6] + 2), dict(raw=dict(K=0)), dict(core=dict(V=0)), dict(core=dict(table=P[5] + 1)), dict(raw=dict(layers=2)),
    dict(O=P[7]), dict(ws_bytes=16), dict(prm=params(Hq=3)), dict(prm=params(g=0)), dict(prm=params(w=0)), dict(prm=params(dtype=4)),
    dict(prm=params(scale=float("inf"))), dict(prm=params(window_mode=2)), dict(prm=params(status=P[6] + 2)), dict(prm=params(B=0)),
])
def test_tree_refuses(lib, kw):
    assert tree_call(lib, **kw) == BAD


@pytest.mark.parametrize("kw", [dict(T=65), dict(T=257, prm=params(w=1024)), dict(prm=params(d=96)), dict(prm=params(B=1025)),
                                dict(prm=params(B=1024, Hq=512, Hkv=512, g=1), raw=dict(rows=1 << 20, cols=1 << 10))])
def test_tree_limits(lib, kw):
    assert tree_call(lib, ws_bytes=1 << 40, **kw) == UNSUP


def test_tree_workspace_size(lib):
    assert lib.cca_tree_workspace_size(params(), 0) == 0 and lib.cca_tree_workspace_size(params(d=96), 4) == 0
    assert lib.cca_tree_workspace_size(None, 4) == 0
    # it depends on the rows of a KV head alone, not on the lengths
    assert lib.cca_tree_workspace_size(params(), 4) == lib.cca_tree_workspace_size(params(B=500, g=4), 4) > 0
    assert lib.cca_tree_workspace_size(params(w=1024), 256) > lib.cca_tree_workspace_size(params(), 4)


def pool_call(lib, T=8, A=4, path=P[8], raw=None, core=None, Q=P[6], lens=P[7], acc=P[9], prm=None):
    return lib.cca_pool_pages(Q or None, pages(**(raw or {})), pages(**{**CORE, **(core or {})}), lens or None, acc or None, path or None,
                              A, T, params() if prm is None else prm, None)


@pytest.mark.parametrize("kw", [
    dict(T=0), dict(A=0), dict(path=0), dict(path=P[8] + 1), dict(Q=0), dict(Q=P[6] + 2), dict(lens=0), dict(acc=0), dict(acc=P[9] + 2),
    dict(raw=dict(cols=0)), dict(core=dict(rows=0)), dict(core=dict(V=P[3])), dict(core=dict(K=P[0])), dict(core=dict(V=P[0] + 4096)),
    dict(prm=params(pool_mode=4)), dict(prm=params(g=0)),
])
def test_pool_pages_refuses(lib, kw):
    assert pool_call(lib, **kw) == BAD


def test_pool_pages_limits(lib):
    assert pool_call(lib, prm=params(Hq=18, pool_mode=3)) == UNSUP      # 9 heads share a KV head
    assert pool_call(lib, prm=params(d=32)) == UNSUP


def test_page_book_refuses(lib):
    ws = lib.cca_pages_reserve_workspace_size(4, 8)
    assert ws >= 4 * (4 * 8 + 4) and lib.cca_pages_reserve_workspace_size(0, 8) == 0
    good = [P[0], 16, P[1], 4, 8, 64, P[2], P[3], P[4], P[5], ws, None, None]
    for k, v in ((0, None), (0, P[0] + 1), (1, 0), (2, None), (3, 0), (4, 0), (5, 0), (6, None), (7, P[3] + 2), (8, None), (9, None),
                 (9, P[5] + 8), (10, ws - 1), (11, P[6] + 1)):
        a = list(good)
        a[k] = v
        assert lib.cca_pages_reserve(*a) == BAD, k
    good = [P[0], 16, P[1], 4, 8, 64, P[2], P[3], 2, P[4], None, None]
    for k, v in ((0, None), (1, -1), (2, P[1] + 1), (3, 0), (4, 0), (5, 0), (6, None), (7, P[3] + 1), (8, -1), (9, None), (10, P[5] + 2)):
        a = list(good)
        a[k] = v
        assert lib.cca_pages_fork(*a) == BAD, k
    assert lib.cca_pages_fork(*good[:8], 65537, *good[9:]) == UNSUP
    good = [P[0], 16, P[1], 4, 8, P[2], P[3], None, None]
    for k, v in ((0, None), (1, 0), (2, None), (3, -1), (4, 0), (5, None), (6, P[3] + 2), (7, P[5] + 1)):
        a = list(good)
        a[k] = v
        assert lib.cca_pages_free(*a) == BAD, k


def test_page_moves_refuse(lib):
    good = [pages(), P[6], 3, params(), None]
    for k, v in ((0, None), (0, pages(K=0)), (0, pages(V=P[1] + 8)), (0, pages(n_pages=0)), (0, pages(layers=0)), (0, pages(V=P[0] + 64)),
                 (1, None), (1, P[6] + 4), (2, -1), (3, None), (3, params(dtype=9)), (3, params(Hkv=0, Hq=0))):
        a = list(good)
        a[k] = v
        assert lib.cca_pages_copy(*a) == BAD, (k, v)
    assert lib.cca_pages_copy(pages(), P[6], 65536, params(), None) == UNSUP
    assert lib.cca_pages_copy(pages(), P[6], 3, params(d=80), None) == UNSUP
    good = [pages(layers=3, K=P[3], V=P[9]), P[6], P[7], 4, P[8], params(), None]
    for k, v in ((0, None), (0, pages(table=0)), (1, None), (2, None), (2, P[7] + 2), (3, 0), (4, None), (5, params(B=0))):
        a = list(good)
        a[k] = v
        assert lib.cca_pages_compact(*a) == BAD, (k, v)
    assert lib.cca_pages_compact(*good[:3], 257, *good[4:]) == UNSUP


def test_no_pages_has_a_text(lib):
    assert "pages" in api.status_string(api.CCA_ERR_NO_PAGES)


def test_binding_refuses_cpu_tensors(lib):
    x, i = torch.zeros(1, 2, 4, 64), torch.zeros(1, dtype=torch.int32)
    f = torch.ones(32, dtype=torch.float64)
    for call in (lambda: api.cca_rope(x, x, f), lambda: api.cca_rope_append(x, x, x, x, x, i[None], i, f),
                 lambda: api.cca_tree_fwd(x, x, x, i[None], x, x, i[None], i, 4, 8),
                 lambda: api.cca_pool_pages(x, x, x, i[None], x, x, i[None], i, i, 4),
                 lambda: api.cca_pages_reserve(i, i[None], i, i, 4), lambda: api.cca_pages_fork(i, i[None], i, i, i, 4),
                 lambda: api.cca_pages_free(i, i[None], i, i), lambda: api.cca_pages_copy(x, x, i.view(1, 1)),
                 lambda: api.cca_pages_compact(x, x, i[None], i, i[None], i), lambda: api.rope(x, x, f)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("kw", [dict(rot=3), dict(rot=0), dict(rot=64, scaling="other"), dict(rot=64, scaling="linear", factor=0.5),
                                dict(rot=2, scaling="ntk", factor=2.0), dict(rot=64, scaling="bands", factor=2.0, low=4.0, high=1.0)])
def test_frequencies_refuse(kw):
    with pytest.raises(ValueError):
        api.rope_frequencies(device="cpu", **kw)


def test_frequencies_on_the_cpu():
    f, a = api.rope_frequencies(8, 10000.0, device="cpu")
    assert f.tolist() == pytest.approx([1.0, 0.1, 0.01, 0.001], rel=1e-15) and a == 1.0
    # bands, by hand: pair 0 makes 8192 / 2 pi = 1303.8 turns over the original context and stays; the last
    # pair 1.30 turns, weight (1.304 - 1) / 3
    f, _ = api.rope_frequencies(8, 10000.0, "bands", 4.0, device="cpu")
    keep = (0.001 * 8192 / (2 * 3.141592653589793) - 1) / 3
    assert f[0] == 1.0 and f[3].item() == pytest.approx(0.001 * (keep + (1 - keep) / 4), rel=1e-12)


def test_binding_refuses_arguments_before_tensors_are_used(lib):
    from sparse_long_context_cca_gb300 import _binding
    with pytest.raises(TypeError):
        _binding.rope(1)
    for args in ((None,) * 10, (3,) * 10, ("Q",) * 10):
        with pytest.raises(ValueError):
            _binding.rope(*args)
    with pytest.raises(ValueError):
        _binding.bind(api.CcaError, {"cca_rope": 0})
    with pytest.raises(TypeError):
        _binding.bind(api.CcaError)


def test_yarn_without_its_limits_takes_the_usual_ones():
    """Unchanged above 32 turns over the original length, stretched below one; "bands" above 4."""
    import math
    plain, _ = api.rope_frequencies(128, 10000.0, device="cpu")
    turns = plain * (8192 / (2 * math.pi))
    for scaling, high in (("yarn", 32.0), ("bands", 4.0)):
        f, _ = api.rope_frequencies(128, 10000.0, scaling, 8.0, 8192, device="cpu")
        given, _ = api.rope_frequencies(128, 10000.0, scaling, 8.0, 8192, 1.0, high, device="cpu")
        assert torch.equal(f, given)
        assert torch.equal(f[turns > high], plain[turns > high])
        assert torch.allclose(f[turns < 1.0][1:], plain[turns < 1.0][1:] / 8, rtol=1e-14, atol=0)
        between = (turns < high / 1.2) & (turns > 1.2)
        assert (f[between] < plain[between]).all() and (f[between] > plain[between] / 8).all()
    with pytest.raises(ValueError):
        api.rope_frequencies(128, 10000.0, "yarn", 8.0, 8192, 40.0, device="cpu")
