"""Host-only checks of the calls that norm queries and keys and of those over packed sequences: sizes, and every refusal that
needs no GPU (the pointers are never dereferenced), of the C ABI and of the binding."""
import ctypes

import pytest
import torch

from sparse_long_context_cca_gb300 import api
from sparse_long_context_cca_gb300 import build as cbuild

BAD, UNSUP = api.CCA_ERR_INVALID_ARG, api.CCA_ERR_UNSUPPORTED
P = [0x1000000 * (k + 1) for k in range(24)]
I64 = ctypes.c_int64 * 3


@pytest.fixture(scope="module")
def lib():
    cbuild.build()
    return api.load_library()


# ---------------------------------------------------------------- norms with rotation

def norm_params(**kw):
    rope = dict(B=1, N=64, d=64, rot=64, layout=0, dtype=api.CCA_F32, inverse=0, factor=1.0, inv_freq=P[8], positions=0, pos_stride=0, start=0)
    own = dict(eps=1e-6, offset=0.0, weight_dtype=api.CCA_F32)
    for k, v in kw.items():
        (own if k in own else rope)[k] = v
    return ctypes.byref(api.CcaNormParams(api.CcaRopeParams(*rope.values()), *own.values()))


def norm_tensor(x=P[0], y=P[1], dy=P[2], weight=P[3], dweight=P[4], H=2, weight_heads=1, xs=(8192, 4096, 64), ys=None, dys=None):
    return api.CcaNormTensor(x, y, dy, weight, dweight, H, weight_heads, I64(*xs), I64(*(ys or xs)), I64(*(dys or xs)))


PARAMS = [dict(B=0), dict(N=0), dict(rot=63), dict(rot=66), dict(layout=2), dict(dtype=7), dict(inverse=1), dict(factor=float("nan")),
          dict(inv_freq=0), dict(inv_freq=P[8] + 4), dict(positions=P[9] + 2), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
          dict(offset=float("nan")), dict(weight_dtype=5)]
TENSORS = [dict(x=0), dict(y=0), dict(x=P[0] + 8), dict(y=P[1] + 4), dict(xs=(8192, 4096, 63)), dict(H=0), dict(H=2 ** 21), dict(weight=P[3] + 2),
           dict(weight_heads=0), dict(weight_heads=3), dict(ys=(8192, 0, 64)), dict(ys=(8192, 32, 64)), dict(weight=P[1] + 256)]


@pytest.mark.parametrize("kw", PARAMS, ids=str)
def test_norm_parameters(lib, kw):
    t = norm_tensor(dy=0, dweight=0)
    assert lib.cca_norm_rope(ctypes.byref(t), 1, norm_params(**kw), None) == BAD
    t = norm_tensor()
    assert lib.cca_norm_rope_bwd(ctypes.byref(t), 1, norm_params(**kw), P[10], 1 << 24, None) == BAD
    assert lib.cca_norm_rope_bwd_workspace_size(ctypes.byref(t), 1, norm_params(**kw)) == 0


@pytest.mark.parametrize("kw", TENSORS, ids=str)
def test_norm_tensors(lib, kw):
    t = norm_tensor(**{"dy": 0, "dweight": 0, **kw})
    assert lib.cca_norm_rope(ctypes.byref(t), 1, norm_params(), None) == BAD
    t = norm_tensor(**kw)
    assert lib.cca_norm_rope_bwd(ctypes.byref(t), 1, norm_params(), P[10], 1 << 24, None) == BAD


@pytest.mark.parametrize("kw", [dict(dy=0), dict(dy=P[2] + 8), dict(y=P[0]), dict(y=P[2]), dict(dweight=P[3]), dict(dweight=P[1]), dict(dweight=P[0]),
                                dict(weight=0), dict(dys=(8192, 4096, 2))], ids=str)
def test_norm_gradients(lib, kw):
    t = norm_tensor(**kw)
    assert lib.cca_norm_rope_bwd(ctypes.byref(t), 1, norm_params(), P[10], 1 << 24, None) == BAD


def test_norm_pairs_and_sizes(lib):
    t = norm_tensor(dy=0, dweight=0)
    for n in (0, 3):
        assert lib.cca_norm_rope(ctypes.byref(t), n, norm_params(), None) == BAD
    assert lib.cca_norm_rope(None, 1, norm_params(), None) == BAD
    assert lib.cca_norm_rope(ctypes.byref(t), 1, None, None) == BAD
    two = (api.CcaNormTensor * 2)(t, norm_tensor(x=P[5], dy=0, dweight=0))                       # one result for both
    assert lib.cca_norm_rope(two, 2, norm_params(), None) == BAD
    two = (api.CcaNormTensor * 2)(t, norm_tensor(x=P[1], y=P[5], dy=0, dweight=0))               # reads the first's result
    assert lib.cca_norm_rope(two, 2, norm_params(), None) == BAD
    two = (api.CcaNormTensor * 2)(norm_tensor(), norm_tensor(x=P[5], y=P[6], dy=P[7], weight=P[9]))   # one dweight for both
    assert lib.cca_norm_rope_bwd(two, 2, norm_params(), P[10], 1 << 24, None) == BAD
    assert lib.cca_norm_rope(ctypes.byref(t), 1, norm_params(d=96, rot=64), None) == UNSUP


def test_norm_append(lib):
    q, k = norm_tensor(dy=0, dweight=0), norm_tensor(x=P[5], y=0, dy=0, dweight=0)
    v = api.CcaRopeTensor(P[6], 0, 2, I64(8192, 4096, 64), I64(0, 0, 0))
    pages = api.CcaPages(P[11], P[12], P[13], 8, 16, 8, 1)

    def call(q=q, k=k, v=v, lens=P[14], status=0, **kw):
        r = [ctypes.byref(x) if x is not None else None for x in (q, k, v)]
        return lib.cca_norm_rope_append(*r, ctypes.byref(pages), lens, None, None, status or None, norm_params(**{"N": 16, **kw}), None)
    assert call(k=None) == call(v=None) == call(lens=0) == call(lens=P[14] + 2) == BAD
    assert call(positions=P[9]) == call(start=3) == call(inverse=1) == call(eps=-1.0) == call(status=P[15] + 1) == BAD
    assert call(q=norm_tensor(y=P[11], dy=0, dweight=0)) == BAD            # queries over the pages
    assert call(k=norm_tensor(x=P[5], y=0, dy=0, dweight=0, weight=P[11] + 64)) == BAD     # weights in the pages
    assert call(k=norm_tensor(x=P[5], y=0, dy=0, dweight=0, weight_heads=3)) == BAD


# ---------------------------------------------------------------- packed sequences

def plan(lib, **kw):
    a = dict(plan=P[0], plan_bytes=None, S=3, T=64, g=4, w=16, window_mode=0)
    a.update(kw)
    if a["plan_bytes"] is None:
        a["plan_bytes"] = max(lib.cca_pack_size(a["S"], a["T"], a["g"]), 1)
    return ctypes.byref(api.CcaPacked(*a.values()))


def params(**kw):
    a = dict(B=1, Hq=4, Hkv=2, N=1, d=128, g=1, w=1, dtype=api.CCA_BF16, scale=0.0, dev_status=0, window_mode=0, pool_mode=0)
    a.update(kw)
    return ctypes.byref(api.CcaParams(*a.values()))


def rows(k, H=4, head=128, row=None):
    return api.CcaPackedRows(k, head, H * 128 if row is None else row)


def calls(lib, pk, prm, only=("pool", "attn", "bwd"), **kw):
    """The packed calls with their tensors by name; {call: status}.  Each has to be refused: a call that is not would run."""
    a = dict(Q=rows(P[1]), K=rows(P[2], 2), V=rows(P[3], 2), Kc=P[4], Vc=P[5], O=rows(P[6]), LSE=P[7], dO=rows(P[8]), dQ=rows(P[9]), dK=rows(P[10], 2),
             dV=rows(P[11], 2), ws=P[12], ws_bytes=1 << 23)
    a.update(kw)
    r = {k: ctypes.byref(v) if isinstance(v, api.CcaPackedRows) else v for k, v in a.items()}
    each = {"pool": lambda: lib.cca_pool_packed(r["Q"], r["K"], r["V"], r["Kc"], r["Vc"], pk, prm, None),
            "attn": lambda: lib.cca_attn_packed(r["Q"], r["K"], r["V"], r["Kc"], r["Vc"], r["O"], r["LSE"], pk, prm, None),
            "bwd": lambda: lib.cca_packed_bwd(r["Q"], r["K"], r["V"], r["Kc"], r["Vc"], r["O"], r["LSE"], r["dO"], r["dQ"], r["dK"], r["dV"],
                                              pk, prm, r["ws"], r["ws_bytes"], None)}
    return {k: each[k]() for k in only}


PLANS = [dict(plan=0), dict(plan=P[0] + 8), dict(plan_bytes=16), dict(S=0), dict(S=65536), dict(T=0), dict(g=0), dict(w=0), dict(window_mode=2)]


@pytest.mark.parametrize("kw", PLANS, ids=str)
def test_plans(lib, kw):
    assert lib.cca_pack(P[1], plan(lib, **kw), None, None) == BAD
    assert set(calls(lib, plan(lib, **kw), params()).values()) == {BAD}
    t, h = (api.CcaPackedRows * 1)(rows(P[6])), (ctypes.c_int32 * 1)(4)
    assert lib.cca_packed_clear(t, h, 1, plan(lib, **kw), params(), None) == BAD


def test_pack_arguments(lib):
    assert lib.cca_pack(None, plan(lib), None, None) == BAD
    assert lib.cca_pack(P[1] + 2, plan(lib), None, None) == BAD
    assert lib.cca_pack(P[1], None, None, None) == BAD
    assert lib.cca_pack(P[1], plan(lib), P[2] + 1, None) == BAD
    assert lib.cca_pack(P[0] + 64, plan(lib), None, None) == BAD       # lengths inside the plan
    assert lib.cca_pack(P[1], plan(lib), P[0] + 64, None) == BAD       # the status inside the plan


@pytest.mark.parametrize("kw,want", [(dict(Hq=0), BAD), (dict(Hkv=0), BAD), (dict(Hq=3), BAD), (dict(Hq=131072), BAD), (dict(dtype=9), BAD),
                                     (dict(scale=float("nan")), BAD), (dict(scale=float("inf")), BAD), (dict(dev_status=P[13] + 1), BAD),
                                     (dict(pool_mode=4), BAD), (dict(pool_mode=-1), BAD), (dict(pool_mode=2), UNSUP), (dict(d=96), UNSUP)], ids=str)
def test_parameters(lib, kw, want):
    assert set(calls(lib, plan(lib), params(**kw)).values()) == {want}
    assert lib.cca_packed_bwd_workspace_size(plan(lib), params(**kw)) == 0


@pytest.mark.parametrize("name", ["Q", "K", "V"])
def test_inputs(lib, name):
    H = 4 if name == "Q" else 2
    k = {"Q": 1, "K": 2, "V": 3}[name]
    for bad in (rows(0, H), rows(P[k] + 8, H), rows(P[k], H, row=H * 128 + 4), rows(P[k], H, head=0), rows(P[k], H, head=64), rows(P[k], H, row=0),
                rows(P[k], H, row=-512), rows(P[k], H, head=-128), rows(P[k], H, row=1 << 40), rows(P[k], H, row=1 << 62), None):
        assert set(calls(lib, plan(lib), params(), **{name: bad}).values()) == {BAD}, name


def test_outputs(lib):
    def status(call, **kw):
        return calls(lib, plan(lib), params(), (call,), **kw)[call]
    for kw in (dict(Kc=0), dict(Vc=0), dict(Kc=P[4] + 8), dict(Kc=P[5]), dict(Kc=P[1]), dict(Vc=P[3] + 128), dict(Kc=P[0])):
        assert status("pool", **kw) == BAD, kw
    for kw in (dict(O=None), dict(O=rows(P[6] + 8)), dict(O=rows(P[6], row=256)), dict(O=rows(P[1])), dict(O=rows(P[1], row=4 * 128)), dict(O=rows(P[0])),
               dict(LSE=0), dict(LSE=P[7] + 2), dict(LSE=P[6]), dict(LSE=P[2]), dict(Kc=0), dict(O=rows(P[4]))):
        assert status("attn", **kw) == BAD, kw
    for kw in (dict(dQ=None), dict(dK=rows(P[9], 2)), dict(dV=rows(P[3], 2)), dict(dQ=rows(P[8])), dict(dK=rows(P[6], 2)), dict(dQ=rows(P[7])),
               dict(dK=rows(P[10], 2, row=128)), dict(ws=0), dict(ws=P[12] + 8), dict(dO=rows(P[8], head=0)), dict(LSE=0), dict(Vc=0)):
        assert status("bwd", **kw) == BAD, kw


def test_clear_arguments(lib):
    def call(n=1, heads=(4,), x=P[6], pk=None, prm=None, second=None):
        t = (api.CcaPackedRows * 5)(rows(x), *([second] if second else []))
        return lib.cca_packed_clear(t, (ctypes.c_int32 * 5)(*heads), n, pk or plan(lib), prm or params(), None)
    assert call(n=0) == call(n=5) == call(heads=(0,)) == call(heads=(70000,)) == call(x=P[6] + 8) == call(x=P[0]) == BAD
    assert call(n=2, heads=(4, 4), second=rows(P[6])) == BAD                  # the same tensor twice
    assert call(prm=params(dtype=5)) == BAD and call(prm=params(d=32)) == UNSUP
    assert lib.cca_packed_clear(None, None, 1, plan(lib), params(), None) == BAD


def test_sizes(lib):
    for S, T, g in ((0, 8, 1), (65536, 8, 1), (1, 0, 1), (1, 8, 0)):
        assert lib.cca_pack_size(S, T, g) == 0 and lib.cca_pack_positions_offset(S, T, g) == 0
    for S, T, g in ((1, 1, 1), (7, 1000, 16), (65535, 5, 3), (12, 147000, 16)):
        size, at = lib.cca_pack_size(S, T, g), lib.cca_pack_positions_offset(S, T, g)
        lists = 16 * sum(T // k + S for k in (256, 128)) + 16 * (T // g // 128 + S)
        assert at >= 64 + lists and at % 16 == 0 and size >= at + 4 * T + 4 * (T // g) and size % 16 == 0
    assert lib.cca_pack_size(65535, 2 ** 31 - 1, 1) > 2 ** 33     # 64 bits throughout


def test_binding_refuses_cpu_tensors(lib):
    x, cu, f = torch.zeros(2, 8, 64), torch.tensor([0, 8], dtype=torch.int32), torch.ones(32, dtype=torch.float64)
    p = api.Packed(torch.zeros(lib.cca_pack_size(1, 8, 4), dtype=torch.uint8), None, 1, 8, 4, 4, 0)
    i = torch.zeros(1, dtype=torch.int32)
    y = x[None]
    for call in (lambda: api.cca_pack(cu, 8), lambda: api.cca_pool_packed(x, x, x, p), lambda: api.cca_attn_packed(x, x, x, None, None, p),
                 lambda: api.cca_packed_bwd(x, x, x, None, None, x, x[..., 0], x, p), lambda: api.cca_packed_clear(p, x),
                 lambda: api.cca_norm_rope(y, y, inv_freq=f), lambda: api.norm_rope(y, y, inv_freq=f),
                 lambda: api.cca_norm_rope_append(y, y, y, y, y, i[None], i), lambda: api.cca_attention_packed(x, x, x, p)):
        with pytest.raises(ValueError):
            call()


def test_a_packed_batch_knows_whether_cores_are_seen():
    for tokens, g, w, want in ((64, 4, 16, True), (64, 4, 64, False), (64, 65, 16, False), (64, 4, 63, True)):
        assert api.Packed(None, None, 1, tokens, g, w, 0).cores is want
