"""Attention of drafted trees over paged caches against a 64-bit row-by-row definition."""
import numpy as np
import pytest
import torch

from paged_ref import close, paged, t64, tree
from sparse_long_context_cca_gb300 import api

pytestmark = pytest.mark.gpu

NAN = float("nan")


def make(B, T, Hq, Hkv, d, lens, g, w, rows, crows, dtype, mode=0, seed=0, trees=True, cols=None):
    """Everything cca_tree_fwd takes.  Only the rows it may read hold numbers; the rest is NaN."""
    rng = np.random.default_rng(seed)
    gen = torch.Generator().manual_seed(seed)
    scale = 1.0 if dtype == torch.float32 else d ** -0.25
    draw = lambda *s: torch.randn(s, generator=gen) * scale  # noqa: E731
    first, raws, cores = [], [], []
    for n in lens:
        lo = max(0, n - w + 1)
        first.append(lo // g * g if mode else lo)
        raws.append((draw(Hkv, n + T - first[-1], d), draw(Hkv, n + T - first[-1], d)))
        top = max(0, n + T - w) // g
        k = draw(Hkv, top, d)
        k[:, ::7] *= 4.0
        cores.append((k, draw(Hkv, top, d)))
    cols = cols or -(-(max(lens) + T) // rows) + 1
    Kp, Vp, table = paged(raws, first, lens, Hkv, d, rows, cols, dtype, seed)
    Kc, Vc, ctable = paged(cores, [0] * B, lens, Hkv, d, crows, max(lens) // g // crows + 2, dtype, seed + 1)
    parents = None
    if trees:
        parents = torch.tensor([[int(rng.integers(max(-1, t - 4), t)) for t in range(T)] for _ in range(B)], dtype=torch.int32)
    Q = draw(B, Hq, T, d).to(dtype)
    return dict(Q=Q, Kp=Kp, Vp=Vp, table=table, Kcp=Kc, Vcp=Vc, core_table=ctable,
                lens=torch.tensor(lens, dtype=torch.int32), parents=parents)


def call(x, g, w, **kw):
    y = {k: v.cuda() if v is not None else None for k, v in x.items()}
    return api.cca_tree_fwd(y["Q"], y["Kp"], y["Vp"], y["table"], y["Kcp"], y["Vcp"], y["core_table"], y["lens"], g, w,
                            parents=y["parents"], **kw)


def check(x, g, w, rows, crows, mode=0, what="", **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    O, LSE = call(x, g, w, window_mode=mode, dev_status=status, **kw)
    torch.cuda.synchronize()
    assert status.item() == 0, what
    ref = tree(x["Q"], x["Kp"], x["Vp"], x["table"], x["Kcp"], x["Vcp"], x["core_table"], x["lens"], x["parents"], g, w, rows,
               crows, mode, kw.get("scale"))
    close(O, ref[0], ref[2], what + " O")
    close(LSE, ref[1], ref[3], what + " LSE")
    return O, LSE


CASES = [  # B, T, Hq, Hkv, d, lens, g, w, rows, crows, mode
    (1, 1, 1, 1, 128, [0], 16, 32, 16, 16, 0),                    # nothing committed
    (1, 1, 4, 4, 128, [500], 16, 64, 64, 64, 0),                  # one token, rows of one warp
    (2, 1, 8, 1, 64, [77, 300], 4, 20, 16, 5, 0),
    (3, 7, 4, 2, 128, [1, 63, 700], 8, 100, 24, 7, 0),            # 14 rows; pages that end inside a tile
    (2, 5, 6, 2, 64, [64, 129], 3, 5, 7, 3, 0),                   # as many nodes as the window is wide; odd pages
    (2, 9, 6, 2, 128, [200, 1000], 16, 128, 64, 64, 1),           # 27 rows, window from the group boundary
    (1, 33, 3, 1, 128, [900], 8, 64, 32, 16, 0),                  # 99 rows: two row tiles
    (2, 64, 8, 2, 128, [130, 2100], 16, 256, 64, 64, 0),          # 256 rows: four row tiles
    (1, 256, 1, 1, 64, [1000], 4, 256, 128, 40, 1),               # the largest tree
    (1, 3, 2, 1, 128, [40], 1, 10, 16, 16, 0),                    # every token its own core
    (1, 2, 2, 2, 64, [50], 64, 60, 1, 1, 0),                      # pages of one row; no core yet
    (5, 4, 4, 2, 128, [0, 3, 31, 32, 33], 16, 16, 16, 16, 1),
    (3, 12, 4, 2, 128, [5000, 20, 2600], 16, 300, 64, 64, 0),     # tensor cores: lists of many tiles, several per CTA
    (40, 10, 8, 4, 128, [17 * i + 3 for i in range(40)], 8, 33, 16, 10, 1),   # more lists than CTAs
    (2, 64, 4, 1, 128, [9000, 4100], 2, 128, 64, 64, 0),          # two halves over runs of many tiles
    (2, 24, 4, 2, 64, [2600, 700], 8, 100, 48, 24, 0),            # d = 64: 48 rows, several lists per CTA
    (2, 96, 4, 1, 128, [333, 4100], 8, 128, 48, 16, 0),           # 384 rows: two row tiles of two halves, the last half empty
]


@pytest.mark.parametrize("trees", [True, False], ids=["tree", "chain"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_matches_definition(case, dtype, trees):
    B, T, Hq, Hkv, d, lens, g, w, rows, crows, mode = CASES[case]
    x = make(B, T, Hq, Hkv, d, lens, g, w, rows, crows, dtype, mode, seed=case, trees=trees)
    check(x, g, w, rows, crows, mode, f"case {case}")


def test_scale():
    x = make(1, 3, 2, 1, 64, [90], 8, 32, 16, 16, torch.float32)
    check(x, 8, 32, 16, 16, what="scale", scale=0.31)


def test_padding_and_broken_chains():
    x = make(2, 6, 4, 2, 128, [100, 300], 8, 64, 16, 16, torch.bfloat16)
    # node 2's chain is broken, node 4 hangs below it; the second tree is padding alone
    x["parents"] = torch.tensor([[-1, 0, 2, 1, 2, 3], [-2] * 6], dtype=torch.int32)
    # what padding nodes' rows hold never matters
    O, LSE = check(x, 8, 64, 16, 16, what="padding")
    assert not O[1].any() and torch.isinf(LSE[1]).all() and not O[0, :, [2, 4]].any()
    x["parents"] = torch.tensor([[-1, 0, 7, -5, 2 ** 31 - 1, -2 ** 31], [-2] * 6], dtype=torch.int32)
    check(x, 8, 64, 16, 16, what="wild parents")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("bad", [NAN, float("inf"), -float("inf")])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads", [2, 4, 24, 40])    # rows for each of the kernels
def test_masked_rows_may_hold_anything(bad, dtype, heads, d):
    """Infinities and NaN in keys and values that a node does not see leave it as it is, and reach the
    nodes that do see them."""
    T = 6
    B, Hq, Hkv, g, w, rows = 1, heads, 1, 8, 40, 16
    x = make(B, T, Hq, Hkv, d, [200], g, w, rows, rows, dtype, seed=3)
    x["parents"] = torch.tensor([[-1, 0, 0, 1, 2, 2]], dtype=torch.int32)
    clean = call(x, g, w)
    page, row = int(x["table"][0, (200 + 2) // rows]), (200 + 2) % rows       # node 2
    x["Vp"][page, 0, row, 5] = bad
    O, LSE = call(x, g, w)
    sees = [2, 4, 5]
    others = [0, 1, 3]
    assert torch.equal(O[:, :, others], clean[0][:, :, others]) and torch.equal(LSE, clean[1])
    want = clean[0].clone().float()
    want[:, :, sees, 5] = bad
    torch.testing.assert_close(O.float(), want, rtol=0, atol=0, equal_nan=True)
    x["Kp"][page, 0, row, 9] = bad
    O, LSE = call(x, g, w)
    assert torch.equal(O[:, :, others], clean[0][:, :, others]) and torch.equal(LSE[:, :, others], clean[1][:, :, others])
    if bad != bad:
        assert torch.isnan(LSE[:, :, sees]).all() and torch.isnan(O[:, :, sees]).all()
    # the first raw row of the shallowest node's window: out of reach of the deeper ones
    x = make(B, T, Hq, Hkv, d, [200], g, w, rows, rows, dtype, seed=3)
    x["parents"] = torch.tensor([[-1, 0, 0, 1, 2, 2]], dtype=torch.int32)
    first = 200 - w + 1
    page, row = int(x["table"][0, first // rows]), first % rows
    x["Vp"][page, 0, row] = bad
    O, _ = call(x, g, w)
    assert torch.equal(O[:, :, 1:], clean[0][:, :, 1:])
    assert (O[:, :, 0].float() == bad).all() if bad == bad else torch.isnan(O[:, :, 0]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_bad_tables_and_lengths_are_reported(dtype):
    g, w, rows = 8, 64, 16
    x = make(3, 4, 2, 1, 64, [150, 200, 170], g, w, rows, rows, dtype)
    clean = call(x, g, w)
    y = dict(x)
    y["lens"] = torch.tensor([150, -1, 10 ** 9], dtype=torch.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    O, LSE = call(y, g, w, dev_status=status)
    assert status.item() == api.CCA_ERR_INVALID_ARG
    assert torch.equal(O[0], clean[0][0]) and not O[1:].any() and torch.isinf(LSE[1:]).all()
    # a page that is not there: its keys are left out, as if masked
    y = dict(x, table=x["table"].clone())
    c = 140 // rows
    y["table"][0, c] = y["Kp"].shape[0]
    y["core_table"] = x["core_table"].clone()
    y["core_table"][0, 0] = -7
    status.zero_()
    O, LSE = call(y, g, w, dev_status=status)
    assert status.item() == api.CCA_ERR_INVALID_ARG and torch.equal(O[1:], clean[0][1:])
    gone = dict(x, Kp=x["Kp"].clone(), Vp=x["Vp"].clone(), Kcp=x["Kcp"].clone(), Vcp=x["Vcp"].clone())
    tau = 64 ** -0.5
    k, v, kc, vc = (t64(gone[n]) for n in ("Kp", "Vp", "Kcp", "Vcp"))
    from paged_ref import chain, row_at, softmax_row, window
    for t in range(4):
        ch = chain(x["parents"][0].tolist(), t)
        cores, start = window(150 + len(ch) - 1, w, g, 0)
        raw = [i for i in range(start, 150) if i // rows != c] + [150 + a for a in ch if (150 + a) // rows != c]
        K = np.stack([row_at(kc, x["core_table"], rows, 0, j) for j in range(rows, cores)] + [row_at(k, x["table"], rows, 0, i) for i in raw], 1)
        V = np.stack([row_at(vc, x["core_table"], rows, 0, j) for j in range(rows, cores)] + [row_at(v, x["table"], rows, 0, i) for i in raw], 1)
        for h in range(2):
            o, lse, do, dl = softmax_row(t64(x["Q"])[0, h, t], K[0], V[0], tau, dtype)
            close(O[0, h, t], o, do, "missing page")
            close(LSE[0, h, t], np.asarray(lse), np.asarray(dl), "missing page LSE")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_contiguous_cache_is_a_pool(dtype):
    """[B, Hkv, Ncap, d] caches with the table 0 .. B - 1: one token equals cca_decode_fwd."""
    B, Hq, Hkv, N, d, g, w, pos = 3, 8, 2, 1024, 128, 16, 200, 777
    gen = torch.Generator().manual_seed(5)
    mk = lambda *s: (torch.randn(s, generator=gen) * 0.3).to(dtype).cuda()  # noqa: E731
    K, V, Kc, Vc, q = mk(B, Hkv, N, d), mk(B, Hkv, N, d), mk(B, Hkv, N // g, d), mk(B, Hkv, N // g, d), mk(B, Hq, d)
    table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous()
    lens = torch.full((B,), pos, dtype=torch.int32, device="cuda")
    O, LSE = api.cca_tree_fwd(q[:, :, None].contiguous(), K, V, table, Kc, Vc, table, lens, g, w)
    Od, Ld = api.cca_decode_fwd(q, K, V, Kc, Vc, pos, g, w)
    # both round once from fp32 sums; in bf16 the tree also rounds its weights
    tol = 2.0 ** -6 if dtype == torch.bfloat16 else 1e-5
    assert (O[:, :, 0].float() - Od.float()).abs().max() <= tol * V.float().abs().max()
    assert (LSE[:, :, 0] - Ld).abs().max() <= 1e-4


def test_long_cache_offsets_pass_32_bits():
    """A pool of more than 2^31 elements: pages at its far end are read where they are."""
    rows, H, d, g, w = 4096, 8, 128, 16, 64
    n = 2 ** 31 // (rows * H * d) + 3
    Kp = torch.zeros(n, H, rows, d, dtype=torch.bfloat16, device="cuda")
    Vp = torch.zeros(n, H, rows, d, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    last = n - 1
    Kp[last] = torch.randn(H, rows, d, generator=gen, device="cuda").to(torch.bfloat16)
    Vp[last] = torch.randn(H, rows, d, generator=gen, device="cuda").to(torch.bfloat16)
    Kc, Vc = Kp[last:, :, :16].contiguous(), Vp[last:, :, :16].contiguous()
    q = torch.randn(1, H, 2, d, generator=gen, device="cuda").to(torch.bfloat16)
    lens = torch.tensor([50], dtype=torch.int32, device="cuda")
    far = torch.tensor([[last]], dtype=torch.int32, device="cuda")
    near = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    got = api.cca_tree_fwd(q, Kp, Vp, far, Kc, Vc, near, lens, g, w)
    want = api.cca_tree_fwd(q, Kp[last:].clone(), Vp[last:].clone(), near, Kc, Vc, near, lens, g, w)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and got[0].any()


def test_repeatable_and_independent_of_the_batch():
    """The same call twice is the same to the bit."""
    x = make(4, 16, 8, 2, 128, [900, 10, 2500, 1300], 16, 256, 64, 64, torch.bfloat16)
    a, b = call(x, 16, 256), call(x, 16, 256)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_graph_serves_later_lengths_and_trees():
    g, w, rows = 16, 128, 32
    x = make(2, 5, 4, 2, 128, [400, 900], g, w, rows, rows, torch.bfloat16, cols=40)
    z = make(2, 5, 4, 2, 128, [1000, 33], g, w, rows, rows, torch.bfloat16, seed=9, cols=40)
    names = ["Q", "Kp", "Vp", "table", "Kcp", "Vcp", "core_table", "lens", "parents"]
    size = {n: [max(p, q) for p, q in zip(x[n].shape, z[n].shape)] for n in names}
    buf = {n: torch.zeros(size[n], dtype=x[n].dtype, device="cuda") for n in names}

    def fill(v):
        for n in names:
            buf[n].fill_(-1 if "table" in n else 0)
            buf[n][tuple(slice(0, s) for s in v[n].shape)] = v[n].cuda()

    fill(x)
    ws = torch.empty(api.tree_workspace_size(2, 4, 2, 5, 128, g, w, torch.bfloat16), dtype=torch.uint8, device="cuda")
    O, LSE = torch.empty_like(buf["Q"]), torch.empty(2, 4, 5, device="cuda")
    args = [buf[n] for n in names[:8]]
    api.cca_tree_fwd(*args, g, w, parents=buf["parents"], O=O, LSE=LSE, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.cca_tree_fwd(*args, g, w, parents=buf["parents"], O=O, LSE=LSE, workspace=ws)
    for v in (z, x):
        fill(v)
        ws.fill_(0xff)
        graph.replay()
        want = call(v, g, w)
        torch.cuda.synchronize()
        assert torch.equal(O, want[0]) and torch.equal(LSE, want[1])


def test_two_streams_with_their_own_workspaces():
    x = make(2, 8, 4, 2, 128, [700, 1500], 16, 128, 64, 64, torch.bfloat16)
    want = call(x, 16, 128)
    y = {k: v.cuda() for k, v in x.items()}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(8):
        got.append(api.cca_tree_fwd(y["Q"], y["Kp"], y["Vp"], y["table"], y["Kcp"], y["Vcp"], y["core_table"], y["lens"], 16,
                                    128, parents=y["parents"], stream=streams[i % 2]))
    torch.cuda.synchronize()
    for O, LSE in got:
        assert torch.equal(O, want[0]) and torch.equal(LSE, want[1])


def test_refusals():
    x = {k: v.cuda() for k, v in make(1, 4, 4, 2, 64, [50], 8, 16, 16, 16, torch.float32).items()}
    args = [x[n] for n in ("Q", "Kp", "Vp", "table", "Kcp", "Vcp", "core_table", "lens")]
    run = lambda a=args, g=8, w=16, **kw: api.cca_tree_fwd(*a, g, w, **kw)  # noqa: E731
    run()
    for bad in (dict(w=3), dict(w=0), dict(g=0), dict(scale=NAN), dict(window_mode=2)):
        with pytest.raises(api.CcaError):
            run(**bad)
    for i, t in ((0, args[0].half()), (0, args[0].transpose(1, 2)), (1, args[1].bfloat16()), (3, args[3].long()), (7, args[7][:0]),
                 (5, args[5][:, :1]), (2, args[2].cpu()), (6, args[6][0])):
        a = list(args)
        a[i] = t
        with pytest.raises(ValueError):
            run(a)
    with pytest.raises(ValueError):
        run(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        run(parents=torch.zeros(1, 3, dtype=torch.int32, device="cuda"))
    with pytest.raises(api.CcaError):
        run(O=args[0])


@pytest.mark.parametrize("T", [8, 40], ids=["one half", "two halves"])
def test_wait_time_out_is_reported(T):
    """Tensor-core kernel with no copies at all: its waits run out, it reports and returns, and the
    next call is as before."""
    x = make(2, T, 8, 2, 128, [300, 900], 16, 64, 32, 32, torch.bfloat16)
    want = call(x, 16, 64)
    torch.cuda.synchronize()
    lib = api.load_library()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.cca_test_set_wait_limit_ns(2_000_000)
    lib.cca_test_skip_q_load(1)
    try:
        call(x, 16, 64, dev_status=status)
        torch.cuda.synchronize()
    finally:
        lib.cca_test_skip_q_load(0)
        lib.cca_test_set_wait_limit_ns(1_000_000_000)
    assert status.item() == api.CCA_ERR_TIMEOUT
    got = call(x, 16, 64)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("d,heads,T", [(128, 1, 3), (128, 4, 40), (64, 2, 5), (64, 1, 20), (64, 4, 40)])
@pytest.mark.parametrize("seed", range(3))
def test_runs_that_begin_and_end_anywhere(d, heads, T, seed):
    """Lists of one tile to many, more of them than groups or fewer: a run may begin inside a list, at its
    end, or hold several; with d = 64 on both kernels."""
    rng = np.random.default_rng([seed, d, T])
    B, Hkv = [(3, 8), (37, 3), (7, 2)][seed]
    lens = [int(rng.choice([0, 5, 100, 900, 2500, 6000])) + int(rng.integers(0, 90)) for _ in range(B)]
    if B > 30:
        lens = [n % 1500 for n in lens]
    g, w, rows, crows = 2, 64, [16, 64, 48][seed], [64, 8, 40][seed]
    x = make(B, T, heads * Hkv, Hkv, d, lens, g, w, rows, crows, torch.bfloat16, seed=seed)
    O, LSE = check(x, g, w, rows, crows, what=f"lens {lens}")
    again = call(x, g, w)
    assert torch.equal(O, again[0]) and torch.equal(LSE, again[1])


WEIGHTS = [  # B, T, Hq, Hkv, d, lens, g, w, mode: up to 16 rows per KV head, few keys or a few that carry the weight
    (1, 1, 1, 1, 128, [9], 4, 16, 0),
    (2, 1, 32, 32, 128, [12, 2600], 16, 24, 0),
    (2, 1, 16, 1, 128, [7, 250], 16, 24, 0),
    (3, 4, 8, 2, 128, [6, 30, 700], 8, 20, 1),
    (2, 5, 6, 2, 128, [1, 5000], 4, 40, 0),
    (2, 1, 4, 1, 64, [10, 900], 8, 12, 0),
    (2, 4, 8, 2, 64, [5, 400], 16, 16, 1),
]


@pytest.mark.parametrize("case", range(len(WEIGHTS)))
def test_few_rows_keep_their_weights(case):
    """Up to 16 rows per KV head the softmax weights meet V as two bf16 parts, so that the output's own
    rounding is nearly all of its error.

    Bound: that of the fp32 call on the same values, the weights' two parts (the first cut off, which
    leaves less than 2^-7 of the weight; the second, cut off as well, leaves 2^-7 of that: 2^-14 of
    sum p |v| / sum p, which max |v| bounds) and the output's rounding.  One part, rounded, is off by up to
    2^-8 of each weight: with ten keys that is some 2^-9 / sqrt(10) of |v|, ten times the bound of an
    output near 0."""
    B, T, Hq, Hkv, d, lens, g, w, mode = WEIGHTS[case]
    x = make(B, T, Hq, Hkv, d, lens, g, w, 16, 16, torch.bfloat16, mode, seed=50 + case)
    O, LSE = call(x, g, w, window_mode=mode)
    wide = {k: v.float() if v is not None and v.is_floating_point() else v for k, v in x.items()}
    ref, lse, dO, dL = tree(wide["Q"], wide["Kp"], wide["Vp"], x["table"], wide["Kcp"], wide["Vcp"], x["core_table"], x["lens"],
                            x["parents"], g, w, 16, 16, mode)
    big = max(float(v[~v.isnan()].abs().max()) for v in (wide["Vp"], wide["Vcp"]) if bool((~v.isnan()).any()))
    near = dO + 2.0 ** -14 * big
    close(O, ref, near + 2.0 ** -8 * (np.abs(ref) + near), f"case {case} O")
    close(LSE, lse, dL, f"case {case} LSE")


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), NAN])
@pytest.mark.parametrize("d,heads", [(128, 1), (128, 40), (64, 1), (64, 16), (64, 40)])
def test_infinities_that_every_row_sees(d, heads, bad):
    """An infinity in the V of a key that every node sees is what each of them puts out, a NaN likewise;
    among runs of whole pages and among the keys around them."""
    g, w, rows = 8, 200, 16
    for at in (150, 299):                  # inside whole pages; next to the nodes
        x = make(1, 3, heads, 1, d, [300], g, w, rows, rows, torch.bfloat16, seed=4)
        clean = call(x, g, w)
        x["Vp"][int(x["table"][0, at // rows]), 0, at % rows, 5] = bad
        O, LSE = call(x, g, w)
        want = clean[0].float()
        want[..., 5] = bad
        torch.testing.assert_close(O.float(), want, rtol=0, atol=0, equal_nan=True)
        assert torch.equal(LSE, clean[1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("heads,d", [(1, 128), (24, 128), (40, 128), (1, 64), (8, 64)])     # rows for each of the kernels
def test_padding_nodes_need_no_page(heads, d, dtype):
    """Trees of different sizes, padded to one T: pages for the real nodes alone, up to the table's last
    row.  Nothing is reported, and the real nodes are as they are with pages for all."""
    T, g, w, rows = 6, 8, 40, 16
    lens = [13, 60, 94, 96, 95]                      # real nodes: 3, 4, 2, none, 1; the table has 96 rows
    real = [3, 4, 2, 0, 1]
    x = make(5, T, heads, 1, d, lens, g, w, rows, rows, dtype, seed=6, cols=7)
    x["parents"] = torch.tensor([[-1, 0, 0, -2, -2, 3], [-1, 0, 1, 2, -2, -2], [-1, 0, -2, -2, -2, -2], [-2] * 6,
                                 [-1, -2, -2, -2, -2, -2]], dtype=torch.int32)
    want = check(x, g, w, rows, rows, what="pages for all")
    y = dict(x, table=x["table"][:, :6].clone())
    for b in range(5):
        y["table"][b, -(-(lens[b] + real[b]) // rows):] = -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    O, LSE = call(y, g, w, dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    # lists may be cut at other keys, so the last bits may differ
    ref = tree(x["Q"], x["Kp"], x["Vp"], x["table"], x["Kcp"], x["Vcp"], x["core_table"], x["lens"], x["parents"], g, w, rows, rows)
    close(O, ref[0], ref[2], "O")
    close(LSE, ref[1], ref[3], "LSE")
    assert torch.isinf(LSE).any() and torch.equal(torch.isinf(LSE), torch.isinf(want[1]))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("chain", [True, False])
def test_real_nodes_past_the_pages_are_reported(dtype, chain):
    """A real node without a page, or past the table's end, is reported and counts as not there for the
    nodes below it; the others are as they were."""
    T, g, w, rows = 5, 8, 32, 16
    x = make(2, T, 4, 2, 64, [60, 30], g, w, rows, rows, dtype, seed=7, cols=5)
    x["parents"] = None if chain else torch.tensor([[-1, 0, 1, 2, 3], [-1, -1, -1, -1, -2]], dtype=torch.int32)
    clean = call(x, g, w)
    for cols in (5, 4):                              # no page for rows 64 .., or no such rows in the table
        y = dict(x, table=x["table"][:, :cols].contiguous())
        if cols == 5:
            y["table"][0, 4] = -1
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        O, LSE = call(y, g, w, dev_status=status)
        assert status.item() == api.CCA_ERR_INVALID_ARG
        assert torch.equal(O[1], clean[0][1]) and torch.equal(LSE[1], clean[1][1])
        assert torch.equal(O[0, :, :4], clean[0][0, :, :4]) and torch.equal(LSE[0, :, :4], clean[1][0, :, :4])
        assert not torch.equal(LSE[0, :, 4], clean[1][0, :, 4]) and torch.isfinite(LSE).equal(torch.isfinite(clean[1]))


MORE_ROWS = [  # as CASES: bf16 with d = 64 and more rows than a CTA has, one KV head each and several
    (1, 100, 3, 1, 64, [700], 8, 128, 16, 24, 0),                 # 300 rows: two row tiles, the second with a half alone
    (2, 72, 16, 2, 64, [90, 3000], 16, 80, 64, 64, 1),            # 576 rows: three row tiles, runs of whole pages
    (3, 256, 2, 1, 64, [1500, 0, 300], 4, 256, 128, 32, 0),       # 512 rows of the largest trees
]


@pytest.mark.parametrize("case", range(len(MORE_ROWS)))
def test_more_rows_than_a_cta_has_at_d_64(case):
    B, T, Hq, Hkv, d, lens, g, w, rows, crows, mode = MORE_ROWS[case]
    x = make(B, T, Hq, Hkv, d, lens, g, w, rows, crows, torch.bfloat16, mode, seed=80 + case)
    check(x, g, w, rows, crows, mode, f"case {case}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d,Hq,T", [(128, 8, 16), (128, 2, 1), (64, 2, 2), (64, 8, 16), (128, 32, 24)])
def test_a_sequence_alone_and_in_a_batch(d, Hq, T, dtype):
    """What else is in the batch decides where a list is cut, and so the last bits alone: each sequence,
    alone and among others, is within the bound of the definition, and so within twice it of itself."""
    g, w, rows, lens = 16, 256, 64, [900, 10, 2500, 1300]
    x = make(4, T, Hq, 2, d, lens, g, w, rows, rows, dtype, seed=90)
    O, LSE = check(x, g, w, rows, rows, what="batch")
    for b in range(4):
        y = {k: v if "cp" in k or k in ("Kp", "Vp") else v[b:b + 1].contiguous() for k, v in x.items()}
        o, lse = check(y, g, w, rows, rows, what=f"sequence {b} alone")
        ref = tree(y["Q"], x["Kp"], x["Vp"], y["table"], x["Kcp"], x["Vcp"], y["core_table"], y["lens"], y["parents"], g, w, rows, rows)
        assert (np.abs(t64(o) - t64(O[b:b + 1])) <= 2 * ref[2]).all() and (np.abs(t64(lse) - t64(LSE[b:b + 1])) <= 2 * ref[3]).all()
