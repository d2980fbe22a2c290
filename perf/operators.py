"""Cases of the rotary, tree-attention, page and paged-pooling operators: what a serving or training
step asks of them, with a plain form in elementary torch operations and a 64-bit definition.

A CCA cache is kept in pages.  A pool is [pages, Hkv, rows, d] (K and V alike); `table[b, c]` names the
page that holds rows c*rows .. of sequence b, -1 where there is none.  Raw tokens and core tokens each
have a pool and a table.  `refs[page]` counts the table entries that hold a page.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- the cases

def _rope(name, **kw):
    c = dict(op="rope", B=1, N=1024, Hq=8, Hkv=8, d=128, rot=128, layout="half", dtype="bf16", base=10000.0,
             stretch=1.0, factor=1.0, given=False, grad=False)
    return {**({"name": name} if name else {}), **c, **kw}


def _append(name, **kw):
    c = dict(op="append", B=1, T=8, Hq=32, Hkv=8, d=128, rot=128, layout="half", dtype="bf16", base=10000.0,
             stretch=1.0, factor=1.0, ctx=8192, rows=64, w=1024, g=16, ragged=0.5)
    return {**({"name": name} if name else {}), **c, **kw}


def _tree(name, **kw):
    c = dict(op="tree", B=1, T=8, Hq=32, Hkv=8, d=128, dtype="bf16", ctx=8192, g=16, w=1024, rows=64, crows=64,
             ragged=0.5, aligned=False, pad=0.1)
    return {**({"name": name} if name else {}), **c, **kw}


def _branch(name, **kw):
    c = dict(op="branch", seqs=4, layers=2, Hkv=8, d=128, dtype="bf16", rows=64, w=1024, T=16)
    return {**({"name": name} if name else {}), **c, **kw}


def _compact(name, **kw):
    c = dict(op="compact", B=4, layers=2, Hkv=8, d=128, dtype="bf16", rows=64, w=1024, T=16, A=6)
    return {**({"name": name} if name else {}), **c, **kw}


def _pool(name, **kw):
    c = dict(op="pool", B=4, T=16, A=6, Hq=32, Hkv=8, d=128, dtype="bf16", ctx=4096, g=16, w=1024, rows=64, crows=64,
             prompt=False)
    return {**({"name": name} if name else {}), **c, **kw}


def listed():
    return [
        # the prompt's queries and keys of a 32 K grouped-query layer, straight from the projections
        _rope("rope-prompt", N=32768, Hq=32, Hkv=8, base=500000.0, stretch=8.0),
        # a training step in fp32 with part of the head rotated, pairs interleaved, positions of packed documents
        _rope("rope-train", B=2, N=4099, Hq=16, Hkv=16, d=64, rot=32, layout="interleaved", dtype="f32", factor=1.1386,
              stretch=4.0, given=True, grad=True),
        # the drafted tokens of a serving step: rotated and stored into their pages
        _append("append-drafts", B=16, T=32, ctx=32768),
        # plain decoding, one token of one sequence
        _tree("tree-one-token", B=1, T=1, Hkv=32, ctx=32768, ragged=0.0, pad=0.0),
        # a serving batch of drafted trees, lengths all different
        _tree("tree-batch", B=8, T=24, ctx=32768),
        # wide trees over the longest contexts
        _tree("tree-long", B=16, T=64, ctx=131072, ragged=0.1),
        # the fp32 path: small heads, pages that end inside a tile, the group-aligned window
        _tree("tree-f32", B=3, T=7, Hq=4, Hkv=2, d=64, dtype="f32", ctx=1500, g=8, w=100, rows=16, crows=48, aligned=True),
        # a few sequences branch and one branch of each is dropped: latency
        _branch("branch-few"),
        # a large beam branches through several layers' pools
        _branch("branch-many", seqs=32, layers=4),
        # accepted tokens of every sequence move to the front, in all layers
        _compact("compact-accepted", B=32, layers=8, T=64, A=9),
        # groups that the accepted tokens complete
        _pool("pool-step", B=32, T=64, A=20, ctx=8192),
        # all groups of a prompt stored in pages
        _pool("pool-prompt", B=1, T=32768, A=32768, Hkv=32, ctx=0, prompt=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "append", "tree", "tree", "tree", "branch", "compact", "pool"])
    d = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 8])
    rows = rng.choice([16, 32, 48, 64, 128])
    g = rng.choice([4, 8, 16, 32])
    w = rng.choice([256, 512, 1024])
    rope = dict(d=d, rot=rng.choice([d, d, d // 2, d // 4, 24]), layout=rng.choice(["half", "interleaved"]), dtype=dtype,
                base=rng.choice([10000.0, 500000.0]), stretch=rng.choice([1.0, 2.0, 8.0]), factor=rng.choice([1.0, 1.25]))
    if op == "rope":
        return _rope(None, B=rng.randint(1, 3), N=_log(rng, 1, 8192), Hq=Hq, Hkv=Hkv, given=rng.random() < 0.5,
                     grad=rng.random() < 0.5, **rope)
    if op == "append":
        return _append(None, B=_log(rng, 1, 32), T=_log(rng, 1, 64), Hq=Hq, Hkv=Hkv, ctx=_log(rng, 64, 32768), rows=rows,
                       w=w, g=g, **rope)
    if op == "tree":
        f32 = dtype == "f32"
        return _tree(None, B=_log(rng, 1, 4 if f32 else 16), T=_log(rng, 1, 16 if f32 else 64), Hq=Hq, Hkv=Hkv, d=d,
                     dtype=dtype, ctx=_log(rng, 64, 4096 if f32 else 65536), g=g, w=w, rows=rows,
                     crows=rng.choice([16, 40, 64]), ragged=rng.choice([0.0, 0.5, 0.9]), aligned=rng.random() < 0.3,
                     pad=rng.choice([0.0, 0.2]))
    if op == "branch":
        return _branch(None, seqs=_log(rng, 1, 32), layers=rng.randint(1, 4), Hkv=Hkv, d=d, dtype=dtype, rows=rows, w=w,
                       T=_log(rng, 1, 64))
    if op == "compact":
        T = _log(rng, 2, 64)
        return _compact(None, B=_log(rng, 1, 32), layers=rng.randint(1, 8), Hkv=Hkv, d=d, dtype=dtype, rows=rows, w=w, T=T,
                        A=rng.randint(1, T))
    T = _log(rng, 1, 64)
    return _pool(None, B=_log(rng, 1, 32), T=T, A=rng.randint(1, T), Hq=Hq, Hkv=Hkv, d=d, dtype=dtype,
                 ctx=_log(rng, 64, 16384), g=g, w=w, rows=rows, crows=rng.choice([16, 40, 64]))


# ---------------------------------------------------------------- the inputs

class _Inputs:
    """Random tensors of one seed; K rows hold a few heavy positions, as long contexts do."""

    def __init__(self, case, seed):
        self.dev = torch.device("cuda")
        self.gen = torch.Generator(device=self.dev)
        self.gen.manual_seed(seed)
        self.dt = DT[case["dtype"]]
        self.scale = 1.0 if case["dtype"] == "f32" else case["d"] ** -0.25

    def normal(self, *shape):
        return (torch.randn(shape, generator=self.gen, device=self.dev) * self.scale).to(self.dt)

    def heavy(self, *shape):
        """Rows [..., n, d] with one in a hundred four times as large."""
        x = torch.randn(shape, generator=self.gen, device=self.dev) * self.scale
        big = torch.rand(shape[:-1], generator=self.gen, device=self.dev) < 0.01
        return (x * (1.0 + 3.0 * big[..., None])).to(self.dt)

    def uniform(self, *shape):
        return torch.rand(shape, generator=self.gen, device=self.dev)

    def integers(self, lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=self.gen, device=self.dev, dtype=torch.int32)

    def lens(self, B, ctx, ragged):
        return (ctx - (self.uniform(B) * ragged * ctx).floor()).to(torch.int32)

    def tree(self, B, T, pad):
        """Parents of drafted nodes: mostly chains that branch, the last ones of some sequences padding (-2)."""
        t = torch.arange(T, device=self.dev)
        back = 1 + (self.uniform(B, T) ** 3 * 6.0).floor()
        par = torch.clamp(t - back, min=-1).to(torch.int32)
        n = T - (self.uniform(B) * pad * T).round()
        return torch.where(t < n[:, None], par, torch.full_like(par, -2))

    def table(self, first, last, cols, most, spare=3):
        """A table whose entries [first, last), `most` of them at most, name pages in random order, and the number of pages."""
        c = torch.arange(cols, device=self.dev)
        held = (c >= first[:, None]) & (c < last[:, None])
        n = min(cols, most) * held.shape[0] + spare
        order = torch.randperm(n, generator=self.gen, device=self.dev).to(torch.int32)
        rank = torch.cumsum(held.flatten().to(torch.int64), 0).reshape(held.shape) - 1
        return torch.where(held, order[rank.clamp(min=0)], torch.full_like(order[:1], -1)), n


def _freq(case, dev):
    """Frequencies of the pairs: base^(-2i/rot), the slow ones stretched for a longer context."""
    rot = case["rot"]
    i = torch.arange(rot // 2, dtype=torch.float64, device=dev)
    f = case["base"] ** (-2.0 * i / rot)
    turns = f * 8192 / (2.0 * math.pi)                       # over the context that was trained on
    keep = ((turns - 1.0) / 3.0).clamp(0.0, 1.0)             # fast pairs stay, slow pairs are stretched
    return f * (keep + (1.0 - keep) / case["stretch"])


def _ceil(a, b):
    return -(-a // b)


def prepare(case, seed):
    x = _Inputs(case, seed)
    op, dev = case["op"], x.dev
    s = {"case": case, "op": op}
    if op in ("rope", "append"):
        s["freq"] = _freq(case, dev)
    if op == "rope":
        B, N, d = case["B"], case["N"], case["d"]
        # the projections' layout [B, N, H, d]; the operator reads it as [B, H, N, d]
        s["Q"] = x.normal(B, N, case["Hq"], d).transpose(1, 2)
        s["K"] = x.normal(B, N, case["Hkv"], d).transpose(1, 2)
        s["positions"] = None
        if case["given"]:
            cut = 1 + (x.uniform(B, 1) * N).floor().to(torch.int32)
            i = torch.arange(N, device=dev, dtype=torch.int32)
            s["positions"] = torch.where(i < cut, i, i - cut).contiguous() + 5 * 8192
        if case["grad"]:
            s["dQ"], s["dK"] = x.normal(B, case["Hq"], N, d), x.normal(B, case["Hkv"], N, d)
            s["Q"], s["K"] = s["Q"].requires_grad_(), s["K"].requires_grad_()
        return s
    if op == "branch":
        n, L, P, T = case["seqs"], case["layers"], case["rows"], case["T"]
        lens = x.integers(case["w"] + T, 4 * case["w"], n)
        lens = torch.cat([lens, torch.zeros_like(lens)])
        cols = _ceil(4 * case["w"] + T, P) + 1
        first, last = (lens - case["w"]).clamp(min=0) // P, _ceil(lens, P)
        s["table"], held = x.table(first, last, cols, _ceil(case["w"], P) + 1)
        s["refs"] = torch.zeros(held + n * (1 + _ceil(T, P)), dtype=torch.int32, device=dev)
        s["refs"][s["table"][s["table"] >= 0].long()] = 1
        s["src"] = torch.randperm(n, generator=x.gen, device=dev).to(torch.int32)
        s["dst"] = torch.arange(n, 2 * n, device=dev, dtype=torch.int32)
        s["lens"] = torch.cat([lens[:n], lens[s["src"].long()]])
        s["extra"] = torch.full_like(lens, T)
        s["drop"] = torch.cat([last[:n], torch.zeros_like(last[n:])]).to(torch.int32)
        s["end"] = torch.full_like(lens, cols)
        s["Kp"] = x.normal(L, s["refs"].numel(), case["Hkv"], P, case["d"])
        s["Vp"] = x.normal(L, s["refs"].numel(), case["Hkv"], P, case["d"])
        return s
    if op == "compact":
        B, L, P, T, A = case["B"], case["layers"], case["rows"], case["T"], case["A"]
        s["lens"] = x.integers(case["w"], 4 * case["w"], B)
        cols = _ceil(4 * case["w"] + T, P)
        s["table"], n = x.table((s["lens"] - case["w"]) // P, _ceil(s["lens"] + T, P), cols, _ceil(case["w"] + T, P) + 1)
        # an increasing choice of A of the T nodes; the first `accepted` of them count
        s["path"] = torch.sort(torch.argsort(x.uniform(B, T), 1)[:, :A], 1)[0].to(torch.int32)
        s["accepted"] = x.integers(0, A + 1, B)
        s["Kp"], s["Vp"] = x.normal(L, n, case["Hkv"], P, case["d"]), x.normal(L, n, case["Hkv"], P, case["d"])
        return s
    B, T, g, w, P = case["B"], case["T"], case["g"], case["w"], case["rows"]
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    s["lens"] = x.lens(B, case["ctx"], case.get("ragged", 0.5))
    behind = torch.zeros_like(s["lens"]) if op == "pool" else (s["lens"] - w - g).clamp(min=0)
    if op == "pool":
        behind = (s["lens"] - g).clamp(min=0)
    s["table"], n = x.table(behind // P, _ceil(s["lens"] + T, P), _ceil(case["ctx"] + T, P),
                            _ceil((0 if op == "pool" else w) + g + T, P) + 1)
    s["Kp"], s["Vp"] = x.heavy(n, Hkv, P, d), x.normal(n, Hkv, P, d)
    if op in ("tree", "append"):
        s["parents"] = x.tree(B, T, case.get("pad", 0.1))
    if op == "append":
        s["Q"] = x.normal(B, T, Hq, d).transpose(1, 2)
        s["K"] = x.normal(B, T, Hkv, d).transpose(1, 2)
        s["V"] = x.normal(B, T, Hkv, d).transpose(1, 2)
        return s
    R = case["crows"]
    cores = (s["lens"] + T) // g + 1
    s["ctable"], n = x.table(torch.zeros_like(cores), _ceil(cores, R), _ceil((case["ctx"] + T) // g + 1 + _ceil(T, g), R) + 1,
                             _ceil((case["ctx"] + T) // g + 1, R))
    s["Kcp"], s["Vcp"] = x.heavy(n, Hkv, R, d), x.normal(n, Hkv, R, d)
    s["Q"] = x.normal(B, Hq, T, d)
    if op == "pool":
        A = case["A"]
        s["path"] = None
        s["accepted"] = torch.full_like(s["lens"], A)
        if not case["prompt"]:
            s["path"] = torch.sort(torch.argsort(x.uniform(B, T), 1)[:, :A], 1)[0].to(torch.int32)
            s["accepted"] = x.integers(0, A + 1, B)
    return s


# ---------------------------------------------------------------- the plain forms

def _turn(X, pos, freq, layout, factor, back=False):
    """X [B, H, N, d] with its first 2 * len(freq) columns rotated by pos [B, N] * freq."""
    r = freq.numel()
    ang = pos[:, None, :, None].to(torch.float64) * freq
    c, s = (ang.cos() * factor).float(), (ang.sin() * (-factor if back else factor)).float()
    x = X.float()
    a, b = (x[..., :r], x[..., r:2 * r]) if layout == "half" else (x[..., 0:2 * r:2], x[..., 1:2 * r:2])
    u, v = a * c - b * s, b * c + a * s
    y = torch.cat([u, v], -1) if layout == "half" else torch.stack([u, v], -1).flatten(-2)
    return torch.cat([y, x[..., 2 * r:]], -1).to(X.dtype)


def _ancestry(parents):
    """(sees [B, T, T]: node, ancestor or itself; depth [B, T]; whole [B, T]: the chain ends at the root)."""
    B, T = parents.shape
    t = torch.arange(T, device=parents.device)
    ok = (parents >= 0) & (parents < t)
    step = ((parents[..., None] == t) & ok[..., None]).float()
    sees = torch.linalg.matrix_power(torch.eye(T, device=parents.device) + step, max(T - 1, 1)) > 0
    whole = (sees & (parents == -1)[:, None, :]).any(-1)
    return sees & whole[..., None], (sees.sum(-1) - 1).to(torch.int64) * whole, whole


def _rows(pool, table, idx):
    """Rows idx [B, n] of each sequence: [B, Hkv, n, d]."""
    P = pool.shape[-2]
    page = table.gather(1, (idx // P).clamp(0, table.shape[1] - 1)).clamp(min=0).long()
    return pool[page, :, idx % P].transpose(1, 2)


def _store(pool, table, idx, rows, valid):
    """Writes rows [B, Hkv, n, d] at idx [B, n] where valid, leaves the others as they are."""
    P = pool.shape[-2]
    page = table.gather(1, idx // P).long()
    old = pool[page, :, idx % P]
    pool[page, :, idx % P] = torch.where(valid[..., None, None], rows.transpose(1, 2).to(pool.dtype), old)


def _plain_tree(s):
    c = s["case"]
    B, T, g, w, Hq, Hkv, d = c["B"], c["T"], c["g"], c["w"], c["Hq"], c["Hkv"], c["d"]
    dev, lens = s["lens"].device, s["lens"].long()
    sees, depth, whole = _ancestry(s["parents"])
    pos = lens[:, None] + depth
    lo = (pos - w + 1).clamp(min=0)
    start = lo // g * g if c["aligned"] else lo
    base = (lens - w + 1).clamp(min=0)
    base = base // g * g if c["aligned"] else base
    core = torch.arange(c["ctx"] // g + 1, device=dev).expand(B, -1)
    raw = base[:, None] + torch.arange(w + g, device=dev)
    node = lens[:, None] + torch.arange(T, device=dev)
    vis = torch.cat([core[:, None, :] < (lo // g)[..., None],
                     (raw[:, None, :] >= start[..., None]) & (raw < lens[:, None])[:, None, :], sees], -1)
    vis &= whole[..., None]
    k = torch.cat([_rows(s["Kcp"], s["ctable"], core), _rows(s["Kp"], s["table"], raw), _rows(s["Kp"], s["table"], node)], 2)
    v = torch.cat([_rows(s["Vcp"], s["ctable"], core), _rows(s["Vp"], s["table"], raw), _rows(s["Vp"], s["table"], node)], 2)
    q = s["Q"].float().reshape(B, Hkv, Hq // Hkv, T, d)
    z = (q @ k.float()[:, :, None].transpose(-1, -2)) * d ** -0.5
    z = z.masked_fill(~vis[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = (z - top).exp()
    total = p.sum(-1, keepdim=True)
    out = (p @ v.float()[:, :, None]) / torch.where(total == 0, torch.ones_like(total), total)
    return out.reshape(B, Hq, T, d).to(s["Q"].dtype), (top + total.log()).reshape(B, Hq, T)


def _plain_branch(s):
    P = s["case"]["rows"]
    table, refs, src, dst = s["table"], s["refs"], s["src"].long(), s["dst"].long()
    B, M = table.shape
    c = torch.arange(M, device=table.device)
    # each destination row holds the source's pages too
    shared = torch.where(c < _ceil(s["lens"][src], P)[:, None], table[src], torch.full_like(table[src], -1))
    table[dst] = shared
    refs.index_add_(0, shared.clamp(min=0).flatten().long(), (shared >= 0).flatten().to(torch.int32))
    # room for the next rows: a page for each missing entry, and for each shared one but its last holder's
    reach = (c >= (s["lens"] // P)[:, None]) & (c < _ceil(s["lens"] + s["extra"], P)[:, None]) & (s["extra"] > 0)[:, None]
    same = (table[:, None, :] == table[None, :, :]) & reach[:, None, :] & reach[None, :, :] & (table >= 0)[:, None, :]
    before = (same & torch.ones(B, B, dtype=torch.bool, device=table.device).tril(-1)[..., None]).sum(1)
    split = reach & (table >= 0) & (refs[table.clamp(min=0).long()] - before > 1)
    need = split | (reach & (table < 0))
    empty = torch.argsort((refs != 0).to(torch.int8), stable=True)
    rank = (torch.cumsum(need.flatten().to(torch.int64), 0) - 1).reshape(B, M)
    fits = need.sum() <= (refs == 0).sum()
    need, split = need & fits, split & fits
    fresh = empty[rank.clamp(0, refs.numel() - 1)].to(torch.int32)
    old = table.clamp(min=0)
    col = (s["lens"] // P).clamp(max=M - 1)[:, None].long()
    moved = split.gather(1, col)[:, 0] & (s["lens"] % P != 0)
    none = torch.full_like(old[:, 0], -1)
    pairs = torch.stack([torch.where(moved, old.gather(1, col)[:, 0], none), torch.where(moved, fresh.gather(1, col)[:, 0], none)], 1)
    refs.index_add_(0, fresh.flatten().long(), need.flatten().to(torch.int32))
    refs.index_add_(0, old.flatten().long(), -split.flatten().to(torch.int32))
    table.copy_(torch.where(need, fresh, table))
    # the pages that were split are copied
    real = pairs[pairs[:, 0] >= 0].long()
    s["Kp"][:, real[:, 1]] = s["Kp"][:, real[:, 0]]
    s["Vp"][:, real[:, 1]] = s["Vp"][:, real[:, 0]]
    held = table.clone()
    # one branch of each is dropped, and the room that was not used
    gone = (c >= s["drop"][:, None]) & (c < s["end"][:, None]) & (table >= 0)
    refs.index_add_(0, table.clamp(min=0).flatten().long(), -gone.flatten().to(torch.int32))
    table.masked_fill_(gone, -1)
    return {"pairs": pairs, "held": held, "table": table, "refs": refs, "Kp": s["Kp"], "Vp": s["Vp"]}


def _plain_compact(s):
    lens, P = s["lens"].long(), s["case"]["rows"]
    j = torch.arange(s["path"].shape[1], device=lens.device)
    valid = j < s["accepted"][:, None]
    a, b = lens[:, None] + s["path"], lens[:, None] + j
    pa, pb = s["table"].gather(1, a // P).long(), s["table"].gather(1, b // P).long()
    pick = valid[None, :, :, None, None]
    s["Kp"][:, pb, :, b % P] = torch.where(pick, s["Kp"][:, pa, :, a % P].movedim(2, 0), s["Kp"][:, pb, :, b % P].movedim(2, 0)).movedim(0, 2)
    s["Vp"][:, pb, :, b % P] = torch.where(pick, s["Vp"][:, pa, :, a % P].movedim(2, 0), s["Vp"][:, pb, :, b % P].movedim(2, 0)).movedim(0, 2)
    return {"Kp": s["Kp"], "Vp": s["Vp"]}


def _plain_pool(s):
    c = s["case"]
    B, T, g, Hq, Hkv, d = c["B"], c["T"], c["g"], c["Hq"], c["Hkv"], c["d"]
    lens, dev = s["lens"].long(), s["lens"].device
    j = lens[:, None] // g + torch.arange((c["A"] - 1) // g + 1, device=dev)
    done = (j + 1) * g <= (lens + s["accepted"])[:, None]
    i = ((j + 1) * g - 1 - lens[:, None]).clamp(0, c["A"] - 1)
    i = i if s["path"] is None else s["path"].gather(1, i).long()
    q = s["Q"].float().reshape(B, Hkv, Hq // Hkv, T, d).mean(2)
    q = q.gather(2, i[:, None, :, None].expand(-1, Hkv, -1, d))
    n = j.shape[1]
    idx = torch.where(done[..., None], j[..., None] * g + torch.arange(g, device=dev), (lens[:, None, None] - 1).clamp(min=0)).reshape(B, n * g)
    k = _rows(s["Kp"], s["table"], idx).float().reshape(B, Hkv, n, g, d)
    v = _rows(s["Vp"], s["table"], idx).float().reshape(B, Hkv, n, g, d)
    z = (k * q[:, :, :, None]).sum(-1) * d ** -0.5
    p = (z - z.amax(-1, keepdim=True)).exp()
    p = p / p.sum(-1, keepdim=True)
    _store(s["Kcp"], s["ctable"], j, (p[..., None] * k).sum(-2), done)
    _store(s["Vcp"], s["ctable"], j, (p[..., None] * v).sum(-2), done)
    return {"Kcp": s["Kcp"], "Vcp": s["Vcp"]}


def _plain(s):
    c, op = s["case"], s["op"]
    if op == "rope":
        B, N = c["B"], c["N"]
        pos = s["positions"] if c["given"] else torch.arange(N, device=s["Q"].device).expand(B, N)
        with torch.no_grad():
            out = [_turn(s["Q"], pos, s["freq"], c["layout"], c["factor"]), _turn(s["K"], pos, s["freq"], c["layout"], c["factor"])]
            if c["grad"]:
                out += [_turn(s["dQ"], pos, s["freq"], c["layout"], c["factor"], True),
                        _turn(s["dK"], pos, s["freq"], c["layout"], c["factor"], True)]
        return out
    if op == "append":
        _, depth, whole = _ancestry(s["parents"])
        pos, slot = s["lens"][:, None] + depth, s["lens"][:, None].long() + torch.arange(c["T"], device=depth.device)
        q = _turn(s["Q"], pos, s["freq"], c["layout"], c["factor"])
        _store(s["Kp"], s["table"], slot, _turn(s["K"], pos, s["freq"], c["layout"], c["factor"]), whole)
        _store(s["Vp"], s["table"], slot, s["V"], whole)
        return {"Q": torch.where(whole[:, None, :, None], q, torch.zeros_like(q)), "Kp": s["Kp"], "Vp": s["Vp"]}
    return {"tree": _plain_tree, "branch": _plain_branch, "compact": _plain_compact, "pool": _plain_pool}[op](s)


# ---------------------------------------------------------------- the framework's calls

def _framework(s):
    from sparse_long_context_cca_gb300 import api
    c, op = s["case"], s["op"]
    if op == "rope":
        if not c["grad"]:
            return list(api.cca_rope(s["Q"], s["K"], s["freq"], positions=s["positions"], layout=c["layout"], factor=c["factor"]))
        q, k = api.rope(s["Q"], s["K"], s["freq"], positions=s["positions"], layout=c["layout"], factor=c["factor"])
        return [q.detach(), k.detach(), *torch.autograd.grad([q, k], [s["Q"], s["K"]], [s["dQ"], s["dK"]])]
    if op == "append":
        q = api.cca_rope_append(s["Q"], s["K"], s["V"], s["Kp"], s["Vp"], s["table"], s["lens"], s["freq"], parents=s["parents"],
                                layout=c["layout"], factor=c["factor"])
        return {"Q": q, "Kp": s["Kp"], "Vp": s["Vp"]}
    if op == "tree":
        return api.cca_tree_fwd(s["Q"], s["Kp"], s["Vp"], s["table"], s["Kcp"], s["Vcp"], s["ctable"], s["lens"], c["g"], c["w"],
                                parents=s["parents"], window_mode=int(c["aligned"]))
    if op == "branch":
        api.cca_pages_fork(s["refs"], s["table"], s["src"], s["dst"], s["lens"], c["rows"])
        pairs = api.cca_pages_reserve(s["refs"], s["table"], s["lens"], s["extra"], c["rows"])
        api.cca_pages_copy(s["Kp"], s["Vp"], pairs)
        held = s["table"].clone()
        api.cca_pages_free(s["refs"], s["table"], s["drop"], s["end"])
        return {"pairs": pairs, "held": held, "table": s["table"], "refs": s["refs"], "Kp": s["Kp"], "Vp": s["Vp"]}
    if op == "compact":
        api.cca_pages_compact(s["Kp"], s["Vp"], s["table"], s["lens"], s["path"], s["accepted"])
        return {"Kp": s["Kp"], "Vp": s["Vp"]}
    api.cca_pool_pages(s["Q"], s["Kp"], s["Vp"], s["table"], s["Kcp"], s["Vcp"], s["ctable"], s["lens"], s["accepted"], c["g"],
                       path=s["path"])
    return {"Kcp": s["Kcp"], "Vcp": s["Vcp"]}


def run(state):
    return _framework(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c, op = case, case["op"]
    e, d = (2 if c["dtype"] == "bf16" else 4), c["d"]
    if op == "rope":
        n = c["B"] * c["N"] * (c["Hq"] + c["Hkv"]) * (2 if c["grad"] else 1)
        return {"bytes": 2.0 * n * d * e, "flops": 3.0 * n * c["rot"]}
    if op == "append":
        n = c["B"] * c["T"] * (c["Hq"] + 2 * c["Hkv"])
        return {"bytes": 2.0 * n * d * e, "flops": 3.0 * c["B"] * c["T"] * (c["Hq"] + c["Hkv"]) * c["rot"]}
    if op == "tree":
        mean = c["ctx"] * (1.0 - c["ragged"] / 2.0)
        keys = max(0.0, mean - c["w"] + 1) / c["g"] + min(mean, c["w"] - 1.0)
        rows = c["B"] * c["Hq"] * c["T"]
        return {"bytes": c["B"] * c["Hkv"] * (keys + c["T"]) * 2.0 * d * e + rows * (2.0 * d * e + 4.0),
                "flops": 4.0 * d * rows * (keys + c["T"] / 4.0)}
    if op == "branch":
        cols = _ceil(4 * c["w"] + c["T"], c["rows"]) + 1
        return {"bytes": c["seqs"] * (4.0 * c["layers"] * c["Hkv"] * c["rows"] * d * e + 8.0 * cols), "flops": 0.0}
    if op == "compact":
        return {"bytes": c["B"] * (c["A"] / 2.0) * c["layers"] * c["Hkv"] * d * e * 4.0, "flops": 0.0}
    groups = c["B"] * (c["A"] if c["prompt"] else c["A"] / 2.0) / c["g"]
    rows = groups * c["Hkv"] * (2.0 * c["g"] + 2.0) + groups * c["Hq"]
    return {"bytes": rows * d * e, "flops": groups * c["Hkv"] * c["g"] * d * 6.0}


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_branch(c, s):
    """One row after the other on the host; the pools in 64 bits."""
    P, table, refs = c["rows"], s["table"].tolist(), s["refs"].tolist()
    lens, extra = s["lens"].tolist(), s["extra"].tolist()
    Kp, Vp = s["Kp"].to(torch.float64), s["Vp"].to(torch.float64)
    for a, z in zip(s["src"].tolist(), s["dst"].tolist()):
        for k in range(-(-lens[a] // P)):
            table[z][k] = table[a][k]
            if table[a][k] >= 0:
                refs[table[a][k]] += 1
    pairs, copies, wanted = [], [], []
    left = list(refs)
    for b, row in enumerate(table):
        for k in range(lens[b] // P, -(-(lens[b] + extra[b]) // P)):
            if row[k] >= 0 and left[row[k]] > 1:
                left[row[k]] -= 1
                wanted.append((b, k, row[k]))
            elif row[k] < 0:
                wanted.append((b, k, -1))
    free = [p for p, held in enumerate(refs) if held == 0]
    got = {b: [-1, -1] for b in range(len(table))}
    for (b, k, old), new in zip(wanted, free):
        table[b][k] = new
        left[new] += 1
        if old >= 0 and k == lens[b] // P and lens[b] % P:
            got[b] = [old, new]
            copies.append((old, new))
    for old, new in copies:
        Kp[:, new], Vp[:, new] = Kp[:, old], Vp[:, old]
    pairs = [got[b] for b in range(len(table))]
    held = [list(row) for row in table]
    for b, (a, z) in enumerate(zip(s["drop"].tolist(), s["end"].tolist())):
        for k in range(a, min(z, len(table[b]))):
            if table[b][k] >= 0:
                left[table[b][k]] -= 1
                table[b][k] = -1
    whole = lambda v: torch.tensor(v, dtype=torch.int32, device=s["table"].device)  # noqa: E731
    return {"pairs": whole(pairs), "held": whole(held), "table": whole(table), "refs": whole(left), "Kp": Kp, "Vp": Vp}


def exact(case, seed):
    c, op = case, case["op"]
    s = prepare(case, seed)
    wide = torch.float64
    if op == "branch":
        return _exact_branch(c, s)
    B, d = c["B"], c["d"]
    if op == "compact":
        P, table, lens = c["rows"], s["table"].tolist(), s["lens"].tolist()
        Kp, Vp = s["Kp"].to(wide), s["Vp"].to(wide)
        for b, path in enumerate(s["path"].tolist()):
            for j in range(int(s["accepted"][b])):   # one row after the other, front to back
                a, z = lens[b] + path[j], lens[b] + j
                for pool in (Kp, Vp):
                    pool[:, table[b][z // P], :, z % P] = pool[:, table[b][a // P], :, a % P]
        return {"Kp": Kp, "Vp": Vp}
    if op in ("rope", "append"):
        half, n = c["layout"] == "half", c["rot"] // 2
        first = list(range(n)) if half else list(range(0, 2 * n, 2))
        second = list(range(n, 2 * n)) if half else list(range(1, 2 * n, 2))

        def complex_turn(X, pos, sign):
            """The pairs as complex numbers, times factor * exp(i * sign * pos * freq)."""
            y = X.detach().to(wide).clone()
            z = torch.complex(y[..., first], y[..., second])
            a = (pos.to(wide)[:, :, None] * s["freq"])[:, None]
            z = z * torch.polar(torch.full_like(a, c["factor"]), sign * a)
            y[..., first], y[..., second] = z.real, z.imag
            return y

    if op == "rope":
        pos = s["positions"] if c["given"] else torch.arange(c["N"], device=s["Q"].device).expand(B, -1)
        out = [complex_turn(s["Q"], pos, 1.0), complex_turn(s["K"], pos, 1.0)]
        return out + [complex_turn(s["dQ"], pos, -1.0), complex_turn(s["dK"], pos, -1.0)] if c["grad"] else out
    lens, table = s["lens"].tolist(), s["table"].tolist()
    P = c["rows"]

    def chains(parents):
        """Each node's chain from itself to the root, None where it does not reach the root."""
        out = []
        for t in range(len(parents)):
            chain, k = [], t
            while k >= 0:
                chain.append(k)
                k = parents[k] if parents[k] < k else -2
            out.append(chain if k == -1 else None)
        return out

    if op == "append":
        parents = s["parents"].tolist()
        up = [chains(p) for p in parents]
        pos = torch.tensor([[lens[b] + (len(ch) - 1 if ch else 0) for ch in up[b]] for b in range(B)], device=s["Q"].device)
        q, k, v = complex_turn(s["Q"], pos, 1.0), complex_turn(s["K"], pos, 1.0), s["V"].to(wide)
        Kp, Vp = s["Kp"].to(wide), s["Vp"].to(wide)
        for b in range(B):
            for t, ch in enumerate(up[b]):
                if ch is None:
                    q[b, :, t] = 0
                    continue
                page, row = table[b][(lens[b] + t) // P], (lens[b] + t) % P
                Kp[page, :, row], Vp[page, :, row] = k[b, :, t], v[b, :, t]
        return {"Q": q, "Kp": Kp, "Vp": Vp}
    ctable, R, g = s["ctable"].tolist(), c["crows"], c["g"]
    Hq, Hkv, T = c["Hq"], c["Hkv"], c["T"]

    def fetch(pool, tab, rows, idx):
        at = torch.tensor([[tab[i // rows], i % rows] for i in idx], device=pool.device, dtype=torch.int64).reshape(-1, 2)
        return pool[at[:, 0], :, at[:, 1]].to(wide).transpose(0, 1)

    if op == "pool":
        Kcp, Vcp = s["Kcp"].to(wide), s["Vcp"].to(wide)
        path = s["path"].tolist() if s["path"] is not None else None
        taken = s["accepted"].tolist()
        for b in range(B):
            groups = [j for j in range(lens[b] // g, (lens[b] + taken[b]) // g)]
            if not groups:
                continue
            last = [(j + 1) * g - 1 - lens[b] for j in groups]
            nodes = last if path is None else [path[b][i] for i in last]
            idx = [j * g + t for j in groups for t in range(g)]
            k = fetch(s["Kp"], table[b], P, idx).reshape(Hkv, len(groups), g, d)
            v = fetch(s["Vp"], table[b], P, idx).reshape(Hkv, len(groups), g, d)
            q = s["Q"][b][:, nodes].to(wide).reshape(Hkv, Hq // Hkv, len(groups), d)
            a = torch.softmax(torch.einsum("hrnd,hngd->hrng", q, k).mean(1) / math.sqrt(d), -1)
            at = torch.tensor([[ctable[b][j // R], j % R] for j in groups], device=k.device)
            Kcp[at[:, 0], :, at[:, 1]] = torch.einsum("hng,hngd->nhd", a, k)
            Vcp[at[:, 0], :, at[:, 1]] = torch.einsum("hng,hngd->nhd", a, v)
        return {"Kcp": Kcp, "Vcp": Vcp}
    w = c["w"]
    out = torch.zeros(B, Hq, T, d, dtype=wide, device=s["Q"].device)
    lse = torch.full((B, Hq, T), -math.inf, dtype=wide, device=s["Q"].device)
    for b, parents in enumerate(s["parents"].tolist()):
        up = chains(parents)
        live = [t for t in range(T) if up[t] is not None]
        if not live:
            continue
        lo = {t: max(0, lens[b] + len(up[t]) - 1 - w + 1) for t in live}
        begin = {t: lo[t] // g * g if c["aligned"] else lo[t] for t in live}
        cores, raw = max(lo.values()) // g, range(min(begin.values()), lens[b])
        k = torch.cat([fetch(s["Kcp"], ctable[b], R, range(cores)), fetch(s["Kp"], table[b], P, [*raw, *range(lens[b], lens[b] + T)])], 1)
        v = torch.cat([fetch(s["Vcp"], ctable[b], R, range(cores)), fetch(s["Vp"], table[b], P, [*raw, *range(lens[b], lens[b] + T)])], 1)
        shut = torch.ones(len(live), cores + len(raw) + T, dtype=torch.bool, device=k.device)
        for n, t in enumerate(live):
            shut[n, :lo[t] // g] = False
            shut[n, cores + begin[t] - raw.start:cores + len(raw)] = False
            shut[n, [cores + len(raw) + a for a in up[t]]] = False
        q = s["Q"][b][:, live].to(wide).reshape(Hkv, Hq // Hkv, len(live), d)
        z = torch.einsum("hrnd,hkd->hrnk", q, k) / math.sqrt(d)
        z.masked_fill_(shut, -math.inf)
        lse[b][:, live] = torch.logsumexp(z, -1).reshape(Hq, len(live))
        out[b][:, live] = torch.einsum("hrnk,hkd->hrnd", torch.softmax(z, -1), v).reshape(Hq, len(live), d)
    return out, lse
