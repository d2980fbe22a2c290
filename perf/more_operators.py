"""Cases of the operators of packed sequences: norms of queries and keys with their rotation, pooling and attention of
sequences of different lengths laid one behind the other, and their gradients.  A plain form in elementary torch
operations and a 64-bit definition stand beside the framework's calls.

Packed tensors are [heads, T, d]; sequence s holds the rows cu[s] .. cu[s+1] - 1.  The core tokens of sequence s, one for
each of its whole groups of g, are the rows cu[s] // g .. of [Hkv, T // g, d].
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ---------------------------------------------------------------- the cases

def _norm(name, **kw):
    c = dict(op="norm", B=1, N=1024, Hq=8, Hkv=8, d=128, rot=128, layout="half", dtype="bf16", base=10000.0, factor=1.0,
             given=False, grad=False, per_head=False, wide_weight=False, offset=0.0)
    return {**({"name": name} if name else {}), **c, **kw}


def _append(name, **kw):
    c = dict(op="append", B=1, T=1, Hq=32, Hkv=8, d=128, rot=128, layout="half", dtype="bf16", base=10000.0, factor=1.0,
             ctx=8192, rows=64, per_head=False, wide_weight=False, offset=0.0)
    return {**({"name": name} if name else {}), **c, **kw}


def _pool(name, **kw):
    c = dict(op="pool", S=4, T=4096, spread=1.0, empty=False, Hq=32, Hkv=8, d=128, dtype="bf16", g=16)
    return {**({"name": name} if name else {}), **c, **kw}


def _attn(name, **kw):
    c = dict(op="attn", S=4, T=4096, spread=1.0, empty=False, Hq=32, Hkv=8, d=128, dtype="bf16", g=16, w=1024, aligned=False)
    return {**({"name": name} if name else {}), **c, **kw}


def _train(name, **kw):
    return _attn(name, op="train", **kw)


def listed():
    return [
        # a 32 K prompt's queries and keys of a grouped-query layer, straight from the projections
        _norm("norm-prompt", N=32768, Hq=32, Hkv=8, base=500000.0),
        # a training step: positions of packed documents, gradients of the inputs and of the norms' weights
        _norm("norm-train", B=2, N=4099, Hq=16, Hkv=4, given=True, grad=True),
        # plain decoding of a serving batch: one token of each sequence, normed, rotated and stored into its page
        _append("append-one", B=64, T=1),
        # drafted tokens of a serving step, pairs interleaved, a norm for each head
        _append("append-drafts", B=8, T=24, ctx=32768, layout="interleaved", per_head=True, wide_weight=True),
        # the groups of a server's packed prompts
        _pool("pool-prompts", S=12, T=32768),
        # many short fp32 sequences with small groups, one of them empty
        _pool("pool-short", S=64, T=2501, Hq=4, Hkv=2, d=64, dtype="f32", g=8, empty=True),
        # a server's packed prompts, core tokens and window
        _attn("attn-prompts", S=12, T=32768),
        # short prompts in one go, every earlier token seen: latency
        _attn("attn-short", S=32, T=1501, w=None),
        # few long documents, most of their keys core tokens
        _attn("attn-long", S=3, T=65536, spread=0.5),
        # the fp32 path: small heads, the group-aligned window, an empty sequence
        _attn("attn-f32", S=5, T=1500, Hq=4, Hkv=2, d=64, dtype="f32", g=8, w=100, aligned=True, empty=True),
        # a training step over packed documents, every earlier token seen
        _train("train-causal", S=6, T=8192, Hq=16, Hkv=4, w=None),
        # the same with core tokens and window, pooled from the step's own keys and values
        _train("train-cores", S=5, T=16384, Hq=32, Hkv=8, spread=0.7),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "append", "pool", "attn", "attn", "train", "train"])
    d = rng.choice([64, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 8])
    norm = dict(d=d, dtype=dtype, Hq=Hq, Hkv=Hkv, rot=rng.choice([d, d, d // 2, d // 4, 24, 0]),
                layout=rng.choice(["half", "interleaved"]), base=rng.choice([10000.0, 500000.0]),
                factor=rng.choice([1.0, 1.25]), per_head=rng.random() < 0.25, wide_weight=rng.random() < 0.5,
                offset=rng.choice([0.0, 1.0]))
    if op == "norm":
        return _norm(None, B=rng.randint(1, 3), N=_log(rng, 1, 8192), given=rng.random() < 0.5, grad=rng.random() < 0.6, **norm)
    if op == "append":
        return _append(None, B=_log(rng, 1, 64), T=_log(rng, 1, 64), ctx=_log(rng, 64, 32768),
                       rows=rng.choice([16, 32, 48, 64, 128]), **norm)
    f32 = dtype == "f32"
    T = _log(rng, 1, {"pool": 32768, "attn": 4096 if f32 else 16384, "train": 2048 if f32 else 8192}[op])
    packed = dict(d=d, dtype=dtype, Hq=Hq, Hkv=Hkv, T=T, S=min(T, _log(rng, 1, 64)), spread=rng.choice([0.0, 1.0, 2.0]),
                  empty=rng.random() < 0.3, g=rng.choice([1, 4, 8, 16, 32, 40]))
    if op == "pool":
        packed["T"] = max(T, packed["S"] * packed["g"])   # one whole group at least
        return _pool(None, **packed)
    c = _attn(None, op=op, w=rng.choice([None, 1, 48, 100, 256, 512, 1024]), aligned=rng.random() < 0.3, **packed)
    while work(c)["flops"] > 1.5e12:
        c["T"] //= 2
        c["S"] = min(c["S"], c["T"])
    return c


def _lengths(c):
    """The lengths of a case's sequences: T in all, one at least each, and a last one of none where the case has it."""
    rng = random.Random(c["S"] * 7919 + c["T"])
    share = [math.exp(c["spread"] * rng.gauss(0.0, 1.0)) for _ in range(c["S"])]
    left, out = c["T"] - c["S"], []
    for k, x in enumerate(share):
        n = left if k == c["S"] - 1 else int(left * x / sum(share[k:]))
        out.append(1 + n)
        left -= n
    return out + ([0] if c["empty"] else [])


# ---------------------------------------------------------------- the inputs

class _Inputs:
    def __init__(self, case, seed):
        self.dev = torch.device("cuda")
        self.gen = torch.Generator(device=self.dev)
        self.gen.manual_seed(seed)
        self.dt = DT[case["dtype"]]

    def normal(self, *shape):
        return torch.randn(shape, generator=self.gen, device=self.dev).to(self.dt)

    def activations(self, *shape):
        """Rows of a projection: sizes that differ from row to row, and a few large columns."""
        size = 0.5 + 2.0 * torch.rand(shape[:-1] + (1,), generator=self.gen, device=self.dev)
        column = 1.0 + 5.0 * (torch.rand(shape[-1], generator=self.gen, device=self.dev) < 0.03)
        return (torch.randn(shape, generator=self.gen, device=self.dev) * size * column).to(self.dt)

    def uniform(self, *shape):
        return torch.rand(shape, generator=self.gen, device=self.dev)

    def integers(self, lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=self.gen, device=self.dev, dtype=torch.int32)


def _ceil(a, b):
    return -(-a // b)


def _prepare_norm(c, x, s):
    d, dev = c["d"], x.dev
    i = torch.arange(c["rot"] // 2, dtype=torch.float64, device=dev)
    s["freq"] = c["base"] ** (-2.0 * i / max(c["rot"], 1))
    wt = torch.float32 if c["wide_weight"] else x.dt
    shape = lambda h: (h, d) if c["per_head"] else (d,)  # noqa: E731
    s["qw"] = (1.0 - c["offset"] + 0.2 * torch.randn(shape(c["Hq"]), generator=x.gen, device=dev)).to(wt)
    s["kw"] = (1.0 - c["offset"] + 0.2 * torch.randn(shape(c["Hkv"]), generator=x.gen, device=dev)).to(wt)
    if c["op"] == "norm":
        B, N = c["B"], c["N"]
        # the projections' layout [B, N, H, d]; the operator reads it as [B, H, N, d]
        s["Q"] = x.activations(B, N, c["Hq"], d).transpose(1, 2)
        s["K"] = x.activations(B, N, c["Hkv"], d).transpose(1, 2)
        s["positions"] = None
        if c["given"]:
            cut = 1 + (x.uniform(B, 1) * N).floor().to(torch.int32)
            n = torch.arange(N, device=dev, dtype=torch.int32)
            s["positions"] = torch.where(n < cut, n, n - cut).contiguous()
        if c["grad"]:
            s["dQ"], s["dK"] = x.normal(B, c["Hq"], N, d), x.normal(B, c["Hkv"], N, d)
            for name in ("Q", "K", "qw", "kw"):
                s[name] = s[name].requires_grad_()
        return s
    B, T, P = c["B"], c["T"], c["rows"]
    s["Q"] = x.activations(B, T, c["Hq"], d).transpose(1, 2)
    s["K"] = x.activations(B, T, c["Hkv"], d).transpose(1, 2)
    s["V"] = x.normal(B, T, c["Hkv"], d).transpose(1, 2)
    s["lens"] = x.integers(c["ctx"] // 2, c["ctx"] + 1, B)
    # pages for the new tokens alone (what lies before them is not touched), in random order
    cols, most = _ceil(c["ctx"] + T, P), _ceil(T, P) + 1
    col = torch.arange(cols, device=dev)
    held = (col >= (s["lens"] // P)[:, None]) & (col < _ceil(s["lens"] + T, P)[:, None])
    n = B * most + 2
    order = torch.randperm(n, generator=x.gen, device=dev).to(torch.int32)
    rank = torch.cumsum(held.flatten().to(torch.int64), 0).reshape(held.shape) - 1
    s["table"] = torch.where(held, order[rank.clamp(min=0)], torch.full_like(order[:1], -1))
    s["Kp"], s["Vp"] = x.normal(n, c["Hkv"], P, d), x.normal(n, c["Hkv"], P, d)
    return s


def _window(c):
    return c["w"] if c["w"] is not None else c["T"]


def prepare(case, seed):
    c, x = case, _Inputs(case, seed)
    s = {"case": c}
    if c["op"] in ("norm", "append"):
        return _prepare_norm(c, x, s)
    lens = _lengths(c)
    random.Random(seed).shuffle(lens)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    s["cu"], T, d, G = cu, c["T"], c["d"], c["T"] // c["g"]
    s["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device=x.dev)
    # queries, keys and values as they come out of the projections and norms: token by token, read as [H, T, d]
    s["Q"] = x.normal(T, c["Hq"], d).transpose(0, 1)
    s["K"] = x.normal(T, c["Hkv"], d).transpose(0, 1)
    s["V"] = x.normal(T, c["Hkv"], d).transpose(0, 1)
    if c["op"] == "pool":
        s["Kc"] = torch.zeros(c["Hkv"], G, d, dtype=x.dt, device=x.dev)
        s["Vc"] = torch.zeros_like(s["Kc"])
    if c["op"] == "attn":
        s["Kc"] = (x.normal(c["Hkv"], G, d) * 0.5).to(x.dt)
        s["Vc"] = (x.normal(c["Hkv"], G, d) * 0.3).to(x.dt)
    if c["op"] == "train":
        s["dO"] = x.normal(c["Hq"], T, d)
        for name in ("Q", "K", "V"):
            s[name] = s[name].requires_grad_()
    if own and c["op"] != "train":
        # the layout of the batch: a program makes it once for all its layers
        from sparse_long_context_cca_gb300 import api
        s["packed"] = api.cca_pack(s["cu_seqlens"], T, c["g"], c.get("w"), window_mode=int(c.get("aligned", False)))
    return s


# ---------------------------------------------------------------- the plain forms

def _turn(x, pos, freq, layout, factor):
    """x [B, H, N, d] (fp32) with its first 2 * len(freq) columns rotated by pos [B, N] * freq."""
    r = freq.numel()
    ang = pos[:, None, :, None].to(torch.float64) * freq
    c, s = (ang.cos() * factor).float(), (ang.sin() * factor).float()
    a, b = (x[..., :r], x[..., r:2 * r]) if layout == "half" else (x[..., 0:2 * r:2], x[..., 1:2 * r:2])
    u, v = a * c - b * s, b * c + a * s
    y = torch.cat([u, v], -1) if layout == "half" else torch.stack([u, v], -1).flatten(-2)
    return torch.cat([y, x[..., 2 * r:]], -1)


def _normed(x, w, offset):
    """x [B, H, N, d] (fp32) over its rows' root mean square, times (offset + w), w [d] or [H, d]."""
    w = w + offset if w.dim() == 1 else (w + offset)[:, None]
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w


def _plain_norm(s):
    c = s["case"]
    B, N = c["B"], c["N"]
    pos = s["positions"] if c["given"] else torch.arange(N, device=s["Q"].device).expand(B, N)
    wide = [s[k].detach().float() for k in ("Q", "K", "qw", "kw")]
    if c["grad"]:
        wide = [x.requires_grad_() for x in wide]
    q = _turn(_normed(wide[0], wide[2], c["offset"]), pos, s["freq"], c["layout"], c["factor"])
    k = _turn(_normed(wide[1], wide[3], c["offset"]), pos, s["freq"], c["layout"], c["factor"])
    out = [q.detach().to(s["Q"].dtype), k.detach().to(s["K"].dtype)]
    if c["grad"]:
        grads = torch.autograd.grad([q, k], wide, [s["dQ"].float(), s["dK"].float()])
        out += [g.to(s[n].dtype) for g, n in zip(grads, ("Q", "K", "qw", "kw"))]
    return out


def _store(pool, table, idx, rows):
    """Writes rows [B, Hkv, n, d] at idx [B, n]."""
    P = pool.shape[-2]
    pool[table.gather(1, idx // P).long(), :, idx % P] = rows.transpose(1, 2).to(pool.dtype)


def _plain_append(s):
    c = s["case"]
    slot = s["lens"][:, None].long() + torch.arange(c["T"], device=s["lens"].device)
    q = _turn(_normed(s["Q"].float(), s["qw"].float(), c["offset"]), slot, s["freq"], c["layout"], c["factor"])
    k = _turn(_normed(s["K"].float(), s["kw"].float(), c["offset"]), slot, s["freq"], c["layout"], c["factor"])
    _store(s["Kp"], s["table"], slot, k)
    _store(s["Vp"], s["table"], slot, s["V"])
    return {"Q": q.to(s["Q"].dtype), "Kp": s["Kp"], "Vp": s["Vp"]}


def _plain_cores(c, q, k, v):
    """Core keys and values [Hkv, n // g, d] of one sequence, fp32."""
    g, d, Hkv = c["g"], c["d"], c["Hkv"]
    n = k.shape[1] // g
    kg, vg = k[:, :n * g].reshape(Hkv, n, g, d), v[:, :n * g].reshape(Hkv, n, g, d)
    ql = q[:, g - 1:n * g:g].reshape(Hkv, -1, n, d).mean(1)
    z = (kg * ql[:, :, None]).sum(-1) * d ** -0.5
    a = (z - z.amax(-1, keepdim=True)).exp()
    a = (a / a.sum(-1, keepdim=True))[..., None]
    return (a * kg).sum(2), (a * vg).sum(2)


def _plain_attention(c, q, k, v, kc, vc):
    """O [Hq, n, d] and LSE [Hq, n] of one sequence, fp32, a block of rows at a time."""
    Hq, n, d = q.shape
    Hkv, g, w = c["Hkv"], c["g"], _window(c)
    step = max(16, min(n, (1 << 27) // (Hq * min(n, 1 << 14))))
    O, L = [], []
    for a in range(0, n, step):
        b = min(a + step, n)
        low = max(0, a - w + 1)
        low = low // g * g if c["aligned"] else low
        m = max(0, b - w) // g
        keys = torch.cat([kc[:, :m], k[:, low:b]], 1)
        vals = torch.cat([vc[:, :m], v[:, low:b]], 1)
        i = torch.arange(a, b, device=q.device)[:, None]
        lo = (i - w + 1).clamp(min=0)
        start = lo // g * g if c["aligned"] else lo
        t = torch.arange(low, b, device=q.device)
        sees = torch.cat([torch.arange(m, device=q.device) < lo // g, (t >= start) & (t <= i)], 1)
        z = (q[:, a:b].reshape(Hkv, Hq // Hkv, b - a, d) @ keys[:, None].transpose(-1, -2)) * d ** -0.5
        z = z.masked_fill(~sees, -math.inf)
        top = z.amax(-1, keepdim=True).detach()
        p = (z - top).exp()
        total = p.sum(-1, keepdim=True)
        O.append(((p @ vals[:, None]) / total).reshape(Hq, b - a, d))
        L.append((top + total.log()).reshape(Hq, b - a))
    return torch.cat(O, 1), torch.cat(L, 1)


def _spans(s):
    return [(a, b) for a, b in zip(s["cu"], s["cu"][1:]) if b > a]


def _plain_pool(s):
    c = s["case"]
    for a, b in _spans(s):
        if b - a >= c["g"]:
            kc, vc = _plain_cores(c, *(s[x][:, a:b].float() for x in "QKV"))
            at = a // c["g"]
            s["Kc"][:, at:at + kc.shape[1]] = kc.to(s["Kc"].dtype)
            s["Vc"][:, at:at + vc.shape[1]] = vc.to(s["Vc"].dtype)
    return {"Kc": s["Kc"], "Vc": s["Vc"]}


def _plain_attn(s):
    c, g = s["case"], s["case"]["g"]
    O = torch.empty(s["Q"].shape, dtype=s["Q"].dtype, device=s["Q"].device)
    L = torch.empty(O.shape[:2], dtype=torch.float32, device=O.device)
    for a, b in _spans(s):
        core = slice(a // g, a // g + (b - a) // g)
        o, lse = _plain_attention(c, *(s[x][:, a:b].float() for x in "QKV"), s["Kc"][:, core].float(), s["Vc"][:, core].float())
        O[:, a:b], L[:, a:b] = o.to(O.dtype), lse
    return {"O": O, "LSE": L}


def _plain_train(s):
    c = s["case"]
    with torch.no_grad():
        out = {n: torch.empty(s[x].shape, dtype=s[x].dtype, device=s[x].device)
               for n, x in (("O", "Q"), ("dQ", "Q"), ("dK", "K"), ("dV", "V"))}
    for a, b in _spans(s):
        q, k, v = (s[x][:, a:b].detach().float().requires_grad_() for x in "QKV")
        kc, vc = _plain_cores(c, q, k, v) if b - a > _window(c) else (k[:, :0], v[:, :0])
        o, _ = _plain_attention(c, q, k, v, kc, vc)
        grads = torch.autograd.grad(o, (q, k, v), s["dO"][:, a:b].float())
        for name, x in zip(("O", "dQ", "dK", "dV"), (o.detach(), *grads)):
            out[name][:, a:b] = x.to(out[name].dtype)
    return out


_PLAIN = {"norm": _plain_norm, "append": _plain_append, "pool": _plain_pool, "attn": _plain_attn, "train": _plain_train}


# ---------------------------------------------------------------- the framework's calls

def _framework(s):
    from sparse_long_context_cca_gb300 import api
    c, op = s["case"], s["case"]["op"]
    if op in ("norm", "append"):
        turn = dict(layout=c["layout"], factor=c["factor"], eps=EPS, offset=c["offset"])
        freq = s["freq"] if c["rot"] else None
    if op == "norm":
        if not c["grad"]:
            return list(api.cca_norm_rope(s["Q"], s["K"], s["qw"], s["kw"], freq, positions=s["positions"], **turn))
        q, k = api.norm_rope(s["Q"], s["K"], s["qw"], s["kw"], freq, positions=s["positions"], **turn)
        return [q.detach(), k.detach(), *torch.autograd.grad([q, k], [s["Q"], s["K"], s["qw"], s["kw"]], [s["dQ"], s["dK"]])]
    if op == "append":
        q = api.cca_norm_rope_append(s["Q"], s["K"], s["V"], s["Kp"], s["Vp"], s["table"], s["lens"], s["qw"], s["kw"], freq, **turn)
        return {"Q": q, "Kp": s["Kp"], "Vp": s["Vp"]}
    if op == "pool":
        api.cca_pool_packed(s["Q"], s["K"], s["V"], s["packed"], Kc=s["Kc"], Vc=s["Vc"])
        return {"Kc": s["Kc"], "Vc": s["Vc"]}
    if op == "attn":
        O, L = api.cca_attn_packed(s["Q"], s["K"], s["V"], s["Kc"], s["Vc"], s["packed"])
        return {"O": O, "LSE": L}
    packed = api.cca_pack(s["cu_seqlens"], c["T"], c["g"], c["w"], window_mode=int(c["aligned"]))
    O = api.cca_attention_packed(s["Q"], s["K"], s["V"], packed)
    dQ, dK, dV = torch.autograd.grad(O, (s["Q"], s["K"], s["V"]), s["dO"])
    return {"O": O.detach(), "dQ": dQ, "dK": dK, "dV": dV}


def run(state):
    return _framework(state) if own else _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without

def _seen(c):
    """(pairs of a query and a key that it sees, core tokens among those keys, for one head)."""
    w, g, pairs = _window(c), c["g"], 0
    cores = 0
    for n in _lengths(c):
        for a in range(0, n, 4096):
            i = torch.arange(a, min(a + 4096, n), dtype=torch.int64)
            lo = (i - w + 1).clamp(min=0)
            pairs += int((i - (lo // g * g if c["aligned"] else lo) + 1 + lo // g).sum())
        cores += max(0, n - w) // g
    return pairs, cores


def work(case):
    c, op = case, case["op"]
    e, d = (2 if c["dtype"] == "bf16" else 4), c["d"]
    if op == "norm":
        n = c["B"] * c["N"] * (c["Hq"] + c["Hkv"]) * (2 if c["grad"] else 1)
        return {"bytes": 2.0 * n * d * e, "flops": n * (4.0 * d + 3.0 * c["rot"])}
    if op == "append":
        n = c["B"] * c["T"] * (c["Hq"] + 2 * c["Hkv"])
        return {"bytes": 2.0 * n * d * e, "flops": c["B"] * c["T"] * (c["Hq"] + c["Hkv"]) * (4.0 * d + 3.0 * c["rot"])}
    if op == "pool":
        groups = sum(n // c["g"] for n in _lengths(c))
        return {"bytes": groups * (c["Hkv"] * (2.0 * c["g"] + 2.0) + c["Hq"]) * d * e,
                "flops": groups * c["Hkv"] * c["g"] * d * 6.0}
    pairs, cores = _seen(c)
    rows = c["T"] * d * e
    if op == "attn":
        return {"bytes": rows * (2.0 * c["Hq"] + 2.0 * c["Hkv"]) + 4.0 * c["T"] * c["Hq"] + 2.0 * cores * c["Hkv"] * d * e,
                "flops": 4.0 * d * pairs * c["Hq"]}
    return {"bytes": rows * (4.0 * c["Hq"] + 4.0 * c["Hkv"]), "flops": 14.0 * d * pairs * c["Hq"]}


# ---------------------------------------------------------------- the definition in 64 bits

def _complex_turn(c, freq, y, pos, sign):
    """The pairs of y [B, H, N, d] as complex numbers, times factor * exp(i * sign * pos * freq)."""
    n = c["rot"] // 2
    half = c["layout"] == "half"
    first = list(range(n)) if half else list(range(0, 2 * n, 2))
    second = list(range(n, 2 * n)) if half else list(range(1, 2 * n, 2))
    y = y.clone()
    z = torch.complex(y[..., first], y[..., second])
    ang = (pos.to(torch.float64)[:, :, None] * freq)[:, None]
    z = z * torch.polar(torch.full_like(ang, c["factor"]), sign * ang)
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_norm(c, s):
    wide = torch.float64
    if c["op"] == "norm":
        pos = s["positions"] if c["given"] else torch.arange(c["N"], device=s["Q"].device).expand(c["B"], -1)
    else:
        pos = s["lens"][:, None] + torch.arange(c["T"], device=s["lens"].device)
    fwd, dx, dw = [], [], []
    for x, w, dy in (("Q", "qw", "dQ"), ("K", "kw", "dK")):
        X, W = s[x].detach().to(wide), s[w].detach().to(wide) + c["offset"]
        W = W.expand(X.shape[1], -1)[None, :, None]
        hat = X / torch.sqrt(torch.square(X).sum(-1, keepdim=True) / c["d"] + EPS)
        fwd.append(_complex_turn(c, s["freq"], hat * W, pos, 1.0))
        if c.get("grad"):
            dn = _complex_turn(c, s["freq"], s[dy].to(wide), pos, -1.0)
            # d hat / d x = (I - hat hat^T / d) / rms
            rms = torch.sqrt(torch.square(X).sum(-1, keepdim=True) / c["d"] + EPS)
            dx.append((dn * W - hat * ((dn * W * hat).sum(-1, keepdim=True) / c["d"])) / rms)
            dw.append((dn * hat).sum((0, 2)) if c["per_head"] else (dn * hat).sum((0, 1, 2)))
    if c["op"] == "norm":
        return fwd + dx + dw
    P, table, lens = c["rows"], s["table"].tolist(), s["lens"].tolist()
    Kp, Vp = s["Kp"].to(wide), s["Vp"].to(wide)
    for b in range(c["B"]):
        for t in range(c["T"]):
            at = lens[b] + t
            Kp[table[b][at // P], :, at % P] = fwd[1][b, :, t]
            Vp[table[b][at // P], :, at % P] = s["V"][b, :, t].to(wide)
    return {"Q": fwd[0], "Kp": Kp, "Vp": Vp}


def _exact_cores(c, q, k):
    """The group weights [Hkv, n // g, g] of one sequence."""
    g, n = c["g"], k.shape[1] // c["g"]
    last = q[:, [j * g + g - 1 for j in range(n)]].unflatten(0, (c["Hkv"], -1)).sum(1) / (c["Hq"] // c["Hkv"])
    return torch.softmax(torch.einsum("hjd,hjtd->hjt", last, k[:, :n * g].unflatten(1, (n, g))) / math.sqrt(c["d"]), -1)


def _visible(c, a, b, n, dev):
    """Rows a .. b - 1 against the sequence's n // g core tokens and its first b tokens: who sees what."""
    i = torch.arange(a, b, device=dev)[:, None]
    first = torch.relu(i - (_window(c) - 1))
    begin = first - first % c["g"] if c["aligned"] else first
    j, t = torch.arange(n // c["g"], device=dev), torch.arange(b, device=dev)
    return torch.cat([(j + 1) * c["g"] <= first, (begin <= t) & (t <= i)], 1)


def _exact_sequence(c, q, k, v, kc, vc, dO):
    """One sequence in 64 bits, a block of rows at a time, every core token and token before the block's end looked at:
    O, LSE and, with dO, the gradients of q, k, v, kc and vc."""
    n, r, tau = q.shape[1], c["Hq"] // c["Hkv"], 1.0 / math.sqrt(c["d"])
    G = kc.shape[1]
    keys, vals = torch.cat([kc, k], 1).repeat_interleave(r, 0), torch.cat([vc, v], 1).repeat_interleave(r, 0)
    O, L = torch.empty_like(q), q.new_empty(q.shape[:2])
    dq, dk, dv = (torch.zeros_like(x) for x in (q, keys, vals)) if dO is not None else (None,) * 3
    step = max(1, (1 << 26) // (c["Hq"] * (G + n)))
    for a in range(0, n, step):
        b = min(a + step, n)
        ks, vs = keys[:, :G + b], vals[:, :G + b]
        z = torch.einsum("hid,hmd->him", q[:, a:b], ks) * tau
        z = torch.where(_visible(c, a, b, n, q.device), z, torch.full_like(z, -math.inf))
        L[:, a:b] = torch.logsumexp(z, -1)
        p = torch.exp(z - L[:, a:b, None])
        O[:, a:b] = torch.einsum("him,hmd->hid", p, vs)
        if dO is not None:
            dp = torch.einsum("hid,hmd->him", dO[:, a:b], vs)
            ds = p * (dp - (dO[:, a:b] * O[:, a:b]).sum(-1, keepdim=True)) * tau
            dq[:, a:b] = torch.einsum("him,hmd->hid", ds, ks)
            dk[:, :G + b] += torch.einsum("him,hid->hmd", ds, q[:, a:b])
            dv[:, :G + b] += torch.einsum("him,hid->hmd", p, dO[:, a:b])
    if dO is None:
        return O, L
    dk, dv = dk.unflatten(0, (-1, r)).sum(1), dv.unflatten(0, (-1, r)).sum(1)
    return O, L, dq, dk[:, G:], dv[:, G:], dk[:, :G], dv[:, :G]


def exact(case, seed):
    c, op = case, case["op"]
    if op in ("attn", "train"):
        cost = sum(float(n) * (n // c["g"] + n) for n in _lengths(c)) * c["Hq"] * c["d"] * (4.0 if op == "attn" else 10.0)
        if cost > 8e12:   # all keys are looked at: some seconds
            return None
    s = prepare(c, seed)
    if op in ("norm", "append"):
        return _exact_norm(c, s)
    wide, g = torch.float64, c["g"]
    if op == "pool":
        out = {"Kc": s["Kc"].to(wide), "Vc": s["Vc"].to(wide)}
    elif op == "attn":
        out = {"O": torch.empty(s["Q"].shape, dtype=wide, device=s["Q"].device)}
        out["LSE"] = torch.empty(out["O"].shape[:2], dtype=wide, device=s["Q"].device)
    else:
        out = {n: torch.empty(s[x].shape, dtype=wide, device=s["Q"].device) for n, x in (("O", "Q"), ("dQ", "Q"), ("dK", "K"), ("dV", "V"))}
    for a, b in _spans(s):
        q, k, v = (s[x][:, a:b].detach().to(wide) for x in "QKV")
        n = (b - a) // g
        core = slice(a // g, a // g + n)
        if op == "attn":
            out["O"][:, a:b], out["LSE"][:, a:b] = _exact_sequence(c, q, k, v, s["Kc"][:, core].to(wide), s["Vc"][:, core].to(wide), None)
            continue
        alpha = _exact_cores(c, q, k)
        kg, vg = k[:, :n * g].unflatten(1, (n, g)), v[:, :n * g].unflatten(1, (n, g))
        kc, vc = torch.einsum("hjt,hjtd->hjd", alpha, kg), torch.einsum("hjt,hjtd->hjd", alpha, vg)
        if op == "pool":
            out["Kc"][:, core], out["Vc"][:, core] = kc, vc
            continue
        O, _, dq, dk, dv, dkc, dvc = _exact_sequence(c, q, k, v, kc, vc, s["dO"][:, a:b].to(wide))
        # back through the groups: the values' weights, then the softmax that made them
        da = torch.einsum("hjd,hjtd->hjt", dkc, kg) + torch.einsum("hjd,hjtd->hjt", dvc, vg)
        ds = alpha * (da - (alpha * da).sum(-1, keepdim=True)) / (math.sqrt(c["d"]) * (c["Hq"] // c["Hkv"]))
        last = torch.arange(n, device=q.device) * g + g - 1
        qsum = q[:, last].unflatten(0, (c["Hkv"], -1)).sum(1)
        dk[:, :n * g] += (alpha[..., None] * dkc[:, :, None] + ds[..., None] * qsum[:, :, None]).flatten(1, 2)
        dv[:, :n * g] += (alpha[..., None] * dvc[:, :, None]).flatten(1, 2)
        dq[:, last] += torch.einsum("hjt,hjtd->hjd", ds, kg).repeat_interleave(c["Hq"] // c["Hkv"], 0)
        out["O"][:, a:b], out["dQ"][:, a:b], out["dK"][:, a:b], out["dV"][:, a:b] = O, dq, dk, dv
    return out
