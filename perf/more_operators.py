"""Cases of the operators that a Gated DeltaNet hybrid's softmax layers need around tree verification, their plain forms
and their definitions in 64 bits.

* ``attend``: every draft node's softmax attention over its request's context, kept in pages of 8-bit keys and values
  (e4m3) with a scale for each page and head, and over its own ancestors in the draft (a lone token: itself);
* ``append``: the accepted path's keys and values (or a prompt's) into those pages; a page's scale grows where a new token
  needs it to, and the tokens that it holds already are then written anew;
* ``norm``: the residual's addition and the RMS norm in front of a projection, with the normed rows in 8 bits and a scale
  for each row or each group of columns.

``own`` chooses between the plain form (elementary torch operations in 32 bits) and the framework's entry points.
"""
import random

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_E4M3 = torch.float8_e4m3fn
_TOP = 448.0      # the largest e4m3 value
_LEAST = -40      # the least exponent of a page's scale


# ------------------------------------------------------------------ cases

def _attend(name, R, lo, hi, nlo, nhi, tree, Hq, Hkv, d, page, dtype="bf16", out="bf16", pad=0):
    """R requests with lo..hi tokens of context and nlo..nhi draft nodes (a chain, or a tree); ``pad``: elements between
    the token rows of q, k and v beyond their own."""
    c = {"op": "attend", "R": R, "lo": lo, "hi": hi, "nlo": nlo, "nhi": nhi, "tree": tree, "Hq": Hq, "Hkv": Hkv, "d": d,
         "page": page, "dtype": dtype, "out": out, "pad": pad}
    return dict(c, name=name) if name else c


def _append(name, R, lo, hi, nlo, nhi, tree, Hkv, d, page, dtype="bf16", pad=0):
    """R requests with lo..hi tokens in the cache already and nlo..nhi new rows: all of them, or (``tree``) the path to
    an accepted node of theirs."""
    c = {"op": "append", "R": R, "lo": lo, "hi": hi, "nlo": nlo, "nhi": nhi, "tree": tree, "Hkv": Hkv, "d": d,
         "page": page, "dtype": dtype, "pad": pad}
    return dict(c, name=name) if name else c


def _norm(name, T, n, dtype, residual, group, both=False, pad=0):
    """T rows of n; ``group``: columns to a scale of the 8-bit rows (0: all); ``both``: the normed rows in their own type too."""
    c = {"op": "norm", "T": T, "n": n, "dtype": dtype, "residual": residual, "group": group, "both": both, "pad": pad}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one request generating without a draft, a context of a few pages: latency counts
        _attend("one token", 1, 1500, 1500, 1, 1, False, 16, 2, 256, 64),
        # a serving step of 64 requests, ragged contexts
        _attend("64 tokens", 64, 2000, 8000, 1, 1, False, 16, 2, 256, 64),
        # one request with a book in its context
        _attend("one long context", 1, 262144, 262144, 1, 1, False, 16, 2, 256, 64),
        # the chain workload (64 requests, drafts of 4 nodes) on a layer with more key heads and small pages, rows of a
        # fused projection
        _attend("drafts of 4", 64, 1000, 4000, 4, 4, False, 32, 8, 128, 16, pad=256),
        # the wide-tree workload: 256 requests, 16 to 64 nodes
        _attend("wide trees", 256, 500, 4000, 16, 64, True, 16, 2, 256, 64),
        # 32-bit rows, no shared heads, contexts from nothing on, small trees
        _attend("f32, odd sizes", 7, 0, 700, 1, 15, True, 5, 5, 80, 32, dtype="f32", out="f32"),
        # 64 requests' single tokens on their way into the cache: latency counts
        _append("64 tokens appended", 64, 1000, 4000, 1, 1, False, 2, 256, 64),
        # the accepted paths of the wide-tree workload
        _append("accepted paths", 256, 500, 4000, 16, 64, True, 2, 256, 64),
        # a batch of prompts, some continuing inside a page
        _append("prompts appended", 16, 0, 999, 3500, 4096, False, 2, 256, 64, pad=512),
        # in front of a projection in a step of 64 requests of 4 nodes, groups of 128 columns to a scale
        _norm("norm of a draft", 256, 2048, "bf16", "bf16", 128),
        # prompts: a scale for each row
        _norm("norm of prompts", 32768, 4096, "bf16", "bf16", 0),
        # a residual in 32 bits, an odd width, both outputs
        _norm("norm, odd width", 1001, 1000, "bf16", "f32", 128, both=True, pad=24),
    ]


def _log(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return int(min(hi, max(lo, round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(("attend", "attend", "attend", "append", "norm"))
    if op == "norm":
        n = rng.choice((rng.randint(64, 8000), 128 * rng.randint(1, 64)))
        T = _log(rng, 1, 134217728 // n // 2)
        return _norm("", T, n, rng.choice(("bf16", "bf16", "f32")), rng.choice(("bf16", "f32")),
                     rng.choice((0, 32, 64, 128)), rng.random() < 0.4, rng.choice((0, 0, 8, 24)))
    Hkv = rng.choice((1, 2, 4, 5, 8))
    d = rng.choice((64, 128, 128, 256, 256))
    page = rng.choice((16, 32, 64, 128))
    if op == "append":
        pad = rng.choice((0, 8, 128))
        if rng.random() < 0.5:
            hi = _log(rng, 1, 4000)
            return _append("", _log(rng, 1, 200), 0, 5 * page, max(1, hi // 64), max(1, hi // 64), False, Hkv, d, page,
                           rng.choice(("bf16", "bf16", "f32")), pad)
        if rng.random() < 0.5:
            n = rng.randint(2, 64)
            return _append("", _log(rng, 1, 256), 0, _log(rng, 1, 4000), max(1, n // 3), n, True, Hkv, d, page, "bf16", pad)
        hi = _log(rng, 64, 3000)
        return _append("", _log(rng, 1, 12), 0, 3 * page, max(1, hi // rng.randint(1, 6)), hi, False, Hkv, d, page, "bf16", pad)
    G = rng.choice((1, 2, 4, 5, 8, 16))
    kind = rng.choice(("tokens", "tokens", "chains", "trees", "long", "f32"))
    pad = rng.choice((0, 0, 8, 200))
    if kind == "long":
        hi = _log(rng, 5000, 150000)
        return _attend("", rng.randint(1, 3), hi // 2, hi, 1, rng.choice((1, 1, 4)), False, 2 * G, 2, d, page, pad=pad)
    if kind == "f32":
        hi = _log(rng, 1, 1000)
        return _attend("", _log(rng, 1, 12), 0, hi, 1, rng.randint(1, 16), True, Hkv * min(G, 4), Hkv, rng.randint(8, 256),
                       page, rng.choice(("bf16", "f32")), "f32", pad)
    hi = _log(rng, 16, 6000)
    lo = rng.choice((0, hi // 4, hi))
    if kind == "tokens":
        return _attend("", _log(rng, 1, 96), lo, hi, 1, 1, False, Hkv * G, Hkv, d, page, pad=pad)
    if kind == "chains":
        n = rng.randint(2, 8)
        return _attend("", _log(rng, 1, 64), lo, hi, max(1, n // 2), n, False, Hkv * G, Hkv, d, page, pad=pad)
    n = rng.randint(8, 64)
    return _attend("", _log(rng, 1, 48), lo, min(hi, 3000), max(1, n // 4), n, True, 2 * G, 2, d, page, pad=pad)


def _spread(R, lo, hi, salt):
    """R whole numbers: hi once, the others spread evenly and out of order between lo and hi."""
    n = np.array([hi - ((hi - lo) * i) // max(1, R - 1) for i in range(R)], dtype=np.int64)
    return n[np.random.RandomState(1000 * salt + R).permutation(R)]


def _shape(c):
    """The requests' lengths, numbers of rows, parents and accepted nodes: the case's own, whatever the seed."""
    length, n = _spread(c["R"], c["lo"], c["hi"], 1), _spread(c["R"], c["nlo"], c["nhi"], 2)
    r = np.random.RandomState(c["R"] + c["nhi"])
    parent, accepted = [], []
    for m in n:
        depth, p = np.zeros(m, np.int64), np.arange(m) - 1
        for i in range(1, m if c["tree"] else 1):  # a parent among the earlier nodes, up to eight levels
            p[i] = r.choice(np.flatnonzero(depth[:i] < 7))
            depth[i] = depth[p[i]] + 1
        parent.append(p)
        accepted.append(r.randint(-1, m))
    return length, n, parent, np.array(accepted)


def _paths(c):
    """The rows (within its request's) that each request appends, in order."""
    _, n, parent, accepted = _shape(c)
    if not c["tree"]:
        return [list(range(m)) for m in n]
    out = []
    for p, a in zip(parent, accepted):
        path = []
        while a >= 0:
            path.append(int(a))
            a = p[a]
        out.append(path[::-1])
    return out


# ------------------------------------------------------------------ inputs

def _rows(T, heads, d, dtype, pad, make):
    """[T][heads][d] with `pad` elements of something else between the tokens' rows."""
    x = make(T, heads, d).to(dtype)
    if not pad:
        return x
    wide = torch.full((T, heads * d + pad), float("nan"), dtype=dtype, device=x.device)
    wide[:, :heads * d] = x.reshape(T, -1)
    return wide[:, :heads * d].view(T, heads, d)


def _pages(c, length, fresh, g, dev):
    """A pool of pages in random order, its table, and pages filled up to the lengths; behind them whatever was there
    before (other requests' tokens, codes that are no numbers among them)."""
    R, Hkv, d, P = c["R"], c["Hkv"], c["d"], c["page"]
    need = -(-(length + fresh) // P)
    width = max(1, int(need.max()))
    total = int(need.sum())
    num = total + 5
    order = torch.randperm(num, generator=g, device=dev)[:total].to(torch.int32).cpu().numpy()
    table = np.full((R, width), -1, np.int32)
    table[np.arange(width) < need[:, None]] = order
    s = {"table": torch.from_numpy(table).to(dev), "length": torch.from_numpy(length.astype(np.int32)).to(dev)}
    used = torch.zeros(num, dtype=torch.int64, device=dev)  # tokens in each page
    fill = np.clip(length[:, None] - P * np.arange(width), 0, P)
    at = table >= 0
    used[torch.from_numpy(table[at].astype(np.int64)).to(dev)] = torch.from_numpy(fill[at]).to(dev)
    live = (torch.arange(P, device=dev) < used[:, None])[:, None, :, None]
    for name in ("k", "v"):
        # keys have a few channels that are larger than the others, values vary from page to page
        size = 1 + 4 * (torch.rand(Hkv, 1, d, generator=g, device=dev) < 0.03) if name == "k" else 0.5 + torch.rand(num, Hkv, 1, 1, generator=g, device=dev)
        x = torch.randn(num, Hkv, P, d, generator=g, device=dev) * size
        x = torch.where(live, x, torch.zeros((), device=dev))
        scale = _scale_for(x.abs().amax((2, 3)))
        codes = (x / scale[..., None, None]).to(_E4M3)
        junk = torch.randint(0, 256, codes.shape, generator=g, device=dev, dtype=torch.uint8).view(_E4M3)
        s[name + "8"] = torch.where(live, codes.view(torch.uint8), junk.view(torch.uint8)).view(_E4M3)
        s[name + "s"] = scale
    return s


def _scale_for(amax):
    """The least power of two that brings amax within e4m3's range."""
    m, e = torch.frexp(amax)
    e = torch.where(amax > 0, e - 9 + (m > 0.875).int(), torch.full_like(e, _LEAST)).clamp(min=_LEAST)
    return torch.ldexp(torch.ones_like(amax), e)


def _cache(s):
    from gdn_speculative_tree_gb300 import binding
    return binding.make_cache(k=s["k8"], v=s["v8"], k_scale=s["ks"], v_scale=s["vs"], page_table=s["table"],
                              length=s["length"])


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)

    c, s = case, {"case": case}
    if c["op"] == "norm":
        T, n, t = c["T"], c["n"], _TYPES[c["dtype"]]
        s["x"] = _rows(T, 1, n, t, c["pad"], normal)[:, 0]
        s["residual"] = _rows(T, 1, n, _TYPES[c["residual"]], c["pad"], lambda *z: 3 * normal(*z))[:, 0]
        s["w"] = 1 + 0.2 * normal(n)
        s["sum"] = torch.zeros(T, n, device=dev, dtype=_TYPES[c["residual"]])
        s["y"] = torch.zeros(T, n, device=dev, dtype=t) if c["both"] else None
        s["y8"] = torch.zeros(T, n, device=dev, dtype=_E4M3)
        s["y8s"] = torch.zeros(T, -(-n // c["group"]) if c["group"] else 1, device=dev)
        if own:
            from gdn_speculative_tree_gb300 import binding
            s["call"] = binding.make_norm(x=s["x"], residual=s["residual"], residual_out=s["sum"], weight=s["w"], eps=1e-6,
                                          y=s["y"], y8=s["y8"], y8_scale=s["y8s"], group=c["group"])
        return s
    length, n, parent, accepted = _shape(c)
    fresh = np.array([len(p) for p in _paths(c)]) if c["op"] == "append" else 0
    s.update(_pages(c, length, fresh, g, dev))
    off = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    T = int(off[-1])
    s["off"] = torch.from_numpy(off).to(dev)
    s["parent"] = torch.from_numpy(np.concatenate(parent).astype(np.int32)).to(dev) if c["tree"] else None
    t = _TYPES[c["dtype"]]
    s["k"] = _rows(T, c["Hkv"], c["d"], t, c["pad"], lambda *z: 1.2 * normal(*z))
    s["v"] = _rows(T, c["Hkv"], c["d"], t, c["pad"], normal)
    s["status"] = torch.zeros(c["R"], device=dev, dtype=torch.int32)
    if c["op"] == "attend":
        s["q"] = _rows(T, c["Hq"], c["d"], t, c["pad"], lambda *z: 1.5 * normal(*z))
        s["o"] = torch.zeros(T, c["Hq"], c["d"], device=dev, dtype=_TYPES[c["out"]])
        if own:
            from gdn_speculative_tree_gb300 import binding
            s["call"] = binding.make_attn(cache=_cache(s), node_offset=s["off"], parent=s["parent"], q=s["q"], k=s["k"],
                                          v=s["v"], o=s["o"], status=s["status"], scale=_softmax_scale(c),
                                          max_nodes=c["nhi"], max_context=c["hi"])
    else:
        s["accepted"] = torch.from_numpy(accepted.astype(np.int32)).to(dev) if c["tree"] else None
        s["new_length"] = torch.zeros(c["R"], device=dev, dtype=torch.int32)
        if own:
            from gdn_speculative_tree_gb300 import binding
            s["call"] = binding.make_append(cache=_cache(s), node_offset=s["off"], parent=s["parent"],
                                            accepted=s["accepted"], k=s["k"], v=s["v"], new_length=s["new_length"],
                                            status=s["status"], max_new=c["nhi"])
    return s


def _softmax_scale(c):
    return c["d"] ** -0.5


# ------------------------------------------------------------------ one pass

def run(state):
    s, op = state, state["case"]["op"]
    if own:
        from gdn_speculative_tree_gb300 import binding
        {"attend": binding.treewy_attend, "append": binding.treewy_append, "norm": binding.treewy_add_norm}[op](s["call"])
    else:
        {"attend": _plain_attend, "append": _plain_append, "norm": _plain_norm}[op](s)
    if op == "attend":
        return {"o": s["o"], "status": s["status"]}
    if op == "append":
        return {"k": s["k8"], "v": s["v8"], "k_scale": s["ks"], "v_scale": s["vs"], "length": s["new_length"],
                "status": s["status"]}
    return {"sum": s["sum"], "y8": s["y8"], "y8_scale": s["y8s"], "y": s["y"]}


def _at(codes, pages):
    """Pages of codes (8-bit types are indexed as bytes)."""
    return codes.view(torch.uint8)[pages].view(_E4M3)


def _padded(s, N):
    """Row of each request's i-th node ([R][N], some row where it has none), and whether it has one."""
    at = s["off"][:-1, None].long() + torch.arange(N, device=s["off"].device)
    live = at < s["off"][1:, None]
    return at.clamp(max=max(0, s["k"].shape[0] - 1)), live


def _ancestors(s, at, live):
    """[R][N][N]: node j is node i's ancestor, or i itself."""
    N, dev = at.shape[1], at.device
    parent = s["parent"][at].long() if s["parent"] is not None else (torch.arange(N, device=dev) - 1).expand(at.shape)
    step = (parent[:, :, None] == torch.arange(N, device=dev)) & live[:, :, None]
    power = step.float()
    reach, far = torch.eye(N, device=dev) + power, 2
    while far < N:  # (I - step)^-1 = (I + step)(I + step^2)(I + step^4)...
        power = power @ power
        reach = reach + reach @ power
        far *= 2
    return reach > 0


def _plain_attend(s):
    c = s["case"]
    R, Hq, Hkv, d, N = c["R"], c["Hq"], c["Hkv"], c["d"], c["nhi"]
    G = Hq // Hkv
    at, live = _padded(s, N)
    pages = s["table"].long().clamp(min=0)
    L = pages.shape[1] * c["page"]
    inside = torch.arange(L, device=pages.device) < s["length"][:, None]  # [R][L]

    def context(codes, scale):  # [R][Hkv][L][d], zeros behind the context
        x = (_at(codes, pages).float() * scale[pages][..., None, None]).transpose(1, 2).reshape(R, Hkv, L, d)
        return torch.where(inside[:, None, :, None], x, torch.zeros((), device=x.device))

    q = s["q"][at].float().view(R, N, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(R, Hkv, N * G, d)
    k = torch.cat([context(s["k8"], s["ks"]), s["k"][at].float().transpose(1, 2)], 2)
    score = q @ k.mT * _softmax_scale(c)
    seen = torch.cat([inside[:, None].expand(R, N, L), _ancestors(s, at, live)], 2).repeat_interleave(G, 1)
    score = torch.where(seen[:, None], score, torch.full((), -torch.inf, device=q.device))
    p = (score - score.amax(-1, keepdim=True)).exp()
    o = p @ torch.cat([context(s["v8"], s["vs"]), s["v"][at].float().transpose(1, 2)], 2) / p.sum(-1, keepdim=True)
    s["o"].copy_(o.view(R, Hkv, N, G, d).permute(0, 2, 1, 3, 4).reshape(R, N, Hq, d)[live])


def _plain_append(s):
    c = s["case"]
    R, Hkv, d, P, N = c["R"], c["Hkv"], c["d"], c["page"], c["nhi"]
    at, live = _padded(s, N)
    dev = at.device
    length = s["length"].long()
    if c["tree"]:  # the rows on the accepted path
        seen = _ancestors(s, at, live)
        accepted = s["accepted"].long()
        on = seen[torch.arange(R, device=dev), accepted.clamp(min=0)] & (accepted >= 0)[:, None]
    else:
        on = live
    place = length[:, None] + on.long().cumsum(1) - 1        # position of each row that is taken
    first = length // P                                      # the first page written
    M = (N + P - 2) // P + 1                                 # pages that N tokens can touch
    page = first[:, None] + torch.arange(M, device=dev)      # [R][M], within the table
    new = length + on.sum(1)
    touched = (page * P < new[:, None]) & (on.sum(1) > 0)[:, None]
    index = s["table"].long().gather(1, page.clamp(max=s["table"].shape[1] - 1))[touched]  # [n]
    slot = page[..., None] * P + torch.arange(P, device=dev)
    old = (slot < length[:, None, None])[touched][:, None, :, None]
    fresh = ((slot >= length[:, None, None]) & (slot < new[:, None, None]))[touched][:, None, :, None]
    to = (place - first[:, None] * P)[on]
    request = torch.arange(R, device=dev)[:, None].expand(R, N)[on]
    for x, codes, scales in ((s["k"], s["k8"], s["ks"]), (s["v"], s["v8"], s["vs"])):
        rows = torch.zeros(R, M * P, Hkv, d, device=dev)
        rows[request, to] = x[at[on]].float()
        rows = rows.view(R, M, P, Hkv, d)[touched].transpose(1, 2)  # [n][Hkv][P][d]
        before, was = _at(codes, index), scales[index]
        amax = rows.abs().amax((2, 3))
        keeps = old.any(2)[..., 0].expand_as(was)
        scale = torch.where(keeps & (amax <= _TOP * was), was, torch.where(keeps, torch.maximum(was, _scale_for(amax)), _scale_for(amax)))
        values = torch.where(old, before.float() * (was / scale)[..., None, None], rows / scale[..., None, None]).to(_E4M3)
        codes.view(torch.uint8)[index] = torch.where(old | fresh, values.view(torch.uint8), before.view(torch.uint8))
        scales[index] = scale
    s["new_length"].copy_(new)


def _plain_norm(s):
    c = s["case"]
    T, n = c["T"], c["n"]
    z = s["x"].float() + s["residual"].float()
    s["sum"].copy_(z)
    y = z * torch.rsqrt(z.square().mean(-1, keepdim=True) + 1e-6) * s["w"]
    if c["both"]:
        s["y"].copy_(y)
    group = c["group"] or n
    m = -(-n // group)
    grouped = torch.cat([y, torch.zeros(T, m * group - n, device=y.device)], 1).view(T, m, group)
    amax = grouped.abs().amax(-1)
    scale = torch.where(amax > 0, amax / _TOP, torch.ones_like(amax))
    s["y8s"].copy_(scale)
    s["y8"].copy_((grouped / scale[..., None]).view(T, -1)[:, :n].to(_E4M3))


# ------------------------------------------------------------------ the definitions, in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"attend": _exact_attend, "append": _exact_append, "norm": _exact_norm}[case["op"]](case, s)


def _exact_attend(c, s):
    """Request by request and key head by key head."""
    length, n, parent, _ = _shape(c)
    P, G, dev = c["page"], c["Hq"] // c["Hkv"], s["o"].device
    if work(c)["flops"] > 1.5e12:  # about 20 seconds in 64 bits
        return None
    o = torch.zeros(s["o"].shape, device=dev, dtype=torch.float64)
    row = 0
    for r in range(c["R"]):
        L, m = int(length[r]), int(n[r])
        seen = np.zeros((m, m), bool)
        for i in range(m):
            if parent[r][i] >= 0:
                seen[i] = seen[parent[r][i]]
            seen[i, i] = True
        mask = torch.from_numpy(np.repeat(seen, G, axis=0)).to(dev)
        pages = s["table"][r, :-(-L // P)].long()
        kc, vc = (_at(s[x + "8"], pages).double() * s[x + "s"][pages].double()[..., None, None] for x in "kv")
        for h in range(c["Hkv"]):
            q = s["q"][row:row + m, h * G:(h + 1) * G].double().reshape(m * G, -1)
            k = torch.cat([kc[:, h].reshape(-1, c["d"])[:L], s["k"][row:row + m, h].double()])
            v = torch.cat([vc[:, h].reshape(-1, c["d"])[:L], s["v"][row:row + m, h].double()])
            w = torch.einsum("id,jd->ij", q, k) / c["d"] ** 0.5
            w[:, L:][~mask] = -torch.inf
            o[row:row + m, h * G:(h + 1) * G] = (torch.softmax(w, dim=1) @ v).view(m, G, -1)
        row += m
    return {"o": o, "status": None}


def _exact_append(c, s):
    """Page by page; the codes' values before they are rounded."""
    length, n, _, _ = _shape(c)
    P, first = c["page"], np.concatenate([[0], np.cumsum(n)])
    out = {"status": None, "length": s["length"].clone()}
    for x in "kv":
        codes, scales = s[x + "8"].double(), s[x + "s"].double()
        for r, path in enumerate(_paths(c)):
            L, at = int(length[r]), 0
            out["length"][r] = L + len(path)
            while at < len(path):
                i, lo = (L + at) // P, (L + at) % P
                m = min(P - lo, len(path) - at)
                rows = torch.as_tensor(path[at:at + m], device=codes.device) + int(first[r])
                new = s[x][rows].double().transpose(0, 1)  # [Hkv][m][d]
                page = int(s["table"][r, i])
                top = new.abs().amax((1, 2)) / 448
                need = torch.where(top > 0, torch.exp2(torch.ceil(torch.log2(top))), torch.zeros_like(top)).clamp(min=2.0 ** _LEAST)
                scale = torch.maximum(need, scales[page]) if lo else need
                if lo:
                    codes[page, :, :lo] *= (scales[page] / scale)[:, None, None]
                codes[page, :, lo:lo + m] = new / scale[:, None, None]
                scales[page] = scale
                at += m
        out[x], out[x + "_scale"] = codes, scales
    return out


def _exact_norm(c, s):
    T, n = c["T"], c["n"]
    z = s["x"].double() + s["residual"].double()
    rms = torch.sqrt(torch.linalg.vector_norm(z, dim=1) ** 2 / n + 1e-6)
    y = s["w"].double() * z / rms[:, None]
    group = c["group"] or n
    m = -(-n // group)
    scale = torch.stack([y[:, i * group:(i + 1) * group].abs().amax(1) for i in range(m)], 1) / 448
    scale[scale == 0] = 1
    y8 = y / scale.repeat_interleave(group, 1)[:, :n]
    return {"sum": z, "y8": y8, "y8_scale": scale, "y": y if c["both"] else None}


# ------------------------------------------------------------------ the work of one pass

def work(case):
    c = case
    size = {"bf16": 2, "f32": 4}
    if c["op"] == "norm":
        T, n = c["T"], c["n"]
        e = size[c["dtype"]]
        per = e + 2 * size[c["residual"]] + 1 + (e if c["both"] else 0)
        return {"bytes": float(T * n * per + 4 * n + 4 * T * (-(-n // c["group"]) if c["group"] else 1)), "flops": 6.0 * T * n}
    length, n, _, _ = _shape(c)
    Hkv, d, e = c["Hkv"], c["d"], size[c["dtype"]]
    if c["op"] == "append":
        taken = np.array([len(p) for p in _paths(c)])
        pages = (-(-(length + taken) // c["page"]) - length // c["page"])[taken > 0].sum()
        # a new row read and its codes written; the scales of the pages
        return {"bytes": float(taken.sum() * 2 * Hkv * d * (e + 1) + pages * 2 * Hkv * 8 + 4 * n.sum()), "flops": float(2 * taken.sum() * 2 * Hkv * d)}
    # each context read once, and every node's rows; scores and weighted sums over the context and half of the draft
    T = int(n.sum())
    rows = T * d * (c["Hq"] * (e + size[c["out"]]) + 2 * Hkv * e)
    pages = int((-(-length // c["page"])).sum())
    return {"bytes": float(length.sum() * 2 * Hkv * d + rows + pages * (8 * Hkv + 4)),
            "flops": 4.0 * d * c["Hq"] * float((n * (length + (n + 1) / 2)).sum())}


if __name__ == "__main__":
    for case in listed() + [draw(random.Random(i)) for i in range(12)]:
        print(case, work(case))
