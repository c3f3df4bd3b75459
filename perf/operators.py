"""Cases of the serving operators around tree verification, their plain forms and their definitions in 64 bits.

Three operators of a Gated DeltaNet server, as a request meets them:

* ``extend``: the gated delta rule over a sequence's new tokens, from and into the state pool (a prompt, a
  chunk of one, or a single token):  S_t = a_t S_{t-1} (I - b_t k_t k_t^T) + b_t v_t k_t^T,  o_t = S_t q_t;
* ``qk``: the norm of every query and key head (L2, or RMS with a weight) with the position rotation, and
  with each head repeated where the heads are shared;
* ``slots``: copying, forking, compacting and clearing slots of the state pools of all layers.

``own`` chooses between the plain form (elementary torch operations in 32 bits) and the framework's entry points.
"""
import random

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_CHUNK = 64  # tokens of one step of extend's plain form
_HEADS = (1, 2, 3, 4, 5, 7, 8, 16, 20, 32)


# ------------------------------------------------------------------ cases

def _extend(name, R, lo, hi, H, Hk, dk, dv, qkv, out, pool, gate=0.9, fresh=0.0, pad=0):
    """R sequences of lo to hi new tokens; ``gate``: the least decay; ``fresh``: the share that starts from a
    zero state; ``pad``: elements between the token rows of q, k and v beyond their own."""
    c = {"op": "extend", "R": R, "lo": lo, "hi": hi, "H": H, "Hk": Hk, "dk": dk, "dv": dv, "qkv": qkv,
         "out": out, "pool": pool, "gate": gate, "fresh": fresh, "pad": pad}
    return dict(c, name=name) if name else c


def _qk(name, T, Hq, Hk, d, dtype, norm, rope=0, interleaved=False, repeat=1, pad=0):
    c = {"op": "qk", "T": T, "Hq": Hq, "Hk": Hk, "d": d, "dtype": dtype, "norm": norm, "rope": rope,
         "interleaved": interleaved, "repeat": repeat, "pad": pad}
    return dict(c, name=name) if name else c


def _slots(name, layers, num_slots, moves, sources, cleared, H, dk, dv, pool):
    """``moves`` slots written from ``sources`` others (fewer sources than moves: forks), ``cleared`` more zeroed."""
    c = {"op": "slots", "layers": layers, "num_slots": num_slots, "moves": moves, "sources": sources,
         "cleared": cleared, "H": H, "dk": dk, "dv": dv, "pool": pool}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one request generating without a draft: one token, latency counts
        _extend("one token", 1, 1, 1, 32, 32, 128, 128, "bf16", "bf16", "f32"),
        # a serving step of 64 requests on a bf16 pool, keys shared by two value heads
        _extend("64 tokens, bf16 pool", 64, 1, 1, 32, 16, 128, 128, "bf16", "bf16", "bf16"),
        # the wide-tree batch (256 requests) in a round without a draft
        _extend("256 tokens", 256, 1, 1, 32, 16, 128, 128, "bf16", "bf16", "f32"),
        # one long prompt: 32 heads, a chain of chunks each
        _extend("one prompt", 1, 4096, 4096, 32, 16, 128, 128, "bf16", "bf16", "f32", fresh=1.0),
        # ragged chunks of prompts joining a batch, odd lengths, some requests continuing, rows of a fused projection
        _extend("ragged prompts, bf16 pool", 13, 1, 2500, 32, 32, 128, 128, "bf16", "bf16", "bf16", gate=0.8,
                fresh=0.5, pad=256),
        # a full batch of prompts: the largest
        _extend("batch of prompts", 16, 4000, 4096, 32, 16, 128, 128, "bf16", "bf16", "f32", fresh=1.0),
        # the small configuration's types (32 bits throughout) at odd head sizes
        _extend("f32, odd sizes", 5, 1, 150, 3, 3, 48, 80, "f32", "f32", "f32"),
        # L2 norm before a tree verification: 64 requests of 4 nodes, 16 key heads shown to 32 value heads
        _qk("norm of a draft", 256, 16, 16, 128, "bf16", "l2", repeat=2),
        # the softmax layers of a hybrid at prefill: RMS norm with weights, a quarter of each head rotated
        _qk("norm and rotation of prompts", 32768, 16, 2, 256, "bf16", "rms", rope=64, pad=512),
        # one request's state shown to 8 samples
        _slots("fork to 8", 1, 32, 8, 1, 0, 32, 128, 128, "f32"),
        # compaction of all 30 layers' pools, some slots cleared
        _slots("compaction of 30 layers", 30, 96, 40, 40, 5, 32, 128, 128, "bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return int(min(hi, max(lo, round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(("extend", "extend", "extend", "qk", "slots"))
    if op == "extend":
        pool = rng.choice(("f32", "bf16"))
        gate = round(rng.uniform(0.5, 0.95), 3)
        if rng.random() < 0.2:  # 32 bits throughout, any head size
            dk, dv = rng.randint(8, 128), rng.randint(8, 128)
            H = rng.choice((1, 2, 3, 5))
            hi = _log(rng, 1, 400)
            return _extend("", _log(rng, 1, 24), max(1, hi // 3), hi, H, H, dk, dv, "f32", "f32", "f32", gate, 0.3)
        H = rng.choice(_HEADS)
        Hk = rng.choice([x for x in (1, 2, 4, 8, 16, 32, H) if H % x == 0])
        dk = dv = rng.choice((128, 128, 128, 64))
        out = rng.choice(("bf16", "bf16", "f32"))
        if rng.random() < 0.4:  # single tokens
            return _extend("", _log(rng, 1, 256), 1, 1, H, Hk, dk, dv, "bf16", out, pool, gate, 0.1,
                           rng.choice((0, 8, 128)))
        R = _log(rng, 1, 16)
        hi = _log(rng, 2, 4095)
        return _extend("", R, max(1, hi // rng.randint(1, 8)), hi, H, Hk, dk, dv, "bf16", out, pool, gate,
                       rng.choice((0.0, 0.5, 1.0)), rng.choice((0, 8, 128)))
    if op == "qk":
        d = rng.choice((64, 80, 128, 256))
        rope = rng.choice((0, d // 4 // 2 * 2, d))
        dtype = rng.choice(("bf16", "bf16", "f32"))
        return _qk("", 2 * _log(rng, 1, 16000) + 1, rng.choice((1, 2, 4, 5, 8, 16)), rng.choice((1, 2, 4, 5, 8)), d,
                   dtype, rng.choice(("l2", "rms")), rope, rng.random() < 0.3, rng.choice((1, 1, 2)),
                   rng.choice((0, 16, 200)))
    layers, n = rng.choice((1, 2, 4, 30)), _log(rng, 1, 40)
    return _slots("", layers, 2 * n + rng.randint(4, 14), n, rng.randint(1, n), rng.randint(0, 3),
                  rng.choice((1, 3, 8, 16)), 128, rng.choice((64, 128)), rng.choice(("f32", "bf16")))


def _lengths(c):
    """The sequences' lengths: hi once, the others spread evenly and out of order between lo and hi."""
    R, lo, hi = c["R"], c["lo"], c["hi"]
    n = np.array([hi - ((hi - lo) * i) // max(1, R - 1) for i in range(R)], dtype=np.int64)
    return n[np.random.RandomState(R).permutation(R)]


# ------------------------------------------------------------------ inputs

def _rows(T, heads, d, dtype, pad, make):
    """[T][heads][d] with `pad` elements of something else between the tokens' rows."""
    x = make(T, heads, d).to(dtype)
    if not pad:
        return x
    wide = torch.full((T, heads * d + pad), float("nan"), dtype=dtype, device=x.device)
    wide[:, :heads * d] = x.reshape(T, -1)
    return wide[:, :heads * d].view(T, heads, d)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=dev, dtype=torch.float32)

    c, s = case, {"case": case}
    if c["op"] == "extend":
        R, H, dk, dv, t = c["R"], c["H"], c["dk"], c["dv"], _TYPES[c["qkv"]]
        n = _lengths(c)
        off = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        T = int(off[-1])
        # keys of neighbouring tokens are alike, as a text's are
        base = normal(1, c["Hk"], dk)

        def unit(T, heads, d):
            x = normal(T, heads, d) + 0.3 * base
            return x / x.norm(dim=-1, keepdim=True)

        s["off"] = torch.from_numpy(off).to(dev)
        s["q"] = _rows(T, c["Hk"], dk, t, c["pad"], unit)
        s["k"] = _rows(T, c["Hk"], dk, t, c["pad"], unit)
        s["v"] = _rows(T, H, dv, t, c["pad"], normal)
        s["alpha"] = c["gate"] + (0.999 - c["gate"]) * uniform(T, H)
        s["beta"] = torch.sigmoid(normal(T, H))
        num = R + 3
        s["slot"] = torch.randperm(num, generator=g, device=dev)[:R].to(torch.int32)
        s["pool"] = (0.05 * normal(num, H, dv, dk)).to(_TYPES[c["pool"]])
        s["fresh"] = (uniform(R) < c["fresh"]).to(torch.uint8)
        s["o"] = torch.zeros(T, H, dv, device=dev, dtype=_TYPES[c["out"]])
        s["status"] = torch.zeros(R, device=dev, dtype=torch.int32)
        if own:
            from gdn_speculative_tree_gb300 import binding
            s["call"] = binding.make_seqs(
                seq_offset=s["off"], q=s["q"], k=s["k"], v=s["v"], alpha=s["alpha"], beta=s["beta"], state=s["pool"],
                state_slot=s["slot"], fresh=s["fresh"], o=s["o"], status=s["status"], max_len=c["hi"])
    elif c["op"] == "qk":
        T, d, t, rep = c["T"], c["d"], _TYPES[c["dtype"]], c["repeat"]
        s["q"] = _rows(T, c["Hq"], d, t, c["pad"], lambda *n: 2.0 * normal(*n))
        s["k"] = _rows(T, c["Hk"], d, t, c["pad"], lambda *n: 2.0 * normal(*n))
        s["wq"] = 1 + 0.2 * normal(d) if c["norm"] == "rms" else None
        s["wk"] = 1 + 0.2 * normal(d) if c["norm"] == "rms" else None
        s["rope"] = s["position"] = None
        if c["rope"]:
            span = 40960  # positions of a long context
            turn = 1e6 ** (-torch.arange(0, c["rope"], 2, device=dev, dtype=torch.float64) / c["rope"])
            angle = torch.arange(span, device=dev, dtype=torch.float64)[:, None] * turn
            s["rope"] = torch.cat([angle.cos(), angle.sin()], dim=1).float()
            s["position"] = torch.randint(0, span, (T,), generator=g, device=dev, dtype=torch.int32)
        s["qo"] = torch.zeros(T, c["Hq"] * rep, d, device=dev, dtype=t)
        s["ko"] = torch.zeros(T, c["Hk"] * rep, d, device=dev, dtype=t)
        s["status"] = torch.zeros(1, device=dev, dtype=torch.int32)
        if own:
            from gdn_speculative_tree_gb300 import binding
            s["call"] = binding.make_qk(
                q=s["q"], k=s["k"], q_out=s["qo"], k_out=s["ko"], status=s["status"], norm=c["norm"], eps=1e-6,
                q_weight=s["wq"], k_weight=s["wk"], q_scale=_scale(c), rope=s["rope"], position=s["position"],
                interleaved=c["interleaved"])
    else:
        n, m = c["moves"], c["moves"] + c["cleared"]
        s["pool"] = torch.empty(c["layers"], c["num_slots"], c["H"], c["dv"], c["dk"], device=dev,
                                dtype=_TYPES[c["pool"]]).normal_(0, 0.05, generator=g)
        at = torch.randperm(c["num_slots"], generator=g, device=dev).to(torch.int32)
        s["dst"] = at[:m].clone()
        src = at[m:m + c["sources"]].repeat(-(-n // c["sources"]))[:n]
        s["src"] = torch.cat([src, torch.full((c["cleared"],), -1, device=dev, dtype=torch.int32)])
        s["status"] = torch.zeros(m, device=dev, dtype=torch.int32)
        if own:
            from gdn_speculative_tree_gb300 import binding
            s["call"] = binding.make_slots(state=s["pool"], src=s["src"], dst=s["dst"], status=s["status"],
                                           layers=c["layers"])
    return s


def _scale(c):
    """Scale of the normed queries: 1/sqrt(d) for the delta rule's read-out, none for a softmax layer's."""
    return c["d"] ** -0.5 if c["norm"] == "l2" else 1.0


# ------------------------------------------------------------------ one pass

def run(state):
    s, op = state, state["case"]["op"]
    if own:
        from gdn_speculative_tree_gb300 import binding
        {"extend": binding.treewy_extend, "qk": binding.treewy_qk_norm, "slots": binding.treewy_copy_slots}[op](s["call"])
    else:
        {"extend": _plain_extend, "qk": _plain_qk, "slots": _plain_slots}[op](s)
    if op == "extend":
        return {"o": s["o"], "state": s["pool"], "status": s["status"]}
    if op == "qk":
        return {"q": s["qo"], "k": s["ko"], "status": s["status"]}
    return {"state": s["pool"], "status": s["status"]}


def _plain_extend(s):
    """The delta rule in chunks: within a chunk, with g_t the product of its decays up to t,
    A[t,i] = b_t (g_t/g_i) k_t.k_i for i < t,  U = (I + A)^-1 diag(b) (V - diag(g) K S^T),
    O = diag(g) Q S^T + M U with M[t,i] = (g_t/g_i) q_t.k_i for i <= t,  S <- g_C S + sum_i (g_C/g_i) u_i k_i^T."""
    c = s["case"]
    R, H, dk, dv, rep, L = c["R"], c["H"], c["dk"], c["dv"], c["H"] // c["Hk"], c["hi"]
    C = min(_CHUNK, L)
    n = -(-L // C)
    at = s["off"][:-1, None] + torch.arange(n * C, device=s["off"].device)  # [R][n C]
    live = at < s["off"][1:, None]
    at = at.clamp(max=max(0, s["q"].shape[0] - 1)).long()

    def chunks(x, fill):  # [T][heads](d) -> [R][H][n][C](d), in 32 bits
        x = x[at].float()
        x = torch.where(live.reshape(live.shape + (1,) * (x.dim() - 2)), x, torch.full_like(x, fill))
        if x.shape[2] != H:
            x = x.repeat_interleave(rep, dim=2)
        return x.reshape((R, n, C) + x.shape[2:]).movedim(3, 1)

    q, k, v = chunks(s["q"], 0.0), chunks(s["k"], 0.0), chunks(s["v"], 0.0)
    alpha, beta = chunks(s["alpha"], 1.0), chunks(s["beta"], 0.0)
    g = alpha.log().cumsum(-1)                                              # [R][H][n][C]
    lower = torch.ones(C, C, device=g.device).tril()
    ratio = torch.where(lower > 0, g[..., :, None] - g[..., None, :], torch.full_like(lower, -torch.inf)).exp()
    A = beta[..., None] * ratio * (k @ k.mT) * lower.tril(-1)
    M = ratio * (q @ k.mT)
    # (I + A)^-1 = (I - A)(I + A^2)(I + A^4)...: A is nilpotent
    inv, power, reach = torch.eye(C, device=g.device) - A, A, 2
    while reach < C:
        power = power @ power
        inv = inv + inv @ power
        reach *= 2
    eg = g.exp()[..., None]
    W, U0 = inv @ (beta[..., None] * eg * k), inv @ (beta[..., None] * v)
    kd = (g[..., -1:] - g).exp()[..., None] * k
    slot = s["slot"].long()
    S = torch.where(s["fresh"][:, None, None, None] != 0, torch.zeros((), device=g.device), s["pool"][slot].float())
    out = torch.empty_like(v)
    for i in range(n):  # the recurrence over chunks
        u = U0[:, :, i] - W[:, :, i] @ S.mT
        out[:, :, i] = eg[:, :, i] * (q[:, :, i] @ S.mT) + M[:, :, i] @ u
        S = eg[:, :, i, -1:] * S + u.mT @ kd[:, :, i]
    s["pool"][slot] = S.to(s["pool"].dtype)
    o = out.movedim(1, 3).reshape(R, n * C, H, dv)
    s["o"].copy_(o[live])


def _plain_qk(s):
    c = s["case"]
    for name, w, scale in (("q", s["wq"], _scale(c)), ("k", s["wk"], 1.0)):
        x = s[name].float()
        square = x.square()
        total = square.sum(-1, keepdim=True) if c["norm"] == "l2" else square.mean(-1, keepdim=True)
        x = x * (scale / (total + 1e-6).sqrt())
        if w is not None:
            x = x * w
        if c["rope"]:
            r = c["rope"]
            table = s["rope"][s["position"].long()][:, None]
            cos, sin = table[..., :r // 2], table[..., r // 2:]
            x, rest = x[..., :r], x[..., r:]
            a, b = (x[..., 0::2], x[..., 1::2]) if c["interleaved"] else (x[..., :r // 2], x[..., r // 2:])
            a, b = a * cos - b * sin, b * cos + a * sin
            x = torch.cat([torch.stack([a, b], -1).flatten(-2) if c["interleaved"] else torch.cat([a, b], -1), rest], -1)
        s[name + "o"].copy_(x.repeat_interleave(c["repeat"], dim=1) if c["repeat"] > 1 else x)


def _plain_slots(s):
    src, dst = s["src"].long(), s["dst"].long()
    new = s["pool"].index_select(1, src.clamp(min=0))
    new = torch.where((src >= 0)[None, :, None, None, None], new, torch.zeros((), device=new.device, dtype=new.dtype))
    s["pool"].index_copy_(1, dst, new)


# ------------------------------------------------------------------ the definitions, in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"extend": _exact_extend, "qk": _exact_qk, "slots": _exact_slots}[case["op"]](case, s)


def _exact_extend(c, s):
    """Token by token, each request and value head from the definition."""
    n = _lengths(c)
    if int(n.max()) * 8e-4 > 18:  # seconds
        return None
    off = s["off"][:-1].long()
    rep = c["H"] // c["Hk"]
    length = torch.from_numpy(n).to(off.device)
    pool = s["pool"].double()
    S = pool[s["slot"].long()]
    S[s["fresh"] != 0] = 0
    o = torch.zeros(s["o"].shape, device=off.device, dtype=torch.float64)
    for t in range(int(n.max())):
        r = torch.nonzero(length > t)[:, 0]
        row = off[r] + t
        q, k = (x[row].double().repeat_interleave(rep, dim=1)[..., None] for x in (s["q"], s["k"]))
        v = s["v"][row].double()[..., None]
        a, b = (x[row].double()[..., None, None] for x in (s["alpha"], s["beta"]))
        old = S if len(r) == len(n) else S[r]
        new = a * (old - b * (old @ k) @ k.mT) + b * v @ k.mT
        o[row] = (new @ q)[..., 0]
        if len(r) == len(n):
            S = new
        else:
            S[r] = new
    pool[s["slot"].long()] = S
    return {"o": o, "state": pool, "status": None}


def _exact_qk(c, s):
    out = {"status": None}
    for name, w, scale in (("q", s["wq"], _scale(c)), ("k", s["wk"], 1.0)):
        x = s[name].double()
        norm = torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2
        y = scale * x / torch.sqrt((norm if c["norm"] == "l2" else norm / c["d"]) + 1e-6)
        y = y * (1 if w is None else w.double())
        r = c["rope"]
        if r:
            i = torch.arange(r // 2, device=x.device)
            first, second = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + r // 2)
            table = s["rope"].double()[s["position"].long()]
            turn = torch.complex(table[:, :r // 2], table[:, r // 2:])[:, None]
            z = torch.complex(y[..., first], y[..., second]) * turn
            y[..., first], y[..., second] = z.real, z.imag
        out[name] = y.repeat_interleave(c["repeat"], dim=1)
    return out


def _exact_slots(c, s):
    pool = s["pool"].double()
    before = s["pool"]
    for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
        pool[:, b] = before[:, a].double() if a >= 0 else 0.0
    return {"state": pool, "status": None}


# ------------------------------------------------------------------ the work of one pass

def work(case):
    c = case
    size = {"bf16": 2, "f32": 4}
    if c["op"] == "extend":
        T, R = int(_lengths(c).sum()), c["R"]
        row = 2 * c["Hk"] * c["dk"] * size[c["qkv"]] + c["H"] * (c["dv"] * (size[c["qkv"]] + size[c["out"]]) + 8)
        block = c["H"] * c["dk"] * c["dv"]
        # S k, the rank-one update and S q of every token and head; each state read (unless it starts from
        # zero) and written once
        return {"bytes": T * row + R * block * size[c["pool"]] * (2 - c["fresh"]), "flops": 6.0 * T * block}
    if c["op"] == "qk":
        e = size[c["dtype"]] * c["T"] * (c["Hq"] + c["Hk"]) * c["d"]
        table = 4 * min(c["T"], 40960) * c["rope"] + (4 * c["T"] if c["rope"] else 0)
        return {"bytes": e * (1 + c["repeat"]) + table, "flops": 4.0 * c["T"] * (c["Hq"] + c["Hk"]) * c["d"]}
    block = c["H"] * c["dk"] * c["dv"] * size[c["pool"]] * c["layers"]
    return {"bytes": float(block * (min(c["sources"], c["moves"]) + c["moves"] + c["cleared"])), "flops": 0.0}


if __name__ == "__main__":
    for case in listed() + [draw(random.Random(i)) for i in range(8)]:
        print(case, work(case))
