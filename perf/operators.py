"""Operators of a served layer next to its prefill: rotary positions, attention
of drafted tokens over a key/value cache, and eviction from that cache.

Each case is one call. `own` false computes it in elementary torch operations
(fp32, or fp64 where fp32 loses what matters); `own` true makes the call of
this package. `exact` is the definition in fp64, written separately.

Layouts: Q [B, Hq, T, 128] and caches [B, Hkv, cap, 128] in bf16; query head hq
reads kv head hq // (Hq // Hkv). Sequence b holds lengths[b] slots, and its
n_draft[b] drafted tokens sit in the slots right after them.
"""
import math

import torch

own = False

D = 128
SCALE = 1.0 / math.sqrt(D)


# ----------------------------------------------------------------- the cases
def _rotary(name, B, Hq, Hkv, T, rd=128, interleaved=False, scaling="none", transpose=False, token_major=False,
            append=False, cap=0, far=0):
    return {"name": name, "op": "rotary", "B": B, "Hq": Hq, "Hkv": Hkv, "T": T, "rd": rd, "interleaved": interleaved,
            "scaling": scaling, "transpose": transpose, "token_major": token_major, "append": append, "cap": cap,
            "far": far}


def _tree(name, B, Hq, Hkv, T, lo, hi, tree=False, weights=False, ragged=False):
    return {"name": name, "op": "tree", "B": B, "Hq": Hq, "Hkv": Hkv, "T": T, "lo": lo, "hi": hi, "tree": tree,
            "weights": weights, "ragged": ragged}


def _evict(name, B, Hkv, lo, hi, keep, T=0, sinks=4, recent=32):
    return {"name": name, "op": "evict", "B": B, "Hkv": Hkv, "lo": lo, "hi": hi, "keep": keep, "T": T,
            "sinks": sinks, "recent": recent}


def listed():
    return [
        # one new token for each of eight sequences: the smallest call, K, V and positions go into the cache
        _rotary("rotary-append-1", 8, 32, 8, 1, append=True, cap=4112, far=120000, scaling="wavelength"),
        # the 32K prefill layer, read as the projections leave it (token-major), with rescaled frequencies
        _rotary("rotary-prefill-32k", 1, 32, 8, 32768, scaling="wavelength", token_major=True),
        # gradients of an 8K layer (two sequences, odd length), interleaved pairs over half of the head
        _rotary("rotary-gradient-8k", 2, 16, 2, 8191, rd=64, interleaved=True, scaling="yarn", transpose=True),
        # one token over a short prompt: latency alone
        _tree("tree-1-short", 1, 2, 1, 1, 37, 37),
        # one token over the 128K context: every key and value is read once
        _tree("tree-1-128k", 1, 32, 8, 1, 131071, 131071),
        # a served batch of ragged contexts, one token each, attention weight kept for eviction
        _tree("tree-1-batch32", 32, 32, 8, 1, 1021, 8190, weights=True),
        # drafted trees of up to 32 tokens over 8K contexts, eight query heads to a kv head
        _tree("tree-32-8k", 4, 16, 2, 32, 7001, 8192, tree=True, weights=True, ragged=True),
        # the last 64 prompt tokens over a 128K cache: scores every slot before the first eviction
        _tree("window-64-128k", 1, 32, 8, 64, 131008, 131008, weights=True),
        # a handful of slots over budget: the smallest eviction
        _evict("evict-few", 4, 2, 2040, 2057, 2048, recent=8),
        # steady serving: a batch drops rejected drafts and goes back to its budget
        _evict("evict-batch32", 32, 8, 4090, 4096, 4096, T=16, recent=64),
        # after the prompt: 128K slots down to 8K
        _evict("evict-128k", 1, 8, 131072, 131072, 8192, recent=64),
        # accepted drafts only, nothing over budget
        _evict("commit-64", 8, 8, 8000, 8192, 1 << 20, T=64),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    Hq, Hkv = rng.choice([(2, 1), (4, 4), (8, 1), (16, 2), (32, 8), (32, 4)])
    op = rng.choice(["rotary", "tree", "tree", "evict"])
    if op == "rotary":
        B = rng.choice([1, 2, 3, 8])
        append = rng.random() < 0.5
        T = log(1, 512) if append else log(1, max(2, 32768 * 40 // ((Hq + Hkv) * B * 2)))
        c = _rotary("", B, Hq, Hkv, T, rd=rng.choice([128, 128, 64, 32, 96]), interleaved=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "wavelength", "yarn"]),
                    transpose=not append and rng.random() < 0.4, token_major=rng.random() < 0.5, append=append,
                    cap=T + log(1, 2000) if append else 0, far=log(1, 1000000))
    elif op == "tree":
        B = rng.choice([1, 1, 2, 5, 16])
        T = rng.choice([1, 1, 2, 3, 7, 16, 33, 64])
        hi = log(1, max(2, 60000 * 8 // (Hkv * B)))
        c = _tree("", B, Hq, Hkv, T, rng.randint(0, hi) if B > 1 else hi, hi, tree=rng.random() < 0.6,
                  weights=rng.random() < 0.5, ragged=rng.random() < 0.5)
    else:
        B = rng.choice([1, 2, 7, 16])
        hi = log(70, max(80, 60000 * 8 // (Hkv * B)))
        T = rng.choice([0, 0, 1, 16, 64])
        c = _evict("", B, Hkv, rng.randint(hi // 2, hi), hi, rng.choice([max(1, hi - T), max(1, hi // 3), hi // 2]), T=T,
                   sinks=rng.choice([0, 4]), recent=rng.choice([0, 1, 32]))
    del c["name"]
    return c


# ----------------------------------------------------------------- sizes that follow from a case
def _lengths(case):
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [hi - (hi - lo) * ((b * 7) % B) // max(B - 1, 1) for b in range(B)]


def _drafts(case):
    T = case["T"]
    return [max(1, T - (b % 3) * (T // 4)) if case["ragged"] else T for b in range(case["B"])]


def _tree_cap(case):
    return case["hi"] + case["T"] + 5


def _evict_cap(case):
    return case["hi"] + case["T"]


def work(case):
    B = case["B"]
    if case["op"] == "rotary":
        rows = B * case["T"] * (case["Hq"] + case["Hkv"])
        if case["append"]:   # V is copied into the cache too, and a position is written for each slot
            return {"bytes": (rows + B * case["T"] * case["Hkv"]) * 512 + B * case["T"] * (8 + 4 * case["Hkv"]),
                    "flops": rows * case["rd"] * 3}
        return {"bytes": rows * 512 + B * case["T"] * 4, "flops": rows * case["rd"] * 3}
    if case["op"] == "tree":
        Hq, Hkv = case["Hq"], case["Hkv"]
        slots = sum(n + t for n, t in zip(_lengths(case), _drafts(case)))
        pairs = sum(t * n + t * (t + 1) // 2 for n, t in zip(_lengths(case), _drafts(case)))
        rows = sum(_drafts(case)) * Hq
        return {"bytes": slots * Hkv * (512 + (8 if case["weights"] else 0)) + rows * 512,
                "flops": 4 * D * Hq * pairs}
    Hkv, T, moved, slots, kept = case["Hkv"], case["T"], 0.0, 0, 0
    for n in _lengths(case):
        have = n + T - T // 2                 # about half of the drafts are accepted
        m = min(have, case["keep"])
        # a slot past the first m moves when it is kept
        moved += (n + T - m) * (m / (n + T))
        slots += n + T
        kept += m
    # weight and position of each slot are read, those of each kept slot and its source are written
    return {"bytes": Hkv * (slots * 8 + kept * 12 + moved * 1024), "flops": Hkv * slots}


# ----------------------------------------------------------------- inputs
def _inv_freq(case):
    """The frequencies of a served model, in fp64, and the factor on its cosines."""
    rd, base = case["rd"], 500000.0
    f = [base ** (-2.0 * i / rd) for i in range(rd // 2)]
    if case["scaling"] == "linear":            # positions squeezed by 4
        return [x / 4 for x in f], 1.0
    if case["scaling"] == "wavelength":        # long waves stretched by 8, short ones kept, a blend between
        out = []
        for x in f:
            turns = 8192.0 * x / (2 * math.pi)
            s = min(1.0, max(0.0, (turns - 1.0) / 3.0))
            out.append(s * x + (1 - s) * x / 8.0)
        return out, 1.0
    if case["scaling"] == "yarn":              # a ramp over the pair index, and a factor on cos and sin
        at = [rd * math.log(8192.0 / (r * 2 * math.pi)) / (2 * math.log(base)) for r in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rd - 1)
        out = []
        for i, x in enumerate(f):
            s = min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3)))
            out.append((1 - s) * x + s * x / 16.0)
        return out, 0.1 * math.log(16.0) + 1.0
    return f, 1.0


def _parents(T, g):
    """A random drafted tree: each token hangs on one of the few before it, or on the context."""
    back = torch.randint(1, 5, (T,), generator=g)
    return torch.clamp(torch.arange(T) - back, min=-1).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    gc = torch.Generator().manual_seed(seed)
    B, T = case["B"], case["T"]

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, device="cuda", generator=g, dtype=torch.float32) * scale).to(torch.bfloat16)

    def ints(v, dtype=torch.int32):
        return torch.tensor(v, device="cuda", dtype=dtype)

    if case["op"] == "rotary":
        Hq, Hkv = case["Hq"], case["Hkv"]
        f, factor = _inv_freq(case)
        s = {"case": case, "inv_freq": ints(f, torch.float64), "factor": factor}
        for name, H in (("Q", Hq), ("K", Hkv), ("V", Hkv)):
            x = normal(B, T, H, D).transpose(1, 2) if case["token_major"] else normal(B, H, T, D)
            s[name] = x
        first = torch.randint(0, case["far"] + 1, (B,), generator=gc)
        s["positions"] = (first[:, None] + torch.arange(T)[None]).to(torch.int32).cuda()
        s["Q_out"] = torch.zeros(B, Hq, T, D, device="cuda", dtype=torch.bfloat16)
        if case["append"]:
            cap = case["cap"]
            s["slots"] = torch.randint(0, cap - T + 1, (B,), generator=gc).to(torch.int32).cuda()
            s["K_out"], s["V_out"] = normal(B, Hkv, cap, D), normal(B, Hkv, cap, D)
            s["pos_out"] = torch.zeros(B, Hkv, cap, device="cuda", dtype=torch.int32)
        else:
            s["K_out"] = torch.zeros(B, Hkv, T, D, device="cuda", dtype=torch.bfloat16)
        return s
    if case["op"] == "tree":
        Hq, Hkv, cap = case["Hq"], case["Hkv"], _tree_cap(case)
        s = {"case": case, "Q": normal(B, Hq, T, D, scale=2.0), "K": normal(B, Hkv, cap, D),
             "V": normal(B, Hkv, cap, D), "lengths": ints(_lengths(case)), "n_draft": ints(_drafts(case)),
             "parents": torch.stack([_parents(T, gc) for _ in range(B)]).cuda() if case["tree"] else None,
             "O": torch.zeros(B, Hq, T, D, device="cuda", dtype=torch.bfloat16)}
        if case["weights"]:
            s["weight"] = torch.rand(B, Hkv, cap, device="cuda", generator=g) * 0.01
            s["weight_out"] = torch.zeros_like(s["weight"])
        return s
    Hkv, cap, lengths = case["Hkv"], _evict_cap(case), _lengths(case)
    s = {"case": case, "K": normal(B, Hkv, cap, D), "V": normal(B, Hkv, cap, D), "lengths": ints(lengths)}
    # accumulated attention spreads over several powers of ten
    s["weight"] = torch.exp(2.5 * torch.randn(B, Hkv, cap, device="cuda", generator=g) - 6.0)
    # slots hold tokens of a longer text, in an order that earlier evictions left
    s["pos"] = torch.argsort(torch.rand(B, Hkv, cap, device="cuda", generator=g), dim=-1).to(torch.int32) * 3
    s["next_pos"] = ints([3 * cap] * B)
    if T:
        s["n_draft"] = ints([T] * B)
        bits = torch.randint(0, 2, (B, T), generator=gc)
        bits[:, 0] = 1
        s["accept"] = ints([int.from_bytes(int("".join(str(x) for x in reversed(r.tolist())), 2).to_bytes(8, "little"),
                                           "little", signed=True) for r in bits], torch.int64)
    s["weight_out"], s["pos_out"] = torch.zeros_like(s["weight"]), torch.zeros_like(s["pos"])
    s["lengths_out"] = torch.zeros_like(s["lengths"])
    s["index"] = torch.zeros(B, Hkv, min(case["keep"], cap), device="cuda", dtype=torch.int32)
    return s


# ----------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return {"rotary": _own_rotary, "tree": _own_tree, "evict": _own_evict}[op](s)
    return {"rotary": _plain_rotary, "tree": _plain_tree, "evict": _plain_evict}[op](s)


def _own_rotary(s):
    from long_context_prefill_dhsa_b200 import binding
    c = s["case"]
    if c["append"]:
        binding.rotary_qkv(s["Q"], s["K"], s["inv_freq"], V=s["V"], positions=s["positions"], slots=s["slots"],
                           interleaved=c["interleaved"], factor=s["factor"], Q_out=s["Q_out"], K_out=s["K_out"],
                           V_out=s["V_out"], pos_out=s["pos_out"])
        return {"Q": s["Q_out"], "K": s["K_out"], "V": s["V_out"], "pos": s["pos_out"]}
    binding.rotary_qkv(s["Q"], s["K"], s["inv_freq"], positions=s["positions"], interleaved=c["interleaved"],
                       transpose=c["transpose"], factor=s["factor"], Q_out=s["Q_out"], K_out=s["K_out"])
    return {"Q": s["Q_out"], "K": s["K_out"]}


def _own_tree(s):
    from long_context_prefill_dhsa_b200 import binding
    if s["case"]["weights"]:
        binding.tree_attn(s["Q"], s["K"], s["V"], s["lengths"], parents=s["parents"], n_draft=s["n_draft"],
                          weight=s["weight"], weight_out=s["weight_out"], out=s["O"])
        return {"O": s["O"], "weight": s["weight_out"]}
    binding.tree_attn(s["Q"], s["K"], s["V"], s["lengths"], parents=s["parents"], n_draft=s["n_draft"], out=s["O"])
    return {"O": s["O"]}


def _own_evict(s):
    from long_context_prefill_dhsa_b200 import binding
    c = s["case"]
    binding.cache_evict(s["K"], s["V"], s["weight"], s["pos"], s["lengths"], c["keep"], next_pos=s["next_pos"],
                        n_draft=s.get("n_draft"), accept=s.get("accept"), sinks=c["sinks"], recent=c["recent"],
                        weight_out=s["weight_out"], pos_out=s["pos_out"], lengths_out=s["lengths_out"],
                        index=s["index"])
    return {"K": s["K"], "V": s["V"], "weight": s["weight_out"], "pos": s["pos_out"], "lengths": s["lengths_out"],
            "index": s["index"]}


def _plain_turn(x, cos, sin, c):
    rd = c["rd"]
    x = x.to(torch.float32)
    rot, rest = x[..., :rd], x[..., rd:]
    if c["interleaved"]:
        a, b = rot[..., 0::2], rot[..., 1::2]
    else:
        a, b = rot[..., : rd // 2], rot[..., rd // 2:]
    if c["transpose"]:
        sin = -sin
    u, v = a * cos - b * sin, a * sin + b * cos
    rot = torch.stack((u, v), dim=-1).flatten(-2) if c["interleaved"] else torch.cat((u, v), dim=-1)
    return torch.cat((rot, rest), dim=-1).to(torch.bfloat16)


def _plain_rotary(s):
    c = s["case"]
    # in fp64: a far position times a frequency needs more digits than fp32 has
    angle = s["positions"].to(torch.float64)[:, None, :, None] * s["inv_freq"]
    cos, sin = ((f(angle) * s["factor"]).to(torch.float32) for f in (torch.cos, torch.sin))
    s["Q_out"].copy_(_plain_turn(s["Q"], cos, sin, c))
    K = _plain_turn(s["K"], cos, sin, c)
    if not c["append"]:
        s["K_out"].copy_(K)
        return {"Q": s["Q_out"], "K": s["K_out"]}
    at = s["slots"].long()[:, None] + torch.arange(c["T"], device="cuda")
    b = torch.arange(c["B"], device="cuda")[:, None]
    s["K_out"][b, :, at] = K.transpose(1, 2)
    s["V_out"][b, :, at] = s["V"].transpose(1, 2)
    s["pos_out"][b, :, at] = s["positions"][:, :, None].expand(-1, -1, c["Hkv"])
    return {"Q": s["Q_out"], "K": s["K_out"], "V": s["V_out"], "pos": s["pos_out"]}


def _plain_tree(s):
    c = s["case"]
    B, Hq, Hkv, T = c["B"], c["Hq"], c["Hkv"], c["T"]
    cap = s["K"].shape[2]
    slot = torch.arange(cap, device="cuda")
    t = torch.arange(T, device="cuda")
    n, nd = s["lengths"].long()[:, None, None], s["n_draft"].long()[:, None, None]
    if s["parents"] is None:
        sees = (t[None, :, None] >= t[None, None, :]).expand(B, T, T)
    else:
        # reach[t, j]: j is t or an ancestor of t; powers of (1 + parent) double the depth they cover
        reach = torch.zeros(B, T, T + 1, device="cuda")
        reach.scatter_(2, s["parents"].long().remainder(T + 1)[..., None], 1.0)
        reach = reach[..., :T] + torch.eye(T, device="cuda")
        reach = torch.linalg.matrix_power(reach.to(torch.float64), 64) if T > 1 else reach
        sees = reach > 0
    j = slot - n                                                      # draft index of a slot
    inside = (j >= 0) & (j < nd)
    drafted = torch.gather(sees, 2, j.clamp(0, T - 1).expand(B, T, cap))
    seen = ((j < 0) | (inside & drafted))[:, None, None]                # [B, 1, 1, T, cap]
    q = s["Q"].to(torch.float32).view(B, Hkv, Hq // Hkv, T, D)
    k, v = s["K"].to(torch.float32)[:, :, None], s["V"].to(torch.float32)[:, :, None]
    score = torch.matmul(q.reshape(B, Hkv, 1, -1, D), k.transpose(-1, -2)).view(B, Hkv, Hq // Hkv, T, cap) * SCALE
    score = score.masked_fill_(~seen, -torch.inf)
    score = score.sub_(score.amax(-1, keepdim=True)).exp_()
    p = score.div_(score.sum(-1, keepdim=True))
    o = torch.matmul(p.view(B, Hkv, 1, -1, cap), v).view(B, Hq, T, D)
    row = (t < s["n_draft"][:, None])                                  # [B, T]
    s["O"].copy_(torch.where(row[:, None, :, None], o.to(torch.bfloat16), s["O"]))
    if not c["weights"]:
        return {"O": s["O"]}
    got = p.masked_fill_(~row[:, None, None, :, None], 0.0).sum((2, 3))
    old = torch.where(j[:, 0][:, None] < 0, s["weight"], 0.0)
    s["weight_out"].copy_(torch.where(((j < 0) | inside)[:, 0][:, None], old + got, s["weight_out"]))
    return {"O": s["O"], "weight": s["weight_out"]}


def _plain_evict(s):
    c = s["case"]
    cap, keep = s["K"].shape[2], c["keep"]
    slot = torch.arange(cap, device="cuda")
    n = s["lengths"].long()[:, None]
    there = slot < n
    if "accept" in s:
        j = slot - n
        bit = (s["accept"][:, None] >> j.clamp(0, 63)) & 1
        there = there | ((j >= 0) & (j < s["n_draft"][:, None]) & (bit == 1))
    m = there.sum(-1).clamp(max=keep)                                  # [B]
    held = (s["pos"] < c["sinks"]) | (s["pos"] >= s["next_pos"][:, None, None] - c["recent"])
    key = s["weight"].masked_fill(held, torch.inf).masked_fill(~there[:, None], -torch.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, slot.expand_as(order))
    kept, low = rank < m[:, None, None], slot < m[:, None, None]
    hole = low & ~kept
    tails = torch.sort(torch.where(kept & ~low, slot, cap), dim=-1).values
    index = torch.where(hole, tails.gather(-1, (hole.cumsum(-1) - 1).clamp(min=0)), slot)
    index = torch.where(low, index, -1)
    take = index.clamp(min=0)
    for name in ("K", "V"):
        x = s[name]
        x.copy_(torch.where(low[..., None], x.gather(2, take[..., None].expand_as(x)), x))
    s["weight_out"].copy_(torch.where(low, s["weight"].gather(-1, take), s["weight_out"]))
    s["pos_out"].copy_(torch.where(low, s["pos"].gather(-1, take), s["pos_out"]))
    s["lengths_out"].copy_(m)
    s["index"].copy_(index[..., : s["index"].shape[-1]])
    return {"K": s["K"], "V": s["V"], "weight": s["weight_out"], "pos": s["pos_out"], "lengths": s["lengths_out"],
            "index": s["index"]}


# ----------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "tree": _exact_tree, "evict": _exact_evict}[case["op"]](case, s)


def _exact_rotary(case, s):
    rd, T = case["rd"], case["T"]
    # a pair is a complex number, and its rotation one product
    turn = torch.polar(torch.full((), s["factor"], dtype=torch.float64, device="cuda").expand(case["B"], T, rd // 2)
                       .contiguous(), s["positions"].double()[..., None] * s["inv_freq"])
    turn = (turn.conj() if case["transpose"] else turn)[:, None]

    def of(x):
        x = x.double().contiguous()
        lead = x[..., :rd]
        if case["interleaved"]:
            z = torch.view_as_complex(lead.reshape(*lead.shape[:-1], rd // 2, 2).contiguous()) * turn
            x[..., :rd] = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(lead[..., : rd // 2].contiguous(), lead[..., rd // 2:].contiguous()) * turn
            x[..., : rd // 2], x[..., rd // 2: rd] = z.real, z.imag
        return x

    if not case["append"]:
        return {"Q": of(s["Q"]), "K": of(s["K"])}
    K, V, pos, new = s["K_out"].double(), s["V_out"].double(), s["pos_out"].clone(), of(s["K"])
    for b, at in enumerate(s["slots"].tolist()):
        K[b, :, at: at + T] = new[b]
        V[b, :, at: at + T] = s["V"][b].double()
        pos[b, :, at: at + T] = s["positions"][b]
    return {"Q": of(s["Q"]), "K": K, "V": V, "pos": pos}


def _exact_tree(case, s):
    B, Hq, Hkv, T = case["B"], case["Hq"], case["Hkv"], case["T"]
    G = Hq // Hkv
    O = s["O"].double()
    W = s["weight_out"].double() if case["weights"] else None
    for b, (n, t) in enumerate(zip(_lengths(case), _drafts(case))):
        up = s["parents"][b].tolist() if case["tree"] else list(range(-1, T - 1))
        sees = torch.zeros(t, t, dtype=torch.bool)
        for r in range(t):
            a = r
            while a >= 0:
                sees[r, a] = True
                a = up[a]
        hidden = (~sees).cuda()
        for h in range(Hkv):
            k, v = s["K"][b, h, : n + t].double(), s["V"][b, h, : n + t].double()
            q = s["Q"][b, h * G: (h + 1) * G, :t].double()
            z = (q @ k.T) / math.sqrt(128.0)
            z[..., n:].masked_fill_(hidden, -torch.inf)
            p = torch.softmax(z, -1)
            O[b, h * G: (h + 1) * G, :t] = p @ v
            if W is not None:
                W[b, h, : n + t] = p.sum((0, 1))
                W[b, h, :n] += s["weight"][b, h, :n].double()
    return {"O": O, "weight": W} if case["weights"] else {"O": O}


def _exact_evict(case, s):
    B, Hkv, T, keep = case["B"], case["Hkv"], case["T"], case["keep"]
    out = {"K": s["K"].double(), "V": s["V"].double(), "weight": s["weight_out"].double(), "pos": s["pos_out"].clone(),
           "lengths": s["lengths_out"].clone(), "index": torch.full_like(s["index"], -1)}
    lengths = _lengths(case)
    for b in range(B):
        there = list(range(lengths[b]))
        if T:
            bits = int(s["accept"][b])
            there += [lengths[b] + j for j in range(T) if bits >> j & 1]
        m = min(len(there), keep)
        out["lengths"][b] = m
        for h in range(Hkv):
            w, pos = s["weight"][b, h].tolist(), s["pos"][b, h].tolist()
            limit = int(s["next_pos"][b]) - case["recent"]
            best = there if m == len(there) else sorted(
                there, key=lambda i: (not (pos[i] < case["sinks"] or pos[i] >= limit), -w[i], i))[:m]
            best = set(best)
            come = iter(sorted(i for i in best if i >= m))
            src = torch.tensor([i if i in best else next(come) for i in range(m)], device="cuda")
            out["index"][b, h, :m] = src.to(torch.int32)
            for name in ("K", "V"):
                out[name][b, h, :m] = s[name][b, h][src].double()
            out["weight"][b, h, :m] = s["weight"][b, h][src].double()
            out["pos"][b, h, :m] = s["pos"][b, h][src]
    return out
