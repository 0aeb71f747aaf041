"""The operators of a speculative decode step on a quantised R-SWA cache, as cases to measure.

  rope     norms of queries and keys per head with the position rotation
  kv       quantising cache rows as they are written, and reading them back
  tree     attention for a tree of drafted tokens over a reference block and a 128-slot ring
  probs    logits to probabilities at a temperature
  verify   verification of the drafted tokens against the target's probabilities

`run` computes them with elementary torch operations (own = False) or through the framework's
public entry points (own = True), on the inputs that `prepare` makes.
"""
import math
import random

import torch

own = False

D = 128        # head dimension
RING = 128     # slots of the generated-token ring
HEADS = 10     # the decoder's attention heads
VOCAB = 129280
THETA = 10000.0
EPS = 1e-6


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token of one sequence: q and k of ten heads, rotated only (this decoder has no q/k norms)
        dict(name="rope_t1", op="rope", T=1, hq=HEADS, hk=HEADS, rot=128, interleaved=False, norm=False, packed=False),
        # the most tokens one call takes, q and k read from the rows of a fused q/k/v projection, norms with weights
        dict(name="rope_t8192", op="rope", T=8192, hq=HEADS, hk=HEADS, rot=128, interleaved=False, norm=True, packed=True),
        # accepted drafts of a batch committed to the ring in int4 (path indices from a verification)
        dict(name="kv_commit_b8", op="kv", kind="int4", B=8, heads=HEADS, cap=RING, new=9, wrap=True),
        # the reference blocks of a ragged batch of prompts written in int8 and read back whole
        dict(name="kv_prefill_b8", op="kv", kind="int8", B=8, heads=HEADS, cap=4096, new=4096, wrap=False),
        # one token after the 289-token prefill of one page: the single-token form, latency counts
        dict(name="tree_t1_r289", op="tree", kind="int8", B=1, R=289, N=1, hq=HEADS, hk=HEADS, n_gen=600, chain=True),
        # eight sequences, sixteen drafted nodes each, after one page
        dict(name="tree_b8_r289", op="tree", kind="int8", B=8, R=289, N=16, hq=HEADS, hk=HEADS, n_gen=600, chain=False),
        # many sequences over long ragged prompts in int4, two query heads to a key head, an odd tree
        dict(name="tree_b32_r4096", op="tree", kind="int4", B=32, R=4096, N=7, hq=2 * HEADS, hk=HEADS, n_gen=100, chain=False),
        # the longest reference block, large trees
        dict(name="tree_b8_r32768", op="tree", kind="int8", B=8, R=32768, N=32, hq=HEADS, hk=HEADS, n_gen=1000, chain=False),
        # one row of the lm_head's logits
        dict(name="probs_t1", op="probs", T=1, V=VOCAB, temperature=1.0),
        # the logits of a prefill-sized batch
        dict(name="probs_t289", op="probs", T=289, V=VOCAB, temperature=0.7),
        # four drafted tokens of one sequence
        dict(name="verify_b1_n4", op="verify", B=1, N=4, V=VOCAB, chain=True, draft=True),
        # drafted trees of a batch
        dict(name="verify_b32_n16", op="verify", B=32, N=16, V=VOCAB, chain=False, draft=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "kv", "tree", "tree", "probs", "verify"])
    if op == "rope":
        hk = rng.choice([1, 2, 5, HEADS])
        return dict(op=op, T=_log(rng, 1, 8192), hq=hk * rng.choice([1, 2]) if hk < HEADS else HEADS, hk=hk,
                    rot=rng.choice([128, 64, 96, 34]), interleaved=rng.random() < 0.5, norm=rng.random() < 0.6,
                    packed=rng.random() < 0.5)
    if op == "kv":
        kind, heads = rng.choice(["int8", "int4"]), rng.choice([1, 2, HEADS])
        if rng.random() < 0.5:
            return dict(op=op, kind=kind, B=_log(rng, 1, 64), heads=heads, cap=RING, new=_log(rng, 1, 150), wrap=True)
        cap = _log(rng, 16, 4096)
        return dict(op=op, kind=kind, B=_log(rng, 1, 8), heads=heads, cap=cap, new=rng.randint(max(1, cap // 2), cap), wrap=False)
    if op == "tree":
        B = _log(rng, 1, 32)
        g = rng.choice([1, 1, 2, 4])
        return dict(op=op, kind=rng.choice(["int8", "int4"]), B=B, R=_log(rng, 1, min(32768, 8 * 32768 // B)),
                    N=_log(rng, 1, 32 // g), hq=g * HEADS, hk=HEADS, n_gen=_log(rng, 1, 2000), chain=rng.random() < 0.4)
    V = rng.choice([VOCAB, _log(rng, 1000, VOCAB)])
    if op == "probs":
        return dict(op=op, T=_log(rng, 1, 289), V=V, temperature=round(rng.uniform(0.3, 1.5), 2))
    return dict(op=op, B=_log(rng, 1, 32), N=_log(rng, 1, 16), V=V, chain=rng.random() < 0.5, draft=rng.random() < 0.7)


def _ragged(most, B):
    """Lengths of a ragged batch: from `most` down to about half of it."""
    return [most - (most * b) // (2 * B) for b in range(B)]


def _counts(case):
    """New tokens of each sequence of a kv case."""
    return _ragged(case["new"], case["B"])


def work(case):
    op = case["op"]
    if op == "rope":
        rows = case["T"] * (case["hq"] + case["hk"])
        return {"bytes": rows * D * 8 + 4 * case["T"], "flops": rows * D * (8 if case["norm"] else 4)}
    if op == "kv":
        packed = (D if case["kind"] == "int8" else D // 2) + 4
        new = sum(_counts(case)) * case["heads"] * 2
        kept = sum(_valid(case)) * case["heads"] * 2
        return {"bytes": new * (4 * D + packed) + kept * (4 * D + packed), "flops": (3 * new + kept) * D}
    if op == "tree":
        row = (D if case["kind"] == "int8" else D // 2) + 4
        B, N = case["B"], case["N"]
        keys = sum(_ragged(case["R"], B)) + B * min(case["n_gen"], RING)
        return {"bytes": keys * case["hk"] * 2 * row + B * N * D * 4 * (2 * case["hq"] + 2 * case["hk"]),
                "flops": 4 * D * case["hq"] * N * keys + 2 * D * case["hq"] * B * N * (N + 1)}
    if op == "probs":
        return {"bytes": 8 * case["T"] * case["V"], "flops": 4 * case["T"] * case["V"]}
    rows = 2 if case["draft"] else 1   # the row that the walk ends on: target (and draft) once
    return {"bytes": case["B"] * rows * 4 * case["V"], "flops": case["B"] * 4 * case["V"]}


# ---------------------------------------------------------------- inputs

def _quantise(x, kind):
    """Codes (int8, or two nibbles a byte) and scales of rows of 128, as a cache holds them."""
    top = 127 if kind == "int8" else 7
    s = x.abs().amax(-1) / torch.full((), top, device="cuda", dtype=x.dtype)   # a true division: by a number it is a product
    q = torch.where(s[..., None] > 0, x / s[..., None], torch.zeros_like(x)).round().clamp_(-top - (kind == "int4"), top)
    if kind == "int8":
        return q.to(torch.int8), s
    q = q.to(torch.int32) & 15
    return (q[..., 0::2] | (q[..., 1::2] << 4)).to(torch.uint8), s


def _trees(case, seed):
    """Parents (-1: the last committed token) of N nodes in each sequence."""
    rng = random.Random(seed)
    B, N = case["B"], case["N"]
    if case["chain"]:
        return [[i - 1 for i in range(N)] for _ in range(B)]
    return [[rng.randint(max(-1, i - 4), i - 1) for i in range(N)] for _ in range(B)]


def _cache(B, heads, cap, kind, gen):
    k = torch.randn(B, heads, cap, D, device="cuda", generator=gen)
    kq = _quantise(k, kind)
    del k
    v = torch.randn(B, heads, cap, D, device="cuda", generator=gen)
    return kq + _quantise(v, kind)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    randn = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    s, op = {"case": case}, case["op"]
    if op == "rope":
        T, hq, hk = case["T"], case["hq"], case["hk"]
        if case["packed"]:   # the rows of a fused projection: q, k and v of a token side by side
            rows = randn(T, (hq + 2 * hk) * D)
            s["q"] = rows[:, :hq * D].view(T, hq, D)
            s["k"] = rows[:, hq * D:(hq + hk) * D].view(T, hk, D)
        else:
            s["q"], s["k"] = randn(T, hq, D), randn(T, hk, D)
        s["pos"] = (torch.arange(T, device="cuda") + 500 * (seed % 64)).to(torch.int32)
        s["gamma_q"], s["gamma_k"] = (1 + 0.2 * randn(D), 1 + 0.2 * randn(D)) if case["norm"] else (None, None)
        s["q_out"], s["k_out"] = torch.empty(T, hq, D, device="cuda"), torch.empty(T, hk, D, device="cuda")
    elif op == "kv":
        B, new, cap = case["B"], case["new"], case["cap"]
        s["k"], s["v"] = randn(B * new, case["heads"], D), randn(B * new, case["heads"], D)
        s["count"] = _ints(_counts(case))
        s["start"] = _ints([600 + 7 * b for b in range(B)] if case["wrap"] else [0] * B)
        s["len"] = _ints(_valid(case))
        # committed drafts are picked by index from a sequence's rows; a prompt's rows are taken as they are
        s["index"] = torch.rand(B, new, device="cuda", generator=gen).argsort(1).to(torch.int32) if case["wrap"] else None
        s["cache"] = _cache(B, case["heads"], cap, case["kind"], gen)
        s["k_out"] = torch.zeros(B, case["heads"], cap, D, device="cuda")
        s["v_out"] = torch.zeros(B, case["heads"], cap, D, device="cuda")
    elif op == "tree":
        B, N, R = case["B"], case["N"], case["R"]
        s["q"] = randn(B, N, case["hq"], D)
        s["k_new"], s["v_new"] = randn(B, N, case["hk"], D), randn(B, N, case["hk"], D)
        s["ref"] = _cache(B, case["hk"], R, case["kind"], gen)
        s["ring"] = _cache(B, case["hk"], RING, case["kind"], gen)
        s["ref_len"] = _ints(_ragged(R, B))
        s["n_gen"] = _ints([max(0, case["n_gen"] - 3 * b) for b in range(B)])
        s["parent"] = _ints(_trees(case, seed))
        s["n_nodes"] = _ints([N - (b % 2 if N > 1 else 0) for b in range(B)])   # every other tree is one node short
        s["out"] = torch.zeros(B, N, case["hq"], D, device="cuda")
    elif op == "probs":
        s["logits"] = 3 * randn(case["T"], case["V"])
        s["probs"] = torch.empty_like(s["logits"])
    else:
        B, N, V = case["B"], case["N"], case["V"]
        base = 3 * randn(B, N + 1, V)
        s["target"] = torch.softmax(base, -1)
        base += 0.7 * randn(B, N + 1, V)   # a draft that knows the target fairly well
        draft = torch.softmax(base[:, :N], -1)
        del base
        s["parent"] = _ints(_trees(case, seed))
        # a node's token is drawn from the draft's distribution behind its parent
        picks = torch.multinomial(draft.view(B * N, V), N, replacement=True, generator=gen).view(B, N, N)
        s["tokens"] = picks.gather(1, s["parent"].long()[:, None] + 1)[:, 0].to(torch.int32)
        s["draft"] = draft if case["draft"] else None
        s["n_nodes"] = _ints([N - (b % 2 if N > 1 else 0) for b in range(B)])
        s["u"] = torch.rand(B, N + 1, device="cuda", generator=gen)
        s["n_accept"] = torch.empty(B, dtype=torch.int32, device="cuda")
        s["path"] = torch.empty(B, N, dtype=torch.int32, device="cuda")
        s["next"] = torch.empty(B, dtype=torch.int32, device="cuda")
    return s


def _valid(case):
    """Rows of each sequence that hold a token after the write of a kv case."""
    if case["wrap"]:
        return [min(case["cap"], 600 + 7 * b + n) for b, n in enumerate(_counts(case))]
    return _counts(case)


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"rope": _rope_own, "kv": _kv_own, "tree": _tree_own, "probs": _probs_own, "verify": _verify_own}[op](s)
    return {"rope": _rope, "kv": _kv, "tree": _tree, "probs": _probs, "verify": _verify}[op](s)


def _rope_own(s):
    from weight_quantized_expert_b200 import api
    c = s["case"]
    return api.focr_qk_norm_rope(s["q"], s["k"], s["pos"], s["gamma_q"], s["gamma_k"], eps=EPS, theta=THETA,
                                 rot_dim=c["rot"], interleaved=c["interleaved"], norm=c["norm"], q_out=s["q_out"],
                                 k_out=s["k_out"])


def _kv_own(s):
    from weight_quantized_expert_b200 import api
    c = s["case"]
    api.focr_kv_write(s["cache"], s["k"], s["v"], s["count"], s["start"], index=s["index"], n_max=c["new"], wrap=c["wrap"])
    return api.focr_kv_read(s["cache"], s["len"], s["k_out"], s["v_out"])


def _tree_own(s):
    from weight_quantized_expert_b200 import api
    return api.focr_rswa_tree(s["q"], s["k_new"], s["v_new"], s["ref"], s["ref_len"], s["ring"], s["n_gen"],
                              s["parent"], s["n_nodes"], out=s["out"])


def _probs_own(s):
    from weight_quantized_expert_b200 import api
    return api.focr_token_probs(s["logits"], s["case"]["temperature"], out=s["probs"])


def _verify_own(s):
    from weight_quantized_expert_b200 import api
    return api.focr_spec_verify(s["target"], s["draft"], s["tokens"], s["parent"], s["n_nodes"], s["u"],
                                n_accept=s["n_accept"], path=s["path"], next_token=s["next"])


# ---------------------------------------------------------------- plain forms

def _rope(s):
    c = s["case"]
    r = c["rot"]
    freq = THETA ** (-torch.arange(0, r, 2, device="cuda", dtype=torch.float64) / r)
    angle = s["pos"].double()[:, None] * freq          # far positions need the angles in 64 bits
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turn(x, gamma):
        if c["norm"]:
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * gamma
        a, b = (x[..., 0:r:2], x[..., 1:r:2]) if c["interleaved"] else (x[..., :r // 2], x[..., r // 2:r])
        pair = (a * cos - b * sin, b * cos + a * sin)
        y = torch.stack(pair, -1).flatten(-2) if c["interleaved"] else torch.cat(pair, -1)
        return torch.cat((y, x[..., r:]), -1)

    return turn(s["q"], s["gamma_q"]), turn(s["k"], s["gamma_k"])


def _values(codes, scale):
    """The fp32 values that codes and scales stand for."""
    if codes.dtype == torch.uint8:
        n = codes.to(torch.int32)
        n = torch.stack((n & 15, n >> 4), -1).flatten(-2)
        return (n - 16 * (n > 7)).float() * scale[..., None]
    return codes.float() * scale[..., None]


def _kv(s):
    c = s["case"]
    B, cap, new = c["B"], c["cap"], c["new"]
    row = torch.arange(cap, device="cuda")[None]
    count, start = s["count"].long()[:, None], s["start"].long()[:, None]
    # the token that ends up in each row of the cache: the last one of those that fall on it
    i = (row - start) % cap if c["wrap"] else row - start
    i = i + torch.div((count - 1 - i).clamp(min=0), cap, rounding_mode="floor") * cap if c["wrap"] else i
    hit = (i >= 0) & (i < count)
    i = i.clamp(0, new - 1)
    src = torch.arange(B, device="cuda")[:, None] * new + (i if s["index"] is None else s["index"].long().gather(1, i))
    keep = (row < s["len"][:, None])[:, None, :, None]
    outs = []
    for x, codes, scale, out in ((s["k"], s["cache"][0], s["cache"][1], s["k_out"]), (s["v"], s["cache"][2], s["cache"][3], s["v_out"])):
        q, f = _quantise(x[src].transpose(1, 2), c["kind"])
        codes.copy_(torch.where(hit[:, None, :, None], q, codes))
        scale.copy_(torch.where(hit[:, None], f, scale))
        outs.append(out.copy_(torch.where(keep, _values(codes, scale), out)))
    return tuple(outs)


def _tree(s):
    c = s["case"]
    B, N, R, hq, hk = c["B"], c["N"], c["R"], c["hq"], c["hk"]
    parent, n = s["parent"].long(), s["n_gen"].long()
    # ancestors: reach[b, i, j] = node j lies on the path from node i to the root (squared up to N steps)
    eye = torch.eye(N, device="cuda")
    reach = eye + (parent[..., None] == torch.arange(N, device="cuda")).float()
    for _ in range(max(1, (N - 1).bit_length())):
        reach = ((reach @ reach) > 0).float()
    depth = reach.sum(-1).long() - 1
    slot = torch.arange(RING, device="cuda")
    p = n[:, None] - 1 - (n[:, None] - 1 - slot) % RING            # the last token before n that lies in the slot
    window = (p[:, None] >= 0) & (p[:, None] > n[:, None, None] + depth[..., None] - RING)
    ref = (torch.arange(R, device="cuda") < s["ref_len"][:, None])[:, None].expand(B, N, R)
    mask = torch.cat((ref, window, reach > 0), -1)[:, None, :, None].expand(B, hk, N, hq // hk, -1).flatten(2, 3)
    k = torch.cat((_values(*s["ref"][:2]), _values(*s["ring"][:2]), s["k_new"].transpose(1, 2)), 2)
    q = s["q"].view(B, N, hk, hq // hk, D).transpose(1, 2).flatten(2, 3)
    w = (q @ k.transpose(-1, -2) / math.sqrt(D)).masked_fill(~mask, -math.inf)
    del k
    w = (w - w.amax(-1, keepdim=True)).exp()
    v = torch.cat((_values(*s["ref"][2:]), _values(*s["ring"][2:]), s["v_new"].transpose(1, 2)), 2)
    o = (w @ v / w.sum(-1, keepdim=True)).view(B, hk, N, hq // hk, D).transpose(1, 2).flatten(2, 3)
    live = (torch.arange(N, device="cuda") < s["n_nodes"][:, None])[..., None, None]
    return s["out"].copy_(torch.where(live, o, s["out"]))


def _probs(s):
    x = s["logits"] / s["case"]["temperature"]
    e = (x - x.amax(-1, keepdim=True)).exp()
    return torch.div(e, e.sum(-1, keepdim=True), out=s["probs"])


def _verify(s):
    """In 64 bits: the answers are whole numbers next to borders.  The nodes are walked in their order because a
    test depends on the one before: whether its parent was accepted, and how much mass its siblings left."""
    B, N, V = s["case"]["B"], s["case"]["N"], s["case"]["V"]
    at = torch.arange(B, device="cuda")
    cur = torch.full((B,), -1, device="cuda")
    c = torch.zeros(B, device="cuda", dtype=torch.float64)
    mass = torch.ones_like(c)
    gone = torch.zeros(B, V, device="cuda", dtype=torch.bool)      # rejected tokens of drafts without probabilities
    taken = torch.zeros(B, N, device="cuda", dtype=torch.bool)
    u = s["u"].double()

    def left(cur, c):
        p = s["target"][at, cur + 1].double()
        if s["draft"] is None:
            return p.masked_fill(gone, 0.0)
        return (p - c[:, None] * s["draft"][at, (cur + 1).clamp(max=N - 1)].double()).clamp(min=0)

    for i in range(N):
        tried = (s["parent"][:, i] == cur) & (i < s["n_nodes"])
        x = s["tokens"][:, i].long()
        w = left(cur, c)
        q = torch.ones_like(c) if s["draft"] is None else s["draft"][at, (cur + 1).clamp(max=N - 1), x].double()
        yes = tried & (u[:, i] * q * mass < w[at, x])
        no = tried & ~yes
        if s["draft"] is None:
            mass = torch.where(no, mass - w[at, x], mass)
            gone[at, x] |= no
        else:
            c = torch.where(no, c + mass, c)
            mass = torch.where(no, left(cur, c).sum(-1), mass)
        taken[:, i] = yes
        cur = torch.where(yes, i, cur)
        c, mass = torch.where(yes, 0.0, c), torch.where(yes, 1.0, mass)
        gone &= ~yes[:, None]
    w = left(cur, c)
    total = w.sum(-1, keepdim=True)
    w = torch.where(total > 0, w, s["target"][at, cur + 1].double())
    run_sum = w.cumsum(-1)
    t = (run_sum <= u[:, N:] * w.sum(-1, keepdim=True)).sum(-1)
    last = V - 1 - (w > 0).flip(-1).int().argmax(-1)
    n = taken.sum(-1)
    order = torch.where(taken, torch.arange(N, device="cuda"), N).sort(-1).values
    return n.int(), torch.where(order < N, order, -1).int(), torch.minimum(t, last).int()


# ---------------------------------------------------------------- in 64 bits, from the definitions

def exact(case, seed):
    of = {"rope": _exact_rope, "kv": _exact_kv, "tree": _exact_tree, "probs": _exact_probs}
    return of[case["op"]](case, prepare(case, seed)) if case["op"] in of else None   # a verification gives whole numbers


def _exact_rope(case, s):
    r = case["rot"]
    i = torch.arange(D, device="cuda")
    half = r // 2
    # the partner of each dimension, its frequency and the sign of the partner's part
    if case["interleaved"]:
        partner, pair, sign = i ^ 1, i // 2, torch.where(i % 2 == 0, -1.0, 1.0)
    else:
        partner, pair, sign = torch.where(i < half, i + half, i - half), torch.where(i < half, i, i - half), torch.where(i < half, -1.0, 1.0)
    angle = s["pos"].double()[:, None] * torch.exp(-2.0 * pair.double() / r * math.log(THETA))
    cos, sin = torch.cos(angle)[:, None], (sign.double() * torch.sin(angle))[:, None]
    outs = []
    for x, g in ((s["q"].double(), s["gamma_q"]), (s["k"].double(), s["gamma_k"])):
        if case["norm"]:
            x = x * torch.rsqrt(x.square().sum(-1, keepdim=True) / D + EPS) * g.double()
        y = x * cos + x[..., partner.clamp(0, D - 1)] * sin
        outs.append(torch.where(i < r, y, x))
    return tuple(outs)


def _exact_rows(codes, scale):
    """Rows of a cache in 64 bits, from bytes."""
    b = codes.to(torch.int64)
    if codes.dtype == torch.uint8:
        v = torch.empty(*b.shape[:-1], 2 * b.shape[-1], dtype=torch.int64, device=b.device)
        v[..., 0::2], v[..., 1::2] = b % 16, b // 16
        b = torch.where(v >= 8, v - 16, v)
    return b.double() * scale.double()[..., None]


def _exact_kv(case, s):
    """A scale is the row's largest magnitude over 127 or 7, rounded to 32 bits; a code is the quotient, rounded to
    32 bits and then to the nearest whole number, ties to even."""
    B, cap, new, lo, hi = case["B"], case["cap"], case["new"], *((-127, 127) if case["kind"] == "int8" else (-8, 7))
    outs = []
    for x, codes, scale in ((s["k"], *s["cache"][:2]), (s["v"], *s["cache"][2:])):
        out = torch.zeros(B, case["heads"], cap, D, device="cuda", dtype=torch.float64)
        for b, (count, valid) in enumerate(zip(_counts(case), _valid(case))):
            rows = x[b * new:(b + 1) * new]
            rows = (rows[:count] if s["index"] is None else rows[s["index"][b, :count].long()]).double()
            f = (rows.abs().amax(-1, keepdim=True) / hi).float().double()
            value = torch.round((rows / f).float().double()).clamp(lo, hi) * f
            out[b, :, :valid] = _exact_rows(codes[b], scale[b])[:, :valid]
            first = 600 + 7 * b if case["wrap"] else 0
            keep = min(count, cap)
            place = (torch.arange(count - keep, count, device="cuda") + first) % cap
            out[b, :, place] = value[count - keep:].transpose(0, 1)
        outs.append(out)
    return tuple(outs)


def _exact_tree(case, s):
    B, N, hq, hk = case["B"], case["N"], case["hq"], case["hk"]
    g = hq // hk
    out = torch.zeros(B, N, hq, D, device="cuda", dtype=torch.float64)
    parents, nodes = s["parent"].tolist(), s["n_nodes"].tolist()
    for b, (R, n) in enumerate(zip(s["ref_len"].tolist(), s["n_gen"].tolist())):
        tokens = list(range(max(0, n - RING), n))
        slots = [t % RING for t in tokens]
        seen = torch.zeros(nodes[b], R + len(tokens) + N, dtype=torch.bool)
        seen[:, :R] = True
        for i in range(nodes[b]):
            line, j = [], i
            while j >= 0:
                line.append(j)
                j = parents[b][j]
            here = n + len(line) - 1   # the node's position; its window ends with itself
            seen[i, R:R + len(tokens)] = torch.tensor([t > here - RING for t in tokens], dtype=torch.bool)
            seen[i, [R + len(tokens) + j for j in line]] = True
        seen = seen.cuda()
        for h in range(hk):
            k, v = (torch.cat((_exact_rows(s["ref"][j][b, h, :R], s["ref"][j + 1][b, h, :R]),
                               _exact_rows(s["ring"][j][b, h, slots], s["ring"][j + 1][b, h, slots]),
                               s[new][b, :, h].double())) for j, new in ((0, "k_new"), (2, "v_new")))
            for x in range(h * g, h * g + g):
                score = torch.einsum("nd,kd->nk", s["q"][b, :nodes[b], x].double(), k) * D ** -0.5
                score[~seen] = -math.inf
                out[b, :nodes[b], x] = torch.softmax(score, -1) @ v
    return out


def _exact_probs(case, s):
    return torch.softmax(s["logits"].double() / case["temperature"], -1)

