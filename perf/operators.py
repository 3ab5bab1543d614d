"""Performance cases of the attention side of a verify step.

Three operators of the step that scores drafted tokens, each with a plain form in
elementary torch operations and the framework's own call:

  rope     rotary positions of q and k (both layouts, part of the head, either direction)
  append   accepted tokens' k and v into an 8-bit paged cache (e4m3 codes, one scale for
           each block of tokens and head)
  attend   attention of the drafted tokens of a chain or a tree over that cache and over
           one another, with an optional tanh cap, distance bias and window

The sizes are those of the framework's verify workloads (B=1 gamma=4 float32; B=64
gamma=5; B=256 gamma=8; B=512 gamma=4; trees of 64 nodes, depth 5, B=32) with ordinary
head layouts and context lengths.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
DEPTH = 5      # deepest node of a drafted tree
BRANCHING = 3  # most children of a node


def listed():
    def attend(name, **k):
        base = dict(op="attend", Hq=32, Hkv=8, D=128, block=64, dtype="bf16", ragged=True,
                    tree=False, softcap=0.0, bias=False, window=0)
        base.update(k)
        return dict(base, name=name)

    def rope(name, **k):
        base = dict(op="rope", Hq=32, Hkv=8, D=128, rot=128, dtype="bf16", interleaved=False,
                    backward=False, tree=False, start=4096, theta=10000.0, magnitude=1.0)
        base.update(k)
        return dict(base, name=name)

    def append(name, **k):
        base = dict(op="append", Hkv=8, D=128, block=64, dtype="bf16", tree=False)
        base.update(k)
        return dict(base, name=name)

    return [
        # one user, no draft: the single next token over a short context (latency)
        attend("attend_b1_n1_777", B=1, N=1, ctx=777, ragged=False),
        # one user, 4 drafted tokens, float32 activations
        attend("attend_b1_n5_f32_2048", B=1, N=5, ctx=2048, dtype="f32", ragged=False, block=32),
        # one user, 4 drafted tokens over a long document
        attend("attend_b1_n5_131071", B=1, N=5, ctx=131071, ragged=False),
        # a served batch, 5 drafted tokens each, contexts of every length
        attend("attend_b64_n6_4096", B=64, N=6, ctx=4096, block=16),
        # the large served batch, 8 drafted tokens each
        attend("attend_b256_n9_4096", B=256, N=9, ctx=4096),
        # drafted trees, capped scores
        attend("attend_tree_b32_n64_cap", B=32, N=64, ctx=4096, tree=True, softcap=50.0),
        # many short requests of a small model: narrow heads, distance bias, sliding window
        attend("attend_b512_n5_bias_window", B=512, N=5, Hq=16, Hkv=4, D=64, ctx=2000, block=32,
               bias=True, window=1024),
        # one user's 5 tokens, float32
        rope("rope_b1_n5_f32", B=1, N=5, dtype="f32"),
        # drafted trees, half of the head rotated in the interleaved layout
        rope("rope_tree_b32_n64_part", B=32, N=64, tree=True, rot=64, interleaved=True),
        # the gradient through long prompts, frequencies and magnitude scaled for their length
        rope("rope_backward_8x8191", B=8, N=8191, backward=True, start=100000, theta=500000.0,
             magnitude=1.2),
        # after a verify step: 1 to 9 accepted tokens of each request
        append("append_b256_n9", B=256, N=9, ctx=1000, commit=True),
        # prompts written at once
        append("append_prompt_8x8191", B=8, N=8191, ctx=100, commit=False),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("attend", "attend", "rope", "append"))
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    D = rng.choice((64, 96, 128))
    Hkv = rng.choice((1, 2, 4, 8))
    group = rng.choice((1, 2, 4, 5, 8))
    tree = rng.random() < 0.3
    block = rng.choice((16, 32, 64, 128))
    if op == "attend":
        B = _log_uniform(rng, 1, 512)
        N = rng.randint(8, 64) if tree else rng.choice((1, 1, _log_uniform(rng, 2, 33)))
        # no more cached tokens, and no more scores, than the largest listed case has
        tokens = min(2.0e8 / (Hkv * D), 1.2e8 / (Hkv * group * N))
        most = max(16, min(131072, int(tokens / B)))
        return dict(op=op, B=B, N=N, Hq=Hkv * group, Hkv=Hkv, D=D, block=block, dtype=dtype,
                    ctx=_log_uniform(rng, 16, most), ragged=rng.random() < 0.7, tree=tree,
                    softcap=rng.choice((0.0, 0.0, 30.0, 50.0)), bias=rng.random() < 0.25,
                    window=rng.choice((0, 0, 0, _log_uniform(rng, 16, 4096))))
    most = 2 ** 25 // (Hkv * D * (group + 1 if op == "rope" else 2))  # tokens in all
    B = _log_uniform(rng, 1, min(512, most))
    N = rng.randint(8, 64) if tree else _log_uniform(rng, 1, max(1, min(8191, most // B)))
    N = max(1, min(N, most // B))
    if op == "rope":
        return dict(op=op, B=B, N=N, Hq=Hkv * group, Hkv=Hkv, D=D, rot=rng.choice((D, D, D // 2)),
                    dtype=dtype, interleaved=rng.random() < 0.5, backward=rng.random() < 0.3,
                    tree=tree, start=_log_uniform(rng, 1, 1000000),
                    theta=rng.choice((10000.0, 500000.0)), magnitude=rng.choice((1.0, 1.2)))
    return dict(op=op, B=B, N=N, Hkv=Hkv, D=D, block=block, dtype=dtype, tree=tree,
                ctx=_log_uniform(rng, 1, 1000), commit=tree or N <= 33)


# ---- sizes that a case fixes (another seed shuffles them over the requests) ----

def _lens(c):
    """Cached tokens of each request: the whole of `ctx`, or every share of it, none and one too."""
    B, ctx = c["B"], c["ctx"]
    if not c.get("ragged", True):
        return [ctx] * B
    lens = [int(ctx * ((b * 0.6180339887498949) % 1.0)) for b in range(B)]
    lens[0] = ctx
    if B >= 8:
        lens[1], lens[2] = 0, 1
    return lens


def _counts(c):
    """Tokens that each request appends."""
    B, N = c["B"], c["N"]
    if not c["commit"]:
        return [N] * B
    most = min(N, DEPTH + 1) if c["tree"] else N
    return [1 + (b * 7) % most for b in range(B)]


def _trees(rng, B, N):
    """Random trees of N nodes, at most DEPTH deep: parents, and one root-to-leaf path of each."""
    parents, paths = [], []
    for _ in range(B):
        parent, depth, kids, free = [-1], [0], [0], [0]
        for n in range(1, N):
            at = rng.randrange(len(free))
            p = free[at]
            parent.append(p)
            depth.append(depth[p] + 1)
            kids.append(0)
            kids[p] += 1
            if kids[p] == BRANCHING:
                free[at] = free[-1]
                free.pop()
            if depth[n] < DEPTH:
                free.append(n)
        n = max(range(N), key=lambda i: (depth[i], rng.random()))
        path = [n]
        while parent[path[-1]] >= 0:
            path.append(parent[path[-1]])
        paths.append((path[::-1] + [-1] * (DEPTH + 1))[:DEPTH + 1])
        parents.append(parent)
    return parents, paths


def _int(rows):
    return torch.tensor(rows, dtype=torch.int32).cuda()


def _frequencies(c):
    """Turns that each pair makes per position, in units of 2^-64 turns (two's complement)."""
    half = c["rot"] // 2
    turns = [c["theta"] ** (-i / half) / (2 * math.pi) for i in range(half)]
    words = [int(math.ldexp(t, 64)) for t in turns]
    return torch.tensor([w - 2 ** 64 if w >= 2 ** 63 else w for w in words], dtype=torch.int64).cuda()


# ---- inputs ----

def _pool(g, n_blocks, c):
    """A pool of 8-bit blocks and their scales, of values of the size of keys and values."""
    shape = (n_blocks, c["Hkv"], c["block"], c["D"])
    codes = torch.empty(shape, dtype=torch.uint8, device="cuda")
    step = max(1, 2 ** 27 // (shape[1] * shape[2] * shape[3]))
    for at in range(0, n_blocks, step):
        x = torch.randn((min(step, n_blocks - at),) + shape[1:], generator=g, device="cuda")
        codes[at:at + step] = (x * 64).to(torch.float8_e4m3fn).view(torch.uint8)
    scale = torch.exp2(torch.randint(-7, -4, shape[:2], generator=g, device="cuda").float())
    return codes, scale


def _table(rng, lens, more, block):
    """Block tables with -1 in the unused entries, and how many blocks there are."""
    need = [-(-(n + m) // block) for n, m in zip(lens, more)]
    ids = list(range(sum(need)))
    rng.shuffle(ids)
    rows, at = [], 0
    for n in need:
        rows.append(ids[at:at + n] + [-1] * (max(need) - n))
        at += n
    return rows, len(ids) + 1  # one block that belongs to nobody


def prepare(case, seed):
    c = dict(case)
    rng = random.Random(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c}
    B, N, D, Hkv = c["B"], c["N"], c["D"], c["Hkv"]
    dt = DTYPES[c["dtype"]]
    s["parent"], s["path"] = None, None
    if c["tree"]:
        parents, paths = _trees(rng, B, N)
        s["parent"], s["path"] = _int(parents), _int(paths)
    if c["op"] == "append":
        lens, counts = [c["ctx"] * (b + 1) // B for b in range(B)], _counts(c)
    else:
        lens, counts = _lens(c) if c["op"] == "attend" else [c["start"]] * B, [N] * B
    order = list(range(B))
    rng.shuffle(order)
    lens, counts = [lens[b] for b in order], [counts[b] for b in order]
    s["len"] = _int(lens)
    Hq = c.get("Hq", Hkv)
    qkv = torch.randn((B, N, Hq + 2 * Hkv, D), generator=g, device="cuda").to(dt)  # a fused projection
    s["q"], s["k"], s["v"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    if c["op"] == "rope":
        s["freq"] = _frequencies(c)
        s["positions"] = None if c["tree"] else s["len"][:, None] + torch.arange(N, dtype=torch.int32, device="cuda")
        return s
    s["rows"], n_blocks = _table(rng, lens, counts if c["op"] == "append" else [1] * B, c["block"])
    s["table"] = _int(s["rows"])
    s["kc"], s["ks"] = _pool(g, n_blocks, c)
    s["vc"], s["vs"] = _pool(g, n_blocks, c)
    if c["op"] == "append":
        s["count"] = _int([n - 1 for n in counts])  # accepted drafts; the token before them joins them
        if not c["tree"]:
            s["path"] = None
        return s
    # the first cached token attracts every query, as the first token of a text does
    u = torch.randint(0, 2, (Hkv, D), generator=g, device="cuda").float() * 2 - 1
    first = s["table"][:, 0].long()
    s["kc"][first, :, 0] = (u * 96).to(torch.float8_e4m3fn).view(torch.uint8)
    s["q"] = (s["q"].float() + 0.4 * u.repeat_interleave(Hq // Hkv, 0)).to(dt)
    s["k"] = s["k"].contiguous()  # q and k come from the rotary pass, v from the projection
    s["slopes"] = torch.tensor([2.0 ** (-8 * (h + 1) / Hq) for h in range(Hq)]).cuda() if c["bias"] else None
    return s


# ---- one pass ----

def run(state):
    op = state["case"]["op"]
    if own:
        return {"attend": _attend_own, "rope": _rope_own, "append": _append_own}[op](state)
    return {"attend": _attend_plain, "rope": _rope_plain, "append": _append_plain}[op](state)


def _cache(s):
    from speculative_decoding_verification_64_gb300 import binding
    if "cache" not in s:
        f8 = torch.float8_e4m3fn
        s["cache"] = binding.KVCache(s["kc"].view(f8), s["vc"].view(f8), s["ks"], s["vs"], s["table"], s["len"])
    return s["cache"]


def _attend_own(s):
    from speculative_decoding_verification_64_gb300 import binding
    c, cache = s["case"], _cache(s)
    if "workspace" not in s:
        s["workspace"] = binding.alloc_attend_workspace(s["q"], cache)
    r = binding.attend(s["q"], s["k"], s["v"], cache, parent=s["parent"], softcap=c["softcap"],
                       slopes=s["slopes"], window=c["window"], workspace=s["workspace"])
    return {"out": r.out, "lse": r.lse, "status": r.row_status}


def _rope_own(s):
    from speculative_decoding_verification_64_gb300 import binding
    c = s["case"]
    q, k = binding.rope(s["q"], s["k"], s["freq"], positions=s["positions"],
                        base=s["len"] if c["tree"] else None, parent=s["parent"],
                        interleaved=c["interleaved"], backward=c["backward"], magnitude=c["magnitude"])
    return {"q": q, "k": k}


def _append_own(s):
    from speculative_decoding_verification_64_gb300 import binding
    cache = _cache(s)
    r = binding.kv_append(s["k"], s["v"], cache, count=s["count"], extra=1, path=s["path"])
    return {"k": cache.k, "v": cache.v, "k_scale": cache.k_scale, "v_scale": cache.v_scale,
            "len": r.length, "status": r.row_status}


# ---- plain forms, in 32 bits ----

def _ancestors(parent, B, N):
    """[B, N, N]: node j is node n or above it (trees at most 8 deep)."""
    if parent is None:
        return torch.ones(N, N, dtype=torch.bool, device="cuda").tril().expand(B, N, N)
    up = (parent[:, :, None] == torch.arange(N, device="cuda")).float() + torch.eye(N, device="cuda")
    up = (up @ up > 0).float()
    up = (up @ up > 0).float()
    return up @ up > 0


def _values(codes, scale, table):
    """The cache's values [B, Hkv, T, D] in the order of the tokens."""
    x = codes[table].view(torch.float8_e4m3fn).float() * scale[table][..., None, None]
    return x.transpose(1, 2).flatten(2, 3)


def _attend_plain(s):
    c = s["case"]
    B, N, Hq, Hkv, D = c["B"], c["N"], c["Hq"], c["Hkv"], c["D"]
    G = Hq // Hkv
    table = s["table"].clamp(min=0).long()
    T = table.shape[1] * c["block"]
    at = torch.arange(T, device="cuda")
    held = at < s["len"][:, None]                                         # [B, T]
    k = torch.cat((_values(s["kc"], s["ks"], table), s["k"].float().transpose(1, 2)), 2)
    v = torch.cat((torch.where(held[:, None, :, None], _values(s["vc"], s["vs"], table), 0.0),
                   s["v"].float().transpose(1, 2)), 2)
    q = s["q"].float().view(B, N, Hkv, G, D).transpose(1, 2).flatten(2, 3)  # [B, Hkv, N G, D]
    x = q @ k.transpose(2, 3) * D ** -0.5
    if c["softcap"]:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    x = x.view(B, Hkv, N, G, T + N)
    sees = _ancestors(s["parent"], B, N)
    depth = sees.sum(2) - 1                                               # [B, N]
    away = torch.cat(((s["len"][:, None] + depth)[:, :, None] - at, depth[:, :, None] - depth[:, None, :]), 2)
    mask = torch.cat((held[:, None, :].expand(B, N, T), sees), 2)
    if c["window"]:
        mask = mask & (away < c["window"])
    if c["bias"]:
        x = x - s["slopes"].view(1, Hkv, 1, G, 1) * away[:, None, :, None, :].float()
    x = x.masked_fill(~mask[:, None, :, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - top)
    total = x.sum(-1, keepdim=True)
    out = (x.flatten(2, 3) @ v).view(B, Hkv, N, G, D) / total
    out = out.transpose(1, 2).reshape(B, N, Hq, D).to(s["q"].dtype)
    lse = (top + torch.log(total)).squeeze(-1).transpose(1, 2).reshape(B, N, Hq)
    return {"out": out, "lse": lse, "status": torch.zeros(B, dtype=torch.int32, device="cuda")}


def _rotate_plain(x, cos, sin, c):
    rot = c["rot"]
    y = x.float()
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if c["interleaved"] else (y[..., :rot // 2], y[..., rot // 2:rot])
    u, w = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((u, w), -1).flatten(-2) if c["interleaved"] else torch.cat((u, w), -1)
    return torch.cat((turned, y[..., rot:]), -1).to(x.dtype)


def _rope_plain(s):
    c = s["case"]
    position = s["positions"]
    if position is None:
        position = s["len"][:, None] + _ancestors(s["parent"], c["B"], c["N"]).sum(2) - 1
    turn = position.long()[..., None] * s["freq"] >> 32                   # whole turns wrap away
    angle = turn.float() * (math.pi / 2 ** 31)
    if c["backward"]:
        angle = -angle
    cos = torch.cos(angle)[:, :, None] * c["magnitude"]
    sin = torch.sin(angle)[:, :, None] * c["magnitude"]
    return {"q": _rotate_plain(s["q"], cos, sin, c), "k": _rotate_plain(s["k"], cos, sin, c)}


def _scale_plain(amax):
    """The smallest power of two, 2^-100 at least, with amax <= 448 times it."""
    m, e = torch.frexp(amax / 448)
    e = torch.where(m == 0.5, e - 1, e)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), 0.0).clamp(min=2.0 ** -100)


def _append_side(x, codes, scale, s, lens, count, first, ids, spare):
    """One of k and v: the touched blocks of each request, whole, and back into the pool."""
    c = s["case"]
    B, N, block = c["B"], c["N"], c["block"]
    M = ids.shape[1]
    at = first[:, None] * block + torch.arange(M * block, device="cuda")   # position of each slot
    old, new = at < lens, (at >= lens) & (at < lens + count)
    j = (at - lens).clamp(0, N - 1)
    if s["path"] is not None:
        j = s["path"].long().gather(1, j.clamp(max=s["path"].shape[1] - 1)).clamp(min=0)
    fresh = x.float().gather(1, j[:, :, None, None].expand(-1, -1, c["Hkv"], c["D"]))
    fresh = fresh.view(B, M, block, c["Hkv"], c["D"]).transpose(2, 3)      # [B, M, Hkv, block, D]
    old, new = (m.view(B, M, 1, block, 1) for m in (old, new))
    held, held_scale = codes[ids], scale[ids]
    amax = torch.where(new, fresh.abs(), 0.0).amax((3, 4))
    to = _scale_plain(amax)
    to = torch.where(old.any(3)[..., 0], torch.maximum(to, held_scale), to)
    to = torch.where(spare[:, :, None], held_scale, to)
    moved = held.view(torch.float8_e4m3fn).float() * (held_scale / to)[..., None, None]
    put = torch.where(new, fresh / to[..., None, None], moved).clamp(-448, 448).to(torch.float8_e4m3fn)
    codes[ids] = torch.where(((old | new) & ~spare[:, :, None, None, None]), put.view(torch.uint8), held)
    scale[ids] = to


def _append_plain(s):
    c = s["case"]
    block = c["block"]
    lens, count = s["len"].long()[:, None], s["count"].long()[:, None] + 1
    first = lens[:, 0] // block
    M = -(-(min(c["N"], s["path"].shape[1]) if s["path"] is not None else c["N"]) // block) + 1
    at = first[:, None] + torch.arange(M, device="cuda")
    spare = at * block >= lens + count                                    # blocks that get no token
    ids = s["table"].long().gather(1, at.clamp(max=s["table"].shape[1] - 1))
    ids = torch.where(spare, s["kc"].shape[0] - 1, ids)
    _append_side(s["k"], s["kc"], s["ks"], s, lens, count, first, ids, spare)
    _append_side(s["v"], s["vc"], s["vs"], s, lens, count, first, ids, spare)
    f8 = torch.float8_e4m3fn
    return {"k": s["kc"].view(f8), "v": s["vc"].view(f8), "k_scale": s["ks"], "v_scale": s["vs"],
            "len": (lens + count)[:, 0].int(), "status": torch.zeros(c["B"], dtype=torch.int32, device="cuda")}


# ---- the definitions in 64 bits, request by request ----

def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _attend_exact, "rope": _rope_exact, "append": _append_exact}[case["op"]](s)


def _up(parent, n):
    """Node n and the nodes above it, n first."""
    chain = [n]
    while (parent[chain[-1]] if parent is not None else chain[-1] - 1) >= 0:
        chain.append(parent[chain[-1]] if parent is not None else chain[-1] - 1)
    return chain


def _attend_exact(s):
    c = s["case"]
    B, N, Hq, Hkv, D, block = (c[k] for k in ("B", "N", "Hq", "Hkv", "D", "block"))
    G = Hq // Hkv
    out = torch.zeros(B, N, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, N, Hq, dtype=torch.float64, device="cuda")
    lens = s["len"].tolist()
    parents = s["parent"].tolist() if s["parent"] is not None else [None] * B
    for b in range(B):
        n_held = lens[b]
        chains = [_up(parents[b], n) for n in range(N)]
        see = torch.zeros(N, N, dtype=torch.bool)
        for n, chain in enumerate(chains):
            see[n, chain] = True
        see = see.cuda()
        where = torch.tensor([n_held + len(chain) - 1 for chain in chains], device="cuda")
        ids = torch.tensor(s["rows"][b][:-(-n_held // block)], dtype=torch.long, device="cuda")
        both = []
        for codes, scale, fresh in ((s["kc"], s["ks"], s["k"]), (s["vc"], s["vs"], s["v"])):
            x = codes[ids].view(torch.float8_e4m3fn).double() * scale[ids].double()[:, :, None, None]
            x = x.permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :n_held]
            both.append(torch.cat((x, fresh[b].double().permute(1, 0, 2)), 1))
        far = where[:, None] - torch.cat((torch.arange(n_held, device="cuda"), where))[None, :]
        hidden = ~torch.cat((torch.ones(N, n_held, dtype=torch.bool, device="cuda"), see), 1)
        if c["window"]:
            hidden |= far >= c["window"]
        for h in range(Hq):
            z = s["q"][b, :, h].double() @ both[0][h // G].T / math.sqrt(D)
            if c["softcap"]:
                z = torch.tanh(z / c["softcap"]) * c["softcap"]
            if c["bias"]:
                z = z - s["slopes"][h].double() * far
            z[hidden] = -math.inf
            lse[b, :, h] = torch.logsumexp(z, 1)
            out[b, :, h] = torch.exp(z - lse[b, :, h, None]) @ both[1][h // G]
    return {"out": out, "lse": lse, "status": None}


def _rope_exact(s):
    c = s["case"]
    B, N, rot = c["B"], c["N"], c["rot"]
    if s["positions"] is not None:
        position = s["positions"].double()
    else:
        parents, lens = s["parent"].tolist(), s["len"].tolist()
        position = torch.tensor([[lens[b] + len(_up(parents[b], n)) - 1 for n in range(N)] for b in range(B)],
                                dtype=torch.float64, device="cuda")
    words = torch.tensor([w % 2 ** 64 / 2 ** 64 for w in s["freq"].tolist()], dtype=torch.float64, device="cuda")
    angle = torch.remainder(position[..., None] * words, 1.0)[:, :, None] * (2 * math.pi)
    turn = torch.polar(torch.full_like(angle, c["magnitude"]), -angle if c["backward"] else angle)
    got = {}
    for name in ("q", "k"):
        y = s[name].double().clone()
        half = rot // 2
        first, second = (slice(0, rot, 2), slice(1, rot, 2)) if c["interleaved"] else (slice(0, half), slice(half, rot))
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        got[name] = y
    return got


def _to_e4m3(x):
    """float64 values to the nearest e4m3 value, ties to even, at most 448 in size."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -30))).clamp(min=-6.0, max=8.0)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _append_exact(s):
    c = s["case"]
    block = c["block"]
    lens, counts = s["len"].tolist(), [n + 1 for n in s["count"].tolist()]
    paths = s["path"].tolist() if s["path"] is not None else None
    got = {"len": None, "status": None}
    for name, codes, scale, fresh in (("k", s["kc"], s["ks"], s["k"]), ("v", s["vc"], s["vs"], s["v"])):
        value, scale = codes.view(torch.float8_e4m3fn).double(), scale.double()
        for b in range(c["B"]):
            nodes = (paths[b] if paths is not None else list(range(c["N"])))[:counts[b]]
            x = fresh[b][torch.tensor(nodes, device="cuda")].double().transpose(0, 1)  # [Hkv, count, D]
            done = 0
            while done < counts[b]:
                slot, off = s["rows"][b][(lens[b] + done) // block], (lens[b] + done) % block
                take = min(block - off, counts[b] - done)
                part = x[:, done:done + take]
                need = torch.exp2(torch.ceil(torch.log2(part.abs().amax((1, 2)) / 448)).clamp(min=-100.0))
                if off:
                    need = torch.maximum(need, scale[slot])
                    value[slot, :, :off] = _to_e4m3(value[slot, :, :off] * (scale[slot] / need)[:, None, None])
                value[slot, :, off:off + take] = _to_e4m3(part / need[:, None, None])
                scale[slot] = need
                done += take
        got[name], got[name + "_scale"] = value, scale
    return got


# ---- what a pass cannot do without ----

def work(case):
    c = case
    es = 2 if c["dtype"] == "bf16" else 4
    B, N, D, Hkv = c["B"], c["N"], c["D"], c["Hkv"]
    if c["op"] == "rope":
        heads = B * N * (c["Hq"] + Hkv)
        return {"bytes": 2.0 * heads * D * es, "flops": 3.0 * heads * c["rot"]}
    if c["op"] == "append":
        tokens = sum(_counts(c))
        return {"bytes": 2.0 * tokens * Hkv * D * (es + 1), "flops": 2.0 * tokens * Hkv * D}
    Hq, held = c["Hq"], _lens(c)
    if c["window"]:
        held = [min(n, c["window"] + (DEPTH if c["tree"] else N) - 1) for n in held]
    seen = N * DEPTH / 2 if c["tree"] else N * (N + 1) / 2               # pairs of drafted tokens
    if c["window"]:
        pairs = sum(sum(min(n, max(0, c["window"] - 1)) for _ in range(N)) for n in _lens(c))
    else:
        pairs = N * sum(held)
    moved = 2.0 * sum(held) * Hkv * D + B * N * ((2 * Hq + 2 * Hkv) * D * es + 4 * Hq)
    return {"bytes": moved, "flops": 4.0 * D * Hq * (pairs + B * seen)}
