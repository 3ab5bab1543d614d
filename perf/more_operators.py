"""Performance cases of the draft side of speculative decoding.

Three operators on rows of logits, each with a plain form in elementary torch operations and
the framework's own call:

  sample   tokens drawn under temperature, top-k, top-p and min-p from given uniforms, with the
           distribution that they were drawn from (the q that the verify step takes), or the
           logits with what the filters remove at -infinity (the target's side of the same)
  top      each row's k largest logits, their tokens and the row's log-sum-exp: what a verify
           step leaves of the target to train the draft with
  distill  the draft's divergence from such a record, and its gradient

The vocabularies and batches are those of the framework's verify workloads (V = 32000, 128256,
152064; B=1 gamma=4 float32; B=64 gamma=5; B=256 gamma=8; trees, B=32), and odd ones.

Of the filters, in this order: top-k keeps a row's k largest logits; top-p the shortest run of
the largest of those that holds at least that share of their mass; min-p what has at least that
share of the largest one's probability. Equal logits rank by index. A draw takes the first
token, by index, whose cumulative mass is above u times the whole.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    def sample(name, **k):
        base = dict(op="sample", R=1, draws=1, give="probs", dtype="bf16", logits="zipf", pad=0,
                    top_k=0, top_p=1.0, min_p=0.0, temperature=0.8, mixed=False)
        base.update(k)
        return dict(base, name=name)

    def top(name, **k):
        base = dict(op="top", dtype="bf16", logits="zipf", pad=0, temperature=1.0)
        base.update(k)
        return dict(base, name=name)

    def distill(name, **k):
        base = dict(op="distill", dtype="bf16", logits="zipf", pad=0, temperature=1.0, rest=True,
                    skip=0.0)
        base.update(k)
        return dict(base, name=name)

    return [
        # one user's draft takes its next token, the usual filters (latency)
        sample("sample_b1_v32000_f32", B=1, V=32000, dtype="f32", top_k=40, top_p=0.95),
        # a draft step of a served batch, every request with its own filters, greedy ones too
        sample("sample_b64_v32000_mixed", B=64, V=32000, top_k=50, top_p=0.9, min_p=0.02, mixed=True),
        # a draft step of the large batch, nucleus sampling over the whole vocabulary
        sample("sample_b256_v128256_top_p", B=256, V=128256, top_p=0.9),
        # children of tree nodes: three draws from each row, flat rows, no filter
        sample("sample_tree_b32_r21_v128256", B=32, R=21, V=128256, draws=3, logits="normal", temperature=1.0),
        # the target's rows of the large verify step under the draft's filter, flat rows
        sample("filter_b256_r9_v128256", B=256, R=9, V=128256, draws=0, give="logits", logits="normal",
               top_p=0.95, min_p=0.001, temperature=0.7),
        # what one user's verify step leaves for training
        top("top_b1_r5_v32000_f32", B=1, R=5, V=32000, dtype="f32", k=16),
        # the same of a served batch, padded rows
        top("top_b64_r6_v32003", B=64, R=6, V=32003, pad=61, k=64),
        # the same of the large verify step
        top("top_b256_r9_v128256", B=256, R=9, V=128256, k=64),
        # a few positions of one request, float32
        distill("distill_b1_r33_v32000_f32", B=1, R=33, V=32000, dtype="f32", k=16),
        # a training batch at a softer temperature, teacher renormalised over its entries, a
        # quarter of the positions without weight
        distill("distill_b16_r255_v32003_soft", B=16, R=255, V=32003, k=200, rest=False, skip=0.25,
                temperature=2.0),
        # a training batch over the large vocabulary
        distill("distill_b8_r512_v128256", B=8, R=512, V=128256, k=64),
        # the same in float32, fewer positions, flat rows
        distill("distill_b4_r127_v152064_f32", B=4, R=127, V=152064, dtype="f32", k=128, logits="normal"),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("sample", "sample", "top", "distill"))
    dtype = "f32" if rng.random() < 0.3 else "bf16"
    V = rng.choice((32000, 128256, 152064, _log_uniform(rng, 1000, 152064), _log_uniform(rng, 1000, 152064) | 1))
    # no more elements than the largest listed case has
    most = int((1.2e8 if op == "sample" else 2.0e8) / V / (2 if dtype == "f32" else 1))
    rows = _log_uniform(rng, 1, most)
    B = rows if rng.random() < 0.4 else _log_uniform(rng, 1, rows)
    c = dict(op=op, B=B, R=max(1, min(4096, rows // B)), V=V, dtype=dtype,
             logits=rng.choice(("zipf", "zipf", "normal")), pad=rng.choice((0, 0, rng.randint(1, 129))))
    if op == "sample":
        give = rng.choice(("probs", "probs", "logits", "none"))
        return dict(c, draws=0 if give == "logits" else rng.randint(1, 4), give=give,
                    top_k=rng.choice((0, 0, 1, _log_uniform(rng, 2, 1000))),
                    top_p=rng.choice((1.0, 1.0, 0.8, 0.9, 0.95, 0.99)),
                    min_p=rng.choice((0.0, 0.0, 0.001, 0.05)),
                    temperature=rng.choice((0.3, 0.7, 1.0, 1.5)), mixed=rng.random() < 0.5)
    k = _log_uniform(rng, 1, 512)
    if op == "top":
        return dict(c, k=k, temperature=rng.choice((0.7, 1.0, 2.0)))
    return dict(c, k=k, rest=rng.random() < 0.6, skip=rng.choice((0.0, 0.0, 0.5)),
                temperature=rng.choice((1.0, 1.0, 2.0)))


# ---- inputs ----

def _logits(g, c):
    """Rows [B, R, V] of a buffer whose rows are `pad` elements longer: falling like the tokens'
    frequencies in text, each row in an order of its own, or all tokens alike."""
    B, R, V = c["B"], c["R"], c["V"]
    buf = torch.empty((B, R, V + c["pad"]), dtype=DTYPES[c["dtype"]], device="cuda")
    order = torch.randperm(V, generator=g, device="cuda")
    level = -1.1 * torch.log(order.float() + 1.0)
    shift = torch.randint(0, V, (B, R), generator=g, device="cuda")
    step = max(1, 2 ** 27 // (R * V))
    for b in range(0, B, step):
        n = min(step, B - b)
        x = torch.randn((n, R, V), generator=g, device="cuda")
        if c["logits"] == "zipf":
            at = (torch.arange(V, device="cuda") + shift[b:b + n, :, None]) % V
            x += level[at]
        else:
            x *= 2.0
        buf[b:b + n, :, :V] = x.to(buf.dtype)
    return buf[:, :, :V]


def _uniforms(g, shape):
    """Values strictly inside (0, 1), exact in float32."""
    k = torch.randint(0, 2 ** 23, shape, generator=g, device="cuda")
    return ((k.double() + 0.5) * 2.0 ** -23).float()


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c, "x": _logits(g, c)}
    B, R, V = c["B"], c["R"], c["V"]
    if c["op"] == "sample":
        T = torch.full((B,), c["temperature"], device="cuda")
        k = torch.full((B,), c["top_k"], dtype=torch.int32, device="cuda")
        p = torch.full((B,), c["top_p"], device="cuda")
        m = torch.full((B,), c["min_p"], device="cuda")
        if c["mixed"]:  # every request its own: some greedy, some without one filter or another
            T = T * (0.5 + torch.rand(B, generator=g, device="cuda"))
            off = torch.rand((4, B), generator=g, device="cuda")
            T = torch.where(off[0] < 0.1, 0.0, T)
            k = torch.where(off[1] < 0.3, 0, k)
            p = torch.where(off[2] < 0.3, 1.0, p)
            m = torch.where(off[3] < 0.3, 0.0, m)
        s.update(T=T, k=k if c["top_k"] else None, p=p if c["top_p"] < 1.0 else None,
                 m=m if c["min_p"] else None, u=_uniforms(g, (B, R, c["draws"])))
    if c["op"] == "distill":
        # the teacher differs from the draft by as much as its logits vary from row to row
        t, K = c["temperature"], min(c["k"], V)
        s["z"] = torch.empty((B, R, K), device="cuda")
        s["ids"] = torch.empty((B, R, K), dtype=torch.int32, device="cuda")
        s["lse"] = torch.empty((B, R), device="cuda")
        step = max(1, 2 ** 27 // (R * V))
        for b in range(0, B, step):
            x = s["x"][b:b + step]
            x = x + torch.randn(x.shape, generator=g, device="cuda")
            z, ids = x.topk(K, dim=-1)
            s["z"][b:b + step], s["ids"][b:b + step] = z, ids.int()
            s["lse"][b:b + step] = torch.logsumexp(x / t, -1)
        if not c["rest"]:
            s["lse"] = None
        w = 0.5 + torch.rand((B, R), generator=g, device="cuda")
        s["w"] = torch.where(torch.rand((B, R), generator=g, device="cuda") < c["skip"], 0.0, w / (B * R))
    return s


# ---- one pass ----

def run(state):
    op = state["case"]["op"]
    if own:
        return {"sample": _sample_own, "top": _top_own, "distill": _distill_own}[op](state)
    return {"sample": _sample_plain, "top": _top_plain, "distill": _distill_plain}[op](state)


def _sample_own(s):
    from speculative_decoding_verification_64_gb300 import binding
    c = s["case"]
    if c["give"] == "logits":
        r = binding.filter_logits(s["x"], s["T"], top_k=s["k"], top_p=s["p"], min_p=s["m"])
        return {"rows": r.rows, "kept": r.kept, "status": r.row_status}
    r = binding.sample(s["x"], s["T"], s["u"], top_k=s["k"], top_p=s["p"], min_p=s["m"],
                       probs=c["give"] == "probs")
    return {"tokens": r.tokens, "rows": r.rows, "kept": r.kept, "status": r.row_status}


def _top_own(s):
    from speculative_decoding_verification_64_gb300 import binding
    c = s["case"]
    r = binding.top_logits(s["x"], min(c["k"], c["V"]), temperature=c["temperature"])
    return {"values": r.values, "ids": r.ids, "lse": r.lse, "status": r.row_status}


def _distill_own(s):
    from speculative_decoding_verification_64_gb300 import binding
    r = binding.distill(s["x"], s["ids"], s["z"], lse=s["lse"], weight=s["w"],
                        temperature=s["case"]["temperature"], grad=True)
    return {"loss": r.loss, "grad": r.grad, "status": r.row_status}


# ---- plain forms ----

def _zeros32(*shape):
    return torch.zeros(shape, dtype=torch.int32, device="cuda")


def _of_request(v, R):
    """A value of every request [B] as one of every row [B R, 1]."""
    return v.repeat_interleave(R)[:, None]


def _sample_plain(s):
    # in 64 bits: the last kept token and the drawn one turn on sums over the whole row
    c, x = s["case"], s["x"]
    B, R, V = c["B"], c["R"], c["V"]
    x = x.reshape(B * R, V)
    T = _of_request(s["T"].double(), R)
    greedy = T == 0
    order = x.sort(dim=-1, descending=True, stable=True)
    z = order.values.double()
    w = torch.exp((z - z[:, :1]) / torch.where(greedy, 1.0, T))
    rank = torch.arange(V, device="cuda")
    keep = torch.ones_like(w, dtype=torch.bool)
    if s["k"] is not None:
        k = _of_request(s["k"], R)
        keep &= (rank < k) | (k == 0)
    if s["p"] is not None:
        p = _of_request(s["p"].double(), R)
        before = torch.where(keep, w, 0.0).cumsum(-1)
        whole = before[:, -1:].clone()
        before = before.roll(1, -1)
        before[:, 0] = 0.0
        keep &= (before < p * whole) | (p >= 1.0)
        del before
    if s["m"] is not None:
        keep &= w >= _of_request(s["m"].double(), R)
    keep = torch.where(greedy, rank == 0, keep)
    kept = keep.sum(-1).int().view(B, R)
    w = torch.where(keep, w, 0.0)
    del z, keep
    w = torch.zeros_like(w).scatter_(1, order.indices, w)  # by index again
    del order
    out = {"kept": kept, "status": _zeros32(B, R)}
    if c["give"] == "logits":
        out["rows"] = torch.where(w > 0, x, -math.inf).view(B, R, V)
        return out
    upto = w.cumsum(-1)
    whole = upto[:, -1:].clone()
    u = s["u"].double().view(B * R, -1)
    out["tokens"] = torch.searchsorted(upto, u * whole, right=True).int().view(B, R, -1)
    out["rows"] = (w / whole).to(x.dtype).view(B, R, V) if c["give"] == "probs" else None
    return out


def _top_plain(s):
    c = s["case"]
    x = s["x"].float()
    order = x.sort(dim=-1, descending=True, stable=True)
    K = min(c["k"], c["V"])
    m = order.values[..., :1]
    lse = m[..., 0] / c["temperature"] + torch.log(torch.exp((x - m) / c["temperature"]).sum(-1))
    return {"values": order.values[..., :K].clone(), "ids": order.indices[..., :K].int(), "lse": lse,
            "status": _zeros32(c["B"], c["R"])}


def _distill_plain(s):
    c, T = s["case"], s["case"]["temperature"]
    x = s["x"].float()
    x = (x - x.amax(-1, keepdim=True)) / T
    e = torch.exp(x)
    whole = e.sum(-1, keepdim=True)
    ids = s["ids"].long()
    at = x.gather(-1, ids) - torch.log(whole)                # ln s of the teacher's entries
    z = s["z"] / T
    if c["rest"]:
        log_p = z - s["lse"][..., None]
        p = torch.exp(log_p)
        r = (1.0 - p.double().sum(-1)).clamp(min=0.0).float()
        rest = e.scatter(-1, ids, 0.0).sum(-1) / whole[..., 0]
        loss = (p * (log_p - at)).sum(-1) + torch.where(r > 0, r * torch.log(r / rest), 0.0)
        y = e * ((1.0 - r / rest) / whole[..., 0])[..., None]
    else:
        z = z - z.amax(-1, keepdim=True)
        log_p = z - torch.log(torch.exp(z).sum(-1, keepdim=True))
        p = torch.exp(log_p)
        loss = (p * (log_p - at)).sum(-1)
        y = e / whole
    y.scatter_(-1, ids, torch.exp(at) - p)
    w = s["w"]
    y *= (w / T)[..., None]
    return {"loss": torch.where(w > 0, loss, 0.0), "grad": y.to(s["x"].dtype), "status": _zeros32(c["B"], c["R"])}


# ---- the definitions in 64 bits ----

def _exact_sample(s):
    c, x = s["case"], s["x"]
    B, R, V = c["B"], c["R"], c["V"]
    rows = torch.empty((B, R, V), dtype=torch.float64, device="cuda")
    T, ks, ps, ms = ([None] * B if v is None else v.tolist() for v in (s["T"], s["k"], s["p"], s["m"]))
    for b in range(B):
        for r in range(R):
            a = x[b, r].double()
            if T[b] == 0:
                one = torch.zeros_like(a)
                one[(a == a.max()).nonzero()[0]] = 1.0
                rows[b, r] = one
                continue
            # distinct values from the largest down, and how many tokens hold each
            v, of, n = torch.unique(a, return_inverse=True, return_counts=True)
            v, of, n = v.flip(0), len(v) - 1 - of, n.flip(0)
            w = ((v - v[0]) / T[b]).exp()
            left = V if not ks[b] else ks[b]
            n = (left - (n.cumsum(0) - n)).clamp(min=0).minimum(n)  # tokens of each that top-k keeps
            if ps[b] is not None and ps[b] < 1.0:
                mass = (w * n).cumsum(0)
                need = ps[b] * mass[-1] - (mass - w * n)
                n = (need / w).ceil().clamp(min=0).long().minimum(n)
                n[0] = n[0].clamp(min=1)
            if ms[b]:
                n = torch.where(w >= ms[b], n, 0)
            # of a value's tokens the first ones by index
            where = torch.sort(of, stable=True).indices
            first = torch.bincount(of, minlength=len(v)).cumsum(0).roll(1)
            first[0] = 0
            nth = torch.empty_like(of)
            nth[where] = torch.arange(V, device="cuda") - first[of[where]]
            p = torch.where(nth < n[of], w[of], 0.0)
            rows[b, r] = p / p.sum()
    return {"tokens": None, "rows": rows, "kept": None, "status": None}


def _exact_top(s):
    c = s["case"]
    lse = torch.stack([torch.logsumexp(row.double() / c["temperature"], -1) for row in s["x"]])
    values = torch.stack([row.double().topk(min(c["k"], c["V"]), dim=-1).values for row in s["x"]])
    return {"values": values, "ids": None, "lse": lse, "status": None}


def _exact_distill(s):
    c, T = s["case"], s["case"]["temperature"]
    B, R, V = c["B"], c["R"], c["V"]
    loss = torch.zeros((B, R), dtype=torch.float64, device="cuda")
    grad = torch.empty((B, R, V), dtype=torch.float64, device="cuda")
    step = max(1, 2 ** 25 // V)
    for b in range(B):
        for r in range(0, R, step):
            at = (b, slice(r, r + step))
            log_s = torch.log_softmax(s["x"][at].double() / T, -1)
            z = s["z"][at].double() / T
            log_p = z - s["lse"][at].double()[:, None] if c["rest"] else torch.log_softmax(z, -1)
            target = torch.zeros_like(log_s).scatter_(-1, s["ids"][at].long(), log_p.exp())
            some = (log_p.exp() * (log_p - log_s.gather(-1, s["ids"][at].long()))).sum(-1)
            if c["rest"]:
                other = torch.ones_like(log_s, dtype=torch.bool).scatter_(-1, s["ids"][at].long(), False)
                of = torch.where(other, log_s.exp(), 0.0)
                r_s = of.sum(-1, keepdim=True)
                r_t = (1.0 - log_p.exp().sum(-1, keepdim=True)).clamp(min=0.0)
                some = some + torch.where(r_t > 0, r_t * (r_t / r_s).log(), 0.0)[:, 0]
                target = target + r_t * of / r_s
            w = s["w"][at].double()
            loss[at] = torch.where(w > 0, some, 0.0)
            grad[at] = (log_s.exp() - target) * (w / T)[:, None]
    return {"loss": loss, "grad": grad, "status": None}


def exact(case, seed):
    if case["op"] == "sample" and (case["give"] != "probs" or case["B"] * case["R"] > 2000):
        return None  # what is computed there are whole numbers; thousands of rows one by one take too long
    s = prepare(case, seed)
    return {"sample": _exact_sample, "top": _exact_top, "distill": _exact_distill}[case["op"]](s)


# ---- what a pass cannot do without ----

def work(case):
    c = case
    rows = c["B"] * c["R"]
    n = rows * c["V"]
    es = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "sample":  # an exponential, a product and two sums for each element
        gives = 0 if c["give"] == "none" else n * es
        return {"bytes": n * es + gives + rows * (8 * c["draws"] + 8) + c["B"] * 16, "flops": 4 * n}
    if c["op"] == "top":
        return {"bytes": n * es + rows * (8 * c["k"] + 8), "flops": 4 * n}
    read = n * es * (1.0 - c["skip"])
    return {"bytes": read + n * es + rows * (8 * c["k"] + 16), "flops": 6 * n}
