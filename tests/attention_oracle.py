"""Plain float64 forms of rotary positions, the 8-bit cache's append and the attention of
drafted tokens, request by request and without the library: what the GPU tests compare with."""
import math

import numpy as np
import torch

E4M3 = torch.float8_e4m3fn


def ancestors(parent, n):
    """Node n and the nodes above it, n first (parent None: a chain)."""
    up = [n]
    while up[-1] > 0:
        nxt = up[-1] - 1 if parent is None else int(parent[up[-1]])
        if nxt < 0:
            break
        up.append(nxt)
    return up


def rope(x, positions, freq, interleaved=False, backward=False, magnitude=1.0):
    """x [B, N, H, D] float64, positions [B, N] ints, freq: words of 2^-64 turns."""
    y = x.clone()
    half = len(freq)
    for i, word in enumerate(freq):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        for bb in range(x.shape[0]):
            for n in range(x.shape[1]):
                turn = (int(positions[bb][n]) * int(word)) % 2 ** 64 / 2.0 ** 64
                ang = 2 * math.pi * turn * (-1 if backward else 1)
                c, s = math.cos(ang) * magnitude, math.sin(ang) * magnitude
                y[bb, n, :, a] = x[bb, n, :, a] * c - x[bb, n, :, b] * s
                y[bb, n, :, b] = x[bb, n, :, b] * c + x[bb, n, :, a] * s
    return y


def to_e4m3(x):
    """float64 -> nearest e4m3 value, ties to even, saturating; NaN for what is not finite."""
    x = np.asarray(x, dtype=np.float64)
    ok = np.isfinite(x)
    a = np.abs(np.where(ok, x, 0.0))
    e = np.clip(np.floor(np.log2(np.maximum(a, 2.0 ** -60))), -6, 8)
    step = 2.0 ** (e - 3)
    r = np.minimum(np.rint(a / step) * step, 448.0)
    return np.where(ok, np.copysign(r, x), np.nan)


def scale_for(amax):
    """Smallest power of two s >= 2^-100 with amax <= 448 s."""
    if amax <= 448 * 2.0 ** -100:
        return 2.0 ** -100
    m, e = math.frexp(amax / 448.0)
    return 2.0 ** (e - 1) if m == 0.5 else 2.0 ** e


def append(values, scale, x, nodes, length, row, block):
    """One request: values float64 [n_blocks, H, block, D] (codes) and scale [n_blocks, H] are
    updated with x[nodes] (x float64 [N, H, D]) at slots length, length + 1, ..."""
    done, count = 0, len(nodes)
    while done < count:
        slot, off = row[(length + done) // block], (length + done) % block
        take = min(block - off, count - done)
        part = x[nodes[done:done + take]]
        for h in range(x.shape[1]):
            y = part[:, h]
            s = scale_for(float(np.max(np.abs(np.where(np.isfinite(y), y, 0.0)))))
            if off:
                s = max(s, float(scale[slot, h]))
                if s > scale[slot, h]:
                    values[slot, h, :off] = to_e4m3(values[slot, h, :off] * (scale[slot, h] / s))
            values[slot, h, off:off + take] = to_e4m3(y / s)
            scale[slot, h] = s
        done += take


def attend(q, k_new, v_new, parent, nodes, k, v, length, scale, softcap=0.0, slopes=None,
           window=0):
    """One request in float64: q [N, Hq, D]; k_new, v_new [N, Hkv, D]; k, v [length, Hkv, D].
    Returns out, lse, and for the tolerances the weighted |v| and the largest sum |q||k| scale."""
    N, Hq, D = q.shape
    Hkv = k_new.shape[1]
    G = Hq // Hkv
    out = torch.zeros(N, Hq, D, dtype=torch.float64)
    lse = torch.full((N, Hq), -math.inf, dtype=torch.float64)
    mag = torch.zeros(N, Hq, D, dtype=torch.float64)
    big = torch.zeros(N, Hq, dtype=torch.float64)
    for n in range(nodes):
        up = ancestors(parent, n)
        where = length + len(up) - 1
        dist = [where - j for j in range(length)] + list(range(len(up)))
        keep = [i for i, d in enumerate(dist) if window == 0 or d < window]
        keys = torch.cat((k, k_new[up]))[keep]
        vals = torch.cat((v, v_new[up]))[keep]
        far = torch.tensor([dist[i] for i in keep], dtype=torch.float64)
        for h in range(Hq):
            kk, vv = keys[:, h // G], vals[:, h // G]
            s = kk @ q[n, h] * scale
            big[n, h] = (kk.abs() @ q[n, h].abs()).nan_to_num(0, 0, 0).max() * abs(scale)
            if softcap:
                s = softcap * torch.tanh(s / softcap)
            if slopes is not None:
                s = s - float(slopes[h]) * far
            if float(s.max()) == -math.inf:
                continue
            p = torch.exp(s - s.max())
            lse[n, h] = torch.log(p.sum()) + s.max()
            out[n, h] = (p / p.sum()) @ vv
            mag[n, h] = (p / p.sum()) @ vv.abs()
    return out, lse, mag, big


def random_tree(rng, N, depth=5, branching=3):
    parent, at, kids = [-1], [0], [0]
    for n in range(1, N):
        free = [i for i in range(n) if at[i] < depth and kids[i] < branching]
        p = int(rng.choice(free)) if free else int(rng.integers(0, n))
        parent.append(p)
        at.append(at[p] + 1)
        kids.append(0)
        kids[p] += 1
    return parent


def make_cache(rng, lens, more, block, Hkv, D, spare=2, scales="pow2"):
    """A paged cache on the CPU: codes uint8 of random finite values, NaN codes in the slots that
    hold no token, scales, a table with junk in its unused entries."""
    need = [-(-(n + m) // block) for n, m in zip(lens, more)]
    ids = rng.permutation(sum(need) + spare)
    width = max(max(need), 1) + 1
    table = np.full((len(lens), width), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        table[b, n:] = rng.choice([-1, 2 ** 31 - 1, -2 ** 31, 0])
        at += n
    nb = sum(need) + spare
    cache = {}
    for name in ("k", "v"):
        x = torch.from_numpy(rng.standard_normal((nb, Hkv, block, D)) * 40).float()
        codes = x.to(E4M3).view(torch.uint8)
        s = 2.0 ** rng.integers(-7, -3, (nb, Hkv)) if scales == "pow2" else \
            rng.uniform(0.004, 0.05, (nb, Hkv))
        cache[name], cache[name + "_scale"] = codes, torch.from_numpy(s).float()
    held = np.zeros((nb, block), dtype=bool)
    for b, n in enumerate(lens):
        for j in range(n):
            held[table[b, j // block], j % block] = True
    junk = torch.from_numpy(~held)[:, None, :, None]
    for name in ("k", "v"):
        cache[name] = torch.where(junk, torch.tensor(0x7F, dtype=torch.uint8), cache[name])
    cache["block_table"], cache["length"] = torch.from_numpy(table), torch.tensor(lens, dtype=torch.int32)
    return cache


def cached_values(cache, name, b, block):
    """float64 [length, Hkv, D] of request b."""
    n = int(cache["length"][b])
    ids = cache["block_table"][b, :-(-n // block)].long()
    x = cache[name][ids].view(E4M3).double() * cache[name + "_scale"][ids].double()[:, :, None, None]
    return x.permute(0, 2, 1, 3).reshape(-1, x.shape[1], x.shape[3])[:n]


def on_gpu(cache):
    from speculative_decoding_verification_64_gb300 import binding
    return binding.KVCache(cache["k"].cuda().view(E4M3), cache["v"].cuda().view(E4M3),
                           cache["k_scale"].cuda(), cache["v_scale"].cuda(),
                           cache["block_table"].cuda(), cache["length"].cuda())
