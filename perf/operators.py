"""What is measured of the paged 8-bit key/value cache: attention over it (full, or a sliding window with a few first
tokens), appending to it, and the moves of its pages.

The cache is a pool of pages of `page` tokens. Keys and values are e4m3 [layers, pages, kv heads, page, dim] with one
fp32 scale for each page and kv head; `table` names each sequence's pages (-1: none), `length` its tokens, `ref` how
many table rows hold a page. `own` False: plain torch in fp32. `own` True: the calls of the package's KVCache.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
E4M3 = torch.float8_e4m3fn
TOP = 448.0           # largest e4m3 value
LOWEST = -120         # smallest exponent of a block scale


# ------------------------------------------------------------------------------------------------ cases

def listed():
    a = dict(kind="attend", layers=1, window=0, sinks=0)
    return [
        # one short sequence of a d 512 model (8 heads of 64), fp32 activations: what one call costs
        dict(a, name="attend_1x333_d512_f32", seqs=1, len_lo=333, len_hi=333, new_lo=1, new_hi=1,
             heads=8, kv_heads=8, dim=64, page=16, type="f32"),
        # one user with a long document, grouped heads: the cache is split over the whole GPU
        dict(a, name="attend_1x131067_gqa", seqs=1, len_lo=131067, len_hi=131067, new_lo=1, new_hi=1,
             heads=64, kv_heads=8, dim=128, page=64, type="bf16"),
        # a batch of 16 at d 5120 (40 heads of 128, each with its own cache), fp32 activations, ragged
        dict(a, name="attend_16x8k_d5120_f32", seqs=16, len_lo=1, len_hi=8191, new_lo=1, new_hi=1,
             heads=40, kv_heads=40, dim=128, page=32, type="f32"),
        # a full serving batch with grouped heads
        dict(a, name="attend_128x16k_gqa", seqs=128, len_lo=129, len_hi=16383, new_lo=1, new_hi=1,
             heads=64, kv_heads=8, dim=128, page=64, type="bf16"),
        # prompt chunks of four users, with a context before each chunk
        dict(a, name="attend_prompt_4x2k", seqs=4, len_lo=1500, len_hi=8191, new_lo=700, new_hi=2048,
             heads=32, kv_heads=8, dim=128, page=64, type="bf16"),
        # streaming decode: a window of 4096 and 4 first tokens, pages that slid out are gone
        dict(a, name="window_64x64k", seqs=64, len_lo=300, len_hi=65535, new_lo=1, new_hi=1,
             heads=32, kv_heads=8, dim=128, page=64, type="bf16", window=4096, sinks=4),
        # a long prompt under a window of 1000 and 70 first tokens, each head with its own cache (d 4096)
        dict(a, name="window_prompt_8191", seqs=1, len_lo=8191, len_hi=8191, new_lo=8191, new_hi=8191,
             heads=32, kv_heads=32, dim=128, page=32, type="f16", window=1000, sinks=70),
        # one decode step's keys and values of 64 sequences (d 5120)
        dict(kind="append", name="append_64x1_d5120", layers=1, seqs=64, len_lo=1, len_hi=4095, new_lo=1, new_hi=1,
             heads=40, kv_heads=40, dim=128, page=32, type="f32"),
        # the keys and values of prompts of different lengths
        dict(kind="append", name="append_prompt_7x4k", layers=1, seqs=7, len_lo=4100, len_hi=8191, new_lo=1000,
             new_hi=4095, heads=32, kv_heads=8, dim=128, page=64, type="bf16"),
        # one sequence forked into four, a token each: bookkeeping latency
        dict(kind="fork", name="fork_1to4_small", layers=2, seqs=1, copies=4, len_lo=75, len_hi=75, new_lo=1, new_hi=1,
             heads=8, kv_heads=8, dim=64, page=16, type="f32"),
        # sampling eight continuations of each of eight prompts (d 4096, 8 layers)
        dict(kind="fork", name="fork_8to64_d4096", layers=8, seqs=8, copies=8, len_lo=500, len_hi=2047, new_lo=1,
             new_hi=40, heads=32, kv_heads=32, dim=128, page=32, type="f16"),
        # a pool left sparse by finished sequences is made dense (d 4096, 8 layers)
        dict(kind="compact", name="compact_d4096", layers=8, seqs=16, gone=16, len_lo=200, len_hi=1500, new_lo=1,
             new_hi=1, heads=32, kv_heads=32, dim=128, page=32, type="f16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["attend", "attend", "prompt", "window", "window_prompt", "append", "fork", "compact"])
    kv = rng.choice([1, 2, 8, 8, 32, 40])
    dim = rng.choice([64, 128, 128, 256])
    group = rng.choice([1, 1, 2, 4, 5, 8, 16])
    c = dict(kind=kind.replace("window_prompt", "attend").replace("prompt", "attend").replace("window", "attend"),
             layers=1, kv_heads=kv, heads=kv * group, dim=dim, page=rng.choice([16, 32, 64]),
             type=rng.choice(["f32", "bf16", "f16"]), window=0, sinks=0, new_lo=1, new_hi=1)
    token = 2 * kv * dim
    if kind in ("attend", "window"):
        c["seqs"] = _log(rng, 1, 128)
        hi = _log(rng, 1, max(64, min(131072, int(1.5e9) // (token * c["seqs"]))))
        c.update(len_lo=max(1, int(hi * rng.choice([0.01, 0.3, 1.0]))), len_hi=hi)
    elif kind in ("prompt", "window_prompt"):
        c["seqs"] = _log(rng, 1, 6)
        c["heads"] = min(c["heads"], 64) // kv * kv
        hi = _log(rng, 17, max(32, min(8191, int(math.sqrt(2.0e9 / (c["seqs"] * c["heads"]))))))
        c.update(len_lo=max(1, hi // 2), len_hi=hi, new_lo=max(1, hi // 8),
                 new_hi=max(1, int(hi * rng.choice([0.3, 1.0]))))
    elif kind == "append":
        c["seqs"] = _log(rng, 1, 64)
        hi = _log(rng, 16, max(64, min(8191, int(5e8) // (token * c["seqs"]))))
        c.update(len_lo=max(1, hi // 3), len_hi=hi, new_hi=rng.choice([1, 1, 7, max(1, hi // 2)]))
    else:
        c["layers"] = rng.choice([1, 2, 4, 8])
        c["seqs"] = _log(rng, 1, 16)
        n = _log(rng, 1, 8 if kind == "fork" else 16)
        c["copies" if kind == "fork" else "gone"] = n
        hi = _log(rng, 4, max(16, min(2047, int(6e8) // (token * c["layers"] * (c["seqs"] + n)))))
        c.update(len_lo=max(1, hi // 4), len_hi=hi, new_hi=rng.choice([1, 5, 40]) if kind == "fork" else 1)
    if kind.startswith("window"):
        c.update(window=_log(rng, 1, 4096), sinks=rng.choice([0, 1, 4, 70]))
    return c


def lengths(case):
    """Tokens of each sequence (its new ones among them) and its new tokens: spread evenly over the case's ranges."""
    n = case["seqs"]
    at = (np.arange(n) * 0.6180339887498949 + 0.5) % 1.0
    at2 = (np.arange(n) * 0.7548776662466927 + 0.25) % 1.0
    total = np.round(case["len_lo"] + at * (case["len_hi"] - case["len_lo"])).astype(np.int64)
    new = np.round(case["new_lo"] + at2 * (case["new_hi"] - case["new_lo"])).astype(np.int64)
    if case["kind"] in ("attend", "append"):
        new = np.minimum(new, total)
    return total, new


def held(case):
    """Truth value for each sequence and column of its table row: does the row name a page there?"""
    total, new = lengths(case)
    P = case["page"]
    col = np.arange(-(-int(total.max() + new.max()) // P) + 1)[None, :]
    has = col * P < total[:, None]
    if case.get("window", 0) > 0:   # what no query from the new tokens on can see has been dropped
        has &= (col * P < case["sinks"]) | (col * P + P - 1 > (total - new - case["window"])[:, None])
    return has


# ------------------------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    total, new = lengths(case)
    L, H, P, D, n = case["layers"], case["kv_heads"], case["page"], case["dim"], case["seqs"]
    has = held(case)
    used = int(has.sum())
    more = 0
    rows = n
    if case["kind"] == "fork":
        rows = n * (1 + case["copies"])
        more = int((-(-(total % P + new.max()) // P) + 1).sum()) * case["copies"]
    if case["kind"] == "compact":
        more = case["gone"] * int(-(-total.max() // P))
    n_pages = used + more + 3

    def pool():
        x = torch.empty((L, n_pages, H, P, D), dtype=E4M3, device=dev)
        for l in range(L):   # values of about unit size once scaled: the largest code is a few deviations out
            y = torch.randn((n_pages, H, P, D), generator=g, device=dev, dtype=torch.float16)
            x[l] = y.mul_(64).clamp_(-TOP, TOP).to(E4M3)
        s = torch.exp2(torch.randint(-7, -4, (L, n_pages, H), generator=g, device=dev).float())
        return x, s

    k, k_scale = pool()
    v, v_scale = pool()
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((rows, has.shape[1]), -1, dtype=torch.int32, device=dev)
    table[:n][torch.from_numpy(has).to(dev)] = order[:used]
    ref = torch.zeros(n_pages, dtype=torch.int32, device=dev)
    ref[order[:used].long()] = 1
    length = torch.zeros(rows, dtype=torch.int32, device=dev)
    length[:n] = torch.from_numpy(total).to(dev)
    s = dict(case=case, k=k, v=v, k_scale=k_scale, v_scale=v_scale, table=table, length=length, ref=ref,
             seqs=torch.arange(n, dtype=torch.int32, device=dev), scale=1.0 / math.sqrt(D), widest=int(new.max()),
             longest=int(total.max()))
    copies = case.get("copies", 1)
    start = np.concatenate([[0], np.cumsum(np.repeat(new, copies))])
    s["start"] = torch.from_numpy(start).to(dev).to(torch.int32)
    if case["kind"] in ("attend", "append"):   # one projection's output: queries, keys and values side by side
        Hq, T = case["heads"], int(start[-1])
        qkv = torch.randn((T, (Hq + 2 * H) * D), generator=g, device=dev).to(TYPES[case["type"]])
        if case["kind"] == "append":   # some heads and tokens larger than others
            qkv[:, Hq * D:].mul_(torch.exp2(torch.randint(-3, 4, (T, 1), generator=g, device=dev).to(qkv.dtype)))
        s["q"] = qkv[:, :Hq * D].unflatten(1, (Hq, D))
        s["k_new"] = qkv[:, Hq * D:(Hq + H) * D].unflatten(1, (H, D))
        s["v_new"] = qkv[:, (Hq + H) * D:].unflatten(1, (H, D))
    if case["kind"] == "fork":
        s["src"] = s["seqs"].repeat_interleave(copies)
        s["dst"] = torch.arange(n, rows, dtype=torch.int32, device=dev)
    if case["kind"] == "compact":
        s["table0"], s["ref0"] = table.clone(), ref.clone()
    if own:   # the handle over these tensors that a program keeps
        from activation_sparse_decode_pi_gb300 import KVCache

        s["cache"] = KVCache([dict(k=k[l], v=v[l], k_scale=k_scale[l], v_scale=v_scale[l]) for l in range(L)],
                             table, length, ref, n_heads=case["heads"])
    return s


# ------------------------------------------------------------------------------------------------ plain forms

def plain_attend(s):
    """Softmax attention of each sequence's last tokens over its pages, in fp32 on padded tensors."""
    c = s["case"]
    H, P, D, W, S = c["kv_heads"], c["page"], c["dim"], c["window"], c["sinks"]
    G, n, Q = c["heads"] // H, c["seqs"], s["widest"]
    dev = s["q"].device
    new = (s["start"][1:] - s["start"][:-1]).long()[:, None]
    total = s["length"][:n].long()[:, None]
    first = total - new                                        # position of the first query
    reach = W + Q - 1
    if W > 0 and S + reach < s["longest"]:                      # only the first tokens and the windows' span
        lo = (first - W + 1).clamp(min=0)
        at = lo + torch.arange(reach, device=dev)[None, :]
        pos = torch.cat([torch.arange(S, device=dev)[None, :].expand(n, S), at], 1)
        there = torch.cat([torch.arange(S, device=dev)[None, :] < lo, at < total], 1)
    else:
        pos = torch.arange(s["longest"], device=dev)[None, :].expand(n, -1)
        there = pos < total
    col = pos.clamp(max=s["table"].shape[1] * P - 1) // P
    page = s["table"][:n].gather(1, col).long()
    there = there & (page >= 0)
    page = page.clamp(min=0)
    slot = pos % P

    def read(pool, scale):
        x = pool[0].view(torch.uint8)[page, :, slot].view(E4M3).float() * scale[0][page][..., None]
        return x.masked_fill(~there[..., None, None], 0.0)      # [n, keys, H, D]

    K, V = read(s["k"], s["k_scale"]), read(s["v"], s["v_scale"])
    t = torch.arange(Q, device=dev)[None, :]
    row = (s["start"][:-1].long()[:, None] + t).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float()[row].view(n, Q, H, G, D)
    logit = torch.einsum("nqhgd,nkhd->nhgqk", q, K) * s["scale"]
    qpos = (first + t)[:, :, None]
    see = there[:, None, :] & (pos[:, None, :] <= qpos)
    if W > 0:
        see = see & ((qpos - pos[:, None, :] < W) | (pos[:, None, :] < S))
    see = see[:, None, None]
    logit = logit.masked_fill(~see, -math.inf)
    top = logit.amax(-1, keepdim=True)
    p = torch.exp(logit - torch.where(torch.isfinite(top), top, 0.0))
    z = p.sum(-1, keepdim=True)
    p = p / torch.where(z > 0, z, 1.0)
    out = torch.einsum("nhgqk,nkhd->nqhgd", p, V).reshape(n, Q, H * G, D)
    return out[t.expand(n, Q) < new].to(s["q"].dtype)


def power_of_two(a):
    """The smallest power of two (of exponent LOWEST or more) that brings a to at most 448."""
    m, e = torch.frexp(a)
    e = torch.where(a > 0, e - 9 + (m > 0.875), LOWEST).clamp(min=LOWEST)
    return torch.exp2(e.float())


def plain_append(s):
    c = s["case"]
    H, P, n = c["kv_heads"], c["page"], c["seqs"]
    start = s["start"].long()
    T = s["k_new"].shape[0]
    tok = torch.arange(T, device=start.device)
    seq = torch.searchsorted(start[1:], tok, right=True)
    pos = s["length"][:n].long()[seq] - start[seq + 1] + tok
    page = s["table"][:n][seq, pos // P].long()
    # the page that the sequence's first new token falls into, and what it held before
    first = s["length"][:n].long() - (start[1:] - start[:-1])
    part = (first % P > 0) & (start[1:] > start[:-1])
    old = s["table"][:n].gather(1, (first // P)[:, None])[:, 0].long()[part]
    before = torch.arange(P, device=start.device)[None, :] < (first % P)[part][:, None]

    def put(pool, scale, x):
        x = x.float()
        top = torch.zeros_like(scale).scatter_reduce(0, page[:, None].expand(T, H), x.abs().amax(-1), "amax")
        s_new = power_of_two(top)
        had = scale[old]
        now = torch.maximum(had, s_new[old])
        codes = pool.view(torch.uint8)
        held = codes[old]
        moved = (held.view(E4M3).float() * (had / now)[..., None, None]).clamp(-TOP, TOP).to(E4M3).view(torch.uint8)
        codes[old] = torch.where(before[:, None, :, None], moved, held)
        scale[page] = s_new[page]
        scale[old] = now
        codes[page, :, pos % P] = (x / scale[page][..., None]).clamp(-TOP, TOP).to(E4M3).view(torch.uint8)

    put(s["k"][0], s["k_scale"][0], s["k_new"])
    put(s["v"][0], s["v_scale"][0], s["v_new"])


def copy_pages(s, src, dst):
    for name in ("k", "v"):
        codes = s[name].view(torch.uint8)
        codes[:, dst] = codes[:, src]
        s[name + "_scale"][:, dst] = s[name + "_scale"][:, src]


def hand_out(s, count):
    """The lowest `count` free pages, now held once."""
    got = torch.nonzero(s["ref"] == 0)[:count, 0]
    s["ref"][got] = 1
    return got


def plain_fork(s):
    """dst gives back its pages, shares src's full ones and gets a copy of the last, and grows by its new tokens."""
    P = s["case"]["page"]
    src, dst, table, length, ref = s["src"].long(), s["dst"].long(), s["table"], s["length"], s["ref"]
    gone = table[dst]
    ref.sub_(torch.bincount(gone[gone >= 0].long(), minlength=ref.numel()).to(torch.int32))
    col = torch.arange(table.shape[1], device=table.device)[None, :]
    have = length[src].long()
    shared = col < (have // P)[:, None]
    row = torch.where(shared, table[src], -1)
    ref.add_(torch.bincount(row[row >= 0].long(), minlength=ref.numel()).to(torch.int32))
    part = have % P > 0
    got = hand_out(s, int(part.sum()))
    copy_pages(s, table[src, (have // P).clamp(max=table.shape[1] - 1)].long()[part], got)
    row[(col == (have // P)[:, None]) & part[:, None]] = got.to(torch.int32)
    now = have + (s["start"][1:] - s["start"][:-1])
    fresh = (col * P >= (-(-have // P) * P)[:, None]) & (col * P < now[:, None])
    row[fresh] = hand_out(s, int(fresh.sum())).to(torch.int32)
    table[dst] = row
    length[dst] = now.to(torch.int32)


def plain_compact(s):
    ref, table = s["ref"], s["table"]
    live = ref > 0
    n = live.sum()
    ids = torch.arange(ref.numel(), device=ref.device)
    hole, mover = ids[~live & (ids < n)], ids[live & (ids >= n)]
    copy_pages(s, mover, hole)
    to = ids.clone()
    to[mover] = hole
    ref[hole] = ref[mover]
    ref[mover] = 0
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].to(torch.int32), table))
    return n.to(torch.int32).reshape(1)


def run(state):
    s, c = state, state["case"]
    if c["kind"] == "attend":
        if own:
            return s["cache"].attend(0, s["seqs"], s["start"], s["q"], scale=s["scale"], window=c["window"],
                                     sinks=c["sinks"])
        return plain_attend(s)
    out = dict(k=s["k"], v=s["v"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    if c["kind"] == "append":
        if own:
            s["cache"].append(0, s["seqs"], s["start"], s["k_new"], s["v_new"])
        else:
            plain_append(s)
        return out
    out.update(table=s["table"], length=s["length"], ref=s["ref"])
    if c["kind"] == "fork":
        if own:
            s["cache"].fork(s["src"], s["dst"])
            s["cache"].reserve(s["dst"], s["start"])
        else:
            plain_fork(s)
        return out
    s["table"].copy_(s["table0"])   # the sparse pool again: its pages are still where they were
    s["ref"].copy_(s["ref0"])
    out["live"] = s["cache"].compact() if own else plain_compact(s)
    return out


# ------------------------------------------------------------------------------------------------ what it takes

def seen(case):
    """Per sequence: keys that some query sees, and (query, key) pairs that count."""
    total, new = lengths(case)
    W, S = case["window"], case["sinks"]
    keys = pairs = 0
    for t, m in zip(total.tolist(), new.tolist()):
        pos = np.arange(t - m, t)
        if W <= 0:
            keys += t
            pairs += int((pos + 1).sum())
        else:
            lo = np.maximum(pos - W + 1, 0)
            keys += t - max(t - m - W + 1, 0) + min(S, max(t - m - W + 1, 0))
            pairs += int((pos + 1 - lo + np.minimum(S, lo)).sum())
    return keys, pairs


def work(case):
    total, new = lengths(case)
    H, D, P, L = case["kv_heads"], case["dim"], case["page"], case["layers"]
    size = {"f32": 4, "bf16": 2, "f16": 2}[case["type"]]
    if case["kind"] == "attend":
        keys, pairs = seen(case)
        io = 2 * int(new.sum()) * case["heads"] * D * size
        return {"bytes": 2 * keys * H * (D + 4.0 / P) + io, "flops": 4.0 * D * case["heads"] * pairs}
    if case["kind"] == "append":
        T = int(new.sum())
        return {"bytes": 2 * T * H * (D * (size + 1) + 4.0 / P), "flops": 2.0 * 2 * T * H * D}
    page = 2 * L * H * (P * D + 4)
    if case["kind"] == "fork":
        copied = int((total % P > 0).sum()) * case["copies"]
        rows = int((-(-total // P)).sum()) * case["copies"]
        return {"bytes": 2 * copied * page + 3 * 4 * rows, "flops": 0.0}
    used = int(held(case).sum())
    n_pages = used + case["gone"] * int(-(-total.max() // P)) + 3
    moved = used * (n_pages - used) / n_pages            # live pages above the dense end of a shuffled pool
    return {"bytes": 2 * moved * page + 4 * (2 * used + n_pages), "flops": 0.0}


# ------------------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "attend":
        if 4.0 * case["dim"] * case["heads"] * seen(case)[1] > 4e12:
            return None
        return exact_attend(s)
    if case["kind"] == "append":
        return exact_append(s)
    return None   # pages are moved, not computed


def exact_attend(s):
    """One sequence and kv head at a time, straight from the definition."""
    c = s["case"]
    H, P, W, S = c["kv_heads"], c["page"], c["window"], c["sinks"]
    G = c["heads"] // H
    start = s["start"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    for i, total in enumerate(s["length"].tolist()):
        m = start[i + 1] - start[i]
        j = torch.arange(total, device=out.device)
        page = s["table"][i].long()[j // P]
        j, page = j[page >= 0], page[page >= 0]
        at = torch.arange(total - m, total, device=out.device)[:, None]
        see = j[None, :] <= at
        if W > 0:
            see &= (at - j[None, :] < W) | (j[None, :] < S)
        for h in range(H):
            read = lambda name: (s[name][0, :, h].view(torch.uint8)[page, j % P].view(E4M3).double()  # noqa: E731
                                 * s[name + "_scale"][0, page, h].double()[:, None])
            q = s["q"][start[i]:start[i + 1], h * G:(h + 1) * G].double()
            k, v = read("k"), read("v")
            for a in range(0, m, 1024):                  # a block of queries at a time
                b = min(m, a + 1024)
                x = (q[a:b].reshape(-1, q.shape[-1]) @ k.T).view(b - a, G, -1) * s["scale"]
                x = x.masked_fill(~see[a:b, None, :], -math.inf)
                p = torch.softmax(x, -1)
                out[start[i] + a:start[i] + b, h * G:(h + 1) * G] = (p.view((b - a) * G, -1) @ v).view(b - a, G, -1)
    return out


def exact_append(s):
    c = s["case"]
    P = c["page"]
    start, total = s["start"].tolist(), s["length"].tolist()
    got = {}
    for name in ("k", "v"):
        pool = s[name][0].view(torch.uint8)
        value = s[name].clone()
        codes = value[0].view(torch.uint8)
        scale = s[name + "_scale"].double()
        x = s[name + "_new"].double()
        for i, n in enumerate(total):
            m = start[i + 1] - start[i]
            at = n - m
            while at < n:                                 # one page at a time
                end = min(n, (at // P + 1) * P)
                page = int(s["table"][i, at // P])
                part = x[start[i + 1] - n + at:start[i + 1] - n + end]          # [tokens, H, D]
                top = part.abs().amax((0, 2))
                e = torch.ceil(torch.log2(top / TOP))
                e += (top > TOP * torch.exp2(e)).double() - (top <= TOP * torch.exp2(e - 1)).double()
                now = torch.exp2(torch.where(top > 0, e, LOWEST).clamp(min=LOWEST))
                old = at % P
                if old:
                    was = scale[0, page]
                    now = torch.maximum(was, now)
                    moved = pool[page, :, :old].view(E4M3).double() * (was / now)[:, None, None]
                    codes[page, :, :old] = moved.clamp(-TOP, TOP).float().to(E4M3).view(torch.uint8)
                scale[0, page] = now
                fresh = (part / now[None, :, None]).clamp(-TOP, TOP).float().to(E4M3).view(torch.uint8)
                codes[page, :, old:old + end - at] = fresh.transpose(0, 1)
                at = end
        got[name], got[name + "_scale"] = value, scale
    return got
