"""What is measured of the steps around the paged cache's attention: projections with 4-bit weights, the norms of queries
and keys with the position rotation, the same with the write into the 8-bit cache, and attention of sequences that
share a long prefix.

`own` False: plain torch in fp32 (angles in fp64). `own` True: the calls of the package: Int4Linear, Rotary, and the
KVCache's append_rotated and attend_shared.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
E4M3 = torch.float8_e4m3fn
TOP = 448.0           # largest e4m3 value
LOWEST = -120         # smallest exponent of a block scale
GROUP = 128           # elements of a 4-bit row that share a scale
EPS = 1e-6            # of the norms


# ------------------------------------------------------------------------------------------------ cases

def listed():
    rot = dict(kind="rotate", heads=32, kv_heads=8, dim=128, rot=128, interleaved=False, norm=True, base=1e4,
               stretch=1.0, trained=8192, pos_lo=0)
    app = dict(rot, kind="append", layers=1)
    sh = dict(kind="shared", layers=1, new=1)
    lin = dict(kind="int4", bias=False, add=False)
    return [
        # one token of one user (32 heads on 8), far along in a long context: what a call costs
        dict(rot, name="rotate_1x_d4096", tokens=1, pos_lo=100003, pos_hi=100003, base=5e5, stretch=8.0, type="bf16"),
        # fp32, 40 heads of 64, the first half of each rotated in neighbouring pairs, no norm, positions up to 10^6
        dict(rot, name="rotate_1003_part_f32", tokens=1003, heads=40, kv_heads=40, dim=64, rot=32, interleaved=True,
             norm=False, pos_hi=1000000, type="f32"),
        # a long prompt of a model with 64 heads on 8
        dict(rot, name="rotate_prompt_8191", tokens=8191, heads=64, pos_hi=8190, type="bf16"),
        # one user's next token into the cache
        dict(app, name="append_rot_1x_d4096", seqs=1, len_lo=30011, len_hi=30011, new_lo=1, new_hi=1, page=64,
             base=5e5, stretch=8.0, type="bf16"),
        # one decode step of 64 sequences (d 5120, each head with its own cache), fp32 activations, no norm
        dict(app, name="append_rot_64x1_d5120", seqs=64, len_lo=1, len_hi=4095, new_lo=1, new_hi=1, heads=40,
             kv_heads=40, page=32, norm=False, type="f32"),
        # prompts of different lengths
        dict(app, name="append_rot_prompt_7x4k", seqs=7, len_lo=4100, len_hi=8191, new_lo=1000, new_hi=4095, page=64,
             type="bf16"),
        # four continuations of a short prompt on a d 512 model (8 heads of 64), fp32: what a call costs
        dict(sh, name="shared_4x_d512_f32", groups=1, seqs=4, pre_lo=1000, pre_hi=1000, own_lo=1, own_hi=70, heads=8,
             kv_heads=8, dim=64, page=16, type="f32"),
        # 64 users behind one long system prompt, grouped heads
        dict(sh, name="shared_64x16k_gqa", groups=1, seqs=64, pre_lo=16400, pre_hi=16400, own_lo=1, own_hi=700,
             heads=64, kv_heads=8, dim=128, page=64, type="bf16"),
        # eight prompts with nine samples each, four proposed tokens a sample, each head with its own cache (d 5120)
        dict(sh, name="shared_8x9_d5120", groups=8, seqs=9, pre_lo=300, pre_hi=6000, own_lo=4, own_hi=300, new=4,
             heads=40, kv_heads=40, dim=128, page=32, type="f16"),
        # queries, keys and values of one token (d 4096, 32 heads on 8 of 128)
        dict(lin, name="int4_1x_d4096", rows=1, n=6144, k=4096, type="bf16"),
        # the same of one token at d 12288, each head with its own keys, fp32 activations and biases
        dict(lin, name="int4_1x_d12288_f32", rows=1, n=36864, k=12288, bias=True, type="f32"),
        # the output projection of 16 tokens, added to the residual stream (d 5120, fp32)
        dict(lin, name="int4_16x_d5120_f32", rows=16, n=5120, k=5120, add=True, type="f32"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rotate", "append", "append", "shared", "shared", "int4", "int4"])
    kind_of = rng.choice(["f32", "bf16", "f16"])
    if kind == "int4":
        k = 128 * _log(rng, 1, 96)
        rows = rng.choice([1, 1, _log(rng, 1, 64)])
        n = _log(rng, 16, max(32, min(49152, int(4e8) // (k * max(1, rows // 8)))))
        return dict(kind=kind, rows=rows, n=n, k=k, bias=rng.random() < 0.5, add=rng.random() < 0.5, type=kind_of)
    kv = rng.choice([1, 2, 8, 8, 32, 40])
    group = rng.choice([1, 1, 2, 4, 5, 8])
    dim = rng.choice([64, 128, 128, 256])
    c = dict(kind=kind, heads=kv * group, kv_heads=kv, dim=dim, type=kind_of)
    if kind == "shared":
        c.update(layers=1, page=rng.choice([16, 32, 64, 128]), new=rng.choice([1, 1, 1, 2, 5]))
        c["groups"] = _log(rng, 1, 12)
        c["seqs"] = _log(rng, 1, max(1, 96 // c["groups"]))
        hi = _log(rng, 64, max(128, min(32768, int(2.6e8) // (2 * kv * dim * c["groups"]),
                                        int(7e9) // (c["groups"] * c["seqs"] * c["new"] * kv * group * dim))))
        c.update(pre_lo=max(1, int(hi * rng.choice([0.05, 0.5, 1.0]))), pre_hi=hi, own_lo=c["new"])
        c["own_hi"] = _log(rng, c["new"], max(c["new"] + 1, min(1500, int(1e8) // (2 * kv * dim * c["groups"] * c["seqs"]))))
        return c
    c.update(rot=rng.choice([dim, dim, dim // 2, dim // 4]), interleaved=rng.random() < 0.4, norm=rng.random() < 0.6,
             base=rng.choice([1e4, 5e5, 1e6]), stretch=rng.choice([1.0, 1.0, 4.0, 32.0]), trained=rng.choice([4096, 8192]))
    token = kv * (group + 2) * dim * SIZE[kind_of]
    if kind == "rotate":
        c.update(pos_lo=0, tokens=_log(rng, 1, max(2, min(8191, int(1.5e8) // token))))
        c["pos_hi"] = _log(rng, c["tokens"], 1000000)
        return c
    c.update(layers=1, page=rng.choice([16, 32, 64, 128]), pos_lo=0)
    c["seqs"] = _log(rng, 1, 64)
    hi = _log(rng, 16, max(64, min(8191, int(3e8) // (token * c["seqs"]))))
    c.update(len_lo=max(1, hi // 3), len_hi=hi, new_lo=1, new_hi=rng.choice([1, 1, 7, max(1, hi // 2)]))
    return c


def spread(n, lo, hi, step, first):
    """n whole numbers spread evenly over lo .. hi."""
    return np.round(lo + (np.arange(n) * step + first) % 1.0 * (hi - lo)).astype(np.int64)


def lengths(case):
    """Tokens of each sequence (its new ones among them) and its new tokens."""
    n = case["seqs"]
    if case["kind"] == "shared":      # a shared prefix of whole pages, and what each sequence has behind it
        pre = np.repeat(prefixes(case), n)
        own_part = spread(len(pre), case["own_lo"], case["own_hi"], 0.6180339887498949, 0.5)
        return pre + own_part, np.full(len(pre), case["new"])
    total = spread(n, case["len_lo"], case["len_hi"], 0.6180339887498949, 0.5)
    return total, np.minimum(spread(n, case["new_lo"], case["new_hi"], 0.7548776662466927, 0.25), total)


def prefixes(case):
    """Tokens that all sequences of a group share: whole pages."""
    return spread(case["groups"], case["pre_lo"], case["pre_hi"], 0.6180339887498949, 0.5) // case["page"] * case["page"]


def frequencies(case):
    """Radians per position of each pair, in fp64. stretch > 1: a context longer than the trained one. Pairs that turn
    at least 32 times within it keep their speed, those that turn at most once go 1 / stretch as fast, in between a
    mean of the two, and the outputs grow by 1 + 0.1 log(stretch)."""
    f = case["base"] ** (-2.0 * np.arange(case["rot"] // 2) / case["rot"])
    if case["stretch"] == 1.0:
        return f, 1.0
    turns = case["trained"] * f / (2 * math.pi)
    keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
    return f * (keep + (1.0 - keep) / case["stretch"]), 1.0 + 0.1 * math.log(case["stretch"])


# ------------------------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case=case)
    {"int4": prepare_int4, "rotate": prepare_rotate, "append": prepare_append, "shared": prepare_shared}[case["kind"]](s, g)
    return s


def prepare_int4(s, g):
    c, dev = s["case"], "cuda"
    t = TYPES[c["type"]]
    s["w"] = torch.randint(0, 256, (c["n"], c["k"] // 2), generator=g, device=dev, dtype=torch.uint8)
    s["scale"] = (torch.rand((c["n"], c["k"] // GROUP), generator=g, device=dev) * 0.4 + 0.1).div_(c["k"] ** 0.5).half()
    s["x"] = torch.randn((c["rows"], c["k"]), generator=g, device=dev).to(t)
    s["bias"] = torch.randn(c["n"], generator=g, device=dev) if c["bias"] else None
    s["add"] = torch.randn((c["rows"], c["n"]), generator=g, device=dev).to(t) if c["add"] else None
    if own:
        from activation_sparse_decode_pi_gb300 import Int4Linear

        s["linear"] = Int4Linear(s["w"], s["scale"], s["bias"])


def heads_of(s, g, tokens):
    """One projection's output: queries, keys and values side by side; the norms' weights; the rotation."""
    c, dev = s["case"], "cuda"
    Hq, H, D = c["heads"], c["kv_heads"], c["dim"]
    qkv = torch.randn((tokens, (Hq + 2 * H) * D), generator=g, device=dev)
    qkv.mul_(torch.exp2(torch.randint(-2, 3, (tokens, 1), generator=g, device=dev).float()))
    qkv = qkv.to(TYPES[c["type"]])
    s["q"] = qkv[:, :Hq * D].unflatten(1, (Hq, D))
    s["k_new"] = qkv[:, Hq * D:(Hq + H) * D].unflatten(1, (H, D))
    s["v_new"] = qkv[:, (Hq + H) * D:].unflatten(1, (H, D))
    freq, s["amp"] = frequencies(c)
    s["freq"] = torch.from_numpy(freq).to(dev)
    s["q_norm"] = s["k_norm"] = None
    if c["norm"]:
        s["q_norm"], s["k_norm"] = (1 + 0.2 * torch.randn(D, generator=g, device=dev) for _ in range(2))
    if own:
        from activation_sparse_decode_pi_gb300 import Rotary

        s["rotary"] = Rotary(freq, D, interleaved=c["interleaved"], amp=s["amp"], norm=c["norm"], q_norm=s["q_norm"],
                             k_norm=s["k_norm"], eps=EPS, device=dev)


def prepare_rotate(s, g):
    c = s["case"]
    heads_of(s, g, c["tokens"])
    if c["pos_hi"] - c["pos_lo"] == c["tokens"] - 1:
        s["pos"] = torch.arange(c["pos_lo"], c["pos_hi"] + 1, device="cuda", dtype=torch.int32)
    else:
        s["pos"] = torch.randint(c["pos_lo"], c["pos_hi"] + 1, (c["tokens"],), generator=g, device="cuda", dtype=torch.int32)


def pools(s, g, n_pages, table, length):
    c, dev = s["case"], "cuda"
    L, H, P, D = c["layers"], c["kv_heads"], c["page"], c["dim"]
    for name in ("k", "v"):
        x = torch.empty((L, n_pages, H, P, D), dtype=E4M3, device=dev)
        for layer in range(L):   # values of about unit size once scaled: the largest code is a few deviations out
            y = torch.randn((n_pages, H, P, D), generator=g, device=dev, dtype=torch.float16)
            x[layer] = y.mul_(64).clamp_(-TOP, TOP).to(E4M3)
        s[name] = x
        s[name + "_scale"] = torch.exp2(torch.randint(-7, -4, (L, n_pages, H), generator=g, device=dev).float())
    s["table"], s["length"] = table, length
    s["ref"] = torch.bincount(table[table >= 0].long(), minlength=n_pages).to(torch.int32)
    if own:
        from activation_sparse_decode_pi_gb300 import KVCache

        s["cache"] = KVCache([dict(k=s["k"][i], v=s["v"][i], k_scale=s["k_scale"][i], v_scale=s["v_scale"][i])
                              for i in range(L)], table, length, s["ref"], n_heads=c["heads"])


def batch(s, total, new):
    dev = "cuda"
    s["seqs"] = torch.arange(len(total), dtype=torch.int32, device=dev)
    s["start"] = torch.from_numpy(np.concatenate([[0], np.cumsum(new)])).to(dev).to(torch.int32)
    s["longest"] = int(total.max())
    return torch.from_numpy(total).to(dev).to(torch.int32)


def prepare_append(s, g):
    c, dev = s["case"], "cuda"
    total, new = lengths(c)
    length = batch(s, total, new)
    pages = -(-total // c["page"])
    n_pages = int(pages.sum()) + 3
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((len(total), int(pages.max()) + 1), -1, dtype=torch.int32, device=dev)
    has = torch.arange(table.shape[1], device=dev)[None, :] < torch.from_numpy(pages).to(dev)[:, None]
    table[has] = order[:int(pages.sum())]
    pools(s, g, n_pages, table, length)
    heads_of(s, g, int(new.sum()))


def prepare_shared(s, g):
    c, dev = s["case"], "cuda"
    total, new = lengths(c)
    length = batch(s, total, new)
    pre = prefixes(c) // c["page"]
    rest = -(-total // c["page"]) - np.repeat(pre, c["seqs"])
    n_pages = int(pre.sum() + rest.sum()) + 3
    order = torch.randperm(n_pages, generator=g, device=dev).cpu().numpy()
    table = np.full((len(total), int(-(-total.max() // c["page"])) + 1), -1, np.int32)
    at = 0
    for i in range(c["groups"]):
        front = order[at:at + pre[i]]
        at += pre[i]
        for j in range(i * c["seqs"], (i + 1) * c["seqs"]):
            table[j, :pre[i]] = front
            table[j, pre[i]:pre[i] + rest[j]] = order[at:at + rest[j]]
            at += rest[j]
    pools(s, g, n_pages, torch.from_numpy(table).to(dev), length)
    s["q"] = torch.randn((int(new.sum()), c["heads"], c["dim"]), generator=g, device=dev).to(TYPES[c["type"]])
    s["scale"] = 1.0 / math.sqrt(c["dim"])
    s["pre"] = torch.from_numpy(prefixes(c)).to(dev)
    s["groups"] = torch.arange(c["groups"] + 1, dtype=torch.int32, device=dev) * c["seqs"]
    if own:   # what the sequences share, found once for the steps of a batch
        s["plan"] = s["cache"].share(s["seqs"], s["start"], s["groups"])


# ------------------------------------------------------------------------------------------------ plain forms

def plain_int4(s):
    c = s["case"]
    q = torch.stack([s["w"] & 15, s["w"] >> 4], -1).view(c["n"], c["k"])     # even elements in the low halves
    q = (q.to(torch.int8) ^ 8) - 8                                           # two's complement
    w = q.view(c["n"], -1, GROUP).float() * s["scale"].float()[..., None]
    y = s["x"].float() @ w.view(c["n"], c["k"]).T
    if s["bias"] is not None:
        y = y + s["bias"]
    if s["add"] is not None:
        y = y + s["add"].float()
    return y.to(s["x"].dtype)


def plain_rotate(s, x, weight, pos):
    """Norm of each head, then the rotation of its first `rot` elements; x [tokens, heads, dim], fp32 out."""
    c = s["case"]
    x = x.float()
    if c["norm"]:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight
    angle = pos.double()[:, None] * s["freq"]
    cos, sin = (f(angle).float()[:, None] for f in (torch.cos, torch.sin))
    R = c["rot"]
    if c["interleaved"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned * s["amp"], x[..., R:]], -1)


def power_of_two(a):
    """The smallest power of two (of exponent LOWEST or more) that brings a to at most 448."""
    m, e = torch.frexp(a)
    e = torch.where(a > 0, e - 9 + (m > 0.875), LOWEST).clamp(min=LOWEST)
    return torch.exp2(e.float())


def plain_append(s):
    c = s["case"]
    H, P, n = c["kv_heads"], c["page"], len(s["seqs"])
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

    put(s["k"][0], s["k_scale"][0], plain_rotate(s, s["k_new"], s["k_norm"], pos))
    put(s["v"][0], s["v_scale"][0], s["v_new"].float())
    return plain_rotate(s, s["q"], s["q_norm"], pos).to(s["q"].dtype)


def plain_shared(s):
    """The prefix of each group once for all its rows, what each sequence has behind it, and the two joined."""
    c = s["case"]
    H, P, D, Gr, n = c["kv_heads"], c["page"], c["dim"], c["groups"], c["seqs"]
    G, Q = c["heads"] // H, c["new"]
    dev = s["q"].device
    pre = s["pre"]

    def read(name, rows, pos, there):
        page = s["table"][rows.long()].gather(1, pos.clamp(max=s["table"].shape[1] * P - 1) // P).long()
        there = there & (page >= 0)
        page = page.clamp(min=0)
        x = s[name][0].view(torch.uint8)[page, :, pos % P].view(E4M3).float() * s[name + "_scale"][0][page][..., None]
        return x.masked_fill(~there[..., None, None], 0.0), there    # [rows, keys, H, D]

    def part(rows, pos, there, q, qpos):
        """Numerators, maxima and sums of q [rows, queries, H, G, D] at positions qpos [rows, queries]."""
        k, there = read("k", rows, pos, there)
        v, _ = read("v", rows, pos, there)
        logit = torch.einsum("nqhgd,nkhd->nhgqk", q, k) * s["scale"]
        see = there[:, None, :] & (pos[:, None, :] <= qpos[:, :, None])
        logit = logit.masked_fill(~see[:, None, None], -math.inf)
        top = logit.amax(-1, keepdim=True)
        p = torch.exp(logit - torch.where(torch.isfinite(top), top, 0.0))
        return torch.einsum("nhgqk,nkhd->nhgqd", p, v), top, p.sum(-1, keepdim=True)

    total = s["length"].long()
    q = s["q"].float()
    qpos = (total - Q)[:, None] + torch.arange(Q, device=dev)
    front = torch.arange(max(1, int(prefixes(c).max())), device=dev)[None, :].expand(Gr, -1)
    o1, m1, z1 = part(s["groups"][:-1], front, front < pre[:, None], q.view(Gr, n * Q, H, G, D), qpos.view(Gr, n * Q))
    split = lambda x: x.view(Gr, H, G, n, Q, -1).permute(0, 3, 1, 2, 4, 5).reshape(Gr * n, H, G, Q, -1)  # noqa: E731
    o1, m1, z1 = split(o1), split(m1), split(z1)
    lo = pre.repeat_interleave(n)[:, None]
    pos = lo + torch.arange(c["own_hi"], device=dev)
    o2, m2, z2 = part(s["seqs"], pos, pos < total[:, None], q.view(Gr * n, Q, H, G, D), qpos)
    top = torch.maximum(m1, m2)
    a, b = torch.exp(m1 - top), torch.exp(m2 - top)
    out = (o1 * a + o2 * b) / (z1 * a + z2 * b)                      # [sequences, H, G, Q, D]
    return out.permute(0, 3, 1, 2, 4).reshape(s["q"].shape).to(s["q"].dtype)


def run(state):
    s, kind = state, state["case"]["kind"]
    if kind == "int4":
        return s["linear"](s["x"], add=s["add"]) if own else plain_int4(s)
    if kind == "rotate":
        if own:
            return s["rotary"].rotate(s["pos"], s["q"], s["k_new"])
        return tuple(plain_rotate(s, x, w, s["pos"]).to(x.dtype) for x, w in ((s["q"], s["q_norm"]), (s["k_new"], s["k_norm"])))
    if kind == "shared":
        if own:
            return s["cache"].attend_shared(0, s["seqs"], s["start"], s["plan"], s["q"], scale=s["scale"])
        return plain_shared(s)
    if own:
        q = s["cache"].append_rotated(0, s["seqs"], s["start"], s["rotary"], s["q"], s["k_new"], s["v_new"])
    else:
        q = plain_append(s)
    return dict(q=q, k=s["k"], v=s["v"], k_scale=s["k_scale"], v_scale=s["v_scale"])


# ------------------------------------------------------------------------------------------------ what it takes

def work(case):
    size, c = SIZE[case["type"]], case
    if c["kind"] == "int4":
        rows, n, k = c["rows"], c["n"], c["k"]
        io = rows * (k + n + n * c["add"]) * size + 4 * n * c["bias"]
        return {"bytes": n * k / 2 + 2 * n * k / GROUP + io, "flops": 2.0 * rows * n * k}
    Hq, H, D = c["heads"], c["kv_heads"], c["dim"]
    if c["kind"] == "rotate":
        T = c["tokens"]
        return {"bytes": 2 * T * (Hq + H) * D * size + 4 * T, "flops": 8.0 * T * (Hq + H) * D}
    total, new = lengths(c)
    T = int(new.sum())
    if c["kind"] == "append":
        return {"bytes": 2 * T * Hq * D * size + 2 * T * H * (D * (size + 1) + 4.0 / c["page"]),
                "flops": 8.0 * T * (Hq + H) * D + 4.0 * T * H * D}
    keys = int(prefixes(c).sum() + (total - np.repeat(prefixes(c), c["seqs"])).sum())
    pairs = sum(int((np.arange(t - m, t) + 1).sum()) for t, m in zip(total.tolist(), new.tolist()))
    return {"bytes": 2 * keys * H * (D + 4.0 / c["page"]) + 2 * T * Hq * D * size, "flops": 4.0 * D * Hq * pairs}


# ------------------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"int4": exact_int4, "rotate": exact_rotate, "append": exact_append, "shared": exact_shared}[case["kind"]](s)


def exact_int4(s):
    c = s["case"]
    out = torch.zeros((c["rows"], c["n"]), dtype=torch.float64, device=s["w"].device)
    for a in range(0, c["n"], 4096):                       # a block of outputs at a time
        low = (s["w"][a:a + 4096] & 15).double()
        high = (s["w"][a:a + 4096] // 16).double()
        scale = s["scale"][a:a + 4096].double().repeat_interleave(GROUP // 2, 1)
        low, high = (torch.where(v > 7, v - 16, v) * scale for v in (low, high))
        out[:, a:a + 4096] = s["x"][:, 0::2].double() @ low.T + s["x"][:, 1::2].double() @ high.T
    for more in (s["bias"], s["add"]):
        if more is not None:
            out += more.double()
    return out


def exact_turn(s, x, weight, pos):
    """The same as plain_rotate from its definition: each pair as a complex number times e^(i angle)."""
    c = s["case"]
    x = x.double().clone()
    if c["norm"]:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / c["dim"] + EPS) * weight.double()
    R = c["rot"]
    first = torch.arange(0, R, 2, device=x.device) if c["interleaved"] else torch.arange(R // 2, device=x.device)
    second = first + (1 if c["interleaved"] else R // 2)
    z = torch.complex(x[..., first], x[..., second])
    angle = pos.double()[:, None, None] * s["freq"]
    z = z * torch.polar(torch.full_like(angle, s["amp"]), angle)
    x[..., first], x[..., second] = z.real, z.imag
    return x


def exact_rotate(s):
    return exact_turn(s, s["q"], s["q_norm"], s["pos"]), exact_turn(s, s["k_new"], s["k_norm"], s["pos"])


def exact_append(s):
    P = s["case"]["page"]
    start, total = s["start"].tolist(), s["length"].tolist()
    pos = torch.cat([torch.arange(n - (b - a), n, device=s["q"].device) for n, a, b in zip(total, start, start[1:])])
    got = dict(q=exact_turn(s, s["q"], s["q_norm"], pos))
    for name, x in (("k", exact_turn(s, s["k_new"], s["k_norm"], pos)), ("v", s["v_new"].double())):
        pool = s[name][0].view(torch.uint8)
        value = s[name].clone()
        codes = value[0].view(torch.uint8)
        scale = s[name + "_scale"].double()
        for i, n in enumerate(total):
            at = n - (start[i + 1] - start[i])
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


def exact_shared(s):
    """One sequence and kv head at a time, straight from the definition: each reads all of its own table row."""
    c = s["case"]
    H, P, Q = c["kv_heads"], c["page"], c["new"]
    G = c["heads"] // H
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    for i, total in enumerate(s["length"].tolist()):
        j = torch.arange(total, device=out.device)
        page = s["table"][i].long()[j // P]
        see = j[None, :] <= torch.arange(total - Q, total, device=out.device)[:, None]
        k, v = (s[name][0].view(torch.uint8)[page, :, j % P].view(E4M3).double() * s[name + "_scale"][0][page].double()[..., None]
                for name in ("k", "v"))                              # [keys, H, D]
        q = s["q"][i * Q:(i + 1) * Q].double().view(Q, H, G, -1)
        x = torch.einsum("qhgd,khd->hgqk", q, k) * s["scale"]
        p = torch.softmax(x.masked_fill(~see, -math.inf), -1)
        out[i * Q:(i + 1) * Q] = torch.einsum("hgqk,khd->qhgd", p, v).reshape(Q, H * G, -1)
    return out
