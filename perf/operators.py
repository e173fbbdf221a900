"""The operators of streaming attention and the cases on which they are timed.

Four kinds of pass, over one family of visibility rules: a query at position i sees key j when
j lies in its sliding window (i - window < j <= i, or |i - j| < window where the attention is
not causal) or is one of the first `sinks` tokens (and j <= i where it is causal).

- "forward":  attention of a whole sequence under that rule (``sla2.window_forward``)
- "training": the same and its gradients (``sla2.window_backward``)
- "append":   keys and values of new tokens into a paged cache of 8-bit codes, one scale for each
              page and head, the rotation of queries and keys applied on the way
              (``sla2.cache_append``)
- "decode":   attention of the newest tokens over that cache (``sla2.cache_attention``)

``run`` computes a pass in its plain form, in elementary torch operations, or, where ``own`` is
set, through the framework's calls.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ the cases

def _window(name, kind, B, Hq, Hkv, N, d, dtype, window, sinks, causal, padded):
    return {"name": name, "kind": kind, "B": B, "Hq": Hq, "Hkv": Hkv, "N": N, "d": d, "dtype": dtype,
            "window": window, "sinks": sinks, "causal": causal, "padded": padded}


def _append(name, B, Hq, Hkv, d, dtype, page, old, new, rot, interleaved):
    return {"name": name, "kind": "append", "B": B, "Hq": Hq, "Hkv": Hkv, "d": d, "dtype": dtype, "page": page,
            "old": old, "new": new, "rot": rot, "interleaved": interleaved}


def _decode(name, B, Hq, Hkv, d, dtype, page, old, new, window, sinks):
    return {"name": name, "kind": "decode", "B": B, "Hq": Hq, "Hkv": Hkv, "d": d, "dtype": dtype, "page": page,
            "old": old, "new": new, "window": window, "sinks": sinks}


def listed():
    return [
        # a short clip in a small model: five query blocks, latency counts
        _window("forward short", "forward", 2, 3, 3, 640, 64, "bf16", 128, 4, True, False),
        # a padded batch of clips of unlike length (one of them empty), both directions, shared key heads
        _window("forward padded", "forward", 4, 16, 4, 4999, 128, "fp16", 512, 16, False, True),
        # one whole video of 32768 tokens, 12 heads of 128, generated in order
        _window("forward long", "forward", 1, 12, 12, 32768, 128, "bf16", 2048, 64, True, False),
        # one step of fine-tuning on a short sequence of odd length
        _window("training short", "training", 1, 4, 2, 515, 64, "fp16", 100, 3, False, False),
        # a training batch of padded sequences, three query heads to a key head
        _window("training padded", "training", 3, 24, 8, 4096, 64, "bf16", 512, 8, True, True),
        # a training step on a long video
        _window("training long", "training", 1, 12, 12, 16384, 128, "bf16", 1024, 64, True, False),
        # one step of generation: one token for each of 32 sequences
        _append("append one each", 32, 32, 8, 128, "bf16", 64, 4096, 1, 128, False),
        # prompts of unlike length into empty and part-filled caches
        _append("append prompts", 5, 12, 4, 128, "fp16", 128, 300, 4001, 64, True),
        # one short sequence, every token visible: the smallest step
        _decode("decode one", 1, 12, 12, 64, "bf16", 16, 1000, 1, 0, 0),
        # a full server: 64 sequences of unlike length, four query heads to a key head
        _decode("decode batch", 64, 32, 8, 128, "bf16", 64, 8192, 1, 0, 0),
        # long videos through a window with sinks, a few tokens of each at once
        _decode("decode window", 24, 16, 2, 128, "fp16", 32, 65536, 4, 4096, 64),
        # two very long sequences, all of them visible, eight query heads to a key head
        _decode("decode long", 2, 16, 2, 128, "bf16", 128, 200000, 1, 0, 0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["forward", "training", "append", "decode"])
    d, dtype = rng.choice([64, 128]), rng.choice(["bf16", "fp16"])
    Hkv, group = rng.choice([1, 2, 3, 4, 8, 12]), rng.choice([1, 2, 3, 4, 7, 8])
    if kind in ("forward", "training"):
        top = 32768 if kind == "forward" else 16384
        while True:
            B, N = rng.choice([1, 1, 2, 3, 4]), _log(rng, 64, top)
            window = _log(rng, 1, 4 * top // 32)
            group = rng.choice([1, 2, 3, 4])
            c = _window("", kind, B, Hkv * group, Hkv, N, d, dtype, window, rng.choice([0, 1, 4, 16, 64, 130]),
                        rng.random() < 0.6, rng.random() < 0.4)
            span = min(N, window * (1 if c["causal"] else 2) + 256)
            # no dearer than the dearest listed case of the kind
            if B * c["Hq"] * N * span * d <= (12 * 32768 * 2304 * 128 if kind == "forward" else 12 * 16384 * 1280 * 128):
                break
    elif kind == "append":
        while True:
            B, new = _log(rng, 1, 256), rng.choice([1, 1, 1, 2, 5, _log(rng, 8, 8192)])
            c = _append("", B, Hkv * group, Hkv, d, dtype, rng.choice([16, 32, 64, 128]), _log(rng, 1, 16384), new,
                        rng.choice([d, d // 2, d - 16]), rng.random() < 0.5)
            if B * new * Hkv * d <= 20000 * 4 * 128 and B * (new + 2 * c["page"]) * Hkv * d <= 1 << 24:
                break
    else:
        while True:
            B, old = _log(rng, 1, 128), _log(rng, 1, 200000)
            window = rng.choice([0, 0, _log(rng, 16, 16384)])
            c = _decode("", B, Hkv * group, Hkv, d, dtype, rng.choice([16, 32, 64, 128]), old, rng.choice([1, 1, 1, 2, 4, 7]),
                        window, rng.choice([0, 4, 64, 100]) if window else 0)
            if B * old * Hkv * d <= 64 * 8192 * 8 * 128 and B * c["new"] * old * c["Hq"] * d <= 1 << 33:
                break
    c.pop("name")
    return c


def _spread(n, lo, hi):
    """n whole numbers between lo and hi, unlike one another, the last of them hi."""
    return [hi if b == n - 1 else lo + int((hi - lo) * ((b + 1) * 0.6180339887 % 1.0)) for b in range(n)]


def _lens(case):
    """The sequences' lengths: of a padded batch, the second of four or more empty."""
    B, N = case["B"], case["N"]
    if not case["padded"]:
        return [N] * B
    lens = _spread(B, N // 3, N)
    if B >= 4:
        lens[1] = 0
    return lens


def _old_new(case):
    """Tokens in the cache before the pass, and new ones, of each sequence."""
    B, old, new = case["B"], case["old"], case["new"]
    if case["kind"] == "append":
        olds = _spread(B, 0, old)
        news = [new] * B if new < 8 else _spread(B, max(1, new // 8), new)
        if B >= 4 and new >= 8:
            olds[0], news[1] = 0, 0           # an empty cache, and a sequence with nothing new
    else:
        olds = _spread(B, old // 2, old)
        news = [new] * B
    return olds, news


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt, d = DTYPES[case["dtype"]], case["d"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    s = dict(case)
    if case["kind"] in ("forward", "training"):
        B, Hq, Hkv, N = case["B"], case["Hq"], case["Hkv"], case["N"]
        # heads side by side in each token's row, as a projection leaves them
        s["q"] = normal(B, N, Hq, d).to(dt).transpose(1, 2)
        s["k"] = normal(B, N, Hkv, d).to(dt).transpose(1, 2)
        s["v"] = normal(B, N, Hkv, d).to(dt).transpose(1, 2)
        s["lens"] = ints(_lens(case)) if case["padded"] else None
        if case["kind"] == "training":
            s["dout"] = normal(B, N, Hq, d).to(dt).transpose(1, 2)
        return s

    B, Hq, Hkv, page = case["B"], case["Hq"], case["Hkv"], case["page"]
    olds, news = _old_new(case)
    T = sum(news)
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    s["kv_lens"], s["cu_new"] = ints(olds), ints(cu)
    held = [-(-(o + n) // page) for o, n in zip(olds, news)]     # pages of each sequence
    width = max(held)
    append = case["kind"] == "append"
    # an append reaches the pages from the last part-filled one on; the others stay out of the case's memory
    first = [o // page if append else 0 for o in olds]
    total = sum(max(h - f, 0) for h, f in zip(held, first)) + 1
    order = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    counts, starts = torch.tensor([max(h - f, 0) for h, f in zip(held, first)]), torch.tensor(first)
    ids = torch.repeat_interleave(torch.arange(B), counts)
    begin = torch.cumsum(counts, 0) - counts
    at = torch.arange(total - 1) - begin[ids] + starts[ids]
    table = torch.full((B, max(width, 1)), -1, dtype=torch.int32, device=dev)
    table[ids.to(dev), at.to(dev)] = order[:total - 1]
    s["page_table"] = table

    def cached():
        x = normal(total, Hkv, page, d)
        x *= (0.5 + torch.rand(total, Hkv, 1, 1, generator=g, device=dev))
        scale = x.abs().amax((2, 3)) / 127
        return x.div_(scale[..., None, None]).round_().to(torch.int8), scale

    s["k_codes"], s["k_scale"] = cached()
    s["v_codes"], s["v_scale"] = cached()
    s["q"] = normal(T, Hq, d).to(dt)
    if append:
        s["k"], s["v"] = normal(T, Hkv, d).to(dt), normal(T, Hkv, d).to(dt)
        far = max(o + n for o, n in zip(olds, news))
        rate = 10000.0 ** (-torch.arange(case["rot"] // 2, device=dev, dtype=torch.float64) * 2 / case["rot"])
        angle = torch.arange(far, device=dev, dtype=torch.float64)[:, None] * rate
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    if own:
        from block_sparse_linear_router_b200 import sla2
        s["cache"] = sla2.KVCache(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    kind = state["kind"]
    if kind == "append":
        (_own_append if own else _plain_append)(state)
        # the cache as the values that its codes stand for
        return {"k": state["k_codes"] * state["k_scale"][..., None, None],
                "v": state["v_codes"] * state["v_scale"][..., None, None],
                "k_scale": state["k_scale"], "v_scale": state["v_scale"], "q": state["q_rot"]}
    if own:
        return {"forward": _own_forward, "training": _own_training, "decode": _own_decode}[kind](state)
    return {"forward": _plain_window, "training": _plain_window, "decode": _plain_decode}[kind](state)


def _rule(s):
    return {"window": s["window"], "sinks": s["sinks"], "causal": s["causal"], "lens": s["lens"]}


def _own_forward(s):
    from block_sparse_linear_router_b200 import sla2
    out, lse = sla2.window_forward(s["q"], s["k"], s["v"], return_lse=True, **_rule(s))
    return {"out": out, "lse": lse}


def _own_training(s):
    from block_sparse_linear_router_b200 import sla2
    out, lse = sla2.window_forward(s["q"], s["k"], s["v"], return_lse=True, **_rule(s))
    dq, dk, dv = sla2.window_backward(s["q"], s["k"], s["v"], out, lse, s["dout"], **_rule(s))
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def _own_append(s):
    from block_sparse_linear_router_b200 import sla2
    s["q_rot"] = sla2.cache_append(s["cache"], s["k"], s["v"], s["page_table"], s["kv_lens"], s["cu_new"],
                                   rope=(s["cos"], s["sin"]), interleaved=s["interleaved"], q=s["q"])


def _own_decode(s):
    from block_sparse_linear_router_b200 import sla2
    return sla2.cache_attention(s["cache"], s["q"], s["page_table"], s["kv_lens"], s["cu_new"],
                                window=s["window"] or None, sinks=s["sinks"])


# ------------------------------------------------------------------ plain forms

def _plain_window(s):
    """Query blocks of 256 against the sinks and the band of keys that any query of the block sees."""
    q, k, v, S, causal = s["q"], s["k"], s["v"], s["sinks"], s["causal"]
    B, Hq, N, d = q.shape
    Hkv = k.shape[1]
    g, C, dev = Hq // Hkv, 256, q.device
    W, S = min(s["window"], N), min(s["sinks"], N)
    nb = -(-N // C)
    first = torch.arange(nb, device=dev)[:, None] * C
    band = first - (W - 1) + torch.arange(W - 1 + C + (0 if causal else W - 1), device=dev)
    idx = torch.cat([torch.arange(S, device=dev).expand(nb, S), band], 1)                      # [nb, M]
    M = idx.shape[1]
    sink = (torch.arange(M, device=dev) < S).expand(nb, M)
    i = (first + torch.arange(C, device=dev))[:, :, None]                                      # [nb, C, 1]
    j, sink = idx[:, None, :], sink[:, None, :]
    near = (j > i - W) & ((j <= i) if causal else (j < i + W)) & (j >= S)
    seen = torch.where(sink, (j <= i) if causal else (j >= 0), near) & (j >= 0)
    lens = s["lens"] if s["lens"] is not None else torch.full((B,), N, device=dev)
    L = lens.view(B, 1, 1, 1)
    seen = (seen[None] & (j[None] < L) & (i[None] < L))[:, None, :, None]                       # [B,1,nb,1,C,M]

    at = idx.clamp(0, N - 1).reshape(-1)
    kg = k[:, :, at].float().view(B, Hkv, nb, M, d)
    vg = v[:, :, at].float().view(B, Hkv, nb, M, d)

    def blocks(x):  # [B, Hq, N, d] -> [B, Hkv, nb, g * C, d]
        x = torch.cat([x.float(), x.new_zeros(B, Hq, nb * C - N, d, dtype=torch.float32)], 2)
        return x.view(B, Hkv, g, nb, C, d).transpose(2, 3).reshape(B, Hkv, nb, g * C, d)

    def rows(x):    # the inverse, for [B, Hkv, nb, g * C, n]
        n = x.shape[-1]
        return x.view(B, Hkv, nb, g, C, n).transpose(2, 3).reshape(B, Hq, nb * C, n)[:, :, :N]

    scale = 1 / math.sqrt(d)
    qb = blocks(q)
    x = (qb @ kg.transpose(-1, -2)).mul_(scale).view(B, Hkv, nb, g, C, M).masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (top + total.log()).view(B, Hkv, nb, g * C, 1)
    p = p.div_(torch.where(total > 0, total, 1)).view(B, Hkv, nb, g * C, M)
    o = p @ vg
    res = {"out": rows(o).to(q.dtype), "lse": rows(lse)[..., 0]}
    if s["kind"] == "forward":
        return res
    do = blocks(s["dout"])
    ds = (do @ vg.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    res["dq"] = rows(ds @ kg).to(q.dtype)
    for name, grad in (("dk", ds.transpose(-1, -2) @ qb), ("dv", p.transpose(-1, -2) @ do)):
        # what a clamped place gathered has a weight of zero
        res[name] = torch.zeros(B, Hkv, N, d, device=dev).index_add_(2, at, grad.reshape(B, Hkv, nb * M, d)).to(q.dtype)
    return res


def _rotated(x, cos, sin, rot, interleaved):
    """x [T, H, d] turned by the angles of its token (in 64 bits, rounded once to x's type)."""
    c, n, y = cos.double()[:, None], sin.double()[:, None], x.double()
    if interleaved:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat([a * c - b * n, b * c + a * n], -1)
    return torch.cat([turned, y[..., rot:]], -1).to(x.dtype)


def _plain_append(s):
    page, table, old, cu = s["page"], s["page_table"], s["kv_lens"].long(), s["cu_new"].long()
    T = s["k"].shape[0]
    t = torch.arange(T, device=table.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    pos = old[b] + t - cu[b]
    cos, sin = s["cos"][pos], s["sin"][pos]
    s["q_rot"] = _rotated(s["q"], cos, sin, s["rot"], s["interleaved"])
    pid, slot = table[b, pos // page].long(), pos % page
    # tokens that the touched pages held before: those of the page that a sequence goes on filling
    pages = s["k_codes"].shape[0]
    going = (cu[1:] > cu[:-1]) & (old % page > 0)
    front = torch.where(going, table.gather(1, (old // page).clamp(max=table.shape[1] - 1)[:, None])[:, 0].long(), pages)
    held = torch.zeros(pages + 1, dtype=torch.int64, device=t.device).scatter_(0, front, torch.where(going, old % page, 0))[:pages]
    new = torch.zeros(pages, dtype=torch.bool, device=t.device).index_fill_(0, pid, True)
    kept = torch.arange(page, device=t.device) < held[:, None]
    for codes, scale, x in ((s["k_codes"], s["k_scale"], _rotated(s["k"], cos, sin, s["rot"], s["interleaved"])),
                            (s["v_codes"], s["v_scale"], s["v"])):
        x = x.float()
        most = torch.zeros_like(scale).index_reduce_(0, pid, x.abs().amax(-1), "amax")
        now = torch.maximum(torch.where(held[:, None] > 0, scale, 0), (most.double() / 127).float())
        now = torch.where(new[:, None], now, scale)
        ratio = torch.where(now > 0, scale.double() / now.double(), 0)
        again = (codes.double() * ratio[..., None, None]).round_().to(torch.int8)
        codes.copy_(torch.where((kept & new[:, None])[:, None, :, None], again, codes))
        at = now[pid][..., None].double()
        codes[pid, :, slot] = torch.where(at > 0, x.double() / at, 0).round_().to(torch.int8)
        scale.copy_(now)


def _plain_decode(s):
    page, table, q, dev = s["page"], s["page_table"], s["q"], s["q"].device
    old, cu = s["kv_lens"].long(), s["cu_new"].long()
    B, (T, Hq, d), Hkv = table.shape[0], q.shape, s["Hkv"]
    g, n = Hq // Hkv, s["new"]
    L = table.shape[1] * page

    def values(codes, scale):   # [B, Hkv, L, d], zero where the sequence has no page
        at = table.clamp(min=0).long()
        x = codes[at].float().mul_(scale[at][..., None, None])                  # [B, pages, Hkv, page, d]
        return x.transpose(1, 2).reshape(B, Hkv, L, d)

    t = cu[:-1, None] + torch.arange(n, device=dev)                              # [B, n]
    pos = (old[:, None] + torch.arange(n, device=dev))[:, None, None, :, None]
    j = torch.arange(L, device=dev)
    seen = (j <= pos) & ((j > pos - s["window"]) | (j < s["sinks"]) if s["window"] else (j >= 0))
    qb = q[t].float().view(B, n, Hkv, g, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, g * n, d)
    x = (qb @ values(s["k_codes"], s["k_scale"]).transpose(-1, -2)).mul_(1 / math.sqrt(d)).view(B, Hkv, g, n, L)
    x = x.masked_fill_(~seen, -math.inf)
    p = x.sub_(x.amax(-1, keepdim=True)).exp_()
    p = p.div_(p.sum(-1, keepdim=True)).view(B, Hkv, g * n, L)
    o = (p @ values(s["v_codes"], s["v_scale"])).view(B, Hkv, g, n, d).permute(0, 3, 1, 2, 4)
    return o.reshape(T, Hq, d).to(q.dtype)


# ------------------------------------------------------------------ the definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "append":
        return _exact_append(s)
    if case["kind"] == "decode":
        return _exact_decode(s)
    return _exact_window(s)


def _softmax(x, seen):
    """Weights over what is seen (none where nothing is) and the logarithm of their sum."""
    x = torch.where(seen, x, -torch.inf)
    lse = torch.logsumexp(x, -1, keepdim=True)
    return torch.where(seen, torch.exp(x - torch.where(lse > -torch.inf, lse, 0)), 0), lse


def _exact_window(s):
    """Sequence by sequence and head by head, 1024 queries against every key that one of them may see."""
    q, k, v, W, S = s["q"], s["k"], s["v"], s["window"], s["sinks"]
    B, Hq, N, d = q.shape
    g = Hq // k.shape[1]
    train = s["kind"] == "training"
    f64 = {"dtype": torch.float64, "device": q.device}
    out, lse = torch.zeros(B, Hq, N, d, **f64), torch.full((B, Hq, N), -math.inf, **f64)
    dq, dk, dv = torch.zeros(B, Hq, N, d, **f64), torch.zeros(B, Hq // g, N, d, **f64), torch.zeros(B, Hq // g, N, d, **f64)
    for b in range(B):
        n = N if s["lens"] is None else int(s["lens"][b])
        for i0 in range(0, n, 1024):
            i1 = min(n, i0 + 1024)
            lo, hi = max(0, i0 - W + 1), i1 if s["causal"] else min(n, i1 + W - 1)
            j = torch.cat([torch.arange(0, min(S, lo), device=q.device), torch.arange(lo, hi, device=q.device)])
            if not s["causal"] and min(S, n) > hi:
                j = torch.cat([j, torch.arange(hi, min(S, n), device=q.device)])
            i = torch.arange(i0, i1, device=q.device)[:, None]
            dist = i - j
            seen = ((dist.abs() < W) | (j < S)) & ((dist >= 0) if s["causal"] else (j < n))
            for h in range(Hq):
                K, V, Q = k[b, h // g, j].double(), v[b, h // g, j].double(), q[b, h, i0:i1].double()
                p, z = _softmax(Q @ K.T / math.sqrt(d), seen)
                out[b, h, i0:i1], lse[b, h, i0:i1] = p @ V, z[:, 0]
                if train:
                    do = s["dout"][b, h, i0:i1].double()
                    dp = do @ V.T
                    ds = p * (dp - (p * dp).sum(-1, keepdim=True)) / math.sqrt(d)
                    dq[b, h, i0:i1] = ds @ K
                    dk[b, h // g, j] += ds.T @ Q
                    dv[b, h // g, j] += p.T @ do
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv} if train else {"out": out, "lse": lse}


def _exact_append(s):
    """The cache after the pass, sequence by sequence and page by page. A rotated key is rounded to
    its type and a scale to 32 bits before they are used; the codes' roundings are the operator's own."""
    page, rot, dt = s["page"], s["rot"], s["q"].dtype
    cache = {"k": [s["k_codes"].double(), s["k_scale"].double()], "v": [s["v_codes"].double(), s["v_scale"].double()]}
    olds, cus, table = s["kv_lens"].tolist(), s["cu_new"].tolist(), s["page_table"].tolist()
    turned = torch.empty_like(s["q"], dtype=torch.float64)
    for b, old in enumerate(olds):
        t0, t1 = cus[b], cus[b + 1]
        phase = torch.complex(s["cos"][old:old + t1 - t0].double(), s["sin"][old:old + t1 - t0].double())[:, None]

        def turn(x):
            y = x.double().clone()
            pairs = [slice(0, rot, 2), slice(1, rot, 2)] if s["interleaved"] else [slice(0, rot // 2), slice(rot // 2, rot)]
            z = torch.complex(y[..., pairs[0]], y[..., pairs[1]]) * phase
            y[..., pairs[0]], y[..., pairs[1]] = z.real, z.imag
            return y

        turned[t0:t1] = turn(s["q"][t0:t1])
        for name, x in (("k", turn(s["k"][t0:t1]).to(dt).double()), ("v", s["v"][t0:t1].double())):
            codes, scales = cache[name]
            at = old
            while at < old + t1 - t0:
                n = min(page - at % page, old + t1 - t0 - at)
                pid, c0, new = table[b][at // page], at % page, x[at - old:at - old + n].transpose(0, 1)   # [Hkv, n, d]
                most = (new.abs().amax((1, 2)) / 127).float().double()
                now = torch.maximum(most, scales[pid]) if c0 else most
                codes[pid, :, :c0] = torch.round(codes[pid, :, :c0] * (scales[pid] / now)[:, None, None])
                codes[pid, :, c0:c0 + n] = torch.round(new / now[:, None, None])
                scales[pid] = now
                at += n
    return {"k": cache["k"][0] * cache["k"][1][..., None, None], "v": cache["v"][0] * cache["v"][1][..., None, None],
            "k_scale": cache["k"][1], "v_scale": cache["v"][1], "q": turned}


def _exact_decode(s):
    page, W, S = s["page"], s["window"], s["sinks"]
    T, Hq, d = s["q"].shape
    g = Hq // s["Hkv"]
    out = torch.zeros(T, Hq, d, dtype=torch.float64, device=s["q"].device)
    olds, cus = s["kv_lens"].tolist(), s["cu_new"].tolist()
    for b, old in enumerate(olds):
        t0, t1 = cus[b], cus[b + 1]
        n = old + t1 - t0
        pages = s["page_table"][b, :-(-n // page)].long()
        j = torch.arange(n, device=out.device)
        i = torch.arange(old, n, device=out.device)[:, None]
        seen = (j <= i) & ((i - j < W) | (j < S)) if W else j <= i
        K, V = ((s[c][pages].double() * s[z][pages].double()[..., None, None]).transpose(0, 1).reshape(s["Hkv"], -1, d)[:, :n]
                for c, z in (("k_codes", "k_scale"), ("v_codes", "v_scale")))
        for h in range(Hq):
            p, _ = _softmax(s["q"][t0:t1, h].double() @ K[h // g].T / math.sqrt(d), seen)
            out[t0:t1, h] = p @ V[h // g]
    return out


# ------------------------------------------------------------------ what a pass cannot do without

def _pairs(n, W, S, causal):
    """(query, key) pairs that the rule lets through in a sequence of n tokens."""
    W, S = min(W, n), min(S, n)
    back = W * n - W * (W - 1) // 2                              # i - W < j <= i
    total = back if causal else 2 * back - n
    # sinks that lie outside the window: key j is behind it for the queries i >= j + W, and before it,
    # where the attention is not causal, for i <= j - W
    behind = sum(max(0, n - j - W) for j in range(S))
    before = 0 if causal else sum(max(0, j - W + 1) for j in range(S))
    return total + behind + before


def work(case):
    d, Hq, Hkv = case["d"], case["Hq"], case["Hkv"]
    if case["kind"] in ("forward", "training"):
        B, N, lens = case["B"], case["N"], _lens(case)
        pairs = Hq * sum(_pairs(n, case["window"], case["sinks"], case["causal"]) for n in lens)
        tokens = sum(lens)
        read = 2 * d * tokens * (Hq + 2 * Hkv)                   # q, k, v
        out = 2 * d * B * N * Hq + 4 * B * N * Hq                # out and lse, padding included
        if case["kind"] == "forward":
            return {"bytes": read + out, "flops": 4 * d * pairs}
        # and dout read, dq, dk, dv written; five products more than the forward pass's two
        return {"bytes": read + out + 2 * d * tokens * Hq + 2 * d * B * N * (Hq + 2 * Hkv), "flops": 14 * d * pairs}
    olds, news = _old_new(case)
    T, page = sum(news), case["page"]
    if case["kind"] == "append":
        rows = 2 * d * T * (Hq + 2 * Hkv) + 2 * d * T * Hq + 4 * case["rot"] * T    # q, k, v, rotated q, angles
        pages = sum(max(-(-(o + n) // page) - o // page, 0) for o, n in zip(olds, news)) + 1
        codes = 2 * Hkv * (T * d + 8 * pages)                    # codes written, scales read and written
        values = 2 * Hkv * pages * page * d * 5                  # the codes read and returned as values
        return {"bytes": rows + codes + values, "flops": 6 * T * d * (Hq + 2 * Hkv)}
    W, S, keys, pairs = case["window"], case["sinks"], 0, 0
    for o, n in zip(olds, news):
        keys += min(o + n, W + n - 1 + S) if W else o + n
        pairs += sum(min(o + i + 1, W + min(S, max(0, o + i + 1 - W))) if W else o + i + 1 for i in range(n))
    return {"bytes": 2 * Hkv * keys * (d + 4 / page) + 4 * d * T * Hq, "flops": 4 * d * Hq * pairs}
