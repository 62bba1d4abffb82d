"""Cases of the attention operators over a paged key-value cache: what is timed, and what it is
compared with.

Three operators make up the attention of one Transformer layer between its column-parallel Q/K/V
projection and its row-parallel output projection:

  append   rotates the new tokens' queries and keys by their positions and writes the keys and
           values into the cache's pages
  decode   attention of one new token of each sequence over its whole cache
  prompt   causal attention of a chunk of new tokens of each sequence over its cache

The cache is two pools [pages, kv heads, page size, head size], in bf16 or in e4m3 with one fp32
scale per kv head, and a page table [sequences, pages]. `run` computes an operator in its plain
form, from elementary torch operations in 32 bits, or (with `own`) calls the library's.
"""
import math
import random

import torch

own = False

THETA = 10000.0


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one generated token of a 7B-shaped layer: the smallest call of every decode step
        dict(name="append_one_token", op="append", B=1, T=1, len=2047, Hq=32, Hkv=32, D=128,
             page=16, kv="bf16", rot=128, pairs="halves"),
        # one token of each of 256 sequences, grouped heads, half of each head rotated, 8-bit cache
        dict(name="append_batch_e4m3", op="append", B=256, T=256, len=1001, Hq=96, Hkv=8, D=128,
             page=32, kv="e4m3", rot=64, pairs="neighbours"),
        # the prompts of a prefill batch
        dict(name="append_prompts", op="append", B=11, T=16384, len=2500, Hq=32, Hkv=8, D=128,
             page=64, kv="bf16", rot=128, pairs="halves"),
        # one sequence of a GPT-2-small-shaped layer: latency
        dict(name="decode_one_gpt2", op="decode", B=1, len=777, ragged=False, Hq=12, Hkv=12, D=64,
             page=16, kv="bf16", window=0),
        # a serving batch of a 7B-shaped layer, every head with its own keys
        dict(name="decode_batch_7b", op="decode", B=64, len=8192, ragged=True, Hq=32, Hkv=32,
             D=128, page=16, kv="bf16", window=0),
        # one sequence with a long cache: the work has to be split over its length
        dict(name="decode_long_one", op="decode", B=1, len=131072, ragged=False, Hq=32, Hkv=8,
             D=128, page=64, kv="bf16", window=0),
        # a ragged batch over an 8-bit cache, 12 query heads to a kv head
        dict(name="decode_batch_e4m3", op="decode", B=48, len=8191, ragged=True, Hq=96, Hkv=8,
             D=128, page=32, kv="e4m3", window=0),
        # a sliding window over longer caches
        dict(name="decode_window", op="decode", B=17, len=20011, ragged=True, Hq=32, Hkv=4, D=128,
             page=128, kv="bf16", window=4096),
        # a short prompt of a GPT-2-small-shaped layer: latency
        dict(name="prompt_short_gpt2", op="prompt", B=1, new=61, len=61, ragged=False, Hq=12,
             Hkv=12, D=64, page=16, kv="bf16", window=0),
        # a prefill batch of ragged prompts, grouped heads
        dict(name="prompt_ragged", op="prompt", B=8, new=2048, len=2048, ragged=True, Hq=32, Hkv=8,
             D=128, page=64, kv="bf16", window=0),
        # one prompt of a GPT-3-175B-shaped layer
        dict(name="prompt_gpt3", op="prompt", B=1, new=4096, len=4096, ragged=False, Hq=96, Hkv=96,
             D=128, page=64, kv="bf16", window=0),
        # chunks of two long prompts over an 8-bit cache
        dict(name="prompt_chunk_e4m3", op="prompt", B=2, new=1000, len=24000, ragged=False, Hq=32,
             Hkv=8, D=128, page=32, kv="e4m3", window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "prompt"])
    kv = rng.choice(["bf16", "e4m3"])
    page = rng.choice([16, 32, 64, 128])
    D = rng.choice([64, 128, 128])
    while True:
        Hkv = rng.choice([1, 2, 4, 5, 8, 8, 12, 16, 32])
        Hq = Hkv * rng.choice([1, 1, 2, 3, 4, 6, 8, 12, 16])
        if Hq > 96:
            continue
        c = dict(op=op, Hq=Hq, Hkv=Hkv, D=D, page=page, kv=kv)
        if op == "append":
            T = _log(rng, 1, 16384)
            c.update(B=min(T, _log(rng, 1, 64)), T=T, len=_log(rng, 64, 4096),
                     rot=rng.choice([D, D, D // 2]), pairs=rng.choice(["halves", "neighbours"]))
            c["len"] = max(c["len"], -(-T // c["B"]))
            if c["B"] * c["len"] * Hkv * D <= 2 ** 27 and T * (Hq + Hkv) * D <= 16384 * 40 * 128:
                return c
        elif op == "decode":
            c.update(B=_log(rng, 1, 128), len=_log(rng, 16, 131072), ragged=rng.random() < 0.7,
                     window=rng.choice([0, 0, 0, 1024]))
            if c["B"] * c["len"] * Hkv * D <= 2 ** 29:
                return c
        else:
            c.update(B=_log(rng, 1, 16), new=_log(rng, 2, 4096), ragged=rng.random() < 0.7,
                     window=rng.choice([0, 0, 0, 1024]))
            c["len"] = c["new"] + rng.choice([0, 0, _log(rng, 1, 16000)])
            if (c["B"] * c["new"] * c["len"] * Hq <= 2 ** 29
                    and c["B"] * c["len"] * Hkv * D <= 2 ** 28):
                return c


def _lengths(case):
    """(keys, new tokens) of each sequence."""
    r = random.Random("%(op)s %(B)d %(len)d" % case)
    B, most = case["B"], case["len"]
    if case["op"] == "append":
        T = case["T"]
        cut = sorted(r.randint(0, T - B) for _ in range(B - 1))  # at least one token each
        new = [b - a + 1 for a, b in zip([0] + cut, cut + [T - B])]
        return [max(most, n) for n in new], new
    if case["op"] == "decode":
        keys = [r.randint(1, most) if case["ragged"] else most for _ in range(B)]
        keys[0] = most
        return keys, [1] * B
    past = most - case["new"]
    new = [r.randint(1, case["new"]) if case["ragged"] else case["new"] for _ in range(B)]
    new[0] = case["new"]
    keys = [n + (r.randint(0, past) if case["ragged"] else past) for n in new]
    keys[0] = most
    return keys, new


def work(case):
    keys, new = _lengths(case)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    size = 2 if case["kv"] == "bf16" else 1
    T = sum(new)
    if case["op"] == "append":
        return {"bytes": T * D * (2 * Hq * 2 + 2 * Hkv * 2 + 2 * Hkv * size) + 8 * T,
                "flops": 3 * T * (Hq + Hkv) * case["rot"]}
    w = case["window"] or max(keys)
    pairs = read = 0
    for s, n in zip(keys, new):
        read += min(s, w + n - 1)
        # query i of n sees min(s - n + 1 + i, w) keys
        full = max(0, min(n, w - (s - n)))  # queries that the window does not cut
        pairs += full * (s - n) + full * (full + 1) // 2 + (n - full) * w
    return {"bytes": 2 * T * Hq * D * 2 + 2 * read * Hkv * D * size, "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------------------ inputs
def _pool(shape, kv, g):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    # an 8-bit cache is filled with values scaled to its range
    return x if kv == "bf16" else x.mul_(60.0).to(torch.float8_e4m3fn)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    keys, new = _lengths(case)
    B, Hq, Hkv, D, page = case["B"], case["Hq"], case["Hkv"], case["D"], case["page"]
    pages = [-(-n // page) for n in keys]
    width, total = max(pages), sum(pages)
    ids = torch.randperm(total + 3, generator=g, device="cuda").to(torch.int32)
    at = torch.tensor([0] + pages, device="cuda").cumsum(0)[:-1, None]
    column = torch.arange(width, device="cuda")[None, :]
    table = ids[torch.clamp(at + column, max=total + 2)].contiguous()
    s = dict(case=case, table=table, B=B, Hq=Hq, Hkv=Hkv, D=D, page=page, width=width,
             K=_pool((total + 3, Hkv, page, D), case["kv"], g),
             V=_pool((total + 3, Hkv, page, D), case["kv"], g),
             lens=torch.tensor(keys, dtype=torch.int32, device="cuda"),
             k_scale=None, v_scale=None)
    if case["kv"] != "bf16":
        s["k_scale"] = 1 / 64 + torch.rand(Hkv, generator=g, device="cuda") / 64
        s["v_scale"] = 1 / 64 + torch.rand(Hkv, generator=g, device="cuda") / 64
    T = sum(new)
    if case["op"] == "append":
        qkv = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g, device="cuda",
                          dtype=torch.bfloat16)
        s["q"], s["k"], s["v"] = qkv.split([Hq * D, Hkv * D, Hkv * D], dim=1)
        s["q_out"] = torch.empty((T, Hq * D), device="cuda", dtype=torch.bfloat16)
        s["seq"] = torch.tensor([b for b, n in enumerate(new) for _ in range(n)],
                                dtype=torch.int32, device="cuda")
        s["pos"] = torch.tensor([m - n + i for m, n in zip(keys, new) for i in range(n)],
                                dtype=torch.int32, device="cuda")
        rot = case["rot"]
        s["freq"] = THETA ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    else:
        s["q"] = torch.randn((T, Hq * D), generator=g, device="cuda", dtype=torch.bfloat16)
        s["out"] = torch.empty((T, Hq * D), device="cuda", dtype=torch.bfloat16)
        s["scale"] = D ** -0.5
        s["most_new"] = max(new)
        s["cu"] = torch.tensor([0] + new, device="cuda").cumsum(0).to(torch.int32)
    if own:
        import tensor_transformer_mlp_tmem_gb300 as tp
        s["attn"] = tp.Attention(Hq, Hkv, D, page, kv_dtype=case["kv"])
        if case["kv"] != "bf16":
            s["attn"].set_scales(s["k_scale"], s["v_scale"])
        if case["op"] == "append":
            s["attn"].set_rope(case["rot"], THETA, interleaved=case["pairs"] == "neighbours")
        s["cache"] = tp.PagedCache(s["attn"], s["K"], s["V"], s["table"], s["lens"])
    return s


# ------------------------------------------------------------------ the operators, plain
def _rotate(x, cos, sin, rot, pairs):
    """x fp32 [T, heads, D]; cos, sin fp32 [T, 1, rot / 2]."""
    y = x.clone()
    if pairs == "halves":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2] = a * cos - b * sin
        y[..., rot // 2:rot] = b * cos + a * sin
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2] = a * cos - b * sin
        y[..., 1:rot:2] = b * cos + a * sin
    return y


def _store(pool, page, slot, x, scale):
    """Rows x fp32 [T, kv heads, D] into their pages."""
    if scale is None:
        pool[page, :, slot] = x.to(pool.dtype)
    else:
        x = (x / scale[None, :, None]).clamp(-448.0, 448.0).to(pool.dtype)
        pool.view(torch.uint8)[page, :, slot] = x.view(torch.uint8)


def _append(s):
    c, D = s["case"], s["D"]
    T = s["q"].shape[0]
    angle = s["pos"].double()[:, None, None] * s["freq"]
    cos, sin = angle.cos().float(), angle.sin().float()
    q = _rotate(s["q"].float().view(T, -1, D), cos, sin, c["rot"], c["pairs"])
    k = _rotate(s["k"].float().view(T, -1, D), cos, sin, c["rot"], c["pairs"])
    s["q_out"].copy_(q.view(T, -1))
    pos = s["pos"].long()
    page = s["table"][s["seq"].long(), pos // s["page"]].long()
    _store(s["K"], page, pos % s["page"], k, s["k_scale"])
    _store(s["V"], page, pos % s["page"], s["v"].float().view(T, -1, D), s["v_scale"])
    return s["q_out"], s["K"], s["V"]


def _gathered(s, pool, scale):
    """The sequences' rows, fp32 [B, kv heads, keys, D] (keys: the widest sequence's pages)."""
    raw = pool if scale is None else pool.view(torch.uint8)
    x = raw[s["table"].long()]  # [B, width, heads, page, D]
    x = x.transpose(1, 2).reshape(s["B"], s["Hkv"], s["width"] * s["page"], s["D"])
    return x.float() if scale is None else x.view(pool.dtype).float() * scale[:, None, None]


def _attend(s, q, first):
    """q fp32 [B, n, Hq, D], query i of sequence b at position first[b] + i: fp32 alike."""
    B, n = q.shape[:2]
    Hkv, D, w = s["Hkv"], s["D"], s["case"]["window"]
    G = s["Hq"] // Hkv
    key = torch.arange(s["width"] * s["page"], device="cuda")
    K = _gathered(s, s["K"], s["k_scale"])
    q = q.view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    p = torch.matmul(q, K.transpose(2, 3)).mul_(s["scale"]).view(B, Hkv, G, n, -1)
    del K
    at = first[:, None] + torch.arange(n, device="cuda")  # [B, n]
    hide = key > at[:, :, None]
    if w:
        hide |= key <= at[:, :, None] - w
    p.masked_fill_(hide[:, None, None], -math.inf)
    p.sub_(p.amax(-1, keepdim=True)).exp_()
    p.div_(p.sum(-1, keepdim=True))
    V = _gathered(s, s["V"], s["v_scale"])
    V.masked_fill_((key >= s["lens"][:, None])[:, None, :, None], 0.0)
    o = torch.matmul(p.view(B, Hkv, G * n, -1), V)
    return o.view(B, Hkv, G, n, D).permute(0, 3, 1, 2, 4)  # [B, n, Hkv, G, D]


def _decode(s):
    B = s["B"]
    o = _attend(s, s["q"].float().view(B, 1, s["Hq"], s["D"]), s["lens"].long() - 1)
    s["out"].copy_(o.reshape(B, -1))
    return s["out"]


def _prompt(s):
    n = s["most_new"]
    new = (s["cu"][1:] - s["cu"][:-1]).long()
    # packed rows [T] -> padded [B, n], and back
    token = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(s["cu"].long(), token, right=True) - 1
    i = token - s["cu"].long()[b]
    q = torch.zeros((s["B"], n, s["Hq"], s["D"]), device="cuda")
    q[b, i] = s["q"].float().view(-1, s["Hq"], s["D"])
    o = _attend(s, q, s["lens"].long() - new)
    s["out"].copy_(o[b, i].reshape(-1, s["Hq"] * s["D"]))
    return s["out"]


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if not own:
        return {"append": _append, "decode": _decode, "prompt": _prompt}[op](s)
    attn, cache = s["attn"], s["cache"]
    if op == "append":
        attn.append(s["q"], s["k"], s["v"], cache, s["pos"], s["seq"], q_out=s["q_out"])
        return s["q_out"], s["K"], s["V"]
    window = s["case"]["window"]
    if op == "decode":
        return attn.decode(s["q"], cache, s["scale"], window, out=s["out"])
    return attn.prompt(s["q"], s["cu"], cache, s["scale"], window, out=s["out"])


# ------------------------------------------------------------------ the definition, in 64 bits
def _exact_append(s):
    rot, D, page = s["case"]["rot"], s["D"], s["page"]
    outs = [s["q"].double(), s["K"].double(), s["V"].double()]
    neighbours = s["case"]["pairs"] == "neighbours"
    turn = torch.exp(1j * s["pos"].double()[:, None] * s["freq"])[:, None, :]

    def turned(x):
        x = x.double().reshape(x.shape[0], -1, D)
        z, rest = x[..., :rot], x[..., rot:]
        if neighbours:
            z = torch.view_as_complex(z.reshape(*z.shape[:-1], rot // 2, 2).contiguous()) * turn
            z = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(z[..., :rot // 2].contiguous(), z[..., rot // 2:].contiguous()) * turn
            z = torch.cat([z.real, z.imag], -1)
        return torch.cat([z, rest], -1)

    outs[0] = turned(s["q"]).reshape(s["q"].shape)
    table = s["table"].tolist()
    pg = torch.tensor([table[b][p // page] for b, p in zip(s["seq"].tolist(), s["pos"].tolist())],
                      device="cuda")
    sl = s["pos"].long() % page
    for pool, x, scale in ((outs[1], turned(s["k"]), s["k_scale"]),
                           (outs[2], s["v"].double().reshape(len(sl), -1, D), s["v_scale"])):
        if scale is not None:
            x = torch.clamp(x / scale.double()[:, None], -448, 448)
        pool[pg, :, sl] = x
    return tuple(outs)


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    if case["op"] == "append":
        return _exact_append(s)
    keys, new = _lengths(case)
    Hq, Hkv, D, page = s["Hq"], s["Hkv"], s["D"], s["page"]
    G, out, t = Hq // Hkv, torch.empty(s["q"].shape, dtype=torch.float64, device="cuda"), 0
    for b, (m, n) in enumerate(zip(keys, new)):
        mine = s["table"][b, :-(-m // page)].long()
        for h in range(Hkv):
            k, v = (pool.view(torch.uint8 if case["kv"] != "bf16" else pool.dtype)[mine, h]
                    .view(pool.dtype).double().reshape(-1, D)[:m] for pool in (s["K"], s["V"]))
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            q = s["q"][t:t + n].view(n, Hkv, G, D)[:, h].double().reshape(n * G, D)
            i = (m - n + torch.arange(n, device="cuda")).repeat_interleave(G)[:, None]
            j = torch.arange(m, device="cuda")[None, :]
            seen = j <= i
            if case["window"]:
                seen &= i - j < case["window"]
            z = torch.where(seen, q @ k.T / math.sqrt(D), -math.inf)
            out[t:t + n].view(n, Hkv, G, D)[:, h] = (torch.softmax(z, -1) @ v).view(n, G, D)
        t += n
    return out
