"""The serving operators of the attention library, in plain torch and through the library.

Four operators that a generation loop uses one after the other:

* ``prompt``: attention over whole prompts of different lengths, packed one behind the other;
* ``store``:  key/value rows written into a cache that holds 4 bits an element, and read back;
* ``decode``: new query rows over that cache, with the attention weight that each cached token
  received added up where the cache is going to be thinned out;
* ``evict``:  the cache thinned out: the newest tokens and the heaviest of the others are kept.

The cache is a uint8 tensor [B, Hkv, blocks, 72 d] of blocks of 64 tokens: K codes [64][d / 2],
V codes [64][d / 2], K parameters [64][d / 64] (fp16 step, fp16 middle), V parameters.  A byte
holds channel 2i in its low and channel 2i + 1 in its high four bits; a code c of a group of 64
channels stands for middle + step (c - 8).
"""

import math

import torch

own = False

GROUP = 64  # channels that share a step and a middle
BLOCK = 64  # tokens of a cache block
LIMIT = 32768.0  # largest magnitude the cache holds
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _ints(text):
    return [int(t) for t in str(text).split(",")]


# --------------------------------------------------------------------------- cases


def listed():
    return [
        # a handful of chat turns, one of them a single token: what the launch costs
        {"name": "prompt_short", "op": "prompt", "lens": "1,37,130,64", "H": 16, "Hkv": 4, "d": 64, "dtype": "fp16",
         "causal": True},
        # a batch of prompts as a server packs them: many short ones, a few long ones
        {"name": "prompt_mixed", "op": "prompt",
         "lens": "4096,17,950,2310,128,1,3001,640,77,1536,255,409,2047,1201,33,700", "H": 32, "Hkv": 8, "d": 128,
         "dtype": "bf16", "causal": True},
        # two long documents
        {"name": "prompt_long", "op": "prompt", "lens": "16384,5001", "H": 32, "Hkv": 8, "d": 128, "dtype": "bf16",
         "causal": True},
        # one generated token of each sequence goes into the cache
        {"name": "store_token", "op": "store", "rows": "1,1,1,1,1,1,1,1", "before": "0,63,64,1000,4095,4096,777,32000",
         "Hkv": 8, "d": 128, "dtype": "bf16"},
        # the keys and values of the packed prompts go into the cache
        {"name": "store_prompt", "op": "store", "rows": "4096,17,8192,2310,0,1,3001,16384",
         "before": "0,0,100,0,50,0,63,0", "Hkv": 8, "d": 128, "dtype": "bf16"},
        # one short conversation: latency
        {"name": "decode_short", "op": "decode", "lens": "500", "C": 512, "H": 16, "Hkv": 4, "Nq": 1, "d": 64,
         "dtype": "fp16", "causal": False, "weights": False},
        # a batch of conversations of very different lengths
        {"name": "decode_ragged", "op": "decode", "lens": "32768,1,20001,777,4096,12345,63,30000", "C": 32768, "H": 32,
         "Hkv": 8, "Nq": 1, "d": 128, "dtype": "bf16", "causal": False, "weights": False},
        # the same with the weight of every cached token added up, for a later eviction
        {"name": "decode_weights", "op": "decode", "lens": "9000,8500,10001,9216,8192,9999,8777,9100", "C": 10240,
         "H": 32, "Hkv": 8, "Nq": 1, "d": 128, "dtype": "fp16", "causal": False, "weights": True},
        # four guessed tokens checked at once, two query heads to a key/value head
        {"name": "decode_rows", "op": "decode", "lens": "10007,5000,3,16000", "C": 16384, "H": 16, "Hkv": 8, "Nq": 4,
         "d": 256, "dtype": "bf16", "causal": True, "weights": False},
        # a full server: the long cache of the decode benchmark in four times its batch
        {"name": "decode_large", "op": "decode", "lens": ",".join(["32768"] * 32), "C": 32768, "H": 32, "Hkv": 8,
         "Nq": 1, "d": 128, "dtype": "bf16", "causal": False, "weights": False},
        # one sequence a little over its budget
        {"name": "evict_step", "op": "evict", "lens": "1100", "C": 1152, "keep": 1024, "recent": 128, "Hkv": 8,
         "d": 128},
        # long prompts cut to a quarter
        {"name": "evict_prompt", "op": "evict", "lens": "32768,30000,8000,32001,20000,32768,16384,28111", "C": 32768,
         "keep": 8192, "recent": 256, "Hkv": 8, "d": 128},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _join(ns):
    return ",".join(str(n) for n in ns)


def draw(rng):
    op = rng.choice(["prompt", "store", "decode", "decode", "evict"])
    d = rng.choice([64, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    dtype = rng.choice(["bf16", "fp16"])
    top = {c["name"]: work(c) for c in listed()}
    while True:
        if op == "prompt":
            lens = [_log(rng, 1, 16384) for _ in range(rng.randint(1, 16))]
            case = {"op": op, "lens": _join(lens), "H": Hkv * rng.choice([1, 2, 4]), "Hkv": Hkv, "d": d, "dtype": dtype,
                    "causal": rng.random() < 0.8}
            most = top["prompt_long"]
            fits = sum(lens) <= 40000
        elif op == "store":
            n = rng.randint(1, 16)
            rows = [rng.choice([0, 1, 1, _log(rng, 1, 16384)]) for _ in range(n)]
            rows[rng.randrange(n)] = _log(rng, 1, 16384)
            case = {"op": op, "rows": _join(rows), "before": _join(rng.choice([0, _log(rng, 1, 8192)]) for _ in rows),
                    "Hkv": Hkv, "d": d, "dtype": rng.choice(["bf16", "fp16", "fp32"])}
            most = top["store_prompt"]
            fits = True
        elif op == "decode":
            lens = [_log(rng, 1, 65536) for _ in range(_log(rng, 1, 32))]
            case = {"op": op, "lens": _join(lens), "C": (max(lens) + rng.choice([0, 1, 100, 1000]) + 63) // 64 * 64,
                    "H": Hkv * rng.choice([1, 2, 3, 4, 7, 8]), "Hkv": Hkv, "Nq": rng.choice([1, 1, 1, 2, 4, 7]), "d": d,
                    "dtype": dtype, "causal": rng.random() < 0.5, "weights": rng.random() < 0.4}
            most = top["decode_large"]
            fits = len(lens) * case["C"] * Hkv * d <= 32 * 32768 * 8 * 128
        else:
            lens = [_log(rng, 1, 65536) for _ in range(_log(rng, 1, 16))]
            keep = _log(rng, 1, 16384)
            case = {"op": op, "lens": _join(lens), "C": (max(lens) + 63) // 64 * 64, "keep": keep,
                    "recent": rng.choice([0, rng.randint(0, keep), min(keep, 64)]), "Hkv": Hkv, "d": d}
            most = top["evict_prompt"]
            fits = len(lens) * case["C"] * Hkv * d <= 8 * 32768 * 8 * 128
        w = work(case)
        if fits and w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"]:
            return case


def work(case):
    op, d, Hkv = case["op"], case["d"], case["Hkv"]
    token = 2 * (d // 2 + d // GROUP * 4)  # bytes of a cached token of one key/value head
    if op == "prompt":
        lens, H = _ints(case["lens"]), case["H"]
        T = sum(lens)
        pairs = sum(n * (n + 1) // 2 if case["causal"] else n * n for n in lens)
        return {"bytes": (2 * H + 2 * Hkv) * T * d * 2 + 4 * H * T, "flops": 4 * d * H * pairs}
    if op == "store":
        T, e = sum(_ints(case["rows"])), 4 if case["dtype"] == "fp32" else 2
        return {"bytes": T * Hkv * (2 * 2 * d * e + token), "flops": T * Hkv * 2 * d * 8}
    lens = _ints(case["lens"])
    if op == "decode":
        rows = case["H"] * case["Nq"] * len(lens)
        slots = sum(lens) * Hkv
        return {"bytes": slots * (token + (8 if case["weights"] else 0)) + rows * (2 * d * 2 + 4),
                "flops": 4 * d * case["H"] * case["Nq"] * sum(lens)}
    kept = sum(min(n, case["keep"]) for n in lens) * Hkv
    return {"bytes": 4 * Hkv * sum(lens) + kept * (2 * token + 4 + 4), "flops": Hkv * sum(lens)}


# --------------------------------------------------------------------------- inputs


def _cu(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def _kv_rows(shape, g):
    """Keys (some channels far off zero, as rotary keys have them) and values."""
    k = torch.randn(shape, generator=g, device="cuda")
    k += 3.0 * (torch.randn(shape[-1], generator=g, device="cuda") ** 3).clamp(-2, 2)
    return k, torch.randn(shape, generator=g, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, d, Hkv = case["op"], case["d"], case["Hkv"]
    randn = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    st = dict(case)
    if op == "prompt":
        lens, dt = _ints(case["lens"]), DTYPES[case["dtype"]]
        T, H = sum(lens), case["H"]
        # the projection's output: query, key and value heads of a token side by side
        qkv = randn(T, H + 2 * Hkv, d).to(dt)
        st.update(lens=lens, cu=_cu(lens), q=qkv[:, :H], k=qkv[:, H:H + Hkv], v=qkv[:, H + Hkv:], scale=d ** -0.5)
    elif op == "store":
        rows, before, dt = _ints(case["rows"]), _ints(case["before"]), DTYPES[case["dtype"]]
        k, v = _kv_rows((sum(rows), Hkv, d), g)
        after = [a + b for a, b in zip(rows, before)]
        st.update(k=k.to(dt), v=v.to(dt), cu=_cu(rows), lens=torch.tensor(after, dtype=torch.int32, device="cuda"),
                  cache=torch.zeros(len(rows), Hkv, (max(after) + BLOCK - 1) // BLOCK, 72 * d, dtype=torch.uint8,
                                    device="cuda"))
    else:
        lens, C = _ints(case["lens"]), case["C"]
        B = len(lens)
        cache = torch.empty(B, Hkv, C // BLOCK, 72 * d, dtype=torch.uint8, device="cuda")
        for b in range(B):
            cache[b] = _packed(*_kv_rows((Hkv, C, d), g))
        st.update(cache=cache, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
        if op == "decode":
            st.update(q=randn(B, case["H"], case["Nq"], d).to(DTYPES[case["dtype"]]), scale=d ** -0.5)
            if case["weights"]:
                st.update(w_in=randn(B, Hkv, C).abs(), w_out=torch.zeros(B, Hkv, C, device="cuda"))
        else:
            keep = case["keep"]
            # what many decode steps have added up: a few heavy tokens, many light ones, some never looked at
            w = torch.exp(2.0 * randn(B, Hkv, C)) * (randn(B, Hkv, C) > -1.5)
            st.update(w=w, cache2=torch.zeros(B, Hkv, (keep + BLOCK - 1) // BLOCK, 72 * d, dtype=torch.uint8,
                                              device="cuda"),
                      w2=torch.zeros(B, Hkv, (keep + BLOCK - 1) // BLOCK * BLOCK, device="cuda"),
                      lens2=torch.zeros(B, dtype=torch.int32, device="cuda"),
                      kept=torch.zeros(B, Hkv, keep, dtype=torch.int32, device="cuda"))
    return st


# --------------------------------------------------------------------------- plain forms


def _quantised(x):
    """x [..., d] -> codes (0..15) [..., d], step and middle [..., d / 64], in 32 bits."""
    x = x.float().unflatten(-1, (-1, GROUP))
    lo, hi = x.amin(-1), x.amax(-1)
    bad = ~((lo >= -LIMIT) & (hi <= LIMIT))
    t = (hi - lo) / torch.full_like(lo, 15.0)  # (a number would be multiplied with as its rounded reciprocal)
    near = t.half()
    step = torch.where(near.float() < t, (near.view(torch.int16) + 1).view(torch.float16), near)  # rounded up
    middle = (lo + 8 * step.float()).half()
    step, middle = step.masked_fill(bad, math.nan), middle.masked_fill(bad, math.nan)
    s, m = step.float()[..., None], middle.float()[..., None]
    code = torch.round((x - m) / s).clamp(-8, 7).nan_to_num(0.0) + 8
    return code.masked_fill(s == 0, 8.0).flatten(-2), step, middle


def _packed_half(x):
    """x [..., C, d] -> code bytes [..., C / 64, 32 d] and parameter bytes [..., C / 64, 4 d]."""
    code, step, middle = _quantised(x)
    code = code.to(torch.uint8)
    by = code[..., 0::2] | (code[..., 1::2] << 4)
    par = torch.stack((step, middle), -1).view(torch.uint8)
    return (by.unflatten(-2, (-1, BLOCK)).flatten(-2), par.flatten(-3).unflatten(-1, (-1, 4 * by.shape[-1] * 2)))


def _packed(k, v):
    """k, v [..., C, d] (C a multiple of 64) -> cache blocks [..., C / 64, 72 d]."""
    (kc, kp), (vc, vp) = _packed_half(k), _packed_half(v)
    return torch.cat((kc, vc, kp, vp), -1)


def _fields(cache):
    """Views of a cache [B, Hkv, blocks, 72 d]: K codes, V codes, K and V parameters by token."""
    d = cache.shape[-1] // 72
    parts = cache.split((32 * d, 32 * d, 4 * d, 4 * d), -1)
    return [p.unflatten(-1, (BLOCK, -1)) for p in parts]


def _values(codes, par):
    """[..., blocks, 64, d / 2] code bytes and parameter bytes -> values [..., blocks * 64, d] in 32 bits."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float().unflatten(-1, (-1, GROUP))
    p = par.contiguous().view(torch.float16).float().unflatten(-1, (-1, 2))
    return (p[..., 1:] + p[..., :1] * (c - 8)).flatten(-2).flatten(-3, -2)


def _plain_prompt(st):
    q, k, v = st["q"], st["k"], st["v"]
    T, H, d = q.shape
    Hkv = k.shape[1]
    g = H // Hkv
    o = torch.empty(T, H, d, dtype=q.dtype, device=q.device)
    lse = torch.empty(H, T, device=q.device)
    at = 0
    for n in st["lens"]:
        heads = max(1, min(Hkv, (1 << 30) // (g * n * n)))  # key/value heads at a time: 4 GB of scores
        qs = q[at:at + n].float().unflatten(1, (Hkv, g)).permute(1, 2, 0, 3)
        ks, vs = k[at:at + n].float().permute(1, 2, 0)[:, None], v[at:at + n].float().transpose(0, 1)[:, None]
        for h in range(0, Hkv, heads):
            s = torch.matmul(qs[h:h + heads], ks[h:h + heads]).mul_(st["scale"])
            if st["causal"]:
                s.masked_fill_(torch.ones(n, n, dtype=torch.bool, device=q.device).triu_(1), -math.inf)
            top = s.amax(-1, keepdim=True)
            p = s.sub_(top).exp_()
            total = p.sum(-1, keepdim=True)
            out = torch.matmul(p, vs[h:h + heads]) / total
            o[at:at + n, h * g:(h + heads) * g] = out.flatten(0, 1).transpose(0, 1).to(q.dtype)
            lse[h * g:(h + heads) * g, at:at + n] = (top + total.log()).squeeze(-1).flatten(0, 1)
        at += n
    return o, lse


def _slots(st):
    """Sequence and slot of each packed row."""
    cu, lens = st["cu"].long(), st["lens"].long()
    row = torch.arange(st["k"].shape[0], device=cu.device)
    b = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    return b, lens[b] - cu[b + 1] + row


def _plain_store(st):
    b, slot = _slots(st)
    out = []
    for x, c, p in ((st["k"], 0, 2), (st["v"], 1, 3)):
        code, step, middle = _quantised(x)
        code = code.to(torch.uint8)
        fields = _fields(st["cache"])
        fields[c][b, :, slot // BLOCK, slot % BLOCK] = code[..., 0::2] | (code[..., 1::2] << 4)
        par = torch.stack((step, middle), -1).flatten(-2).view(torch.uint8)
        fields[p][b, :, slot // BLOCK, slot % BLOCK] = par
        # read back
        got = fields[c][b, :, slot // BLOCK, slot % BLOCK], fields[p][b, :, slot // BLOCK, slot % BLOCK]
        out.append(_values(got[0][:, :, None, None], got[1][:, :, None, None]).squeeze(-2).to(x.dtype))
    return out


def _plain_decode(st):
    q, lens = st["q"].float(), st["lens"].long()
    B, H, Nq, d = q.shape
    Hkv, C = st["cache"].shape[1], st["cache"].shape[2] * BLOCK
    kc, vc, kp, vp = _fields(st["cache"])
    slot = torch.arange(C, device=q.device)
    last = lens[:, None] - 1  # the newest slot that a row may look at
    if st["causal"]:
        last = lens[:, None] - Nq + torch.arange(Nq, device=q.device)
    last = last.expand(B, Nq)
    dark = (slot > last[..., None])[:, None, None]  # [B, 1, 1, Nq, C]
    s = torch.matmul(q.view(B, Hkv, -1, d), _values(kc, kp).transpose(-1, -2)).view(B, Hkv, -1, Nq, C) * st["scale"]
    s = s.masked_fill(dark, -math.inf)
    top = s.amax(-1, keepdim=True).clamp_min(-3e38)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    v = _values(vc, vp).masked_fill((slot >= lens[:, None])[:, None, :, None], 0.0)
    p = p / total.clamp_min(1e-38)
    o = torch.matmul(p.flatten(2, 3), v).view(B, H, Nq, d).to(st["q"].dtype)
    lse = torch.where(total > 0, top + total.log(), -math.inf).view(B, H, Nq)
    if not st["weights"]:
        return o, lse
    w = st["w_in"] + p.sum((2, 3))
    st["w_out"].copy_(torch.where((slot < lens[:, None])[:, None], w, st["w_out"]))
    return o, lse, st["w_out"]


def _plain_evict(st):
    w, lens, keep, recent = st["w"], st["lens"].long(), st["keep"], st["recent"]
    B, Hkv, C = w.shape
    n = lens.clamp_max(keep)
    slot = torch.arange(C, device=w.device)
    kind = torch.where(slot < (lens[:, None] - recent), 1, 0) + 2 * (slot >= lens[:, None])  # 0 newest, 1 others
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices
    by_kind = torch.sort(kind[:, None].expand(B, Hkv, C).gather(-1, order), dim=-1, stable=True).indices
    order = order.gather(-1, by_kind)[..., :keep]
    rank = torch.arange(order.shape[-1], device=w.device)
    order = order.masked_fill((rank >= n[:, None])[:, None], C).sort(-1).values
    there = order < C
    b, h, to = torch.nonzero(there, as_tuple=True)
    src = order[b, h, to]
    st["kept"].fill_(-1)[b, h, to] = src.int()
    st["w2"][b, h, to] = w[b, h, src]
    for x, y in zip(_fields(st["cache"]), _fields(st["cache2"])):
        y[b, h, to // BLOCK, to % BLOCK] = x[b, h, src // BLOCK, src % BLOCK]
    st["lens2"].copy_(n)
    return st["cache2"], st["w2"], st["lens2"], st["kept"]


# --------------------------------------------------------------------------- one pass


def run(state):
    op = state["op"]
    if own:
        return _own(state)
    if op == "prompt":
        return _plain_prompt(state)
    if op == "store":
        return _plain_store(state)
    return _plain_decode(state) if op == "decode" else _plain_evict(state)


def _own(st):
    from exact_tiled_attention_07_gb300 import binding as fa

    op = st["op"]
    if op == "prompt":
        return fa.attention_forward_varlen(st["q"], st["k"], st["v"], st["cu"], causal=st["causal"], scale=st["scale"])
    if op == "store":
        fa.fa_kv4_append(st["k"], st["v"], st["cu"], st["lens"], st["cache"])
        return fa.kv4_read(st["cache"], st["cu"], st["lens"], st["k"].shape[0], dtype=st["k"].dtype)
    if op == "decode":
        if not st["weights"]:
            return fa.attention_decode_kv4(st["q"], st["cache"], st["lens"], causal=st["causal"], scale=st["scale"])
        o, lse = fa.attention_decode_kv4(st["q"], st["cache"], st["lens"], causal=st["causal"], scale=st["scale"],
                                         weights_in=st["w_in"], weights_out=st["w_out"])
        return o, lse, st["w_out"]
    fa.fa_kv4_evict(st["cache"], st["w"], st["lens"], st["keep"], st["recent"], st["cache2"], st["w2"], st["lens2"],
                    st["kept"])
    return st["cache2"], st["w2"], st["lens2"], st["kept"]


# --------------------------------------------------------------------------- the definitions in 64 bits


def exact(case, seed):
    w = work(case)
    if w["flops"] > 3e12:
        return None
    st = prepare(case, seed)
    op, d, Hkv = case["op"], case["d"], case["Hkv"]
    if op == "prompt":
        T, H, at = st["q"].shape[0], case["H"], 0
        o = torch.empty(T, H, d, dtype=torch.float64, device="cuda")
        lse = torch.empty(H, T, dtype=torch.float64, device="cuda")
        for n in st["lens"]:
            for h in range(H):
                q, k, v = (st[x][at:at + n, i].double() for x, i in (("q", h), ("k", h * Hkv // H), ("v", h * Hkv // H)))
                s = q @ k.T * st["scale"]
                if case["causal"]:
                    i = torch.arange(n, device="cuda")
                    s[i[:, None] < i] = -math.inf
                lse[h, at:at + n] = torch.logsumexp(s, -1)
                o[at:at + n, h] = torch.softmax(s, -1) @ v
            at += n
        return o, lse
    if op == "store":
        return [_exact_values(st[x]) for x in ("k", "v")]
    if op == "decode":
        B, H, Nq = len(_ints(case["lens"])), case["H"], case["Nq"]
        o = torch.zeros(B, H, Nq, d, dtype=torch.float64, device="cuda")
        lse = torch.full((B, H, Nq), -math.inf, dtype=torch.float64, device="cuda")
        add = torch.zeros(B, Hkv, case["C"], dtype=torch.float64, device="cuda")
        for b, n in enumerate(_ints(case["lens"])):
            for hk in range(Hkv):
                k, v = _exact_rows(st["cache"][b, hk], n)
                g = H // Hkv
                for i in range(Nq):
                    m = n - Nq + i + 1 if case["causal"] else n
                    if m <= 0:
                        continue
                    s = st["q"][b, hk * g:(hk + 1) * g, i].double() @ k[:m].T * st["scale"]
                    p = torch.softmax(s, -1)
                    o[b, hk * g:(hk + 1) * g, i] = p @ v[:m]
                    lse[b, hk * g:(hk + 1) * g, i] = torch.logsumexp(s, -1)
                    add[b, hk, :m] += p.sum(0)
        if not case["weights"]:
            return o, lse
        for b, n in enumerate(_ints(case["lens"])):
            add[b, :, :n] += st["w_in"][b, :, :n].double()
        return o, lse, add
    # eviction moves what is there: whole values and copies
    w = st["w"].cpu()
    keep, recent = case["keep"], case["recent"]
    for b, n in enumerate(_ints(case["lens"])):
        m = min(n, keep)
        for h in range(Hkv):
            newest = list(range(max(0, n - recent), n))
            others = torch.sort(w[b, h, :n - len(newest)].double(), descending=True, stable=True).indices
            src = torch.tensor(sorted(newest[len(newest) - min(m, len(newest)):] + others[:max(0, m - len(newest))].tolist()),
                               dtype=torch.int64, device="cuda")
            st["kept"][b, h] = -1
            st["kept"][b, h, :m] = src.int()
            st["w2"][b, h, :m] = st["w"][b, h, src]
            to = torch.arange(m, device="cuda")
            for lo, size in ((0, d // 2), (32 * d, d // 2), (64 * d, d // 16), (68 * d, d // 16)):
                x = st["cache"][b, h, :, lo:lo + 64 * size].reshape(-1, size)
                at = (to // BLOCK)[:, None], lo + (to % BLOCK)[:, None] * size + torch.arange(size, device="cuda")
                st["cache2"][b, h][at] = x[src]
        st["lens2"][b] = m
    return st["cache2"], st["w2"].double(), st["lens2"], st["kept"]


def _exact_values(x):
    """What the cache holds of x: the format's own roundings (steps to fp16 upwards, middles to fp16, quotients to 32 bits) taken
    on 64-bit results."""
    x = x.double().reshape(*x.shape[:-1], -1, GROUP)
    lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
    f32 = lambda t: t.float().double()  # noqa: E731
    t = f32(f32(hi - lo) / 15)
    step = t.half()
    step = torch.where(step.double() < t, torch.nextafter(step.cpu(), torch.tensor(math.inf, dtype=torch.float16)).to(t.device),
                       step).double()
    middle = f32(lo + 8 * step).half().double()
    code = torch.round(f32(f32(x - middle) / step.clamp_min(1e-30))).clamp(-8, 7)
    return (middle + step * code).reshape(*x.shape[:-2], -1)


def _exact_rows(blocks, n):
    """The first n keys and values of one cache head [blocks, 72 d], in 64 bits."""
    d = blocks.shape[-1] // 72
    got = []
    for code_at, par_at in ((0, 64 * d), (32 * d, 68 * d)):
        by = blocks[:, code_at:code_at + 32 * d].reshape(-1, d // 2)[:n].int()
        code = torch.empty(n, d, dtype=torch.float64, device=blocks.device)
        code[:, 0::2], code[:, 1::2] = (by % 16).double(), (by // 16).double()
        par = blocks[:, par_at:par_at + 4 * d].reshape(-1, d // 16)[:n].contiguous().view(torch.float16).double()
        step, middle = par[:, 0::2].repeat_interleave(GROUP, -1), par[:, 1::2].repeat_interleave(GROUP, -1)
        got.append(middle + step * (code - 8))
    return got
