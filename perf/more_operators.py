"""The attention block's operators around and beside plain causal attention, in plain torch and through the library.

* ``norm``:   queries and keys normed head by head (root mean square, learned weight) and rotated by their position, from
  the fused projection's output to what attention takes; with ``train`` the gradients of both inputs and weights too;
* ``window``: attention with a sliding window and a few first tokens (sinks) that stay visible: query i sees key j when
  j <= i and (i - j < window or j < sinks).  ``train``: forward and gradients of a padded batch; ``prompt``: packed
  prompts of different lengths; ``decode``: new rows over a key/value cache;
* ``prefix``: new rows of many sequences that begin with the same tokens: keys and values of the shared prefix are held
  once, those behind it in a cache of each sequence's own.

A rotation table [positions, rotary] holds cos of the rotary / 2 angles of a position, then their sin.  Rotated pairs are
channels (i, i + rotary / 2), or (2i, 2i + 1) where ``interleaved``; channels from ``rotary`` on are not rotated.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6


def _ints(text):
    return [int(t) for t in str(text).split(",")]


# --------------------------------------------------------------------------- cases


def listed():
    return [
        # one generated token of each of 32 conversations, far into their texts: what the launch costs
        {"name": "norm_token", "op": "norm", "kind": "packed", "B": 1, "N": 32, "H": 32, "Hkv": 8, "d": 128,
         "rotary": 128, "interleaved": False, "dtype": "bf16", "wdtype": "bf16", "table": 32768},
        # the packed prompts of a server
        {"name": "norm_prompt", "op": "norm", "kind": "packed", "B": 1, "N": 34001, "H": 32, "Hkv": 8, "d": 128,
         "rotary": 128, "interleaved": False, "dtype": "bf16", "wdtype": "bf16", "table": 16384},
        # a small training step whose heads rotate half of their channels, in adjacent pairs
        {"name": "norm_train_short", "op": "norm", "kind": "train", "B": 3, "N": 1001, "H": 12, "Hkv": 4, "d": 64,
         "rotary": 32, "interleaved": True, "dtype": "fp16", "wdtype": "fp32", "table": 1024},
        # the causal language model's training step
        {"name": "norm_train", "op": "norm", "kind": "train", "B": 8, "N": 4096, "H": 16, "Hkv": 16, "d": 128,
         "rotary": 128, "interleaved": False, "dtype": "bf16", "wdtype": "fp32", "table": 4096},
        # a small model's training step, ragged length, sinks that end inside a tile
        {"name": "window_train_short", "op": "window", "kind": "train", "B": 2, "N": 1000, "H": 16, "Hkv": 16, "d": 64,
         "window": 256, "sinks": 5, "dtype": "fp16"},
        # the causal language model's training step with a window of a quarter of its length
        {"name": "window_train", "op": "window", "kind": "train", "B": 8, "N": 4096, "H": 16, "Hkv": 16, "d": 128,
         "window": 1024, "sinks": 4, "dtype": "bf16"},
        # a batch of prompts as a server packs them
        {"name": "window_prompt", "op": "window", "kind": "prompt", "lens": "16384,17,950,2310,8001,1,3001,640", "H": 32,
         "Hkv": 8, "d": 128, "window": 2048, "sinks": 16, "dtype": "bf16"},
        # two conversations, one shorter than its window: latency
        {"name": "window_decode_short", "op": "window", "kind": "decode", "lens": "700,90", "C": 768, "H": 16, "Hkv": 4,
         "Nq": 1, "d": 64, "window": 128, "sinks": 4, "dtype": "fp16"},
        # a full server with long caches, of which a window is looked at
        {"name": "window_decode", "op": "window", "kind": "decode",
         "lens": "32768,32001,20001,777,4096,12345,30000,32768,31999,5000,16384,28111,9000,8192,27001,32000", "C": 32768,
         "H": 32, "Hkv": 8, "Nq": 1, "d": 128, "window": 4096, "sinks": 4, "dtype": "bf16"},
        # a few requests behind one system prompt
        {"name": "prefix_short", "op": "prefix", "P": 1000, "lens": "30,1,200,77", "C": 256, "H": 16, "Hkv": 4, "Nq": 1,
         "d": 64, "dtype": "fp16"},
        # guessed tokens of requests about one document, checked at once
        {"name": "prefix_rows", "op": "prefix", "P": 20001, "lens": "130,4,999,2047,64,700,1,350,8,1200,90,512", "C": 2048,
         "H": 16, "Hkv": 8, "Nq": 4, "d": 128, "dtype": "fp16"},
        # a full server whose requests share a long prefix
        {"name": "prefix_large", "op": "prefix", "P": 32768, "lens": ",".join(str(100 + 61 * i) for i in range(64)),
         "C": 4096, "H": 32, "Hkv": 8, "Nq": 1, "d": 128, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _join(ns):
    return ",".join(str(n) for n in ns)


def draw(rng):
    top = {c["name"]: work(c) for c in listed()}
    op, kind, most = rng.choice([
        ("norm", "packed", "norm_prompt"), ("norm", "train", "norm_train"), ("window", "train", "window_train"),
        ("window", "prompt", "window_prompt"), ("window", "decode", "window_decode"), ("prefix", None, "prefix_large")])
    while True:
        Hkv, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256])
        H = Hkv * rng.choice([1, 2, 3, 4, 7, 8])
        case = {"op": op, "kind": kind, "H": H, "Hkv": Hkv, "d": d, "dtype": rng.choice(["bf16", "fp16"])}
        fits = True
        if op == "norm":
            case["d"] = d = rng.choice([64, 64, 80, 96, 128, 128, 256])
            B = 1 if kind == "packed" else _log(rng, 1, 16)
            case.update(B=B, N=_log(rng, 1, 65536 // B), rotary=rng.choice([d, d, d // 2 // 8 * 8, 16]),
                        interleaved=rng.random() < 0.4, dtype=rng.choice(["bf16", "fp16", "fp32"]), table=0)
            case.update(wdtype=rng.choice(["fp32", case["dtype"]]), table=max(case["N"], _log(rng, 16, 131072)))
        elif kind == "train":
            case.update(B=_log(rng, 1, 8), N=_log(rng, 1, 16384), window=_log(rng, 1, 8192),
                        sinks=rng.choice([0, 1, 4, _log(rng, 1, 300)]))
            fits = case["B"] * H * case["N"] <= 8 * 16 * 4096
        elif kind == "prompt":
            lens = [_log(rng, 1, 16384) for _ in range(rng.randint(1, 16))]
            case.update(lens=_join(lens), window=_log(rng, 1, 8192), sinks=rng.choice([0, 1, 4, _log(rng, 1, 300)]))
            fits = sum(lens) <= 40000
        elif kind == "decode":
            lens = [_log(rng, 1, 65536) for _ in range(_log(rng, 1, 32))]
            case.update(lens=_join(lens), C=max(lens) + rng.choice([0, 1, 100, 1000]), Nq=rng.choice([1, 1, 1, 2, 4, 7]),
                        window=_log(rng, 1, 32768), sinks=rng.choice([0, 1, 4, _log(rng, 1, 300)]))
            fits = len(lens) * case["C"] * Hkv * d <= 16 * 32768 * 8 * 128
        else:
            lens = [rng.choice([0, _log(rng, 1, 8192)]) for _ in range(_log(rng, 1, 96))]
            case.update(P=_log(rng, 1, 65536), lens=_join(lens), C=max(1, max(lens) + rng.choice([0, 1, 100])),
                        Nq=rng.choice([1, 1, 1, 2, 4, 7]))
            fits = len(lens) * case["C"] * Hkv * d <= 64 * 4096 * 8 * 128
        w = work(case)
        if fits and w["bytes"] <= top[most]["bytes"] and w["flops"] <= top[most]["flops"]:
            return case


def _seen(n, window, sinks):
    """Visible (query, key) pairs of one sequence of n tokens."""
    w = min(n, window)
    pairs = w * (w + 1) // 2 + (n - w) * w
    s = min(sinks, max(0, n - window))  # sink j is outside the window of the n - window - j last queries
    return pairs + s * (n - window) - s * (s - 1) // 2


def _seen_slots(n, window, sinks):
    return min(n, window) + min(sinks, max(0, n - window))


def work(case):
    d, H, Hkv = case["d"], case["H"], case["Hkv"]
    e = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "norm":
        T = case["B"] * case["N"]
        one = T * (H + Hkv) * d
        rows = T if case["kind"] == "packed" else case["N"]
        passes = 2 if case["kind"] == "train" else 1
        return {"bytes": passes * 2 * one * e + rows * case["rotary"] * 4, "flops": one * (8 if passes == 1 else 22)}
    if case["op"] == "window" and case["kind"] == "train":
        B, N = case["B"], case["N"]
        return {"bytes": B * N * d * e * (4 * H + 4 * Hkv) + 4 * B * H * N,
                "flops": 14 * d * B * H * _seen(N, case["window"], case["sinks"])}
    lens = _ints(case["lens"])
    if case["op"] == "window" and case["kind"] == "prompt":
        T = sum(lens)
        return {"bytes": (2 * H + 2 * Hkv) * T * d * e + 4 * H * T,
                "flops": 4 * d * H * sum(_seen(n, case["window"], case["sinks"]) for n in lens)}
    B, Nq = len(lens), case["Nq"]
    rows = H * Nq * B
    if case["op"] == "window":
        slots = sum(_seen_slots(n, case["window"], case["sinks"]) for n in lens)
        shared = 0
    else:
        slots, shared = sum(lens), case["P"]
    return {"bytes": (slots + shared) * Hkv * 2 * d * e + rows * (2 * d * e + 4),
            "flops": 4 * d * H * Nq * (slots + B * shared)}


# --------------------------------------------------------------------------- inputs


def _cu(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def _rotation_table(n, rotary):
    """What a user's program computes once: cos, then sin of each position's angles, in 64 bits before they are rounded."""
    freq = 10000.0 ** (-torch.arange(0, rotary, 2, dtype=torch.float64, device="cuda") / max(rotary, 1))
    angle = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat((angle.cos(), angle.sin()), -1).float()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    d, H, Hkv, dt = case["d"], case["H"], case["Hkv"], DTYPES[case["dtype"]]
    st = dict(case)
    if case["op"] == "norm":
        B, N = case["B"], case["N"]
        # the projection's output: query, key and value heads of a token side by side
        qkv = (randn(B, N, H + 2 * Hkv, d) * (1.0 + randn(H + 2 * Hkv, d).abs())).to(dt)
        if case["kind"] == "packed":
            qkv = qkv[0]
            st["pos"] = torch.randint(0, case["table"], (N,), generator=g, device="cuda", dtype=torch.int32)
        else:
            st["pos"] = None  # 0 .. N - 1
            st.update(dq=randn(B, H, N, d).to(dt), dk=randn(B, Hkv, N, d).to(dt))
        wdt = DTYPES[case["wdtype"]]
        st.update(q=qkv[..., :H, :], k=qkv[..., H:H + Hkv, :], wq=(1.0 + 0.3 * randn(d)).to(wdt),
                  wk=(1.0 + 0.3 * randn(d)).to(wdt), table=_rotation_table(case["table"], case["rotary"]))
        return st
    st["scale"] = d ** -0.5
    if case["op"] == "window" and case["kind"] == "train":
        B, N = case["B"], case["N"]
        st.update(q=randn(B, H, N, d).to(dt), k=randn(B, Hkv, N, d).to(dt), v=randn(B, Hkv, N, d).to(dt),
                  do=randn(B, H, N, d).to(dt))
        return st
    lens = _ints(case["lens"])
    B = len(lens)
    if case["op"] == "window" and case["kind"] == "prompt":
        qkv = randn(sum(lens), H + 2 * Hkv, d).to(dt)
        st.update(lens=lens, cu=_cu(lens), q=qkv[:, :H], k=qkv[:, H:H + Hkv], v=qkv[:, H + Hkv:])
        return st
    C = case["C"]
    k, v = (torch.empty(B, Hkv, C, d, dtype=dt, device="cuda") for _ in range(2))
    for b in range(B):
        k[b], v[b] = randn(Hkv, C, d), randn(Hkv, C, d)
    st.update(k=k, v=v, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), q=randn(B, H, case["Nq"], d).to(dt))
    if case["op"] == "prefix":
        st.update(kp=randn(Hkv, case["P"], d).to(dt), vp=randn(Hkv, case["P"], d).to(dt))
    return st


# --------------------------------------------------------------------------- plain forms


def _turned(y, c, s, rotary, interleaved):
    """y [..., d] rotated by cos, sin [..., rotary / 2]; with -s the inverse, which is also the transpose."""
    a, b = (y[..., 0:rotary:2], y[..., 1:rotary:2]) if interleaved else (y[..., :rotary // 2], y[..., rotary // 2:rotary])
    ra, rb = a * c - b * s, b * c + a * s
    turned = torch.stack((ra, rb), -1).flatten(-2) if interleaved else torch.cat((ra, rb), -1)
    return torch.cat((turned, y[..., rotary:]), -1)


def _plain_norm(st):
    rotary, half = st["rotary"], st["rotary"] // 2
    pos = st["pos"].long() if st["pos"] is not None else torch.arange(st["N"], device="cuda")
    c, s = st["table"][pos][:, None, :half], st["table"][pos][:, None, half:]  # [N, 1, half]
    out, grads, wgrads = [], [], []
    for x, w, dy in ((st["q"], st["wq"], st.get("dq")), (st["k"], st["wk"], st.get("dk"))):
        dt, xf, wf = x.dtype, x.float(), w.float()
        r = torch.rsqrt(xf.square().mean(-1, keepdim=True) + EPS)
        y = _turned(xf * r * wf, c, s, rotary, st["interleaved"])
        out.append(y.to(dt) if dy is None else y.transpose(1, 2).to(dt).contiguous())
        if dy is not None:
            u = _turned(dy.float().transpose(1, 2), c, -s, rotary, st["interleaved"])
            xh = xf * r
            g = u * wf
            grads.append((r * (g - xh * (g * xh).mean(-1, keepdim=True))).to(dt))
            wgrads.append((u * xh).flatten(0, -2).sum(0).to(w.dtype))
    return out + grads + wgrads


def _band(i0, i1, window, sinks):
    """The keys that queries i0 .. i1 - 1 of a sequence may see: [0, first) and [lo, i1)."""
    lo = max(0, i0 - window + 1)
    return min(sinks, lo), lo


def _band_scores(q, k, i0, i1, window, sinks, scale):
    """Scores of queries i0 .. i1 - 1 (q [..., Hkv, g, rows, d]) and their keys (k [..., Hkv, N, d]): with the keys' numbers."""
    first, lo = _band(i0, i1, window, sinks)
    j = torch.cat((torch.arange(first, device=q.device), torch.arange(lo, i1, device=q.device)))
    i = torch.arange(i0, i1, device=q.device)[:, None]
    dark = (j > i) | ((i - j >= window) & (j >= sinks))
    s = torch.matmul(q, k[..., j, :].unsqueeze(-3).transpose(-1, -2)).mul_(scale).masked_fill_(dark, -math.inf)
    return s, j


def _rows_at_once(heads, window, sinks):
    rows = 4096
    while rows > 64 and heads * rows * (rows + window + sinks) * 4 > 1 << 31:
        rows //= 2
    return rows


def _plain_window_train(st):
    q, k, v, do = (st[x].float() for x in ("q", "k", "v", "do"))
    B, H, N, d = q.shape
    Hkv, w, sk, scale = k.shape[1], st["window"], st["sinks"], st["scale"]
    q, do = q.unflatten(1, (Hkv, -1)), do.unflatten(1, (Hkv, -1))
    o, dq, lse = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q[..., 0])
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    step = _rows_at_once(B * H, min(w, N), min(sk, N))
    for i0 in range(0, N, step):
        i1 = min(N, i0 + step)
        qs, dos = q[..., i0:i1, :], do[..., i0:i1, :]
        s, j = _band_scores(qs, k, i0, i1, w, sk, scale)
        top = s.amax(-1, keepdim=True)
        p = s.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        p = p.div_(total)
        vj = v[..., j, :].unsqueeze(-3)
        out = torch.matmul(p, vj)
        o[..., i0:i1, :] = out
        lse[..., i0:i1] = (top + total.log()).squeeze(-1)
        dv[..., j, :] += torch.matmul(p.transpose(-1, -2), dos).sum(2)
        ds = torch.matmul(dos, vj.transpose(-1, -2)).sub_((dos * out).sum(-1, keepdim=True)).mul_(p).mul_(scale)
        dq[..., i0:i1, :] = torch.matmul(ds, k[..., j, :].unsqueeze(-3))
        dk[..., j, :] += torch.matmul(ds.transpose(-1, -2), qs).sum(2)
    dt = st["q"].dtype
    return (o.flatten(1, 2).to(dt), lse.flatten(1, 2), dq.flatten(1, 2).to(dt), dk.to(dt), dv.to(dt))


def _plain_window_prompt(st):
    q, k, v = st["q"], st["k"], st["v"]
    T, H, d = q.shape
    Hkv, w, sk = k.shape[1], st["window"], st["sinks"]
    o = torch.empty(T, H, d, dtype=q.dtype, device=q.device)
    lse = torch.empty(H, T, device=q.device)
    at = 0
    for n in st["lens"]:
        qs = q[at:at + n].float().transpose(0, 1).unflatten(0, (Hkv, -1))
        ks, vs = k[at:at + n].float().transpose(0, 1), v[at:at + n].float().transpose(0, 1)
        step = _rows_at_once(H, min(w, n), min(sk, n))
        for i0 in range(0, n, step):
            i1 = min(n, i0 + step)
            s, j = _band_scores(qs[..., i0:i1, :], ks, i0, i1, w, sk, st["scale"])
            top = s.amax(-1, keepdim=True)
            p = s.sub_(top).exp_()
            total = p.sum(-1, keepdim=True)
            out = torch.matmul(p, vs[:, None, j]) / total
            o[at + i0:at + i1] = out.flatten(0, 1).transpose(0, 1).to(q.dtype)
            lse[:, at + i0:at + i1] = (top + total.log()).squeeze(-1).flatten(0, 1)
        at += n
    return o, lse


def _softmaxed(s):
    """Weights, their sum and the largest score of rows that may see nothing."""
    top = s.amax(-1, keepdim=True).clamp_min(-3e38)
    p = torch.exp(s - top)
    return p, p.sum(-1, keepdim=True), top


def _plain_window_decode(st):
    q, k, v, lens = st["q"], st["k"], st["v"], st["lens"].long()
    B, H, Nq, d = q.shape
    Hkv, C = k.shape[1], k.shape[2]
    w, sk = min(st["window"], C), min(st["sinks"], C)
    lo = (lens - Nq - w + 1).clamp_min(0)  # the first row's window starts here
    j = torch.cat((torch.arange(sk, device=q.device).expand(B, sk),
                   lo[:, None] + torch.arange(min(C, w + Nq - 1), device=q.device)), -1)  # [B, slots]
    twice = torch.cat((torch.zeros(sk, dtype=torch.bool, device=q.device),
                       torch.ones(j.shape[1] - sk, dtype=torch.bool, device=q.device))) & (j < sk)
    i = lens[:, None] - Nq + torch.arange(Nq, device=q.device)  # a row's own slot
    dark = (j[:, None] > i[..., None]) | ((i[..., None] - j[:, None] >= w) & (j[:, None] >= sk)) | twice[:, None]
    gone = (j >= lens[:, None]) | twice
    at = (torch.arange(B, device=q.device)[:, None], slice(None), j.clamp_max(C - 1))
    ks, vs = (x[at].float().transpose(1, 2) for x in (k, v))  # [B, Hkv, slots, d]
    s = torch.matmul(q.float().view(B, Hkv, -1, d), ks.transpose(-1, -2)).view(B, Hkv, -1, Nq, j.shape[1])
    p, total, top = _softmaxed(s.mul_(st["scale"]).masked_fill_(dark[:, None, None], -math.inf))
    vs = vs.masked_fill(gone[:, None, :, None], 0.0)
    o = torch.matmul(p.flatten(2, 3), vs).view(B, H, Nq, d) / total.clamp_min(1e-38).view(B, H, Nq, 1)
    return o.to(q.dtype), torch.where(total > 0, top + total.log(), -math.inf).view(B, H, Nq)


def _plain_prefix(st):
    q, lens = st["q"], st["lens"].long()
    B, H, Nq, d = q.shape
    Hkv, C, P = st["k"].shape[1], st["k"].shape[2], st["P"]
    g = H // Hkv
    o = torch.empty_like(q)
    lse = torch.empty(B, H, Nq, device=q.device)
    slot = torch.arange(C, device=q.device)
    i = lens[:, None] - Nq + torch.arange(Nq, device=q.device)
    dark = (slot > i[..., None])[:, None]  # [B, 1, Nq, C]
    for h in range(Hkv):
        qs = q[:, h * g:(h + 1) * g].float()
        s = torch.cat((torch.matmul(qs.flatten(0, 2), st["kp"][h].float().T).view(B, g, Nq, P),
                       torch.matmul(qs.flatten(1, 2), st["k"][:, h].float().transpose(-1, -2)).view(B, g, Nq, C)
                       .masked_fill(dark, -math.inf)), -1)
        p, total, top = _softmaxed(s.mul_(st["scale"]))
        v = st["v"][:, h].float().masked_fill((slot >= lens[:, None])[..., None], 0.0)
        out = torch.matmul(p[..., :P].flatten(0, 2), st["vp"][h].float()).view(B, g, Nq, d)
        out = out + torch.matmul(p[..., P:].flatten(1, 2), v).view(B, g, Nq, d)
        o[:, h * g:(h + 1) * g] = (out / total).to(q.dtype)
        lse[:, h * g:(h + 1) * g] = (top + total.log()).squeeze(-1)
    return o, lse


# --------------------------------------------------------------------------- one pass


def run(state):
    if own:
        return _own(state)
    if state["op"] == "norm":
        return _plain_norm(state)
    if state["op"] == "prefix":
        return _plain_prefix(state)
    return {"train": _plain_window_train, "prompt": _plain_window_prompt,
            "decode": _plain_window_decode}[state["kind"]](state)


def _own(st):
    from exact_tiled_attention_07_gb300 import binding as fa

    if st["op"] == "norm":
        args = (st["q"], st["k"], st["wq"], st["wk"], st["table"])
        opts = {"positions": st["pos"], "eps": EPS, "interleaved": st["interleaved"]}
        out = fa.qk_norm_rope(*args, **opts)
        if st["kind"] == "packed":
            return list(out)
        return [*out, *fa.qk_norm_rope_backward(st["dq"], st["dk"], *args, **opts)]
    if st["op"] == "prefix":
        return fa.attention_decode_prefix(st["q"], st["kp"], st["vp"], st["k"], st["v"], st["lens"], scale=st["scale"])
    band = {"scale": st["scale"], "window": st["window"], "sinks": st["sinks"]}
    if st["kind"] == "decode":
        return fa.attention_decode_window(st["q"], st["k"], st["v"], st["lens"], **band)
    if st["kind"] == "prompt":
        return fa.attention_forward_varlen(st["q"], st["k"], st["v"], st["cu"], causal=True, **band)
    o, lse = fa.attention_forward(st["q"], st["k"], st["v"], causal=True, **band)
    return (o, lse, *fa.attention_backward(st["q"], st["k"], st["v"], o, st["do"], lse, causal=True, **band))


# --------------------------------------------------------------------------- the definitions in 64 bits


def exact(case, seed):
    if work(case)["flops"] > 4e12:
        return None
    st = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(st)
    if case["op"] == "window" and case["kind"] != "decode":
        return _exact_train(st) if case["kind"] == "train" else _exact_prompt(st)
    return _exact_decode(st)


def _exact_norm(st):
    """Row by row of the definition: the rotation as a matrix of its own for each position."""
    d, rotary = st["d"], st["rotary"]
    half = rotary // 2
    pos = st["pos"].long() if st["pos"] is not None else torch.arange(st["N"], device="cuda")
    c = torch.ones(len(pos), d, dtype=torch.float64, device="cuda")
    s = torch.zeros_like(c)
    ch = torch.arange(rotary, device="cuda")
    pair = ch // 2 if st["interleaved"] else ch % max(half, 1)
    second = (ch % 2 == 1) if st["interleaved"] else ch >= half  # the pair's other half
    mate = torch.arange(d, device="cuda")
    mate[:rotary] = torch.where(second, ch - (1 if st["interleaved"] else half), ch + (1 if st["interleaved"] else half))
    t = st["table"].double()[pos]
    c[:, :rotary], s[:, :rotary] = t[:, pair], t[:, half + pair] * torch.where(second, 1.0, -1.0)
    c, s = c[:, None], s[:, None]
    out, grads, wgrads = [], [], []
    for x, w, dy in ((st["q"], st["wq"], st.get("dq")), (st["k"], st["wk"], st.get("dk"))):
        x, w = x.double(), w.double()
        norm = torch.sqrt((x * x).sum(-1, keepdim=True) / d + EPS)
        y = x / norm * w
        y = y * c + y[..., mate] * s
        if dy is None:
            out.append(y)
            continue
        out.append(y.transpose(1, 2))
        dy = dy.double().transpose(1, 2)
        u = dy * c + (dy * s)[..., mate]
        wgrads.append((u * x / norm).sum((0, 1, 2)))
        grads.append(u * w / norm - x * (u * w * x).sum(-1, keepdim=True) / (d * norm ** 3))
    return out + grads + wgrads


def _visible(n, window, sinks, rows):
    j = torch.arange(n, device="cuda")
    i = rows[:, None]
    near = torch.logical_and(j <= i, j > i - window)
    return torch.logical_or(near, torch.logical_and(j <= i, j < sinks))


def _exact_head(q, k, v, st, do=None):
    """One head: outputs, log-sum-exps and, with do, the three gradients, some rows at a time over all keys they may see."""
    n = q.shape[0]
    o, lse = torch.empty_like(q), torch.empty(n, dtype=q.dtype, device=q.device)
    dq, dk, dv = torch.empty_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for i0 in range(0, n, 2048):
        rows = torch.arange(i0, min(n, i0 + 2048), device="cuda")
        end = int(rows[-1]) + 1
        begin = 0 if st["sinks"] else max(0, i0 - st["window"] + 1)
        s = q[rows] @ k[begin:end].T * st["scale"]
        s.masked_fill_(~_visible(end, st["window"], st["sinks"], rows)[:, begin:], -math.inf)
        lse[rows] = torch.logsumexp(s, -1)
        p = torch.exp(s - lse[rows, None])
        o[rows] = p @ v[begin:end]
        if do is None:
            continue
        g = do[rows]
        dv[begin:end] += p.T @ g
        ds = p * (g @ v[begin:end].T - (g * o[rows]).sum(-1, keepdim=True)) * st["scale"]
        dq[rows] = ds @ k[begin:end]
        dk[begin:end] += ds.T @ q[rows]
    return o, lse, dq, dk, dv


def _exact_train(st):
    B, H, N, d = st["q"].shape
    g = H // st["Hkv"]
    new = lambda like: torch.zeros(like.shape, dtype=torch.float64, device="cuda")  # noqa: E731
    o, dq, dk, dv = new(st["q"]), new(st["q"]), new(st["k"]), new(st["v"])
    lse = new(st["q"][..., 0])
    for b in range(B):
        for h in range(H):
            r = _exact_head(*(st[x][b, i].double() for x, i in (("q", h), ("k", h // g), ("v", h // g))), st,
                            st["do"][b, h].double())
            o[b, h], lse[b, h], dq[b, h] = r[:3]
            dk[b, h // g] += r[3]
            dv[b, h // g] += r[4]
    return o, lse, dq, dk, dv


def _exact_prompt(st):
    T, H, d = st["q"].shape
    g = H // st["Hkv"]
    o = torch.empty(T, H, d, dtype=torch.float64, device="cuda")
    lse = torch.empty(H, T, dtype=torch.float64, device="cuda")
    at = 0
    for n in st["lens"]:
        for h in range(H):
            r = _exact_head(*(st[x][at:at + n, i].double() for x, i in (("q", h), ("k", h // g), ("v", h // g))), st)
            o[at:at + n, h], lse[h, at:at + n] = r[:2]
        at += n
    return o, lse


def _exact_decode(st):
    B, H, Nq, d = st["q"].shape
    g = H // st["Hkv"]
    o = torch.zeros(B, H, Nq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, Nq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(st["lens"].tolist()):
        for hk in range(st["Hkv"]):
            for i in range(Nq):
                last = n - Nq + i  # the row's own slot
                parts = []
                if st["op"] == "prefix":
                    parts.append((st["kp"][hk], st["vp"][hk]))
                    first = 0
                else:
                    first = max(0, last - st["window"] + 1)
                    m = min(st["sinks"], first, last + 1)
                    parts.append((st["k"][b, hk, :m], st["v"][b, hk, :m]) if m > 0 else (st["k"][b, hk, :0],) * 2)
                if last >= 0:
                    parts.append((st["k"][b, hk, first:last + 1], st["v"][b, hk, first:last + 1]))
                k, v = (torch.cat([p[x].double() for p in parts]) for x in (0, 1))
                if k.shape[0] == 0:
                    continue
                s = st["q"][b, hk * g:(hk + 1) * g, i].double() @ k.T * st["scale"]
                lse[b, hk * g:(hk + 1) * g, i] = torch.logsumexp(s, -1)
                o[b, hk * g:(hk + 1) * g, i] = torch.softmax(s, -1) @ v
    return o, lse
