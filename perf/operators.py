"""What is measured of the 8-bit product and of the cache held in 4 bits.

Five paths, each with a plain form in torch (``own`` false) and as the calls
that a user makes of this framework (``own`` true):

  linear   y = x W^T: x's rows rounded to 8-bit integers with a scale of their
           own, multiplied with W's 8-bit rows and their scales
  product  the same product from codes and scales that are there already
  append   new tokens' K and V into a paged cache of 4 bits, and what the cache
           then holds of them
  decode,  attention over that cache: a token of each sequence, a few, or a
  extend   chunk of a prompt

An 8-bit row: s = max|x| / 127 and q = round(127 x / max|x|), half to even.  A
group of 64 values of a head in 4 bits: z = fp16(min), a = fp16((max - min) /
15), c = round((x - z) / a) in 0..15, half to even, standing for a c + z.  Byte
b of a head's vector holds value 2b in its low four bits and 2b + 1 in its
high ones.  Page t of the cache is [kv head][position][D / 2] bytes of K and
as many of V, and [kv head][position][D / 64] pairs (a, z) of each.
"""
import random

import torch

own = False

GROUP = 64
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one token through a gate or up projection kept at 8 bits: latency and the weight's bytes
        {"name": "linear 1x14336x4096", "op": "linear", "m": 1, "n": 14336, "k": 4096, "type": "fp16"},
        # a batch of 16 decoding through a down projection, codes at hand
        {"name": "product 16x4096x14336", "op": "product", "m": 16, "n": 4096, "k": 14336, "type": "bf16"},
        # a small odd layer: no size a multiple of anything
        {"name": "product 77x1111x1003", "op": "product", "m": 77, "n": 1111, "k": 1003, "type": "fp32"},
        # a ragged prompt through a wide layer
        {"name": "linear 333x28672x8192", "op": "linear", "m": 333, "n": 28672, "k": 8192, "type": "bf16"},
        # a long prompt: the tensor cores' rate
        {"name": "linear 4096x14336x4096", "op": "linear", "m": 4096, "n": 14336, "k": 4096, "type": "fp16"},
        # a decode step's new tokens, one of each of 64 sequences
        {"name": "append 64x1", "op": "append", "batch": 64, "new": 1, "len": 2000, "hq": 32, "hkv": 8, "d": 128,
         "page": 16, "type": "fp16"},
        # ragged prompts, 8192 tokens at most in all
        {"name": "append 8x1024", "op": "append", "batch": 8, "new": 1024, "len": 1500, "hq": 32, "hkv": 8, "d": 128,
         "page": 64, "type": "bf16"},
        # one user decoding: latency
        {"name": "decode 1x4001", "op": "decode", "batch": 1, "new": 1, "len": 4001, "hq": 32, "hkv": 8, "d": 128,
         "page": 16, "window": 0, "type": "fp16"},
        # a ragged batch decoding, an empty slot among it
        {"name": "decode 64x8192", "op": "decode", "batch": 64, "new": 1, "len": 8192, "hq": 32, "hkv": 8, "d": 128,
         "page": 64, "window": 0, "type": "fp16"},
        # one user with a long document
        {"name": "decode 1x131072", "op": "decode", "batch": 1, "new": 1, "len": 131072, "hq": 32, "hkv": 8, "d": 128,
         "page": 64, "window": 0, "type": "bf16"},
        # drafts of five tokens checked at once, one kv head for each query head
        {"name": "extend 16x5", "op": "extend", "batch": 16, "new": 5, "len": 3000, "hq": 16, "hkv": 16, "d": 64,
         "page": 32, "window": 1000, "type": "bf16"},
        # a prompt's chunk behind what the cache holds of it
        {"name": "extend 2x2048", "op": "extend", "batch": 2, "new": 2048, "len": 6000, "hq": 32, "hkv": 8, "d": 128,
         "page": 64, "window": 0, "type": "fp16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["linear", "product", "append", "decode", "decode", "extend"])
    if op in ("linear", "product"):
        m, n, k = _log(rng, 1, 4096), _log(rng, 64, 28672), _log(rng, 64, 16384)
        m = max(1, min(m, 2 ** 37 // (n * k)))
        return {"op": op, "m": m, "n": n, "k": k,
                "type": rng.choice(["fp16", "bf16"] if op == "linear" else ["fp16", "bf16", "fp32"])}
    hq, hkv = rng.choice([(32, 8), (32, 32), (8, 1), (28, 4), (16, 16), (12, 4), (40, 8), (16, 1)])
    d = rng.choice([64, 128, 128, 256])
    case = {"op": op, "hq": hq, "hkv": hkv, "d": d, "page": rng.choice([16, 32, 48, 64, 128]),
            "type": rng.choice(["fp16", "bf16"])}
    if op == "append":
        case["batch"] = _log(rng, 1, 64)
        case["new"] = _log(rng, 1, max(1, 2 ** 23 // (case["batch"] * hkv * d)))
        case["len"] = case["new"] + _log(rng, 1, 2000)
        return case
    case["window"] = rng.choice([0, 0, 0, 128, 1000])
    if op == "decode":
        case["batch"], case["new"] = _log(rng, 1, 128), 1
        case["len"] = max(1, min(_log(rng, 16, 65536), 2 ** 28 // (case["batch"] * hkv * d)))
    else:
        case["batch"] = _log(rng, 1, 32)
        case["new"] = max(2, min(_log(rng, 2, 2048), 4096 // case["batch"]))
        case["len"] = case["new"] + max(1, min(_log(rng, 16, 4096), 2 ** 27 // (case["batch"] * hkv * d)))
    return case


# ----------------------------------------------------------------- the inputs

def _lengths(case, seed):
    """(tokens in the cache, new ones among them) of each sequence."""
    r, one = random.Random(seed), case["batch"] == 1
    rows = random.Random(case["batch"] * 8191 + case["new"])  # the outputs' sizes are the case's
    lens, new = [], []
    for b in range(case["batch"]):
        n = case["new"] if one or case["new"] == 1 else rows.randint(max(1, case["new"] // 2), case["new"])
        if one:
            t = case["len"] - r.randint(0, case["len"] // 64)
        else:
            t = r.randint(case["len"] // 8, case["len"])
        lens.append(max(t, n))
        new.append(n)
    if case["batch"] >= 16 and case["op"] == "decode":
        lens[r.randrange(case["batch"])] = 0  # a slot that no request has
    return lens, new


def _pages(case, seed, g):
    lens, new = _lengths(case, seed)
    page, batch = case["page"], case["batch"]
    width = -(-case["len"] // page)
    pages = width * batch + 3
    table = torch.randperm(pages, generator=g, device="cuda")[:width * batch].view(batch, width).to(torch.int32)
    i32 = {"dtype": torch.int32, "device": "cuda"}
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return {"table": table.contiguous(), "kv_len": torch.tensor(lens, **i32), "cu": torch.tensor(cu, **i32),
            "tokens": cu[-1], "max_new": max(new), "max_len": max(1, max(lens)), "pages": pages,
            "max_seen": case["len"]}


def _cache(case, pages, g):
    """A cache of drawn codes (a group's lie about its middle) with scales and
    offsets as of values about N(0, 1)."""
    size = (pages, case["hkv"], case["page"])
    out = {}
    for part in ("k", "v"):
        code = torch.empty(*size, case["d"] // 2, dtype=torch.uint8, device="cuda")
        for p in range(0, pages, 512):  # in parts: the draws take eight times the codes' bytes
            c = torch.randn(code[p:p + 512].shape + (2,), generator=g, device="cuda")
            c = c.mul_(3.3).add_(7.5).round_().clamp_(0, 15).to(torch.uint8)
            code[p:p + 512] = c[..., 0] | (c[..., 1] << 4)
        a = torch.rand(*size, case["d"] // GROUP, generator=g, device="cuda") * 0.2 + 0.2
        z = a * (torch.randn(a.shape, generator=g, device="cuda") * 0.5 - 7.5)
        out[part], out[part + "_param"] = code, torch.stack([a, z], -1).to(torch.float16)
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    t = TYPES[case["type"]]
    s = {"case": dict(case)}
    if op in ("linear", "product"):
        m, n, k = case["m"], case["n"], case["k"]
        kp = -(-k // 16) * 16  # rows of codes start on 16 bytes
        w = torch.randn(n, k, generator=g, device="cuda") * 0.02
        top = w.abs().amax(1, keepdim=True)
        codes = torch.zeros(n, kp, dtype=torch.int8, device="cuda")
        codes[:, :k] = (w * (127 / top)).round().clamp(-127, 127).to(torch.int8)
        s["w"], s["w_scale"] = codes[:, :k], (top / 127).view(n)
        del w
        x = torch.randn(m, k, generator=g, device="cuda")
        x[:, torch.randperm(k, generator=g, device="cuda")[:max(1, k // 1000)]] *= 20  # channels that stick out
        if op == "linear":
            s["x"] = x.to(t)
        else:
            top = x.abs().amax(1, keepdim=True)
            codes = torch.zeros(m, kp, dtype=torch.int8, device="cuda")
            codes[:, :k] = (x * (127 / top)).round().clamp(-127, 127).to(torch.int8)
            s["x"], s["x_scale"] = codes[:, :k], (top / 127).view(m)
        return s
    s.update(_pages(case, seed, g))
    if op == "append":
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        qkv = torch.randn(s["tokens"], (hq + 2 * hkv) * d, generator=g, device="cuda").to(t)  # one projection's rows
        s["k_new"] = qkv[:, hq * d:(hq + hkv) * d].view(-1, hkv, d)
        s["v_new"] = qkv[:, (hq + hkv) * d:].view(-1, hkv, d)
        size = (s["pages"], hkv, case["page"])
        for part in ("k", "v"):
            s[part] = torch.zeros(*size, d // 2, dtype=torch.uint8, device="cuda")
            s[part + "_param"] = torch.zeros(*size, d // GROUP, 2, dtype=torch.float16, device="cuda")
    else:
        s["q"] = torch.randn(s["tokens"], case["hq"], case["d"], generator=g, device="cuda").to(t)
        s.update(_cache(case, s["pages"], g))
        # what no token has written yet: NaN in a page's last positions
        at = torch.arange(s["table"].shape[1] * case["page"], device="cuda").view(1, -1, case["page"])
        dead = at >= s["kv_len"].view(-1, 1, 1)
        page, pos = s["table"].long()[:, :, None].expand_as(dead)[dead], (at % case["page"]).expand_as(dead)[dead]
        for part in ("k_param", "v_param"):
            s[part][page, :, pos] = float("nan")
    if own:
        from bit_gemv_bcq_b200 import api
        s["cache"] = api.Kv4Cache(s["k"], s["k_param"], s["v"], s["v_param"])
    return s


# ------------------------------------------------------------------- one pass

def run(s):
    c = s["case"]
    if own:
        from bit_gemv_bcq_b200 import api
        if c["op"] == "linear":
            return api.linear_i8(s["x"], s["w"], s["w_scale"])
        if c["op"] == "product":
            return api.gemm_i8(s["x"], s["x_scale"], s["w"], s["w_scale"], dtype=TYPES[c["type"]])
        if c["op"] == "append":
            api.kv4_append(s["cache"], s["k_new"], s["v_new"], s["table"], s["kv_len"], s["cu"])
            return api.kv4_read(s["cache"], s["table"], s["kv_len"], s["cu"], tokens=s["tokens"], dtype=TYPES[c["type"]])
        return api.kv4_attention(s["q"], s["cache"], s["table"], s["kv_len"], s["cu"], max_q=s["max_new"],
                                 max_kv=s["max_seen"], window=c["window"], return_lse=True)
    if c["op"] == "linear":
        x = s["x"].float()
        top = x.abs().amax(1, keepdim=True)
        # in 64 bits: whether 127 x / top lies on a half decides the code
        codes = torch.where(top > 0, (x.double() * 127 / top.double()).round(), 0.0).float()
        return _scaled(codes, (top / 127).view(-1), s["w"], s["w_scale"]).to(s["x"].dtype)
    if c["op"] == "product":
        return _scaled(s["x"].float(), s["x_scale"], s["w"], s["w_scale"]).to(TYPES[c["type"]])
    if c["op"] == "append":
        return _held(s["k_new"]), _held(s["v_new"])
    return _attention(s, c)


def _scaled(codes, scale, w, w_scale):
    return (codes @ w.float().t()) * scale[:, None] * w_scale[None, :]


def _held(x):
    """What the cache holds for x [T][heads][D]."""
    v = x.double().view(*x.shape[:2], -1, GROUP)
    lo, hi = v.amin(-1, keepdim=True).float(), v.amax(-1, keepdim=True).float()
    z, a = lo.half().double(), ((hi - lo) / 15).half().double()
    code = torch.where(a > 0, (v - z) / a, 0.0).round().clamp(0, 15)
    return (code * a + z).float().to(x.dtype).view(x.shape)


def _values(code, param):
    """[pages][heads][position][D] in 32 bits."""
    x = torch.stack([code & 15, code >> 4], -1).flatten(-2).float()
    x = x.view(*x.shape[:-1], -1, GROUP)
    return (x * param[..., :1].float() + param[..., 1:].float()).flatten(-2)


def _attention(s, c):
    hkv, d, group = c["hkv"], c["d"], c["hq"] // c["hkv"]
    table, kv_len, cu = s["table"].long(), s["kv_len"].long(), s["cu"].long()
    new = cu[1:] - cu[:-1]
    # K and V of every sequence in order, [batch][kv head][position][D]; zeros where there is no token
    width = -(-s["max_len"] // c["page"])
    table = table[:, :width]
    key = _values(s["k"][table], s["k_param"][table]).transpose(1, 2).flatten(2, 3)
    value = _values(s["v"][table], s["v_param"][table]).transpose(1, 2).flatten(2, 3)
    at = torch.arange(key.shape[2], device=key.device)
    dead = (at[None] >= kv_len[:, None])[:, None, :, None]
    key.masked_fill_(dead, 0.0)
    value.masked_fill_(dead, 0.0)
    # queries of a sequence side by side, [batch][kv head][group x new][D]
    i = torch.arange(s["max_new"], device=key.device)
    row = (cu[:-1, None] + i[None]).clamp(max=s["tokens"] - 1)
    q = s["q"].float()[row].view(*row.shape, hkv, group, d).permute(0, 2, 3, 1, 4).flatten(2, 3)
    score = (q @ key.transpose(-1, -2)) * d ** -0.5
    pos = (kv_len - new)[:, None] + i[None]  # [batch][new]
    hide = at[None, None] > pos[..., None]
    if c["window"]:
        hide |= at[None, None] <= pos[..., None] - c["window"]
    hide |= at[None, None] >= kv_len[:, None, None]
    hide = hide[:, None, None].expand(-1, 1, group, -1, -1).flatten(2, 3)
    score.masked_fill_(hide, float("-inf"))
    top = score.amax(-1, keepdim=True)
    top = torch.where(top.isinf(), 0.0, top)
    score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    out = torch.where(total > 0, (score @ value) / total, 0.0)
    lse = (top + total.log()).squeeze(-1)
    # back to rows of tokens
    token = torch.arange(s["tokens"], device=key.device)
    seq = torch.searchsorted(cu[1:].contiguous(), token, right=True)
    k = token - cu[seq]
    out = out.view(len(kv_len), hkv, group, -1, d)[seq, :, :, k]
    lse = lse.view(len(kv_len), hkv, group, -1)[seq, :, :, k]
    return out.reshape(s["tokens"], c["hq"], d).to(s["q"].dtype), lse.reshape(s["tokens"], c["hq"])


# --------------------------------------------------------- what a pass cannot do without

def work(case):
    size = 4 if case["type"] == "fp32" else 2
    op = case["op"]
    if op in ("linear", "product"):
        m, n, k = case["m"], case["n"], case["k"]
        x = m * k * size if op == "linear" else m * k + 4 * m
        return {"bytes": x + n * k + 4 * n + m * n * size, "flops": 2 * m * n * k}
    lens, new = _lengths(case, 1)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    held = 2 * hkv * (d // 2 + d // GROUP * 4)  # bytes of a token in the cache
    if op == "append":
        return {"bytes": sum(new) * (2 * 2 * 2 * hkv * d + held), "flops": 8 * sum(new) * hkv * d}
    seen = pairs = 0
    window = case["window"] or 1 << 40
    for t, n in zip(lens, new):
        seen += max(0, t - max(0, t - n - window + 1))
        pairs += sum(min(window, max(0, t - n + i + 1)) for i in range(n))
    return {"bytes": seen * held + sum(new) * hq * (2 * d * size + 4), "flops": 4 * d * hq * pairs}


# --------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("linear", "product"):
        if op == "linear":
            x = s["x"].double()
            most = x.abs().max(dim=1, keepdim=True).values
            codes = torch.round(127 * x / most.clamp(min=1e-300))  # 127 x is exact and a half stays one
            scale = most.squeeze(1) / 127
        else:
            codes, scale = s["x"].double(), s["x_scale"].double()
        return torch.einsum("mk,nk->mn", codes, s["w"].double()) * torch.outer(scale, s["w_scale"].double())
    if op == "append":
        both = []
        for x in (s["k_new"], s["v_new"]):
            x = x.cpu().numpy() if x.dtype == torch.float16 else x.cpu().float().numpy()
            both.append(torch.from_numpy(_held_numpy(x)))
        return tuple(both)
    hkv, d, page = case["hkv"], case["d"], case["page"]
    group = case["hq"] // hkv
    lens, cu = s["kv_len"].tolist(), s["cu"].tolist()
    out = torch.zeros(s["tokens"], case["hq"], d, dtype=torch.float64, device="cuda")
    lse = torch.full((s["tokens"], case["hq"]), float("-inf"), dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        if n == 0:
            continue
        at = torch.arange(n, device="cuda")
        where = s["table"][b].long()[at // page], at % page
        new = cu[b + 1] - cu[b]
        seen = at[None, :] <= (n - new + torch.arange(new, device="cuda"))[:, None]
        if case["window"]:
            seen &= at[None, :] > (n - new + torch.arange(new, device="cuda"))[:, None] - case["window"]
        for h in range(hkv):
            kv = []
            for part in ("k", "v"):
                byte, param = s[part][where[0], h, where[1]].long(), s[part + "_param"][where[0], h, where[1]].double()
                x = torch.empty(n, d, dtype=torch.float64, device="cuda")
                x[:, 0::2], x[:, 1::2] = byte % 16, byte // 16
                kv.append(x * param[..., 0].repeat_interleave(GROUP, 1) + param[..., 1].repeat_interleave(GROUP, 1))
            for e in range(h * group, (h + 1) * group):
                score = s["q"][cu[b]:cu[b + 1], e].double() @ kv[0].t() / d ** 0.5
                score = torch.where(seen, score, float("-inf"))
                lse[cu[b]:cu[b + 1], e] = torch.logsumexp(score, 1)
                out[cu[b]:cu[b + 1], e] = torch.softmax(score, 1) @ kv[1]
    return out, lse


def _held_numpy(x):
    import numpy as np
    v = x.astype(np.float64).reshape(*x.shape[:2], -1, GROUP)
    lo, hi = v.min(-1, keepdims=True), v.max(-1, keepdims=True)
    z = lo.astype(np.float16).astype(np.float64)
    a = ((hi - lo).astype(np.float32) / np.float32(15)).astype(np.float16).astype(np.float64)
    code = np.clip(np.rint((v - z) / np.where(a > 0, a, np.inf)), 0, 15)
    return (code * a + z).reshape(x.shape)
