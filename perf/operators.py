"""Measured cases of the operators between the ternary matmuls of a layer:

* ``norm``  -- the block boundary: norm after the block, gate, residual scale, residual
  add, norm before the next block, int8 tokens (or the float tokens) for it;
* ``cache`` -- keys and values quantised to 4 bits as they are written into a paged
  cache, and read back;
* ``attn``  -- causal attention over that cache, with an optional sliding window and
  a few first tokens that stay visible.

With ``own`` false the operators are computed in elementary torch operations,
with ``own`` true by this package's calls.
"""
import math

import numpy as np
import torch

own = False

PAGE = 64        # tokens of a cache page
GROUP = 64       # channels that share one (step, middle) pair
CLAMP = 57344.0  # what a cached value saturates at
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases

def _norm(n, f, b="fp32", stream="bf16", post=False, gate="none", scale=1.0, tokens="int8"):
    return {"op": "norm", "n": n, "f": f, "b": b, "stream": stream, "post": post, "gate": gate,
            "scale": scale, "tokens": tokens}


def _cache(seqs, new, old, kv_heads, dim, dtype, read):
    return {"op": "cache", "seqs": seqs, "new": new, "old": old, "kv_heads": kv_heads,
            "dim": dim, "dtype": dtype, "read": read}


def _attn(seqs, new, old, heads, kv_heads, dim, dtype, window=0, sinks=0):
    return {"op": "attn", "seqs": seqs, "new": new, "old": old, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "dtype": dtype, "window": window, "sinks": sinks}


def listed():
    return [
        # one decoded token of the 2B-class layer (hidden 2560) crossing a block boundary
        dict(_norm(1, 2560), name="norm 1 token"),
        # a decode batch of the large layer with norms on both sides of the block
        dict(_norm(64, 8192, stream="fp32", post=True, gate="channel", scale=0.22),
             name="norm 64 tokens"),
        # a prompt of the 2B-class layer, gated per token and channel
        dict(_norm(4096, 2560, post=True, gate="token", scale=0.5), name="norm prompt"),
        # the last norm before the output projection, float tokens, an odd batch
        dict(_norm(333, 1024, b="bf16", stream="bf16", tokens="float"), name="norm float"),
        # a decode batch writing one token per sequence, and reading it back
        dict(_cache(64, 1, 1000, 5, 128, "fp32", "new"), name="cache 1 token"),
        # prompts of three sequences written into fresh pages and read back
        dict(_cache(3, 2731, 0, 8, 128, "bf16", "new"), name="cache prompt"),
        # a stored history read back after a short continuation
        dict(_cache(16, 5, 2043, 5, 128, "fp32", "all"), name="cache history"),
        # one sequence, one token, a short history: latency
        dict(_attn(1, 1, 514, 20, 5, 128, "fp32"), name="attn 1 token"),
        # a decode batch of the large layer's heads, ragged histories
        dict(_attn(64, 1, 4095, 64, 8, 128, "bf16"), name="attn 64 tokens"),
        # one token over a very long history
        dict(_attn(1, 1, 131071, 20, 5, 128, "fp32"), name="attn long"),
        # prompts of three sequences, from nothing
        dict(_attn(3, 2048, 0, 16, 8, 128, "bf16"), name="attn prompt"),
        # a chunk of a long prompt under a sliding window with four sinks
        dict(_attn(2, 300, 16000, 32, 8, 64, "fp32", 4096, 4), name="attn window"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    most = {"norm": 9e7, "cache": 3e7, "attn": 1.5e8}
    while True:
        op = rng.choice(["norm", "cache", "attn", "attn"])
        if op == "norm":
            c = _norm(_log(rng, 1, 4096), 128 * _log(rng, 2, 128), rng.choice(["fp32", "bf16"]),
                      rng.choice(["fp32", "bf16"]), rng.random() < 0.5,
                      rng.choice(["none", "channel", "token"]), round(rng.uniform(0.1, 1.5), 3),
                      rng.choice(["int8", "int8", "float"]))
        elif op == "cache":
            c = _cache(_log(rng, 1, 64), _log(rng, 1, 4096), rng.choice([0, _log(rng, 1, 4096)]),
                       rng.choice([1, 2, 4, 5, 8]), rng.choice([64, 128, 256]),
                       rng.choice(["fp32", "bf16"]), rng.choice(["new", "all"]))
        else:
            kv = rng.choice([1, 2, 4, 5, 8])
            c = _attn(_log(rng, 1, 64), rng.choice([1, 1, _log(rng, 2, 2048)]), _log(rng, 1, 100000),
                      kv * rng.choice([1, 2, 4, 6, 8]), kv, rng.choice([64, 128, 128, 256]),
                      rng.choice(["fp32", "bf16"]))
            if rng.random() < 0.3:
                c["window"], c["sinks"] = _log(rng, 16, 8192), rng.choice([0, 1, 4, 64])
        # the scores of the plain form, and its whole histories in 32 bits, have to fit
        n, t = c.get("new", 0), c.get("new", 0) + c.get("old", 0)
        if op == "attn" and (c["seqs"] * c["heads"] * n * t > 3e8 or
                             c["seqs"] * c["kv_heads"] * t * c["dim"] > 3e8):
            continue
        if _cost(c) <= most[op]:
            return c


# ---------------------------------------------------------------- inputs

def _lengths(case):
    """Tokens that each sequence adds and holds already: the first sequence has the
    stated numbers, the others fewer (ragged), the same ones for every seed."""
    r = np.random.RandomState(case["seqs"])
    new = [case["new"]] + [max(1, int(case["new"] * r.uniform(0.3, 1))) for _ in range(case["seqs"] - 1)]
    old = [case["old"]] + [int(case["old"] * r.uniform(0.2, 1)) for _ in range(case["seqs"] - 1)]
    return np.array(new), np.array(old)


def _kv(shape, g, dev):
    """Keys or values: near normal, a few channels many times as large (as keys have
    them) and a middle that differs between channels."""
    d = shape[-1]
    gain = 1 + 7 * (torch.rand(d, generator=g, device=dev) < 0.04).float()
    mid = 0.5 * torch.randn(d, generator=g, device=dev)
    return torch.randn(shape, generator=g, device=dev).mul_(gain).add_(mid)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    s = {"case": case}
    if case["op"] == "norm":
        n, f, bt, st = case["n"], case["f"], DTYPES[case["b"]], DTYPES[case["stream"]]
        s["b"] = torch.randn((n, f), generator=g, device=dev).mul_(1.7).to(bt)
        gain = 1 + 20 * (torch.rand(f, generator=g, device=dev) < 0.005).float()
        s["res"] = (torch.randn((n, f), generator=g, device=dev) * gain).to(st)
        s["gamma"] = 1 + 0.2 * torch.randn(f, generator=g, device=dev)
        s["post_gamma"] = 1 + 0.2 * torch.randn(f, generator=g, device=dev) if case["post"] else None
        s["gate"] = {"none": None, "channel": torch.rand(f, generator=g, device=dev) + 0.5,
                     "token": torch.rand((n, f) if case["gate"] == "token" else (1, 1), generator=g,
                                         device=dev) + 0.5}[case["gate"]]
        return s
    new, old = _lengths(case)
    dim, kvh, dt = case["dim"], case["kv_heads"], DTYPES[case["dtype"]]
    kv_len = new + old
    pages = -(-kv_len // PAGE)
    total = int(pages.sum()) + 3
    perm = torch.randperm(total, generator=g, device=dev).cpu().numpy()
    table = np.full((case["seqs"], int(pages.max())), -1, np.int32)
    at = 0
    for b, p in enumerate(pages):
        table[b, :p] = perm[at:at + p]
        at += p
    put = lambda a: torch.from_numpy(np.asarray(a, np.int32)).to(dev)  # noqa: E731
    s["table"], s["kv_len"] = put(table), put(kv_len)
    s["q_start"] = put(np.concatenate([[0], np.cumsum(new)]))
    s["max_kv"], s["n"] = int(kv_len.max()), int(new.sum())
    s["max_new"] = int(new.max())
    # pages are handed out as they are: what no token was written to holds anything
    s["cache"] = torch.full((total, kvh, 72 * dim), 255, dtype=torch.uint8, device=dev)
    if case["op"] == "cache":
        first, filled = np.zeros(len(old)), old
        s["k"], s["v"] = (_kv((s["n"], kvh, dim), g, dev).to(dt) for _ in range(2))
        span = kv_len if case["read"] == "all" else new
        s["r_start"], s["n_read"] = put(np.concatenate([[0], np.cumsum(span)])), int(span.sum())
    else:
        first, filled = np.zeros(len(old)), kv_len
        s["q"] = torch.randn((s["n"], case["heads"], dim), generator=g, device=dev).to(dt)
    if filled.sum():
        start = put(np.concatenate([[0], np.cumsum(filled)]))
        k, v = (_kv((int(filled.sum()), kvh, dim), g, dev) for _ in range(2))
        _write(s["cache"], *_where(s["table"], put(filled), start, int(filled.sum())), k, v)
    return s


# ---------------------------------------------------------------- plain forms

def _where(table, kv_len, start, n):
    """Page and place in it of n tokens: token start[b] + i of sequence b is at position
    kv_len[b] - (start[b + 1] - start[b]) + i."""
    r = torch.arange(n, device=table.device)
    b = torch.searchsorted(start[1:].contiguous(), r.to(start.dtype), right=True)
    pos = kv_len[b].long() - start[b + 1].long() + r
    return table[b, pos // PAGE].long(), pos % PAGE


def _parts(cache):
    """The four parts of every page record: key codes [token][quad][32 channels][byte], value
    codes [four tokens][lane][group][token, two bytes], and their (step, middle) pairs."""
    d = cache.shape[2] // 72
    return (cache[:, :, :32 * d].unflatten(2, (PAGE, 4, d // 32, 4)),
            cache[:, :, 32 * d:64 * d].unflatten(2, (16, 16, d // 64, 4, 2)),
            cache[:, :, 64 * d:68 * d].view(torch.float16).unflatten(2, (PAGE, d // 64, 2)),
            cache[:, :, 68 * d:].view(torch.float16).unflatten(2, (16, d // 64, 2, 4)))


def _quantise(x):
    """x[n][heads][dim] -> codes 0..15, step and middle of each group, both 16-bit."""
    x = x.float().clamp(-CLAMP, CLAMP).unflatten(2, (-1, GROUP))
    lo, hi = x.amin(3, True), x.amax(3, True)
    mid = (lo + (hi - lo) * np.float32(8 / 15).item()).half()
    m = mid.float()
    step = torch.maximum((hi - m) * np.float32(1 / 7).item(), (m - lo) * 0.125).half()
    inv = torch.where(step > 0, 1 / step.float(), torch.zeros_like(m))
    code = ((x - m) * inv + 8).round().clamp(0, 15).to(torch.uint8)
    return code.flatten(2), step.squeeze(3), mid.squeeze(3)


def _write(cache, page, place, k, v):
    kc, vc, km, vm = _parts(cache)
    n, heads, d = k.shape
    code, step, mid = _quantise(k)
    code = code.view(n, heads, d // 32, 4, 4, 2).transpose(2, 3)
    kc[page, :, place] = code[..., 0] | code[..., 1] << 4
    km[page, :, place] = torch.stack([step, mid], 3)
    code, step, mid = _quantise(v)
    code = code.view(n, heads, d // 64, 16, 2, 2).transpose(2, 3)
    vc[page, :, place // 4, :, :, place % 4] = code[..., 0] | code[..., 1] << 4
    vm[page, :, place // 4, :, :, place % 4] = torch.stack([step, mid], 3)


def _value(code, step, mid):
    """codes [..., groups, 64] -> fp32 values."""
    return mid.float()[..., None] + step.float()[..., None] * (code.float() - 8)


def _nibbles(x):
    return torch.stack([x & 15, x >> 4], -1).flatten(-2)


def _key_rows(codes, meta):
    """[..., quad, 32 channels, byte] and [..., group, 2] -> [..., dim]."""
    c = _nibbles(codes).transpose(-3, -2).flatten(-3).unflatten(-1, (-1, GROUP))
    return _value(c, meta[..., 0], meta[..., 1]).flatten(-2)


def _value_rows(codes, step, mid):
    """[..., lane, group, 2] and [..., group] -> [..., dim]."""
    c = _nibbles(codes).transpose(-3, -2).flatten(-2)
    return _value(c, step, mid).flatten(-2)


def _read(cache, page, place):
    kc, vc, km, vm = _parts(cache)
    m = vm[page, :, place // 4, :, :, place % 4]
    return (_key_rows(kc[page, :, place], km[page, :, place]),
            _value_rows(vc[page, :, place // 4, :, :, place % 4], m[..., 0], m[..., 1]))


def _plain_cache(s):
    c = s["case"]
    _write(s["cache"], *_where(s["table"], s["kv_len"], s["q_start"], s["n"]), s["k"], s["v"])
    k, v = _read(s["cache"], *_where(s["table"], s["kv_len"], s["r_start"], s["n_read"]))
    return k.to(DTYPES[c["dtype"]]), v.to(DTYPES[c["dtype"]])


def _plain_attn(s):
    c, dev = s["case"], s["q"].device
    seqs, heads, kvh, d = c["seqs"], c["heads"], c["kv_heads"], c["dim"]
    kc, vc, km, vm = _parts(s["cache"][s["table"].clamp(min=0).long()].flatten(0, 1))
    k = _key_rows(kc, km).unflatten(0, (seqs, -1)).transpose(1, 2).flatten(2, 3)
    vm = vm.permute(0, 1, 2, 5, 3, 4)   # [page][head][four tokens][token][group][2]
    v = _value_rows(vc.permute(0, 1, 2, 5, 3, 4, 6), vm[..., 0], vm[..., 1]).flatten(2, 3)
    v = v.unflatten(0, (seqs, -1)).transpose(1, 2).flatten(2, 3)
    t = k.shape[2]
    j = torch.arange(t, device=dev)
    held = j < s["kv_len"][:, None]                                    # [seqs][t]
    k = k.masked_fill(~held[:, None, :, None], 0.0)
    v = v.masked_fill(~held[:, None, :, None], 0.0)
    # queries padded to the longest continuation, the heads of a group side by side
    n = s["max_new"]
    i = torch.arange(n, device=dev)
    count = (s["q_start"][1:] - s["q_start"][:-1])[:, None]
    row = (s["q_start"][:-1, None] + i).clamp(max=s["n"] - 1).long()
    q = s["q"][row].float().unflatten(2, (kvh, heads // kvh)).permute(0, 2, 1, 3, 4)
    score = torch.matmul(q.reshape(seqs, kvh, -1, d), k.transpose(2, 3)) * (1 / math.sqrt(d))
    score = score.view(seqs, kvh, n, heads // kvh, t)
    pos = s["kv_len"][:, None] - count + i                             # [seqs][n]
    see = held[:, None] & (j <= pos[:, :, None])
    if c["window"]:
        see &= (j > pos[:, :, None] - c["window"]) | (j < c["sinks"])
    score.masked_fill_(~see[:, None, :, None], -math.inf)
    score -= score.amax(4, True).clamp(min=-3e38)
    score.exp_()
    den = score.sum(4)
    o = torch.matmul(score.flatten(2, 3), v).view(seqs, kvh, n, heads // kvh, d)
    o = torch.where(den[..., None] > 0, o / den[..., None], torch.zeros_like(o))
    o = o.permute(0, 2, 1, 3, 4).reshape(seqs, n, heads, d)
    return o[i < count].to(s["q"].dtype)


def _factor(x, eps):
    """fp32(1 / sqrt(mean of squares + eps)), the mean in binary64."""
    return (1 / (x.double().square().mean(1, True) + eps).sqrt()).float()


EPS = np.float32(1e-5).item()


def _plain_norm(s):
    c = s["case"]
    t = s["b"].float()
    if c["post"]:
        t = t * _factor(t, EPS) * s["post_gamma"]
    if s["gate"] is not None:
        t = t * s["gate"]
    h = (s["res"].float() + t * np.float32(c["scale"]).item()).to(s["res"].dtype)
    v = h.float() * _factor(h, EPS) * s["gamma"]
    if c["tokens"] == "float":
        return h, v.to(h.dtype)
    scale = (127.0 / v.abs().amax(1).clamp(min=np.float32(1e-5).item()).double()).float()
    code = (v * scale[:, None]).round().clamp(-128, 127).to(torch.int8)
    return h, code / scale[:, None], scale, code.sum(1, dtype=torch.int32)


def run(s):
    c = s["case"]
    if own:
        return _own(s)
    return {"norm": _plain_norm, "cache": _plain_cache, "attn": _plain_attn}[c["op"]](s)


# ---------------------------------------------------------------- the package's calls

def _own(s):
    import ternary_weight_i2_amd as bn
    c = s["case"]
    if c["op"] == "attn":
        return bn.attn_kv4(s["q"], s["cache"], s["table"], s["kv_len"], s["q_start"],
                           window=c["window"], sinks=c["sinks"], max_kv=s["max_kv"])
    if c["op"] == "cache":
        bn.kv4_append(s["cache"], s["table"], s["kv_len"], s["q_start"], s["k"], s["v"])
        return bn.kv4_read(s["cache"], s["table"], s["kv_len"], s["r_start"], s["n_read"],
                           dtype=s["k"].dtype)
    floats = c["tokens"] == "float"
    h, v, tokens = bn.block_norm_quant(
        s["b"], s["res"], post_norm=c["post"], post_gamma=s["post_gamma"], gate=s["gate"],
        scale=c["scale"], gamma=s["gamma"], eps=1e-5, want_v=floats, want_q=not floats)
    if floats:
        return h, v
    code, scale, total = tokens
    return h, code / scale[:, None], scale, total


# ---------------------------------------------------------------- work

def work(case):
    if case["op"] == "norm":
        n, f = case["n"], case["f"]
        size = {"fp32": 4, "bf16": 2}
        each = size[case["b"]] + 2 * size[case["stream"]]
        each += 1 if case["tokens"] == "int8" else size[case["stream"]]
        each += 4 if case["gate"] == "token" else 0
        return {"bytes": n * f * each + 8 * f, "flops": n * f * (12 if case["post"] else 8)}
    new, old = _lengths(case)
    n, dim, kvh = int(new.sum()), case["dim"], case["kv_heads"]
    size = {"fp32": 4, "bf16": 2}[case["dtype"]]
    token = kvh * dim * 9 // 8          # one token's keys and values with their pairs
    if case["op"] == "cache":
        read = int((new + old).sum()) if case["read"] == "all" else n
        values = (n + read) * 2 * kvh * dim
        return {"bytes": values * size + (n + read) * token, "flops": 6 * values}
    pairs = seen = 0
    for a, o in zip(new.tolist(), old.tolist()):
        pos = np.arange(o, o + a)
        low = np.zeros_like(pos)
        if case["window"]:
            low = np.maximum(0, pos - case["window"] + 1)
        pairs += int((pos + 1 - low + np.minimum(low, case["sinks"])).sum())
        seen += int(o + a - low[0] + min(low[0], case["sinks"]))
    return {"bytes": seen * token + 2 * n * case["heads"] * dim * size,
            "flops": 4 * dim * case["heads"] * pairs}


# ---------------------------------------------------------------- from the definitions, in 64 bits

def _bits(a, count):
    return [(a >> (4 * i)) & 15 for i in range(count)]


def _exact_rows(rec, d):
    """One page record (a numpy row of bytes) -> keys and values [64][d] in binary64."""
    g = d // 64
    k, v = np.empty((PAGE, d)), np.empty((PAGE, d))
    kw = rec[:32 * d].view("<u4").reshape(PAGE, 4, d // 32)
    for quad in range(4):
        for step in range(d // 32):
            for i, c in enumerate(_bits(kw[:, quad, step], 8)):
                k[:, 32 * step + 8 * quad + i] = c
    vw = rec[32 * d:64 * d].view("<u2").reshape(16, 16, g, 4)
    for lane in range(16):
        for p in range(g):
            for i, c in enumerate(_bits(vw[:, lane, p], 4)):
                v[:, 64 * p + 4 * lane + i] = c.reshape(-1)
    km = rec[64 * d:68 * d].view("<f2").astype(np.float64).reshape(PAGE, g, 2)
    vm = rec[68 * d:].view("<f2").astype(np.float64).reshape(16, g, 2, 4).transpose(0, 3, 1, 2)
    vm = vm.reshape(PAGE, g, 2)
    with np.errstate(invalid="ignore"):
        for p in range(g):
            at = slice(64 * p, 64 * p + 64)
            k[:, at] = km[:, p, 1:] + km[:, p, :1] * (k[:, at] - 8)
            v[:, at] = vm[:, p, 1:] + vm[:, p, :1] * (v[:, at] - 8)
    return k, v


def _exact_cached(x):
    """What x[n][heads][dim] stands for once cached: the quantiser as it is defined, with
    each of its roundings to 32 and 16 bits."""
    f4 = np.float32
    x = np.clip(x.astype(f4), -f4(CLAMP), f4(CLAMP))
    x = x.reshape(x.shape[0], x.shape[1], -1, GROUP)
    lo, hi = x.min(3, keepdims=True), x.max(3, keepdims=True)
    mid = (lo + (hi - lo) * f4(8 / 15)).astype(np.float16).astype(f4)
    step = np.maximum((hi - mid) * f4(1 / 7), (mid - lo) * f4(1 / 8)).astype(np.float16).astype(f4)
    with np.errstate(divide="ignore"):
        inv = np.where(step > 0, f4(1) / step, f4(0))
    code = np.clip(np.rint((x - mid) * inv + f4(8)), 0, 15).astype(np.float64)
    return (mid + step.astype(np.float64) * (code - 8)).reshape(x.shape[0], x.shape[1], -1)


def exact(case, seed):
    s = prepare(case, seed)
    host = lambda t: None if t is None else t.float().cpu().numpy()  # noqa: E731
    if case["op"] == "norm":
        return _exact_norm(case, s, host)
    if case["op"] == "cache" and case["read"] == "new":
        return [torch.from_numpy(_exact_cached(host(s[x]))) for x in ("k", "v")]
    new, old = _lengths(case)
    if case["op"] == "cache":
        fresh = [_exact_cached(host(s[x])) for x in ("k", "v")]
        outs, at = ([], []), 0
        for b in range(case["seqs"]):
            kv = _exact_history(s, b, int(old[b]))
            for o, h, f in zip(outs, kv, fresh):
                o += [h[:old[b]], f[at:at + new[b]]]
            at += new[b]
        return [torch.from_numpy(np.concatenate(o)) for o in outs]
    out, at = [], 0
    for b in range(case["seqs"]):
        n, t = int(new[b]), int(new[b] + old[b])
        k, v = (torch.from_numpy(x[:t]).cuda() for x in _exact_history(s, b, t))
        q = s["q"][at:at + n].double()
        pos = torch.arange(t - n, t, device="cuda")[:, None]
        j = torch.arange(t, device="cuda")[None]
        hide = j > pos
        if case["window"]:
            hide = hide | ((j <= pos - case["window"]) & (j >= case["sinks"]))
        heads = []
        for h in range(case["heads"]):
            kvh = h // (case["heads"] // case["kv_heads"])
            w = (q[:, h] @ k[:, kvh].t().contiguous()) / math.sqrt(case["dim"])
            heads.append(torch.softmax(w.masked_fill(hide, -math.inf), 1) @ v[:, kvh].contiguous())
        out.append(torch.stack(heads, 1))
        at += n
    return torch.cat(out)


def _exact_history(s, b, t):
    """Keys and values [t][heads][dim] of sequence b's first t tokens (and what pads the page)."""
    d, kvh = s["cache"].shape[2] // 72, s["cache"].shape[1]
    pages = s["table"][b, :-(-t // PAGE)].long()
    rec = s["cache"][pages].cpu().numpy()
    k, v = np.empty((len(rec) * PAGE, kvh, d)), np.empty((len(rec) * PAGE, kvh, d))
    for p in range(len(rec)):
        for h in range(kvh):
            k[p * PAGE:p * PAGE + PAGE, h], v[p * PAGE:p * PAGE + PAGE, h] = _exact_rows(rec[p, h], d)
    return k, v


def _exact_norm(case, s, host):
    """The boundary as it is defined: every product and sum of two numbers formed in
    binary64 and rounded to the 32 bits that the definition gives it."""
    f4, f8 = np.float32, np.float64
    stored = (lambda a: torch.from_numpy(a).to(DTYPES[case["stream"]]).float().numpy())

    def factor(a):
        return (1 / np.sqrt((a.astype(f8) ** 2).mean(1, keepdims=True) + f8(f4(1e-5)))).astype(f4)

    def times(a, b):
        return (a.astype(f8) * np.asarray(b).astype(f8)).astype(f4)

    t = host(s["b"])
    if case["post"]:
        t = times(times(t, factor(t)), host(s["post_gamma"]))
    if s["gate"] is not None:
        t = times(t, host(s["gate"]))
    t = times(t, f4(case["scale"]))
    h = stored((host(s["res"]).astype(f8) + t.astype(f8)).astype(f4))
    v = times(times(h, factor(h)), host(s["gamma"]))
    if case["tokens"] == "float":
        return torch.from_numpy(h.astype(f8)), torch.from_numpy(v.astype(f8))
    scale = (127.0 / np.maximum(np.abs(v).max(1), f4(1e-5)).astype(f8)).astype(f4)
    code = np.clip(np.rint(times(v, scale[:, None])), -128, 127).astype(f8)
    return (torch.from_numpy(h.astype(f8)), torch.from_numpy(code / scale[:, None].astype(f8)),
            torch.from_numpy(scale.astype(f8)), None)
