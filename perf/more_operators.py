"""Measured cases of the operators around a decode step of a ternary layer:

* ``place`` -- rotary positions of queries and keys, the keys and values appended to the
  4-bit cache in the same call (and read back);
* ``turn``  -- rotary positions of rows at given positions, forward or inverse;
* ``w4``    -- a matrix of 4-bit weights with a step for each group, times float tokens;
* ``weigh`` -- the attention weight that each cached token gets from a call's rows, added to
  what it had got before;
* ``evict`` -- the tokens of the largest weight, the first and the last ones, moved to new
  pages (and read back).

With ``own`` false the operators are computed in elementary torch operations,
with ``own`` true by this package's calls.
"""
import math

import numpy as np
import torch

own = False

PAGE = 64        # tokens of a cache page
GROUP = 64       # cached channels that share one (step, middle) pair
CLAMP = 57344.0  # what a cached value saturates at
W4MAX = 7 * 65504.0
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"fp32": 4, "bf16": 2}


# ---------------------------------------------------------------- cases

def _place(seqs, new, old, heads, kv_heads, dim, rot, dtype, offset=0, pairs="half", base=10000.0,
           factor=1.0, magnitude=1.0):
    return {"op": "place", "seqs": seqs, "new": new, "old": old, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "rot": rot, "dtype": dtype, "offset": offset,
            "pairs": pairs, "base": base, "factor": factor, "magnitude": magnitude}


def _turn(n, heads, dim, rot, dtype, far, pairs="half", inverse=False, base=10000.0, factor=1.0,
          magnitude=1.0):
    return {"op": "turn", "n": n, "heads": heads, "dim": dim, "rot": rot, "dtype": dtype,
            "far": far, "pairs": pairs, "inverse": inverse, "base": base, "factor": factor,
            "magnitude": magnitude}


def _w4(n, rows, k, group, dtype):
    return {"op": "w4", "n": n, "rows": rows, "k": k, "group": group, "dtype": dtype}


def _weigh(seqs, new, old, heads, kv_heads, dim, dtype, decay=1.0, window=0, sinks=0):
    return {"op": "weigh", "seqs": seqs, "new": new, "old": old, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "dtype": dtype, "decay": decay, "window": window,
            "sinks": sinks}


def _evict(seqs, held, keep, kv_heads, dim, sinks, recent):
    return {"op": "evict", "seqs": seqs, "new": 0, "old": held, "keep": keep,
            "kv_heads": kv_heads, "dim": dim, "sinks": sinks, "recent": recent}


def listed():
    return [
        # one decoded token of the 2B-class layer: latency
        dict(_place(1, 1, 514, 20, 5, 128, 128, "fp32"), name="place 1 token"),
        # prompts of three sequences, written into fresh pages, stretched positions
        dict(_place(3, 2731, 0, 16, 8, 128, 128, "bf16", base=500000.0, factor=4.0,
                    magnitude=1.1386), name="place prompt"),
        # a decode batch far into a context that was cut before: part of the head, neighbours paired
        dict(_turn(64, 32, 128, 64, "fp32", 1000000, "interleaved"), name="turn 64 tokens"),
        # the gradient of a long prompt's rotated queries, an odd head
        dict(_turn(8191, 32, 80, 80, "bf16", 8191, inverse=True), name="turn back"),
        # one token times a projection of the 2B-class layer: latency
        dict(_w4(1, 2560, 2560, 64, "fp32"), name="w4 1 token"),
        # one token's logits over a vocabulary
        dict(_w4(1, 128000, 2560, 64, "bf16"), name="w4 head"),
        # a small batch, an odd number of rows, small groups
        dict(_w4(5, 50001, 1024, 32, "fp32"), name="w4 5 tokens"),
        # the down projection of the large layer for a full decode batch
        dict(_w4(64, 8192, 28672, 128, "bf16"), name="w4 64 tokens"),
        # a decode batch of the large layer's heads, ragged histories
        dict(_weigh(64, 1, 4095, 64, 8, 128, "bf16", 0.97), name="weigh 64 tokens"),
        # the end of a long prompt, whose rows vote for what is kept, an odd count
        dict(_weigh(2, 131, 12000, 20, 5, 128, "fp32", 0.0, 4096, 4), name="weigh chunk"),
        # a decode batch cut back to its budget
        dict(_evict(16, 2176, 1024, 8, 128, 4, 256), name="evict 16 sequences"),
        # one very long history cut to a small part
        dict(_evict(1, 131072, 4096, 5, 128, 4, 512), name="evict long"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def _spin(rng, dim):
    """How positions are applied: channels, pairing, base, stretch, magnitude."""
    return dict(rot=rng.choice([dim, dim, dim // 2, dim // 4, 2 * rng.randint(1, dim // 2)]),
                dtype=rng.choice(["fp32", "bf16"]), pairs=rng.choice(["half", "interleaved"]),
                base=rng.choice([10000.0, 500000.0]), factor=rng.choice([1.0, 1.0, 4.0, 8.0]),
                magnitude=rng.choice([1.0, 1.0, 1.1386]))


def draw(rng):
    most = {"place": 1.26e8, "turn": 8.3e7, "w4": 6e8, "weigh": 9.7e7, "evict": 1.1e8}
    while True:
        op = rng.choice(["place", "turn", "w4", "w4", "weigh", "evict"])
        kv, dim = rng.choice([1, 2, 4, 5, 8]), rng.choice([64, 128, 128, 256])
        if op == "place":
            c = _place(_log(rng, 1, 64), rng.choice([1, _log(rng, 1, 4096)]),
                       rng.choice([0, _log(rng, 1, 4096)]), kv * rng.choice([1, 2, 4, 6, 8]), kv,
                       dim, offset=rng.choice([0, _log(rng, 1, 1000000)]), **_spin(rng, dim))
        elif op == "turn":
            dim = rng.choice([64, 80, 96, 128, 192, 256])
            c = _turn(_log(rng, 1, 16384), _log(rng, 1, 64), dim, far=_log(rng, 1000, 1000000),
                      inverse=rng.random() < 0.4, **_spin(rng, dim))
        elif op == "w4":
            c = _w4(rng.choice([1, _log(rng, 1, 64), _log(rng, 1, 300)]), _log(rng, 50, 128000),
                    128 * _log(rng, 2, 224), rng.choice([32, 64, 64, 128]),
                    rng.choice(["fp32", "bf16"]))
            if c["rows"] * c["k"] > 3.3e8:
                continue
        elif op == "weigh":
            c = _weigh(_log(rng, 1, 64), rng.choice([1, 1, _log(rng, 2, 1024)]), _log(rng, 1, 100000),
                       kv * rng.choice([1, 2, 4, 6, 8]), kv, dim, rng.choice(["fp32", "bf16"]),
                       rng.choice([0.0, 0.9, 1.0]))
            if rng.random() < 0.3:
                c["window"], c["sinks"] = _log(rng, 16, 8192), rng.choice([0, 1, 4, 64])
        else:
            held = _log(rng, 2, 131072)
            keep = _log(rng, 1, held)
            sinks = min(rng.choice([0, 1, 4, 64]), keep // 2)
            c = _evict(_log(rng, 1, 64), held, keep, kv, dim, sinks,
                       rng.choice([0, _log(rng, 1, keep), keep]) * (keep - sinks) // keep)
        # the scores of the plain form, and its whole histories in 32 bits, have to fit
        n, t = c.get("new", 0), c.get("new", 0) + c.get("old", 0)
        if op == "weigh" and (c["seqs"] * c["heads"] * n * t > 3e8 or c["seqs"] * kv * t * dim > 3e8):
            continue
        if op == "evict" and c["seqs"] * kv * t * dim > 3e8:
            continue
        if _cost(c) <= most[op]:
            return c


# ---------------------------------------------------------------- inputs

def _lengths(case):
    """Tokens that each sequence adds and holds already: the first sequence has the
    stated numbers, the others fewer (ragged), the same ones for every seed."""
    r = np.random.RandomState(case["seqs"])
    new = [case["new"]] + [max(min(1, case["new"]), int(case["new"] * r.uniform(0.3, 1)))
                           for _ in range(case["seqs"] - 1)]
    old = [case["old"]] + [int(case["old"] * r.uniform(0.2, 1)) for _ in range(case["seqs"] - 1)]
    return np.array(new), np.array(old)


def _kv(shape, g, dev):
    """Keys or values: near normal, a few channels many times as large (as keys have
    them) and a middle that differs between channels."""
    d = shape[-1]
    gain = 1 + 7 * (torch.rand(d, generator=g, device=dev) < 0.04).float()
    mid = 0.5 * torch.randn(d, generator=g, device=dev)
    return torch.randn(shape, generator=g, device=dev).mul_(gain).add_(mid)


def _turns(case, dev):
    """Turns per position of each pair, as 64-bit fractions of one: base^(-2 i / rot) radians,
    divided by the factor."""
    half = case["rot"] // 2
    f = [case["base"] ** (-2 * i / case["rot"]) / case["factor"] / (2 * math.pi) for i in range(half)]
    f = [int(x * 2.0 ** 64) for x in f]
    return torch.tensor([x - 2 ** 64 if x >= 2 ** 63 else x for x in f], dtype=torch.int64, device=dev)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    s = {"case": case}
    if case["op"] == "w4":
        n, m, k = case["n"], case["rows"], case["k"]
        gain = 1 + 15 * (torch.rand(k, generator=g, device=dev) < 0.005).float()
        s["x"] = (torch.randn((n, k), generator=g, device=dev) * gain).to(DTYPES[case["dtype"]])
        w = torch.randn((m, k), generator=g, device=dev)
        w.mul_(0.02 * torch.exp(0.3 * torch.randn((m, 1), generator=g, device=dev)))
        s["codes"], s["steps"] = _pack_w4(w, case["group"])
        return s
    if case["op"] in ("place", "turn"):
        s["turns"], dt = _turns(case, dev), DTYPES[case["dtype"]]
    if case["op"] == "turn":
        s["x"] = torch.randn((case["n"], case["heads"], case["dim"]), generator=g, device=dev).to(dt)
        s["at"] = torch.randint(0, case["far"], (case["n"],), generator=g, device=dev, dtype=torch.int32)
        return s
    new, old = _lengths(case)
    dim, kvh = case["dim"], case["kv_heads"]
    kv_len = new + old
    pages = np.maximum(-(-kv_len // PAGE), 1)
    fresh = np.minimum(kv_len, case["keep"]) if case["op"] == "evict" else 0 * kv_len
    fresh = -(-fresh // PAGE)
    total = int(pages.sum() + fresh.sum()) + 3
    perm = torch.randperm(total, generator=g, device=dev).cpu().numpy()

    def hand_out(count, at):
        t = np.full((case["seqs"], max(int(count.max()), 1)), -1, np.int32)
        for b, p in enumerate(count):
            t[b, :p] = perm[at:at + p]
            at += p
        return t

    put = lambda a: torch.from_numpy(np.asarray(a, np.int32)).to(dev)  # noqa: E731
    s["table"], s["kv_len"] = put(hand_out(pages, 0)), put(kv_len)
    s["q_start"] = put(np.concatenate([[0], np.cumsum(new)]))
    s["max_kv"], s["n"], s["max_new"] = int(kv_len.max()), int(new.sum()), int(new.max())
    # pages are handed out as they are: what no token was written to holds anything
    s["cache"] = torch.full((total, kvh, 72 * dim), 255, dtype=torch.uint8, device=dev)
    if case["op"] == "place":
        s["q"] = torch.randn((s["n"], case["heads"], dim), generator=g, device=dev).to(dt)
        s["k"], s["v"] = (_kv((s["n"], kvh, dim), g, dev).to(dt) for _ in range(2))
        s["offset"] = put(np.arange(case["seqs"]) + case["offset"])
        return s
    start = put(np.concatenate([[0], np.cumsum(kv_len)]))
    k, v = (_kv((int(kv_len.sum()), kvh, dim), g, dev) for _ in range(2))
    _write(s["cache"], *_where(s["table"], s["kv_len"], start, int(kv_len.sum())), k, v)
    # weights of many steps: few tokens have most of it, and some none at all
    w = 0.02 * torch.exp(2 * torch.randn((total, kvh, PAGE), generator=g, device=dev))
    s["weights"] = w * (torch.rand((total, kvh, PAGE), generator=g, device=dev) < 0.9)
    if case["op"] == "weigh":
        s["q"] = torch.randn((s["n"], case["heads"], dim), generator=g, device=dev).to(DTYPES[case["dtype"]])
        s["out"] = torch.zeros_like(s["weights"])
        return s
    s["new_table"] = put(hand_out(fresh, int(pages.sum())))
    keep = np.minimum(kv_len, case["keep"])
    s["read_start"], s["kept"] = put(np.concatenate([[0], np.cumsum(keep)])), int(keep.sum())
    return s


# ---------------------------------------------------------------- plain forms

def _where(table, kv_len, start, n):
    """Page and place in it of n tokens: token start[b] + i of sequence b is at position
    kv_len[b] - (start[b + 1] - start[b]) + i."""
    b, pos = _positions(kv_len, start, n)
    return table[b, pos // PAGE].long(), pos % PAGE


def _positions(kv_len, start, n):
    r = torch.arange(n, device=kv_len.device)
    b = torch.searchsorted(start[1:].contiguous(), r.to(start.dtype), right=True)
    return b, kv_len[b].long() - start[b + 1].long() + r


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


def _rotate(x, turns, at, c, back=False):
    """Rows x[n][heads][dim] turned to the positions at[n]; the angle of a far position is a
    64-bit fraction of a turn, so whole turns fall away exactly."""
    angle = (at.long()[:, None] * turns).double() * (2 * math.pi / 2.0 ** 64)
    cos = (angle.cos() * c["magnitude"]).float()[:, None]
    sin = (angle.sin() * (-c["magnitude"] if back else c["magnitude"])).float()[:, None]
    x = x.float()
    r = c["rot"]
    t, rest = x[..., :r], x[..., r:]
    if c["pairs"] == "half":
        a, b = t[..., :r // 2], t[..., r // 2:]
        t = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = t[..., ::2], t[..., 1::2]
        t = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([t, rest], -1).to(DTYPES[c["dtype"]])


def _plain_turn(s):
    c = s["case"]
    return _rotate(s["x"], s["turns"], s["at"], c, c["inverse"])


def _plain_place(s):
    c = s["case"]
    b, pos = _positions(s["kv_len"], s["q_start"], s["n"])
    at = pos + s["offset"][b]
    q, k = _rotate(s["q"], s["turns"], at, c), _rotate(s["k"], s["turns"], at, c)
    page, place = s["table"][b, pos // PAGE].long(), pos % PAGE
    _write(s["cache"], page, place, k, s["v"])
    k, v = _read(s["cache"], page, place)
    return q, k.to(q.dtype), v.to(q.dtype)


def _pack_w4(w, group):
    """w[m][k] -> codes [16 rows][128 channels][quad, row][four times 8 channels of 4 bits] and
    steps [16 rows][128 channels][group][row]; rows up to a multiple of 16 are zeros."""
    m, k = w.shape
    tiles = -(-m // 16)
    w = torch.nn.functional.pad(w.float().clamp(-W4MAX, W4MAX), (0, 0, 0, 16 * tiles - m))
    w = w.view(16 * tiles, k // group, group)
    lo, hi = w.amin(2, True), w.amax(2, True)
    step = torch.maximum(hi * np.float32(1 / 7).item(), lo * -0.125).half()
    inv = torch.where(step > 0, 1 / step.float(), torch.zeros_like(lo))
    code = ((w * inv).round().clamp(-8, 7) + 8).to(torch.uint8)
    code = code.view(tiles, 16, k // 128, 4, 4, 4, 2).permute(0, 2, 4, 1, 3, 5, 6)
    code = (code[..., 0] | code[..., 1] << 4).reshape(tiles, k // 128, 64, 16)
    return code, step.view(tiles, 16, k // 128, -1).permute(0, 2, 3, 1).contiguous()


def _plain_w4(s):
    c = s["case"]
    code = s["codes"].view(-1, c["k"] // 128, 4, 16, 4, 4).permute(0, 3, 1, 4, 2, 5)
    w = _nibbles(code).float().sub_(8).view(-1, c["k"] // c["group"], c["group"])
    w.mul_(s["steps"].permute(0, 3, 1, 2).float().reshape(w.shape[0], -1, 1))
    return torch.matmul(s["x"].float(), w.view(-1, c["k"])[:c["rows"]].t())


def _plain_weigh(s):
    c, dev = s["case"], s["q"].device
    seqs, heads, kvh, d = c["seqs"], c["heads"], c["kv_heads"], c["dim"]
    pages = s["table"].clamp(min=0).long()
    kc, _, km, _ = _parts(s["cache"][pages].flatten(0, 1))
    k = _key_rows(kc, km).unflatten(0, (seqs, -1)).transpose(1, 2).flatten(2, 3)
    t = k.shape[2]
    j = torch.arange(t, device=dev)
    held = j < s["kv_len"][:, None]                                    # [seqs][t]
    k = k.masked_fill(~held[:, None, :, None], 0.0)
    # queries padded to the longest continuation, the heads of a group side by side
    n = s["max_new"]
    i = torch.arange(n, device=dev)
    count = (s["q_start"][1:] - s["q_start"][:-1])[:, None]
    row = (s["q_start"][:-1, None] + i).clamp(max=s["n"] - 1).long()
    q = s["q"][row].float().unflatten(2, (kvh, heads // kvh)).permute(0, 2, 1, 3, 4)
    score = torch.matmul(q.reshape(seqs, kvh, -1, d), k.transpose(2, 3)) * (1 / math.sqrt(d))
    score = score.view(seqs, kvh, n, heads // kvh, t)
    pos = s["kv_len"][:, None] - count + i                             # [seqs][n]
    see = held[:, None] & (j <= pos[:, :, None]) & (i < count)[:, :, None]
    if c["window"]:
        see &= (j > pos[:, :, None] - c["window"]) | (j < c["sinks"])
    score.masked_fill_(~see[:, None, :, None], -math.inf)
    score -= score.amax(4, True).clamp(min=-3e38)
    score.exp_()
    score /= score.sum(4, True).clamp(min=1e-30)
    got = score.flatten(2, 3).sum(2)                                   # [seqs][kvh][t]
    old = s["weights"][pages].transpose(1, 2).flatten(2)               # [seqs][kvh][t]
    first = (s["kv_len"][:, None] - count)[:, None]
    got = got + torch.where(j < first, old * np.float32(c["decay"]).item(), torch.zeros_like(old))
    b, p = held.nonzero(as_tuple=True)
    s["out"][pages[b, p // PAGE], :, p % PAGE] = got[b, :, p]
    return s["out"]


def _plain_evict(s):
    c = s["case"]
    kvh, dev = c["kv_heads"], s["cache"].device
    pages = s["table"].clamp(min=0).long()
    w = s["weights"][pages].transpose(1, 2).flatten(2)                 # [seqs][kvh][t]
    j = torch.arange(w.shape[2], device=dev)
    held = s["kv_len"][:, None]
    rank = (j < held).int() + ((j < held) & ((j < c["sinks"]) | (j >= held - c["recent"]))).int()
    by = torch.sort(w, dim=2, descending=True, stable=True)[1]
    again = torch.sort(rank[:, None].expand_as(w).gather(2, by), dim=2, descending=True, stable=True)[1]
    by = by.gather(2, again)[:, :, :c["keep"]]                         # the best first
    new_len = s["kv_len"].clamp(max=c["keep"])
    inside = torch.arange(by.shape[2], device=dev) < new_len[:, None]
    by = torch.where(inside[:, None], by, torch.full_like(by, 1 << 40)).sort(2)[0]
    index = torch.full((c["seqs"], kvh, c["keep"]), -1, dtype=torch.int32, device=dev)
    index[:, :, :by.shape[2]] = torch.where(inside[:, None], by, torch.full_like(by, -1)).int()
    # moved as they are, head by head
    b, p = inside.nonzero(as_tuple=True)
    h = torch.arange(kvh, device=dev)[:, None]
    src = index[b, :, p].long().t()                                    # [kvh][n]
    sp, st = pages[b, src // PAGE], src % PAGE
    tp, tt = s["new_table"][b, p // PAGE].long()[None], (p % PAGE)[None]
    kc, vc, km, vm = _parts(s["cache"])
    kc[tp, h, tt] = kc[sp, h, st]
    km[tp, h, tt] = km[sp, h, st]
    vc[tp, h, tt // 4, :, :, tt % 4] = vc[sp, h, st // 4, :, :, st % 4]
    vm[tp, h, tt // 4, :, :, tt % 4] = vm[sp, h, st // 4, :, :, st % 4]
    s["weights"][tp, h, tt] = s["weights"][sp, h, st]
    k, v = _read(s["cache"], tp[0], tt[0])
    return new_len, index, k.bfloat16(), v.bfloat16(), s["weights"]


def run(s):
    c = s["case"]
    if own:
        return _own(s)
    return {"place": _plain_place, "turn": _plain_turn, "w4": _plain_w4, "weigh": _plain_weigh,
            "evict": _plain_evict}[c["op"]](s)


# ---------------------------------------------------------------- the package's calls

def _own(s):
    import ternary_weight_i2_amd as bn
    c = s["case"]
    if c["op"] == "w4":
        return bn.linear_w4(s["x"], bn.W4Matrix(s["codes"], s["steps"], c["rows"]))
    if c["op"] == "weigh":
        return bn.kv4_weigh(s["weights"], s["q"], s["cache"], s["table"], s["kv_len"], s["q_start"],
                            decay=c["decay"], window=c["window"], sinks=c["sinks"],
                            max_kv=s["max_kv"], out=s["out"])
    if c["op"] == "evict":
        new_len, index = bn.kv4_evict(s["cache"], s["weights"], s["table"], s["kv_len"], s["new_table"],
                                      c["keep"], sinks=c["sinks"], recent=c["recent"])
        k, v = bn.kv4_read(s["cache"], s["new_table"], new_len, s["read_start"], s["kept"],
                           dtype=torch.bfloat16)
        return new_len, index, k, v, s["weights"]
    plan = bn.Rotary(s["turns"], interleaved=c["pairs"] == "interleaved", magnitude=c["magnitude"])
    if c["op"] == "turn":
        return bn.rotary(s["x"], plan, s["at"], inverse=c["inverse"])
    q = bn.rotary_kv4_append(s["cache"], s["table"], s["kv_len"], s["q_start"], s["q"], s["k"], s["v"],
                             plan, offset=s["offset"])
    k, v = bn.kv4_read(s["cache"], s["table"], s["kv_len"], s["q_start"], s["n"], dtype=q.dtype)
    return q, k, v


# ---------------------------------------------------------------- work

def work(case):
    if case["op"] == "w4":
        n, m, k = case["n"], case["rows"], case["k"]
        return {"bytes": m * k // 2 + 2 * m * k // case["group"] + n * k * SIZE[case["dtype"]] + 4 * n * m,
                "flops": 2 * n * m * k}
    if case["op"] == "turn":
        values = case["n"] * case["heads"] * case["dim"]
        return {"bytes": 2 * values * SIZE[case["dtype"]], "flops": 3 * values}
    new, old = _lengths(case)
    n, dim, kvh = int(new.sum()), case["dim"], case["kv_heads"]
    token = kvh * dim * 9 // 8          # one token's keys and values with their pairs
    if case["op"] == "place":
        size = SIZE[case["dtype"]]
        q, kv = n * case["heads"] * dim, n * 2 * kvh * dim
        return {"bytes": 2 * q * size + 2 * kv * size + 2 * n * token, "flops": 3 * q + 12 * kv}
    if case["op"] == "evict":
        held, kept = int(old.sum()), int(np.minimum(old, case["keep"]).sum())
        # weights looked at; tokens, weights and indices moved; values read back
        return {"bytes": 4 * held * kvh + kept * (3 * token + 12 * kvh + 4 * kvh * dim),
                "flops": held * kvh + 4 * kept * kvh * dim}
    pairs = seen = 0
    for a, o in zip(new.tolist(), old.tolist()):
        pos = np.arange(o, o + a)
        low = np.zeros_like(pos)
        if case["window"]:
            low = np.maximum(0, pos - case["window"] + 1)
        pairs += int((pos + 1 - low + np.minimum(low, case["sinks"])).sum())
        seen += int(o + a - low[0] + min(low[0], case["sinks"]))
    held = int((new + old).sum())
    return {"bytes": seen * token // 2 + (8 if case["decay"] else 4) * held * kvh
            + n * case["heads"] * dim * SIZE[case["dtype"]],
            "flops": 2 * dim * case["heads"] * pairs}


# ---------------------------------------------------------------- from the definitions, in 64 bits

def _exact_kv(cache, page, place, head, keys):
    """Keys (or values) of tokens, from the places of their nibbles in a record: binary64."""
    d = cache.shape[2] // 72
    c = torch.arange(d, device=cache.device)
    rec = cache[page, head]
    if keys:
        at = place[:, None] * (d // 2) + ((c % 32 // 8) * (d // 32) + c // 32) * 4 + c % 8 // 2
        pair = 64 * d + (place[:, None] * (d // 64) + c // 64) * 4
        step, mid = pair, pair + 2
    else:
        lane = ((place[:, None] // 4 * 16 + c % 64 // 4) * (d // 64) + c // 64) * 4 + place[:, None] % 4
        at = 32 * d + 2 * lane + c % 4 // 2
        pair = 68 * d + (place[:, None] // 4 * (d // 64) + c // 64) * 16 + place[:, None] % 4 * 2
        step, mid = pair, pair + 8
    half = lambda p: torch.stack([rec.gather(1, p), rec.gather(1, p + 1)], -1).view(torch.float16)[..., 0].double()  # noqa: E731,E501
    code = rec.gather(1, at) >> (4 * (c % 2)).to(torch.uint8) & 15
    return half(mid) + half(step) * (code.double() - 8)


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


def _exact_turn(x, turns, at, c, sign, exactly):
    """The rotation as a product of complex numbers in binary64; `exactly`: with the
    roundings to 32 bits that the definition gives the factors, the products and the sums."""
    angle = np.longdouble(2 * np.pi) * ((at.astype(np.uint64)[:, None] * turns.view(np.uint64)).astype(np.longdouble) / np.longdouble(2.0) ** 64)
    cos, sin = (c["magnitude"] * f(angle.astype(np.float64)) for f in (np.cos, np.sin))
    low = (lambda a: a.astype(np.float32).astype(np.float64)) if exactly else (lambda a: a)
    cos, sin = low(cos)[:, None], low(sign * sin)[:, None]
    out = x.astype(np.float64).copy()
    r = c["rot"]
    a, b = (slice(0, r // 2), slice(r // 2, r)) if c["pairs"] == "half" else (slice(0, r, 2), slice(1, r, 2))
    re, im = out[..., a].copy(), out[..., b].copy()
    out[..., a] = low(low(re * cos) - low(im * sin))
    out[..., b] = low(low(im * cos) + low(re * sin))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    host = lambda t: t.float().cpu().numpy()  # noqa: E731
    if case["op"] == "w4":
        m, k, g = case["rows"], case["k"], case["group"]
        c = torch.arange(k, device="cuda")
        x, outs = s["x"].double(), []
        for t in range(0, s["codes"].shape[0], 256):
            words = s["codes"][t:t + 256].view(-1, k // 128, 4, 16, 16)     # [.][.][quad][row][byte]
            byte = c % 128 // 32 * 4 + c % 8 // 2
            code = words[:, c // 128, c % 32 // 8, :, byte].permute(1, 2, 0)  # [tile][row][k]
            code = (code >> (4 * (c % 2)).to(torch.uint8) & 15).double() - 8
            step = s["steps"][t:t + 256][:, c // 128, c % 128 // g].transpose(1, 2).double()
            outs.append(x @ (code * step).flatten(0, 1).t().contiguous())
        return torch.cat(outs, 1)[:, :m]
    if case["op"] == "turn":
        at = s["at"].cpu().numpy().astype(np.int64)
        return torch.from_numpy(_exact_turn(host(s["x"]), s["turns"].cpu().numpy(), at, case,
                                            -1 if case["inverse"] else 1, False))
    new, old = _lengths(case)
    if case["op"] == "place":
        at = np.concatenate([np.arange(o, o + n) + case["offset"] + b
                             for b, (n, o) in enumerate(zip(new.tolist(), old.tolist()))])
        turns = s["turns"].cpu().numpy()
        q = _exact_turn(host(s["q"]), turns, at, case, 1, False)
        k = _exact_turn(host(s["k"]), turns, at, case, 1, True)
        k = torch.from_numpy(k.astype(np.float32)).to(s["k"].dtype).float().numpy()
        return [torch.from_numpy(o) for o in (q, _exact_cached(k), _exact_cached(host(s["v"])))]
    if case["op"] == "evict":
        return _exact_evict(case, s, old)
    out, at = s["out"].double(), 0
    for b in range(case["seqs"]):
        n, t = int(new[b]), int(new[b] + old[b])
        p = torch.arange(t, device="cuda")
        page, place = s["table"][b, p // PAGE].long(), p % PAGE
        pos = torch.arange(t - n, t, device="cuda")[:, None]
        hide = p > pos
        if case["window"]:
            hide = hide | ((p <= pos - case["window"]) & (p >= case["sinks"]))
        per = case["heads"] // case["kv_heads"]
        for h in range(case["kv_heads"]):
            k = _exact_kv(s["cache"], page, place, h, True)
            q = s["q"][at:at + n, h * per:(h + 1) * per].double().transpose(0, 1)
            w = torch.matmul(q, k.t().contiguous()) / math.sqrt(case["dim"])
            w = torch.softmax(w.masked_fill(hide, -math.inf), 2).sum((0, 1))
            past = s["weights"][page, h, place].double() * float(np.float32(case["decay"]))
            out[page, h, place] = w + torch.where(p < t - n, past, torch.zeros_like(past))
        at += n
    return out


def _exact_evict(case, s, held):
    """Only moves: which tokens, by numpy's own order, and what they stand for."""
    table, new_table = (s[x].cpu().numpy() for x in ("table", "new_table"))
    weights, kvh = s["weights"].cpu().numpy(), case["kv_heads"]
    w = weights.astype(np.float64)
    ks, vs = [], []
    for b in range(case["seqs"]):
        t, keep = int(held[b]), min(int(held[b]), case["keep"])
        p = np.arange(t)
        heads = [[], []]
        for h in range(kvh):
            mine = weights[table[b, p // PAGE], h, p % PAGE]
            spared = (p < case["sinks"]) | (p >= t - case["recent"])
            kept = np.sort(np.lexsort((p, -mine, ~spared))[:keep])
            d = np.arange(keep)
            w[new_table[b, d // PAGE], h, d % PAGE] = mine[kept]
            page, place = (torch.from_numpy(x.astype(np.int64)).cuda()
                           for x in (table[b, kept // PAGE], kept % PAGE))
            for o, keys in zip(heads, (True, False)):
                o.append(_exact_kv(s["cache"], page, place, h, keys))
        ks.append(torch.stack(heads[0], 1))
        vs.append(torch.stack(heads[1], 1))
    return None, None, torch.cat(ks), torch.cat(vs), torch.from_numpy(w)
