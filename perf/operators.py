"""The attention-side operators of the EXL3 layer library, as a user's program calls them.

Four operators around the quantised linear layers, on the packed tokens of a batch of sequences:

rope    rotary positions on the heads of a fused projection's output
cache   keys and values written into a paged cache (rotary positions applied on the way, 8- and 4-bit
        formats quantised) and read back
prompt  causal attention over whole prompts of different lengths, packed one after the other
paged   attention of new tokens (one, a few, or a chunk) over a paged cache

``own`` false computes the plain form in 32-bit torch; ``own`` true calls the library.  ``exact``
computes the same from the definition in 64 bits.

The formats.  A frequency is a phase, in turns of 2^64, that one position adds; a position's angle is
position * phase modulo 2^64.  The quantised formats hold, for each token and head, the Hadamard transform of the
head's vector times 2^-3 as offset codes (code + 128 in a byte, code + 8 in a nibble, low nibble first)
and one bfloat16 scale.
"""
import functools
import math

import numpy as np
import torch

own = False

_TURN = math.pi / 2.0**31  # radians of one unit of a phase's upper 32 bits
_BIAS = {"int8": 128, "int4": 8}
_TOP = {"int8": 127.0, "int4": 7.0}


def _dt(name):
    return {"bf16": torch.bfloat16, "f16": torch.float16}[name]


def _ints(text):
    return [int(v) for v in text.split(",")]


# --------------------------------------------------------------------------------------------------
# cases


def listed():
    return [
        # one decode step's q and k heads, batch of 37, whole head rotated
        dict(name="rope_step", op="rope", tokens=37, heads=40, skip=8, dim=128, rot=128, layout="half", dtype="bf16",
             long=False),
        # a prompt of 8191 tokens, half of each head, interleaved pairs, frequencies stretched for long contexts
        dict(name="rope_prompt", op="rope", tokens=8191, heads=48, skip=8, dim=128, rot=64, layout="interleaved",
             dtype="bf16", long=True),
        # a decode step of 61 sequences: rotary q and k, 8-bit write, and the new rows read back
        dict(name="cache_step_int8", op="cache", tokens=61, heads=32, kv=8, dim=128, rot=128, layout="half",
             dtype="bf16", fmt="int8", page=16, long=False),
        # a long prompt's keys and values into the 4-bit cache
        dict(name="cache_prompt_int4", op="cache", tokens=16381, heads=32, kv=8, dim=128, rot=128, layout="half",
             dtype="bf16", fmt="int4", page=64, long=True),
        # a handful of short prompts, small heads
        dict(name="prompt_short", op="prompt", lens="1,17,200,63,128", heads=16, kv=4, dim=64, window=0, dtype="f16"),
        # a packed batch of prompts of ordinary lengths, five query heads a key head
        dict(name="prompt_packed", op="prompt", lens="2011,640,77,1500,1,333,1024,2048,129,911", heads=40, kv=8,
             dim=128, window=0, dtype="bf16"),
        # one long document
        dict(name="prompt_long", op="prompt", lens="16384", heads=32, kv=8, dim=128, window=0, dtype="bf16"),
        # one user, one token, 16-bit cache
        dict(name="paged_one", op="paged", q_lens="1", kv_lens="4097", heads=32, kv=8, dim=128, page=16, fmt="bf16",
             window=0, dtype="bf16"),
        # a serving batch of single tokens at ragged lengths, 8-bit cache (one slot of the batch is empty)
        dict(name="paged_batch_int8", op="paged", q_lens=",".join(["1"] * 48),
             kv_lens="0," + ",".join(str(257 + (i * 7919) % 14000) for i in range(46)) + ",16384", heads=32, kv=8,
             dim=128, page=64, fmt="int8", window=0, dtype="bf16"),
        # drafted tokens checked together, 4-bit cache, long contexts
        dict(name="paged_draft_int4", op="paged", q_lens="3,4,1,2,4,4,3,1", kv_lens="32768,30011,9000,27777,32001,16000,"
             "25000,31234", heads=32, kv=8, dim=128, page=32, fmt="int4", window=0, dtype="f16"),
        # a chunk of a long prompt over what is already cached
        dict(name="paged_chunk", op="paged", q_lens="512", kv_lens="32768", heads=32, kv=8, dim=128, page=64,
             fmt="bf16", window=0, dtype="bf16"),
        # chunks and single tokens together over the 8-bit cache, sliding window
        dict(name="paged_mixed_int8", op="paged", q_lens="300,1,129,1,1,700", kv_lens="9000,8111,129,1,15000,6001",
             heads=96, kv=8, dim=128, page=32, fmt="int8", window=4096, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    v = max(lo, min(hi, v))
    return v + 1 if v == 3072 else v


def draw(rng):
    op = rng.choice(["rope", "cache", "prompt", "prompt", "paged", "paged", "paged"])
    dtype = rng.choice(["bf16", "f16"])
    dim = rng.choice([64, 128, 128])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 12])
    heads = min(96, kv * group)
    heads -= heads % kv
    if op == "rope":
        rot = rng.choice([dim, dim, dim // 2, dim // 4])
        return dict(op=op, tokens=_log(rng, 1, 8192), heads=heads + kv, skip=kv, dim=dim, rot=rot,
                    layout=rng.choice(["half", "interleaved"]), dtype=dtype, long=rng.random() < 0.5)
    if op == "cache":
        return dict(op=op, tokens=_log(rng, 1, 16384), heads=min(32, heads) // kv * kv, kv=kv, dim=dim,
                    rot=rng.choice([dim, dim // 2]), layout=rng.choice(["half", "interleaved"]), dtype=dtype,
                    fmt=rng.choice(["int8", "int4", dtype]), page=rng.choice([16, 32, 64, 128, 256]),
                    long=rng.random() < 0.5)
    if op == "prompt":
        if rng.random() < 0.4:
            lens = [_log(rng, 1, 8192)]
        else:
            lens = [_log(rng, 1, 2048) for _ in range(rng.randint(2, 10))]
        return dict(op=op, lens=",".join(map(str, lens)), heads=min(heads, 32) // kv * kv, kv=kv, dim=dim,
                    window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]), dtype=dtype)
    kind = rng.choice(["one", "draft", "chunk"])
    if kind == "chunk":
        heads = min(heads, 32) // kv * kv
        q_lens = [_log(rng, 1, 700) for _ in range(rng.randint(1, 4))]
        kv_lens = [q + _log(rng, 1, 16000) for q in q_lens]
    else:
        q_lens = [1 if kind == "one" else rng.randint(1, 5) for _ in range(_log(rng, 1, 32))]
        kv_lens = [_log(rng, 1, 16384) for _ in q_lens]
    return dict(op=op, q_lens=",".join(map(str, q_lens)), kv_lens=",".join(map(str, kv_lens)), heads=heads, kv=kv,
                dim=dim, page=rng.choice([16, 32, 64, 128, 256]), fmt=rng.choice(["int8", "int4", dtype]),
                window=rng.choice([0, 0, 0, _log(rng, 16, 4096)]), dtype=dtype)


# --------------------------------------------------------------------------------------------------
# what a program has in hand


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _phases(rot, long):
    """Turns a position, as 64-bit fixed point; `long` stretches the slow half of the frequencies by 8."""
    f = 10000.0 ** (-2.0 * np.arange(rot // 2) / rot)
    if long:
        f = np.where(f * 4096 / (2 * math.pi) < 4.0, f / 8.0, f)
    turns = f / (2 * math.pi)
    return torch.tensor([int(t * 2.0**64) - (2**64 if t >= 0.5 else 0) for t in turns], dtype=torch.int64,
                        device="cuda")


def _offsets(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def _mixed(g, shape, dtype, channels):
    """Activations of a projection: normal, with a few channels that stand out as those of keys do."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    loud = torch.rand((channels,), generator=g, device="cuda") < 0.02
    return (x * torch.where(loud, 5.0, 1.0)).to(dtype)


def prepare(case, seed):
    g = _gen(seed)
    dev = "cuda"
    op, d, dtype = case["op"], case["dim"], _dt(case["dtype"])
    s = dict(case=case, dtype=dtype)
    if op in ("rope", "cache"):
        t = case["tokens"]
        rows = case["heads"] + (case["skip"] if op == "rope" else 2 * case["kv"])
        # a projection's fused output; the operators take views of it
        s["qkv"] = _mixed(g, (t, rows * d), dtype, rows * d).view(t, rows, d)
        top = 131072 if case["long"] else 8192
        start = int(torch.randint(0, max(1, top - t), (1,), generator=g, device=dev))
        if t > 256:  # a prompt's consecutive positions
            s["positions"] = torch.arange(start, start + t, dtype=torch.int32, device=dev)
        else:  # a batch's own positions
            s["positions"] = torch.randint(0, top, (t,), generator=g, device=dev, dtype=torch.int32)
        s["phases"] = _phases(case["rot"], case["long"])
        s["amplitude"] = 1.0 + 0.1 * math.log(8.0) if case["long"] else 1.0
    if op == "cache":
        pages = (t + case["page"] - 1) // case["page"] + 3
        s.update(_cache(g, case, pages))
        s["slots"] = torch.randperm(pages * case["page"], generator=g, device=dev)[:t]
        if t > 256:  # a prompt's tokens fill pages in order, the pages lie anywhere
            at = torch.arange(t, device=dev)
            order = torch.randperm(pages, generator=g, device=dev)
            s["slots"] = order[at // case["page"]] * case["page"] + at % case["page"]
    if op == "prompt":
        lens = _ints(case["lens"])
        h, kv = case["heads"], case["kv"]
        x = _mixed(g, (sum(lens), (h + 2 * kv) * d), dtype, (h + 2 * kv) * d).view(sum(lens), h + 2 * kv, d)
        s["q"], s["k"], s["v"] = x[:, :h], x[:, h:h + kv], x[:, h + kv:]
        s["cu"] = _offsets(lens)
        s["max_len"] = max(lens)
    if op == "paged":
        q_lens, kv_lens = _ints(case["q_lens"]), _ints(case["kv_lens"])
        s["q"] = _mixed(g, (sum(q_lens), case["heads"] * d), dtype, case["heads"] * d).view(-1, case["heads"], d)
        need = [(n + case["page"] - 1) // case["page"] for n in kv_lens]
        pages = sum(need) + 5
        s.update(_cache(g, case, pages))
        order = torch.randperm(pages, generator=g, device=dev).to(torch.int32).cpu().numpy()
        table = np.full((len(need), max(1, max(need)) + 1), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        s["table"] = torch.tensor(table, device=dev)
        s["cu"] = _offsets(q_lens)
        s["kv_lens"] = torch.tensor(kv_lens, dtype=torch.int32, device=dev)
        s["max_q"], s["max_kv"] = max(q_lens), max(kv_lens)
    return s


def _cache(g, case, pages):
    """A cache in use: every page holds some sequence's rows."""
    kv, d, ps, fmt = case["kv"], case["dim"], case["page"], case["fmt"]
    out = {"page": ps}
    for name in ("k", "v"):
        if fmt in ("bf16", "f16"):
            out["cache_" + name] = torch.randn((pages, kv, ps, d), generator=g, device="cuda",
                                               dtype=torch.float32).to(_dt(fmt))
            out[name + "_scale"] = None
            continue
        width = d if fmt == "int8" else d // 2
        # codes of rotated vectors are close to normal, the largest of a row at the top code
        if fmt == "int8":
            c = torch.randn((pages, kv, ps, width), generator=g, device="cuda") * 46.0
            codes = (c.round().clamp(-127, 127) + 128).to(torch.uint8)
        else:
            c = torch.randn((pages, kv, ps, width, 2), generator=g, device="cuda") * 2.6
            c = (c.round().clamp(-7, 7) + 8).to(torch.uint8)
            codes = c[..., 0] | (c[..., 1] << 4)
        out["cache_" + name] = codes
        size = 1.4 / (46.0 if fmt == "int8" else 2.6)
        out[name + "_scale"] = ((0.7 + 0.6 * torch.rand((pages, kv, ps), generator=g, device="cuda")) * size).to(
            torch.bfloat16)
    return out


# --------------------------------------------------------------------------------------------------
# one pass


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import exl3_trellis_quantized_gb300 as E

    case = s["case"]
    op = case["op"]
    if op == "rope":
        return E.rope(s["qkv"][:, :case["heads"]], s["positions"], s["phases"], layout=case["layout"],
                      amplitude=s["amplitude"])
    if op == "prompt":
        return E.attention_prompt(s["q"], s["k"], s["v"], s["cu"], s["max_len"], window=case["window"])
    cache = E.KVCache(s["cache_k"], s["cache_v"], s["k_scale"], s["v_scale"], case["fmt"])
    if op == "cache":
        h, kv = case["heads"], case["kv"]
        x = s["qkv"]
        q = E.kv_write(cache, x[:, h:h + kv], x[:, h + kv:], s["slots"], q=x[:, :h], positions=s["positions"],
                       phases=s["phases"], layout=case["layout"], amplitude=s["amplitude"])
        k, v = E.kv_read(cache, s["slots"], dtype=s["dtype"])
        return q, k, v
    return E.attention_paged(s["q"], cache, s["table"], s["cu"], s["kv_lens"], s["max_q"], s["max_kv"],
                             window=case["window"])


def _rotate(x, positions, phases, layout, amplitude):
    """x [T, H, D] in 32 bits, its first 2 * len(phases) values of each head rotated."""
    angle = ((positions.long()[:, None] * phases[None, :]) >> 32).float() * _TURN
    c, n = (torch.cos(angle) * amplitude)[:, None], (torch.sin(angle) * amplitude)[:, None]
    half = phases.numel()
    if layout == "half":
        a, b, rest = x[..., :half], x[..., half:2 * half], x[..., 2 * half:]
        return torch.cat([a * c - b * n, b * c + a * n, rest], -1)
    a, b, rest = x[..., 0:2 * half:2], x[..., 1:2 * half:2], x[..., 2 * half:]
    pairs = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    return torch.cat([pairs, rest], -1)


def _stage(x, stride):
    p = x.unflatten(-1, (-1, 2, stride))
    return torch.stack([p[..., 0, :] + p[..., 1, :], p[..., 0, :] - p[..., 1, :]], -2).flatten(-3)


def _hadamard(x):
    """The Hadamard transform of the last axis, not normalised: adds and subtracts in strides 1, 2, 4 and up."""
    return functools.reduce(_stage, [1 << i for i in range(x.shape[-1].bit_length() - 1)], x)


def _quantise(x, fmt):
    """(codes, scale) of rows x [..., D] in 32 bits."""
    y = _hadamard(x) * 0.125
    top = y.abs().amax(-1, keepdim=True)
    up = ((top / _TOP[fmt]).view(torch.int32) + 0xFFFF) & ~0xFFFF
    scale = up.view(torch.float32).clamp_min(2.0**-100)
    scale = torch.where(top == 0, 1.0, scale)
    codes = torch.round(y * (1.0 / scale)).clamp(-_TOP[fmt], _TOP[fmt])
    return codes, scale


def _store(codes, fmt):
    c = (codes + _BIAS[fmt]).to(torch.uint8)
    return c if fmt == "int8" else c[..., 0::2] | (c[..., 1::2] << 4)


def _load(stored, fmt):
    if fmt == "int8":
        return stored.float() - 128.0
    return torch.stack([stored & 15, stored >> 4], -1).flatten(-2).float() - 8.0


def _plain(s):
    case = s["case"]
    return {"rope": _plain_rope, "cache": _plain_cache, "prompt": _plain_prompt, "paged": _plain_paged}[case["op"]](s)


def _plain_rope(s):
    case = s["case"]
    x = s["qkv"][:, :case["heads"]].float()
    return _rotate(x, s["positions"], s["phases"], case["layout"], s["amplitude"]).to(s["dtype"])


def _plain_cache(s):
    case = s["case"]
    h, kv, d, fmt, ps = case["heads"], case["kv"], case["dim"], case["fmt"], case["page"]
    x = s["qkv"].float()
    turned = _rotate(x[:, :h + kv], s["positions"], s["phases"], case["layout"], s["amplitude"]).to(s["dtype"])
    page, at = s["slots"] // ps, s["slots"] % ps
    if fmt in ("bf16", "f16"):
        s["cache_k"][page, :, at] = turned[:, h:]
        s["cache_v"][page, :, at] = x[:, h + kv:].to(s["dtype"])
        return turned[:, :h], s["cache_k"][page, :, at], s["cache_v"][page, :, at]
    ck, sk = _quantise(turned[:, h:].float(), fmt)
    cv, sv = _quantise(x[:, h + kv:], fmt)
    s["cache_k"][page, :, at] = _store(ck, fmt)
    s["cache_v"][page, :, at] = _store(cv, fmt)
    s["k_scale"][page, :, at] = sk[..., 0].to(torch.bfloat16)
    s["v_scale"][page, :, at] = sv[..., 0].to(torch.bfloat16)
    back = 8.0 / d
    k = _hadamard(_load(s["cache_k"][page, :, at], fmt)) * (s["k_scale"][page, :, at].float()[..., None] * back)
    v = _hadamard(_load(s["cache_v"][page, :, at], fmt)) * (s["v_scale"][page, :, at].float()[..., None] * back)
    return turned[:, :h], k.to(s["dtype"]), v.to(s["dtype"])


def _attend(q, k, v, seen):
    """q [B, KV, G, Lq, D], k and v [B, KV, Lk, D], seen [B, 1, Lq, Lk]: softmax attention, zeros where nothing is seen."""
    b, kv, g, lq, d = q.shape
    p = torch.matmul(q.reshape(b, kv, g * lq, d) * d**-0.5, k.transpose(-1, -2)).view(b, kv, g, lq, -1)
    p.masked_fill_(~seen[:, None], -math.inf)
    top = p.amax(-1, keepdim=True)
    p.sub_(top.masked_fill_(top == -math.inf, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(b, kv, g * lq, -1), v).view(b, kv, g, lq, d)
    return o / total.masked_fill_(total == 0, 1.0)


def _grid(lens, most, total):
    """[B, most] packed indices of the sequences' tokens, and which of them exist."""
    at = torch.arange(most, device=lens.device)
    there = at[None, :] < (lens[1:] - lens[:-1])[:, None]
    return (lens[:-1, None] + at[None, :]).clamp(0, max(0, total - 1)).long(), there


def _sight(pos, there, keys, lens, window):
    """[B, 1, Lq, Lk]: key j is seen from position p if j <= p, j < the sequence's length and, with a window, j > p - window."""
    j = torch.arange(keys, device=pos.device)[None, None, :]
    seen = (j <= pos[..., None]) & (j < lens[:, None, None]) & there[..., None]
    return (seen & (j > pos[..., None] - window) if window else seen)[:, None]


def _plain_prompt(s):
    case = s["case"]
    h, kv, d = case["heads"], case["kv"], case["dim"]
    total = s["q"].shape[0]
    idx, there = _grid(s["cu"], s["max_len"], total)
    q = s["q"].float()[idx].view(*idx.shape, kv, h // kv, d).permute(0, 2, 3, 1, 4)
    k, v = (s[n].float()[idx].transpose(1, 2) for n in ("k", "v"))
    pos = torch.arange(s["max_len"], device=idx.device)[None, :].expand(idx.shape)
    o = _attend(q, k, v, _sight(pos, there, s["max_len"], s["cu"][1:] - s["cu"][:-1], case["window"]))
    return o.permute(0, 3, 1, 2, 4).reshape(*idx.shape, h, d)[there].to(s["dtype"])


def _rows(s, name):
    """A cache side's rows by sequence, [B, KV, Lk, D] in 32 bits (in the rotated basis for the quantised formats)."""
    case = s["case"]
    most = (s["max_kv"] + case["page"] - 1) // case["page"]
    table = s["table"][:, :max(1, most)].clamp_min(0).long()
    c = s["cache_" + name][table]
    x = c.float() if s[name + "_scale"] is None else _load(c, case["fmt"])
    if s[name + "_scale"] is not None:
        x = x * s[name + "_scale"][table].float()[..., None]
    return x.transpose(1, 2).flatten(2, 3)


def _plain_paged(s):
    case = s["case"]
    h, kv, d = case["heads"], case["kv"], case["dim"]
    idx, there = _grid(s["cu"], s["max_q"], s["q"].shape[0])
    q = s["q"].float()[idx]
    turned = s["k_scale"] is not None
    if turned:
        q = _hadamard(q) * (8.0 / d)
    q = q.view(*idx.shape, kv, h // kv, d).permute(0, 2, 3, 1, 4)
    k, v = _rows(s, "k"), _rows(s, "v")
    first = s["kv_lens"] - (s["cu"][1:] - s["cu"][:-1])
    pos = first[:, None] + torch.arange(s["max_q"], device=idx.device)[None, :]
    o = _attend(q, k, v, _sight(pos, there, k.shape[2], s["kv_lens"], case["window"]))
    if turned:
        o = _hadamard(o) * (8.0 / d)
    return o.permute(0, 3, 1, 2, 4).reshape(*idx.shape, h, d)[there].to(s["dtype"])


# --------------------------------------------------------------------------------------------------
# what a pass cannot do without


def _pairs(q_len, kv_len, window):
    """Query-key pairs of one sequence's head."""
    n = 0
    first = kv_len - q_len
    pos = np.arange(max(0, first), kv_len, dtype=np.int64)
    low = np.maximum(0, pos - window + 1) if window else np.zeros_like(pos)
    n = int((pos + 1 - low).sum())
    return n, (int(kv_len - low.min()) if pos.size else 0)


def _row_bytes(case):
    """Bytes of one cached row of one head, key or value."""
    return {"bf16": 2 * case["dim"], "f16": 2 * case["dim"], "int8": case["dim"] + 2,
            "int4": case["dim"] // 2 + 2}[case["fmt"]]


def work(case):
    op, d = case["op"], case["dim"]
    if op == "rope":
        n = case["tokens"] * case["heads"]
        return {"bytes": n * d * 4 + case["tokens"] * 4, "flops": n * case["rot"] * 3}
    if op == "cache":
        t, h, kv = case["tokens"], case["heads"], case["kv"]
        turn = d.bit_length() - 1 if case["fmt"].startswith("int") else 0
        moved = t * (h * d * 4 + 2 * kv * (2 * d + 2 * _row_bytes(case) + 2 * d) + 4 + 16)
        return {"bytes": moved, "flops": t * ((h + kv) * case["rot"] * 3 + 2 * kv * d * (2 * turn + 3))}
    if op == "prompt":
        lens = _ints(case["lens"])
        pairs = sum(_pairs(n, n, case["window"])[0] for n in lens)
        return {"bytes": sum(lens) * (2 * case["heads"] + 2 * case["kv"]) * d * 2,
                "flops": 4 * d * case["heads"] * pairs}
    q_lens, kv_lens = _ints(case["q_lens"]), _ints(case["kv_lens"])
    both = [_pairs(q, n, case["window"]) for q, n in zip(q_lens, kv_lens)]
    return {"bytes": sum(q_lens) * case["heads"] * d * 4 + sum(b for _, b in both) * case["kv"] * 2 * _row_bytes(case),
            "flops": 4 * d * case["heads"] * sum(a for a, _ in both)}


# --------------------------------------------------------------------------------------------------
# the definition, in 64 bits


def _h64(d):
    i = np.arange(d)
    bits = np.zeros((d, d), dtype=np.int64)
    a = i[:, None] & i[None, :]
    while a.any():
        bits += a & 1
        a = a >> 1
    return torch.tensor(1.0 - 2.0 * (bits & 1), dtype=torch.float64, device="cuda")


def _turn64(x, s):
    """Rotation of x [T, H, D] (64 bits) as a product of complex numbers."""
    case = s["case"]
    r = case["rot"]
    turns = torch.tensor([[int(p) * int(f) % 2**64 / 2.0**64 for f in s["phases"].tolist()]
                          for p in s["positions"].tolist()], dtype=torch.float64, device="cuda")
    w = torch.polar(torch.full_like(turns, s["amplitude"]), 2 * math.pi * turns)[:, None]
    y = x.clone()
    if case["layout"] == "half":
        z = torch.complex(x[..., :r // 2], x[..., r // 2:r]) * w
        y[..., :r // 2], y[..., r // 2:r] = z.real, z.imag
    else:
        z = torch.complex(x[..., 0:r:2].contiguous(), x[..., 1:r:2].contiguous()) * w
        y[..., 0:r:2], y[..., 1:r:2] = z.real, z.imag
    return y


def _one64(q, k, v, first, window):
    """One sequence: q [Lq, H, D], k and v [Lk, KV, D] in 64 bits; query i stands at position first + i."""
    lq, h, d = q.shape
    lk, kv, _ = k.shape
    out = torch.zeros_like(q)
    if lk == 0:
        return out
    pos = first + torch.arange(lq, device=q.device)
    j = torch.arange(lk, device=q.device)
    for head in range(h):
        for a in range(0, lq, 4096):
            p = pos[a:a + 4096, None]
            bad = j[None, :] > p
            if window:
                bad |= j[None, :] <= p - window
            x = (q[a:a + 4096, head] @ k[:, head * kv // h].T) / math.sqrt(d)
            w = torch.softmax(x.masked_fill(bad, -math.inf), -1)
            out[a:a + 4096, head] = torch.where(bad.all(-1, keepdim=True), 0.0, torch.nan_to_num(w)) @ v[:, head * kv // h]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op, d = case["op"], case["dim"]
    if op == "rope":
        if case["tokens"] * case["rot"] > 2_000_000:
            return None
        return _turn64(s["qkv"][:, :case["heads"]].double(), s)
    if op == "cache":
        if case["tokens"] * case["rot"] > 4_000_000:
            return None
        h, kv = case["heads"], case["kv"]
        q = _turn64(s["qkv"][:, :h].double(), s)
        if case["fmt"] not in _TOP:  # the key held is the rotated one in its own type
            return q, _turn64(s["qkv"][:, h:h + kv].double(), s), s["qkv"][:, h + kv:].double()
        # a quantised row has no 64-bit value: its codes are roundings
        return q, None, None
    if op == "prompt":
        lens = _ints(case["lens"])
        q, k, v = (s[n].double() for n in ("q", "k", "v"))
        ends = np.cumsum(lens)
        return torch.cat([_one64(q[e - n:e], k[e - n:e], v[e - n:e], 0, case["window"]) for n, e in zip(lens, ends)])
    q_lens, kv_lens = _ints(case["q_lens"]), _ints(case["kv_lens"])
    hm = _h64(d)
    out, at = [], 0
    for b, (n, m) in enumerate(zip(q_lens, kv_lens)):
        need = (m + case["page"] - 1) // case["page"]
        pages = s["table"][b, :need].long()
        sides = []
        for name in ("k", "v"):
            c = s["cache_" + name][pages]
            if case["fmt"] == "int8":
                x = c.double() - 128
            elif case["fmt"] == "int4":
                x = torch.empty(*c.shape[:-1], d, dtype=torch.float64, device="cuda")
                x[..., 0::2] = (c % 16).double() - 8
                x[..., 1::2] = (c // 16).double() - 8
            else:
                x = c.double()
            if case["fmt"] in _TOP:
                x = (x * s[name + "_scale"][pages].double()[..., None]) @ hm * (8.0 / d)
            sides.append(x.permute(0, 2, 1, 3).reshape(-1, case["kv"], d)[:m])
        out.append(_one64(s["q"][at:at + n].double(), *sides, m - n, case["window"]))
        at += n
    return torch.cat(out)
