"""The operators of a serving step around the paged cache, as a user's program calls them.

pages   the step's page tables, slots, positions and packing built on the GPU from the requests' lengths (plan), and
        the pages of ended requests given back (release)
norm    the norms of query and key heads, with the rotary positions (of one or several axes) in the same pass: on a
        fused projection's heads (rope), and with keys and values written into the paged cache (cache)
shared  attention of a batch whose sequences begin with the same cached tokens, read once for all of them

``own`` false computes the plain form in 32-bit torch; ``own`` true calls the library.  ``exact``
computes the same from the definition in 64 bits (whole numbers one by one).

The formats are those of the library's cache: a frequency is a phase, in turns of 2^64, that one position adds; the
quantised formats hold, for each token and head, the Hadamard transform of the head's vector times 2^-3 as offset codes
(code + 128 in a byte, code + 8 in a nibble, low nibble first) and one bfloat16 scale.
"""
import functools
import math

import numpy as np
import torch

own = False

_TURN = math.pi / 2.0**31  # radians of one unit of a phase's upper 32 bits
_BIAS = {"int8": 128, "int4": 8}
_TOP = {"int8": 127.0, "int4": 7.0}
_EPS = 1e-6


def _dt(name):
    return {"bf16": torch.bfloat16, "f16": torch.float16}[name]


def _ints(text):
    return [int(v) for v in text.split(",")] if text else []


def _text(values):
    return ",".join(str(v) for v in values)


# --------------------------------------------------------------------------------------------------
# cases


def listed():
    return [
        # a decode step's plan: every request has one new token, one in sixteen needs a page
        dict(name="plan_step", op="plan", batch=61, new="one", top=1, longest=16000, page=16, short=False),
        # a mixed step: prompts of up to 2000 tokens beside single tokens
        dict(name="plan_prompts", op="plan", batch=203, new="mixed", top=2000, longest=8000, page=64, short=False),
        # drafted tokens of a large batch, the pool nearly empty: the last requests are refused
        dict(name="plan_draft_short", op="plan", batch=2001, new="draft", top=5, longest=3000, page=16, short=True),
        # half of a batch ends, some of it with a shared beginning that stays
        dict(name="release_half", op="release", batch=250, longest=16000, page=16, shared=True),
        # one user's token: norms, rotation and the 16-bit write
        dict(name="norm_one", op="cache", tokens=1, heads=32, kv=8, dim=128, rot=128, layout="half", dtype="bf16",
             fmt="bf16", page=16, axes=1),
        # a decode step of 61 sequences into the 8-bit cache, and the new rows read back
        dict(name="norm_step_int8", op="cache", tokens=61, heads=40, kv=8, dim=128, rot=128, layout="half",
             dtype="bf16", fmt="int8", page=64, axes=3),
        # the patches of an image, whose query and key heads turn by height and width; keys are not cached
        dict(name="norm_image", op="rope", tokens=4099, heads=32, skip=16, dim=64, rot=64, layout="interleaved",
             dtype="f16", axes=2),
        # a long prompt with images in it: time, height and width
        dict(name="norm_prompt", op="cache", tokens=16381, heads=32, kv=8, dim=128, rot=128, layout="half",
             dtype="bf16", fmt="bf16", page=64, axes=3),
        # three answers to one short question, small heads
        dict(name="shared_small", op="shared", sizes="3", prefixes="700", q_lens="1,1,1", tails="1,17,130", heads=16,
             kv=4, dim=64, page=16, fmt="f16", dtype="f16"),
        # a serving batch behind one long system prompt
        dict(name="shared_step", op="shared", sizes="64", prefixes="8192", q_lens=_text([1] * 64),
             tails=_text([1 + (i * 7919) % 2000 for i in range(64)]), heads=32, kv=8, dim=128, page=16, fmt="bf16",
             dtype="bf16"),
        # drafted tokens behind two long documents, some sequences alone, 8-bit cache
        dict(name="shared_draft_int8", op="shared", sizes="24,9", prefixes="6011,30000",
             q_lens=_text([1 + i % 3 for i in range(39)]), tails=_text([3 + (i * 613) % 900 for i in range(39)]),
             heads=40, kv=8, dim=128, page=64, fmt="int8", dtype="bf16"),
        # questions of different lengths about one long document, 4-bit cache
        dict(name="shared_chunk_int4", op="shared", sizes="7", prefixes="16000", q_lens="300,1,129,512,64,700,33",
             tails="300,1211,129,2000,64,701,500", heads=32, kv=8, dim=128, page=32, fmt="int4", dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "plan", "release", "rope", "cache", "cache", "shared", "shared", "shared", "shared"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "plan":
        new = rng.choice(["one", "draft", "mixed"])
        batch = _log(rng, 1, 2000 if new != "mixed" else 200)
        return dict(op=op, batch=batch, new=new, top={"one": 1, "draft": 5, "mixed": _log(rng, 10, 2000)}[new],
                    longest=_log(rng, 30, 16000), page=page, short=rng.random() < 0.3)
    if op == "release":
        return dict(op=op, batch=_log(rng, 1, 250), longest=_log(rng, 30, 16000), page=page,
                    shared=rng.random() < 0.5)
    dtype = rng.choice(["bf16", "f16"])
    dim = rng.choice([64, 128, 128])
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 2, 3, 4, 5, 7, 8, 12])
    if op == "rope":
        return dict(op=op, tokens=_log(rng, 1, 8192), heads=min(48, heads + kv), skip=kv, dim=dim,
                    rot=rng.choice([dim, dim, dim // 2]), layout=rng.choice(["half", "interleaved"]), dtype=dtype,
                    axes=rng.choice([1, 2, 3]))
    if op == "cache":
        return dict(op=op, tokens=_log(rng, 1, 12000), heads=min(32, heads), kv=kv, dim=dim,
                    rot=rng.choice([dim, dim // 2]), layout=rng.choice(["half", "interleaved"]), dtype=dtype,
                    fmt=rng.choice(["int8", "int4", dtype]), page=page, axes=rng.choice([1, 2, 3]))
    kind = rng.choice(["one", "draft", "chunk"])
    sizes = [_log(rng, 1, 3 if kind == "chunk" else 24) for _ in range(rng.randint(1, 2))]
    prefixes = [_log(rng, 100, 10000) for _ in sizes]
    batch = sum(sizes) + rng.choice([0, 0, 1, 3])
    if kind == "chunk":
        heads = min(heads, 32) // kv * kv
        q_lens = [_log(rng, 1, 300) for _ in range(batch)]
    else:
        q_lens = [1 if kind == "one" else rng.randint(1, 4) for _ in range(batch)]
    tails = [q + _log(rng, 1, 600) - 1 for q in q_lens]
    return dict(op=op, sizes=_text(sizes), prefixes=_text(prefixes), q_lens=_text(q_lens), tails=_text(tails),
                heads=heads, kv=kv, dim=dim, page=page, fmt=rng.choice(["int8", "int4", dtype]), dtype=dtype)


# --------------------------------------------------------------------------------------------------
# what a program has in hand


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _mixed(g, shape, dtype, channels):
    """Activations of a projection: normal, with a few channels that stand out as those of keys do."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    loud = torch.rand((channels,), generator=g, device="cuda") < 0.02
    return (x * torch.where(loud, 5.0, 1.0)).to(dtype)


def _i32(values):
    return torch.tensor(np.asarray(values), dtype=torch.int32, device="cuda")


def _phases(rot):
    """Turns a position, as 64-bit fixed point."""
    turns = 10000.0 ** (-2.0 * np.arange(rot // 2) / rot) / (2 * math.pi)
    return torch.tensor([int(t * 2.0**64) for t in turns], dtype=torch.int64, device="cuda")


def prepare(case, seed):
    op = case["op"]
    s = dict(case=case)
    if op in ("plan", "release"):
        _prepare_pages(s, case, seed)
    elif op in ("rope", "cache"):
        _prepare_norm(s, case, seed)
    else:
        _prepare_shared(s, case, seed)
    return s


def _rows_of_step(case):
    """Rows of a captured step, for the requests' tokens and padding."""
    b, top = case["batch"], case["top"]
    if case["new"] == "mixed":  # a fifth of the requests with top / ln(top) tokens, and some room
        return int(b + 0.3 * b * top / math.log(top) + top)
    return b * top + 5


def _prepare_pages(s, case, seed):
    rng = np.random.default_rng(seed)
    b, page = case["batch"], case["page"]
    lens = np.exp(rng.uniform(0, math.log(case["longest"]), b)).astype(np.int64)
    held = (lens + page - 1) // page
    width = (case["longest"] + case.get("top", 0)) // page + 3
    if case["op"] == "plan":
        if case["new"] == "one":
            new = np.ones(b, dtype=np.int64)
        elif case["new"] == "draft":
            new = rng.integers(0, case["top"] + 1, b)
        else:  # one request in five brings a prompt (or a part of one)
            new = np.where(rng.random(b) < 0.2, np.exp(rng.uniform(0, math.log(case["top"]), b)).astype(np.int64), 1)
        held += rng.random(b) < 0.05  # drafted tokens that were refused have left a page ahead
        need = int(np.maximum((lens + new + page - 1) // page - held, 0).sum())
        spare = int(0.9 * need) if case["short"] else need + 100
        s["new"] = _i32(new)
        s["total"] = _rows_of_step(case)
    else:
        spare = int(rng.integers(0, 200))
        s["ended"] = torch.tensor(rng.random(b) < 0.5, device="cuda")
        s["shared"] = _i32(np.where(rng.random(b) < 0.3, held // 2, 0)) if case["shared"] else None
    pages = b * width + 200  # of the pool; those that are neither held nor free are another batch's
    order = rng.permutation(pages)
    table = np.full((b, width), -1, dtype=np.int32)
    ends = np.cumsum(held)
    for r in range(b):
        table[r, :held[r]] = order[ends[r] - held[r]:ends[r]]
    stack = np.full(pages, -1, dtype=np.int32)
    stack[:spare] = order[ends[-1]:][:spare]
    s["table"], s["lens"], s["held"] = _i32(table), _i32(lens), _i32(held)
    s["stack"], s["free"] = _i32(stack), _i32([spare])
    s["next"] = [torch.zeros_like(s[n]) for n in ("lens", "held", "free")]
    if own:
        import exl3_trellis_quantized_gb300 as E

        s["tables"] = E.KVTables(s["table"], s["lens"], s["held"], s["stack"], s["free"], page)
        s["into"] = E.KVTables(s["table"], s["next"][0], s["next"][1], s["stack"], s["next"][2], page)


def _prepare_norm(s, case, seed):
    g = _gen(seed)
    t, d, dtype = case["tokens"], case["dim"], _dt(case["dtype"])
    s["dtype"] = dtype
    turned = case["heads"] + (case["kv"] if case["op"] == "cache" else 0)
    rows = turned + (case["skip"] if case["op"] == "rope" else case["kv"])
    # a projection's fused output; the operators take views of it
    s["qkv"] = _mixed(g, (t, rows * d), dtype, rows * d).view(t, rows, d)
    s["phases"] = _phases(case["rot"])
    top = 131072
    start = int(torch.randint(0, top - t, (1,), generator=g, device="cuda"))
    at = torch.arange(t, device="cuda", dtype=torch.int32)
    if t > 256:  # time runs on, height and width go over the patches of images 61 wide
        rows_of = [start + at, start + at // 61 % 48, start + at % 61]
    else:  # a batch's own positions
        rows_of = [torch.randint(0, top, (t,), generator=g, device="cuda", dtype=torch.int32) for _ in range(3)]
    n = case["axes"]
    if n == 1:
        s["positions"], s["axes"] = rows_of[0].contiguous(), None
    else:
        s["positions"] = torch.stack(rows_of[3 - n:])
        i = torch.arange(case["rot"] // 2, device="cuda")
        # three axes in sections of the frequencies, two in turn
        third = max(1, case["rot"] // 6)
        s["axes"] = ((i // third).clamp_max(2) if n == 3 else i % 2).to(torch.uint8)

    def weight(*shape):
        return (1.0 + 0.3 * torch.randn(shape, generator=g, device="cuda")).to(dtype)

    if case["op"] == "rope":  # heads of queries and keys in one call, each row with its own weights
        s["weight"] = weight(case["heads"], d)
        return
    s["q_weight"], s["k_weight"] = weight(d), weight(d)
    pages = (t + case["page"] - 1) // case["page"] + 3
    s.update(_cache(g, case, pages))
    order = torch.randperm(pages, generator=g, device="cuda")
    where = at.long()
    if t <= 256:
        where = torch.randperm(pages * case["page"], generator=g, device="cuda")[:t]
    s["slots"] = order[where // case["page"]] * case["page"] + where % case["page"]


def _prepare_shared(s, case, seed):
    g = _gen(seed)
    d, ps = case["dim"], case["page"]
    s["dtype"] = _dt(case["dtype"])
    sizes, prefixes, q_lens, tails = (_ints(case[n]) for n in ("sizes", "prefixes", "q_lens", "tails"))
    prefix = [p for n, p in zip(sizes, prefixes) for _ in range(n)]
    prefix += [0] * (len(q_lens) - len(prefix))  # sequences of no group
    lens = [p + t for p, t in zip(prefix, tails)]
    s["q"] = _mixed(g, (sum(q_lens), case["heads"] * d), s["dtype"], case["heads"] * d).view(-1, case["heads"], d)
    # a group's whole pages of the prefix are shared; what is left of it lies in each sequence's own next page
    first = [sum(sizes[:i]) for i in range(len(sizes))]
    need = [(n + ps - 1) // ps for n in lens]
    width = max(need) + 1
    pages = sum(need) + 5
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).cpu().numpy()
    table = np.full((len(lens), width), -1, dtype=np.int32)
    copies = []  # page from, page to, rows
    at = 0
    for b, n in enumerate(need):
        lead = max([f for f in first if f <= b and b < sum(sizes)], default=b)
        keep = prefix[b] // ps if lead != b else 0
        table[b, :keep] = table[lead, :keep]
        table[b, keep:n] = order[at:at + n - keep]
        at += n - keep
        if lead != b and prefix[b] % ps:
            copies.append((table[lead, keep], table[b, keep], prefix[b] % ps))
    s.update(_cache(g, case, pages))
    for name in ("cache_k", "cache_v", "k_scale", "v_scale"):
        if s[name] is not None:
            for a, b, n in copies:
                s[name][int(b), :, :n] = s[name][int(a), :, :n]
    s["table"] = torch.tensor(table, device="cuda")
    s["cu"] = _i32(np.concatenate([[0], np.cumsum(q_lens)]))
    s["kv_lens"] = _i32(lens)
    s["groups"] = _i32(np.concatenate([[0], np.cumsum(sizes)]))
    s["prefix"] = _i32(prefixes)
    s["max_q"], s["max_kv"], s["max_prefix"] = max(q_lens), max(lens), max(prefixes)


def _cache(g, case, pages):
    """A cache in use: every page holds some sequence's rows."""
    kv, d, ps, fmt = case["kv"], case["dim"], case["page"], case["fmt"]
    out = {}
    for name in ("k", "v"):
        if fmt in ("bf16", "f16"):
            out["cache_" + name] = torch.randn((pages, kv, ps, d), generator=g, device="cuda",
                                               dtype=torch.float32).to(_dt(fmt))
            out[name + "_scale"] = None
            continue
        # codes of rotated vectors are close to normal, the largest of a row at the top code
        if fmt == "int8":
            c = torch.randn((pages, kv, ps, d), generator=g, device="cuda") * 46.0
            codes = (c.round().clamp(-127, 127) + 128).to(torch.uint8)
        else:
            c = torch.randn((pages, kv, ps, d // 2, 2), generator=g, device="cuda") * 2.6
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
    if own:
        return _own(s)
    return {"plan": _plain_plan, "release": _plain_release, "rope": _plain_rope, "cache": _plain_cache,
            "shared": _plain_shared}[s["case"]["op"]](s)


def _own(s):
    import exl3_trellis_quantized_gb300 as E

    case = s["case"]
    op = case["op"]
    if op == "plan":
        cu, positions, slots, granted = E.kv_plan(s["tables"], s["new"], s["total"], into=s["into"])
        return (cu, positions, slots, granted, *s["next"], s["table"])
    if op == "release":
        E.kv_release(s["tables"], s["ended"], shared=s["shared"], into=s["into"])
        return (*s["next"], s["stack"])
    if op == "rope":
        return E.rope(s["qkv"][:, :case["heads"]], s["positions"], s["phases"], layout=case["layout"], axes=s["axes"],
                      weight=s["weight"], eps=_EPS)
    cache = E.KVCache(s["cache_k"], s["cache_v"], s["k_scale"], s["v_scale"], case["fmt"])
    if op == "cache":
        h, kv, x = case["heads"], case["kv"], s["qkv"]
        q = E.kv_write(cache, x[:, h:h + kv], x[:, h + kv:], s["slots"], q=x[:, :h], positions=s["positions"],
                       phases=s["phases"], layout=case["layout"], axes=s["axes"], q_weight=s["q_weight"],
                       k_weight=s["k_weight"], eps=_EPS)
        if case["fmt"] in _TOP:
            return (q, *E.kv_read(cache, s["slots"], dtype=s["dtype"]))
        return q, s["cache_k"], s["cache_v"]
    return E.attention_shared(s["q"], cache, s["table"], s["cu"], s["kv_lens"], s["groups"], s["prefix"], s["max_q"],
                              s["max_kv"], s["max_prefix"])


def _plain_plan(s):
    page, total, width = s["case"]["page"], s["total"], s["table"].shape[1]
    new, lens, held = (s[n].long() for n in ("new", "lens", "held"))
    new = new.clamp_min(0)
    ends = new.cumsum(0)
    want = (lens + new + page - 1) // page
    can = (ends <= total) & (want <= width)
    need = torch.where(can & (new > 0), (want - held).clamp_min(0), 0)
    upto = need.cumsum(0)
    granted = can & ((need == 0) | (upto <= s["free"]))
    need = torch.where(granted, need, 0)
    # the table's new entries: column c of request b is its page c - held[b], counted from the top of the stack
    col = torch.arange(width, device=lens.device)[None, :]
    mine = (col >= held[:, None]) & (col < (held + need)[:, None])
    at = s["free"] - 1 - ((upto - need)[:, None] + col - held[:, None])
    s["table"].copy_(torch.where(mine, s["stack"][at.clamp(0, s["stack"].numel() - 1)], s["table"]))
    cu = torch.cat([ends.new_zeros(1), ends]).clamp_max(total).to(torch.int32)
    # tokens: the request of each, and its place in it
    t = torch.arange(total, device=lens.device)
    b = (t[:, None] >= ends[None, :]).sum(1) if total * new.numel() < 1 << 28 else torch.searchsorted(ends, t, right=True)
    there = b < new.numel()
    b = b.clamp_max(new.numel() - 1)
    pos = lens[b] + t - (ends - new)[b]
    positions = torch.where(there, pos, 0)
    entry = s["table"][b, (pos // page).clamp(0, width - 1)].long()
    slots = torch.where(there & granted[b] & (entry >= 0), entry * page + pos % page, -1)
    s["next"][0].copy_(torch.where(granted, lens + new, lens))
    s["next"][1].copy_(held + need)
    s["next"][2].copy_(s["free"] - need.sum())
    return (cu, positions.to(torch.int32), slots, granted, *s["next"], s["table"])


def _plain_release(s):
    width = s["table"].shape[1]
    held, ended = s["held"].long(), s["ended"]
    keep = torch.zeros_like(held) if s["shared"] is None else torch.minimum(s["shared"].long(), held)
    give = torch.where(ended, held - keep, 0)
    before = give.cumsum(0) - give
    col = torch.arange(width, device=held.device)[None, :]
    mine = (col >= keep[:, None]) & (col < held[:, None]) & ended[:, None]
    at = s["free"].long() + before[:, None] + col - keep[:, None]
    s["stack"][at[mine]] = s["table"][mine]
    s["next"][0].copy_(torch.where(ended, 0, s["lens"]))
    s["next"][1].copy_(torch.where(ended, 0, s["held"]))
    s["next"][2].copy_(s["free"] + give.sum())
    return (*s["next"], s["stack"])


def _normed(x, weight):
    """x [T, H, D] in 32 bits over its root mean square, times weight [D] or [H, D]."""
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS) * weight.float()


def _rotate(x, s):
    """x [T, H, D] in 32 bits, its first 2 * len(phases) values of each head rotated."""
    half = s["phases"].numel()
    p = s["positions"].long()
    p = p[:, None] if s["axes"] is None else p.T[:, s["axes"].long()]  # [T, half]
    angle = ((p * s["phases"][None, :]) >> 32).float() * _TURN
    c, n = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    if s["case"]["layout"] == "half":
        a, b, rest = x[..., :half], x[..., half:2 * half], x[..., 2 * half:]
        return torch.cat([a * c - b * n, b * c + a * n, rest], -1)
    a, b, rest = x[..., 0:2 * half:2], x[..., 1:2 * half:2], x[..., 2 * half:]
    return torch.cat([torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2), rest], -1)


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
    return torch.round(y * (1.0 / scale)).clamp(-_TOP[fmt], _TOP[fmt]), scale


def _store(codes, fmt):
    c = (codes + _BIAS[fmt]).to(torch.uint8)
    return c if fmt == "int8" else c[..., 0::2] | (c[..., 1::2] << 4)


def _load(stored, fmt):
    if fmt == "int8":
        return stored.float() - 128.0
    return torch.stack([stored & 15, stored >> 4], -1).flatten(-2).float() - 8.0


def _plain_rope(s):
    x = s["qkv"][:, :s["case"]["heads"]].float()
    return _rotate(_normed(x, s["weight"]), s).to(s["dtype"])


def _plain_cache(s):
    case = s["case"]
    h, kv, d, fmt, ps = case["heads"], case["kv"], case["dim"], case["fmt"], case["page"]
    x = s["qkv"].float()
    weight = torch.cat([s["q_weight"].expand(h, d), s["k_weight"].expand(kv, d)])
    turned = _rotate(_normed(x[:, :h + kv], weight), s).to(s["dtype"])
    page, at = s["slots"] // ps, s["slots"] % ps
    if fmt not in _TOP:
        s["cache_k"][page, :, at] = turned[:, h:]
        s["cache_v"][page, :, at] = x[:, h + kv:].to(s["dtype"])
        return turned[:, :h], s["cache_k"], s["cache_v"]
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


def _plain_shared(s):
    case = s["case"]
    h, kv, d = case["heads"], case["kv"], case["dim"]
    cu, lens = s["cu"], s["kv_lens"]
    q_lens = cu[1:] - cu[:-1]
    at = torch.arange(s["max_q"], device=cu.device)
    there = at[None, :] < q_lens[:, None]
    idx = (cu[:-1, None] + at[None, :]).clamp(0, s["q"].shape[0] - 1).long()
    q = s["q"].float()[idx]
    turned = s["k_scale"] is not None
    if turned:
        q = _hadamard(q) * (8.0 / d)
    q = q.view(*idx.shape, kv, h // kv, d).permute(0, 2, 3, 1, 4)
    k, v = _rows(s, "k"), _rows(s, "v")
    pos = (lens - q_lens)[:, None] + at[None, :]
    j = torch.arange(k.shape[2], device=cu.device)[None, None, :]
    seen = (j <= pos[..., None]) & there[..., None]
    o = _attend(q, k, v, seen[:, None])
    if turned:
        o = _hadamard(o) * (8.0 / d)
    return o.permute(0, 3, 1, 2, 4).reshape(*idx.shape, h, d)[there].to(s["dtype"])


# --------------------------------------------------------------------------------------------------
# what a pass cannot do without


def _row_bytes(case):
    """Bytes of one cached row of one head, key or value."""
    return {"bf16": 2 * case["dim"], "f16": 2 * case["dim"], "int8": case["dim"] + 2,
            "int4": case["dim"] // 2 + 2}[case["fmt"]]


def work(case):
    op = case["op"]
    if op == "plan":
        b = case["batch"]
        tokens = _rows_of_step(case)
        pages = tokens // case["page"]
        # lengths, held pages and new tokens of a request in and out, its flag; a row's position and slot; a page's
        # id from the stack into the table, and one entry of every request's table
        return {"bytes": 29 * b + 12 * tokens + 8 * pages, "flops": 8 * b + 6 * tokens}
    if op == "release":
        pages = int(case["batch"] * case["longest"] / math.log(case["longest"]) / case["page"] / 2)
        return {"bytes": 17 * case["batch"] + 8 * pages, "flops": 4 * case["batch"] + 2 * pages}
    d = case["dim"]
    if op == "rope":
        n = case["tokens"] * case["heads"]
        return {"bytes": n * d * 4 + case["tokens"] * 4 * case["axes"], "flops": n * (4 * d + 3 * case["rot"])}
    if op == "cache":
        t, h, kv = case["tokens"], case["heads"], case["kv"]
        quant = case["fmt"] in _TOP
        turn = 2 * (d.bit_length() - 1) + 3 if quant else 0
        # rows in, rotated queries out, rows into the cache; the quantised rows read back and out
        moved = t * (h * d * 4 + 2 * kv * (2 * d + _row_bytes(case)) + 4 * case["axes"] + 8)
        back = t * 2 * kv * (_row_bytes(case) + 2 * d) if quant else 0
        return {"bytes": moved + back, "flops": t * ((h + kv) * (4 * d + 3 * case["rot"]) + 2 * kv * d * turn)}
    sizes, prefixes, q_lens, tails = (_ints(case[n]) for n in ("sizes", "prefixes", "q_lens", "tails"))
    prefix = [p for n, p in zip(sizes, prefixes) for _ in range(n)]
    prefix += [0] * (len(q_lens) - len(prefix))
    pairs = sum(q * (p + t - q) + q * (q + 1) // 2 for q, p, t in zip(q_lens, prefix, tails))
    rows = sum(prefixes) + sum(tails)
    return {"bytes": sum(q_lens) * case["heads"] * d * 4 + rows * case["kv"] * 2 * _row_bytes(case),
            "flops": 4 * d * case["heads"] * pairs}


# --------------------------------------------------------------------------------------------------
# the definition, in 64 bits


def exact(case, seed):
    return {"plan": _exact_plan, "release": _exact_release, "rope": _exact_norm, "cache": _exact_norm,
            "shared": _exact_shared}[case["op"]](case, prepare(case, seed))


def _exact_plan(case, s):
    page, total = case["page"], s["total"]
    table, stack = s["table"].cpu().numpy().copy(), s["stack"].cpu().tolist()
    new, lens, held = (s[n].cpu().tolist() for n in ("new", "lens", "held"))
    free = int(s["free"])
    cu, positions, slots, granted = [0], [], [], []
    left, dry = free, False
    for b, n in enumerate(new):
        n = max(n, 0)
        at = cu[-1]
        want = -(-(lens[b] + n) // page)
        need = max(0, want - held[b]) if n else 0
        ok = at + n <= total and want <= table.shape[1]
        if ok and need:
            dry = dry or need > left  # who comes after a request that got no pages gets none either
            ok = not dry
        if ok:
            for _ in range(need):
                left -= 1
                table[b, held[b]] = stack[left]
                held[b] += 1
        for i in range(min(n, total - at)):
            positions.append(lens[b] + i)
            slots.append(int(table[b, positions[-1] // page]) * page + positions[-1] % page if ok else -1)
        granted.append(ok)
        lens[b] += n if ok else 0
        cu.append(min(at + n, total))
    positions += [0] * (total - len(positions))
    slots += [-1] * (total - len(slots))
    return (_i32(cu), _i32(positions), torch.tensor(slots, dtype=torch.int64, device="cuda"),
            torch.tensor(granted, device="cuda"), _i32(lens), _i32(held), _i32([left]), _i32(table))


def _exact_release(case, s):
    table, stack = s["table"].cpu().numpy(), s["stack"].cpu().tolist()
    lens, held, ended = (s[n].cpu().tolist() for n in ("lens", "held", "ended"))
    shared = [0] * len(lens) if s["shared"] is None else s["shared"].cpu().tolist()
    free = int(s["free"])
    for b, done in enumerate(ended):
        if done:
            for page in table[b, min(shared[b], held[b]):held[b]]:
                stack[free] = int(page)
                free += 1
            lens[b] = held[b] = 0
    return _i32(lens), _i32(held), _i32([free]), _i32(stack)


def _exact_norm(case, s):
    t, r, n = case["tokens"], case["rot"], case["heads"] + case.get("kv", 0)
    if t * r > 2_200_000:
        return None
    x = s["qkv"][:, :n].double()
    size = torch.linalg.vector_norm(x, dim=-1, keepdim=True)
    if case["op"] == "rope":
        w = s["weight"].double()
    else:
        w = torch.stack([s["q_weight"]] * case["heads"] + [s["k_weight"]] * case["kv"]).double()
    y = x / torch.sqrt(size**2 / case["dim"] + _EPS) * w
    p = s["positions"].cpu().numpy().astype(object).reshape(case["axes"], t)
    axis = [0] * (r // 2) if s["axes"] is None else s["axes"].tolist()
    f = s["phases"].tolist()
    turns = np.stack([np.array([v * f[i] % 2**64 / 2.0**64 for v in p[axis[i]]], dtype=np.float64)
                      for i in range(r // 2)], -1)
    spin = torch.polar(torch.ones(t, 1, r // 2, dtype=torch.float64, device="cuda"),
                       2 * math.pi * torch.tensor(turns, device="cuda")[:, None])
    first, second = (slice(0, r // 2), slice(r // 2, r)) if case["layout"] == "half" else (slice(0, r, 2), slice(1, r, 2))
    z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * spin
    y[..., first], y[..., second] = z.real, z.imag
    if case["op"] == "rope":
        return y
    if case["fmt"] in _TOP:  # a quantised row has no 64-bit value: its codes are roundings
        return y[:, :case["heads"]], None, None
    k, v = s["cache_k"].double(), s["cache_v"].double()
    where, row = s["slots"] // case["page"], s["slots"] % case["page"]
    k[where, :, row] = y[:, case["heads"]:]
    v[where, :, row] = s["qkv"][:, n:].double()
    return y[:, :case["heads"]], k, v


def _h64(d):
    i = np.arange(d)
    bits = np.zeros((d, d), dtype=np.int64)
    a = i[:, None] & i[None, :]
    while a.any():
        bits += a & 1
        a = a >> 1
    return torch.tensor(1.0 - 2.0 * (bits & 1), dtype=torch.float64, device="cuda")


def _exact_shared(case, s):
    d, h, kv = case["dim"], case["heads"], case["kv"]
    hm = _h64(d)
    lens, cu = s["kv_lens"].tolist(), s["cu"].tolist()
    out = torch.zeros((cu[-1], h, d), dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        pages = s["table"][b, :(n + case["page"] - 1) // case["page"]].long()
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
            sides.append(x.permute(1, 0, 2, 3).reshape(kv, -1, d)[:, :n])
        k, v = sides
        q = s["q"][cu[b]:cu[b + 1]].double()
        pos = n - q.shape[0] + torch.arange(q.shape[0], device="cuda")
        hidden = torch.arange(n, device="cuda")[None, :] > pos[:, None]
        for head in range(h):
            x = (q[:, head] @ k[head * kv // h].T) / math.sqrt(d)
            out[cu[b]:cu[b + 1], head] = torch.softmax(x.masked_fill(hidden, -math.inf), -1) @ v[head * kv // h]
    return out
