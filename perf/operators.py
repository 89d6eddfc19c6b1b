"""The quantised key/value cache: writing it, reading it back, and decode attention over it.

Three operators, each in its plain form (elementary torch operations) and as the
library's call:

  write  new keys and values of T tokens are quantised into the cache (Q8_0 or
         Q4_0 codes per 32-block, fp16 scale) at their slots; the tokens are
         then read back, so that the outputs are the values the cache stands for
  read   T cached tokens, given by their slots, as values
  attn   M query tokens (1 .. 8) of each of B sequences attend to their pages of
         the cache: softmax(scale q.k) v, causal among the M, an optional
         sliding window, grouped heads

The cache is one byte buffer of pages; a page holds, for each key/value head,
groups of 16 tokens, a group its key codes, key scales, value codes and value
scales. ``_codes_at`` and ``_scales_at`` give the place of each byte.
"""
import functools
import math

import torch

own = False

BLOCK, GROUP = 32, 16
QTYPE = {"q8": 0, "q4": 1}
DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}


def _case(name, op, **kw):
    return {"name": name, "op": op, **kw}


def listed():
    kv = dict(page=64, kt="q4", vt="q4", dtype="f32")
    return [
        # one new token of a 14-head / 2-kv-head decoder of head size 64: the smallest call, latency only
        _case("write_1_token", "write", tokens=1, hkv=2, d=64, **{**kv, "kt": "q8", "vt": "q8"}),
        # one new token of each of 64 sequences
        _case("write_64_tokens", "write", tokens=64, hkv=8, d=128, **kv),
        # a prompt of odd length, bf16 projections, finer keys than values, small pages
        _case("write_prompt_1021", "write", tokens=1021, hkv=8, d=128, page=16, kt="q8", vt="q4", dtype="bf16"),
        # several prompts at once: the widest write
        _case("write_prompt_16384", "write", tokens=16384, hkv=8, d=128, **{**kv, "dtype": "bf16"}),
        # an odd number of cached tokens, head size 96
        _case("read_777", "read", tokens=777, hkv=4, d=96, **{**kv, "kt": "q8"}),
        # a long context handed on as bf16
        _case("read_65536", "read", tokens=65536, hkv=8, d=128, **{**kv, "dtype": "bf16"}),
        # a chat's first tokens, one sequence: latency only
        _case("attn_b1_33", "attn", batch=1, queries=1, hq=14, hkv=2, d=64, length=33, ragged=False, window=0,
              **{**kv, "kt": "q8", "vt": "q8"}),
        # one sequence of the same decoder at an ordinary context, four-bit cache
        _case("attn_b1_4096", "attn", batch=1, queries=1, hq=14, hkv=2, d=64, length=4096, ragged=False, window=0, **kv),
        # one very long sequence of a 40-head decoder: little batch, much context
        _case("attn_b1_131072", "attn", batch=1, queries=1, hq=40, hkv=8, d=128, length=131072, ragged=False, window=0, **kv),
        # four drafted tokens of each of eight sequences of uneven lengths, one slot empty
        _case("attn_b8_m4_2500", "attn", batch=8, queries=4, hq=40, hkv=8, d=128, length=2500, ragged=True, window=0,
              **{**kv, "dtype": "bf16"}),
        # a serving batch at uneven lengths, one slot empty: the largest
        _case("attn_b64_8192", "attn", batch=64, queries=1, hq=40, hkv=8, d=128, length=8192, ragged=True, window=0, **kv),
        # head size 256 and a sliding window over small pages, finer keys than values
        _case("attn_window_d256", "attn", batch=16, queries=1, hq=8, hkv=4, d=256, length=6000, ragged=False, window=1024,
              page=16, kt="q8", vt="q4", dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("write", "read", "attn", "attn"))
    case = {"op": op, "page": rng.choice((16, 32, 64, 128)), "kt": rng.choice(("q8", "q4")),
            "vt": rng.choice(("q8", "q4", "q4")), "dtype": rng.choice(("f32", "bf16"))}
    if op != "attn":
        top = 16384 if op == "write" else 65536
        case |= {"hkv": rng.choice((1, 2, 3, 4, 8)), "d": rng.choice((64, 96, 128)), "tokens": _log(rng, 1, top)}
        return case
    d = rng.choice((64, 96, 128, 256))
    hkv, ratio, m = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 4, 5, 7, 8)), rng.choice((1, 1, 1, 2, 4, 7, 8))
    case |= {"hkv": hkv, "d": d, "hq": hkv * ratio, "queries": m}
    # as many keys as cost what the largest listed case does, whatever the head size, the types and the rows per key
    most = 64 * 4096 * 8 * 128 // (hkv * d * (2 if "q8" in (case["kt"], case["vt"]) else 1) * max(1, -(-ratio * m // 8)))
    length = min(_log(rng, 1, 131072), most)
    case |= {"length": length, "batch": _log(rng, 1, max(1, min(64, most // length))), "ragged": rng.choice((True, False)),
             "window": rng.choice((0, 0, _log(rng, 1, 8192)))}
    return case


# --------------------------------------------------------------------------- the cache's layout

def _part(d, qt):
    """Bytes of one group's codes and scales (keys or values)."""
    return GROUP * (d if qt == "q8" else d // 2) + GROUP * (d // BLOCK) * 2


def _run_of(b, nb, widest):
    """Blocks are laid in runs of `widest`, then of the powers of two below: (first block of b's run, its length)."""
    first, n = 0, widest
    while True:
        while first + n <= nb:
            if b < first + n:
                return first, n
            first += n
        n //= 2


@functools.lru_cache(maxsize=None)  # a table of the layout, the same for every call
def _codes_at(d, qt, part, device):
    """Byte offset in a group of code byte x of block b of token t: int64 [16, d/32, 32 (q8) or 16 (q4)]."""
    nb, widest, size = d // BLOCK, (2 if qt == "q8" else 4), (32 if qt == "q8" else 16)
    runs = [_run_of(b, nb, widest) for b in range(nb)]
    first = torch.tensor([r[0] for r in runs], device=device).view(1, nb, 1)
    n = torch.tensor([r[1] for r in runs], device=device).view(1, nb, 1)
    t = torch.arange(GROUP, device=device).view(GROUP, 1, 1)
    r = torch.arange(nb, device=device).view(1, nb, 1) - first
    x = torch.arange(size, device=device).view(1, 1, size)
    base = first * GROUP * size
    if part == "k":
        row = 8 * (t // 8) + 2 * (t % 4) + (t // 4) % 2
        if qt == "q8":
            return base + ((row * 4 + (x % 16) // 4) * n + r) * 8 + (x // 16) * 4 + x % 4
        return base + ((row * 4 + x // 4) * n + r) * 4 + x % 4
    g = (x % 16) // 2
    unit = 4 if qt == "q8" else 2
    inside = r * unit + (x // 16) * 2 + x % 2
    halves = (((g // 4) * GROUP + t) * 4 + g % 4) * 8
    whole = (t * 8 + g) * (n * unit)
    return base + torch.where(n == widest, halves, whole) + inside


@functools.lru_cache(maxsize=None)
def _scales_at(d, qt, device):
    """Byte offset in a group of the fp16 scale of block b of token t: int64 [16, d/32]."""
    nb = d // BLOCK
    t = torch.arange(GROUP, device=device).view(GROUP, 1)
    b = torch.arange(nb, device=device).view(1, nb)
    return GROUP * (d if qt == "q8" else d // 2) + ((t % 4) * nb + b) * 8 + (t // 4) * 2


def _quantise(x, qt):
    """x fp32 [..., d] -> (code bytes uint8 [..., d/32, 32 or 16], scales fp16 [..., d/32]): ggml's rules, each step in binary32."""
    x = x.unflatten(-1, (-1, BLOCK))
    amax = x.abs().amax(-1, keepdim=True)
    if qt == "q8":
        d = amax / torch.full_like(amax, 127.0)  # by a tensor: a division by a number is done as a product
        inv = torch.where(d != 0, 1.0 / d, torch.zeros_like(d))
        y = (x * inv).double()
        y = torch.trunc(y.abs() + 0.5) * torch.sign(y)  # half away from zero; in 64 bits, as 0.5 - 2^-25 plus 0.5 is 1 in 32
        return y.clamp(-127, 127).to(torch.int8).view(torch.uint8), d.squeeze(-1).to(torch.float16)
    place = torch.arange(BLOCK, device=x.device)  # the scale takes its sign from the first of the largest
    at = torch.where(x.abs() == amax, place, BLOCK).amin(-1, keepdim=True).clamp(max=BLOCK - 1)
    d = x.gather(-1, at) / -8.0
    inv = torch.where(d != 0, 1.0 / d, torch.zeros_like(d))
    q = torch.trunc(x * inv + 8.5).clamp(0, 15).to(torch.uint8)
    return q[..., :16] | (q[..., 16:] << 4), d.squeeze(-1).to(torch.float16)


def _values(codes, scales, qt):
    """Code bytes uint8 [..., d/32, 32 or 16] and scales fp16 [..., d/32] -> fp32 [..., d]."""
    if qt == "q8":
        q = codes.contiguous().view(torch.int8).float()
    else:
        q = torch.cat((codes & 15, codes >> 4), -1).float() - 8.0
    return (q * scales.float().unsqueeze(-1)).flatten(-2)


def _group_values(groups, d, qt, part, start):
    """groups uint8 [..., bytes of a group] -> fp32 [..., 16, d]."""
    codes = groups[..., start + _codes_at(d, qt, part, groups.device)]
    at = start + _scales_at(d, qt, groups.device)
    scales = groups[..., torch.stack((at, at + 1), -1)].view(torch.float16).squeeze(-1)
    return _values(codes, scales, qt)


# --------------------------------------------------------------------------- inputs

class State:
    pass


def _lens(case):
    """Tokens of each sequence: all alike, or spread from few to `length`, with an empty slot where there are four sequences or more."""
    n, top = case["batch"], case["length"]
    if not case["ragged"]:
        return [top] * n
    return [0 if b == 0 and n >= 4 else max(1, top * (b + 1) // n - (b * 7) % 13) for b in range(n)]


def _fill(s, gen, dev):
    """A cache whose every page holds quantised keys and values: channels of uneven size, as projections give."""
    s.cache = torch.empty((s.pages, s.hkv, s.page // GROUP, _part(s.d, s.kt) + _part(s.d, s.vt)), dtype=torch.uint8, device=dev)
    size = [torch.exp(0.5 * torch.randn((s.hkv, 1, 1, s.d), generator=gen, device=dev)) for _ in range(2)]
    step = max(1, (1 << 25) // (s.hkv * s.page * s.d))
    for at in range(0, s.pages, step):
        out = s.cache[at:at + step]
        for k, (part, qt, start) in enumerate((("k", s.kt, 0), ("v", s.vt, _part(s.d, s.kt)))):
            x = torch.randn((out.shape[0], s.hkv, s.page // GROUP, GROUP, s.d), generator=gen, device=dev) * size[k]
            codes, scales = _quantise(x, qt)
            out[..., (start + _codes_at(s.d, qt, part, dev)).flatten()] = codes.flatten(-3)
            at2 = start + _scales_at(s.d, qt, dev)
            out[..., torch.stack((at2, at2 + 1), -1).flatten()] = scales.unsqueeze(-1).view(torch.uint8).flatten(-3)
    s.cache = s.cache.view(s.pages, -1)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    s = State()
    s.op, s.hkv, s.d, s.page, s.kt, s.vt = (case[k] for k in ("op", "hkv", "d", "page", "kt", "vt"))
    s.dtype = DTYPE[case["dtype"]]
    if s.op == "attn":
        lens = _lens(case)
        s.hq, s.window, s.scale = case["hq"], case["window"], case["d"] ** -0.5
        held = [-(-n // s.page) for n in lens]
        s.pages = sum(held) + 1
        _fill(s, gen, dev)
        order = torch.randperm(s.pages, generator=gen, device=dev).to(torch.int32)
        s.table = torch.full((len(lens), max(max(held), 1)), -1, dtype=torch.int32, device=dev)
        at = 0
        for b, n in enumerate(held):
            s.table[b, :n] = order[at:at + n]
            at += n
        s.lens = torch.tensor(lens, dtype=torch.int32, device=dev)
        # the queries are a slice of the fused projections' rows
        row = torch.randn((case["batch"], case["queries"], (s.hq + 2 * s.hkv) * s.d), generator=gen, device=dev) * 1.5
        s.q = row.to(s.dtype)[..., : s.hq * s.d].unflatten(-1, (s.hq, s.d))
        return s
    held = -(-case["tokens"] // s.page)
    s.pages = held + 1
    if case["tokens"] <= 64:  # one token of each sequence: every token on a page of its own
        s.pages = case["tokens"] + 1
        order = torch.randperm(s.pages, generator=gen, device=dev)[: case["tokens"]]
        s.slots = order * s.page + torch.randint(s.page, (case["tokens"],), generator=gen, device=dev)
    else:  # prompts: runs of tokens, page after page
        order = torch.randperm(s.pages, generator=gen, device=dev)
        t = torch.arange(case["tokens"], device=dev)
        s.slots = order[t // s.page] * s.page + t % s.page
    _fill(s, gen, dev)
    if s.op == "write":  # keys and values are slices of the fused projections' rows, behind the queries
        size = torch.exp(0.5 * torch.randn((3, s.hkv, s.d), generator=gen, device=dev))
        row = (torch.randn((case["tokens"], 3, s.hkv, s.d), generator=gen, device=dev) * size).to(s.dtype)
        s.k, s.v = row[:, 1], row[:, 2]
    return s


# --------------------------------------------------------------------------- the operators

def _plain_read(s):
    group = s.slots // GROUP
    page, inside, t = group // (s.page // GROUP), group % (s.page // GROUP), s.slots % GROUP
    groups = s.cache.view(s.pages, s.hkv, s.page // GROUP, -1)[page, :, inside]  # [T, hkv, bytes]
    out = []
    for part, qt, start in (("k", s.kt, 0), ("v", s.vt, _part(s.d, s.kt))):
        at = (start + _codes_at(s.d, qt, part, groups.device))[t]  # [T, d/32, n]
        codes = groups.gather(2, at.flatten(1).unsqueeze(1).expand(-1, s.hkv, -1)).unflatten(-1, at.shape[1:])
        at = (start + _scales_at(s.d, qt, groups.device))[t]
        at = torch.stack((at, at + 1), -1)
        scales = groups.gather(2, at.flatten(1).unsqueeze(1).expand(-1, s.hkv, -1)).view(torch.float16)
        out.append(_values(codes, scales, qt).to(s.dtype))
    return tuple(out)


def _plain_write(s):
    group = s.slots // GROUP
    page, inside, t = group // (s.page // GROUP), group % (s.page // GROUP), s.slots % GROUP
    size = _part(s.d, s.kt) + _part(s.d, s.vt)
    head = torch.arange(s.hkv, device=s.slots.device)
    base = ((page.unsqueeze(1) * s.hkv + head) * (s.page // GROUP) + inside.unsqueeze(1)) * size  # [T, hkv]
    flat = s.cache.view(-1)
    for x, part, qt, start in ((s.k, "k", s.kt, 0), (s.v, "v", s.vt, _part(s.d, s.kt))):
        codes, scales = _quantise(x.float(), qt)
        at = (start + _codes_at(s.d, qt, part, flat.device))[t]
        flat[base[:, :, None, None] + at[:, None]] = codes
        at = (start + _scales_at(s.d, qt, flat.device))[t]
        at = torch.stack((at, at + 1), -1)
        flat[base[:, :, None, None] + at[:, None]] = scales.unsqueeze(-1).view(torch.uint8)
    return _plain_read(s)


def _plain_attn(s):
    nseq, m = s.q.shape[:2]
    groups = s.cache.view(s.pages, s.hkv, s.page // GROUP, -1)[s.table.clamp(min=0).long()]  # [B, pages, hkv, groups, bytes]
    groups = groups.transpose(1, 2)
    k = _group_values(groups, s.d, s.kt, "k", 0).reshape(nseq, s.hkv, -1, s.d)
    v = _group_values(groups, s.d, s.vt, "v", _part(s.d, s.kt)).reshape(nseq, s.hkv, -1, s.d)
    q = s.q.float().unflatten(2, (s.hkv, -1)).permute(0, 2, 1, 3, 4)  # [B, hkv, M, ratio, d]
    scores = (q.flatten(2, 3) @ k.transpose(2, 3)).unflatten(2, q.shape[2:4]) * s.scale  # [B, hkv, M, ratio, keys]
    pos = torch.arange(k.shape[2], device=k.device)
    last = s.lens.view(-1, 1) - m + torch.arange(m, device=k.device)  # the last key that each query sees
    seen = pos <= last.unsqueeze(-1)
    if s.window:
        seen &= pos > last.unsqueeze(-1) - s.window
    seen = seen[:, None, :, None]
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    out = (p.flatten(2, 3) @ v).unflatten(2, q.shape[2:4]) / torch.where(total > 0, total, torch.ones_like(total))
    return out.permute(0, 2, 1, 3, 4).flatten(2, 3).to(s.dtype)


def run(state):
    s = state
    if own:
        import decode_gemv_qmm_b200 as qmm

        form = {"page": s.page, "ktype": QTYPE[s.kt], "vtype": QTYPE[s.vt]}
        if s.op == "attn":
            return qmm.qmm_kv_attn(s.q, s.cache, s.table, s.lens, s.hkv, scale=s.scale, window=s.window, **form)
        if s.op == "write":
            qmm.qmm_kv_write(s.cache, s.k, s.v, s.slots, **form)
        return qmm.qmm_kv_read(s.cache, s.slots, s.hkv, s.d, dtype=s.dtype, **form)
    return {"attn": _plain_attn, "write": _plain_write, "read": _plain_read}[s.op](s)


def work(case):
    d, hkv, size = case["d"], case["hkv"], 4 if case["dtype"] == "f32" else 2
    token = (_part(d, case["kt"]) + _part(d, case["vt"])) // GROUP * hkv
    if case["op"] == "read":
        return {"bytes": case["tokens"] * (token + 2 * hkv * d * size + 8), "flops": 2 * case["tokens"] * hkv * d}
    if case["op"] == "write":  # the values in, the cache written and read, the values out
        return {"bytes": case["tokens"] * (2 * token + 4 * hkv * d * size + 16), "flops": 10 * case["tokens"] * hkv * d}
    m, keys, pairs = case["queries"], 0, 0
    for n in _lens(case):
        seen = [max(0, n - m + i + 1) for i in range(m)]
        low = max(0, seen[0] - case["window"]) if case["window"] else 0
        keys += max(0, n - low)
        pairs += sum(min(c, case["window"]) if case["window"] else c for c in seen)
    rows = case["batch"] * m * case["hq"]
    return {"bytes": keys * token + 2 * rows * d * size + 4 * case["batch"] + 4 * keys // case["page"],
            "flops": 4 * pairs * case["hq"] * d}


# --------------------------------------------------------------------------- 64 bits

@functools.lru_cache(maxsize=None)
def _places(d, qt, part, start):
    """Byte, shift and scale byte of each token and dim of a group, as the layout is defined: lane by lane of the reader's tiles."""
    nb, size, widest = d // BLOCK, (32 if qt == "q8" else 16), (2 if qt == "q8" else 4)
    byte, shift = ([[0] * d for _ in range(GROUP)] for _ in range(2))
    runs, left, n = [], nb, widest
    while left:
        if n <= left:
            runs.append(n)
            left -= n
        else:
            n //= 2
    at, block, unit = start, 0, 4 if qt == "q8" else 2
    for n in runs:
        for lane in range(32):
            g, t = lane // 4, lane % 4
            for r in range(n):
                dim = (block + r) * BLOCK
                for k in range(4):
                    if part == "v":  # the lane's tokens are t, t + 4, t + 8, t + 12; its dims are 2g, 2g + 1 of each half
                        tok = t + 4 * k
                        chunk = at + ((g // 4 * 64 + tok * 4 + g % 4) * 8 if n == widest else (tok * 8 + g) * n * unit)
                        for half in range(2):
                            for e in range(2):
                                x = dim + half * 16 + 2 * g + e
                                if qt == "q8":
                                    byte[tok][x] = chunk + r * 4 + half * 2 + e
                                else:
                                    byte[tok][x], shift[tok][x] = chunk + r * 2 + e, 4 * half
                    elif k < 2:  # the lane's keys are column g of either half of the group; its dims are 4t .. 4t + 3 of each half
                        tok = g // 2 + 4 * (g % 2) + 8 * k
                        for half in range(2):
                            for e in range(4):
                                x = dim + half * 16 + 4 * t + e
                                row = (8 * k + g) * 4 + t
                                if qt == "q8":
                                    byte[tok][x] = at + (row * n + r) * 8 + half * 4 + e
                                else:
                                    byte[tok][x], shift[tok][x] = at + (row * n + r) * 4 + e, 4 * half
        at += n * size * GROUP
        block += n
    scale = [[at + ((tok % 4) * nb + x // BLOCK) * 8 + tok // 4 * 2 for x in range(d)] for tok in range(GROUP)]
    return tuple(torch.tensor(v) for v in (byte, shift, scale))


def _decode(raw, d, qt, part, start):
    """Bytes [..., group bytes] -> fp64 [..., 16, d]."""
    byte, shift, scale = (v.to(raw.device) for v in _places(d, qt, part, start))
    q = raw[..., byte].to(torch.int32)
    q = torch.where(q > 127, q - 256, q) if qt == "q8" else ((q >> shift) & 15) - 8
    bits = raw[..., scale].to(torch.int32) | (raw[..., scale + 1].to(torch.int32) << 8)
    return q.double() * bits.to(torch.int16).view(torch.float16).double()


def _exact_quantised(x, qt):
    """The values that a quantised row stands for. The codes are defined in binary32 steps; their products with the scale are exact."""
    import numpy as np

    f = np.float32
    x = x.float().cpu().numpy().reshape(*x.shape[:-1], -1, BLOCK)
    mag = np.abs(x)
    big = np.take_along_axis(x, mag.argmax(-1)[..., None], -1)  # numpy's argmax is the first of equals
    d = (np.abs(big) / f(127)).astype(f) if qt == "q8" else (big / f(-8)).astype(f)
    with np.errstate(divide="ignore"):
        inv = np.where(d == 0, f(0), f(1) / d).astype(f)
    y = (x * inv).astype(f)
    if qt == "q8":
        q = np.copysign(np.floor(np.abs(y.astype(np.float64)) + 0.5), y).clip(-127, 127)
    else:
        q = np.floor((y + f(8.5)).astype(f)).clip(0, 15).astype(np.float64) - 8
    return torch.from_numpy((q * d.astype(np.float16).astype(np.float64)).reshape(*x.shape[:-2], -1))


def exact(case, seed):
    s = prepare(case, seed)
    if s.op == "write":
        return _exact_quantised(s.k, s.kt), _exact_quantised(s.v, s.vt)
    cut = _part(s.d, s.kt)
    groups = s.page // GROUP
    cache = s.cache.view(s.pages, s.hkv, groups, -1)

    def tokens(which, at):  # fp64 [n, hkv, d] of n slots
        held, inverse = torch.unique(at // GROUP, return_inverse=True)
        return _decode(cache[held // groups, :, held % groups], s.d, *which)[inverse, :, at % GROUP]

    parts = ((s.kt, "k", 0), (s.vt, "v", cut))
    if s.op == "read":
        return tuple(tokens(p, s.slots) for p in parts)
    m, ratio = s.q.shape[1], s.hq // s.hkv
    out = torch.zeros(s.q.shape, dtype=torch.float64, device=s.q.device)
    for b, n in enumerate(_lens(case)):
        low = max(0, n - m + 1 - s.window) if s.window else 0
        pos = torch.arange(low, n, device=s.q.device)
        if not n:
            continue
        at = s.table[b, pos // s.page].long() * s.page + pos % s.page
        k, v = (tokens(p, at) for p in parts)
        for i in range(m):
            last = n - m + i
            keep = (pos <= last) & (pos > last - s.window if s.window else pos >= 0)
            if last < 0:
                continue
            for h in range(s.hkv):
                q = s.q[b, i, h * ratio:(h + 1) * ratio].double()
                w = torch.softmax(q @ k[keep, h].T * s.scale, -1)
                out[b, i, h * ratio:(h + 1) * ratio] = w @ v[keep, h]
    return out
