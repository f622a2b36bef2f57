"""The operators of the per-stream token cache as cases that can be timed and checked.

A stream's audio reaches a decoder as rows that arrive chunk by chunk.  Four operators
carry a chunk through the stream's paged key / value cache:

  append  turns the chunk's queries and keys by their positions and writes its keys and
          values into the stream's pages;
  attend  attends from the chunk's queries to everything cached, the chunk included;
  weigh   adds up the attention weight that each cached key received;
  evict   keeps the keys of largest weight and the newest ones, in other pages.

``run`` computes a case in its plain form with elementary torch operations in float32
or, where ``own`` is true, through the calls that a user of this package makes.
``exact`` computes it from the definition in float64.

Sizes: 16 query heads over 8 key heads of 128 dimensions are the decoder's, 20 heads of
64 dimensions with a window of 750 keys the causal audio tower's, 1024 streams that push
80 ms each are the streaming workload's, 375 tokens are 30 s of audio at 12.5 tokens a
second, and 65,536 tokens the decoder's context for a recording of 87 minutes.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _case(name, op, streams, new, cached, hq, hkv, d, page, half="bf16", **more):
    c = {"name": name, "op": op, "streams": streams, "new_lo": new[0], "new_hi": new[1], "cached_lo": cached[0],
         "cached_hi": cached[1], "hq": hq, "hkv": hkv, "d": d, "page": page, "half": half}
    c.update(more)
    return c


def listed():
    return [
        # one new decoder token for each of 1024 live streams, the angles stretched for a long context: runs every step
        _case("append one token", "append", 1024, (1, 1), (0, 64), 16, 8, 128, 16, rot=128, interleaved=False,
              scaling="ramp", far=60000),
        # 30 s chunks of uneven length into the audio tower's cache, pairs side by side, half of the head turned
        _case("append ragged chunks", "append", 64, (1, 375), (0, 375), 20, 20, 64, 32, "fp16", rot=32,
              interleaved=True, scaling="linear", far=100000),
        # one live caption stream: a single token against the audio tower's window; all latency
        _case("attend one stream", "attend", 1, (1, 1), (900, 900), 20, 20, 64, 16, window=750, causal=True, lse=False),
        # the decode step of 1024 streams of very different age
        _case("attend decode", "attend", 1024, (1, 1), (1, 1500), 16, 8, 128, 16, window=0, causal=True, lse=False),
        # the decode step of a few recordings of up to 87 minutes: one long axis, few rows
        _case("attend long decode", "attend", 8, (1, 1), (40000, 65535), 16, 8, 128, 64, window=0, causal=True,
              lse=False),
        # 160 ms pushes (16 rows) of 256 streams through the audio tower's window
        _case("attend windowed push", "attend", 256, (16, 16), (0, 1500), 20, 20, 64, 32, "fp16", window=750,
              causal=True, lse=False),
        # 30 s chunks of uneven length, some streams new and some with a few minutes behind them
        _case("attend ragged chunks", "attend", 48, (1, 375), (0, 2000), 16, 8, 128, 16, window=0, causal=True,
              lse=True),
        # the last piece of an 87 minute prompt: the arithmetic of a long chunk over a long cache
        _case("attend long chunk", "attend", 1, (4096, 4096), (61440, 61440), 16, 8, 128, 64, window=0, causal=True,
              lse=True),
        # the weights of one decode step, taken for streams whose caches are about to be cut
        _case("weigh decode", "weigh", 256, (1, 1), (500, 4000), 16, 8, 128, 16, window=0, causal=True, decay=0.99),
        # the weights that a chunk of prompt gives to a cache of some minutes
        _case("weigh chunks", "weigh", 4, (900, 1100), (4000, 9000), 16, 8, 128, 64, "fp16", window=0, causal=True,
              decay=1.0),
        # live streams cut to the newest minute and what mattered before
        _case("evict live streams", "evict", 256, (0, 0), (600, 2500), 16, 8, 128, 16, budget=750, recent=250),
        # two long recordings cut to a quarter of the context
        _case("evict long streams", "evict", 2, (0, 0), (60000, 65536), 16, 8, 128, 64, budget=16384, recent=1024),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the ranges above: any operator, type, head layout, page size, raggedness."""
    op = rng.choice(["append", "attend", "attend", "attend", "weigh", "evict"])
    hq, hkv, d = rng.choice([(16, 8, 128), (20, 20, 64), (14, 2, 64), (16, 16, 64), (16, 8, 64), (8, 1, 128)])
    c = {"op": op, "hq": hq, "hkv": hkv, "d": d, "page": rng.choice([16, 32, 64, 128]),
         "half": rng.choice(["bf16", "fp16"])}
    if op == "append":
        tokens = _log(rng, 1, 16000)
        c["streams"] = _log(rng, 1, min(tokens, 1024))
        each = max(1, tokens // c["streams"])
        c.update(new_lo=rng.choice([each, 1]), new_hi=each, cached_lo=0, cached_hi=_log(rng, 1, 300),
                 rot=rng.choice([d, d // 2]), interleaved=rng.random() < 0.5,
                 scaling=rng.choice(["none", "linear", "ramp"]), far=_log(rng, 1, 100000))
    elif op == "evict":
        length = _log(rng, 200, 65536)
        c["streams"] = _log(rng, 1, max(1, min(512, 400000 // length)))
        budget = max(1, int(length * rng.uniform(0.05, 0.9)))
        c.update(new_lo=0, new_hi=0, cached_lo=length // 2, cached_hi=length, budget=budget,
                 recent=int(budget * rng.uniform(0.0, 0.9)))
    else:
        each = rng.choice([1, 1, rng.randint(2, 16), _log(rng, 16, 2000)])
        length = _log(rng, 1, 60000)
        room = 300000 if each <= 16 else max(60000, 40000000 // each) if op == "attend" else 120000
        c["streams"] = _log(rng, 1, max(1, min(1024, room // (length + each))))
        c.update(new_lo=rng.choice([each, 1]), new_hi=each, cached_lo=rng.choice([0, length]), cached_hi=length,
                 window=rng.choice([0, 0, rng.randint(20, 2000)]), causal=rng.random() < 0.8)
        if op == "attend":
            c["lse"] = rng.random() < 0.5
        else:
            c["decay"] = rng.choice([1.0, 0.9])
    return c


def _lengths(case):
    """New and total tokens of every stream: part of the case, the same for every seed."""
    r = random.Random("%s %d %d %d" % (case["op"], case["streams"], case["new_hi"], case["cached_hi"]))
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["streams"])]
    return new, [n + r.randint(case["cached_lo"], case["cached_hi"]) for n in new]


def _seen(case, n, length, i):
    """Keys [lo, hi) that new token i of a stream sees."""
    at = length - n + i
    hi = min(length, at + 1) if case["causal"] else length
    return (max(0, at + 1 - case["window"]) if case["window"] else 0), hi


def work(case):
    new, lens = _lengths(case)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    t, row = sum(new), d * 2
    if case["op"] == "append":
        return {"bytes": 2 * t * (hq + 2 * hkv) * row + 4 * t, "flops": 3 * t * (hq + hkv) * case["rot"]}
    if case["op"] == "evict":
        kept = sum(min(x, case["budget"]) for x in lens)
        return {"bytes": hkv * (4 * sum(lens) + kept * (4 * row + 4) + 4 * case["streams"] * case["budget"]),
                "flops": hkv * sum(lens)}
    pairs = keys = 0
    for n, length in zip(new, lens):
        first, last = _seen(case, n, length, 0), _seen(case, n, length, n - 1)
        keys += last[1] - first[0]
        pairs += sum(h - l for l, h in (_seen(case, n, length, i) for i in range(n)))
    if case["op"] == "attend":
        out = 2 * t * hq * row + (4 * t * hq if case["lse"] else 0)
        return {"bytes": out + 2 * keys * hkv * row, "flops": 4 * pairs * hq * d}
    return {"bytes": t * hq * (row + 4) + keys * hkv * row + 8 * sum(lens) * hkv, "flops": 2 * pairs * hq * d}


def _table(lens, page, dev, gen, spare=3):
    """Pages handed out in a shuffled order, as a pool looks after some hours."""
    need = [-(-x // page) for x in lens]
    order = torch.randperm(sum(need) + spare, device=dev, generator=gen).to(torch.int32)
    table = torch.zeros(len(lens), max(max(need), 1), dtype=torch.int32, device=dev)
    at = torch.tensor([0] + need, device=dev).cumsum(0)
    col = torch.arange(table.shape[1], device=dev)
    live = col < torch.tensor(need, device=dev)[:, None]
    table[live] = order[(at[:-1, None] + col)[live]]
    return table, sum(need) + spare


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    new, lens = _lengths(case)
    hq, hkv, d, page, half = case["hq"], case["hkv"], case["d"], case["page"], TYPES[case["half"]]
    s = {"case": case, "new": new, "lens_host": lens, "t": sum(new)}
    offs = [0]
    for n in new:
        offs.append(offs[-1] + n)
    s["offsets_host"] = offs
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["table"], pages = _table(lens, page, dev, gen)
    s["k_pages"] = torch.randn(pages, hkv, page, d, device=dev, generator=gen, dtype=half)
    s["v_pages"] = torch.randn(pages, hkv, page, d, device=dev, generator=gen, dtype=half)
    scale = 1.0 / math.sqrt(d)
    if case["op"] == "append":
        # queries, keys and values are slices of one projection's rows, as a decoder block has them
        s["qkv"] = torch.randn(s["t"], (hq + 2 * hkv) * d, device=dev, generator=gen, dtype=half)
        begin = torch.randint(0, case["far"], (case["streams"],), device=dev, generator=gen)
        step = torch.cat([torch.arange(n, device=dev) for n in new])
        own_row = torch.repeat_interleave(torch.arange(case["streams"], device=dev), torch.tensor(new, device=dev))
        s["positions"] = (begin[own_row] + step).to(torch.int32)
        slot = torch.tensor([x - n for x, n in zip(lens, new)], device=dev)[own_row] + step
        s["row_page"] = s["table"][own_row, slot // page].long()
        s["row_slot"] = slot % page
    elif case["op"] == "evict":
        # weights as attention leaves them: a few large, many small, some keys never looked at (exact ties)
        w = torch.exp(2.0 * torch.randn(pages, hkv, page, device=dev, generator=gen))
        s["mass"] = torch.where(torch.rand(pages, hkv, page, device=dev, generator=gen) < 0.2, torch.zeros_like(w), w)
        kept = [min(x, case["budget"]) for x in lens]
        s["to_table"], to_pages = _table(kept, page, dev, gen)
        s["to_k"] = torch.zeros(to_pages, hkv, page, d, device=dev, dtype=half)
        s["to_v"] = torch.zeros(to_pages, hkv, page, d, device=dev, dtype=half)
        s["to_mass"] = torch.zeros(to_pages, hkv, page, device=dev)
        s["to_lens"] = torch.zeros(case["streams"], dtype=torch.int32, device=dev)
    else:
        # scores with a deviation of 2: a few keys carry a row, as in a trained block
        s["q"] = (2.0 * torch.randn(s["t"], hq, d, device=dev, generator=gen)).to(half)
        if case["op"] == "weigh":
            s["lse"] = _attend_plain(s, scale)[1]
            s["mass"] = torch.rand(pages, hkv, page, device=dev, generator=gen)
            s["to_mass"] = torch.zeros_like(s["mass"])
    if own:
        import log_mel_spectrogram_logmel_b200 as lm
        more = {}
        if case["op"] == "append":
            more = dict(rotary_dim=case["rot"], interleaved=case["interleaved"], rotary_base=ROPE_BASE,
                        **SCALINGS[case["scaling"]])
        plan = lm.CachePlan(hq, hkv, d, page, dtype=half, **more)
        s["cache"] = lm.TokenCache(plan, s["k_pages"], s["v_pages"], s["table"], s["lens"], mass=s.get("mass"))
        if case["op"] == "evict":
            s["to"] = lm.TokenCache(plan, s["to_k"], s["to_v"], s["to_table"], s["to_lens"], mass=s["to_mass"])
        s["offsets"] = None if case["new_lo"] == case["new_hi"] else offs
    return s


ROPE_BASE = 1000000.0
SCALINGS = {"none": {}, "linear": {"rotary_scaling": "linear", "rotary_factor": 4.0},
            "ramp": {"rotary_scaling": "ramp", "rotary_factor": 4.0, "rotary_context": 32768}}


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    case, cache = s["case"], s["cache"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "append":
        x = s["qkv"].view(s["t"], hq + 2 * hkv, d)
        q = cache.append(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], s["offsets"], positions=s["positions"])
        return q, s["k_pages"], s["v_pages"]
    if case["op"] == "attend":
        return cache.attend(s["q"], s["offsets"], causal=case["causal"], window=case["window"], return_lse=case["lse"])
    if case["op"] == "weigh":
        return cache.weigh(s["q"], s["lse"], s["offsets"], causal=case["causal"], window=case["window"],
                           decay=case["decay"], out=s["to_mass"])
    kept = cache.evict(s["to"], case["budget"], recent=case["recent"])
    return kept, s["to_k"], s["to_v"], s["to_mass"], s["to_lens"]


# --- plain forms ------------------------------------------------------------------------------------------


def _run_plain(s):
    case = s["case"]
    if case["op"] == "append":
        return _append_plain(s)
    if case["op"] == "attend":
        out, lse = _attend_plain(s, 1.0 / math.sqrt(case["d"]))
        return (out, lse) if case["lse"] else out
    if case["op"] == "weigh":
        return _weigh_plain(s, 1.0 / math.sqrt(case["d"]))
    return _evict_plain(s)


def _frequencies(case, dev):
    """Radians a position for every pair, in float64, and the factor on the turned pair's length."""
    rot = case["rot"]
    i = torch.arange(rot // 2, device=dev, dtype=torch.float64)
    inv = ROPE_BASE ** (-2.0 * i / rot)
    if case["scaling"] == "none":
        return inv, 1.0
    more = SCALINGS[case["scaling"]]
    if case["scaling"] == "linear":
        return inv / more["rotary_factor"], 1.0
    # pairs that turn more than 32 times within the trained context stay, those below one turn are slowed by
    # the factor, and those between are mixed in proportion to their index
    def index_of(turns):
        return rot * math.log(more["rotary_context"] / (turns * 2 * math.pi)) / (2 * math.log(ROPE_BASE))
    low, high = max(math.floor(index_of(32.0)), 0), min(math.ceil(index_of(1.0)), rot - 1)
    slow = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
    return inv * (1 - slow) + inv / more["rotary_factor"] * slow, 0.1 * math.log(more["rotary_factor"]) + 1.0


def _turn(case, x, cos, sin):
    rot = case["rot"]
    y = x.float()
    if case["interleaved"]:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, y[..., rot:]], -1).to(x.dtype)


def _append_plain(s):
    case = s["case"]
    hq, hkv = case["hq"], case["hkv"]
    x = s["qkv"].view(s["t"], hq + 2 * hkv, case["d"])
    inv, length = _frequencies(case, x.device)
    angle = s["positions"].double()[:, None] * inv
    cos, sin = (length * angle.cos()).float()[:, None], (length * angle.sin()).float()[:, None]
    s["k_pages"][s["row_page"], :, s["row_slot"]] = _turn(case, x[:, hq:hq + hkv], cos, sin)
    s["v_pages"][s["row_page"], :, s["row_slot"]] = x[:, hq + hkv:]
    return _turn(case, x[:, :hq], cos, sin), s["k_pages"], s["v_pages"]


def _keys(pool, table, page, length):
    """The cached rows of some streams, [streams, heads, length, d] in float32."""
    x = pool[table[:, :-(-length // page)].long()].transpose(1, 2).flatten(2, 3)
    return x[:, :, :length].float()


def _blocks(s):
    """Streams that can go through one product: runs of equal token counts whose scores stay moderate."""
    case, new, lens = s["case"], s["new"], s["lens_host"]
    a = 0
    while a < len(new):
        b, top = a + 1, lens[a]
        while b < len(new) and new[b] == new[a] and (b - a + 1) * max(top, lens[b]) * case["hkv"] * case["d"] <= 1 << 27:
            top = max(top, lens[b])
            b += 1
        if new[a]:
            yield a, b, new[a], top
        a = b


def _mask(s, a, b, i0, i1, n, top):
    case = s["case"]
    lens = s["lens"][a:b, None, None].long()
    key = torch.arange(top, device=lens.device)
    at = lens - n + torch.arange(i0, i1, device=lens.device)[:, None]
    seen = (key < lens) & ((key <= at) if case["causal"] else (key >= 0))
    return seen & (key > at - case["window"]) if case["window"] else seen


def _scores(s, scale, a, b, n, i0, i1, keys, top):
    """Scores [streams, key heads, group, tokens, keys], minus infinity where a token does not see the key."""
    case = s["case"]
    hkv, g = case["hkv"], case["hq"] // case["hkv"]
    q = s["q"][s["offsets_host"][a]:s["offsets_host"][b]].view(b - a, n, hkv, g, case["d"])[:, i0:i1].float()
    q = q.permute(0, 2, 3, 1, 4).reshape(b - a, hkv, g * (i1 - i0), case["d"])
    x = torch.matmul(q, keys.transpose(-1, -2)).mul_(scale).view(b - a, hkv, g, i1 - i0, top)
    return x.masked_fill_(~_mask(s, a, b, i0, i1, n, top)[:, None, None], -math.inf)


def _attend_plain(s, scale):
    case = s["case"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    out = torch.empty_like(s["q"])
    lse = torch.empty(s["t"], hq, device=out.device)
    for a, b, n, top in _blocks(s):
        k = _keys(s["k_pages"], s["table"][a:b], case["page"], top)
        v = _keys(s["v_pages"], s["table"][a:b], case["page"], top)
        piece = max(1, (1 << 28) // ((b - a) * hq * top))
        for i0 in range(0, n, piece):
            i1 = min(n, i0 + piece)
            x = _scores(s, scale, a, b, n, i0, i1, k, top)
            high = x.amax(-1, keepdim=True).clamp(min=-3e38)
            p = x.sub_(high).exp_()
            total = p.sum(-1, keepdim=True)
            o = torch.matmul(p.flatten(2, 3), v).view(b - a, hkv, hq // hkv, i1 - i0, d) / total.clamp(min=1e-30)
            rows = slice(s["offsets_host"][a], s["offsets_host"][b])
            out[rows].view(b - a, n, hq, d)[:, i0:i1] = o.permute(0, 3, 1, 2, 4).flatten(2, 3).to(out.dtype)
            lse[rows].view(b - a, n, hq)[:, i0:i1] = (high + total.log())[..., 0].permute(0, 3, 1, 2).flatten(2, 3)
    return out, lse


def _weigh_plain(s, scale):
    case = s["case"]
    hq, hkv, page = case["hq"], case["hkv"], case["page"]
    for a, b, n, top in _blocks(s):
        k = _keys(s["k_pages"], s["table"][a:b], page, top)
        w = torch.zeros(b - a, hkv, top, device=k.device)
        piece = max(1, (1 << 28) // ((b - a) * hq * top))
        for i0 in range(0, n, piece):
            i1 = min(n, i0 + piece)
            x = _scores(s, scale, a, b, n, i0, i1, k, top)
            l = s["lse"][s["offsets_host"][a]:s["offsets_host"][b]].view(b - a, n, hkv, hq // hkv)[:, i0:i1]
            w += x.sub_(l.permute(0, 2, 3, 1)[..., None]).exp_().sum((2, 3))
        key = torch.arange(top, device=k.device)
        live = key < s["lens"][a:b, None]
        pages = s["table"][a:b].long()[:, key // page][live]
        slots = (key % page).expand(b - a, top)[live]
        was = s["mass"][pages, :, slots]
        s["to_mass"][pages, :, slots] = case["decay"] * was + w.transpose(1, 2)[live]
    return s["to_mass"]


def _evict_plain(s):
    case, lens, page = s["case"], s["lens_host"], s["case"]["page"]
    budget, recent, hkv = case["budget"], case["recent"], case["hkv"]
    dev = s["k_pages"].device
    kept = torch.full((case["streams"], hkv, budget), -1, dtype=torch.int32, device=dev)
    head = torch.arange(hkv, device=dev)[:, None]
    for i, length in enumerate(lens):
        m = min(length, budget)
        slot = torch.arange(length, device=dev)
        at = s["table"][i].long()[slot // page]
        w = s["mass"][at, :, slot % page].t()
        newest = slot >= length - recent
        w = torch.where(newest, torch.full_like(w, math.inf), w)
        order = torch.sort(w, dim=1, descending=True, stable=True).indices[:, :m]
        keep = torch.sort(order, dim=1).values
        kept[i, :, :m] = keep.int()
        src, src_slot = at[keep], keep % page
        to = torch.arange(m, device=dev)
        dst, dst_slot = s["to_table"][i].long()[to // page], to % page
        for a, b in (("k_pages", "to_k"), ("v_pages", "to_v"), ("mass", "to_mass")):
            s[b][dst, head, dst_slot] = s[a][src, head, src_slot]
        s["to_lens"][i] = m
    return kept, s["to_k"], s["to_v"], s["to_mass"], s["to_lens"]


# --- the definition in float64 ------------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return {"append": _append_exact, "attend": _attend_exact, "weigh": _weigh_exact, "evict": _evict_exact}[
            case["op"]](case, s)


def _append_exact(case, s):
    hq, hkv, d, rot = case["hq"], case["hkv"], case["d"], case["rot"]
    x = s["qkv"].double().view(s["t"], hq + 2 * hkv, d)
    inv = torch.tensor([ROPE_BASE ** (-2.0 * j / rot) for j in range(rot // 2)], dtype=torch.float64)
    length = 1.0
    if case["scaling"] == "linear":
        inv = inv / 4.0
    elif case["scaling"] == "ramp":
        first = rot * math.log(32768 / (32 * 2 * math.pi)) / (2 * math.log(ROPE_BASE))
        last = rot * math.log(32768 / (2 * math.pi)) / (2 * math.log(ROPE_BASE))
        first, last = max(math.floor(first), 0), min(math.ceil(last), rot - 1)
        part = [min(max((j - first) / max(last - first, 0.001), 0.0), 1.0) for j in range(rot // 2)]
        part = torch.tensor(part, dtype=torch.float64)
        inv = inv * (1 - part) + inv * part / 4.0
        length = 1.0 + 0.1 * math.log(4.0)
    angle = torch.outer(s["positions"].double(), inv.to(x.device))
    turn = torch.polar(torch.full_like(angle, length), angle)[:, None]
    y = x.clone()
    first = slice(0, rot, 2) if case["interleaved"] else slice(0, rot // 2)
    second = slice(1, rot, 2) if case["interleaved"] else slice(rot // 2, rot)
    z = torch.complex(x[:, :hq + hkv, first].contiguous(), x[:, :hq + hkv, second].contiguous()) * turn
    y[:, :hq + hkv, first], y[:, :hq + hkv, second] = z.real, z.imag
    k_pages, v_pages = s["k_pages"].double(), s["v_pages"].double()
    k_pages[s["row_page"], :, s["row_slot"]] = y[:, hq:hq + hkv]
    v_pages[s["row_page"], :, s["row_slot"]] = y[:, hq + hkv:]
    return y[:, :hq].contiguous(), k_pages, v_pages


def _stream_rows(case, s, i, pool):
    at = torch.arange(s["lens_host"][i], device=pool.device)
    return pool[s["table"][i].long()[at // case["page"]], :, at % case["page"]].double().transpose(0, 1)


def _weights_exact(case, s, i):
    """For stream i, pieces (first token, weights [key heads, group x tokens, keys] in float64, log of their sum)."""
    n, length = s["new"][i], s["lens_host"][i]
    hkv, g = case["hkv"], case["hq"] // case["hkv"]
    keys = _stream_rows(case, s, i, s["k_pages"])
    piece = max(1, (1 << 27) // (case["hq"] * length))
    for t0 in range(0, n, piece):
        t1 = min(n, t0 + piece)
        rows = s["q"][s["offsets_host"][i] + t0:s["offsets_host"][i] + t1].double()
        rows = rows.view(t1 - t0, hkv, g, case["d"]).permute(1, 2, 0, 3).flatten(1, 2)
        x = rows @ keys.mT / math.sqrt(case["d"])
        bounds = torch.tensor([_seen(case, n, length, t) for t in range(t0, t1)], device=keys.device).repeat(g, 1)
        at = torch.arange(length, device=keys.device)
        hidden = (at < bounds[:, :1]) | (at >= bounds[:, 1:])
        x = torch.where(hidden, -math.inf, x)
        total = torch.logsumexp(x, -1, keepdim=True)
        yield t0, t1, x, total


def _attend_exact(case, s):
    hq, d = case["hq"], case["d"]
    out = torch.empty(s["t"], hq, d, dtype=torch.float64, device=s["q"].device)
    lse = torch.empty(s["t"], hq, dtype=torch.float64, device=s["q"].device)
    for i in range(case["streams"]):
        if not s["new"][i]:
            continue
        values = _stream_rows(case, s, i, s["v_pages"])
        for t0, t1, x, total in _weights_exact(case, s, i):
            o = torch.exp(x - total) @ values
            rows = slice(s["offsets_host"][i] + t0, s["offsets_host"][i] + t1)
            out[rows] = o.unflatten(1, (-1, t1 - t0)).permute(2, 0, 1, 3).flatten(1, 2)
            lse[rows] = total[..., 0].unflatten(1, (-1, t1 - t0)).permute(2, 0, 1).flatten(1, 2)
    return (out, lse) if case["lse"] else out


def _weigh_exact(case, s):
    result = s["to_mass"].double()
    hkv, g = case["hkv"], case["hq"] // case["hkv"]
    for i in range(case["streams"]):
        w = 0.0
        for t0, t1, x, _ in _weights_exact(case, s, i):
            l = s["lse"][s["offsets_host"][i] + t0:s["offsets_host"][i] + t1].double()
            w = w + torch.exp(x - l.view(t1 - t0, hkv, g).permute(1, 2, 0).flatten(1)[..., None]).sum(1)
        if s["new"][i]:
            at = torch.arange(s["lens_host"][i], device=result.device)
            page, slot = s["table"][i].long()[at // case["page"]], at % case["page"]
            result[page, :, slot] = case["decay"] * s["mass"][page, :, slot].double() + w.t()
    return result


def _evict_exact(case, s):
    budget, page, hkv = case["budget"], case["page"], case["hkv"]
    kept = torch.full((case["streams"], hkv, budget), -1, dtype=torch.int32)
    k, v, mass = s["to_k"].double(), s["to_v"].double(), s["to_mass"].double()
    to_lens = torch.zeros(case["streams"], dtype=torch.int32)
    for i, length in enumerate(s["lens_host"]):
        m = min(budget, length)
        to_lens[i] = m
        at = torch.arange(length, device=k.device)
        where, slot = s["table"][i].long()[at // page], at % page
        weight = s["mass"][where, :, slot].cpu().numpy()
        to = torch.arange(m, device=k.device)
        for h in range(hkv):
            old = max(0, length - case["recent"])
            best = (-weight[:old, h]).argsort(kind="stable")[:max(0, m - (length - old))].tolist()
            keep = sorted(best + list(range(max(old, length - m), length) if length - old > m else range(old, length)))
            keep = torch.tensor(keep)
            kept[i, h, :m] = keep.int()
            keep = keep.to(k.device)
            dst, dst_slot = s["to_table"][i].long()[to // page], to % page
            k[dst, h, dst_slot] = s["k_pages"][where[keep], h, slot[keep]].double()
            v[dst, h, dst_slot] = s["v_pages"][where[keep], h, slot[keep]].double()
            mass[dst, h, dst_slot] = s["mass"][where[keep], h, slot[keep]].double()
    return kept, k, v, mass, to_lens
