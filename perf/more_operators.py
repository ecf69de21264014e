"""Many continuations of one cached prompt, as measured cases.

What generation over the paged FP8 cache needs around its attention: rotary
positions of queries and keys (alone, or with the keys and values quantized into
the cache in the same step), the pages of the cache (forked for another
continuation, reserved for new tokens, given back, copied, moved together), and
attention of a batch whose sequences share long prefixes, each read once for all.
``run`` computes each in its plain form, or, with ``own`` set, calls the framework.

A batch is B sequences.  Sequence b holds ``kv_len[b]`` tokens in the cache; its
last n_b = cu[b+1] - cu[b] tokens are those of the call, packed in rows cu[b] ..
cu[b+1] - 1.  Position p lies in page table[b][p // page], at p % page.  A pool
counts in refs[p] the table entries that name page p; bit p % 32 of free[p // 32]
is set where there is none.
"""
import math
import random

import torch

own = False

CLIP = 75600   # 21 x 45 x 80 latent tokens
FRAME = 3600   # one latent frame of 45 x 80 tokens


def listed():
    return [
        # serving: the queries of one new token of each sequence, all channels
        dict(name="rotate, one token each", op="rotate", T=100, H=32, d=128, rot=128, layout="halves", scaling="none", base=10000.0, factor=1.0, far=8192, inverse=False),
        # the way back through the rotation of a long prompt's keys: half of the channels, neighbouring pairs, a context stretched eight times
        dict(name="rotate back, a long prompt", op="rotate", T=20011, H=40, d=128, rot=64, layout="pairs", scaling="ramp", base=500000.0, factor=8.0, far=262144, inverse=True),
        # serving: a new token of each sequence on its way into the cache, grouped heads
        dict(name="rotate and append, a token", op="append", B=100, n_lo=1, n_hi=1, kv_lo=1, kv_hi=8192, H=8, G=4, d=128, page=16, rot=128, layout="halves", scaling="none",
             base=10000.0, factor=1.0, lens=21),
        # prompts of different lengths, one of them empty, far into a stretched context
        dict(name="rotate and append, prompts", op="append", B=7, n_lo=0, n_hi=6007, kv_lo=6007, kv_hi=131072, H=8, G=5, d=128, page=64, rot=96, layout="halves",
             scaling="ramp", base=1000000.0, factor=4.0, lens=22),
        # 64 continuations of a prompt begin: the old ones' pages are given back, the prompt is forked, and each gets a page of its own for its first token
        dict(name="pages, a prompt forked", op="fork", B=1, N=64, kv_lo=8183, kv_hi=8183, n=1, H=8, d=128, page=64, used=0.3, pages=4096, lens=23),
        # drafts of 512 sequences are taken back to what was accepted, and pages reserved for the next ones
        dict(name="pages, drafts", op="drafts", B=512, N=0, kv_lo=100, kv_hi=4000, n=8, H=1, d=64, page=16, used=0.7, pages=190001, lens=24),
        # half of a pool's pages moved together after many sequences have ended
        dict(name="pages, moved together", op="compact", B=40, N=0, kv_lo=2000, kv_hi=16000, n=0, H=8, d=128, page=64, used=0.5, pages=12000, lens=25),
        # one sequence's pages to another pool
        dict(name="pages, to another pool", op="copy", B=1, N=0, kv_lo=20000, kv_hi=20000, n=0, H=4, d=64, page=32, used=0.5, pages=1500, lens=26),
        # the smallest: four continuations of a short prompt
        dict(name="shared, a short prompt", op="shared", B=4, N=1, p_lo=700, p_hi=700, s_lo=1, s_hi=60, n_lo=1, n_hi=1, H=2, G=2, d=64, page=16, causal=True, lens=27),
        # 100 continuations of a prompt of 8,000 tokens, one token each
        dict(name="shared, one token each", op="shared", B=100, N=1, p_lo=8000, p_hi=8000, s_lo=1, s_hi=900, n_lo=1, n_hi=1, H=8, G=4, d=128, page=16, causal=True, lens=28),
        # several prompts with continuations, a few drafted tokens each
        dict(name="shared, prompts with drafts", op="shared", B=60, N=5, p_lo=300, p_hi=30000, s_lo=7, s_hi=700, n_lo=1, n_hi=7, H=4, G=8, d=128, page=64, causal=True, lens=29),
        # two versions of the next latent frame over six frames that they have in common, 40 heads
        dict(name="shared, frames of a clip", op="shared", B=2, N=1, p_lo=6 * FRAME, p_hi=6 * FRAME, s_lo=FRAME, s_hi=FRAME, n_lo=FRAME, n_hi=FRAME, H=40, G=1, d=128, page=128,
             causal=False, lens=30),
    ]


def _between(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_rotation(rng, d):
    scaling = rng.choice(["none", "positions", "base", "ramp"])
    return dict(rot=rng.choice([r for r in (16, 32, 48, 64, 96, 128) if r <= d]), layout=rng.choice(["halves", "pairs"]), scaling=scaling, base=rng.choice([10000.0, 500000.0, 1000000.0]),
                factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 32.0]))


def draw(rng):
    op = rng.choice(["rotate", "append", "fork", "drafts", "compact", "copy", "shared", "shared", "shared"])
    d = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128, 256])
    lens = rng.randrange(1 << 30)
    if op == "rotate":
        H = rng.choice([1, 2, 3, 8, 24, 32, 40])
        return dict(op=op, T=_between(rng, 1, 800000 // H), H=H, d=d, far=_between(rng, 1, 4000000), inverse=rng.random() < 0.4, **_draw_rotation(rng, d))
    if op == "append":
        H, G = rng.choice([(1, 1), (2, 8), (3, 2), (8, 4), (8, 5), (24, 1), (40, 1)])
        kv_hi = _between(rng, 1, 100000)
        B = _between(rng, 1, max(1, min(200, 400000 // kv_hi)))
        n_hi = _between(rng, 1, max(1, min(kv_hi, 800000 // (B * H * G))))
        return dict(op=op, B=B, n_lo=rng.choice([0, 1, n_hi]), n_hi=n_hi, kv_lo=rng.choice([0, kv_hi // 2, kv_hi]), kv_hi=kv_hi, H=H, G=G, d=d, page=page, lens=lens,
                    **_draw_rotation(rng, d))
    if op != "shared":
        H = rng.choice([1, 2, 4, 8])
        kv_hi = _between(rng, 1, 30000)
        B = 1 if op == "copy" else _between(rng, 1, max(1, min(400, 300000 // kv_hi)))
        N = _between(rng, 1, max(1, min(300, 1000000 // kv_hi))) if op == "fork" else 0
        n = {"fork": rng.choice([1, 5]), "drafts": rng.choice([1, 3, 8, 40])}.get(op, 0)
        need = B * (-(-kv_hi // page) + 2 + n // page) + N * (2 + n // page)
        used = rng.choice([0.2, 0.5, 0.9])
        return dict(op=op, B=B, N=N, kv_lo=rng.choice([0, kv_hi // 2, kv_hi]), kv_hi=kv_hi, n=n, H=H, d=d, page=page, used=used, pages=int(need / used) + rng.randint(3, 99), lens=lens)
    H, G = rng.choice([(1, 1), (2, 8), (4, 3), (4, 8), (8, 4), (8, 5), (24, 1)])
    p_hi = _between(rng, 1, 60000)
    form = rng.choice(["token", "token", "few", "chunk"])
    n_hi = 1 if form == "token" else rng.randint(2, 9) if form == "few" else _between(rng, 10, 700)
    s_hi = n_hi + _between(rng, 1, 2000)
    B = _between(rng, 2, max(2, min(128, 3000000000 // (n_hi * (p_hi + s_hi) * H * G), 8000000 // ((p_hi + s_hi) * H))))
    return dict(op=op, B=B, N=_between(rng, 1, max(1, min(12, B // 2))), p_lo=rng.choice([0, p_hi // 2, p_hi]), p_hi=p_hi, s_lo=rng.choice([n_hi, s_hi]), s_hi=s_hi, n_lo=rng.choice([0, 1, n_hi]),
                n_hi=n_hi, H=H, G=G, d=d, page=page, causal=rng.random() < 0.7, lens=lens)


# ------------------------------------------------------------ what a case says


def _lengths(c):
    """Tokens in the cache and in the call of each sequence: the case alone gives them.  One is the longest."""
    rng = random.Random(c["lens"])
    kv = [rng.randint(c["kv_lo"], c["kv_hi"]) for _ in range(c["B"])]
    kv[rng.randrange(c["B"])] = c["kv_hi"]
    if c["op"] != "append":
        return kv, [c["n"]] * c["B"]
    n = [min(k, rng.randint(c["n_lo"], c["n_hi"])) for k in kv]
    if sum(n) == 0:
        n[kv.index(max(kv))] = min(c["n_hi"], max(kv))
    return kv, n


def _families(c):
    """Of a batch with shared prefixes: the sequences' groups (offsets), the groups' prefixes, and of each sequence
    its tokens in the cache and in the call."""
    rng = random.Random(c["lens"])
    cuts = sorted(rng.sample(range(1, c["B"]), c["N"] - 1)) if c["N"] > 1 else []
    groups = [0] + cuts + [c["B"]]
    prefix = [rng.randint(c["p_lo"], c["p_hi"]) for _ in range(c["N"])]
    prefix[rng.randrange(c["N"])] = c["p_hi"]
    kv, n = [], []
    for g, p in enumerate(prefix):
        for _ in range(groups[g + 1] - groups[g]):
            s = rng.randint(c["s_lo"], c["s_hi"])
            kv.append(p + s)
            n.append(min(s, rng.randint(c["n_lo"], c["n_hi"])))
    if sum(n) == 0:
        n[0] = min(c["n_hi"], kv[0] - prefix[0])
    return groups, prefix, kv, n


def _turns(c):
    """Radians a position of each pair of channels, in fp64 on the CPU, and what the rotated channels are multiplied by."""
    i = torch.arange(c["rot"] // 2, dtype=torch.float64)
    base, f = c["base"], c["factor"]
    if c["scaling"] == "base":
        base = base * f ** (c["rot"] / (c["rot"] - 2.0))
    w = base ** (-2.0 * i / c["rot"])
    if c["scaling"] == "positions":
        w = w / f
    if c["scaling"] != "ramp":
        return w, 1.0
    # channels that turn 32 times or more over the original 4,096 positions stay, those that turn once or less slow down
    keep = ((4096.0 * w / (2.0 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0)
    return w * keep + w / f * (1.0 - keep), 0.1 * math.log(f) + 1.0


def _random(shape, g):
    return torch.randn(shape, generator=g, device="cuda")


def _keys(rows, H, d, g):
    """Keys (and queries, and their gradients): N(0, 1) about a mean of each head and channel, as bf16."""
    return (_random((rows, H, d), g) + _random((1, H, d), g)).to(torch.bfloat16)


def _values(rows, H, d, g):
    """Values: N(0, 1), one token in a hundred times 20 on four channels, as bf16."""
    v = _random((rows, H, d), g)
    v[:, :, torch.randperm(d, generator=g, device="cuda")[:4]] *= torch.where(torch.rand((rows, 1, 1), generator=g, device="cuda") < 0.01, 20.0, 1.0)
    return v.to(torch.bfloat16)


def _codes(x):
    """[..., d] fp32 -> E4M3 codes (their bytes) and the fp32 scale of each row."""
    amax = x.abs().amax(-1, keepdim=True)
    inv = torch.where(amax > 0, 448.0 / amax, torch.zeros_like(amax))
    return (x * inv).to(torch.float8_e4m3fn).view(torch.uint8), (amax / 448.0)[..., 0]


def _cache(pages, c, g):
    """A filled pool."""
    H, d, page = c["H"], c["d"], c["page"]
    cache = {}
    for code, scale, make in (("K8", "sk", _keys), ("V8", "sv", _values)):
        # made for one head after the other: the fp32 parts of a large pool are large
        cache[code] = torch.empty((pages, H, page, d), dtype=torch.uint8, device="cuda")
        cache[scale] = torch.empty((pages, H, page), dtype=torch.float32, device="cuda")
        for h in range(H):
            x, s = _codes(make(pages * page, 1, d, g).view(pages, page, d).float())
            cache[code][:, h], cache[scale][:, h] = x, s
    return cache


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _offsets(n):
    starts = [0]
    for m in n:
        starts.append(starts[-1] + m)
    return _ints(starts)


def _table(need, cols, pages, g):
    """A table of sequences that hold `need` pages each, in random order of the pool."""
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    need = _ints(need)
    first = need.cumsum(0) - need
    at = torch.arange(cols, device="cuda")
    return torch.where(at < need[:, None], order[(first[:, None] + at).clamp(max=pages - 1)], -1).to(torch.int32)


def _free_bits(refs):
    """The words that say which pages no entry names."""
    bits = torch.zeros(-(-refs.numel() // 32) * 32, dtype=torch.int64, device="cuda")
    bits[:refs.numel()] = refs == 0
    words = (bits.view(-1, 32) << torch.arange(32, device="cuda")).sum(1)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)


def _pool(table, pages):
    refs = torch.bincount(table[table >= 0].long(), minlength=pages).to(torch.int32)
    return {"refs": refs, "free": _free_bits(refs)}


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case=c)
    if c["op"] in ("rotate", "append"):
        w, times = _turns(c)
        s["radians"] = w.cuda()
        # the same in turns, as 64-bit fixed-point fractions
        turns = torch.round(torch.remainder(w / (2.0 * math.pi), 1.0) * 2.0 ** 62).to(torch.int64) << 2
        s["rope"] = dict(turns=turns.cuda(), layout=c["layout"], magnitude=times)
    if c["op"] == "rotate":
        s["X"] = _keys(c["T"], c["H"], c["d"], g)
        s["pos"] = torch.randint(c["far"], (c["T"],), generator=g, device="cuda").to(torch.int32)
        return s
    page = c["page"]
    if c["op"] == "shared":
        groups, prefix, kv, n = _families(c)
        # a prefix's pages, the one that it ends in too, are named by all sequences of its group; their own follow
        need = [-(-p // page) for p in prefix] + [-(-(k - prefix[sum(b >= e for e in groups[1:-1])]) // page) + 1 for b, k in enumerate(kv)]
        whole = _table(need, max(need), sum(need) + 3, g)
        member = torch.bucketize(torch.arange(c["B"], device="cuda"), _ints(groups[1:-1]), right=True) if c["N"] > 1 else torch.zeros(c["B"], dtype=torch.int64, device="cuda")
        at, split = torch.arange(-(-max(kv) // page), device="cuda"), (_ints(prefix) // page)[member][:, None]
        common = whole[:c["N"]][member][:, at.clamp(max=whole.shape[1] - 1)]
        alone = whole[c["N"]:].gather(1, (at - split).clamp(min=0, max=whole.shape[1] - 1))
        s["table"] = torch.where(at < split, common, torch.where(at * page < _ints(kv)[:, None], alone, -1)).to(torch.int32)
        s.update(cache=_cache(sum(need) + 3, c, g), T=sum(n), n=n, max_q=max(n), cu=_offsets(n), kv_len=_ints(kv), groups=_ints(groups), prefix=_ints(prefix))
        # what lies in the page where a prefix ends is the same in each of its sequences: a fork has copied it
        inside = _ints(prefix)[member] % page
        for k in ("K8", "V8", "sk", "sv"):
            own_page = s["table"].gather(1, split.clamp(max=s["table"].shape[1] - 1).long())[:, 0].long()
            old_page = whole[:c["N"]].gather(1, (_ints(prefix) // page).clamp(max=whole.shape[1] - 1).long()[:, None])[member, 0].long()
            part = torch.arange(page, device="cuda") < inside[:, None]
            part = (part & (inside > 0)[:, None])[:, None].reshape([c["B"], 1, page] + [1] * (s["cache"][k].dim() - 3))
            x = s["cache"][k][own_page.clamp(min=0)]
            s["cache"][k][own_page.clamp(min=0)] = torch.where(part, s["cache"][k][old_page.clamp(min=0)], x)
        s["Q"] = _keys(sum(n), c["H"] * c["G"], c["d"], g)
        s["most"] = max(sum(n[a:b]) for a, b in zip(groups, groups[1:]))
        return s
    kv, n = _lengths(c)
    need = [-(-k // page) for k in kv]
    if c["op"] == "append":
        s.update(table=_table(need, max(1, max(need)), sum(need) + 3, g), cache=_cache(sum(need) + 3, c, g), T=sum(n), n=n, cu=_offsets(n), kv_len=_ints(kv))
        s["Q"], s["K"], s["V"] = _keys(sum(n), c["H"] * c["G"], c["d"], g), _keys(sum(n), c["H"], c["d"], g), _values(sum(n), c["H"], c["d"], g)
        return s
    pages = c["pages"]
    s["cache"] = _cache(pages, c, g)
    cols = max(need) + 2 + c["n"] // page
    s["table"], s["kv_len"] = _table(need, cols, pages, g), _ints(kv)
    s["pool"] = _pool(s["table"], pages)
    if c["op"] == "fork":
        s["parents"] = torch.randint(c["B"], (c["N"],), generator=g, device="cuda").to(torch.int32)
        s["none"], s["cu"] = torch.zeros(c["N"], dtype=torch.int32, device="cuda"), _offsets([c["n"]] * c["N"])
        s["new_table"] = torch.full((c["N"], cols), -1, dtype=torch.int32, device="cuda")
        s["new_len"] = torch.zeros(c["N"], dtype=torch.int32, device="cuda")
    if c["op"] == "drafts":
        s["accepted"], s["cu"] = s["kv_len"].clone(), _offsets(n)
    if c["op"] == "compact":
        s["before"] = (s["table"].clone(), s["pool"]["refs"].clone(), s["pool"]["free"].clone())
    if c["op"] == "copy":
        s["other"] = {k: torch.zeros_like(v) for k, v in s["cache"].items()}
        s["from"] = s["table"][0, :need[0]].clone()
        s["to"] = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[:need[0]]
    return s


# ------------------------------------------------------------ plain forms


def _places(s):
    """Sequence, position, page and place in the page of each row of the call."""
    page = s["case"]["page"]
    cu, kv = s["cu"].long(), s["kv_len"].long()
    n = cu[1:] - cu[:-1]
    b = torch.repeat_interleave(torch.arange(n.numel(), device="cuda"), n, output_size=s["T"])
    pos = torch.arange(s["T"], device="cuda") - cu[b] + (kv - n)[b]
    return b, pos, s["table"][b, pos // page].long(), pos % page


def _rotated(x, pos, s, back=False):
    """fp32 [T, H, d] with its first `rot` channels turned by the angles of the rows' positions."""
    c, rot = s["case"], s["case"]["rot"]
    angle = pos.double()[:, None] * s["radians"]  # in 64 bits: far positions
    cos, sin = ((f(angle) * s["rope"]["magnitude"]).float()[:, None] for f in (torch.cos, torch.sin))
    if back:
        sin = -sin
    if c["layout"] == "halves":
        x0, x1 = x[..., :rot // 2], x[..., rot // 2:rot]
    else:
        x0, x1 = x[..., 0:rot:2], x[..., 1:rot:2]
    y0, y1 = x0 * cos - x1 * sin, x0 * sin + x1 * cos
    turned = torch.cat([y0, y1], -1) if c["layout"] == "halves" else torch.stack([y0, y1], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_append(s):
    _, pos, at, off = _places(s)
    for x, code, scale in ((_rotated(s["K"].float(), pos, s), "K8", "sk"), (s["V"].float(), "V8", "sv")):
        codes, scales = _codes(x)
        s["cache"][code][at, :, off] = codes
        s["cache"][scale][at, :, off] = scales
    return _rotated(s["Q"].float(), pos, s).to(torch.bfloat16)


def _plain_trim(s, table, kv_len, lens):
    """Each sequence keeps the pages of its first `lens` tokens."""
    page, pool = s["case"]["page"], s["pool"]
    drop = (torch.arange(table.shape[1], device="cuda") >= ((lens + page - 1) // page)[:, None]) & (table >= 0)
    pool["refs"] -= torch.bincount(table[drop].long(), minlength=pool["refs"].numel()).to(torch.int32)
    table[drop] = -1
    kv_len.copy_(torch.minimum(kv_len, lens))
    pool["free"].copy_(_free_bits(pool["refs"]))


def _plain_fork(s):
    """New rows that name the pages of their parents."""
    page, pool, parents = s["case"]["page"], s["pool"], s["parents"].long()
    s["new_len"].copy_(s["kv_len"][parents])
    held = torch.arange(s["table"].shape[1], device="cuda") < ((s["new_len"] + page - 1) // page)[:, None]
    s["new_table"].copy_(torch.where(held, s["table"][parents], -1))
    pool["refs"] += torch.bincount(s["new_table"][held].long(), minlength=pool["refs"].numel()).to(torch.int32)


def _plain_reserve(s, table, kv_len):
    """Pages that a sequence alone names for the positions of its new tokens: the lowest free ones, in the order of the
    sequences and of their positions.  What a page holds of the tokens before is copied."""
    c, page, pool, cache = s["case"], s["case"]["page"], s["pool"], s["cache"]
    n = (s["cu"][1:] - s["cu"][:-1])
    first = kv_len - n
    cols = torch.arange(table.shape[1], device="cuda")
    written = (cols >= (first // page)[:, None]) & (cols < ((kv_len + page - 1) // page)[:, None]) & (n > 0)[:, None]
    where = written.nonzero()
    entry = table[written].long()
    held = entry >= 0
    # of the rows that write into one page, all but the last take another; the last too, if others hold it
    writers = torch.bincount(entry[held], minlength=pool["refs"].numel())
    order = torch.arange(entry.numel(), device="cuda")
    last = torch.full_like(writers, -1).scatter_reduce(0, entry[held], order[held], "amax")
    shared = held & (pool["refs"][entry.clamp(min=0)] > 1)
    keep = shared & (writers[entry.clamp(min=0)] >= pool["refs"][entry.clamp(min=0)]) & (last[entry.clamp(min=0)] == order)
    fresh = ~held | (shared & ~keep)
    new = (pool["refs"] == 0).nonzero()[:, 0][:fresh.sum()]
    left, old = shared & ~keep, entry.clone()
    pool["refs"] -= torch.bincount(entry[left], minlength=pool["refs"].numel()).to(torch.int32)
    pool["refs"][new] = 1
    entry[fresh] = new
    table[written] = entry.to(torch.int32)
    pool["free"].copy_(_free_bits(pool["refs"]))
    # the tokens before the new ones in the pages that were left
    b, col = where[left].unbind(1)
    tokens = (first[b] - col * page).clamp(min=0)
    part = torch.arange(page, device="cuda") < tokens[:, None]
    for x in cache.values():
        m = part.reshape([part.shape[0], 1, page] + [1] * (x.dim() - 3))
        x[entry[left]] = torch.where(m, x[old[left]], x[entry[left]])


def _plain_compact(s):
    """The pages in use from the first number on."""
    pool, cache, table = s["pool"], s["cache"], s["table"]
    used = pool["refs"] > 0
    count = used.sum()
    at = torch.arange(used.numel(), device="cuda")
    to, old = (~used & (at < count)).nonzero()[:, 0], (used & (at >= count)).nonzero()[:, 0]
    for x in cache.values():
        x[to] = x[old]
    number = at.clone()
    number[old] = to
    table.copy_(torch.where(table >= 0, number[table.clamp(min=0).long()], -1))
    pool["refs"][to] = pool["refs"][old]
    pool["refs"][old] = 0
    pool["free"].copy_(_free_bits(pool["refs"]))
    return count.to(torch.int32).reshape(1)


def _plain_copy(s):
    for k, x in s["other"].items():
        x[s["to"].long()] = s["cache"][k][s["from"].long()]


def _plain_shared(s):
    c, cache = s["case"], s["cache"]
    H, G, d, page, B, T = c["H"], c["G"], c["d"], c["page"], c["B"], s["T"]
    cu, kv = s["cu"].long(), s["kv_len"].long()
    n = cu[1:] - cu[:-1]
    L, N = c["p_hi"] + c["s_hi"], s["max_q"]
    # every sequence padded to the longest: keys and values [B, H, L, d], queries [B, H, N * G, d]
    pos = torch.arange(L, device="cuda")
    at = s["table"].long().clamp(min=0)[:, (pos // page).clamp(max=s["table"].shape[1] - 1)]
    off = (pos % page).expand(B, L)
    value = lambda code, scale: (cache[code][at, :, off].view(torch.float8_e4m3fn).float() * cache[scale][at, :, off][..., None]).transpose(1, 2)  # noqa: E731
    K, V = value("K8", "sk"), value("V8", "sv")
    V = V.masked_fill((pos >= kv[:, None])[:, None, :, None], 0.0)
    i = torch.arange(N, device="cuda")
    row = (cu[:-1, None] + i).clamp(max=T - 1)
    Q = s["Q"].float()[row].view(B, N, H, G, d).permute(0, 2, 1, 3, 4).reshape(B, H, N * G, d)
    scores = Q @ K.transpose(-1, -2)
    scores *= 1.0 / math.sqrt(d)
    last = (kv - n)[:, None] + i if c["causal"] else (kv - 1)[:, None].expand(B, N)
    seen = (pos <= last[..., None]) & (pos < kv[:, None, None])
    scores.view(B, H, N, G, L).masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    scores -= top
    scores.exp_()
    total = scores.sum(-1, keepdim=True)
    O = (scores @ V) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + total.log())[..., 0]
    b, p, _, _ = _places(s)
    i = p - (kv - n)[b]
    O = O.view(B, H, N, G, d).permute(0, 2, 1, 3, 4)[b, i].reshape(T, H * G, d)
    lse = lse.view(B, H, N, G).permute(0, 2, 1, 3)[b, i].reshape(T, H * G)
    return O.to(torch.bfloat16), lse


def _pages_of(s, table, kv_len):
    return {"table": table, "kv_len": kv_len, "refs": s["pool"]["refs"], "free": s["pool"]["free"], **_stored(s["cache"])}


def _stored(cache):
    return {"K8": cache["K8"].view(torch.float8_e4m3fn), "sk": cache["sk"], "V8": cache["V8"].view(torch.float8_e4m3fn), "sv": cache["sv"]}


def run(state):
    s = state
    c = s["case"]
    if own:
        from bit_fp8_attention_means_gb300 import vc
        trim = lambda table, kv_len, lens: vc.vc_pages_trim(s["cache"], s["pool"], table, kv_len, lens)  # noqa: E731
        fork = lambda: vc.vc_pages_fork(s["cache"], s["pool"], s["table"], s["kv_len"], s["parents"], s["new_table"], s["new_len"])  # noqa: E731
        reserve = lambda table, kv_len: vc.vc_pages_reserve(s["cache"], s["pool"], s["cu"], kv_len, table, T=c["n"] * (s["cu"].numel() - 1))  # noqa: E731
    else:
        trim = lambda table, kv_len, lens: _plain_trim(s, table, kv_len, lens)  # noqa: E731
        fork = lambda: _plain_fork(s)  # noqa: E731
        reserve = lambda table, kv_len: _plain_reserve(s, table, kv_len)  # noqa: E731
    if c["op"] == "rotate":
        if own:
            return vc.vc_rope(s["X"], s["rope"], pos=s["pos"], inverse=int(c["inverse"]))
        return _rotated(s["X"].float(), s["pos"], s, c["inverse"]).to(torch.bfloat16)
    if c["op"] == "append":
        if own:
            Q = vc.vc_cache_append_rope(s["Q"], s["K"], s["V"], s["cache"], s["cu"], s["kv_len"], s["table"], s["rope"])
        else:
            Q = _plain_append(s)
        return {"Q": Q, **_stored(s["cache"])}
    if c["op"] == "fork":
        trim(s["new_table"], s["new_len"], s["none"])
        fork()
        s["new_len"] += c["n"]
        reserve(s["new_table"], s["new_len"])
        return _pages_of(s, s["new_table"], s["new_len"])
    if c["op"] == "drafts":
        trim(s["table"], s["kv_len"], s["accepted"])
        s["kv_len"] += c["n"]
        reserve(s["table"], s["kv_len"])
        return _pages_of(s, s["table"], s["kv_len"])
    if c["op"] == "compact":
        # from the same tables each time: what is moved stays where it was, too
        for x, y in zip((s["table"], s["pool"]["refs"], s["pool"]["free"]), s["before"]):
            x.copy_(y)
        count = vc.vc_pages_compact(s["cache"], s["pool"], s["table"]) if own else _plain_compact(s)
        return {"count": count, **_pages_of(s, s["table"], s["kv_len"])}
    if c["op"] == "copy":
        if own:
            vc.vc_cache_copy(s["cache"], s["other"], s["from"], s["to"])
        else:
            _plain_copy(s)
        return _stored(s["other"])
    if own:
        return vc.vc_attn_paged_shared(s["Q"], s["cache"], s["cu"], s["kv_len"], s["table"], s["groups"], s["prefix"], causal=int(c["causal"]), max_q=s["max_q"], max_rows=s["most"])
    return _plain_shared(s)


# ------------------------------------------------------------ work


def work(case):
    c = case
    if c["op"] == "rotate":
        return {"bytes": c["T"] * (c["H"] * c["d"] * 4 + 4), "flops": c["T"] * c["H"] * c["rot"] * 3}
    H, d, page = c["H"], c["d"], c["page"]
    token = H * (2 * d + 8)  # codes and scales of a cached token
    if c["op"] == "shared":
        groups, prefix, kv, n = _families(c)
        pairs = keys = 0
        for g, p in enumerate(prefix):
            keys += p
            for b in range(groups[g], groups[g + 1]):
                keys += kv[b] - p if n[b] else 0
                pairs += sum(kv[b] - n[b] + i + 1 if c["causal"] else kv[b] for i in range(n[b]))
        rows = sum(n) * H * c["G"]
        return {"bytes": rows * (4 * d + 4) + keys * token, "flops": 4.0 * d * pairs * H * c["G"]}
    kv, n = _lengths(c)
    if c["op"] == "append":
        T = sum(n)
        return {"bytes": T * (H * c["G"] * 4 * d + H * 4 * d + token), "flops": T * H * (c["rot"] * 3 * (c["G"] + 1) + 4 * d)}
    held = [-(-k // page) for k in kv]
    if c["op"] == "fork":
        parents = c["N"] * (sum(held) // c["B"])  # entries that a fork writes, about
        copied = c["N"] * (sum(k % page for k in kv) // c["B"]) * token
        return {"bytes": 8 * parents + 4 * sum(held) + 2 * copied, "flops": parents}
    if c["op"] == "drafts":
        return {"bytes": c["B"] * 40 + c["B"] * (c["n"] // page + 1) * 16 + c["pages"] // 8, "flops": c["B"]}
    if c["op"] == "compact":
        used = sum(held)
        moved = used * (1.0 - used / c["pages"])  # those of random numbers behind the first `used`
        return {"bytes": 2 * moved * page * token + 8 * sum(held) + 8 * c["pages"], "flops": used}
    return {"bytes": 2 * held[0] * page * token + 8 * held[0], "flops": held[0]}


# ------------------------------------------------------------ from the definitions, in 64 bits


def _exact_rotation(x, pos, c, back):
    """fp64 [T, H, d], pair by pair."""
    w, times = _turns(c)
    y = x.double().clone()
    for i in range(c["rot"] // 2):
        p, q = (i, i + c["rot"] // 2) if c["layout"] == "halves" else (2 * i, 2 * i + 1)
        angle = pos.double() * float(w[i])
        z = torch.polar(torch.full_like(angle, times), -angle if back else angle)[:, None] * torch.complex(x[..., p].double(), x[..., q].double())
        y[..., p], y[..., q] = z.real, z.imag
    return y


def _exact_codes(x):
    """The nearest E4M3 value of each channel times 448 over the row's largest, as bytes, and the scale."""
    top = x.abs().amax(-1)
    q = torch.where(top[..., None] > 0, x * 448.0 / top[..., None], torch.zeros((), dtype=torch.float64, device="cuda"))
    # a step is 2^-3 of the value's power of two, 2^-9 at the least
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(q / step) * step).float().to(torch.float8_e4m3fn).view(torch.uint8), (top / 448.0).float()


def _exact_pages(s):
    """The page calls of `run` on lists, one entry after the other."""
    c, page = s["case"], s["case"]["page"]
    table, kv = s["table"].tolist(), s["kv_len"].tolist()
    refs, cache = s["pool"]["refs"].tolist(), {k: v.clone() for k, v in s["cache"].items()}
    count, moves = 0, []                       # moves: from a page, to a page, so many tokens
    if c["op"] == "fork":
        parents = s["parents"].tolist()
        old, old_len = table, kv
        table, kv = [[-1] * len(table[0]) for _ in parents], [old_len[p] for p in parents]
        for row, p in zip(table, parents):
            for j in range(-(-old_len[p] // page)):
                row[j] = old[p][j]
                refs[row[j]] += 1
    if c["op"] in ("fork", "drafts"):
        # in the sequences' order: a page that others still hold is left to them, the last one keeps it
        lowest = iter([p for p, r in enumerate(refs) if r == 0])
        for b, row in enumerate(table):
            first, kv[b] = kv[b], kv[b] + c["n"]
            for j in range(first // page, -(-kv[b] // page)):
                if row[j] >= 0 and refs[row[j]] == 1:
                    continue
                new = next(lowest)
                if row[j] >= 0:
                    refs[row[j]] -= 1
                    moves.append((row[j], new, max(0, first - j * page)))
                row[j], refs[new] = new, 1
    if c["op"] == "compact":
        count = sum(r > 0 for r in refs)
        holes = [p for p in range(count) if refs[p] == 0]
        to = dict(zip([p for p in range(count, len(refs)) if refs[p]], holes))
        moves = [(a, b, page) for a, b in to.items()]
        table = [[to.get(e, e) for e in row] for row in table]
        for a, b in to.items():
            refs[a], refs[b] = 0, refs[a]
    if moves:
        a, b, m = (torch.tensor(x, device="cuda") for x in zip(*moves))
        for k, x in cache.items():
            part = (torch.arange(page, device="cuda") < m[:, None]).reshape([len(moves), 1, page] + [1] * (x.dim() - 3))
            x[b] = torch.where(part, s["cache"][k][a], x[b])
    words = [sum(1 << i for i in range(32) if p + i < len(refs) and refs[p + i] == 0) for p in range(0, len(refs), 32)]
    out = {"table": _ints(table), "kv_len": _ints(kv), "refs": _ints(refs), "free": _ints([w - (1 << 32) if w >> 31 else w for w in words]), **_stored(cache)}
    return {"count": _ints([count]), **out} if c["op"] == "compact" else out


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "rotate":
        return _exact_rotation(s["X"], s["pos"], c, c["inverse"])
    if c["op"] in ("fork", "drafts", "compact"):
        return _exact_pages(s)
    cache = s["cache"]
    if c["op"] == "copy":
        for k, x in s["other"].items():
            for a, b in zip(s["from"].tolist(), s["to"].tolist()):
                x[b] = cache[k][a]
        return _stored(s["other"])
    H, G, d, page, T = c["H"], c["G"], c["d"], c["page"], s["T"]
    if c["op"] == "append":
        kv, n = _lengths(c)
        pos = torch.cat([torch.arange(k - m, k, device="cuda") for k, m in zip(kv, n)])
        K = _exact_rotation(s["K"], pos, c, False)
        for x, code, scale in ((K, "K8", "sk"), (s["V"].double(), "V8", "sv")):
            q, t = _exact_codes(x)
            row = 0
            for b in range(c["B"]):
                p = pos[row:row + n[b]]
                at = s["table"][b].long()[p // page]
                cache[code][at, :, p % page] = q[row:row + n[b]]
                cache[scale][at, :, p % page] = t[row:row + n[b]]
                row += n[b]
        return {"Q": _exact_rotation(s["Q"], pos, c, False), **_stored(cache)}
    groups, prefix, kv, n = _families(c)
    if 4.0 * d * H * G * sum(k * m for k, m in zip(kv, n)) > 8e12:
        return None

    def cached(code, scale, b, h, L):
        """Keys or values of head h at the first L positions of sequence b."""
        pages = s["table"][b, :-(-L // page)].long()
        x = cache[code][pages, h].view(torch.float8_e4m3fn).double() * cache[scale][pages, h].double()[..., None]
        return x.reshape(-1, d)[:L]

    O = torch.zeros((T, H * G, d), dtype=torch.float64, device="cuda")
    lse = torch.full((T, H * G), -math.inf, dtype=torch.float64, device="cuda")
    row = 0
    for b in range(c["B"]):
        for h in range(H if n[b] else 0):
            K, V = cached("K8", "sk", b, h, kv[b]), cached("V8", "sv", b, h, kv[b])
            at, part = torch.arange(kv[b], device="cuda"), max(1, (1 << 28) // (kv[b] * G))
            for i in range(0, n[b], part):
                q = s["Q"][row + i:row + min(i + part, n[b]), h * G:(h + 1) * G].double()
                m = q.shape[0]
                z = (q.reshape(m * G, d) @ K.T).view(m, G, -1) / math.sqrt(d)
                if c["causal"]:
                    z.masked_fill_((at > (kv[b] - n[b] + i + torch.arange(m, device="cuda"))[:, None])[:, None], -math.inf)
                lse[row + i:row + i + m, h * G:(h + 1) * G] = torch.logsumexp(z, -1)
                O[row + i:row + i + m, h * G:(h + 1) * G] = (torch.softmax(z, -1).view(m * G, -1) @ V).view(m, G, d)
        row += n[b]
    return O, lse
