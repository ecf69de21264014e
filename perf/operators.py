"""The paged FP8 key/value cache and the attention that reads it, as measured cases.

Three operators: quantising new keys and values into the pages of a cache as
they are written, reading cached tokens back as bf16, and attention of a chunk
of new tokens (down to one) over the paged cache.  ``run`` computes each in its
plain form in 32 bits, or, with ``own`` set, calls the framework.

A batch is B sequences.  Sequence b holds ``kv_len[b]`` tokens in the cache;
its last n_b = cu[b+1] - cu[b] tokens are the ones a call writes, reads or asks
from, packed in rows cu[b] .. cu[b+1] - 1, so row cu[b] + i is the token at
position kv_len[b] - n_b + i.  Position p lies in page table[b][p // page], at
p % page.  Codes are E4M3 with one fp32 scale for each token and head,
amax / 448.
"""
import math
import random

import torch

own = False

CLIP = 75600   # 21 x 45 x 80 latent tokens
FRAME = 3600   # one latent frame of 45 x 80 tokens


def listed():
    return [
        # serving: every sequence of a batch writes its newest token
        dict(name="append, one token each", op="append", B=96, n_lo=1, n_hi=1, kv_lo=1, kv_hi=8192, H=8, G=1, d=128, page=16, causal=True, window=0, lens=1),
        # chunk-wise video generation: a finished latent frame enters the cache, 40 heads
        dict(name="append, a latent frame", op="append", B=1, n_lo=FRAME, n_hi=FRAME, kv_lo=3 * FRAME, kv_hi=3 * FRAME, H=40, G=1, d=128, page=128, causal=False, window=0, lens=2),
        # prompts of different lengths (one of them empty), small heads
        dict(name="append, ragged chunks", op="append", B=9, n_lo=0, n_hi=517, kv_lo=0, kv_hi=700, H=6, G=1, d=64, page=32, causal=True, window=0, lens=3),
        # the whole clip back to bf16, as for leaving the cache or checking it
        dict(name="read, a whole clip", op="read", B=1, n_lo=CLIP, n_hi=CLIP, kv_lo=CLIP, kv_hi=CLIP, H=40, G=1, d=128, page=128, causal=False, window=0, lens=4),
        # cached prefixes of a small batch
        dict(name="read, ragged prefixes", op="read", B=17, n_lo=0, n_hi=900, kv_lo=0, kv_hi=900, H=2, G=1, d=64, page=16, causal=False, window=0, lens=5),
        # the smallest step: one token of one short sequence
        dict(name="attend, one token, short", op="attend", B=1, n_lo=1, n_hi=1, kv_lo=219, kv_hi=219, H=2, G=1, d=64, page=16, causal=True, window=0, lens=6),
        # serving a batch of different lengths, grouped heads
        dict(name="attend, one token each", op="attend", B=96, n_lo=1, n_hi=1, kv_lo=100, kv_hi=8192, H=8, G=4, d=128, page=16, causal=True, window=0, lens=7),
        # one token against a clip-long cache: few rows, a long axis
        dict(name="attend, one token, long", op="attend", B=1, n_lo=1, n_hi=1, kv_lo=CLIP, kv_hi=CLIP, H=8, G=5, d=128, page=128, causal=True, window=0, lens=8),
        # a few tokens of each sequence at once (drafts that are checked)
        dict(name="attend, a few tokens each", op="attend", B=24, n_lo=1, n_hi=7, kv_lo=500, kv_hi=6000, H=4, G=8, d=128, page=64, causal=True, window=0, lens=9),
        # prompts in chunks, some with a cached prefix
        dict(name="attend, ragged chunks", op="attend", B=7, n_lo=0, n_hi=700, kv_lo=300, kv_hi=4096, H=8, G=4, d=128, page=32, causal=True, window=0, lens=10),
        # long causal chunks that see a sliding window
        dict(name="attend, window", op="attend", B=2, n_lo=4001, n_hi=8192, kv_lo=9000, kv_hi=16384, H=4, G=6, d=64, page=64, causal=True, window=4096, lens=11),
        # one latent frame attends to the clip in both directions, 40 heads
        dict(name="attend, a frame over a clip", op="attend", B=1, n_lo=FRAME, n_hi=FRAME, kv_lo=CLIP, kv_hi=CLIP, H=40, G=1, d=128, page=128, causal=False, window=0, lens=12),
    ]


def _between(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "read", "attend", "attend", "attend"])
    d = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128, 256])
    lens = rng.randrange(1 << 30)
    if op != "attend":
        H = rng.choice([1, 2, 3, 6, 8, 24, 40])
        kv_hi = _between(rng, 1, 20000 if H > 8 else 60000)
        B = _between(rng, 1, max(1, min(200, 120000 // kv_hi)))
        n_hi = kv_hi if op == "read" else _between(rng, 1, kv_hi)
        return dict(op=op, B=B, n_lo=rng.choice([0, 1, n_hi]), n_hi=n_hi, kv_lo=rng.choice([0, kv_hi // 2, kv_hi]), kv_hi=kv_hi, H=H, G=1, d=d, page=page, causal=False,
                    window=0, lens=lens)
    form = rng.choice(["token", "token", "few", "chunk", "chunk"])
    H, G = rng.choice([(1, 1), (2, 8), (4, 3), (4, 6), (8, 4), (8, 5), (24, 1), (40, 1)])
    kv_hi = _between(rng, 1, 60000)
    if form == "token":
        n_hi, B = 1, _between(rng, 1, max(1, min(200, 2400000 // (kv_hi * H))))
    elif form == "few":
        n_hi, B = rng.randint(2, 9), _between(rng, 1, max(1, min(60, 1600000 // (kv_hi * H))))
    else:
        n_hi = _between(rng, 10, max(10, min(6000, 4000000000 // (kv_hi * H * G))))
        B = _between(rng, 1, max(1, min(12, 4000000000 // (n_hi * kv_hi * H * G))))
    causal = rng.random() < 0.7
    window = _between(rng, 1, 2 * kv_hi) if rng.random() < 0.3 else 0
    return dict(op=op, B=B, n_lo=rng.choice([0, 1, n_hi]), n_hi=n_hi, kv_lo=rng.choice([0, kv_hi // 2, kv_hi]), kv_hi=kv_hi, H=H, G=G, d=d, page=page, causal=causal,
                window=window, lens=lens)


def _lengths(c):
    """The sequences' lengths in the cache and in the call: the case alone gives them.  One is the longest, and no
    call asks for more tokens of a sequence than it holds."""
    rng = random.Random(c["lens"])
    kv = [rng.randint(c["kv_lo"], c["kv_hi"]) for _ in range(c["B"])]
    kv[rng.randrange(c["B"])] = c["kv_hi"]
    whole = c["op"] == "read"
    n = [k if whole else min(k, rng.randint(c["n_lo"], c["n_hi"])) for k in kv]
    if not whole and sum(n) == 0:
        n[kv.index(max(kv))] = min(c["n_hi"], max(kv))
    return kv, n


def _random(shape, g):
    return torch.randn(shape, generator=g, device="cuda")


def _keys(rows, H, d, g):
    """Keys (and queries): N(0, 1) about a mean of each head and channel, as bf16."""
    return (_random((rows, H, d), g) + _random((1, H, d), g)).to(torch.bfloat16)


def _values(rows, H, d, g):
    """Values: N(0, 1), one token in a hundred times 20 on four channels, as bf16."""
    v = _random((rows, H, d), g)
    v[:, :, torch.randperm(d, generator=g, device="cuda")[:4]] *= torch.where(torch.rand((rows, 1, 1), generator=g, device="cuda") < 0.01, 20.0, 1.0)
    return v.to(torch.bfloat16)


def _codes(x):
    """[..., d] -> E4M3 codes (their bytes) and the fp32 scale of each row."""
    x = x.float()
    amax = x.abs().amax(-1, keepdim=True)
    inv = torch.where(amax > 0, 448.0 / amax, torch.zeros_like(amax))
    return (x * inv).to(torch.float8_e4m3fn).view(torch.uint8), (amax / 448.0)[..., 0]


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kv, n = _lengths(c)
    H, d, page, T = c["H"], c["d"], c["page"], sum(n)
    need = [-(-k // page) for k in kv]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((c["B"], max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    cache = {}
    for code, scale, make in (("K8", "sk", _keys), ("V8", "sv", _values)):
        # made for one head after the other: the fp32 parts of a clip are large
        cache[code] = torch.empty((pages, H, page, d), dtype=torch.uint8, device="cuda")
        cache[scale] = torch.empty((pages, H, page), dtype=torch.float32, device="cuda")
        for h in range(H):
            x, s = _codes(make(pages * page, 1, d, g).view(pages, page, d))
            cache[code][:, h], cache[scale][:, h] = x, s
    starts = [0]
    for m in n:
        starts.append(starts[-1] + m)
    state = dict(case=c, cache=cache, table=table, T=T, max_q=max(n), n=n,
                 cu=torch.tensor(starts, dtype=torch.int32, device="cuda"), kv_len=torch.tensor(kv, dtype=torch.int32, device="cuda"))
    if c["op"] == "append":
        state["K"], state["V"] = _keys(T, H, d, g), _values(T, H, d, g)
    if c["op"] == "attend":
        state["Q"] = _keys(T, H * c["G"], d, g)
    return state


def _places(s):
    """Sequence, position, page and place in the page of each row of the call."""
    page = s["case"]["page"]
    cu, kv = s["cu"].long(), s["kv_len"].long()
    n = cu[1:] - cu[:-1]
    b = torch.repeat_interleave(torch.arange(n.numel(), device="cuda"), n, output_size=s["T"])
    pos = torch.arange(s["T"], device="cuda") - cu[b] + (kv - n)[b]
    return b, pos, s["table"][b, pos // page].long(), pos % page


def _plain_append(s):
    _, _, at, off = _places(s)
    for x, code, scale in ((s["K"], "K8", "sk"), (s["V"], "V8", "sv")):
        codes, scales = _codes(x)
        s["cache"][code][at, :, off] = codes
        s["cache"][scale][at, :, off] = scales
    return _state_of(s["cache"])


def _state_of(cache):
    return {"K8": cache["K8"].view(torch.float8_e4m3fn), "sk": cache["sk"], "V8": cache["V8"].view(torch.float8_e4m3fn), "sv": cache["sv"]}


def _plain_read(s):
    _, _, at, off = _places(s)
    c = s["cache"]
    value = lambda code, scale: (c[code].view(torch.uint8)[at, :, off].view(torch.float8_e4m3fn).float() * c[scale][at, :, off][..., None]).to(torch.bfloat16)  # noqa: E731
    return value("K8", "sk"), value("V8", "sv")


def _plain_attend(s):
    c, cache = s["case"], s["cache"]
    H, G, d, page, B, T = c["H"], c["G"], c["d"], c["page"], c["B"], s["T"]
    cu, kv = s["cu"].long(), s["kv_len"].long()
    n = cu[1:] - cu[:-1]
    L, N = c["kv_hi"], s["max_q"]
    # every sequence padded to the longest: keys and values [B, H, L, d], queries [B, H, N * G, d]
    pos = torch.arange(L, device="cuda")
    at = s["table"].long().clamp(min=0)[:, pos // page]
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
    if c["window"]:
        seen &= pos > last[..., None] - c["window"]
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


def run(state):
    s = state
    c = s["case"]
    if own:
        from bit_fp8_attention_means_gb300 import vc
        if c["op"] == "append":
            vc.vc_cache_append(s["K"], s["V"], s["cache"], s["cu"], s["kv_len"], s["table"])
            return _state_of(s["cache"])
        if c["op"] == "read":
            return vc.vc_cache_read(s["cache"], s["cu"], s["kv_len"], s["table"], s["T"])
        return vc.vc_attn_paged(s["Q"], s["cache"], s["cu"], s["kv_len"], s["table"], causal=int(c["causal"]), window=c["window"], max_q=s["max_q"])
    if c["op"] == "append":
        return _plain_append(s)
    if c["op"] == "read":
        return _plain_read(s)
    return _plain_attend(s)


def _seen(c, kv, n):
    """First and last key that each of a sequence's n rows sees."""
    last = [kv - n + i if c["causal"] else kv - 1 for i in range(n)]
    return [(max(0, e - c["window"] + 1) if c["window"] else 0, e) for e in last]


def work(case):
    c = case
    kv, n = _lengths(c)
    T, H, d = sum(n), c["H"], c["d"]
    token = H * (2 * d + 8)  # codes and scales of a cached token
    if c["op"] != "attend":
        return {"bytes": T * (H * 4 * d + token), "flops": T * H * d * 4}
    pairs = keys = 0
    for k, m in zip(kv, n):
        span = _seen(c, k, m)
        pairs += sum(e - a + 1 for a, e in span)
        keys += max((e for _, e in span), default=-1) + 1 - min((a for a, _ in span), default=0)
    rows = T * H * c["G"]
    return {"bytes": rows * (4 * d + 4) + keys * token, "flops": 4.0 * d * pairs * H * c["G"]}


def exact(case, seed):
    s = prepare(case, seed)
    c, cache = s["case"], s["cache"]
    H, G, d, page, T = c["H"], c["G"], c["d"], c["page"], s["T"]
    kv, n = _lengths(c)

    def cached(code, scale, b, h, a, e):
        """Keys or values of head h at positions a .. e - 1 of sequence b."""
        pages = s["table"][b, a // page:-(-e // page)].long()
        x = cache[code][pages, h].view(torch.float8_e4m3fn).double() * cache[scale][pages, h].double()[..., None]
        return x.reshape(-1, d)[a % page:a % page + e - a]

    if c["op"] == "append":
        out = {k: v.clone() for k, v in cache.items()}
        for x, code, scale in ((s["K"], "K8", "sk"), (s["V"], "V8", "sv")):
            top = x.double().abs().amax(-1)
            q = torch.where(top[..., None] > 0, x.double() * 448.0 / top[..., None], torch.zeros((), dtype=torch.float64, device="cuda"))
            # nearest E4M3 value: a step is 2^-3 of the value's power of two, 2^-9 at the least
            step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
            q = (torch.round(q / step) * step).float().to(torch.float8_e4m3fn).view(torch.uint8)
            row = 0
            for b in range(c["B"]):
                p = torch.arange(kv[b] - n[b], kv[b], device="cuda")
                at = s["table"][b].long()[p // page]
                out[code][at, :, p % page] = q[row:row + n[b]]
                out[scale][at, :, p % page] = (top[row:row + n[b]] / 448.0).float()
                row += n[b]
        return _state_of(out)
    if c["op"] == "read":
        whole = []
        for code, scale in (("K8", "sk"), ("V8", "sv")):
            whole.append(torch.cat([torch.stack([cached(code, scale, b, h, kv[b] - n[b], kv[b]) for h in range(H)], 1) for b in range(c["B"]) if n[b]]).float())
        return tuple(whole)
    if 4.0 * d * H * G * sum(e - a + 1 for k, m in zip(kv, n) for a, e in _seen(c, k, m)) > 8e12:
        return None
    O = torch.zeros((T, H * G, d), dtype=torch.float64, device="cuda")
    lse = torch.full((T, H * G), -math.inf, dtype=torch.float64, device="cuda")
    row = 0
    for b in range(c["B"]):
        span = torch.tensor(_seen(c, kv[b], n[b]), device="cuda").view(-1, 2)
        if n[b] and kv[b]:
            for h in range(H):
                K, V = cached("K8", "sk", b, h, 0, kv[b]), cached("V8", "sv", b, h, 0, kv[b])
                at = torch.arange(kv[b], device="cuda")
                part = max(1, (1 << 28) // (kv[b] * G))
                for i in range(0, n[b], part):
                    q = s["Q"][row + i:row + min(i + part, n[b]), h * G:(h + 1) * G].double()
                    m = q.shape[0]
                    z = (q.reshape(m * G, d) @ K.T).view(m, G, -1) / math.sqrt(d)
                    hidden = (at < span[i:i + m, :1]) | (at > span[i:i + m, 1:])
                    z.masked_fill_(hidden[:, None], -math.inf)
                    lse[row + i:row + i + m, h * G:(h + 1) * G] = torch.logsumexp(z, -1)
                    p = torch.softmax(z, -1).view(m * G, -1)
                    O[row + i:row + i + m, h * G:(h + 1) * G] = (p @ V).view(m, G, d)
        row += n[b]
    return O, lse
