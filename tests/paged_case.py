"""Batches over a paged cache for the tests, on the CPU, and the operators' definitions in fp64.

Shares no code with the library: codes are decoded through torch's float8 type
on the CPU and encoded by a nearest-value search over its 256 values.
"""
import math
import random

import torch

E4M3 = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()   # value of every code
LOG2E = 1.4426950408889634


def encode(x):
    """E4M3 byte of fp64 values within +-448: the nearest, ties to the even code, the sign kept on zero."""
    pos = E4M3[:127]                                        # 0 .. 448, ascending
    a = x.abs().clamp(max=448.0)
    hi = torch.searchsorted(pos, a).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up = (pos[hi] - a < a - pos[lo]) | ((pos[hi] - a == a - pos[lo]) & (hi % 2 == 0))
    code = torch.where(up, hi, lo)
    return (code + 128 * torch.signbit(x)).to(torch.uint8)


def quantize(x):
    """bf16 [..., d] -> codes, fp32 scales, by the definition in fp32 steps."""
    xf = x.float()
    amax = xf.abs().amax(-1, keepdim=True)
    zero = amax < 2.0 ** -100
    bad = ~torch.isfinite(xf).all(-1, keepdim=True)
    inv = torch.where(zero | bad, torch.zeros(()), torch.tensor(448.0) / amax)
    y = torch.where(zero | bad, torch.zeros(()), xf * inv)
    scale = torch.where(bad, torch.tensor(math.nan), torch.where(zero, torch.zeros(()), amax / 448.0))[..., 0]
    codes = encode(y.double())
    codes[(zero | bad).expand_as(codes)] = 0
    return codes, scale


class Case:
    """A batch: lengths, a page pool in random order, queries, and new keys and values."""

    def __init__(self, n, kv, H=2, G=1, d=128, page=16, seed=0, spare=2, tail=0, qmul=1.0, cols=None):
        g = torch.Generator().manual_seed(seed)
        self.n, self.kv, self.H, self.G, self.d, self.page = list(n), list(kv), H, G, d, page
        self.B, self.T = len(n), sum(n) + tail            # `tail` rows behind the last sequence
        need = [-(-k // page) for k in kv]
        self.pages = sum(need) + spare
        order = list(range(self.pages))
        random.Random(seed).shuffle(order)
        self.table = torch.full((self.B, cols or max(1, max(need))), -1, dtype=torch.int32)
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = torch.tensor(order[at:at + m], dtype=torch.int32)
            at += m
        cu = [0]
        for m in n:
            cu.append(cu[-1] + m)
        self.cu, self.kv_len = torch.tensor(cu, dtype=torch.int32), torch.tensor(kv, dtype=torch.int32)

        def bf(*shape, mul=1.0):
            return (torch.randn(shape, generator=g) * mul).to(torch.bfloat16)
        self.Q = bf(self.T, H * G, d, mul=qmul)
        self.K, self.V = bf(self.T, H, d), bf(self.T, H, d)
        self.K8, self.sk = quantize(bf(self.pages, H, page, d))
        self.V8, self.sv = quantize(bf(self.pages, H, page, d))

    def cache(self, device=None):
        return {k: getattr(self, k).clone() if device is None else getattr(self, k).to(device)
                for k in ("K8", "sk", "V8", "sv")}

    def args(self, device):
        return tuple(t.to(device) for t in (self.cu, self.kv_len, self.table))

    def places(self):
        """(row, sequence, position) of every row of the call."""
        return [(int(self.cu[b]) + i, b, self.kv[b] - self.n[b] + i) for b in range(self.B) for i in range(self.n[b])]

    def page_of(self, b, p):
        pg = int(self.table[b, p // self.page])
        return pg if 0 <= pg < self.pages else None

    # ---------------------------------------------------------------- definitions

    def appended(self):
        """The cache after the call's keys and values are written."""
        c = self.cache()
        for code, scale, x in (("K8", "sk", self.K), ("V8", "sv", self.V)):
            q, s = quantize(x)
            for r, b, p in self.places():
                if p >= 0 and self.page_of(b, p) is not None:
                    c[code][self.page_of(b, p), :, p % self.page] = q[r]
                    c[scale][self.page_of(b, p), :, p % self.page] = s[r]
        return c

    def read(self, c, K, V):
        """K and V with the cached rows in them."""
        K, V = K.clone(), V.clone()
        for r, b, p in self.places():
            pg = self.page_of(b, p) if p >= 0 else None
            for out, code, scale in ((K, "K8", "sk"), (V, "V8", "sv")):
                if pg is None:
                    out[r] = 0
                else:
                    x = E4M3[c[code][pg, :, p % self.page].long()].float() * c[scale][pg, :, p % self.page, None]
                    out[r] = x.to(torch.bfloat16)
        return K, V

    def sequence(self, c, code, scale, b, h):
        """(codes' values, scales, there) of a sequence's positions 0 .. kv - 1 in head h, fp64."""
        L = self.kv[b]
        pgs = [self.page_of(b, p) for p in range(0, L, self.page)]
        there = torch.tensor([pg is not None for pg in pgs]).repeat_interleave(self.page)[:L]
        idx = torch.tensor([0 if pg is None else pg for pg in pgs])
        x = E4M3[c[code][idx, h].long()].reshape(-1, self.d)[:L]
        return x, c[scale][idx, h].double().reshape(-1)[:L], there

    def attend(self, c, causal=1, window=0, scale=0.0, rows=None):
        """O, lse in fp64 and how far a kernel may be off them, element by element.

        The bars count, for a row with visible keys t, probabilities p_t, and
        scores s_t: the output's rounding to bf16 (half a step, 2^-8); the
        probabilities' rounding to fp16 (2^-11 of each, or 2^-25 of the largest
        P = p_t sv_t where that is more); and e^(error of s_t), the error of a
        score being that of the query's two-part E4M3 form (2^-17 of the row's
        largest channel in each channel), of fp32 sums of 2d products, and of
        its fp32 scaling and exponential; n 2^-24 for the row sums."""
        T, Hq, d, G = self.T, self.H * self.G, self.d, self.G
        scale = scale if scale > 0 else 1.0 / math.sqrt(d)
        O, tolO = torch.zeros((T, Hq, d), dtype=torch.float64), torch.zeros((T, Hq, d), dtype=torch.float64)
        lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
        told = torch.zeros((T, Hq), dtype=torch.float64)
        Q = self.Q.double()
        for b in range(self.B):
            if self.n[b] == 0 or self.kv[b] == 0:
                continue
            r0, n, L = int(self.cu[b]), self.n[b], self.kv[b]
            last = (L - n + torch.arange(n)) if causal else torch.full((n,), L - 1)
            pos = torch.arange(L)
            for h in range(self.H):
                kc, ks, there = self.sequence(c, "K8", "sk", b, h)
                vc_, vs, _ = self.sequence(c, "V8", "sv", b, h)
                k, v = kc * ks[:, None], vc_ * vs[:, None]
                seen = (pos <= last[:, None]) & there
                if window:
                    seen &= pos > last[:, None] - window
                k, v = torch.where(there[:, None], k, 0.0), torch.where(there[:, None], v, 0.0)
                vabs = torch.where(there[:, None], vc_.abs(), 0.0)
                for j in range(G):
                    q = Q[r0:r0 + n, h * G + j]
                    s = (q @ k.T * scale).masked_fill(~seen, -math.inf)
                    some = seen.any(-1)
                    top = torch.where(some, s.amax(-1), 0.0)
                    p = torch.exp(s - top[:, None]).masked_fill(~seen, 0.0)
                    tot = torch.where(some, p.sum(-1), 1.0)
                    # a key whose values are not numbers spoils the rows that see it, and no other
                    spoil = (seen[:, :, None] & ~torch.isfinite(v)).any(1) | ~torch.isfinite(top)[:, None]
                    vz = torch.nan_to_num(v, 0.0, 0.0, 0.0)
                    o = p @ vz / tot[:, None]
                    O[r0:r0 + n, h * G + j] = o.masked_fill(spoil, math.nan)
                    lse[r0:r0 + n, h * G + j] = torch.where(some, top + tot.log(), -math.inf)
                    kz = torch.nan_to_num(k, 0.0, 0.0, 0.0)
                    qmax = q.abs().amax(-1, keepdim=True)
                    err = scale * (2.0 ** -17 * qmax * kz.abs().sum(-1) + 2 * (d + 16) * 2.0 ** -24 * (q.abs() @ kz.abs().T))
                    fin = torch.where(seen, s, 0.0)
                    err = err + 2.0 ** -21 * (fin.abs() * LOG2E + 16)
                    delta = torch.where(seen, err, 0.0).amax(-1)
                    rel = (L + 64) * 2.0 ** -24
                    w = p * torch.nan_to_num(vs)
                    small = 2.0 ** -25 * w.amax(-1, keepdim=True) * (seen.double() @ vabs) / tot[:, None]
                    tolO[r0:r0 + n, h * G + j] = (2.0 ** -8 * o.abs() + small
                                                  + (2.0 ** -11 + 3 * delta[:, None] + rel) * (p @ vz.abs()) / tot[:, None])
                    told[r0:r0 + n, h * G + j] = delta + rel + 2.0 ** -22 * (top.abs() + tot.log().abs())
        return O, tolO, lse, told

    def check(self, got, c, **kw):
        """Compares (O, lse) of a kernel with the definition; returns the worst shares of the bars."""
        O, lse = (t.double().cpu() for t in got)
        O_ref, tolO, lse_ref, told = self.attend(c, **kw)
        worst = []
        for x, ref, tol in ((O, O_ref, tolO), (lse, lse_ref, told)):
            x, ref, tol = x[:int(self.cu[-1])], ref[:int(self.cu[-1])], tol[:int(self.cu[-1])]
            assert torch.equal(torch.isnan(x), torch.isnan(ref)), "NaN in other places"
            fin = torch.isfinite(ref)
            assert torch.equal(x[~fin & ~torch.isnan(ref)], ref[~fin & ~torch.isnan(ref)])
            off = (x - ref).abs()[fin]
            share = off / tol[fin].clamp(min=1e-300)
            share[off == 0] = 0
            worst.append(float(share.max()) if share.numel() else 0.0)
            assert worst[-1] <= 1.0, "off by %.3g of its bar" % worst[-1]
        return worst
