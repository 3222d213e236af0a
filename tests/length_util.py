"""Shared helpers of the tests of key weights, kept keys and their move: a paged batch on the GPU, and the
definitions in 64 bits."""
import math

import numpy as np
import torch

BF, FP = torch.bfloat16, torch.float16


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def starts(lens):
    return [sum(lens[:i]) for i in range(len(lens) + 1)]


class Paged:
    """Requests of kv_lens keys in pages of P rows scattered over a pool, with queries of qo_lens rows (None: one
    row each and no row pointer).  Slots that hold no key are NaN."""

    def __init__(self, kv_lens, P, hkv, d=128, dtype=BF, kv8=False, qo_lens=None, group=4, seed=0, spread=0.0, extra=3):
        g = torch.Generator("cuda").manual_seed(seed)
        self.kv_lens, self.P, self.hkv, self.d, self.dtype, self.group = list(kv_lens), P, hkv, d, dtype, group
        self.rows = [1] * len(kv_lens) if qo_lens is None else list(qo_lens)
        counts = [-(-n // P) for n in kv_lens]
        self.pool = sum(counts) + extra
        order = torch.randperm(self.pool, generator=g, device="cuda").to(torch.int32)
        self.indices = order[:sum(counts)].contiguous()
        self.indptr = ints(starts(counts))
        self.last = ints([n - (k - 1) * P if n else 0 for n, k in zip(kv_lens, counts)])
        self.qo = None if qo_lens is None else ints(starts(qo_lens))
        shape = (self.pool, 2, hkv, P, d)
        x = torch.randn(shape, generator=g, device="cuda")
        if spread:
            x = x * torch.exp2(torch.randn(shape[:-1], generator=g, device="cuda") * spread).unsqueeze(-1)
        held = torch.zeros(self.pool, P, dtype=torch.bool, device="cuda")
        for b, n in enumerate(kv_lens):
            page, slot = self.places(b, torch.arange(n, device="cuda"))
            held[page, slot] = True
        self.held = held
        if kv8:
            s = ((x.abs().amax(-1).view(torch.int32) >> 23) - 7).clamp(min=1)
            codes = torch.ldexp(x, (127 - s).unsqueeze(-1)).to(torch.float8_e4m3fn)
            codes.view(torch.uint8).masked_fill_(~held[:, None, None, :, None], 0x7F)
            self.kv, self.scales = codes, s.to(torch.uint8).masked_fill_(~held[:, None, None, :], 255)
        else:
            self.kv, self.scales = x.to(dtype).masked_fill_(~held[:, None, None, :, None], float("nan")), None
        self.q = torch.randn(sum(self.rows), hkv * group, d, generator=g, device="cuda").to(dtype)

    def places(self, b, token):
        """(page, slot) of request b's tokens."""
        first = int(self.indptr[b])
        return self.indices[first + token // self.P].long(), token % self.P

    def values(self, b, which):
        """Keys (0) or values (1) [hkv, n, d] of request b in 64 bits."""
        page, slot = self.places(b, torch.arange(self.kv_lens[b], device="cuda"))
        if self.scales is None:
            x = self.kv[page, which, :, slot].double()
        else:
            x = self.kv.view(torch.uint8)[page, which, :, slot].view(torch.float8_e4m3fn).double()
            x = x * torch.exp2(self.scales[page, which, :, slot].double() - 127).unsqueeze(-1)
        return x.transpose(0, 1)

    def logits(self, b, sm_scale, cap=0.0, causal=False):
        """[hkv, group, rows, keys] in 64 bits, -inf where a row does not see a key."""
        r0 = sum(self.rows[:b])
        n, keys = self.rows[b], self.kv_lens[b]
        q = self.q[r0:r0 + n].double().view(n, self.hkv, self.group, self.d).permute(1, 2, 0, 3)
        y = sm_scale * torch.matmul(q, self.values(b, 0).transpose(1, 2).unsqueeze(1))
        if cap > 0:
            y = cap * torch.tanh(y / cap)
        if causal:
            y = y.masked_fill(torch.ones_like(y, dtype=torch.bool).triu(keys - n + 1), -math.inf)
        return y

    def lse(self, sm_scale, cap=0.0, causal=False):
        """What the attention call of these rows returns, float32 [rows, heads]."""
        out = [torch.logsumexp(self.logits(b, sm_scale, cap, causal), -1).permute(2, 0, 1).reshape(-1, self.hkv * self.group)
               for b in range(len(self.rows))]
        return torch.cat(out).float() if out else torch.zeros(0, self.hkv * self.group, device="cuda")

    def new_weights(self, lse, before, sm_scale, cap=0.0, causal=False, decay=1.0, weighed=None):
        """(weights, the bound of their error): the definition in 64 bits.  A logit is a sum of d exact
        products in fp32, off by at most d 2^-24 sum |q k| sm_scale (<= 2^-16 sum |q k| sm for d = 128, counted
        once more for the scaling, the cap and lse), and a probability by that share and 2^-21 for its
        exponential; fp32 sums of n terms in blocks lose at most 2^-24 for each of the up to 64 + n / 64 additions
        that a term goes through."""
        w, err = before.double().clone(), torch.zeros_like(before, dtype=torch.float64)
        for b, n in enumerate(self.kv_lens):
            if n == 0:
                continue
            page, slot = self.places(b, torch.arange(n, device="cuda"))
            r0, r1 = sum(self.rows[:b]), sum(self.rows[:b + 1])
            old = w[page, :, slot] * decay if decay else torch.zeros(n, self.hkv, dtype=torch.float64, device="cuda")
            if weighed is not None:
                old[weighed[b]:] = 0
            y = self.logits(b, sm_scale, cap, causal)
            l = lse[r0:r1].double().view(r1 - r0, self.hkv, self.group).permute(1, 2, 0).unsqueeze(-1)
            p = torch.where(torch.isneginf(y) | torch.isneginf(l), 0.0, torch.exp(y - l))
            q = self.q[r0:r1].double().view(r1 - r0, self.hkv, self.group, self.d).permute(1, 2, 0, 3)
            size = sm_scale * torch.matmul(q.abs(), self.values(b, 0).abs().transpose(1, 2).unsqueeze(1))
            adds = 64 + p.shape[1] * p.shape[2] / 64
            off = p * (size * 2.0 ** -15 + l.abs().masked_fill(torch.isneginf(l), 0) * 2.0 ** -22 + 2.0 ** -21 + (cap or 0) * 2.0 ** -20)
            w[page, :, slot] = old + p.sum((1, 2)).transpose(0, 1)
            err[page, :, slot] = off.sum((1, 2)).transpose(0, 1) + (adds * 2.0 ** -24) * (old.abs() + p.sum((1, 2)).transpose(0, 1)) + 1e-30
        return w, err
