"""Cases of the cache operators: appending with rotary positions on several axes, appending to the
8-bit paged cache, and attention (decode and ragged prefill) over the 8-bit cache.

``run`` computes them in elementary torch operations, or with ``own`` set makes the library's calls.
A case fixes the sizes (lengths come from the case's own ``lens`` seed); the data come from the seed.

The 8-bit cache: kv8 [num_pages, 2, Hkv, P, D] e4m3 codes, and one power-of-two scale per (token, kv head,
K|V), kept as its exponent byte s (the scale is 2^(s - 127)) in scales [num_pages, 2, Hkv, P].  A row x with
largest magnitude amax gets s = max(exponent field of float32(amax) - 7, 1), so that amax * 2^(127 - s) lies
in [128, 256) and the row stays below 448 however it is turned.
"""
import math
import random

import numpy as np
import torch

own = False

F8 = torch.float8_e4m3fn
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # one decode step of a batch of requests: a token each, its query, key and value turned and stored
        dict(name="append16 step", op="append16", dtype="bf16", hq=32, hkv=8, d=128, p=16, batch=64, new_lo=1, new_hi=1,
             ctx_lo=50, ctx_hi=900, rotary=128, axes=3, sections="16,24,24", interleaved=False, theta=1e6, lens=1),
        # prompts with pictures, axes dealt to the pairs in turn, no earlier context
        dict(name="append16 prompts", op="append16", dtype="fp16", hq=32, hkv=8, d=128, p=16, batch=16, new_lo=128,
             new_hi=2048, ctx_lo=0, ctx_hi=1024, rotary=128, axes=3, sections="24,20,20", interleaved=True, theta=5e6, lens=2),
        # the decode step again, into the 8-bit cache; an odd number of requests
        dict(name="append8 step", op="append8", dtype="bf16", hq=32, hkv=8, d=128, p=16, batch=61, new_lo=1, new_hi=1,
             ctx_lo=50, ctx_hi=900, rotary=128, axes=3, sections="16,24,24", interleaved=False, theta=1e6, lens=3),
        # the ragged prompts into the 8-bit cache
        dict(name="append8 prompts", op="append8", dtype="bf16", hq=32, hkv=8, d=128, p=16, batch=16, new_lo=128,
             new_hi=2048, ctx_lo=0, ctx_hi=1024, rotary=128, axes=3, sections="24,20,20", interleaved=True, theta=5e6, lens=4),
        # chunks of odd lengths, half of each head turned, one kv head, pages of 5 rows
        dict(name="append8 partial rotation", op="append8", dtype="fp16", hq=7, hkv=1, d=64, p=5, batch=9, new_lo=3,
             new_hi=401, ctx_lo=0, ctx_hi=77, rotary=32, axes=2, sections="7,9", interleaved=False, theta=1e4, lens=5),
        # the small batch: latency
        dict(name="decode8 tiny", op="decode8", dtype="fp16", hq=8, hkv=2, d=64, p=16, batch=4, kv_lo=1, kv_hi=256, cap=0.0, lens=6),
        # the serving batch of an 8B-class model
        dict(name="decode8 batch", op="decode8", dtype="bf16", hq=32, hkv=8, d=128, p=16, batch=64, kv_lo=512, kv_hi=4096,
             cap=0.0, lens=7),
        # two long contexts, 8 query heads per kv head: the keys of one request spread over the whole card
        dict(name="decode8 long group 8", op="decode8", dtype="bf16", hq=64, hkv=8, d=128, p=64, batch=2, kv_lo=100001,
             kv_hi=131072, cap=0.0, lens=8),
        # one-row pages with a soft cap on the logits
        dict(name="decode8 one-row pages", op="decode8", dtype="fp16", hq=16, hkv=8, d=128, p=1, batch=23, kv_lo=300,
             kv_hi=5000, cap=30.0, lens=9),
        # two short prompts
        dict(name="prefill8 small", op="prefill8", dtype="fp16", hq=8, hkv=2, d=128, p=8, batch=2, qo_lo=40, qo_hi=150,
             ctx_lo=0, ctx_hi=60, causal=True, cap=0.0, lens=10),
        # ragged causal prompts behind cached prefixes
        dict(name="prefill8 prompts", op="prefill8", dtype="bf16", hq=32, hkv=8, d=128, p=16, batch=10, qo_lo=128, qo_hi=1500,
             ctx_lo=0, ctx_hi=1024, causal=True, cap=0.0, lens=11),
        # 64 requests' queries against the prefix that they share, every row seeing every key
        dict(name="prefill8 shared prefix", op="prefill8", dtype="bf16", hq=32, hkv=8, d=128, p=16, batch=1, qo_lo=64,
             qo_hi=64, ctx_lo=8192, ctx_hi=8192, causal=False, cap=30.0, lens=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["append16", "append8", "decode8", "decode8", "prefill8"])
    hkv = rng.choice([1, 2, 3, 4, 5, 8])
    g = rng.choice([1, 2, 4, 8])
    d = 128 if op == "prefill8" else rng.choice([64, 128])
    p = rng.choice([1, 2, 4, 8, 16, 32, 64, 128] + ([] if op == "append16" else [3, 5, 7, 11, 48]))
    c = dict(op=op, dtype=rng.choice(["bf16", "fp16"]), hq=hkv * g, hkv=hkv, d=d, p=p, lens=rng.randrange(1 << 20))
    if op in ("append16", "append8"):
        axes = rng.choice([1, 2, 3, 3, 4])
        rotary = rng.choice([d, d, d // 2, d // 4])
        cuts = sorted(rng.randrange(rotary // 2 + 1) for _ in range(axes - 1))
        sections = [b - a for a, b in zip([0] + cuts, cuts + [rotary // 2])]
        total = _log(rng, 1, 16000 * 24 // (g + 2) // hkv)
        batch = min(total, _log(rng, 1, 64))
        hi = max(1, 2 * total // batch - 1)
        return dict(c, batch=batch, new_lo=1, new_hi=hi, ctx_lo=0, ctx_hi=_log(rng, 1, 1000), rotary=rotary, axes=axes,
                    sections=",".join(map(str, sections)), interleaved=rng.random() < 0.5, theta=rng.choice([1e4, 5e5, 5e6]))
    cap = rng.choice([0.0, 0.0, 30.0])
    if op == "decode8":
        total = _log(rng, 64, 100000)
        batch = min(total, _log(rng, 1, 96))
        hi = max(2, 2 * total // batch)
        return dict(c, batch=batch, kv_lo=1, kv_hi=hi, cap=cap)
    total = _log(rng, 16, min(4000, 128000 // (hkv * g)))
    batch = min(total, _log(rng, 1, 8))
    return dict(c, batch=batch, qo_lo=1, qo_hi=max(1, min(1500, 2 * total // batch - 1)), ctx_lo=0, ctx_hi=_log(rng, 1, 2000),
                causal=rng.random() < 0.7, cap=cap)


def _lengths(c):
    """(rows of each request, keys of each request, these rows' keys among them where the rows are new)."""
    r = random.Random(c["lens"])
    if c["op"] == "decode8":
        return [1] * c["batch"], [r.randint(c["kv_lo"], c["kv_hi"]) for _ in range(c["batch"])]
    lo, hi = (c["new_lo"], c["new_hi"]) if c["op"].startswith("append") else (c["qo_lo"], c["qo_hi"])
    rows = [r.randint(lo, hi) for _ in range(c["batch"])]
    ctx = [r.randint(c["ctx_lo"], c["ctx_hi"]) for _ in range(c["batch"])]
    if c["op"] == "prefill8" and not c["causal"]:
        return rows, [max(1, x) for x in ctx]  # keys that are not the rows' own: a shared prefix, an encoder's states
    return rows, [a + b for a, b in zip(rows, ctx)]


def _cumsum(v):
    return torch.tensor([0] + list(np.cumsum(v)), dtype=torch.int32)


def _quantise(x):
    """(codes, exponent bytes) of rows x [..., D] in float32."""
    field = x.abs().amax(-1).view(torch.int32) >> 23
    s = (field - 7).clamp(min=1)
    return torch.ldexp(x, (127 - s).unsqueeze(-1)).to(F8), s.to(torch.uint8)


def _positions(rows, kv, axes, seed):
    """int32 [axes, tokens]: text counts on all axes together; a picture's tokens share the first axis and walk a
    grid on the others."""
    r = random.Random(seed)
    cols = []
    for n, length in zip(rows, kv):
        base, left = length - n + r.randint(0, 3000), n
        while left > 0:
            if left >= 24 and r.random() < 0.6:
                h = r.randint(2, max(2, min(32, int(math.sqrt(left)))))
                w = max(1, min(left // h, r.randint(2, 40)))
                i = np.arange(h * w)
                grid = [np.full(h * w, base), base + i // w, base + i % w, base + (i * 7) % (h * w)]
                cols.append(np.stack([grid[a] for a in range(axes)]))
                base += max(h, w)
                left -= h * w
            else:
                m = min(left, r.randint(1, 400))
                cols.append(np.tile(base + np.arange(m), (axes, 1)))
                base += m
                left -= m
    return torch.from_numpy(np.concatenate(cols, 1).astype(np.int32))


def prepare(case, seed):
    c = case
    g = torch.Generator("cuda").manual_seed(seed)
    rows, kv = _lengths(c)
    dtype, hq, hkv, d, p = DT[c["dtype"]], c["hq"], c["hkv"], c["d"], c["p"]
    counts = [-(-n // p) for n in kv]
    pool = sum(counts) + 3
    s = dict(case=c, rows=rows, kv=kv, n=sum(rows), pool=pool)
    s["indices"] = torch.randperm(pool, generator=g, device="cuda")[: sum(counts)].to(torch.int32)
    s["indptr_h"], s["last_h"] = _cumsum(counts), torch.tensor([n - (k - 1) * p for n, k in zip(kv, counts)], dtype=torch.int32)
    s["rows_h"] = _cumsum(rows)
    for k in ("indptr", "last", "rows"):
        s[k + "_d"] = s[k + "_h"].cuda()

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if c["op"] == "append16":
        s["cache"] = normal(pool, 2, hkv, p, d).to(dtype)
    else:
        # keys and values whose size differs from token to token
        s["cache"], s["scales"] = _quantise(normal(pool, 2, hkv, p, d) * torch.exp(0.5 * normal(pool, 2, hkv, p, 1)))
    s["q"] = normal(s["n"], hq, d).to(dtype)
    if c["op"].startswith("append"):
        s["k_new"], s["v_new"] = (normal(s["n"], hkv, d) * torch.exp(0.5 * normal(s["n"], hkv, 1)) for _ in range(2))
        s["k_new"], s["v_new"] = s["k_new"].to(dtype), s["v_new"].to(dtype)
        s["positions"] = _positions(rows, kv, c["axes"], seed).cuda()
        s["q_out"] = torch.empty_like(s["q"])
        if own:
            from paged_kv_cache_bsr_gb300 import api
            s["params"] = api.make_params(hq, hkv, d, p, dtype, 1.0)
            s["rope"] = api.make_rope_axes(c["theta"], c["rotary"], [int(x) for x in c["sections"].split(",")], c["interleaved"])
    else:
        s["sm_scale"] = 1.0 / math.sqrt(d)
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["n"], hq, device="cuda")
        if own:  # the plan that a serving loop makes once for a step and runs in every layer
            from paged_kv_cache_bsr_gb300 import api
            decode = c["op"] == "decode8"
            s["plan"] = api.Plan(api.PLAN_DECODE_KV8 if decode else api.PLAN_PREFILL_KV8, num_qo_heads=hq, num_kv_heads=hkv,
                                 head_dim=d, page_size=p, dtype=dtype, sm_scale=s["sm_scale"], logits_cap=c["cap"],
                                 causal=bool(c.get("causal")), max_batch=c["batch"], max_total_q=s["n"], max_kv_pages=sum(counts))
            s["plan"].plan(s["indptr_h"], s["last_h"], pool, qo_indptr_h=None if decode else s["rows_h"],
                           kv_indices_h=s["indices"].cpu())
    return s


def run(state):
    s = state
    if s["case"]["op"].startswith("append"):
        return _append_own(s) if own else _append(s)
    return _attend_own(s) if own else _attend(s)


def _append_own(s):
    from paged_kv_cache_bsr_gb300 import api
    if s["case"]["op"] == "append16":
        api.append_paged_kv_axes(s["params"], s["rope"], s["rows_d"], s["indptr_d"], s["indices"], s["last_d"], s["positions"],
                                 s["k_new"], s["v_new"], s["cache"], s["q"], s["q_out"])
        return {"kv": s["cache"], "q": s["q_out"]}
    api.append_paged_kv8(s["params"], s["rope"], s["rows_d"], s["indptr_d"], s["indices"], s["last_d"], s["positions"],
                         s["k_new"], s["v_new"], s["cache"], s["scales"], s["q"], s["q_out"])
    return {"kv": s["cache"], "scales": s["scales"], "q": s["q_out"]}


def _attend_own(s):
    s["plan"].run(s["q"], s["cache"], s["indices"], s["indptr_d"], s["last_d"], s["o"], s["lse"],
                  qo_indptr=s["rows_d"] if s["case"]["op"] == "prefill8" else None, kv_scales=s["scales"])
    return {"o": s["o"], "lse": s["lse"]}


def _axis_of_pair(c):
    """The axis that each pair of elements turns by."""
    sections = [int(x) for x in c["sections"].split(",")]
    axis = np.repeat(np.arange(len(sections)), sections)
    if c["interleaved"]:  # dealt in turn, an axis without pairs left passed over
        turn = np.concatenate([np.arange(n) for n in sections])
        axis = axis[np.lexsort((axis, turn))]
    return torch.from_numpy(axis).cuda()


def _turn(x, cos, sin, rotary):
    """x [n, heads, D] in float32, cos and sin [n, rotary / 2]."""
    h = rotary // 2
    a, b = x[..., :h], x[..., h:rotary]
    cos, sin = cos.unsqueeze(1), sin.unsqueeze(1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., rotary:]], -1)


def _append(s):
    c, p = s["case"], s["case"]["p"]
    t = torch.arange(s["n"], device="cuda")
    b = torch.searchsorted(s["rows_d"], t, right=True) - 1
    first, end = s["rows_d"][b], s["rows_d"][b + 1]
    length = (s["indptr_d"][b + 1] - s["indptr_d"][b] - 1) * p + s["last_d"][b]
    place = length - (end - first) + (t - first)
    page, slot = s["indices"][s["indptr_d"][b] + place // p].long(), place % p
    pair = torch.arange(c["rotary"] // 2, device="cuda", dtype=torch.float64)
    angle = s["positions"][_axis_of_pair(c)].T.double() * c["theta"] ** (-2.0 * pair / c["rotary"])
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    k, v = s["k_new"].float(), s["v_new"].float()
    s["q_out"].copy_(_turn(s["q"].float(), cos, sin, c["rotary"]))
    if c["op"] == "append16":
        s["cache"][page, 0, :, slot] = _turn(k, cos, sin, c["rotary"]).to(s["cache"].dtype)
        s["cache"][page, 1, :, slot] = s["v_new"]
        return {"kv": s["cache"], "q": s["q_out"]}
    field = k.abs().amax(-1).view(torch.int32) >> 23
    k_s = (field - 7).clamp(min=1)
    k8 = torch.ldexp(_turn(k, cos, sin, c["rotary"]), (127 - k_s).unsqueeze(-1)).to(F8)
    v8, v_s = _quantise(v)
    codes = s["cache"].view(torch.uint8)
    codes[page, 0, :, slot], codes[page, 1, :, slot] = k8.view(torch.uint8), v8.view(torch.uint8)
    s["scales"][page, 0, :, slot], s["scales"][page, 1, :, slot] = k_s.to(torch.uint8), v_s
    return {"kv": s["cache"], "scales": s["scales"], "q": s["q_out"]}


def _attend(s):
    """The requests side by side, filled up to the longest with masked rows and keys."""
    c = s["case"]
    hq, hkv, d, p, batch = c["hq"], c["hkv"], c["d"], c["p"], c["batch"]
    group, rows, keys = hq // hkv, max(s["rows"]), max(s["kv"])
    b = torch.arange(batch, device="cuda").unsqueeze(1)
    n_keys = ((s["indptr_d"][1:] - s["indptr_d"][:-1] - 1) * p + s["last_d"]).unsqueeze(1)
    n_rows = (s["rows_d"][1:] - s["rows_d"][:-1]).unsqueeze(1)
    j = torch.arange(keys, device="cuda").unsqueeze(0)
    at = (s["indptr_d"][:-1].unsqueeze(1) + j // p).clamp(max=s["indices"].numel() - 1)
    page, slot = s["indices"][at].long(), j % p
    codes = s["cache"].view(torch.uint8)

    def read(which):  # [batch, hkv, keys, d]
        x = codes[page, which, :, slot].view(F8).float()
        e = s["scales"][page, which, :, slot].to(torch.int32) - 127
        return torch.ldexp(x, e.unsqueeze(-1)).transpose(1, 2)

    i = torch.arange(rows, device="cuda").unsqueeze(0)
    row = (s["rows_d"][:-1].unsqueeze(1) + i).clamp(max=s["n"] - 1)
    q = s["q"][row].float().view(batch, rows, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(batch, hkv, group * rows, d)
    x = torch.matmul(q, read(0).transpose(2, 3)).mul_(s["sm_scale"])
    if c["cap"] > 0:
        x = c["cap"] * torch.tanh(x / c["cap"])
    seen = (j < n_keys).unsqueeze(1)  # [batch, rows, keys]
    if c.get("causal"):
        seen = seen & (j.unsqueeze(1) <= (i + n_keys - n_rows).unsqueeze(2))
    x = x.view(batch, hkv, group, rows, keys).masked_fill_(~seen.view(batch, 1, 1, -1, keys), -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(batch, hkv, group * rows, keys), read(1)).view(batch, hkv, group, rows, d) / total
    lse = (top + total.log()).squeeze(-1)
    mine = i < n_rows
    s["o"].copy_(o.permute(0, 3, 1, 2, 4).reshape(batch, rows, hq, d)[mine])
    s["lse"].copy_(lse.permute(0, 3, 1, 2).reshape(batch, rows, hq)[mine])
    return {"o": s["o"], "lse": s["lse"]}


def _pairs(c):
    """(query row, key) pairs that are attended."""
    rows, kv = _lengths(c)
    return sum(n * k - (n * (n - 1) // 2 if c.get("causal") else 0) for n, k in zip(rows, kv))


def work(case):
    c = case
    rows, kv = _lengths(c)
    n, hq, hkv, d = sum(rows), c["hq"], c["hkv"], c["d"]
    if c["op"].startswith("append"):
        out = 2 * hkv * d * 2 if c["op"] == "append16" else 2 * hkv * (d + 1)
        table = 4 * sum(-(-a // c["p"]) for a in rows) + 12 * c["batch"]
        return {"bytes": n * (2 * hkv * d * 2 + out + 2 * hq * d * 2 + 4 * c["axes"]) + table,
                "flops": n * (hq + hkv) * c["rotary"] * 3}
    table = 4 * sum(-(-k // c["p"]) for k in kv) + 12 * c["batch"]
    return {"bytes": sum(kv) * 2 * hkv * (d + 1) + n * hq * (2 * d * 2 + 4) + table, "flops": 4 * d * hq * _pairs(c)}


def _e4m3(x):
    """The e4m3 value next to x (|x| < 464), ties to the even one."""
    step = torch.exp2(torch.frexp(x)[1].double().sub(1).clamp(min=-6) - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    s, c = prepare(case, seed), case
    rows, kv, p, hkv, d = s["rows"], s["kv"], c["p"], c["hkv"], c["d"]
    start, r0 = s["indptr_h"].tolist(), s["rows_h"].tolist()
    if c["op"].startswith("append"):
        axis = [[a] * int(n) for a, n in enumerate(c["sections"].split(","))]
        if c["interleaved"]:
            order = [x.pop() for _ in range(c["rotary"] // 2) for x in axis if x]
        else:
            order = sum(axis, [])
        h = c["rotary"] // 2
        angle = torch.stack([s["positions"][a].double() * math.exp(-2.0 * i / c["rotary"] * math.log(c["theta"]))
                             for i, a in enumerate(order)], 1)
        z = torch.polar(torch.ones_like(angle), angle).unsqueeze(1)

        def turned(x):
            y = torch.complex(x[..., :h], x[..., h : 2 * h]) * z
            return torch.cat([y.real, y.imag, x[..., 2 * h :]], -1)

        out = s["cache"].double()
        k, v, k_to = s["k_new"].double(), s["v_new"].double(), s.get("scales")
        k_new, v_new = turned(k), v
        if c["op"] == "append8":
            k_e, v_e = (torch.frexp(x.abs().amax(-1).clamp(min=2.0**-126))[1].sub(1).add(120).clamp(min=1) for x in (k, v))
            k_new = _e4m3(k_new * torch.exp2(127.0 - k_e.double()).unsqueeze(-1))
            v_new = _e4m3(v_new * torch.exp2(127.0 - v_e.double()).unsqueeze(-1))
        for b in range(c["batch"]):
            place = torch.arange(kv[b] - rows[b], kv[b], device="cuda")
            page = s["indices"][start[b] + place // p].long()
            new = slice(r0[b], r0[b + 1])
            out[page, 0, :, place % p], out[page, 1, :, place % p] = k_new[new], v_new[new]
            if c["op"] == "append8":
                k_to[page, 0, :, place % p], k_to[page, 1, :, place % p] = k_e[new].to(torch.uint8), v_e[new].to(torch.uint8)
        got = {"kv": out, "q": turned(s["q"].double())}
        return got if c["op"] == "append16" else dict(got, scales=k_to)
    if _pairs(c) * c["hq"] * d > 2e12:
        return None
    o, lse = torch.empty(s["n"], c["hq"], d, dtype=torch.float64, device="cuda"), torch.empty(s["n"], c["hq"], dtype=torch.float64, device="cuda")
    for b in range(c["batch"]):
        pages = s["indices"][start[b] : start[b + 1]].long()
        x = s["cache"].view(torch.uint8)[pages].view(F8).double() * torch.exp2(s["scales"][pages].double() - 127).unsqueeze(-1)
        x = x.permute(1, 2, 0, 3, 4).reshape(2, hkv, -1, d)[:, :, : kv[b]]
        for head in range(c["hq"]):
            k, v = x[:, head // (c["hq"] // hkv)]
            y = s["q"][r0[b] : r0[b + 1], head].double() @ k.T * (1 / math.sqrt(d))
            if c["cap"] > 0:
                y = c["cap"] * torch.tanh(y / c["cap"])
            if c.get("causal"):
                y = y.masked_fill(torch.ones_like(y, dtype=torch.bool).triu(kv[b] - rows[b] + 1), -math.inf)
            o[r0[b] : r0[b + 1], head] = torch.softmax(y, -1) @ v
            lse[r0[b] : r0[b + 1], head] = torch.logsumexp(y, -1)
    return {"o": o, "lse": lse}
