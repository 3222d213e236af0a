"""Cases of the operators that bound a cache's length: attention over whole prompts that are packed one
behind another (no pages yet), the accumulated attention weight of every cached key, the choice of the keys
to keep, and the move of the kept keys to the front of a page list.

``run`` computes them in elementary torch operations, or with ``own`` set makes the library's calls.
A case fixes the sizes (lengths come from the case's own ``lens`` seed); the data come from the seed.

Key weights [num_pages, Hkv, P] float32 lie beside the cache.  A call adds, for every key j of a request, kv head
h and the call's query rows i of the heads that share h, the probabilities exp(logit - lse) that the attention
over the same keys gave:  w[j, h] = decay * w[j, h] + sum over i of p[i, j],  where a key from the request's
``weighed`` on (keys that were not there before) starts from 0.  The kept keys of a request are, up to its budget,
its last ``window`` keys, then its first ``sink`` ones, then those of the largest weight (the lower index first
where weights are equal), for each kv head its own; they stay in their order.
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
        # two short prompts of odd lengths: latency
        dict(name="ragged short", op="ragged", dtype="fp16", hq=8, hkv=2, batch=2, qo_lo=33, qo_hi=150, ctx_lo=0, ctx_hi=0,
             causal=True, cap=0.0, fused=True, lens=1),
        # ragged prompts of an 8B-class model, queries, keys and values as views of one projection's output
        dict(name="ragged prompts", op="ragged", dtype="bf16", hq=32, hkv=8, batch=10, qo_lo=128, qo_hi=1500, ctx_lo=0,
             ctx_hi=0, causal=True, cap=0.0, fused=True, lens=2),
        # rows that attend to another sequence's states (every row sees every key), a head each, logits capped
        dict(name="ragged across", op="ragged", dtype="bf16", hq=12, hkv=12, batch=5, qo_lo=40, qo_hi=900, ctx_lo=200,
             ctx_hi=1501, causal=False, cap=30.0, fused=False, lens=3),
        # the small batch's decode step: latency
        dict(name="weights tiny", op="weights", dtype="fp16", hq=8, hkv=2, d=64, p=16, batch=4, qo_lo=1, qo_hi=1, ctx_lo=0,
             ctx_hi=255, causal=False, cap=0.0, kv8=False, decay=1.0, lens=4),
        # one decode step of the serving batch of an 8B-class model
        dict(name="weights step", op="weights", dtype="bf16", hq=32, hkv=8, d=128, p=16, batch=64, qo_lo=1, qo_hi=1,
             ctx_lo=511, ctx_hi=4095, causal=False, cap=0.0, kv8=False, decay=1.0, lens=5),
        # a decode step of two long contexts in the 8-bit cache, 8 query heads per kv head, older weight fading
        dict(name="weights 8-bit long", op="weights", dtype="bf16", hq=64, hkv=8, d=128, p=64, batch=2, qo_lo=1, qo_hi=1,
             ctx_lo=100000, ctx_hi=131071, causal=False, cap=0.0, kv8=True, decay=0.95, lens=6),
        # whole prompts, every row weighing the keys it sees
        dict(name="weights prompts", op="weights", dtype="bf16", hq=32, hkv=8, d=128, p=16, batch=10, qo_lo=128, qo_hi=1500,
             ctx_lo=0, ctx_hi=0, causal=True, cap=0.0, kv8=False, decay=0.0, lens=7),
        # the last rows of long prompts weigh the keys before them; small pages, logits capped
        dict(name="weights last rows", op="weights", dtype="fp16", hq=16, hkv=8, d=128, p=4, batch=7, qo_lo=32, qo_hi=64,
             ctx_lo=2000, ctx_hi=9001, causal=True, cap=30.0, kv8=False, decay=0.0, lens=8),
        # the serving batch keeps half of its keys
        dict(name="select batch", op="select", hkv=8, p=16, batch=64, kv_lo=512, kv_hi=4096, part=0.5, sink=4, window=32, lens=9),
        # two long contexts keep a sixteenth
        dict(name="select long", op="select", hkv=8, p=64, batch=2, kv_lo=100001, kv_hi=131072, part=0.0625, sink=4,
             window=128, lens=10),
        # the serving batch's kept keys move to the front of their own pages, each with its weight
        dict(name="compact batch", op="compact", dtype="bf16", hkv=8, d=128, p=16, batch=64, kv_lo=512, kv_hi=4096, part=0.5,
             kv8=False, weights=True, in_place=True, lens=11),
        # one long prompt of the 8-bit cache into other pages (its own are shared)
        dict(name="compact 8-bit prompt", op="compact", dtype="bf16", hkv=8, d=128, p=16, batch=1, kv_lo=8001, kv_hi=12000,
             part=0.2, kv8=True, weights=False, in_place=False, lens=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["ragged", "weights", "weights", "select", "compact"])
    hkv = rng.choice([1, 2, 3, 4, 5, 8])
    g = rng.choice([1, 2, 4, 8])
    p = rng.choice([1, 2, 3, 4, 5, 7, 8, 11, 16, 32, 48, 64, 128])
    lens = rng.randrange(1 << 20)
    dtype = rng.choice(["bf16", "fp16"])
    cap = rng.choice([0.0, 0.0, 30.0])
    if op in ("select", "compact"):
        total = _log(rng, 16, 200000 if op == "select" else 100000)
        batch = min(total, _log(rng, 1, 64))
        c = dict(op=op, hkv=hkv, p=p, batch=batch, kv_lo=1, kv_hi=max(2, 2 * total // batch), part=rng.choice([0.05, 0.25, 0.5, 0.9, 1.0]), lens=lens)
        if op == "select":
            return dict(c, sink=rng.choice([0, 1, 4]), window=rng.choice([0, 1, 16, 64]))
        kv8 = rng.random() < 0.4
        return dict(c, dtype=dtype, d=rng.choice([64, 128]), kv8=kv8, weights=rng.random() < 0.5, in_place=rng.random() < 0.6)
    causal = rng.random() < 0.7
    if op == "ragged" or rng.random() < 0.5:
        total = _log(rng, 16, min(4000, 128000 // (hkv * g)))
        batch = min(total, _log(rng, 1, 8))
        c = dict(op=op, dtype=dtype, hq=hkv * g, hkv=hkv, batch=batch, qo_lo=1, qo_hi=max(1, min(1500, 2 * total // batch - 1)),
                 ctx_lo=0, ctx_hi=_log(rng, 1, 2000), causal=causal, cap=cap, lens=lens)
        if op == "ragged":
            fused = causal and rng.random() < 0.6
            return dict(c, fused=fused, ctx_hi=0 if fused else c["ctx_hi"])
    else:
        total = _log(rng, 64, 100000)
        batch = min(total, _log(rng, 1, 96))
        c = dict(op=op, dtype=dtype, hq=hkv * g, hkv=hkv, batch=batch, qo_lo=1, qo_hi=1, ctx_lo=0, ctx_hi=max(1, 2 * total // batch),
                 causal=causal, cap=cap, lens=lens)
    return dict(c, d=128 if c["qo_hi"] > 1 else rng.choice([64, 128]), p=p, kv8=rng.random() < 0.4, decay=rng.choice([0.0, 1.0, 0.9]))


def _lengths(c):
    """(query rows of each request, keys of each request)."""
    r = random.Random(c["lens"])
    if c["op"] in ("select", "compact"):
        return [0] * c["batch"], [r.randint(c["kv_lo"], c["kv_hi"]) for _ in range(c["batch"])]
    rows = [r.randint(c["qo_lo"], c["qo_hi"]) for _ in range(c["batch"])]
    ctx = [r.randint(c["ctx_lo"], c["ctx_hi"]) for _ in range(c["batch"])]
    if c["op"] == "ragged" and not c["causal"]:
        return rows, [max(1, x) for x in ctx]  # another sequence's keys
    return rows, [a + b for a, b in zip(rows, ctx)]


def _kept(c):
    return [max(1, int(n * c["part"])) for n in _lengths(c)[1]]


def _cumsum(v):
    return torch.tensor([0] + list(np.cumsum(v)), dtype=torch.int32)


def _quantise(x):
    """(codes, exponent bytes) of rows x [..., D] in float32: the 8-bit cache's power-of-two scale for each row."""
    s = ((x.abs().amax(-1).view(torch.int32) >> 23) - 7).clamp(min=1)
    return torch.ldexp(x, (127 - s).unsqueeze(-1)).to(F8), s.to(torch.uint8)


def prepare(case, seed):
    c = case
    g = torch.Generator("cuda").manual_seed(seed)
    rows, kv = _lengths(c)
    hkv, batch, op = c["hkv"], c["batch"], c["op"]
    s = dict(case=c, rows=rows, kv=kv, n=sum(rows))

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s["rows_h"] = _cumsum(rows)
    s["rows_d"] = s["rows_h"].cuda()
    if op == "ragged":
        hq, d, dtype = c["hq"], 128, DT[c["dtype"]]
        s["kv_h"] = _cumsum(kv)
        s["kv_d"] = s["kv_h"].cuda()
        if c["fused"]:
            x = normal(s["n"], hq + 2 * hkv, d).to(dtype)
            s["q"], s["k"], s["v"] = x[:, :hq], x[:, hq : hq + hkv], x[:, hq + hkv :]
        else:
            s["q"], s["k"], s["v"] = (normal(n, h, d).to(dtype) for n, h in ((s["n"], hq), (sum(kv), hkv), (sum(kv), hkv)))
        s["sm_scale"] = 1.0 / math.sqrt(d)
        s["o"] = torch.empty(s["n"], hq, d, dtype=dtype, device="cuda")
        s["lse"] = torch.empty(s["n"], hq, device="cuda")
        if own:  # the plan that a serving loop makes once for a batch of prompts and runs in every layer
            from paged_kv_cache_bsr_gb300 import api
            s["plan"] = api.Plan(api.PLAN_PREFILL_RAGGED, num_qo_heads=hq, num_kv_heads=hkv, head_dim=d, page_size=1, dtype=dtype,
                                 sm_scale=s["sm_scale"], logits_cap=c["cap"], causal=c["causal"], max_batch=batch,
                                 max_total_q=s["n"], max_kv_pages=sum(kv))
            s["plan"].plan(s["kv_h"], None, sum(kv), qo_indptr_h=s["rows_h"])
        return s
    p = c["p"]
    counts = [-(-n // p) for n in kv]
    to = _kept(c) if op == "compact" and not c["in_place"] else []
    pool = sum(counts) + sum(-(-n // p) for n in to) + 3
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    s["indices"] = order[: sum(counts)].clone()
    s["indptr_d"] = _cumsum(counts).cuda()
    s["last_d"] = torch.tensor([n - (k - 1) * p for n, k in zip(kv, counts)], dtype=torch.int32).cuda()
    if op == "select":
        # the sums of many small probabilities and a few large ones, on a grid so that some are equal
        s["weights"] = torch.exp(1.5 * normal(pool, hkv, p)).mul_(256).round_().div_(256)
        s["budget"] = torch.tensor(_kept(c), dtype=torch.int32).cuda()
        s["keep"] = torch.empty(batch, hkv, max(_kept(c)), dtype=torch.int32, device="cuda")
        s["kept_len"] = torch.empty(batch, dtype=torch.int32, device="cuda")
        return s
    d, dtype = c["d"], DT[c["dtype"]]
    s["cache"], s["scales"] = normal(pool, 2, hkv, p, d).mul_(torch.exp(0.5 * normal(pool, 2, hkv, p, 1))), None
    if c["kv8"]:
        s["cache"], s["scales"] = _quantise(s["cache"])
    else:
        s["cache"] = s["cache"].to(dtype)
    if op == "compact":
        s["weights"] = torch.exp(1.5 * normal(pool, hkv, p)) if c["weights"] else None
        most = max(_kept(c))
        s["keep"] = torch.full((batch, hkv, most), -1, dtype=torch.int32, device="cuda")
        for b, n in enumerate(_kept(c)):
            x = torch.rand(hkv, kv[b], generator=g, device="cuda").argsort(-1)[:, :n].sort(-1)[0]
            s["keep"][b, :, :n] = x.to(torch.int32)
        s["kept_len"] = torch.tensor(_kept(c), dtype=torch.int32).cuda()
        s["to_indptr"] = s["to_indices"] = None
        if not c["in_place"]:
            s["to_indptr"] = _cumsum([-(-n // p) for n in to]).cuda()
            s["to_indices"] = order[sum(counts) : pool - 3].clone()
        return s
    s["q"] = normal(s["n"], c["hq"], d).to(dtype)
    s["sm_scale"] = 1.0 / math.sqrt(d)
    s["lse"] = _paged_logits(s)[1]  # what the attention call of the same rows gave
    s["weights"] = torch.rand(pool, hkv, p, generator=g, device="cuda").mul_(3.0)
    s["weighed"] = torch.tensor([k - n for n, k in zip(rows, kv)], dtype=torch.int32).cuda()
    if own:
        from paged_kv_cache_bsr_gb300 import api
        s["params"] = api.make_params(c["hq"], hkv, d, p, dtype, s["sm_scale"], c["cap"], c["causal"])
    return s


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        from paged_kv_cache_bsr_gb300 import api
        if op == "ragged":
            s["plan"].run_ragged(s["q"], s["k"], s["v"], s["o"], s["lse"])
        elif op == "weights":
            one = s["case"]["qo_hi"] == 1
            api.add_key_weights(s["params"], s["indptr_d"], s["indices"], s["last_d"], s["q"], s["lse"], s["cache"], s["weights"],
                                qo_indptr=None if one else s["rows_d"], kv_scales=s["scales"], decay=s["case"]["decay"],
                                weighed_len=s["weighed"])
        elif op == "select":
            api.select_keys(s["indptr_d"], s["indices"], s["last_d"], s["weights"], s["budget"], s["keep"], s["kept_len"],
                            sink=s["case"]["sink"], window=s["case"]["window"])
        else:
            api.compact_paged_kv(s["indptr_d"], s["indices"], s["last_d"], s["keep"], s["kept_len"], s["cache"],
                                 kv_scales=s["scales"], weights=s["weights"], dst_indptr=s["to_indptr"], dst_indices=s["to_indices"])
    else:
        {"ragged": _ragged, "weights": _weights, "select": _select, "compact": _compact}[op](s)
    if op == "ragged":
        return {"o": s["o"], "lse": s["lse"]}
    if op == "weights":
        return {"weights": s["weights"]}
    if op == "select":
        return {"keep": s["keep"], "kept_len": s["kept_len"]}
    return {"cache": s["cache"], "scales": s["scales"], "weights": s["weights"]}


# ---- plain forms: the requests side by side, filled up to the longest with masked rows and keys


def _seen(s, n_rows, n_keys):
    """[batch, 1, 1, rows, keys]: which keys each row sees."""
    i = torch.arange(max(s["rows"]), device="cuda").view(1, -1, 1)
    j = torch.arange(max(s["kv"]), device="cuda").view(1, 1, -1)
    n_rows, n_keys = n_rows.view(-1, 1, 1), n_keys.view(-1, 1, 1)
    seen = (j < n_keys) & (i < n_rows)
    if s["case"]["causal"]:
        seen = seen & (j <= i + n_keys - n_rows)
    return seen.view(len(s["rows"]), 1, 1, max(s["rows"]), -1)


def _logits(s, k, n_keys):
    """Masked logits [batch, hkv, group, rows, keys] of k [batch, keys, hkv, d] in float32, their lse, and the rows'
    places."""
    c = s["case"]
    hq, hkv, batch = c["hq"], c["hkv"], c["batch"]
    group, d = hq // hkv, k.shape[-1]
    i = torch.arange(max(s["rows"]), device="cuda").unsqueeze(0)
    n_rows = (s["rows_d"][1:] - s["rows_d"][:-1]).unsqueeze(1)
    row = (s["rows_d"][:-1].unsqueeze(1) + i).clamp(max=s["n"] - 1)
    q = s["q"][row].float().view(batch, -1, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(batch, hkv, -1, d)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(s["sm_scale"]).view(batch, hkv, group, i.numel(), -1)
    if c["cap"] > 0:
        x = x.div_(c["cap"]).tanh_().mul_(c["cap"])
    x.masked_fill_(~_seen(s, n_rows, n_keys), -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-3e38)
    lse = (top + (x - top).exp_().sum(-1, keepdim=True).log_())
    return x, lse, i < n_rows


def _places(s, keys):
    """Keys 0 .. keys - 1 of every request: (page, slot) [batch, keys], and the requests' lengths."""
    p = s["case"]["p"]
    n_keys = (s["indptr_d"][1:] - s["indptr_d"][:-1] - 1) * p + s["last_d"]
    j = torch.arange(keys, device="cuda").unsqueeze(0)
    at = (s["indptr_d"][:-1].unsqueeze(1) + j // p).clamp(max=s["indices"].numel() - 1)
    return s["indices"][at].long(), (j % p).expand(at.shape), n_keys


def _paged_logits(s):
    page, slot, n_keys = _places(s, max(s["kv"]))
    if s["scales"] is None:
        k = s["cache"][page, 0, :, slot].float()
    else:
        k = s["cache"].view(torch.uint8)[page, 0, :, slot].view(F8).float()
        k = torch.ldexp(k, (s["scales"][page, 0, :, slot].to(torch.int32) - 127).unsqueeze(-1))
    x, lse, mine = _logits(s, k, n_keys)
    return x, lse.squeeze(-1).permute(0, 3, 1, 2).reshape(len(s["rows"]), -1, s["case"]["hq"])[mine]


def _ragged(s):
    c = s["case"]
    hq, hkv, batch = c["hq"], c["hkv"], c["batch"]
    j = torch.arange(max(s["kv"]), device="cuda").unsqueeze(0)
    n_keys = s["kv_d"][1:] - s["kv_d"][:-1]
    at = (s["kv_d"][:-1].unsqueeze(1) + j).clamp(max=s["k"].shape[0] - 1)
    x, lse, mine = _logits(s, s["k"][at].float(), n_keys)
    x = x.sub_(lse).exp_()
    o = torch.matmul(x.view(batch, hkv, -1, j.numel()), s["v"][at].float().transpose(1, 2)).view(batch, hkv, hq // hkv, -1, 128)
    s["o"].copy_(o.permute(0, 3, 1, 2, 4).reshape(batch, -1, hq, 128)[mine])
    s["lse"].copy_(lse.squeeze(-1).permute(0, 3, 1, 2).reshape(batch, -1, hq)[mine])


def _weights(s):
    c = s["case"]
    hkv, batch = c["hkv"], c["batch"]
    x = _paged_logits(s)[0]
    i = torch.arange(max(s["rows"]), device="cuda").unsqueeze(0)
    row = (s["rows_d"][:-1].unsqueeze(1) + i).clamp(max=s["n"] - 1)
    lse = s["lse"][row].view(batch, -1, hkv, c["hq"] // hkv).permute(0, 2, 3, 1).unsqueeze(-1)
    add = x.sub_(lse).exp_().sum((2, 3))  # [batch, hkv, keys]
    page, slot, n_keys = _places(s, max(s["kv"]))
    j = torch.arange(max(s["kv"]), device="cuda").unsqueeze(0)
    old = s["weights"][page, :, slot] * ((j < s["weighed"].unsqueeze(1)) * c["decay"]).unsqueeze(-1)
    mine = j < n_keys.unsqueeze(1)
    s["weights"][page[mine], :, slot[mine]] = (old + add.transpose(1, 2))[mine]


def _select(s):
    c = s["case"]
    page, slot, n_keys = _places(s, max(s["kv"]))
    j = torch.arange(max(s["kv"]), device="cuda").view(1, 1, -1)
    n = torch.minimum(s["budget"], n_keys.to(torch.int32))
    kept, n_keys = n.view(-1, 1, 1), n_keys.view(-1, 1, 1)
    window, sink = (j >= n_keys - c["window"]) & (j < n_keys), j < c["sink"]
    w = s["weights"][page, :, slot].transpose(1, 2)  # [batch, hkv, keys]
    # the last keys from the back, the first ones from the front, the others by weight, what is past the end last
    w = torch.where(window, j.float(), torch.where(sink, -j.float(), w))
    kind = torch.where(j >= n_keys, 3, torch.where(window, 0, torch.where(sink, 1, 2))).expand(w.shape)
    order = torch.argsort(w, dim=-1, descending=True, stable=True)
    order = torch.gather(order, -1, torch.argsort(torch.gather(kind, -1, order), dim=-1, stable=True))
    most = s["keep"].shape[-1]
    order = order[..., :most]
    first = torch.arange(most, device="cuda").view(1, 1, -1) < kept
    order = torch.where(first, order, 1 << 30).sort(-1)[0]
    s["keep"].copy_(torch.where(first, order, -1))
    s["kept_len"].copy_(n)


def _compact(s):
    c = s["case"]
    p, batch = c["p"], c["batch"]
    src = s["keep"].clamp(min=0).long()  # [batch, hkv, most]
    i = torch.arange(src.shape[-1], device="cuda").view(1, 1, -1)
    head = torch.arange(c["hkv"], device="cuda").view(1, -1, 1).expand(src.shape)
    mine = (i < s["kept_len"].view(-1, 1, 1)).expand(src.shape)
    start, to_start = s["indptr_d"][:-1].view(-1, 1, 1), s["indptr_d"][:-1].view(-1, 1, 1)
    to_table = s["indices"]
    if s["to_indptr"] is not None:
        to_start, to_table = s["to_indptr"][:-1].view(-1, 1, 1), s["to_indices"]
    page = s["indices"][start + src // p].long()[mine]
    to = to_table[(to_start + i // p).expand(src.shape)[mine]].long()
    at, to_slot, head = (src % p)[mine], (i % p).expand(src.shape)[mine], head[mine]
    x = s["cache"].view(torch.uint8) if c["kv8"] else s["cache"]
    x[to, :, head, to_slot] = x[page, :, head, at]
    if c["kv8"]:
        s["scales"][to, :, head, to_slot] = s["scales"][page, :, head, at]
    if s["weights"] is not None:
        s["weights"][to, head, to_slot] = s["weights"][page, head, at]


def _pairs(c):
    """(query row, key) pairs that are attended."""
    rows, kv = _lengths(c)
    return sum(n * k - (n * (n - 1) // 2 if c["causal"] else 0) for n, k in zip(rows, kv))


def work(case):
    c = case
    rows, kv = _lengths(c)
    n, hkv = sum(rows), c["hkv"]
    if c["op"] == "ragged":
        return {"bytes": 2 * 128 * (2 * n * c["hq"] + 2 * sum(kv) * hkv) + 4 * n * c["hq"], "flops": 4 * 128 * c["hq"] * _pairs(c)}
    table = 4 * sum(-(-k // c["p"]) for k in kv) + 12 * c["batch"]
    if c["op"] == "weights":
        row = c["d"] + 1 if c["kv8"] else 2 * c["d"]
        return {"bytes": sum(kv) * hkv * (row + (8 if c["decay"] else 4)) + n * c["hq"] * (2 * c["d"] + 4) + table,
                "flops": 2 * c["d"] * c["hq"] * _pairs(c)}
    kept = sum(min(a, b) for a, b in zip(_kept(c), kv))
    if c["op"] == "select":
        return {"bytes": 4 * hkv * (sum(kv) + kept) + table, "flops": hkv * sum(kv)}
    row = 2 * (c["d"] + 1 if c["kv8"] else 2 * c["d"]) + (4 if c["weights"] else 0)
    return {"bytes": kept * hkv * (2 * row + 4) + table, "flops": 0}


def _plain_kv(s, b, which):
    """Keys (0) or values (1) [hkv, keys, d] of request b in 64 bits."""
    lo, hi = s["indptr_d"][b : b + 2].tolist()
    pages = s["indices"][lo:hi].long()
    x = s["cache"][pages, which]
    x = x.double() if s["scales"] is None else x.view(torch.uint8).view(F8).double() * torch.exp2(s["scales"][pages, which].double() - 127).unsqueeze(-1)
    return x.transpose(0, 1).reshape(x.shape[1], -1, x.shape[-1])[:, : s["kv"][b]]


def _exact_rows(s, b, head, k):
    """Capped and masked logits of request b's rows of one head against keys k."""
    c = s["case"]
    r0, r1 = s["rows_h"][b : b + 2].tolist()
    y = s["q"][r0:r1, head].double() @ k.T * (1 / math.sqrt(k.shape[-1]))
    if c["cap"] > 0:
        y = c["cap"] * torch.tanh(y / c["cap"])
    if c["causal"]:
        y = y.masked_fill(torch.ones_like(y, dtype=torch.bool).triu(s["kv"][b] - s["rows"][b] + 1), -math.inf)
    return y, slice(r0, r1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    rows, kv, hkv, batch = s["rows"], s["kv"], c["hkv"], c["batch"]
    if c["op"] in ("ragged", "weights"):
        group = c["hq"] // hkv
        if _pairs(c) * c["hq"] * 128 > 2e12:
            return None
    if c["op"] == "ragged":
        o = torch.empty(s["n"], c["hq"], 128, dtype=torch.float64, device="cuda")
        lse = torch.empty(s["n"], c["hq"], dtype=torch.float64, device="cuda")
        for b in range(batch):
            k0, k1 = s["kv_h"][b : b + 2].tolist()
            for head in range(c["hq"]):
                y, at = _exact_rows(s, b, head, s["k"][k0:k1, head // group].double())
                o[at, head], lse[at, head] = torch.softmax(y, -1) @ s["v"][k0:k1, head // group].double(), torch.logsumexp(y, -1)
        return {"o": o, "lse": lse}
    start, p = s["indptr_d"].tolist(), c["p"]

    def slots(b, token):
        return s["indices"][start[b] + token // p].long(), token % p

    if c["op"] == "weights":
        w = s["weights"].double()
        for b in range(batch):
            keys = _plain_kv(s, b, 0)
            page, slot = slots(b, torch.arange(kv[b], device="cuda"))
            for h in range(hkv):
                old = w[page, h, slot] * c["decay"]
                old[kv[b] - rows[b] :] = 0
                for head in range(h * group, (h + 1) * group):
                    y, at = _exact_rows(s, b, head, keys[h])
                    old += torch.exp(y - s["lse"][at, head].double().unsqueeze(1)).sum(0)
                w[page, h, slot] = old
        return {"weights": w}
    if c["op"] == "select":
        keep = torch.full(s["keep"].shape, -1, dtype=torch.int64)
        kept_len = torch.zeros(batch, dtype=torch.int64)
        for b in range(batch):
            n = kept_len[b] = min(_kept(c)[b], kv[b])
            page, slot = slots(b, torch.arange(kv[b], device="cuda"))
            tail = min(c["window"], int(n))
            front = min(c["sink"], int(n) - tail, kv[b] - tail)
            left = int(n) - tail - front
            sure = list(range(front)) + list(range(kv[b] - tail, kv[b]))
            for h in range(hkv):
                w = s["weights"][page, h, slot].cpu().numpy()[front : kv[b] - tail]
                best = np.lexsort((np.arange(w.size), -w.astype(np.float64)))[:left] + front
                keep[b, h, : int(n)] = torch.tensor(sorted(sure + best.tolist()))
        return {"keep": keep, "kept_len": kept_len}
    out = {k: None if s[k] is None else (s[k].double() if k != "scales" else s[k].long()) for k in ("cache", "scales", "weights")}
    old = {k: None if v is None else v.clone() for k, v in out.items()}
    for b, n in enumerate(_kept(c)):
        i = torch.arange(n, device="cuda")
        if s["to_indptr"] is None:
            to, to_slot = slots(b, i)
        else:
            to, to_slot = s["to_indices"][int(s["to_indptr"][b]) + i // p].long(), i % p
        for h in range(hkv):
            page, slot = slots(b, s["keep"][b, h, :n].long())
            out["cache"][to, :, h, to_slot] = old["cache"][page, :, h, slot]
            if out["scales"] is not None:
                out["scales"][to, :, h, to_slot] = old["scales"][page, :, h, slot]
            if out["weights"] is not None:
                out["weights"][to, h, to_slot] = old["weights"][page, h, slot]
    return out
