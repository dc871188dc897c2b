"""Attention of many query rows over keys they share: the workloads it is measured on.

Two operators, each in its plain form (elementary torch operations in fp32)
and as the library's kernels compute it:

``cross``   cross attention of a decoder's tokens to an encoder's states,
            which have a length of their own for each batch entry;
``prefix``  decode attention of a batch whose sequences all begin with the
            same long prefix, held once, before keys of their own.

A case is a dict: ``op``; ``batch``, ``tokens`` (new query tokens of a batch
entry), ``q_heads``, ``kv_heads``, ``dim`` (head_dim), ``dtype``; ``keys``,
the capacity along the encoder's states or the sequences' own keys, of which
the entries use between ``least`` and ``keys``; and for ``prefix`` also
``prefix`` (the length), ``room`` (the capacity that holds it) and
``causal``.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}

# The largest work of a listed case: what a drawn one may cost.
MOST_FLOPS = 4 * 4 * 2048 * 32 * 8192 * 128
MOST_BYTES = 4 * 128 * 131072 * 8


def _cross(name, batch, tokens, heads, dim, keys, least, dtype):
    return {"name": name, "op": "cross", "batch": batch, "tokens": tokens, "q_heads": heads[0], "kv_heads": heads[1],
            "dim": dim, "keys": keys, "least": least, "dtype": dtype}


def _prefix(name, batch, tokens, heads, dim, prefix, room, keys, least, dtype, causal=False):
    return {"name": name, "op": "prefix", "batch": batch, "tokens": tokens, "q_heads": heads[0],
            "kv_heads": heads[1], "dim": dim, "prefix": prefix, "room": room, "keys": keys, "least": least,
            "dtype": dtype, "causal": causal}


def listed():
    return [
        # one token of one request against a short input: nothing but latency
        _cross("cross_token", 1, 1, (8, 1), 64, 512, 512, "bf16"),
        # a decode step of a batch of eight, inputs of unequal length
        _cross("cross_step", 8, 1, (32, 8), 128, 4096, 1000, "bf16"),
        # short prompts, a KV head for every query head, nothing a multiple of anything
        _cross("cross_odd", 3, 77, (12, 12), 64, 1023, 200, "fp16"),
        # prompts of ordinary length against inputs of unequal length
        _cross("cross_prompt", 8, 256, (32, 8), 128, 4096, 1000, "bf16"),
        # wide heads: eight query heads on a KV head of 256 elements
        _cross("cross_wide", 2, 333, (16, 2), 256, 5001, 4000, "bf16"),
        # a few tokens against one very long input: little to share the work by but the keys
        _cross("cross_document", 1, 64, (64, 8), 128, 131072, 131072, "fp16"),
        # long prompts against long inputs: all arithmetic
        _cross("cross_large", 4, 2048, (32, 8), 128, 8192, 8000, "bf16"),
        # four short requests behind a short instruction
        _prefix("prefix_small", 4, 1, (8, 1), 64, 512, 512, 64, 1, "bf16"),
        # an ordinary batch behind one system prompt, early in its answers
        _prefix("prefix_batch", 32, 1, (32, 8), 128, 4000, 4096, 512, 1, "bf16"),
        # speculative decoding: four new tokens a sequence, causal among them
        _prefix("prefix_drafts", 32, 4, (16, 2), 64, 8191, 8191, 2048, 4, "fp16", True),
        # wide heads behind a long document
        _prefix("prefix_wide", 24, 1, (16, 2), 256, 20000, 20480, 300, 10, "bf16"),
        # a large batch behind a long document, with long answers of its own
        _prefix("prefix_large", 128, 1, (64, 8), 128, 32768, 32768, 2048, 1, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    c = {"op": rng.choice(["cross", "prefix"]), "dtype": rng.choice(["bf16", "fp16"]),
         "dim": rng.choice([64, 64, 128, 128, 128, 256])}
    c["q_heads"], c["kv_heads"] = rng.choice([(8, 1), (12, 12), (16, 2), (32, 8), (64, 8), (24, 8), (10, 2), (28, 4)])
    group = c["q_heads"] // c["kv_heads"]
    if c["op"] == "cross":
        c["batch"] = _log(rng, 1, 32)
        c["tokens"] = _log(rng, 1, 2048)
        c["keys"] = _log(rng, 128, 131072)
    else:
        c["batch"] = _log(rng, 2, 160)
        c["tokens"] = rng.randint(1, max(1, 32 // group)) if rng.random() < 0.3 else 1
        c["prefix"] = _log(rng, 100, 65536)
        c["room"] = c["prefix"] + rng.choice([0, 0, rng.randint(1, 999)])
        c["keys"] = _log(rng, max(8, c["tokens"]), 4096)
        c["causal"] = rng.random() < 0.5
    c["least"] = rng.randint(c["tokens"] if c["op"] == "prefix" else 1, c["keys"])
    while work(c)["flops"] > MOST_FLOPS or work(c)["bytes"] > MOST_BYTES:
        for k in ("batch", "tokens") if c["op"] == "cross" else ("batch",):
            c[k] = max(1, c[k] * 3 // 4)
        low = c["tokens"] if c["op"] == "prefix" else 1
        c["keys"], c["least"] = max(low, c["keys"] * 3 // 4), max(low, c["least"] * 3 // 4)
    return c


def _lengths(case):
    """The batch's lengths, spread evenly over their range (a seed shuffles them)."""
    n, lo, hi = case["batch"], case["least"], case["keys"]
    return [hi - (hi - lo) * i // max(1, n - 1) for i in range(n)]


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    B, T, H, K, d = case["batch"], case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(dtype)

    lens = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
    s = {"case": case, "q": normal(B, T, H, d), "k": normal(B, case["keys"], K, d), "v": normal(B, case["keys"], K, d),
         "lens": lens[torch.randperm(B, generator=gen, device="cuda")].contiguous()}
    if case["op"] == "prefix":
        s["k_prefix"], s["v_prefix"] = normal(case["room"], K, d), normal(case["room"], K, d)
        s["prefix_len"] = torch.tensor([case["prefix"]], dtype=torch.int32, device="cuda")
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(B, T, H, dtype=torch.float32, device="cuda")
    return s


def run(state):
    if own:
        return _kernels(state)
    return _plain_cross(state) if state["case"]["op"] == "cross" else _plain_prefix(state)


def _kernels(s):
    import gqa_decode_blackwell_gb300 as g

    # the workspace of these shapes, kept from the first call on
    if s["case"]["op"] == "cross":
        if "workspace" not in s:
            s["workspace"] = _bytes(g.gqa_cross_workspace_size(s["q"], s["k"]))
        g.gqa_cross_attn(s["q"], s["k"], s["v"], s["lens"], s["out"], s["lse"], s["workspace"])
    else:
        if "workspace" not in s:
            s["workspace"] = _bytes(g.gqa_prefix_workspace_size(s["q"], s["k_prefix"], s["k"],
                                                                causal=s["case"]["causal"]))
        g.gqa_prefix_attn(s["q"], s["k_prefix"], s["v_prefix"], s["prefix_len"], s["k"], s["v"], s["lens"], s["out"],
                          s["lse"], s["workspace"], causal=s["case"]["causal"])
    return s["out"], s["lse"]


def _bytes(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda") if n else None


def _softmax(scores):
    """(weights, logarithm of their sum) of each row of scores; a row that sees nothing gives 0 and -inf."""
    top = scores.amax(-1, keepdim=True)
    weights = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    total = weights.sum(-1, keepdim=True)
    return weights / torch.where(total == 0, 1.0, total), (top + torch.log(total)).squeeze(-1)


def _plain_cross(s):
    B, T, H, d = s["q"].shape
    N, K = s["k"].shape[1:3]
    G = H // K
    # [B, K, T G, d]: the rows of the query heads that share a KV head together
    q = s["q"].float().view(B, T, K, G, d).permute(0, 2, 1, 3, 4).reshape(B, K, T * G, d)
    scores = q @ s["k"].float().permute(0, 2, 3, 1) / math.sqrt(d)
    hidden = torch.arange(N, device="cuda")[None, :] >= s["lens"][:, None]
    w, lse = _softmax(scores.masked_fill(hidden[:, None, None, :], -math.inf))
    out = w @ s["v"].float().permute(0, 2, 1, 3)
    out = out.view(B, K, T, G, d).permute(0, 2, 1, 3, 4).reshape(B, T, H, d)
    return out.to(s["q"].dtype), lse.view(B, K, T, G).permute(0, 2, 1, 3).reshape(B, T, H)


def _plain_prefix(s):
    B, T, H, d = s["q"].shape
    P, (N, K) = s["k_prefix"].shape[0], s["k"].shape[1:3]
    G = H // K
    q = s["q"].float().view(B, T, K, G, d).permute(2, 0, 1, 3, 4)  # [K, B, T, G, d]
    shared = q.reshape(K, B * T * G, d) @ s["k_prefix"].float().permute(1, 2, 0)
    alone = q.reshape(K, B, T * G, d) @ s["k"].float().permute(2, 0, 3, 1)
    shared, alone = shared.view(K, B, T, G, P) / math.sqrt(d), alone.view(K, B, T, G, N) / math.sqrt(d)
    shared = shared.masked_fill(torch.arange(P, device="cuda") >= s["prefix_len"], -math.inf)
    end = s["lens"][:, None].expand(B, T)
    if s["case"]["causal"]:
        end = s["lens"][:, None] - T + 1 + torch.arange(T, device="cuda")[None, :]
    hidden = torch.arange(N, device="cuda")[None, None, :] >= end[:, :, None]
    alone = alone.masked_fill(hidden[None, :, :, None, :], -math.inf)
    w, lse = _softmax(torch.cat([shared, alone], -1))
    out = w[..., :P].reshape(K, B * T * G, P) @ s["v_prefix"].float().permute(1, 0, 2)
    out = out.view(K, B, T * G, d) + w[..., P:].reshape(K, B, T * G, N) @ s["v"].float().permute(2, 0, 1, 3)
    out = out.view(K, B, T, G, d).permute(1, 2, 0, 3, 4).reshape(B, T, H, d)
    return out.to(s["q"].dtype), lse.permute(1, 2, 0, 3).reshape(B, T, H)


def work(case):
    B, T, H, K, d = case["batch"], case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
    keys = sum(_lengths(case))
    seen, held = keys * T, keys  # (query token, key) pairs; positions of K and V to read
    if case["op"] == "prefix":
        if case["causal"]:
            seen -= B * T * (T - 1) // 2
        seen, held = seen + B * T * case["prefix"], held + case["prefix"]
    return {"bytes": 4 * d * K * held + 4 * d * B * T * H + 4 * B * T * H, "flops": 4 * d * H * seen}


def exact(case, seed):
    """The definition in fp64, one KV head of one batch entry at a time over the keys it sees."""
    s = prepare(case, seed)
    B, T, H, K, d = case["batch"], case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
    G = H // K
    lens = s["lens"].tolist()
    out = torch.zeros(B, T, H, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, T, H), -math.inf, dtype=torch.float64, device="cuda")
    for h in range(K):
        heads = slice(h * G, (h + 1) * G)
        if case["op"] == "prefix":
            kp = s["k_prefix"][: case["prefix"], h].double()
            vp = s["v_prefix"][: case["prefix"], h].double()
        for b in range(B):
            keys, values = s["k"][b, : lens[b], h].double(), s["v"][b, : lens[b], h].double()
            first = 0
            if case["op"] == "prefix":
                keys, values, first = torch.cat([kp, keys]), torch.cat([vp, values]), case["prefix"]
            x = torch.einsum("tgd,jd->tgj", s["q"][b, :, heads].double(), keys) * d ** -0.5
            if case.get("causal"):
                position = torch.arange(first + lens[b], device="cuda") - first
                last = lens[b] - T + torch.arange(T, device="cuda")
                future = (position[None, :] >= 0) & (position[None, :] > last[:, None])
                x[future[:, None, :].expand(T, G, -1)] = -math.inf
            total = torch.logsumexp(x, -1)
            lse[b, :, heads] = total
            out[b, :, heads] = torch.einsum("tgj,jd->tgd", torch.exp(x - total[..., None]), values)
    return out, lse
