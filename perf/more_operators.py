"""Serving with a paged cache and drafted tokens: the workloads it is measured on.

Four operators, each in its plain form (elementary torch operations in fp32,
angles in fp64) and as the library's kernels compute it:

``rotary``  the position rotation of a tensor of heads;
``append``  new queries and keys rotated, keys and values put into a paged
            cache (pages of ``page`` positions, a table of pages a sequence);
``tree``    attention of a tree of drafted tokens over the paged cache that
            holds them; one token is an ordinary decode step;
``step``    a verification step as a serving loop makes it: the drafts' tree
            from their parents, append, attention, and the accepted branch
            moved together in the cache.

A case is a dict: ``op``; ``batch``, ``tokens`` (new tokens of a sequence, at
most), ``q_heads``, ``kv_heads``, ``dim`` (head_dim), ``dtype``; ``keys``, the
most positions a sequence has with its new tokens, of which the sequences use
between ``least`` and ``keys``; ``ragged``: sequences have unequal numbers of
new tokens; ``page``; ``heads_first``: a page is [kv_heads, page, dim] and not
[page, kv_heads, dim]; and for the rotation ``rotated`` (elements of a head),
``interleaved``, ``base``, ``scaling``, ``factor``, ``original`` (the length
before scaling) and ``inverse``.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}

# Turns over the original length between which the scaling by parts goes from
# positions divided by the factor to positions as they are.
SLOW, FAST = 1.0, 32.0


def _rope(rotated, interleaved=False, base=10000.0, scaling="none", factor=1.0, original=0):
    return {"rotated": rotated, "interleaved": interleaved, "base": base, "scaling": scaling, "factor": factor,
            "original": original}


def _rotary(name, batch, tokens, heads, dim, keys, least, dtype, rope, inverse=False):
    return {"name": name, "op": "rotary", "batch": batch, "tokens": tokens, "q_heads": heads, "kv_heads": heads,
            "dim": dim, "keys": keys, "least": least, "dtype": dtype, "inverse": inverse, **rope}


def _append(name, batch, tokens, heads, dim, page, keys, least, dtype, rope, ragged=False, heads_first=False):
    return {"name": name, "op": "append", "batch": batch, "tokens": tokens, "q_heads": heads[0],
            "kv_heads": heads[1], "dim": dim, "page": page, "keys": keys, "least": least, "dtype": dtype,
            "ragged": ragged, "heads_first": heads_first, **rope}


def _tree(name, batch, tokens, heads, dim, page, keys, least, dtype, ragged=False, heads_first=False):
    return {"name": name, "op": "tree", "batch": batch, "tokens": tokens, "q_heads": heads[0], "kv_heads": heads[1],
            "dim": dim, "page": page, "keys": keys, "least": least, "dtype": dtype, "ragged": ragged,
            "heads_first": heads_first}


def _step(name, batch, tokens, heads, dim, page, keys, least, dtype, rope, ragged=False):
    return {**_append(name, batch, tokens, heads, dim, page, keys, least, dtype, rope, ragged), "op": "step"}


def listed():
    return [
        # the queries of one decode step of a batch of eight: latency
        _rotary("rotary_step", 8, 1, 32, 128, 4096, 1000, "bf16", _rope(128, base=500000.0)),
        # the gradient of long prompts' queries, half of each head rotated in pairs of neighbours, context
        # stretched eightfold by parts
        _rotary("rotary_prompt", 4, 2048, 32, 128, 65536, 60000, "bf16",
                _rope(64, True, 10000.0, "parts", 8.0, 8192), inverse=True),
        # one new token of each of eight sequences
        _append("append_step", 8, 1, (32, 8), 128, 16, 4096, 1000, "bf16", _rope(128, base=500000.0)),
        # odd sizes: a KV head for every query head, 20 of 64 elements rotated, prompts of unequal length
        _append("append_odd", 3, 77, (12, 12), 64, 16, 1023, 200, "fp16",
                _rope(20, True, 10000.0, "linear", 4.0), ragged=True),
        # chunks of long prompts, of unequal length, into pages with the heads first
        _append("append_prompt", 8, 1024, (32, 8), 128, 64, 8192, 3000, "bf16",
                _rope(128, False, 10000.0, "base", 4.0), ragged=True, heads_first=True),
        # one token of one sequence: nothing but latency
        _tree("tree_token", 1, 1, (8, 1), 64, 16, 512, 512, "bf16"),
        # a decode step of a batch of eight over pages, sequences of unequal length
        _tree("tree_step", 8, 1, (32, 8), 128, 16, 4096, 1000, "bf16"),
        # an ordinary tree for each of a batch, of unequal size
        _tree("tree_drafts", 16, 26, (32, 8), 128, 32, 8192, 1000, "bf16", ragged=True),
        # wide heads, a larger tree, pages with the heads first
        _tree("tree_wide", 8, 40, (16, 2), 256, 64, 10007, 5000, "fp16", heads_first=True),
        # large trees behind long documents: 512 query rows of a KV head
        _tree("tree_long", 4, 64, (64, 8), 128, 128, 100000, 90000, "bf16"),
        # a whole step of four short requests with small trees
        _step("step_small", 4, 7, (8, 1), 64, 16, 600, 100, "bf16", _rope(64), ragged=True),
        # and of an ordinary batch
        _step("step_batch", 32, 16, (32, 8), 128, 32, 2048, 300, "bf16", _rope(128, base=500000.0), ragged=True),
    ]


# What a drawn case may cost: the largest work of a listed case of its operator, and its scores in fp32.
MOST = {"rotary": 2 ** 26, "append": 2 ** 26, "step": 2 ** 27}  # elements of x; of q, k, v; of the caches
MOST_FLOPS = 4 * 128 * 64 * 64 * 4 * 95000
MOST_SCORES = 4 * 64 * 64 * 100000
MOST_KEYS = 4 * 100000 * 8 * 128  # elements of K


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "append", "tree", "tree", "step"])
    c = {"op": op, "dtype": rng.choice(["bf16", "fp16"]), "dim": rng.choice([64, 64, 128, 128, 128, 256])}
    c["q_heads"], c["kv_heads"] = rng.choice([(8, 1), (12, 12), (16, 2), (32, 8), (64, 8), (24, 8), (10, 2), (28, 4)])
    if op == "rotary":
        c["kv_heads"] = c["q_heads"]
        c["batch"], c["tokens"], c["keys"] = _log(rng, 1, 64), _log(rng, 1, 4096), _log(rng, 4096, 500000)
        c["dtype"], c["inverse"] = rng.choice(["bf16", "fp16", "fp32"]), rng.random() < 0.5
    else:
        c["page"] = rng.choice([16, 16, 32, 64, 128, 256])
        c["ragged"], c["heads_first"] = rng.random() < 0.5, rng.random() < 0.3
        c["batch"] = _log(rng, 1, 64)
        c["tokens"] = _log(rng, 1, 2048 if op == "append" else 64)
        c["keys"] = _log(rng, max(64, c["tokens"]), 131072 if op == "tree" else 16384)
    if op != "tree":
        c["rotated"] = rng.choice([c["dim"], c["dim"], c["dim"] // 2, 2 * rng.randint(1, c["dim"] // 2)])
        c["interleaved"], c["base"] = rng.random() < 0.5, rng.choice([10000.0, 500000.0])
        c["scaling"] = rng.choice(["none", "linear", "base", "parts"])
        c["factor"] = 1.0 if c["scaling"] == "none" else rng.choice([2.0, 4.0, 8.0])
        c["original"] = 4096 if c["scaling"] == "parts" else 0

    def costs():
        new = c["batch"] * c["tokens"] * c["dim"]
        held = c["batch"] * c["keys"] * c["kv_heads"] * c["dim"]
        if op == "rotary":
            return new * c["q_heads"] > MOST["rotary"]
        if op == "append":
            return new * (c["q_heads"] + 2 * c["kv_heads"]) > MOST["append"] or held > MOST["step"]
        if op == "step" and held > MOST["step"]:
            return True
        c["least"] = c["keys"]
        return (held > MOST_KEYS or work(c)["flops"] > MOST_FLOPS
                or c["batch"] * c["tokens"] * c["q_heads"] * c["keys"] > MOST_SCORES)

    while costs():
        for k in ("batch", "tokens"):
            c[k] = max(1, c[k] * 3 // 4)
        if op != "rotary":
            c["keys"] = max(c["tokens"], c["keys"] * 3 // 4)
    c["least"] = rng.randint(c["tokens"], max(c["tokens"], c["keys"]))
    return c


def _lengths(case):
    """The batch's lengths with their new tokens, spread evenly over their range (a seed shuffles them)."""
    n, lo, hi = case["batch"], case["least"], case["keys"]
    return [hi - (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _news(case):
    """And their numbers of new tokens."""
    n, most = case["batch"], case["tokens"]
    return [max(1, most - (most - 1) * i // max(1, n - 1)) if case.get("ragged") else most for i in range(n)]


def _frequencies(case):
    """Radians a position of each pair of elements, in fp64."""
    r, base, s = case["rotated"], case["base"], case["factor"]
    if case["scaling"] == "base" and r > 2:
        base = base * s ** (r / (r - 2))
    f = base ** (-torch.arange(0, r, 2, dtype=torch.float64, device="cuda") / r)
    if case["scaling"] == "linear":
        f = f / s
    if case["scaling"] == "parts":
        keep = ((f * case["original"] / (2 * math.pi) - SLOW) / (FAST - SLOW)).clamp(0, 1)
        f = f / s * (1 - keep) + f * keep
    return f


def _magnitude(case):
    return 0.1 * math.log(case["factor"]) + 1 if case["scaling"] == "parts" else 1.0


def _words(seen):
    """[..., n] truth values as int32 words of 32 bits, the first the lowest."""
    n = seen.shape[-1]
    seen = torch.nn.functional.pad(seen, (0, -n % 32)).view(*seen.shape[:-1], -1, 32)
    return (seen.long() << torch.arange(32, device="cuda")).sum(-1).to(torch.int32)


def _bits(words, n):
    """The inverse of _words."""
    return ((words.long()[..., None] >> torch.arange(32, device="cuda")) & 1).bool().flatten(-2)[..., :n]


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    B, T, H, K, d = case["batch"], case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(dtype)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    order = torch.randperm(B, generator=gen, device="cuda")
    lens = ints(_lengths(case))[order].contiguous()
    s = {"case": case}
    if case["op"] != "tree":
        s["frequencies"] = _frequencies(case)
        if own:
            import gqa_decode_blackwell_gb300 as g

            s["turns"] = g.rotary_turns(case["rotated"], case["base"], scaling=case["scaling"], factor=case["factor"],
                                        original_length=case["original"], device="cuda")
    if case["op"] == "rotary":
        s["x"] = normal(B, T, H, d)
        s["out"] = torch.empty_like(s["x"])
        s["positions"] = (lens[:, None] - T + torch.arange(T, device="cuda")).to(torch.int32).contiguous()
        return s
    news = ints(_news(case))[torch.randperm(B, generator=gen, device="cuda")].contiguous()
    s["lens"], s["news"] = lens, news if case["ragged"] else None

    # pages in no order, and -1 behind a sequence's last
    P = case["page"]
    most = (case["keys"] + P - 1) // P
    pages = B * most + 3
    table = torch.randperm(pages, generator=gen, device="cuda")[: B * most].view(B, most).to(torch.int32)
    used = torch.arange(most, device="cuda")[None, :] * P < lens[:, None]
    s["table"] = torch.where(used, table, -1).contiguous()
    shape = (pages, K, P, d) if case["heads_first"] else (pages, P, K, d)
    for name in ("k_cache", "v_cache"):
        cache = normal(*shape)
        s[name] = cache.transpose(1, 2) if case["heads_first"] else cache

    if case["op"] in ("append", "step"):
        # as a projection of all three leaves them: views of one tensor
        qkv = normal(B, T, H + 2 * K, d)
        s["q"], s["k"], s["v"] = qkv[:, :, :H], qkv[:, :, H: H + K], qkv[:, :, H + K:]
        s["q_out"] = torch.zeros(B, T, H, d, dtype=dtype, device="cuda")
    else:
        s["q"] = normal(B, T, H, d)
    if case["op"] in ("tree", "step"):
        # a token's parent is an earlier one or (-1) the last token before them
        u = torch.rand(B, T, generator=gen, device="cuda")
        s["parents"] = (u * (torch.arange(T, device="cuda") + 1)).floor().long().sub(1).to(torch.int32)
        seen = _ancestors(s["parents"].long())
        if case["op"] == "tree":
            s["tree"] = _words(seen) if T > 1 else None
        else:
            # the branch that a target model accepted ends at some token
            last = (torch.rand(B, generator=gen, device="cuda") * news).floor().long()
            branch = seen[torch.arange(B, device="cuda"), last]
            s["keep"] = branch.sum(-1).to(torch.int32)
            at = torch.where(branch, torch.arange(T, device="cuda"), T).sort(-1).values
            s["path"] = torch.where(at < T, at, -1).to(torch.int32).contiguous()
            W = (T + 31) // 32
            s["tree"] = torch.zeros(B, T, W, dtype=torch.int32, device="cuda")
            s["positions"] = torch.zeros(B, T, dtype=torch.int32, device="cuda")
            s["lens_out"] = torch.zeros_like(lens)
        s["out"] = torch.empty(B, T, H, d, dtype=dtype, device="cuda")
        s["lse"] = torch.empty(B, T, H, dtype=torch.float32, device="cuda")
    return s


def run(state):
    return (_kernels if own else _plain)(state)


def _kernels(s):
    import gqa_decode_blackwell_gb300 as g

    c, op = s["case"], s["case"]["op"]
    if op == "rotary":
        g.gqa_rotary_apply(s["x"], s["positions"], s["turns"], s["out"], interleaved=c["interleaved"],
                           inverse=c["inverse"], magnitude=_magnitude(c))
        return s["out"]
    if op == "step":
        g.gqa_tree_from_parents(s["parents"], s["lens"], s["tree"], s["positions"], new_lens=s["news"])
    if op != "tree":
        g.gqa_paged_append(s["q"], s["k"], s["v"], s["q_out"], s["k_cache"], s["v_cache"], s["table"], s["lens"],
                           new_lens=s["news"], positions=s["positions"] if op == "step" else None, turns=s["turns"],
                           interleaved=c["interleaved"], magnitude=_magnitude(c))
    if op == "append":
        return s["q_out"], s["k_cache"], s["v_cache"]
    q = s["q"] if op == "tree" else s["q_out"]
    if "workspace" not in s:  # of these shapes, kept from the first call on
        n = g.gqa_tree_workspace_size(q, s["k_cache"], s["table"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    g.gqa_tree_attn(q, s["k_cache"], s["v_cache"], s["table"], s["lens"], s["out"], s["lse"], s["workspace"],
                    new_lens=s["news"], tree=s["tree"])
    if op == "tree":
        return s["out"], s["lse"]
    g.gqa_paged_keep(s["k_cache"], s["v_cache"], s["table"], s["lens"], s["path"], s["keep"], s["lens_out"],
                     new_lens=s["news"], tokens=c["tokens"])
    return s["tree"], s["positions"], s["out"], s["lse"], s["k_cache"], s["v_cache"], s["lens_out"]


# ------------------------------------------------------------- plain forms
def _ancestors(parents):
    """[B, T, T]: whether token j is token t itself or one of its ancestors."""
    B, T = parents.shape
    seen = torch.zeros(B, T, T, dtype=torch.bool, device="cuda")
    rows = torch.arange(B, device="cuda")
    for t in range(T):
        above = parents[:, t]
        if t:
            seen[:, t] = seen[rows, above.clamp(min=0)] & (above >= 0)[:, None]
        seen[:, t, t] = True
    return seen


def _turned(x, positions, case, frequencies):
    """x [B, T, heads, d] rotated in fp32, rounded once."""
    r = case["rotated"]
    angle = positions.double()[..., None] * frequencies * (-1 if case.get("inverse") else 1)
    cos, sin = (torch.cos(angle) * _magnitude(case)).float(), (torch.sin(angle) * _magnitude(case)).float()
    cos, sin = cos[:, :, None], sin[:, :, None]
    y = x.float()
    if case["interleaved"]:
        a, b = y[..., 0:r:2], y[..., 1:r:2]
        front = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = y[..., : r // 2], y[..., r // 2: r]
        front = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([front, y[..., r:]], -1).to(x.dtype)


def _counts(s):
    T = s["case"]["tokens"]
    return s["news"] if s["news"] is not None else torch.full_like(s["lens"], T)


def _places(s, index):
    """Pages and positions within them of each sequence's positions [B, n] (those outside it anywhere)."""
    P = s["case"]["page"]
    index = index.clamp(min=0, max=s["table"].shape[1] * P - 1)
    return s["table"].long().gather(1, index // P).clamp(min=0), index % P


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "rotary":
        return _turned(s["x"], s["positions"], case, s["frequencies"])
    T = case["tokens"]
    t = torch.arange(T, device="cuda")
    first = (s["lens"] - _counts(s)).long()
    tree, positions = s.get("tree"), first[:, None] + t
    if op == "step":
        live = t[None, :] < _counts(s)[:, None]
        seen = _ancestors(s["parents"].long()) & live[:, :, None] & live[:, None, :]
        tree, positions = _words(seen), torch.where(live, first[:, None] + seen.sum(-1) - 1, 0)
    if op != "tree":
        b, i = (t[None, :] < _counts(s)[:, None]).nonzero(as_tuple=True)
        page, at = (x[b, i] for x in _places(s, first[:, None] + t))
        s["q_out"][b, i] = _turned(s["q"], positions, case, s["frequencies"])[b, i]
        s["k_cache"][page, at] = _turned(s["k"], positions, case, s["frequencies"])[b, i]
        s["v_cache"][page, at] = s["v"][b, i]
    if op == "append":
        return s["q_out"], s["k_cache"], s["v_cache"]
    out, lse = _plain_attention(s, s["q"] if op == "tree" else s["q_out"], tree)
    if op == "tree":
        return out, lse
    b, i = (t[None, :] < s["keep"][:, None]).nonzero(as_tuple=True)
    old = [x[b, i] for x in _places(s, first[:, None] + s["path"].long())]
    new = [x[b, i] for x in _places(s, first[:, None] + t)]
    for cache in (s["k_cache"], s["v_cache"]):
        cache[new[0], new[1]] = cache[old[0], old[1]]
    return (tree, positions.to(torch.int32), out, lse, s["k_cache"], s["v_cache"],
            (first + s["keep"]).to(torch.int32))


def _plain_attention(s, q, tree):
    B, T, H, d = q.shape
    N, K = s["table"].shape[1] * s["case"]["page"], s["k_cache"].shape[2]
    G = H // K
    j = torch.arange(N, device="cuda")
    page, at = _places(s, j.expand(B, N))
    news, lens = _counts(s).long(), s["lens"].long()
    first = lens - news
    # the keys before the new ones, and of the new ones those in a token's branch
    own = (j[None, :] - first[:, None]).clamp(0, T - 1)
    branch = torch.ones(B, T, T, dtype=torch.bool, device="cuda") if tree is None else _bits(tree, T)
    sees = branch.gather(2, own[:, None, :].expand(B, T, N)) | (j[None, :] < first[:, None])[:, None, :]
    sees &= (j[None, :] < lens[:, None])[:, None, :] & (torch.arange(T, device="cuda")[None, :] < news[:, None])[..., None]
    # [B, K, T G, d]: the rows of the query heads that share a KV head together
    rows = q.float().view(B, T, K, G, d).permute(0, 2, 1, 3, 4).reshape(B, K, T * G, d)
    keys, values = (s[name][page, at].float().permute(0, 2, 1, 3) for name in ("k_cache", "v_cache"))
    scores = (rows @ keys.transpose(2, 3) / math.sqrt(d)).view(B, K, T, G, N)
    scores = scores.masked_fill(~sees[:, None, :, None, :], -math.inf)
    top = scores.amax(-1, keepdim=True)
    weights = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    total = weights.sum(-1, keepdim=True)
    weights = weights / torch.where(total == 0, 1.0, total)
    out = (weights.view(B, K, T * G, N) @ values).view(B, K, T, G, d).permute(0, 2, 1, 3, 4).reshape(B, T, H, d)
    lse = (top + torch.log(total)).squeeze(-1).permute(0, 2, 1, 3).reshape(B, T, H)
    return out.to(q.dtype), lse


# ---------------------------------------------------------------- the work
def work(case):
    B, T, H, K, d = case["batch"], case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "rotary":
        return {"bytes": 2 * size * B * T * H * d + 4 * B * T, "flops": 3 * B * T * H * case["rotated"]}
    lens, news = _lengths(case), _news(case)
    new = sum(news)
    b = f = 0
    if case["op"] in ("append", "step"):
        b += 2 * size * new * (H + 2 * K) * d
        f += 3 * new * (H + K) * case["rotated"]
    if case["op"] in ("tree", "step"):
        # (which sequence has how many new tokens, the seed says: each with the mean)
        seen = sum(max(0, L - new / B) for L in lens) * new / B + sum(n * (n + 1) / 2 for n in news)
        b += 2 * size * K * d * sum(lens) + size * (new + B * T) * H * d + 4 * B * T * H
        f += 4 * d * H * seen
    return {"bytes": int(b), "flops": int(f)}


# ------------------------------------------------- the definition in 64 bits
def _exact_turned(x, positions, case):
    """Each pair as a complex number times magnitude e^(i angle); x [T, heads, d], positions [T]."""
    r, base, s = case["rotated"], case["base"], case["factor"]
    z = torch.zeros(x.shape[0], r // 2, dtype=torch.complex128, device="cuda")
    for i in range(r // 2):
        f = (base * s ** (r / (r - 2)) if case["scaling"] == "base" and r > 2 else base) ** (-2 * i / r)
        if case["scaling"] == "linear":
            f /= s
        if case["scaling"] == "parts":
            keep = min(1.0, max(0.0, (case["original"] * f / (2 * math.pi) - SLOW) / (FAST - SLOW)))
            f = f * (keep + (1 - keep) / s)
        angle = positions.double() * (-f if case.get("inverse") else f)
        z[:, i] = torch.polar(torch.full_like(angle, _magnitude(case)), angle)
    y = x.double().clone()
    at = torch.arange(r // 2, device="cuda")
    re, im = (2 * at, 2 * at + 1) if case["interleaved"] else (at, at + r // 2)
    turned = torch.complex(y[..., re], y[..., im]) * z[:, None]
    y[..., re], y[..., im] = turned.real, turned.imag
    return y


def exact(case, seed):
    """One sequence at a time over the positions it has, in the order it has them."""
    s = prepare(case, seed)
    B, T, H, K, d = case["batch"], case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "rotary":
        return torch.stack([_exact_turned(s["x"][b], s["positions"][b], case) for b in range(B)])
    dtype, P = DTYPES[case["dtype"]], case["page"]
    lens = s["lens"].tolist()
    news = s["news"].tolist() if s["news"] is not None else [T] * B
    rotates, attends = case["op"] != "tree", case["op"] != "append"
    k64, v64 = s["k_cache"].double(), s["v_cache"].double()
    q64 = torch.zeros(B, T, H, d, dtype=torch.float64, device="cuda")
    words = torch.zeros(B, T, (T + 31) // 32, dtype=torch.int64)
    depth = torch.zeros(B, T, dtype=torch.int32)
    out = torch.zeros(B, T, H, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, T, H), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        L, n = lens[b], news[b]
        j = torch.arange(L, device="cuda")
        page, at = s["table"][b].long()[j // P], j % P
        branch = [set(range(n)) for _ in range(n)]
        if attends and (T > 1 or case["op"] == "step"):
            for t, up in enumerate(s["parents"][b, :n].tolist()):
                branch[t] = {t} | (branch[up] if up >= 0 else set())
        if case["op"] == "step":
            for t in range(n):
                depth[b, t] = L - n + len(branch[t]) - 1
                for i in branch[t]:
                    words[b, t, i // 32] += 1 << (i % 32)
        if rotates:
            at_positions = depth[b, :n].cuda() if case["op"] == "step" else torch.arange(L - n, L, device="cuda")
            q64[b, :n] = _exact_turned(s["q"][b, :n], at_positions, case)
            k64[page[L - n:], at[L - n:]] = _exact_turned(s["k"][b, :n], at_positions, case)
            v64[page[L - n:], at[L - n:]] = s["v"][b, :n].double()
        if not attends:
            continue
        # what attention reads are the rounded keys and queries
        q = q64[b, :n].to(dtype).double() if rotates else s["q"][b, :n].double()
        sees = torch.ones(n, L, dtype=torch.bool, device="cuda")
        for t in range(n):
            for i in range(n):
                if i not in branch[t]:
                    sees[t, L - n + i] = False
        for h in range(K):
            heads = slice(h * (H // K), (h + 1) * (H // K))
            keys, values = k64[page, at, h].to(dtype).double(), v64[page, at, h].to(dtype).double()
            x = torch.einsum("tgd,jd->tgj", q[:, heads], keys) * d ** -0.5
            x = x.masked_fill(~sees[:, None, :], -math.inf)
            total = torch.logsumexp(x, -1)
            lse[b, :n, heads] = total
            out[b, :n, heads] = torch.einsum("tgj,jd->tgd", torch.exp(x - total[..., None]), values)
    if case["op"] == "append":
        return q64, k64, v64
    if case["op"] == "tree":
        return out, lse
    for b in range(B):
        n, m = news[b], s["keep"].tolist()[b]
        kept = s["path"][b, :m].long() + lens[b] - n
        left = torch.arange(lens[b] - n, lens[b] - n + m, device="cuda")
        for cache in (k64, v64):
            rows = cache[s["table"][b].long()[kept // P], kept % P].clone()
            cache[s["table"][b].long()[left // P], left % P] = rows
    words = torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32).cuda()
    ends = torch.tensor([L - n for L, n in zip(lens, news)], dtype=torch.int32, device="cuda") + s["keep"]
    return words, depth.cuda(), out, lse, k64, v64, ends
