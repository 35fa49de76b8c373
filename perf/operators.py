"""The paged-cache operators of a Medusa server, as a benchmark calls them.

A step of such a server rotates the new tokens' queries and keys and writes
keys and values into a paged cache (``rope``), attends to it (``attention``),
applies each request's penalties, biases and grammar mask to the base logits
(``logits``) and, after acceptance, compacts the accepted rows inside the
pages (``accept``).  ``run`` computes an operator in its plain form, with
elementary torch operations, or, where ``own`` is set, through
``speculative_decoding_heads_b200``.

The shapes are those of the repository's Vicuna-shaped workloads (32 / 40 / 52
heads of 128, vocabulary 32000, trees of 15 to 129 tokens, prefixes of 256 to
8192 rows) and of generic grouped-query models next to them.
"""

import functools
import itertools
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------


def listed():
    rope = dict(op="rope", dtype="bf16", hd=128, rot=128, layout="half", scaling="none", factor=1.0, page=64)
    attn = dict(op="attention", dtype="bf16", hd=128, page=64)
    return [
        # one new token of one request: the smallest call, latency alone
        dict(rope, name="rope_token", B=1, n_lo=1, n_hi=1, L_lo=1024, L_hi=1024, H=32, Hkv=32, page=16),
        # prompts of three requests at once, far positions in a context extended with YaRN, half of each head rotated in interleaved pairs
        dict(rope, name="rope_prompts_yarn", B=3, n_lo=1537, n_hi=4093, L_lo=0, L_hi=100003, H=32, Hkv=8, rot=64,
             layout="interleaved", scaling="yarn", factor=16.0),
        # the 15-token fp32 tree, its nodes at their depths' positions
        dict(rope, name="rope_tree_f32", dtype="f32", K=3, topk=2, nodes=14, B=2, L_lo=64, L_hi=64, H=4, Hkv=4, hd=64,
             rot=64, page=16, scaling="linear", factor=2.0),
        # plain decoding of one request at the 7B shape: the smallest attention
        dict(attn, name="attn_token", kind="chunk", B=1, n_lo=1, n_hi=1, L_lo=1024, L_hi=1024, H=32, Hkv=32, page=16),
        # single tokens of a batch of long ragged requests, grouped heads
        dict(attn, name="attn_tokens_long", kind="chunk", B=13, n_lo=1, n_hi=1, L_lo=4099, L_hi=60001, H=40, Hkv=8),
        # one verification step's tree at the 33B shape
        dict(attn, name="attn_tree_33b", kind="tree", K=5, topk=10, nodes=64, B=4, L_lo=8192, L_hi=8192, H=52, Hkv=52),
        # a chunk of a long prompt, grouped heads: the largest
        dict(attn, name="attn_prompt_chunk", kind="chunk", B=2, n_lo=3001, n_hi=4096, L_lo=2048, L_hi=4095, H=32, Hkv=8),
        # the 15-token fp32 tree over short prefixes
        dict(attn, name="attn_tree_f32", kind="tree", dtype="f32", K=3, topk=2, nodes=14, B=2, L_lo=64, L_hi=301, H=4,
             Hkv=4, hd=64, page=16),
        # compaction after one accepted path of a 7B-shaped request
        dict(op="accept", name="accept_b1", dtype="bf16", K=5, topk=10, nodes=63, layers=32, B=1, L_lo=1024, L_hi=1024,
             Hkv=32, hd=128, page=16, a=3),
        # the same for a batch at the 13B shape
        dict(op="accept", name="accept_b8", dtype="bf16", K=4, topk=8, nodes=48, layers=40, B=8, L_lo=17, L_hi=251,
             Hkv=40, hd=128, page=64, a=4),
        # every node of one 64-token tree: penalties, bias and a grammar mask
        dict(op="logits", name="logits_tree_b1", K=5, topk=10, nodes=63, B=1, V=32000, hist_lo=900, hist_hi=900, bias=8,
             mask=True),
        # a batch of trees with long histories, no grammar
        dict(op="logits", name="logits_trees_b16", K=4, topk=8, nodes=48, B=16, V=32003, hist_lo=257, hist_hi=8191, bias=0,
             mask=False),
    ]


def _log_int(rng, lo, hi):
    """An integer of lo..hi, spread evenly over its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _draw_tree(rng):
    K, topk = rng.randint(2, 5), rng.choice([2, 4, 8, 10])
    return K, topk, rng.randint(1, min(128, sum(topk ** l for l in range(1, K + 1))))


def _draw_one(rng):
    op = rng.choice(["rope", "attention", "attention", "accept", "logits"])
    c = {"op": op}
    if op in ("rope", "attention", "accept"):
        c["dtype"] = rng.choice(["bf16", "bf16", "bf16", "f32"])
        c["hd"] = rng.choice([128, 128, 64])
        c["page"] = rng.choice([16, 32, 64, 128])
        c["Hkv"] = rng.choice([1, 2, 4, 8, 16, 32, 40])
        c["H"] = c["Hkv"] * rng.choice([g for g in (1, 2, 3, 4, 5, 7, 8) if g * c["Hkv"] <= 64])
        c["B"] = _log_int(rng, 1, 32)
    if op == "rope":
        if rng.random() < 0.3:
            c["K"], c["topk"], c["nodes"] = _draw_tree(rng)
        else:
            c["n_lo"] = _log_int(rng, 1, 4096)
            c["n_hi"] = c["n_lo"] if rng.random() < 0.4 else _log_int(rng, c["n_lo"], 4096)
        c["L_lo"] = rng.choice([0, _log_int(rng, 1, 1 << 17)])
        c["L_hi"] = _log_int(rng, c["L_lo"] + 1, 1 << 17) if rng.random() < 0.6 else c["L_lo"]
        c["L_hi"] = max(c["L_lo"], c["L_hi"])
        c["rot"] = rng.choice([c["hd"], c["hd"], c["hd"] // 2, c["hd"] // 4])
        c["layout"] = rng.choice(["half", "interleaved"])
        c["scaling"] = rng.choice(["none", "linear", "ntk", "yarn"])
        c["factor"] = 1.0 if c["scaling"] == "none" else float(rng.choice([2, 4, 16]))
    elif op == "attention":
        c["kind"] = rng.choice(["token", "chunk", "tree"])
        if c["kind"] == "tree":
            c["K"], c["topk"], c["nodes"] = _draw_tree(rng)
        else:
            c["n_lo"] = 1 if c["kind"] == "token" else _log_int(rng, 2, 4096)
            c["n_hi"] = c["n_lo"] if c["kind"] == "token" or rng.random() < 0.4 else _log_int(rng, c["n_lo"], 4096)
            c["kind"] = "chunk"
        c["L_lo"] = rng.choice([0, _log_int(rng, 1, 30000)])
        c["L_hi"] = max(c["L_lo"], _log_int(rng, c["L_lo"] + 1, 60000) if rng.random() < 0.6 else c["L_lo"])
        if c["dtype"] == "f32":
            c["L_hi"] = c["L_lo"] = min(c["L_lo"], 4000)
            if c["kind"] == "chunk":
                c["n_lo"] = c["n_hi"] = min(c["n_lo"], 257)
    elif op == "accept":
        del c["H"]
        c["K"], c["topk"], c["nodes"] = _draw_tree(rng)
        c["layers"] = rng.randint(1, 40)
        c["L_lo"] = _log_int(rng, 1, 256)
        c["L_hi"] = _log_int(rng, c["L_lo"], 256)
        c["a"] = rng.randint(0, c["K"])
    else:
        c["K"], c["topk"], c["nodes"] = _draw_tree(rng) if rng.random() < 0.6 else (1, 2, 0)
        c["B"] = _log_int(rng, 1, 64)
        c["V"] = _log_int(rng, 999, 130000)
        c["hist_lo"] = _log_int(rng, 1, 8192)
        c["hist_hi"] = _log_int(rng, c["hist_lo"], 8192)
        c["bias"] = rng.choice([0, 0, 8, 100])
        c["mask"] = rng.random() < 0.5
    return c


def _fits(c):
    """No more work than the largest listed cases, and a plain form that fits the card."""
    most = {"rope": 2e8, "attention": 1.7e9, "accept": 3.2e7, "logits": 2e8}[c["op"]]
    w = work(c)
    if w["bytes"] > most or w["flops"] > 5.4e11:
        return False
    if c["op"] == "attention":
        lens, news = _lengths(c), _news(c)
        S = max(L + n for L, n in zip(lens, news)) + c["page"]
        return (c["B"] * c["H"] * max(news) * S <= 1.2e9 and c["B"] * S * c["Hkv"] * c["hd"] <= 1.5e9
                and (c["dtype"] != "f32" or w["flops"] < 3e10))
    if c["op"] == "accept":
        return c["layers"] * c["B"] * (max(_lengths(c)) + 256) * c["Hkv"] * c["hd"] <= 4e8
    if c["op"] == "rope":
        return sum(L + n + c["page"] for L, n in zip(_lengths(c), _news(c))) * c["Hkv"] * c["hd"] <= 1e9
    return True


def draw(rng):
    while True:
        c = _draw_one(rng)
        if _fits(c):
            return c


# ---------------------------------------------------------------------------
# sizes that follow from a case alone
# ---------------------------------------------------------------------------


def _spread(lo, hi, n):
    """n integers of lo..hi in an irregular fixed order, both ends among them where n allows."""
    if n == 1:
        return [hi]
    return [lo + (hi - lo) * ((7 * k) % n if n % 7 else k) // (n - 1) for k in range(n)]


def _lengths(c):
    return _spread(c["L_lo"], c["L_hi"], c["B"])


def _news(c):
    """New tokens of every sequence."""
    if "nodes" in c:
        return [c["nodes"] + 1] * c["B"]
    return _spread(c["n_lo"], c["n_hi"], c["B"])[::-1]


@functools.lru_cache(maxsize=64)
def _tree(K, topk, nodes):
    """(rank tuples, parent, depth, paths) of the static tree: the first tuples by (rank sum, length, order), breadth first."""
    got = []
    for total in itertools.count():
        if len(got) >= nodes:
            break
        for length in range(1, K + 1):
            got += [t for t in itertools.product(range(min(topk, total + 1)), repeat=length) if sum(t) == total]
    tuples = sorted(got[:nodes], key=lambda t: (len(t), t))
    at = {(): 0, **{t: i + 1 for i, t in enumerate(tuples)}}
    parent = [-1] + [at[t[:-1]] for t in tuples]
    depth = [0] + [len(t) for t in tuples]
    leaves = [i for i in range(len(parent)) if i not in set(parent)]
    paths = []
    for leaf in leaves:
        p = [leaf]
        while parent[p[-1]] >= 0:
            p.append(parent[p[-1]])
        paths.append(p[::-1])
    return tuples, parent, depth, paths


def _sees(parent):
    """[T, T] truth values: j is i or one of its ancestors."""
    T = len(parent)
    m = torch.zeros(T, T, dtype=torch.bool)
    for i in range(T):
        j = i
        while j >= 0:
            m[i, j] = True
            j = parent[j]
    return m


def _accepted(c):
    """(path, accept length) of every sequence: paths that the compaction can run on twice with the same result."""
    _, parent, _, paths = _tree(c["K"], c["topk"], c["nodes"])
    got = []
    for b in range(c["B"]):
        a = max(0, c["a"] - b % 2)
        fit = [p for p, path in enumerate(paths) if len(path) > a and all(n == j or n > a for j, n in enumerate(path[:a + 1]))]
        got.append((fit[(5 * b + 3) % len(fit)], a) if fit else (0, 0))
    return got


def work(case):
    c = case
    if c["op"] == "logits":
        T = c["nodes"] + 1
        n = c["B"] * T * c["V"]
        hist = sum(_spread(c["hist_lo"], c["hist_hi"], c["B"]))
        return {"bytes": 8 * n + (n / 8 if c["mask"] else 0) + 4 * hist + 4 * c["B"] * T, "flops": 2 * n}
    es = BYTES[c["dtype"]]
    if c["op"] == "accept":
        _, _, _, paths = _tree(c["K"], c["topk"], c["nodes"])
        moved = sum(sum(n != j for j, n in enumerate(paths[p][:a + 1])) for p, a in _accepted(c))
        return {"bytes": 4 * c["layers"] * c["Hkv"] * c["hd"] * es * moved + 24 * c["B"], "flops": 0}
    lens, news = _lengths(c), _news(c)
    N = sum(news)
    if c["op"] == "rope":
        return {"bytes": 2 * N * (c["H"] + 2 * c["Hkv"]) * c["hd"] * es + 4 * N, "flops": 3 * N * (c["H"] + c["Hkv"]) * c["rot"]}
    if c["kind"] == "tree":
        own_rows = sum(d + 1 for d in _tree(c["K"], c["topk"], c["nodes"])[2])
        pairs = sum(n * L + own_rows for L, n in zip(lens, news))
    else:
        pairs = sum(n * L + n * (n + 1) // 2 for L, n in zip(lens, news))
    kv = 2 * sum(L + n for L, n in zip(lens, news)) * c["Hkv"] * c["hd"] * es
    return {"bytes": kv + 2 * N * c["H"] * c["hd"] * es, "flops": 4 * c["hd"] * c["H"] * pairs}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _paged(c, seed, layers, g):
    """Pages filled with unit normals, handed out to the sequences in a shuffled order."""
    lens, news, page = _lengths(c), _news(c), c["page"]
    used = [-(-(L + n) // page) for L, n in zip(lens, news)]
    n_pages, cap = sum(used), max(used)
    shuffled = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).tolist()
    table = [[shuffled.pop() for _ in range(u)] + [0] * (cap - u) for u in used]
    shape = (layers, n_pages, c["Hkv"], page, c["hd"])
    t = TYPES[c["dtype"]]
    pages = [torch.empty(shape, dtype=t, device=DEV).normal_(generator=g) for _ in range(2)]
    return {"k_pages": pages[0], "v_pages": pages[1], "table": _ints(table), "lens": _ints(lens), "n_max": max(news)}


def _starts(news):
    return _ints([0] + list(itertools.accumulate(news)))


def _frequencies(c):
    """(angle per position of every pair in 64 bits, amplitude): rotary frequencies scaled for long contexts."""
    rot, base, s = c["rot"], 10000.0, c["factor"]
    pair = torch.arange(rot // 2, dtype=torch.float64)
    if c["scaling"] == "ntk":
        base = base * s ** (rot / (rot - 2))
    f = base ** (-2.0 * pair / rot)
    if c["scaling"] == "linear":
        f = f / s
    if c["scaling"] == "yarn":
        # pairs that turn more than 32 times over the original length keep their frequency, those below one turn are
        # interpolated, those between are blended linearly in the pair's index
        at = lambda turns: rot * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
        ramp = ((pair - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f / s * ramp + f * (1 - ramp)
        return f, 0.1 * math.log(s) + 1.0
    return f, 1.0


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    rand = lambda *shape: torch.randn(shape, generator=g, device=DEV)  # noqa: E731
    s = {"case": c}
    if "nodes" in c:
        tuples, parent, depth, paths = _tree(c["K"], c["topk"], c["nodes"])
        s["sees"] = _sees(parent).to(DEV)
        D = max(depth)
        s["paths"] = _ints([p + [-1] * (D + 1 - len(p)) for p in paths])
        if own:
            import speculative_decoding_heads_b200 as mb
            s["tree"] = mb.Tree(tuples, c["K"], c["topk"])
    if c["op"] == "logits":
        T = c["nodes"] + 1
        hist = _spread(c["hist_lo"], c["hist_hi"], c["B"])
        # token ids as texts have them: a few often, most of them rarely
        ids = lambda *shape: (torch.rand(shape, generator=g, device=DEV) ** 3 * c["V"]).int()  # noqa: E731
        s.update(logits=3 * rand(c["B"], T, c["V"]), tokens=ids(c["B"], T), history=ids(c["B"], max(hist)),
                 history_lens=_ints(hist), prompt_lens=_ints([h * 2 // 3 for h in hist]),
                 repetition=1.0 + 0.3 * torch.rand(c["B"], generator=g, device=DEV),
                 frequency=0.2 * torch.rand(c["B"], generator=g, device=DEV),
                 presence=0.5 * torch.rand(c["B"], generator=g, device=DEV),
                 bias_ids=None, bias=None, allowed=None)
        if c["bias"]:
            s.update(bias_ids=ids(c["B"], c["bias"]), bias=2 * rand(c["B"], c["bias"]))
        if c["mask"]:
            s["allowed"] = torch.randint(-2 ** 31, 2 ** 31, (c["B"], T, -(-c["V"] // 32)), generator=g, device=DEV).int()
        s["out"] = torch.empty_like(s["logits"])
        return s
    t = TYPES[c["dtype"]]
    s.update(_paged(c, int(seed), c.get("layers", 1), g))
    if own:
        import speculative_decoding_heads_b200 as mb
        s["kv"] = mb.PagedKV(s["k_pages"], s["v_pages"], s["table"], s["lens"])
    if c["op"] == "accept":
        took = _accepted(c)
        s.update(best=_ints([p for p, _ in took]), accept=_ints([a for _, a in took]), new_lens=torch.empty_like(s["lens"]))
        if own:
            s["ws"] = mb.workspace(mb.medusa_paged_accept_workspace_size(s["kv"]))
        return s
    news = _news(c)
    N = sum(news)
    # equal chunks need no table of starts
    s["starts"] = None if min(news) == max(news) else _starts(news)
    s["q"] = rand(N, c["H"], c["hd"]).to(t)
    s["out"] = torch.empty_like(s["q"])
    if c["op"] == "rope":
        # queries, keys and values as one fused product leaves them: the rows of a token side by side
        qkv = rand(N, (c["H"] + 2 * c["Hkv"]) * c["hd"]).to(t)
        q, k, v = qkv.split([c["H"] * c["hd"], c["Hkv"] * c["hd"], c["Hkv"] * c["hd"]], dim=1)
        if "nodes" in c:  # a tree's node sits at its depth's position, whatever row it takes
            s["positions"] = (s["lens"][:, None] + _ints(depth)).flatten()
        s.update(q=q.unflatten(1, (c["H"], c["hd"])), k=k.unflatten(1, (c["Hkv"], c["hd"])), v=v.unflatten(1, (c["Hkv"], c["hd"])))
        f, s["amplitude"] = _frequencies(c)
        s["f"] = f.to(DEV)
        if own:
            kind = {"none": mb.MEDUSA_ROPE_NONE, "linear": mb.MEDUSA_ROPE_LINEAR, "ntk": mb.MEDUSA_ROPE_NTK,
                    "yarn": mb.MEDUSA_ROPE_YARN}[c["scaling"]]
            s["rotary"] = mb.Rotary(c["rot"], layout=mb.MEDUSA_ROPE_HALF if c["layout"] == "half" else mb.MEDUSA_ROPE_INTERLEAVED,
                                    base=10000.0, scaling=kind, factor=c["factor"], original_length=4096)
    elif own:
        s["ws"] = mb.workspace(mb.medusa_paged_attention_workspace_size(s["kv"], N, c["H"]))
    return s


# ---------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        import speculative_decoding_heads_b200 as mb
        if op == "rope":
            mb.medusa_rope_append(s["kv"], 0, s["q"], s["k"], s["v"], s["out"], s["rotary"],
                                 positions=s.get("positions"), chunk_starts=s["starts"])
            return [s["out"], s["k_pages"], s["v_pages"]]
        if op == "attention":
            mb.medusa_paged_attention(s["kv"], 0, s["q"], s["out"], s["case"]["hd"] ** -0.5, s["ws"], tree=s.get("tree"),
                                      chunk_starts=s["starts"])
            return [s["out"]]
        if op == "accept":
            mb.medusa_paged_accept_kv(s["tree"], s["kv"], s["best"], s["accept"], s["new_lens"], s["ws"])
            return [s["k_pages"], s["v_pages"], s["new_lens"]]
        mb.medusa_adjust_logits(s["tree"], s["logits"], s["tokens"], s["out"], history=s["history"],
                                history_lens=s["history_lens"], prompt_lens=s["prompt_lens"], repetition=s["repetition"],
                                presence=s["presence"], frequency=s["frequency"], bias_ids=s["bias_ids"], bias=s["bias"],
                                allowed=s["allowed"])
        return [s["out"]]
    return {"rope": _plain_rope, "attention": _plain_attention, "accept": _plain_accept, "logits": _plain_logits}[op](s)


def _place(s, N):
    """(sequence, index in its chunk) of each of the N packed tokens."""
    n = torch.arange(N, device=DEV)
    B = s["lens"].shape[0]
    if s["starts"] is None:
        return n // (N // B), n % (N // B)
    b = torch.searchsorted(s["starts"].long(), n, right=True) - 1
    return b, n - s["starts"].long()[b]


def _rotate(x, cos, sin, rot, layout):
    """x [N, heads, hd] in 32 bits, cos and sin [N, 1, rot / 2]."""
    a, b = (x[..., :rot // 2], x[..., rot // 2:rot]) if layout == "half" else (x[..., 0:rot:2], x[..., 1:rot:2])
    y = x.clone()
    ya, yb = a * cos - b * sin, b * cos + a * sin
    if layout == "half":
        y[..., :rot // 2], y[..., rot // 2:rot] = ya, yb
    else:
        y[..., 0:rot:2], y[..., 1:rot:2] = ya, yb
    return y


def _plain_rope(s):
    c = s["case"]
    N, page = s["q"].shape[0], c["page"]
    b, i = _place(s, N)
    row = s["lens"].long()[b] + i
    angle = s.get("positions", row).double()[:, None] * s["f"]
    cos = (angle.cos() * s["amplitude"]).float()[:, None]
    sin = (angle.sin() * s["amplitude"]).float()[:, None]
    q = _rotate(s["q"].float(), cos, sin, c["rot"], c["layout"])
    k = _rotate(s["k"].float(), cos, sin, c["rot"], c["layout"])
    at = s["table"].long()[b, row // page]
    s["out"].copy_(q)
    s["k_pages"][0][at, :, row % page] = k.to(s["k_pages"].dtype)
    s["v_pages"][0][at, :, row % page] = s["v"]
    return [s["out"], s["k_pages"], s["v_pages"]]


def _plain_attention(s):
    c = s["case"]
    N, H, hd = s["q"].shape
    B, Hkv, n_max = c["B"], c["Hkv"], s["n_max"]
    table, lens = s["table"].long(), s["lens"].long()
    S = table.shape[1] * c["page"]
    k = s["k_pages"][0][table].transpose(1, 2).reshape(B, Hkv, S, hd).float()
    v = s["v_pages"][0][table].transpose(1, 2).reshape(B, Hkv, S, hd).float()
    new = torch.arange(n_max, device=DEV)
    first = s["starts"].long()[:-1] if s["starts"] is not None else torch.arange(B, device=DEV) * (N // B)
    q = s["q"][(first[:, None] + new).clamp(max=N - 1)].float()                       # [B, n_max, H, hd]
    q = q.reshape(B, n_max, Hkv, H // Hkv, hd).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, hd)
    z = (q @ k.transpose(2, 3)).mul_(hd ** -0.5).view(B, Hkv, H // Hkv, n_max, S)
    col = torch.arange(S, device=DEV)
    if c["kind"] == "tree":
        rel = col - lens[:, None]                                                     # [B, S]
        inside = (rel >= 0) & (rel < n_max)
        seen = s["sees"][:, rel.clamp(0, n_max - 1)].transpose(0, 1)                  # [B, T, S]
        seen = (rel < 0)[:, None] | (inside[:, None] & seen)
    else:
        seen = col <= (lens[:, None] + new)[..., None]
    z.masked_fill_(~seen[:, None, None], -torch.inf)
    z.sub_(z.amax(-1, keepdim=True)).exp_()
    z.div_(z.sum(-1, keepdim=True))
    o = (z.view(B, Hkv, -1, S) @ v).view(B, Hkv, H // Hkv, n_max, hd).permute(0, 3, 1, 2, 4).reshape(B, n_max, H, hd)
    b, i = _place(s, N)
    s["out"].copy_(o[b, i])
    return [s["out"]]


def _plain_accept(s):
    page = s["case"]["page"]
    lens, a = s["lens"].long()[:, None], s["accept"].long()[:, None]
    D1 = s["paths"].shape[1]
    j = torch.minimum(torch.arange(D1, device=DEV)[None], a)
    node = s["paths"].long()[s["best"].long()].gather(1, j)
    src, dst = lens + node, lens + j
    table = s["table"].long()
    ps, pd = table.gather(1, src // page), table.gather(1, dst // page)
    for pages in (s["k_pages"], s["v_pages"]):
        pages[:, pd, :, dst % page] = pages[:, ps, :, src % page]
    s["new_lens"].copy_(s["lens"] + s["accept"] + 1)
    return [s["k_pages"], s["v_pages"], s["new_lens"]]


def _plain_logits(s):
    z = s["logits"]
    B, T, V = z.shape
    at = torch.arange(s["history"].shape[1], device=DEV)
    live = at < s["history_lens"][:, None]
    made = live & (at >= s["prompt_lens"][:, None])
    none = torch.zeros(B, V, device=DEV)
    ever = none.scatter_add(1, s["history"].long(), live.float())[:, None]
    out = none.scatter_add(1, s["history"].long(), made.float())[:, None]
    path = torch.zeros(B, T, V, device=DEV)
    path.scatter_add_(2, s["tokens"].long()[:, None].expand(B, T, T), s["sees"].float().expand(B, T, T))
    ever, out = ever + path, out + path
    rep = s["repetition"][:, None, None]
    z = torch.where(ever > 0, torch.where(z > 0, z / rep, z * rep), z)
    z = z - (s["frequency"][:, None, None] * out + s["presence"][:, None, None] * (out > 0))
    if s["bias"] is not None:
        z = z + none.scatter_add(1, s["bias_ids"].long(), s["bias"])[:, None]
    if s["allowed"] is not None:
        bits = (s["allowed"][..., None] >> torch.arange(32, device=DEV, dtype=torch.int32)) & 1
        z = torch.where(bits.flatten(2)[..., :V] != 0, z, -torch.inf)
    s["out"].copy_(z)
    return [s["out"]]


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------


def exact(case, seed):
    c = dict(case)
    if c["op"] == "accept" or work(c)["flops"] > 2e12:
        return None
    s = prepare(c, seed)
    if c["op"] == "logits":
        return _exact_logits(s)
    lens, news = _lengths(c), _news(c)
    table = s["table"].tolist()
    first = [0] + list(itertools.accumulate(news))
    page = c["page"]
    if c["op"] == "rope":
        q, k, pages = s["q"].double(), s["k"].double(), s["k_pages"].double()
        f, amp = _frequencies(c)
        half = c["layout"] == "half"
        turned = []
        for x in (q, k):
            depth = _tree(c["K"], c["topk"], c["nodes"])[2] if "nodes" in c else None
            p = torch.cat([L + torch.tensor(depth or range(n), dtype=torch.float64) for L, n in zip(lens, news)])
            e = torch.polar(torch.full((1,), amp, dtype=torch.float64), p[:, None] * f).to(DEV)[:, None]
            r = x[..., :c["rot"]]
            r = r.unflatten(-1, (2, -1)).transpose(-1, -2) if half else r.unflatten(-1, (-1, 2))
            r = torch.view_as_real(torch.view_as_complex(r.contiguous()) * e)
            r = r.transpose(-1, -2).flatten(-2) if half else r.flatten(-2)
            turned.append(torch.cat([r, x[..., c["rot"]:]], -1))
        for b in range(c["B"]):
            rows = range(lens[b], lens[b] + news[b])
            at = torch.tensor([table[b][r // page] for r in rows], device=DEV)
            pages[0, at, :, torch.tensor([r % page for r in rows], device=DEV)] = turned[1][first[b]:first[b + 1]]
        return [turned[0], pages, None]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    group = c["H"] // c["Hkv"]
    for b in range(c["B"]):
        L, n = lens[b], news[b]
        ids = torch.tensor(table[b][:-(-(L + n) // page)], device=DEV)
        k, v = (s[x][0][ids].permute(1, 0, 2, 3).flatten(1, 2)[:, :L + n].double() for x in ("k_pages", "v_pages"))
        seen = torch.ones(n, L + n, dtype=torch.bool, device=DEV)
        seen[:, L:] = s["sees"] if c["kind"] == "tree" else torch.ones(n, n, dtype=torch.bool, device=DEV).tril()
        for h in range(c["H"]):
            z = torch.einsum("id,jd->ij", s["q"][first[b]:first[b + 1], h].double(), k[h // group]) / math.sqrt(c["hd"])
            p = torch.softmax(z.masked_fill(~seen, -math.inf), 1)
            out[first[b]:first[b + 1], h] = torch.einsum("ij,jd->id", p, v[h // group])
    return [out]


def _exact_logits(s):
    c = s["case"]
    parent = _tree(c["K"], c["topk"], c["nodes"])[1]
    z = s["logits"].double()
    V = c["V"]
    tokens = s["tokens"].tolist()
    numbers = {k: s[k].tolist() for k in ("history_lens", "prompt_lens", "repetition", "presence", "frequency")}
    for b in range(c["B"]):
        h, m = numbers["history_lens"][b], numbers["prompt_lens"][b]
        past = s["history"][b, :h].long()
        ever0, out0 = torch.bincount(past, minlength=V), torch.bincount(past[m:], minlength=V)
        extra = torch.zeros(V, dtype=torch.float64, device=DEV)
        if s["bias"] is not None:
            extra.index_add_(0, s["bias_ids"][b].long(), s["bias"][b].double())
        rep, pres, freq = (numbers[k][b] for k in ("repetition", "presence", "frequency"))
        for i in range(len(parent)):
            seen, j = [], i
            while j >= 0:
                seen.append(tokens[b][j])
                j = parent[j]
            more = torch.bincount(torch.tensor(seen, device=DEV), minlength=V)
            ever, out = ever0 + more, out0 + more
            r = z[b, i]
            r = torch.where(ever > 0, torch.where(r > 0, r / rep, r * rep), r)
            z[b, i] = r - freq * out.double() - pres * out.clamp(max=1).double() + extra
    if s["allowed"] is not None:
        word = torch.arange(V, device=DEV)
        ok = torch.bitwise_and(s["allowed"].long()[..., word // 32], torch.bitwise_left_shift(torch.ones_like(word), word % 32)) != 0
        z.masked_fill_(~ok, -math.inf)
    return [z]
