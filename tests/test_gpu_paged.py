"""The paged-cache calls and the logit adjustment on the GPU, against the fp64
definitions of ``oracle.paged_oracle``.

Rows of the pages that no sequence owns, and the rows past a sequence's end,
are NaN in every test: reading one of them shows.
"""

import numpy as np
import pytest
import torch

import oracle.medusa_oracle as O
import oracle.paged_oracle as PO

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}   # a rounding's largest relative error


@pytest.fixture(scope="module")
def mb(built):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_heads_b200 as mb
    return mb


@pytest.fixture(autouse=True)
def no_device_error(mb):
    mb.device_status()
    yield
    assert mb.device_status() == (0, 0)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def f64(t):
    return t.detach().double().cpu().numpy()


class Cache:
    """A paged cache whose sequences hold lens[b] + news[b] rows of unit normals; everything else is NaN."""

    def __init__(self, mb, dtype, hd, page, Hkv, lens, news, layers=1, seed=0, spare=2, extra_table=1):
        self.g = torch.Generator().manual_seed(seed)
        used = [-(-(L + n) // page) for L, n in zip(lens, news)]
        n_pages = sum(used) + spare
        order = torch.randperm(n_pages, generator=self.g).tolist()
        width = max(used) + extra_table
        self.table = [[order.pop() for _ in range(u)] + [-7] * (width - u) for u in used]   # unused entries are not read
        shape = (layers, n_pages, Hkv, page, hd)
        t = TYPES[dtype]
        k = torch.full(shape, float("nan"), dtype=t)
        v = torch.full(shape, float("nan"), dtype=t)
        for b, (L, n) in enumerate(zip(lens, news)):
            for r in range(L + n):
                p = self.table[b][r // page]
                k[:, p, :, r % page] = torch.randn(layers, Hkv, hd, generator=self.g).to(t)
                v[:, p, :, r % page] = torch.randn(layers, Hkv, hd, generator=self.g).to(t)
        self.k, self.v = k.cuda(), v.cuda()
        self.lens = list(lens)
        self.kv = mb.PagedKV(self.k, self.v, ints(self.table), ints(lens))

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.g)


def starts_of(news):
    return np.concatenate([[0], np.cumsum(news)]).astype(int).tolist()


# ---------------------------------------------------------------------------
# rotary positions and the write into the pages
# ---------------------------------------------------------------------------

ROPE = [
    # dtype, hd, rot, layout, scaling, factor, page, H, Hkv, lens, news
    ("bf16", 128, 128, "half", "none", 1.0, 16, 4, 4, [0], [1]),
    ("bf16", 128, 64, "interleaved", "yarn", 16.0, 64, 8, 2, [63, 0, 5], [3, 70, 1]),
    ("bf16", 64, 32, "half", "ntk", 4.0, 8, 6, 2, [7, 8, 9, 1], [1, 0, 9, 2]),
    ("bf16", 96, 96, "half", "linear", 2.0, 32, 3, 1, [31, 33], [40, 40]),
    ("bf16", 80, 20, "half", "none", 1.0, 16, 5, 5, [3], [9]),            # rotated part not whole 16-byte vectors
    ("bf16", 72, 6, "interleaved", "none", 1.0, 16, 2, 1, [3], [9]),
    ("f32", 64, 64, "half", "linear", 2.0, 16, 4, 4, [64, 64], [15, 15]),
    ("f32", 128, 64, "interleaved", "yarn", 4.0, 256, 7, 1, [300, 2], [17, 400]),
    ("f32", 256, 256, "half", "none", 1.0, 128, 2, 2, [120], [20]),
    ("f32", 8, 2, "half", "none", 1.0, 8, 1, 1, [0, 7], [0, 2]),
    ("f32", 256, 16, "interleaved", "none", 1.0, 8, 3, 3, [1], [33]),
    ("bf16", 128, 128, "half", "none", 1.0, 64, 40, 8, [0] * 3, [2000, 1300, 701]),   # several tokens per block
]


@pytest.mark.parametrize("case", ROPE, ids=lambda c: "-".join(str(x) for x in c[:8]))
@pytest.mark.parametrize("fused", [False, True], ids=["apart", "fused"])
def test_rope_append(mb, case, fused):
    dtype, hd, rot, layout, scaling, factor, page, H, Hkv, lens, news = case
    c = Cache(mb, dtype, hd, page, Hkv, lens, news, layers=2, seed=hd + rot)
    before_k, before_v = c.k.clone(), c.v.clone()
    t = TYPES[dtype]
    N, starts = sum(news), starts_of(news)
    qkv = c.randn(N, H + 2 * Hkv, hd).to(t).cuda()
    q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    rotary = mb.Rotary(rot, layout=mb.MEDUSA_ROPE_HALF if layout == "half" else mb.MEDUSA_ROPE_INTERLEAVED,
                       scaling=["none", "linear", "ntk", "yarn"].index(scaling), factor=factor)
    out = torch.full((N + 2, H, hd), 7.0, dtype=t, device="cuda")
    equal = len(set(news)) == 1
    mb.medusa_rope_append(c.kv, 1, q, k, v, out[:N], rotary, chunk_starts=None if equal else ints(starts))
    freq, amp = PO.rope_frequencies(rot, 10000.0, scaling, factor)
    pos = np.concatenate([np.arange(L, L + n) for L, n in zip(lens, news)])

    def check(got, x):
        x = f64(x)
        want = PO.rotate(x, pos, freq, amp, rot, layout)
        # cos and sin: the angle's fraction of a half turn is rounded once (pi 2^-24) after 2^-32 turns were cut off,
        # sincospi is within 2 units (2^-23), the amplitude and three more roundings: below 2^-20 of |x| + |y|.
        pair = PO.rotate(np.abs(x), np.zeros(len(x)), freq, 1.0, rot, layout)
        span = np.zeros_like(x)
        for i in range(rot // 2):
            a, b = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
            span[..., a] = span[..., b] = pair[..., a] + pair[..., b]
        tol = span * amp * 2.0 ** -20 + (HALF_STEP[dtype] * np.abs(want) if dtype == "bf16" else 0)
        assert (np.abs(got - want) <= tol).all()

    check(f64(out[:N]), q)
    assert (out[N:] == 7).all()
    rows = [(c.table[b][(L + i) // page], (L + i) % page) for b, (L, n) in enumerate(zip(lens, news)) for i in range(n)]
    pg, rw = (torch.tensor(x, device="cuda") for x in zip(*rows))
    check(f64(c.k[1][pg, :, rw]), k)
    assert torch.equal(c.v[1][pg, :, rw], v)
    # nothing else moved
    for now, was in ((c.k, before_k), (c.v, before_v)):
        now[1][pg, :, rw] = was[1][pg, :, rw]
        assert torch.equal(now.view(torch.uint8), was.view(torch.uint8))


def test_rope_far_positions(mb):
    """At positions near 2^31 the angle still follows the definition (computed here in exact integers)."""
    c = Cache(mb, "f32", 64, 16, 2, [3], [6])
    rotary = mb.Rotary(64)
    turns, amp = mb.medusa_rotary_turns(64)
    pos = [0, 1, 999_999, 1_000_003, 2 ** 31 - 1, 123_456_789]
    x = c.randn(6, 2, 64).cuda()
    out = torch.empty_like(x)
    mb.medusa_rope_append(c.kv, 0, x, x.clone(), x.clone(), out, rotary, positions=ints(pos))
    xs, want = f64(x), np.zeros((6, 2, 64))
    for n, p in enumerate(pos):
        for i in range(32):
            th = (p * turns[i] % 2 ** 64) / 2 ** 64 * 2 * np.pi
            c_, s_ = np.cos(th), np.sin(th)
            want[n, :, i] = xs[n, :, i] * c_ - xs[n, :, i + 32] * s_
            want[n, :, i + 32] = xs[n, :, i + 32] * c_ + xs[n, :, i] * s_
    span = np.abs(xs[..., :32]) + np.abs(xs[..., 32:])
    assert (np.abs(f64(out) - want) <= np.concatenate([span, span], -1) * 2.0 ** -20).all()


def test_rope_in_place_and_behind_the_last_sequence(mb):
    lens, news = [4, 0, 9], [3, 0, 5]
    c = Cache(mb, "bf16", 128, 8, 2, lens, news)
    q = c.randn(12, 4, 128).bfloat16().cuda()     # 8 tokens, 4 rows behind the last sequence
    k = c.randn(12, 2, 128).bfloat16().cuda()
    apart = q.clone()
    want = torch.empty_like(q)
    rotary = mb.Rotary(128)
    mb.medusa_rope_append(c.kv, 0, apart, k, k, want, rotary, chunk_starts=ints(starts_of(news)))
    mb.medusa_rope_append(c.kv, 0, q, k, k, q, rotary, chunk_starts=ints(starts_of(news)))
    assert torch.equal(q[:8], want[:8]) and torch.equal(q[8:], apart[8:])


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------


def check_attention(mb, dtype, hd, page, H, Hkv, lens, news, choices=None, K=0, topk=0, seed=0, scale=None, layers=1,
                    layer=0, ws=None):
    tree = sees = None
    if choices is not None:
        tree = mb.Tree(choices, K, topk)
        tab = tree.tables()
        sees = np.array([[(tab["anc"][i][j // 64] >> (j % 64)) & 1 for j in range(tree.T)] for i in range(tree.T)], bool)
        news = [tree.T] * len(lens)
    c = Cache(mb, dtype, hd, page, Hkv, lens, news, layers=layers, seed=seed)
    N, starts = sum(news), starts_of(news)
    q = c.randn(N, H, hd).to(TYPES[dtype]).cuda()
    out = torch.full((N + 1, H, hd), 7.0, dtype=TYPES[dtype], device="cuda")
    scale = hd ** -0.5 if scale is None else scale
    equal = len(set(news)) == 1
    ws = mb.workspace(mb.medusa_paged_attention_workspace_size(c.kv, N, H)) if ws is None else ws
    args = dict(tree=tree, chunk_starts=None if equal else ints(starts))
    mb.medusa_paged_attention(c.kv, layer, q, out[:N], scale, ws, **args)
    first = out.clone()
    mb.medusa_paged_attention(c.kv, layer, q, out[:N], scale, ws, **args)     # the workspace is as it was
    assert torch.equal(out, first), "a second call gives other bits"
    assert (out[N] == 7).all()
    want, mass = PO.attention(f64(q), f64(c.k[layer]), f64(c.v[layer]), c.table, lens, starts, scale, sees)
    # Scores: a sum of hd products in fp32 and two more roundings move a score by at most (hd + 2) 2^-24 sum |q k| scale,
    # exp2 by 2^-22; probabilities move by twice that, sums of n terms by n 2^-24, twice (numerator and denominator).
    n_max = max(L + n for L, n in zip(lens, news))
    qk = np.abs(f64(q)).sum(-1).max() * 6.0 * abs(scale)      # |k| < 6 for these normals
    d = (hd + 2) * 2.0 ** -24 * qk + 2.0 ** -22
    tol = mass * (2 * d + 2 * (n_max + 8) * 2.0 ** -24)
    if dtype == "bf16":   # probabilities rounded before the second product, the output after it
        tol = tol + mass * HALF_STEP["bf16"] + (np.abs(want) + tol) * HALF_STEP["bf16"]
    err = np.abs(f64(out[:N]) - want)
    assert (err <= tol).all(), f"max error {err.max():.3g}, tolerance there {tol.flat[err.argmax()]:.3g}"
    return c, q, out[:N].clone()


ATTN = [
    # dtype, hd, page, H, Hkv, lens, news
    ("bf16", 128, 16, 4, 4, [0], [1]),
    ("bf16", 128, 64, 4, 4, [127, 128, 129, 1], [1, 1, 1, 1]),
    ("bf16", 128, 8, 8, 1, [1000], [1]),
    ("bf16", 128, 256, 14, 2, [255, 700, 0], [1, 1, 1]),
    ("bf16", 128, 32, 6, 2, [33, 0, 200], [17, 0, 130]),
    ("bf16", 128, 128, 5, 1, [0, 300], [301, 64]),
    ("bf16", 128, 64, 3, 1, [511], [129]),
    ("bf16", 128, 64, 32, 2, [63], [9]),
    ("bf16", 128, 64, 8, 2, [300], [2048]),      # many tiles to a CTA, whole ones and pieces, one key tile and more
    ("bf16", 128, 64, 64, 8, [300, 40], [500, 140]),      # from here to 63 heads: enough rows for two groups to a unit
    ("bf16", 64, 32, 64, 8, [0, 130], [303, 300]),
    ("bf16", 128, 64, 32, 8, [300, 0, 90], [1300, 1, 30]),
    ("bf16", 128, 16, 63, 9, [1, 500], [600, 50]),
    ("bf16", 64, 16, 4, 2, [100, 5], [3, 140]),
    ("bf16", 64, 64, 9, 3, [1500, 3], [1, 1]),
    ("bf16", 96, 16, 2, 2, [70], [20]),
    ("bf16", 256, 32, 4, 2, [90, 20], [5, 33]),
    ("bf16", 8, 8, 2, 1, [9], [4]),
    ("f32", 64, 16, 4, 4, [64, 301], [15, 15]),
    ("f32", 128, 32, 4, 1, [0, 257], [80, 2]),
    ("f32", 128, 64, 4, 4, [900], [1]),
    ("f32", 256, 8, 2, 1, [40], [30]),
    ("f32", 40, 16, 3, 3, [17, 0], [0, 5]),
]


@pytest.mark.parametrize("case", ATTN, ids=lambda c: "-".join(str(x) for x in c))
def test_paged_attention_chunks(mb, case):
    check_attention(mb, *case, seed=sum(case[5]))


TREES = [
    # dtype, hd, page, H, Hkv, lens, K, topk, nodes
    ("bf16", 128, 16, 4, 4, [0, 100], 3, 2, 14),
    ("bf16", 128, 64, 2, 2, [320], 5, 10, 63),
    ("bf16", 128, 64, 2, 2, [127, 1], 5, 10, 64),
    ("bf16", 128, 32, 4, 2, [65, 250, 3], 5, 10, 128),
    ("bf16", 128, 16, 1, 1, [77], 5, 10, 255),
    ("bf16", 64, 8, 8, 2, [40], 4, 8, 48),
    ("bf16", 128, 16, 4, 4, [50], 1, 1, 0),
    ("bf16", 128, 64, 8, 1, [700, 2], 5, 10, 63),          # several tiles of one key head
    ("bf16", 64, 16, 20, 2, [300, 90, 0], 5, 10, 100),
    ("bf16", 128, 64, 64, 4, [260, 70, 31], 5, 10, 254),   # enough rows for two groups to a unit
    ("f32", 64, 16, 4, 4, [64, 5], 3, 2, 14),
    ("f32", 128, 64, 2, 1, [130], 5, 10, 64),
]


@pytest.mark.parametrize("case", TREES, ids=lambda c: "-".join(str(x) for x in c))
def test_paged_attention_trees(mb, case):
    dtype, hd, page, H, Hkv, lens, K, topk, nodes = case
    choices = O.ranksum_choices(K, topk, nodes) if nodes else []
    check_attention(mb, dtype, hd, page, H, Hkv, lens, None, choices=choices, K=K, topk=topk, seed=nodes)


def test_paged_attention_other_layer_and_scales(mb):
    check_attention(mb, "bf16", 128, 16, 4, 2, [40, 200], [3, 3], layers=3, layer=2)
    check_attention(mb, "bf16", 128, 16, 4, 2, [40, 200], [3, 3], scale=0.0)
    check_attention(mb, "f32", 64, 16, 4, 2, [40, 200], [3, 3], scale=-0.3)


def test_paged_attention_large_scores(mb):
    """Scores of hundreds: one key takes nearly all the weight, and the running maximum moves a lot."""
    check_attention(mb, "f32", 64, 16, 2, 2, [700], [4], scale=4.0)
    check_attention(mb, "bf16", 128, 16, 2, 2, [700], [4], scale=2.0)


def test_paged_attention_nan_in_masked_keys(mb):
    """A NaN key of a later token does not reach the rows that do not see it."""
    for dtype in ("bf16", "f32"):
        c, q, out = check_attention(mb, dtype, 128, 16, 2, 2, [20], [6])
        row = 20 + 5
        c.k[0, c.table[0][row // 16], :, row % 16] = float("nan")
        again = torch.empty_like(out)
        ws = mb.workspace(mb.medusa_paged_attention_workspace_size(c.kv, 6, 2))
        mb.medusa_paged_attention(c.kv, 0, q, again, 128 ** -0.5, ws)
        assert torch.equal(again[:5], out[:5]) and again[5].isnan().all()


def test_paged_attention_shared_prefix(mb):
    """Two sequences whose tables name the same prefix pages read the same rows."""
    c = Cache(mb, "bf16", 128, 16, 2, [64, 64], [2, 2])
    c.table[1][:4] = c.table[0][:4]
    kv = mb.PagedKV(c.k, c.v, ints(c.table), ints(c.lens))
    q = c.randn(4, 4, 128).bfloat16().cuda()
    out = torch.empty_like(q)
    ws = mb.workspace(mb.medusa_paged_attention_workspace_size(kv, 4, 4))
    mb.medusa_paged_attention(kv, 0, q, out, 0.09, ws)
    want, mass = PO.attention(f64(q), f64(c.k[0]), f64(c.v[0]), c.table, c.lens, [0, 2, 4], 0.09)
    # as in check_attention, its fp32 terms below 2^-14 for 66 keys and scores under 8 * 6 * 11.4 * 0.09
    tol = mass * (HALF_STEP["bf16"] + 2.0 ** -10) + np.abs(want) * HALF_STEP["bf16"]
    assert (np.abs(f64(out) - want) <= tol).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_paged_attention_one_workspace_in_turn(mb, dtype):
    """Calls of all kinds share one workspace: none leaves in it what another takes for a count."""
    big = 0
    calls = [(128, 64, 8, 2, [300], [700]), (128, 64, 4, 4, [500, 90], [1, 1]), (128, 16, 4, 2, [40, 200, 0], [60, 7, 300]),
             (64, 16, 4, 4, [900], [2]), (64, 8, 4, 1, [100] * 9, [9, 0, 30, 1, 1, 64, 2, 0, 5]), (256, 32, 2, 1, [600], [40])]
    for hd, page, H, Hkv, lens, news in calls:
        c = Cache(mb, dtype, hd, page, Hkv, lens, news)
        big = max(big, mb.medusa_paged_attention_workspace_size(c.kv, sum(news), H))
    ws = mb.workspace(big)
    for turn in range(2):
        for hd, page, H, Hkv, lens, news in calls[::1 - 2 * turn]:
            check_attention(mb, dtype, hd, page, H, Hkv, lens, news, ws=ws)
            check_attention(mb, dtype, hd, page, H, Hkv, lens, news, ws=ws, scale=-0.05)     # the CUDA-core kernel for bf16 too


@pytest.mark.parametrize("dtype,hd,H,Hkv", [("bf16", 128, 4, 2), ("bf16", 64, 3, 3), ("bf16", 40, 4, 2), ("f32", 64, 2, 1)])
def test_paged_attention_64_sequences(mb, dtype, hd, H, Hkv):
    """The most sequences of a call, some with nothing to do and some with no prefix; then a single token each."""
    rng = np.random.default_rng(hd)
    lens = [int(x) for x in rng.integers(0, 70, 64)]
    news = [int(x) for x in rng.integers(0, 9, 64)]
    lens[0] = lens[63] = 0
    news[5], news[0], news[63] = 150, 0, 0
    check_attention(mb, dtype, hd, 8, H, Hkv, lens, news)
    lens[7] = 1700
    check_attention(mb, dtype, hd, 16, H, Hkv, lens, [1] * 64)


def test_paged_attention_wide_groups(mb):
    """Groups of more than 128 query heads, that 128 is no multiple of, and of the most heads."""
    check_attention(mb, "bf16", 128, 16, 256, 1, [33], [3])
    check_attention(mb, "bf16", 128, 16, 128, 1, [130], [3])
    check_attention(mb, "bf16", 64, 16, 100, 1, [200, 3], [5, 2])
    check_attention(mb, "bf16", 128, 16, 75, 1, [200], [1])
    check_attention(mb, "bf16", 64, 8, 256, 256, [9], [1])


def test_offsets_past_32_bits(mb):
    """Pages whose elements lie past 2^31 (and bytes past 2^32), in the second layer: append, attention, compaction."""
    hd, page, Hkv, H, n_pages = 128, 256, 40, 40, 1700                # 1700 * 40 * 256 * 128 > 2^31 elements a layer
    k = torch.empty(2, n_pages, Hkv, page, hd, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    tree = mb.Tree(O.ranksum_choices(3, 2, 14), 3, 2)
    T, L = tree.T, 250                                                # the new rows begin in one page and end in the next
    used = [n_pages - 1, n_pages - 2]
    g = torch.Generator(device="cuda").manual_seed(5)
    k[1, used] = torch.randn(2, Hkv, page, hd, generator=g, device="cuda").bfloat16()
    v[1, used] = torch.randn(2, Hkv, page, hd, generator=g, device="cuda").bfloat16()
    k[0, used], v[0, used] = 0, 0
    lens = ints([L])
    kv = mb.PagedKV(k, v, ints([used]), lens)
    q = torch.randn(T, H, hd, generator=g, device="cuda").bfloat16()
    nk, nv = (torch.randn(T, Hkv, hd, generator=g, device="cuda").bfloat16() for _ in range(2))
    small = mb.PagedKV(k[:, used].contiguous(), v[:, used].contiguous(), ints([[0, 1]]), ints([L]))
    assert k[1, used[0]].data_ptr() - k.data_ptr() > 2 ** 33
    outs = []
    for cache in (kv, small):                                         # the same pages near the buffer's start: the same bits
        qr, out = torch.empty_like(q), torch.empty_like(q)
        mb.medusa_rope_append(cache, 1, q, nk, nv, qr, mb.Rotary(hd))
        ws = mb.workspace(mb.medusa_paged_attention_workspace_size(cache, T, H))
        mb.medusa_paged_attention(cache, 1, qr, out, hd ** -0.5, ws, tree=tree)
        best = max(range(tree.P), key=lambda p: sum(x >= 0 for x in tree.tables()["retrieve"][p]))
        mb.medusa_paged_accept_kv(tree, cache, ints([best]), ints([tree.D]), cache.seq_lens,
                                  mb.workspace(mb.medusa_paged_accept_workspace_size(cache)))
        outs.append((out, cache.seq_lens.clone()))
    assert torch.equal(outs[0][0], outs[1][0]) and outs[0][0].isfinite().all() and outs[0][1].tolist() == [L + tree.D + 1]
    for far, near in ((k, small.k_pages), (v, small.v_pages)):
        assert torch.equal(far[:, used], near)
    rows = [(0, r) if r < page else (1, r - page) for r in range(L, L + T)]
    moved = small.v_pages[1][[p for p, _ in rows], :, [r for _, r in rows]]
    path = tree.tables()["retrieve"][best]
    assert torch.equal(moved[:tree.D + 1], nv[[int(x) for x in path[:tree.D + 1]]])


# ---------------------------------------------------------------------------
# compaction
# ---------------------------------------------------------------------------


CHAIN = [(0,), (1,)] + [(1,) + (0,) * n for n in range(1, 16)]    # depth 16, every node one row behind its depth
ACCEPT_TREES = {"d4": (4, 8, O.ranksum_choices(4, 8, 48)), "d5": (5, 10, O.ranksum_choices(5, 10, 63)), "d16": (16, 2, CHAIN)}


@pytest.mark.parametrize("tree_of", sorted(ACCEPT_TREES))
@pytest.mark.parametrize("dtype,hd,page,Hkv,lens,in_place", [
    ("bf16", 128, 16, 4, [0, 15, 33], True), ("bf16", 64, 8, 1, [7], False), ("f32", 64, 64, 3, [62, 1, 130, 64], True),
    ("f32", 8, 8, 2, [5, 2], False), ("bf16", 128, 256, 40, [250, 3], True)])
def test_paged_accept(mb, dtype, hd, page, Hkv, lens, in_place, tree_of):
    K, topk, choices = ACCEPT_TREES[tree_of]
    tree = mb.Tree(choices, K, topk)
    ret = tree.tables()["retrieve"]
    rng = np.random.default_rng(len(lens) + hd)
    ws = None
    for trial in range(4):
        c = Cache(mb, dtype, hd, page, Hkv, lens, [tree.T] * len(lens), layers=3, seed=trial)
        best = [int(rng.integers(tree.P)) for _ in lens]
        acc = [int(rng.integers(sum(x >= 0 for x in ret[p]))) for p in best]
        if trial == 3:                            # the deepest path, all of it
            best = [max(range(tree.P), key=lambda p: sum(x >= 0 for x in ret[p]))] * len(lens)
            acc = [tree.D] * len(lens)
        want = [PO.accept(t.cpu().float().numpy(), c.table, lens, ret, best, acc) for t in (c.k, c.v)]
        ws = mb.workspace(mb.medusa_paged_accept_workspace_size(c.kv)) if ws is None else ws
        new = c.kv.seq_lens if in_place else torch.full_like(c.kv.seq_lens, -5)
        mb.medusa_paged_accept_kv(tree, c.kv, ints(best), ints(acc), new, ws)
        for t, w in zip((c.k, c.v), want):
            assert np.array_equal(t.cpu().float().numpy(), w, equal_nan=True)
        assert new.tolist() == [L + a + 1 for L, a in zip(lens, acc)]
        if not in_place:
            assert c.kv.seq_lens.tolist() == lens


# ---------------------------------------------------------------------------
# logits
# ---------------------------------------------------------------------------

LOGITS = [
    # B, V, (K, topk, nodes), history lengths, what is asked
    (1, 1000, (3, 2, 14), [40], "rpfbm"),
    (3, 4099, (4, 8, 48), [0, 700, 33], "rpf"),
    (2, 2048, (1, 1, 0), [300, 5], "rpfbm"),
    (2, 31, (2, 2, 6), [64, 64], "rpfbm"),
    (1, 513, (5, 10, 63), [10], "m"),
    (1, 5000, (2, 2, 6), [10], "b"),
    (2, 1, (2, 2, 6), [3, 0], "rpfbm"),
    (2, 6000, (2, 2, 6), None, "rf"),
    (5, 2052, (3, 2, 14), [9, 1, 0, 2, 400], "p"),
    (1, 300, (2, 2, 6), [5], ""),
    (64, 20_003, (1, 1, 0), [(37 * b) % 900 for b in range(64)], "rpfbm"),    # single tokens, several chunks to a block
    (33, 65_536, (1, 1, 0), [40] * 33, "rpfm"),
]


def logits_case(B, V, tree_of, lens, asked, seed=0):
    rng = np.random.default_rng(seed + V)
    K, topk, nodes = tree_of
    T = nodes + 1
    ids = lambda *s: np.minimum((rng.random(s) ** 3 * V).astype(np.int32), V - 1)  # noqa: E731
    kw, plain = {}, {}
    tokens = ids(B, T)
    if T > 4:
        tokens[:, 3] = -1                        # padding inside a path
        tokens[:, 4] = tokens[:, 0]              # the same token twice on a path
    if lens is not None:
        cap = max(lens) + 3
        hist = ids(B, cap)
        hist[:, -3:] = 0                         # behind every history
        if max(lens) > 4:
            hist[:, 1], hist[:, 2] = V, -1       # outside the vocabulary
        prompt = [L // 2 for L in lens]
        kw.update(history=ints(hist.tolist()), history_lens=ints(lens), prompt_lens=ints(prompt))
        plain.update(history=[hist[b, :lens[b]].tolist() for b in range(B)], prompt_lens=prompt)
    for letter, name, lo, hi in (("r", "repetition", 0.7, 1.6), ("p", "presence", -0.5, 1.0), ("f", "frequency", -0.2, 0.5)):
        if letter in asked:
            x = rng.uniform(lo, hi, B).astype(np.float32)
            kw[name], plain[name] = torch.from_numpy(x).cuda(), x.astype(np.float64)
    if "b" in asked:
        bi = ids(B, 9)
        bi[:, 4] = bi[:, 1]                      # a token biased twice
        bi[:, 7] = -1
        bv = rng.normal(size=(B, 9)).astype(np.float32)
        kw.update(bias_ids=ints(bi.tolist()), bias=torch.from_numpy(bv).cuda())
        plain["bias"] = [list(zip(bi[b].tolist(), bv[b].astype(np.float64))) for b in range(B)]
    if "m" in asked:
        ok = rng.random((B, T, V)) < 0.5
        ok[0, 0] = False                         # a node where nothing may follow
        W = -(-V // 32)
        bits = np.zeros((B, T, W * 32), np.uint8)
        bits[..., :V] = ok
        words = np.packbits(bits, axis=-1, bitorder="little").view(np.uint32).astype(np.int64)
        kw["allowed"] = torch.from_numpy((words - ((words >> 31) << 32)).astype(np.int32)).cuda()
        plain["allowed"] = ok
    z = (3 * rng.normal(size=(B, T, V))).astype(np.float32)
    return z, tokens, kw, plain


@pytest.mark.parametrize("case", LOGITS, ids=lambda c: f"B{c[0]}-V{c[1]}-{c[4]}")
@pytest.mark.parametrize("in_place", [False, True], ids=["apart", "in_place"])
def test_adjust_logits(mb, case, in_place):
    B, V, (K, topk, nodes), lens, asked = case
    tree = mb.Tree(O.ranksum_choices(K, topk, nodes) if nodes else [], K, topk)
    z, tokens, kw, plain = logits_case(*case)
    dev = torch.from_numpy(z).cuda()
    out = dev if in_place else torch.empty_like(dev)
    mb.medusa_adjust_logits(tree, dev, ints(tokens.tolist()), out, **kw)
    want = PO.adjust_logits(z, tokens.tolist(), tree.tables()["parent"], **plain)
    got = f64(out)
    assert np.array_equal(np.isinf(got), np.isinf(want))
    # At most six roundings, each below 2^-24 of a partial result that |z| 1.6 + c (|f| + |p|) + the biases bound.
    biggest = np.abs(z).max() * 1.6 + 700 * 1.5 + 40
    fin = np.isfinite(want)
    span = np.abs(z) * 1.6 + np.abs(want, where=fin, out=np.zeros_like(want)) + 40
    few = np.abs(got[fin] - want[fin]) <= 6 * 2.0 ** -24 * np.maximum(span[fin], biggest * 0.05)
    assert few.all()


def test_adjust_logits_past_32_bits(mb):
    """Rows that begin past 2^31 elements, in place: the last sequence's equal those of a call of its own."""
    tree = mb.Tree(O.ranksum_choices(5, 10, 63), 5, 10)
    B, T, V = 35, 64, 960_001
    assert B * T * V > 2 ** 31
    z = torch.empty(B, T, V, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    last = torch.randn(1, T, V, generator=g, device="cuda")
    z[:-1], z[-1:] = 0, last
    tokens = ints([[(7 * i) % V for i in range(T)]] * B)
    kw = dict(presence=torch.full((B,), 0.5, device="cuda"), repetition=torch.full((B,), 1.25, device="cuda"),
              bias_ids=ints([[V - 1, 5]] * B), bias=torch.ones(B, 2, device="cuda"))
    mb.medusa_adjust_logits(tree, z, tokens, z, **kw)
    want = torch.empty_like(last)
    mb.medusa_adjust_logits(tree, last, tokens[-1:].contiguous(), want, **{k: x[-1:].contiguous() for k, x in kw.items()})
    assert torch.equal(z[-1:], want) and not torch.equal(want, last)
    assert (z[0, 0, V - 1], z[0, 0, 5], z[0, 0, 0], z[0, 0, 1]) == (1.0, 1.0, -0.5, 0.0)


def test_adjust_logits_infinite(mb):
    """Infinite and NaN logits and biases follow the definition's arithmetic."""
    tree = mb.Tree([], 1, 1)
    inf, nan = float("inf"), float("nan")
    z = torch.tensor([[[inf, -inf, nan, 1.0, -2.0, 3.0, -inf, 0.0]]], device="cuda")
    out = torch.empty_like(z)
    ok = ints([[[0b01111111]]])
    mb.medusa_adjust_logits(tree, z, ints([[1]]), out, repetition=torch.tensor([2.0], device="cuda"),
                            presence=torch.tensor([0.25], device="cuda"), history=ints([[0, 2, 3, 4]]), history_lens=ints([4]),
                            bias_ids=ints([[5, 6]]), bias=torch.tensor([[-inf, 9.0]], device="cuda"), allowed=ok)
    got = out.flatten().tolist()
    assert got[:2] == [inf, -inf] and np.isnan(got[2]) and got[3:] == [0.25, -4.25, -inf, -inf, -inf]


def test_adjust_logits_odd_alignment(mb):
    """Logits that start 4 bytes past a 16-byte boundary take the element path."""
    tree = mb.Tree(O.ranksum_choices(2, 2, 6), 2, 2)
    case = (1, 2048, (2, 2, 6), [50], "rpfbm")
    z, tokens, kw, plain = logits_case(*case)
    room = torch.empty(z.size + 1, device="cuda")
    dev = room[1:].view(z.shape)
    dev.copy_(torch.from_numpy(z))
    a, b = torch.empty(z.shape, device="cuda"), torch.empty(z.shape, device="cuda")
    mb.medusa_adjust_logits(tree, dev, ints(tokens.tolist()), a, **kw)
    mb.medusa_adjust_logits(tree, torch.from_numpy(z).cuda(), ints(tokens.tolist()), b, **kw)
    assert torch.equal(a, b)


# ---------------------------------------------------------------------------
# errors that only the device sees
# ---------------------------------------------------------------------------


def test_device_checks_leave_the_sequence_alone(mb):
    """A sequence past its table, and a bad page id: status set, that sequence untouched, the others right."""
    lens, news = [20, 10], [2, 2]
    c = Cache(mb, "bf16", 128, 16, 2, lens, news, extra_table=0)
    q = c.randn(4, 4, 128).bfloat16().cuda()
    k = c.randn(4, 2, 128).bfloat16().cuda()
    ws = mb.workspace(mb.medusa_paged_attention_workspace_size(c.kv, 4, 4))
    good, out = torch.empty_like(q), torch.full_like(q, 7.0)
    mb.medusa_paged_attention(c.kv, 0, q, good, 0.09, ws)
    over = mb.PagedKV(c.k, c.v, c.kv.page_table, ints([31, 10]))       # 31 + 2 > 2 pages of 16
    mb.medusa_paged_attention(over, 0, q, out, 0.09, ws)
    assert mb.device_status() == (mb.MEDUSA_ERR_DEVICE_CHECK, 11)
    assert (out[:2] == 7).all() and torch.equal(out[2:], good[2:])
    for bad in (-1, c.k.shape[1], 2 ** 31 - 1):
        table = [row[:] for row in c.table]
        table[0][0] = bad
        kv = mb.PagedKV(c.k, c.v, ints(table), ints(lens))
        mb.medusa_paged_attention(kv, 0, q, out, 0.09, ws)
        assert mb.device_status() == (mb.MEDUSA_ERR_DEVICE_CHECK, 12)
        assert torch.equal(out[2:], good[2:]) and out.isfinite().all()
    qo = torch.full_like(q, 7.0)
    before = c.k.clone()
    mb.medusa_rope_append(over, 0, q, k, k, qo, mb.Rotary(128))
    assert mb.device_status() == (mb.MEDUSA_ERR_DEVICE_CHECK, 11)
    assert (qo[:2] == 7).all() and not (qo[2:] == 7).all()
    assert torch.equal(c.k[0, c.table[0]].view(torch.uint8), before[0, c.table[0]].view(torch.uint8))


def test_device_checks_of_chunks(mb):
    c = Cache(mb, "bf16", 128, 16, 2, [20, 10, 0], [2, 2, 2])
    q = c.randn(6, 2, 128).bfloat16().cuda()
    ws = mb.workspace(mb.medusa_paged_attention_workspace_size(c.kv, 6, 2))
    good = torch.empty_like(q)
    mb.medusa_paged_attention(c.kv, 0, q, good, 0.09, ws)
    for starts, ok in (([0, 2, 1, 3], []), ([0, 2, 4, 9], [0, 1, 2, 3]), ([-3, 0, 2, 4], [])):
        out = torch.full_like(q, 7.0)
        mb.medusa_paged_attention(c.kv, 0, q, out, 0.09, ws, chunk_starts=ints(starts))
        assert mb.device_status() == (mb.MEDUSA_ERR_DEVICE_CHECK, 11)
        for n in ok:
            assert torch.equal(out[n], good[n])
        if starts[-1] == 9:
            assert (out[4:] == 7).all()


def test_device_checks_of_rope_chunks(mb):
    """A chunk that begins before row 0 or ends behind the last is not written; the others are."""
    c = Cache(mb, "bf16", 128, 16, 2, [20, 10, 0], [2, 2, 2])
    q, k = c.randn(6, 2, 128).bfloat16().cuda(), c.randn(6, 2, 128).bfloat16().cuda()
    rotary = mb.Rotary(128)
    good = torch.empty_like(q)
    mb.medusa_rope_append(c.kv, 0, q, k, k, good, rotary)
    for starts, ok in (([0, 2, 4, 9], [0, 1, 2, 3]), ([-3, 2, 4, 6], [2, 3, 4, 5])):
        out, before = torch.full_like(q, 7.0), c.k.clone()
        mb.medusa_rope_append(c.kv, 0, q, k, k, out, rotary, chunk_starts=ints(starts))
        assert mb.device_status() == (mb.MEDUSA_ERR_DEVICE_CHECK, 11)
        for n in range(6):
            assert torch.equal(out[n], good[n]) if n in ok else (out[n] == 7).all()
        assert torch.equal(c.k.view(torch.uint8), before.view(torch.uint8))      # the same rows, written again


def test_device_checks_of_accept_and_logits(mb):
    tree = mb.Tree(O.ranksum_choices(2, 2, 6), 2, 2)
    c = Cache(mb, "bf16", 64, 16, 2, [20, 10], [7, 7])
    before = c.k.clone()
    ws = mb.workspace(mb.medusa_paged_accept_workspace_size(c.kv))
    mb.medusa_paged_accept_kv(tree, c.kv, ints([99, 0]), ints([1, 1]), c.kv.seq_lens, ws)
    assert mb.device_status() == (mb.MEDUSA_ERR_DEVICE_CHECK, 13)
    assert c.kv.seq_lens.tolist() == [20, 12]
    assert torch.equal(c.k[0, c.table[0][:2]].view(torch.uint8), before[0, c.table[0][:2]].view(torch.uint8))
    z = torch.randn(2, 7, 100, device="cuda")
    out = torch.full_like(z, 7.0)
    mb.medusa_adjust_logits(tree, z, ints([[1] * 7] * 2), out, history=ints([[1, 2], [3, 4]]), history_lens=ints([3, 2]),
                            presence=torch.ones(2, device="cuda"))
    assert mb.device_status() == (mb.MEDUSA_ERR_DEVICE_CHECK, 15)
    assert (out[0] == 7).all() and not (out[1] == 7).any()


# ---------------------------------------------------------------------------
# streams, graphs, together
# ---------------------------------------------------------------------------


def test_other_stream_and_graph(mb):
    lens, news = [300, 40, 129], [1, 1, 1]
    c, q, out = check_attention(mb, "bf16", 128, 16, 8, 2, lens, news)
    side = torch.cuda.Stream()
    ws = mb.workspace(mb.medusa_paged_attention_workspace_size(c.kv, 3, 8))
    got = torch.zeros_like(out)
    side.wait_stream(torch.cuda.current_stream())
    mb.medusa_paged_attention(c.kv, 0, q, got, 128 ** -0.5, ws, stream=side)
    side.synchronize()
    assert torch.equal(got, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mb.medusa_paged_attention(c.kv, 0, q, got, 128 ** -0.5, ws)
    # replayed on other lengths and queries than it was captured with
    c.kv.seq_lens.copy_(ints([17, 41, 128]))
    q2 = c.randn(3, 8, 128).bfloat16().cuda()
    q.copy_(q2)
    for _ in range(3):
        graph.replay()
    want = torch.empty_like(got)
    ws2 = mb.workspace(mb.medusa_paged_attention_workspace_size(c.kv, 3, 8))
    mb.medusa_paged_attention(c.kv, 0, q, want, 128 ** -0.5, ws2)
    # sequence 1's own row (41) was never written: NaN in both
    assert np.array_equal(f64(got), f64(want), equal_nan=True) and got[[0, 2]].isfinite().all()


def test_two_graphs_at_once(mb):
    """Two captured calls with workspaces of their own, replayed at the same time on two streams, many times."""
    jobs = []
    for seed, (lens, news) in enumerate((([300, 1200], [70, 5]), ([2000, 40, 129], [1, 1, 1]))):
        c, q, want = check_attention(mb, "bf16", 128, 16, 8, 2, lens, news, seed=seed)
        ws = mb.workspace(mb.medusa_paged_attention_workspace_size(c.kv, sum(news), 8))
        got, starts = torch.zeros_like(want), ints(starts_of(news))
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph):
            mb.medusa_paged_attention(c.kv, 0, q, got, 128 ** -0.5, ws, chunk_starts=starts)
        jobs.append((graph, stream, got, want, c, q, ws, starts))
    torch.cuda.synchronize()
    for _ in range(50):
        for graph, stream, *_ in jobs:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, _, got, want, *_ in jobs:
        assert torch.equal(got, want)


def test_a_verification_step_over_pages(mb):
    """Rotary + append, attention, logits, acceptance and compaction, as a server runs them, and captured in a graph."""
    H, Hkv, hd, page, V = 8, 2, 128, 16, 1200
    lens = [37, 150]
    tree = mb.Tree(O.ranksum_choices(4, 8, 48), 4, 8)
    tab = tree.tables()
    T, B = tree.T, len(lens)
    c = Cache(mb, "bf16", hd, page, Hkv, lens, [T] * B, seed=5)
    k0, v0 = c.k.clone(), c.v.clone()
    rng = np.random.default_rng(3)
    qkv = c.randn(B * T, H + 2 * Hkv, hd).bfloat16().cuda()
    topk_ids = ints(rng.integers(0, V, (B, 4, 8)).tolist())
    root = ints([5, 9])
    tokens, cand, pos = (torch.empty(s, dtype=torch.int32, device="cuda") for s in ((B, T), (B, tree.P, tree.D + 1), (B, T)))
    logits = (3 * c.randn(B, T, V)).cuda()
    rep = torch.tensor([1.2, 1.05], device="cuda")
    hist = ints(rng.integers(0, V, (B, 160)).tolist())
    rotary = mb.Rotary(hd)
    rq, att, adj = torch.empty(B * T, H, hd, dtype=torch.bfloat16, device="cuda"), None, torch.empty_like(logits)
    att = torch.empty_like(rq)
    out = {n: torch.zeros(B, dtype=torch.int32, device="cuda") for n in ("best", "acc", "next")}
    accepted = torch.zeros(B, tree.D + 1, dtype=torch.int32, device="cuda")
    ws_a = mb.workspace(mb.medusa_paged_attention_workspace_size(c.kv, B * T, H))
    ws_p = mb.workspace(mb.medusa_posterior_workspace_size(tree, B))
    ws_c = mb.workspace(mb.medusa_paged_accept_workspace_size(c.kv))

    def step():
        mb.medusa_build_tree(tree, root, topk_ids, c.kv.seq_lens, tokens, cand, pos)
        mb.medusa_rope_append(c.kv, 0, qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:], rq, rotary, positions=pos.view(-1))
        mb.medusa_paged_attention(c.kv, 0, rq, att, hd ** -0.5, ws_a, tree=tree)
        mb.medusa_adjust_logits(tree, logits, tokens, adj, history=hist, history_lens=c.kv.seq_lens, repetition=rep)
        mb.medusa_evaluate_posterior(tree, adj, cand, mb.MEDUSA_GREEDY, out["best"], out["acc"], accepted, out["next"], ws_p)
        mb.medusa_paged_accept_kv(tree, c.kv, out["best"], out["acc"], c.kv.seq_lens, ws_c)

    # an accepted path: the adjusted argmax of node 0 is its first child's token
    mb.medusa_build_tree(tree, root, topk_ids, c.kv.seq_lens, tokens, cand, pos)
    child = tab["parent"].index(0)
    for b in range(B):
        logits[b, 0, tokens[b, child]] = 40.0
    step()
    torch.cuda.synchronize()
    # the same from the definitions
    qs, ks, vs = f64(qkv[:, :H]), f64(qkv[:, H:H + Hkv]), qkv[:, H + Hkv:]
    p = np.array([L + d for L in lens for d in tab["depth"]])
    freq, amp = PO.rope_frequencies(hd)
    ko, vo = f64(k0[0]), f64(v0[0])
    kr = PO.rotate(ks, p, freq, amp, hd, "half")
    qr = PO.rotate(qs, p, freq, amp, hd, "half")
    for b, L in enumerate(lens):
        for i in range(T):
            ko[c.table[b][(L + i) // page], :, (L + i) % page] = kr[b * T + i]
            vo[c.table[b][(L + i) // page], :, (L + i) % page] = f64(vs[b * T + i])
    sees = np.array([[(tab["anc"][i][j // 64] >> (j % 64)) & 1 for j in range(T)] for i in range(T)], bool)
    want, mass = PO.attention(qr, ko, vo, c.table, lens, starts_of([T] * B), hd ** -0.5, sees)
    # q and k rounded to bf16 move a score by 2 * 2^-8 sum |q k| scale at most; probabilities by twice that
    qk = np.abs(qr).sum(-1).max() * 6.0 * hd ** -0.5
    tol = mass * (2 * 2 * HALF_STEP["bf16"] * qk + HALF_STEP["bf16"]) + np.abs(want) * HALF_STEP["bf16"]
    err = np.abs(f64(att) - want)
    assert (err <= tol).all()
    assert np.sqrt((err ** 2).mean()) < 4 * HALF_STEP["bf16"] * np.sqrt((mass ** 2).mean())   # roundings of random sign
    zs = PO.adjust_logits(logits.cpu().numpy(), tokens.tolist(), tab["parent"],
                          history=[hist[b, :lens[b]].tolist() for b in range(B)], repetition=rep.double().cpu().numpy())
    post = O.evaluate_posterior(O.tree_tables(O.ranksum_choices(4, 8, 48), 4, 8), zs, cand.cpu().numpy(), "greedy")
    assert out["best"].tolist() == list(post["best_path"]) and out["acc"].tolist() == list(post["accept_len"])
    assert all(a >= 1 for a in out["acc"].tolist())
    assert c.kv.seq_lens.tolist() == [L + a + 1 for L, a in zip(lens, out["acc"].tolist())]
    # captured: the same results from the same start
    after = (c.k.clone(), c.v.clone(), att.clone(), c.kv.seq_lens.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    c.k.copy_(k0), c.v.copy_(v0), c.kv.seq_lens.copy_(ints(lens)), att.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for got, ref in zip((c.k, c.v, att, c.kv.seq_lens), after):
        assert torch.equal(got.contiguous().view(torch.uint8), ref.contiguous().view(torch.uint8))
