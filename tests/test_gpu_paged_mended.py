"""The paged-cache calls on the GPU where arguments or the machine let them down."""

import numpy as np
import pytest
import torch

import oracle.medusa_oracle as O
import oracle.paged_oracle as PO
from test_gpu_paged import Cache, check_attention, f64, ints, starts_of

pytestmark = pytest.mark.gpu


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


@pytest.mark.parametrize("starts", [[0, 10, 5, 12], [0, 12, 12, 11], [3, 2, 7, 12], [12, 8, 4, 0]], ids=str)
@pytest.mark.parametrize("dtype,hd,rot", [("bf16", 128, 128), ("f32", 64, 6)], ids=["vectors", "elements"])
def test_rope_append_writes_nothing_for_chunks_that_descend(mb, dtype, hd, rot, starts):
    """Overlapping chunks: a row would belong to two sequences, and one of them would be left with a hole."""
    c = Cache(mb, dtype, hd, 16, 2, [20, 10, 0], [12, 12, 12])
    q, k = c.randn(12, 4, hd).to(c.k.dtype).cuda(), c.randn(12, 2, hd).to(c.k.dtype).cuda()
    out = torch.full_like(q, 7.0)
    before = c.k.clone(), c.v.clone()
    rotary = mb.Rotary(rot)
    mb.medusa_rope_append(c.kv, 0, q, k, k, out, rotary, chunk_starts=ints(starts))
    assert mb.device_status() == (mb.MEDUSA_ERR_DEVICE_CHECK, 11)
    assert (out == 7).all()
    for now, was in zip((c.k, c.v), before):
        assert torch.equal(now.view(torch.uint8), was.view(torch.uint8))
    mb.medusa_rope_append(c.kv, 0, q, k, k, out, rotary, chunk_starts=ints([0, 5, 5, 12]))     # one that does not, empty chunk and all
    assert not (out == 7).any() and not torch.equal(c.k.view(torch.uint8), before[0].view(torch.uint8))


WAITS = {  # hd, page, H, Hkv, lens, news
    "few rows": (128, 16, 8, 2, [300, 1500, 40], [1, 1, 1]),
    "alternating tiles": (64, 16, 8, 2, [300, 90], [40, 11]),
    "two groups of rows": (128, 64, 64, 8, [300, 40], [500, 140]),
}


@pytest.mark.parametrize("case", sorted(WAITS))
def test_a_wait_that_runs_out_ends_the_call(mb, case):
    """A barrier between two roles expects one arrival that nobody makes, for at most 1 ms: the call reports it, writes
    none of the rows (no piece is finished), and leaves a context in which the next call, its workspace zeroed, is exact."""
    hd, page, H, Hkv, lens, news = WAITS[case]
    c = Cache(mb, "bf16", hd, page, Hkv, lens, news)
    N, starts = sum(news), ints([sum(news[:b]) for b in range(len(news) + 1)])
    q = c.randn(N, H, hd).bfloat16().cuda()
    ws = mb.workspace(mb.medusa_paged_attention_workspace_size(c.kv, N, H))
    want, out = torch.empty_like(q), torch.full_like(q, 7.0)
    args = dict(chunk_starts=None if case == "few rows" else starts)
    mb.medusa_paged_attention(c.kv, 0, q, want, hd ** -0.5, ws, **args)
    torch.cuda.synchronize()
    assert mb.device_status() == (0, 0)
    try:
        mb.medusa_test_paged_wait(1, 1_000_000)
        mb.medusa_paged_attention(c.kv, 0, q, out, hd ** -0.5, ws, **args)
        torch.cuda.synchronize()
    finally:
        mb.medusa_test_paged_wait(0, 0)
    assert mb.device_status() == (mb.MEDUSA_ERR_TIMEOUT, 14)
    assert (out == 7).all()
    ws.zero_()
    for _ in range(2):
        mb.medusa_paged_attention(c.kv, 0, q, out, hd ** -0.5, ws, **args)
        assert torch.equal(out, want)
        out.fill_(7.0)


MOST_ROWS = 2 ** 31 - 257


def test_the_most_rows_of_a_sequence(mb):
    """Row numbers stay inside 31 bits: the append, attention and the compaction refuse a sequence that would pass them,
    as one that outgrows its table, and serve the longest that does not.  Every entry of the table is page 0, so a cache
    of two pages stands for all of it; the first sequence is short and always served."""
    hd, page, T = 8, 256, 7
    pages = torch.zeros(1, 2, 1, page, hd, device="cuda")
    table = torch.zeros(2, 2 ** 31 // page + 2, dtype=torch.int32, device="cuda")
    table[0] = 1
    tree = mb.Tree(O.ranksum_choices(2, 2, T - 1), 2, 2)
    assert tree.T == T
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(2 * T, 1, hd, generator=g, device="cuda")
    rotary = mb.Rotary(hd)
    for L, ok in ((MOST_ROWS - T, True), (MOST_ROWS - T + 1, False), (2 ** 31 - 3, False), (2 ** 31 - 1, False)):
        kv = mb.PagedKV(pages.clone(), pages.clone(), table, ints([3, L]))
        before = kv.v_pages.clone()
        out = torch.full_like(x, 7.0)
        mb.medusa_rope_append(kv, 0, x, x, x, out, rotary)
        assert mb.device_status() == ((0, 0) if ok else (mb.MEDUSA_ERR_DEVICE_CHECK, 11))
        assert not (out[:T] == 7).any() and (out[T:] == 7).all() == (not ok)
        assert torch.equal(kv.v_pages[0, 1, 0, 3:3 + T], x[:T, 0])
        assert torch.equal(kv.v_pages[0, 0], before[0, 0]) == (not ok)
        if ok:
            assert torch.equal(kv.v_pages[0, 0, 0, [r % page for r in range(L, L + T)]], x[T:, 0])
        new = ints([-5, -5])
        ws = mb.workspace(mb.medusa_paged_accept_workspace_size(kv))
        mb.medusa_paged_accept_kv(tree, kv, ints([0, 0]), ints([1, 1]), new, ws)
        assert mb.device_status() == ((0, 0) if ok else (mb.MEDUSA_ERR_DEVICE_CHECK, 13))
        assert new.tolist() == [5, L + 2 if ok else -5]
    # attention computes over such a sequence only where it is refused: 2^31 rows would take the test's time
    kv = mb.PagedKV(pages, pages, table, ints([3, MOST_ROWS]))
    ws = mb.workspace(mb.medusa_paged_attention_workspace_size(kv, 2, 1))
    out = torch.full_like(x[:2], 7.0)
    mb.medusa_paged_attention(kv, 0, x[:2].contiguous(), out, 1.0, ws)
    assert mb.device_status() == (mb.MEDUSA_ERR_DEVICE_CHECK, 11)
    assert out[0].isfinite().all() and not (out[0] == 7).any() and (out[1] == 7).all()


ERRORS = [
    # hd, page, H, Hkv, lens, news (None: a tree of so many nodes), nodes, probabilities as a pair
    (128, 16, 8, 8, [700, 1100, 33], [1, 1, 1], 0, True),
    (64, 16, 8, 2, [700], [4], 0, True),
    (128, 64, 4, 4, [300, 77], None, 64, False),              # alternating tiles
    (64, 16, 8, 2, [200], None, 48, False),
    (128, 16, 4, 4, [127, 500], [130, 3], 0, False),          # ragged chunks, one group of rows
    (128, 64, 64, 8, [300, 40], [400, 140], 0, False),        # two groups of rows
    (64, 32, 64, 8, [0, 130], [303, 300], 0, False),
    (128, 16, 8, 8, [400, 9, 33], [1, 1, 20], 0, False),      # single tokens that travel with a prompt
]


@pytest.mark.parametrize("case", ERRORS, ids=lambda c: "-".join(str(x) for x in c))
def test_the_error_of_bf16_attention(mb, case):
    """Root mean square against 64 bits: the output's one rounding and, where the probabilities are one bf16 each, theirs.
    A rounding to bf16 is off by at most 2^-8 of the value, evenly spread and so 2^-8 / sqrt(3) in root mean square; those
    of different keys are independent, so their squares add up: (2^-8)^2 / 3 times the sum over the keys of (p v)^2.  A
    pair leaves half a step of a remainder that is itself half a step, 2^-16; scores, exponentials and sums in fp32 stay
    below 2^-13 for these up to 1100 keys.  Beside the output's rounding of over 2^-10 that is less than 1% in squares,
    and 5% leaves room for values that round the other way."""
    hd, page, H, Hkv, lens, news, nodes, as_pair = case
    tree = sees = None
    if news is None:
        tree = mb.Tree(O.ranksum_choices(5, 10, nodes), 5, 10)
        anc = tree.tables()["anc"]
        sees = np.array([[(anc[i][j // 64] >> (j % 64)) & 1 for j in range(tree.T)] for i in range(tree.T)], bool)
    count = [tree.T] * len(lens) if news is None else news
    starts = starts_of(count)
    c = Cache(mb, "bf16", hd, page, Hkv, lens, count, seed=nodes)
    q = c.randn(sum(count), H, hd).bfloat16().cuda()
    out = torch.full_like(q, 7.0)
    ws = mb.workspace(mb.medusa_paged_attention_workspace_size(c.kv, q.shape[0], H))
    mb.medusa_paged_attention(c.kv, 0, q, out, hd ** -0.5, ws, tree=tree,
                              chunk_starts=None if len(set(count)) == 1 else ints(starts))
    k, v, q = f64(c.k[0]), f64(c.v[0]), f64(q)
    want, _ = PO.attention(q, k, v, c.table, lens, starts, hd ** -0.5, sees)
    once = np.mean((f64(torch.from_numpy(want).bfloat16()) - want) ** 2)
    theirs = np.zeros_like(want)
    for b, (L, n) in enumerate(zip(lens, count)):
        kb, vb = (np.repeat(PO.gather_rows(x, c.table[b], L + n), H // Hkv, 0) for x in (k, v))
        qb = q[starts[b]:starts[b + 1]].transpose(1, 0, 2)
        visible = np.concatenate([np.ones((n, L), bool), sees if sees is not None else np.tril(np.ones((n, n), bool))], 1)
        p = np.exp(np.where(visible, qb @ kb.transpose(0, 2, 1) * hd ** -0.5, -np.inf))
        p /= p.sum(-1, keepdims=True)
        theirs[starts[b]:starts[b + 1]] = (p ** 2 @ vb ** 2).transpose(1, 0, 2)
    assert once > 2.0 ** -20 * np.mean(want ** 2)
    most = once + (0 if as_pair else np.mean(theirs) * 2.0 ** -16 / 3)
    assert np.mean((f64(out) - want) ** 2) < 1.05 ** 2 * most


# ---------------------------------------------------------------------------
# calls that the documentation allows, at the ends of their ranges
# ---------------------------------------------------------------------------


@pytest.mark.parametrize("dtype,hd", [("bf16", 128), ("bf16", 64), ("bf16", 40), ("f32", 64)])
@pytest.mark.parametrize("news,rows", [([0, 0, 0], 4), ([0, 0, 0], 40), ([2, 0, 1], 5), ([30, 0, 11], 60)], ids=str)
def test_rows_behind_the_last_chunk_stay(mb, dtype, hd, news, rows):
    """More packed rows than chunks, and chunks that are all empty, by every kernel: those rows keep what they held."""
    c = Cache(mb, dtype, hd, 16, 2, [20, 300, 5], news)
    q = c.randn(rows, 4, hd).to(c.k.dtype).cuda()
    starts = starts_of(news)
    ws = mb.workspace(mb.medusa_paged_attention_workspace_size(c.kv, rows, 4))
    out = torch.full_like(q, 7.0)
    for _ in range(2):
        mb.medusa_paged_attention(c.kv, 0, q, out, 0.1, ws, chunk_starts=ints(starts))
        assert (out[starts[-1]:] == 7).all()
    if starts[-1]:
        want, mass = PO.attention(f64(q[:starts[-1]]), f64(c.k[0]), f64(c.v[0]), c.table, [20, 300, 5], starts, 0.1)
        # probabilities and output rounded to bf16 (2^-8 each); fp32 terms far below 2^-10 for these scores
        tol = mass * (2.0 ** -8 + 2.0 ** -10) + np.abs(want) * 2.0 ** -8 if dtype == "bf16" else mass * 2.0 ** -10
        assert (np.abs(f64(out[:starts[-1]]) - want) <= tol).all()


@pytest.mark.parametrize("case", [
    ("f32", 64, 16, 4, 1, [40, 3, 0, 9, 100, 7, 7, 7], [8, 0, 0, 0, 0, 0, 0, 0]),     # 32 rows where the average is 4: two tiles of 16
    ("bf16", 40, 16, 4, 1, [40, 3, 0, 9, 100, 7, 7, 7], [0, 1, 0, 7, 0, 0, 0, 0]),
    ("bf16", 128, 16, 20, 10, [3 * b for b in range(64)], [1] * 64),                  # 640 units: few rows, and more than four
    ("bf16", 128, 16, 20, 10, [3 * b for b in range(64)], [3] * 64),
    ("bf16", 64, 16, 20, 10, [3 * b for b in range(64)], [3] * 64),
], ids=["f32-tiles", "bf16-tiles", "many-units", "many-units-6-rows", "many-units-64"])
def test_attention_at_the_bounds_between_the_kernels(mb, case):
    check_attention(mb, *case)


def test_too_many_blocks_of_keys(mb):
    """Over 2^30 blocks of keys in a call: refused, with nothing computed."""
    hd, page, Hkv = 8, 256, 40
    pages = torch.zeros(1, 1, Hkv, page, hd, device="cuda")
    table = torch.zeros(1, MOST_ROWS // page + 1, dtype=torch.int32, device="cuda")
    kv = mb.PagedKV(pages, pages.clone(), table, ints([MOST_ROWS - 1]))
    assert (MOST_ROWS // 32) * Hkv > 2 ** 30
    q = torch.zeros(1, Hkv, hd, device="cuda")
    out = torch.full_like(q, 7.0)
    ws = mb.workspace(mb.medusa_paged_attention_workspace_size(kv, 1, Hkv))
    mb.medusa_paged_attention(kv, 0, q, out, 1.0, ws)
    assert mb.device_status() == (mb.MEDUSA_ERR_DEVICE_CHECK, 11)
    assert (out == 7).all() and not ws.any()


@pytest.mark.parametrize("dtype,hd", [("bf16", 64), ("f32", 8)])
def test_a_prefix_of_millions_of_rows(mb, dtype, hd):
    """A prefix whose pages are all the same page: every row has the weight of its copies, so the output is that of the
    one page, the new token aside.  Scores are zero, which makes the weights equal: the mean of the values."""
    page, L = 256, 3_000_000 * 2 - 1
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(2)
    k = torch.randn(1, 2, 1, page, hd, generator=g, device="cuda").to(t)
    v = (torch.randn(1, 2, 1, page, hd, generator=g, device="cuda") + 1).to(t)
    table = torch.zeros(1, L // page + 1, dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    kv = mb.PagedKV(k, v, table, ints([L]))
    q = torch.zeros(1, 4, hd, dtype=t, device="cuda")
    out = torch.full_like(q, 7.0)
    ws = mb.workspace(mb.medusa_paged_attention_workspace_size(kv, 1, 4))
    mb.medusa_paged_attention(kv, 0, q, out, 1.0, ws)
    copies, last = (L + 1) // page, (L + 1) % page
    want = (f64(v[0, 0, 0]).sum(0) * copies + f64(v[0, 1, 0, :last]).sum(0)) / (L + 1)
    # A block's range is at most 6 million / 148 rows, below 2^16, and at most 2^10 ranges are joined: a sum of n terms is
    # off by n 2^-24 of their absolute sum at the very most, twice (numerator and denominator); then the output's rounding.
    mass = (np.abs(f64(v[0, 0, 0])).sum(0) * copies + np.abs(f64(v[0, 1, 0, :last])).sum(0)) / (L + 1)
    tol = mass * 2 * (2.0 ** -8 + 2.0 ** -14) + (np.abs(want) * 2.0 ** -8 if dtype == "bf16" else 0)
    assert (np.abs(f64(out[0]) - want) <= tol).all()
