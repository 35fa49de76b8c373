"""The paged-cache calls and the logit adjustment without a GPU: the fp64
definitions against independent forms of the same formulas, the table of
rotary frequencies, and every refusal.  No compute call reaches a device."""

import ctypes
import math

import numpy as np
import pytest
import torch

import oracle.medusa_oracle as O
import oracle.paged_oracle as PO

bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def mb(built):
    import speculative_decoding_heads_b200 as mb
    return mb


@pytest.fixture(scope="module")
def tree(mb):
    t = mb.Tree([(0,), (1,), (0, 0), (0, 1), (1, 0), (1, 1)], 2, 2, upload=False)
    yield t
    t.close()


# ---------------------------------------------------------------------------
# the definitions
# ---------------------------------------------------------------------------


def paged(dense, page, rng):
    """Dense rows [B][Hkv, rows, hd] in shuffled pages: (pages, table)."""
    Hkv, _, hd = dense[0].shape
    used = [-(-d.shape[1] // page) for d in dense]
    order = rng.permutation(sum(used)).tolist()
    pages = np.full((sum(used), Hkv, page, hd), np.nan)
    table = []
    for d, u in zip(dense, used):
        ids = [order.pop() for _ in range(u)]
        for r in range(d.shape[1]):
            pages[ids[r // page], :, r % page] = d[:, r]
        table.append(ids)
    return pages, table


@pytest.mark.parametrize("H,Hkv", [(4, 4), (6, 2)])
def test_attention_definition_against_torch(H, Hkv):
    rng = np.random.default_rng(H)
    lens, news, hd, page = [5, 0, 17], [4, 3, 1], 16, 8
    K = [rng.normal(size=(Hkv, L + n, hd)) for L, n in zip(lens, news)]
    V = [rng.normal(size=k.shape) for k in K]
    kp, table = paged(K, page, np.random.default_rng(1))
    vp, _ = paged(V, page, np.random.default_rng(1))
    q = rng.normal(size=(sum(news), H, hd))
    starts = [0, 4, 7, 8]
    out, _ = PO.attention(q, kp, vp, table, lens, starts, 0.25)
    for b, (L, n) in enumerate(zip(lens, news)):
        qb = torch.from_numpy(q[starts[b]:starts[b + 1]]).transpose(0, 1)
        kb, vb = (torch.from_numpy(x[b]).repeat_interleave(H // Hkv, 0) for x in (K, V))
        mask = torch.ones(n, L + n, dtype=torch.bool).tril(L)
        ref = torch.nn.functional.scaled_dot_product_attention(qb, kb, vb, attn_mask=mask, scale=0.25).transpose(0, 1)
        assert np.allclose(out[starts[b]:starts[b + 1]], ref.numpy(), atol=1e-12)


def test_tree_attention_definition_against_the_dense_one():
    tr = O.tree_tables(O.ranksum_choices(3, 2, 14), 3, 2)
    T, H, hd, page, lens = tr["T"], 2, 8, 4, [3, 10]
    rng = np.random.default_rng(2)
    q = rng.normal(size=(1, 2, T, H, hd))
    kc, vc = (rng.normal(size=(1, 2, H, 30, hd)) for _ in range(2))
    ref = O.tree_attention(tr, q, kc, vc, np.array(lens), 0.3)
    dense = lambda c: [c[0, b][:, :lens[b] + T] for b in range(2)]  # noqa: E731
    kp, table = paged(dense(kc), page, np.random.default_rng(1))
    vp, _ = paged(dense(vc), page, np.random.default_rng(1))
    out, _ = PO.attention(q[0].reshape(2 * T, H, hd), kp, vp, table, lens, [0, T, 2 * T], 0.3,
                          np.asarray(tr["anc"], bool))
    assert np.allclose(out.reshape(2, T, H, hd), ref[0], atol=1e-12)


def test_accept_definition_against_the_dense_one():
    tr = O.tree_tables(O.ranksum_choices(3, 2, 14), 3, 2)
    T, page, lens = tr["T"], 4, [3, 10]
    rng = np.random.default_rng(4)
    kc = rng.normal(size=(1, 2, 2, 30, 8))
    best, acc = [3, 5], [min(2, sum(x >= 0 for x in tr["retrieve"][3]) - 1), 1]
    pages, table = paged([kc[0, b][:, :lens[b] + T] for b in range(2)], page, rng)
    got = PO.accept(pages[None], table, lens, tr["retrieve"], best, acc)
    for b in range(2):
        rows = PO.gather_rows(got[0], table[b], lens[b] + acc[b] + 1)
        want = kc[0, b].copy()
        for j in range(acc[b] + 1):
            want[:, lens[b] + j] = kc[0, b][:, lens[b] + tr["retrieve"][best[b]][j]]
        assert np.array_equal(rows, want[:, :lens[b] + acc[b] + 1])


def test_rotate_keeps_lengths_and_relative_positions():
    """A rotation preserves every pair's length, and products of rotated vectors depend on the distance alone."""
    rng = np.random.default_rng(5)
    x, y = rng.normal(size=(1, 1, 16)), rng.normal(size=(1, 1, 16))
    freq, _ = PO.rope_frequencies(8)
    for layout in ("half", "interleaved"):
        r = lambda v, p: PO.rotate(v, [p], freq, 1.0, 8, layout)[0, 0]  # noqa: E731
        assert np.allclose(np.linalg.norm(r(x, 77)), np.linalg.norm(x))
        assert np.allclose(r(x, 10) @ r(y, 4), r(x, 1006) @ r(y, 1000))
        assert np.array_equal(r(x, 3)[8:], x[0, 0, 8:])
    half, inter = PO.rotate(x, [9], freq, 1.0, 8, "half"), PO.rotate(x[..., [0, 4, 1, 5, 2, 6, 3, 7] + list(range(8, 16))], [9], freq, 1.0, 8, "interleaved")
    assert np.allclose(half[..., [0, 4, 1, 5, 2, 6, 3, 7]], inter[..., :8])


def test_logits_definition_closed_forms():
    z = np.array([[[2.0, -2.0, 1.0, 0.0]] * 3])
    parent = [-1, 0, 0]
    out = PO.adjust_logits(z, [[0, 1, 1]], parent, history=[[1, 2, 2]], prompt_lens=[2], repetition=[2.0], presence=[0.5],
                           frequency=[0.25], bias=[[(3, 1.0), (3, 1.0)]])
    # node 0: path {0}; token 1 only in the prompt, token 2 once generated
    assert np.allclose(out[0, 0], [2 / 2 - 0.75, -4.0, 0.5 - 0.75, 2.0])
    # node 1: path {0, 1}
    assert np.allclose(out[0, 1], [2 / 2 - 0.75, -4.0 - 0.75, 0.5 - 0.75, 2.0])
    assert np.array_equal(out[0, 1], out[0, 2])
    allowed = np.ones((1, 3, 4), bool)
    allowed[0, 2, 1:3] = False
    assert np.isneginf(PO.adjust_logits(z, [[0, 1, 1]], parent, allowed=allowed)).tolist() == (~allowed).tolist()


# ---------------------------------------------------------------------------
# rotary frequencies
# ---------------------------------------------------------------------------


@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 4.0), ("ntk", 2.0), ("yarn", 16.0), ("yarn", 1.0)])
@pytest.mark.parametrize("rot", [4, 32, 64, 128, 256])
def test_rotary_turns(mb, rot, scaling, factor):
    turns, amp = mb.medusa_rotary_turns(rot, 10000.0, ["none", "linear", "ntk", "yarn"].index(scaling), factor, 4096)
    freq, want_amp = PO.rope_frequencies(rot, 10000.0, scaling, factor, 4096)
    # both in double precision: a few units of 2^-53 each, and the table's last bit, 2^-64 turns = 2 pi 2^-64 radians
    assert np.allclose(np.array(turns, dtype=np.float64) / 2.0 ** 64 * 2 * math.pi, freq, rtol=1e-14, atol=2 * math.pi * 2.0 ** -64)
    assert amp == np.float32(want_amp)


@pytest.mark.parametrize("over", [dict(rot=0), dict(rot=3), dict(rot=258), dict(base=1.0), dict(base=math.inf), dict(scaling=4),
                                  dict(factor=0.5), dict(factor=math.nan), dict(rot=2, scaling=2), dict(scaling=3, original_length=0),
                                  dict(scaling=3, beta_fast=1.0, beta_slow=1.0), dict(scaling=3, beta_slow=0.0)])
def test_rotary_turns_refuses(mb, over):
    with pytest.raises(mb.MedusaError) as e:
        mb.medusa_rotary_turns(**{**dict(rot=64), **over})
    assert e.value.code == mb.MEDUSA_ERR_INVALID_ARG


# ---------------------------------------------------------------------------
# the binding's refusals (each before it looks at where a tensor lives)
# ---------------------------------------------------------------------------

B, N, H, Hkv, hd, page = 2, 6, 4, 2, 64, 16


def _cache(**over):
    a = dict(k_pages=torch.zeros(2, 5, Hkv, page, hd, dtype=bf), v_pages=torch.zeros(2, 5, Hkv, page, hd, dtype=bf),
             page_table=torch.zeros(B, 4, dtype=i32), seq_lens=torch.zeros(B, dtype=i32))
    a.update(over)
    return a


@pytest.mark.parametrize("over", [
    dict(k_pages=torch.zeros(5, Hkv, page, hd, dtype=bf)), dict(v_pages=torch.zeros(2, 5, Hkv, page, hd)),
    dict(v_pages=torch.zeros(2, 4, Hkv, page, hd, dtype=bf)), dict(page_table=torch.zeros(B, 4, dtype=torch.int64)),
    dict(page_table=torch.zeros(B, 8, dtype=i32)[:, ::2]), dict(seq_lens=torch.zeros(B + 1, dtype=i32)),
    dict(k_pages=torch.zeros(2, 5, page, Hkv, hd, dtype=bf).transpose(2, 3)), dict(page_table=torch.zeros(4, dtype=i32))])
def test_paged_kv_refuses(mb, over):
    with pytest.raises(ValueError):
        mb.PagedKV(**_cache(**over))


def test_paged_kv_refuses_other_dtypes(mb):
    with pytest.raises(mb.MedusaError):
        mb.PagedKV(**_cache(k_pages=torch.zeros(2, 5, Hkv, page, hd, dtype=torch.float16)))


def _rotary(mb):
    r = mb.Rotary.__new__(mb.Rotary)
    r.turns, r.rot, r.layout, r.amplitude = torch.zeros(hd // 2, dtype=torch.int64), hd, 0, 1.0
    r.c = mb.RotaryArgs(0, hd, r.turns.data_ptr(), 1.0)
    r.ref = ctypes.byref(r.c)
    return r


ROPE = {
    "q of another head size": dict(q=torch.zeros(N, H, hd + 8, dtype=bf)),
    "q fp32": dict(q=torch.zeros(N, H, hd)),
    "q heads strided": dict(q=torch.zeros(N, 2 * H, hd, dtype=bf)[:, ::2]),
    "k of H heads": dict(k=torch.zeros(N, H, hd, dtype=bf)),
    "v short": dict(v=torch.zeros(N - 2, Hkv, hd, dtype=bf)),
    "q_out strided": dict(q_out=torch.zeros(N, 2 * H, hd, dtype=bf)[:, :H]),
    "q_out fp32": dict(q_out=torch.zeros(N, H, hd)),
    "positions int64": dict(positions=torch.zeros(N, dtype=torch.int64)),
    "positions short": dict(positions=torch.zeros(N - 1, dtype=i32)),
    "starts short": dict(chunk_starts=torch.zeros(B, dtype=i32)),
    "uneven chunks without starts": dict(q=torch.zeros(5, H, hd, dtype=bf), k=torch.zeros(5, Hkv, hd, dtype=bf),
                                         v=torch.zeros(5, Hkv, hd, dtype=bf), q_out=torch.zeros(5, H, hd, dtype=bf)),
    "no token": dict(q=torch.zeros(0, H, hd, dtype=bf), k=torch.zeros(0, Hkv, hd, dtype=bf),
                     v=torch.zeros(0, Hkv, hd, dtype=bf), q_out=torch.zeros(0, H, hd, dtype=bf)),
    "host tensors": {},
}


@pytest.mark.parametrize("case", sorted(ROPE))
def test_rope_append_refuses(mb, case):
    kv = mb.PagedKV(**_cache())
    a = dict(q=torch.zeros(N, H, hd, dtype=bf), k=torch.zeros(N, Hkv, hd, dtype=bf), v=torch.zeros(N, Hkv, hd, dtype=bf),
             q_out=torch.zeros(N, H, hd, dtype=bf), positions=None, chunk_starts=None)
    a.update(ROPE[case])
    with pytest.raises(ValueError, match="CUDA tensors" if case == "host tensors" else None):
        mb.medusa_rope_append(kv, 0, a["q"], a["k"], a["v"], a["q_out"], _rotary(mb), positions=a["positions"],
                              chunk_starts=a["chunk_starts"])


ATTN = {
    "q fp32": lambda t: dict(q=torch.zeros(N, H, hd)),
    "q strided": lambda t: dict(q=torch.zeros(N, H + 2, hd, dtype=bf)[:, :H]),
    "out fp32": lambda t: dict(out=torch.zeros(N, H, hd)),
    "out short": lambda t: dict(out=torch.zeros(N - 1, H, hd, dtype=bf)),
    "uneven chunks without starts": lambda t: dict(q=torch.zeros(5, H, hd, dtype=bf), out=torch.zeros(5, H, hd, dtype=bf)),
    "starts int64": lambda t: dict(chunk_starts=torch.zeros(B + 1, dtype=torch.int64)),
    "tree of another size": lambda t: dict(tree=t),
    "tree with starts": lambda t: dict(tree=t, q=torch.zeros(14, H, hd, dtype=bf), out=torch.zeros(14, H, hd, dtype=bf),
                                       chunk_starts=torch.zeros(B + 1, dtype=i32)),
    "workspace strided": lambda t: dict(ws=torch.zeros(8192, dtype=torch.uint8)[::2]),
    "host tensors": lambda t: {},
}


@pytest.mark.parametrize("case", sorted(ATTN))
def test_paged_attention_refuses(mb, tree, case):
    kv = mb.PagedKV(**_cache())
    a = dict(q=torch.zeros(N, H, hd, dtype=bf), out=torch.zeros(N, H, hd, dtype=bf), ws=torch.zeros(4096, dtype=torch.uint8),
             tree=None, chunk_starts=None)
    a.update(ATTN[case](tree))
    with pytest.raises(ValueError, match="CUDA tensors" if case == "host tensors" else None):
        mb.medusa_paged_attention(kv, 0, a["q"], a["out"], 0.1, a["ws"], tree=a["tree"], chunk_starts=a["chunk_starts"])


ACCEPT = {"best int64": dict(best=torch.zeros(B, dtype=torch.int64)), "accept short": dict(acc=torch.zeros(B - 1, dtype=i32)),
          "lens float": dict(new=torch.zeros(B)), "host tensors": {}}


@pytest.mark.parametrize("case", sorted(ACCEPT))
def test_paged_accept_refuses(mb, tree, case):
    kv = mb.PagedKV(**_cache())
    a = dict(best=torch.zeros(B, dtype=i32), acc=torch.zeros(B, dtype=i32), new=torch.zeros(B, dtype=i32))
    a.update(ACCEPT[case])
    with pytest.raises(ValueError, match="CUDA tensors" if case == "host tensors" else None):
        mb.medusa_paged_accept_kv(tree, kv, a["best"], a["acc"], a["new"], torch.zeros(256, dtype=torch.uint8))


T, V = 7, 50
LOGITS = {
    "another tree": dict(logits=torch.zeros(B, T + 1, V)),
    "bf16 logits": dict(logits=torch.zeros(B, T, V, dtype=bf)),
    "logits strided": dict(logits=torch.zeros(B, T, 2 * V)[..., :V]),
    "out short": dict(out=torch.zeros(B, T, V - 1)),
    "penalty without tree tokens": dict(tree_tokens=None, presence=torch.zeros(B)),
    "penalty fp64": dict(repetition=torch.ones(B, dtype=torch.float64)),
    "penalty per node": dict(frequency=torch.ones(B, T)),
    "history without lengths": dict(history=torch.zeros(B, 3, dtype=i32)),
    "lengths without history": dict(history_lens=torch.zeros(B, dtype=i32)),
    "prompt lengths without history": dict(prompt_lens=torch.zeros(B, dtype=i32)),
    "history int64": dict(history=torch.zeros(B, 3, dtype=torch.int64), history_lens=torch.zeros(B, dtype=i32)),
    "history of no room": dict(history=torch.zeros(B, 0, dtype=i32), history_lens=torch.zeros(B, dtype=i32)),
    "bias without ids": dict(bias=torch.zeros(B, 2)),
    "bias of another shape": dict(bias=torch.zeros(B, 3), bias_ids=torch.zeros(B, 2, dtype=i32)),
    "too many biases": dict(bias=torch.zeros(B, 1025), bias_ids=torch.zeros(B, 1025, dtype=i32)),
    "mask of too few words": dict(allowed=torch.zeros(B, T, 1, dtype=i32)),
    "mask of bytes": dict(allowed=torch.zeros(B, T, 2, dtype=torch.uint8)),
    "host tensors": {},
}


@pytest.mark.parametrize("case", sorted(LOGITS))
def test_adjust_logits_refuses(mb, tree, case):
    a = dict(logits=torch.zeros(B, T, V), tree_tokens=torch.zeros(B, T, dtype=i32), out=torch.zeros(B, T, V))
    a.update(LOGITS[case])
    with pytest.raises(ValueError, match="CUDA tensors" if case == "host tensors" else None):
        mb.medusa_adjust_logits(tree, **a)


# ---------------------------------------------------------------------------
# the C ABI's own refusals (made-up device pointers; only where there is no device to run on)
# ---------------------------------------------------------------------------

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up pointers: only without a device")
P = 0x10000000


def c_kv(mb, **over):
    a = dict(dtype=mb.MEDUSA_BF16, layers=2, n_pages=5, Hkv=2, page=16, hd=64, k_pages=P, v_pages=2 * P, B=2, max_pages=4,
             page_table=3 * P, seq_lens=4 * P)
    a.update(over)
    return mb.PagedKVArgs(*[a[f] for f, _ in mb.PagedKVArgs._fields_])


def rope_call(mb, kv=None, layer=0, N=6, H=4, q=5 * P, qs=256, k=6 * P, ks=128, v=7 * P, vs=128, out=8 * P, layout=0, rot=64,
              turns=9 * P, amplitude=1.0, positions=None, starts=None):
    return mb._lib.medusa_rope_append(ctypes.byref(kv if kv is not None else c_kv(mb)), layer, N, H, q, qs, k, ks, v, vs, out,
                                      ctypes.byref(mb.RotaryArgs(layout, rot, turns, amplitude)), positions, starts, None)


BAD_KV = [dict(dtype=2), dict(layers=0), dict(n_pages=0), dict(Hkv=0), dict(page=12), dict(page=4), dict(page=512), dict(hd=0),
          dict(hd=60), dict(hd=264), dict(k_pages=None), dict(v_pages=P + 8), dict(B=0), dict(B=65), dict(max_pages=0),
          dict(page_table=None), dict(seq_lens=None), dict(seq_lens=P + 2)]


@no_gpu
@pytest.mark.parametrize("over", BAD_KV, ids=str)
def test_c_paged_kv(mb, over):
    kv = c_kv(mb, **over)
    assert rope_call(mb, kv) in (mb.MEDUSA_ERR_INVALID_ARG, mb.MEDUSA_ERR_UNSUPPORTED)
    assert mb._lib.medusa_paged_attention(ctypes.byref(kv), 0, 6, 4, 5 * P, 0.1, None, None, 6 * P, 7 * P, 1 << 40, None) in (1, 2)
    assert mb._lib.medusa_paged_attention_workspace_size(ctypes.byref(kv), 6, 4) == 0


@no_gpu
@pytest.mark.parametrize("over", [dict(layer=2), dict(layer=-1), dict(N=0), dict(N=7), dict(H=0), dict(q=None), dict(out=None),
                                  dict(qs=255), dict(ks=100), dict(vs=132), dict(rot=3), dict(rot=66), dict(layout=2),
                                  dict(turns=None), dict(amplitude=math.nan), dict(q=5 * P + 8), dict(out=5 * P + 512),
                                  dict(out=5 * P, qs=512), dict(out=6 * P), dict(starts=P + 1)], ids=str)
def test_c_rope_append(mb, over):
    assert rope_call(mb, **over) in (mb.MEDUSA_ERR_INVALID_ARG, mb.MEDUSA_ERR_UNSUPPORTED)


@no_gpu
def test_c_well_formed_calls_reach_the_device_check(mb, tree):
    assert rope_call(mb) == mb.MEDUSA_ERR_CUDA
    assert rope_call(mb, out=5 * P) == mb.MEDUSA_ERR_CUDA            # in place
    kv = c_kv(mb)
    assert mb._lib.medusa_paged_attention(ctypes.byref(kv), 0, 6, 4, 5 * P, 0.1, None, None, 6 * P, 7 * P, 1 << 40, None) == 3


@no_gpu
@pytest.mark.parametrize("over", [dict(H=3), dict(q=None), dict(ws=None), dict(out=5 * P), dict(scale=math.inf), dict(scale=-math.inf),
                                  dict(scale=math.nan), dict(scale=2.0 ** 65), dict(ws=7 * P + 16),
                                  dict(layer=9), dict(N=5)], ids=str)
def test_c_paged_attention(mb, over):
    a = dict(layer=0, N=6, H=4, q=5 * P, scale=0.1, out=6 * P, ws=7 * P)
    a.update(over)
    kv = c_kv(mb)
    assert mb._lib.medusa_paged_attention(ctypes.byref(kv), a["layer"], a["N"], a["H"], a["q"], a["scale"], None, None, a["out"],
                                          a["ws"], 1 << 40, None) == mb.MEDUSA_ERR_INVALID_ARG


@no_gpu
def test_c_accept_and_logits(mb, tree):
    kv = c_kv(mb)
    acc = lambda t, best=5 * P, n=6 * P, new=4 * P, ws=8 * P, size=256: mb._lib.medusa_paged_accept_kv(  # noqa: E731
        t, ctypes.byref(kv), best, n, new, ws, size, None)
    assert acc(None) == 1 and acc(tree.handle) == 1                  # no tree; a tree without device tables
    assert acc(tree.handle, new=4 * P + 4) == 1 and b"overlaps" in mb._lib.medusa_last_error()
    assert acc(tree.handle, new=5 * P) == 1 and b"overlaps" in mb._lib.medusa_last_error()
    assert acc(tree.handle, size=0) == 1 and b"too small" in mb._lib.medusa_last_error()
    r = mb.LogitRules()
    adj = lambda rules, B=2, V=50, z=5 * P, tok=6 * P, out=7 * P: mb._lib.medusa_adjust_logits(  # noqa: E731
        tree.handle, B, V, z, tok, ctypes.byref(rules), out, None)
    for kw in (dict(B=0), dict(B=65), dict(V=0), dict(V=2 ** 30 + 1), dict(z=None), dict(out=None)):
        assert adj(r, **kw) == 1
    assert adj(r) == 1 and b"without upload" in mb._lib.medusa_last_error()
    for fields, kw in ((dict(history=P), {}), (dict(history=P, history_lens=P), {}), (dict(prompt_lens=P), {}),
                       (dict(bias=P), {}), (dict(bias=P, bias_ids=P, n_bias=0), {}), (dict(bias=P, bias_ids=P, n_bias=1025), {}),
                       (dict(presence=P), dict(tok=None)), (dict(allowed=P + 1), {})):
        r = mb.LogitRules()
        for k, v in fields.items():
            setattr(r, k, v)
        assert adj(r, **kw) == 1 and b"without upload" not in mb._lib.medusa_last_error(), fields
