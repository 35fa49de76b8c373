"""The paged-cache calls without a GPU: what their sources must keep to, and refusals of the C ABI."""

import ctypes
import os
import re

import pytest

from test_paged_cpu import P, c_kv, no_gpu, rope_call

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_decoding_heads_b200", "csrc")


@pytest.fixture(scope="module")
def mb(built):
    import speculative_decoding_heads_b200 as mb
    return mb


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_a_warpgroup_moves_its_registers_in_one_place():
    """setmaxnreg must be the same instruction for all of a warpgroup's threads: each kernel that uses it has one
    branch per warpgroup range, and the instruction is the first thing in it."""
    used = 0
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith((".cu", ".cuh")):
            continue
        text = _source(name)
        moves = re.findall(r"setmaxnreg\.(dec|inc)", text)
        if not moves:
            continue
        used += 1
        shape = re.search(r"if \(warp < 4\) \{\s*asm volatile\(\"setmaxnreg\.dec\.sync\.aligned\.u32 (\d+);\"\);", text)
        rest = re.search(r"\n  \} else \{\s*asm volatile\(\"setmaxnreg\.inc\.sync\.aligned\.u32 (\d+);\"\);", text)
        assert moves == ["dec", "inc"] and shape and rest, name
        # the pool that the block was launched with: 384 threads of 168 registers
        assert 128 * int(shape[1]) + 256 * int(rest[1]) <= 384 * 168, name
    assert used == 1


@pytest.mark.parametrize("bad", [(-1, 0), (1025, 0), (0, -5)], ids=str)
def test_the_wait_hook_refuses(mb, bad):
    with pytest.raises(mb.MedusaError) as e:
        mb.medusa_test_paged_wait(*bad)
    assert e.value.code == mb.MEDUSA_ERR_INVALID_ARG
    mb.medusa_test_paged_wait(0, 0)


def test_every_wait_of_the_paged_kernels_is_bounded():
    """A spin on a barrier goes through mbar_wait and its limit."""
    for name in ("paged_attention_tc.cu", "paged_attention_few.cu"):
        text = _source(name)
        assert text.count("mbar_try_wait") == 1, name                   # the first try of wait(), then mbar_wait
        assert not re.search(r"while\s*\(\s*!|for\s*\(;;\)\s*;", text), name
        assert all("wait_limit" in m for m in re.findall(r"mbar_wait\([^;]*;", text)), name


# the made-up cache of test_paged_cpu: k_pages at P, v_pages at 2 P, 2 layers of 5 pages of 2 heads of 16 rows of 64 bf16
PAGES = 2 * 5 * 2 * 16 * 64 * 2


@no_gpu
@pytest.mark.parametrize("over", [dict(out=P), dict(out=2 * P + PAGES - 16), dict(out=P - 16), dict(q=P + 4096, out=P + 4096),
                                  dict(k=2 * P), dict(v=P + 256), dict(q=2 * P - 16)], ids=str)
def test_rope_append_refuses_tensors_in_the_pages(mb, over):
    assert rope_call(mb, **over) == mb.MEDUSA_ERR_INVALID_ARG
    assert b"the pages" in mb._lib.medusa_last_error()


@no_gpu
@pytest.mark.parametrize("out,refused", [(P, True), (2 * P + PAGES - 16, True), (2 * P - 6 * 4 * 64 * 2 + 16, True),
                                         (P + PAGES, False), (2 * P - 6 * 4 * 64 * 2, False)])
def test_paged_attention_refuses_an_output_in_the_pages(mb, out, refused):
    kv = c_kv(mb)
    got = mb._lib.medusa_paged_attention(ctypes.byref(kv), 0, 6, 4, 5 * P, 0.1, None, None, out, 7 * P, 1 << 40, None)
    if refused:
        assert got == mb.MEDUSA_ERR_INVALID_ARG and b"the pages" in mb._lib.medusa_last_error()
    else:
        assert got == mb.MEDUSA_ERR_CUDA             # well-formed: it gets as far as the missing device
