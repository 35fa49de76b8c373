"""The paged-cache calls without a GPU: what their sources must keep to, and refusals of the C ABI."""

import os
import re

import pytest

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
