"""The tree-drafting operators' arguments at the ends of their ranges, without a GPU (addresses here are never
touched)."""
import os
import re

import pytest
import torch

import test_abi_host

pa = test_abi_host.pa  # the module fixture that builds and loads the library

INVALID, UNSUPPORTED, MISALIGNED = -1, -2, -3


# ------------------------------------------------------------------------------------------ the rows' grants

@pytest.mark.parametrize("granted,rc", [(0x1e0002, MISALIGNED), (0x100000, INVALID), (0x110004, INVALID), (0x160008, INVALID),
                                        (0x150010, INVALID), (0x190000, INVALID), (0x1a0008, INVALID)])
def test_plan_refuses_grants_over_other_arrays(pa, granted, rc):
    assert pa.lib.pa_plan_step_granted(0x100000, 0x110000, 0x120000, 0x130000, 0x140000, None, 0x150000, 0x160000, 0x170000,
                                       0x180000, 0x190000, 0x1a0000, 0x1b0000, None, granted, 4, 16, 10, 5, 64, None, None) == rc


def test_tree_and_compact_refuse_misplaced_grants(pa):
    args = (0x100000, 0x200000, 0x300000, 0x400000, 0x410000, 0x420000, 0x430000, 0x440002, 0x500000, None, 2, 16, 8, 8, 2, 128, 16,
            10, 5, 80, 0.1)
    rest = (0, 0, 0x700000, 1 << 30, None)
    assert pa.lib.pa_tree_gqa_granted(*args, *rest) == MISALIGNED
    assert pa.lib.pa_tree_gqa_fp8_granted(*args, 0.5, 0.5, *rest) == MISALIGNED
    assert pa.lib.pa_tree_gqa_nvfp4_granted(*args, 0.5, 0.5, *rest) == MISALIGNED
    for granted, rc in ((0x360002, MISALIGNED), (0x350000, INVALID), (0x350004, INVALID)):
        assert pa.lib.pa_kv_compact_granted(0x100000, 0x200000, 0x300000, 0x310000, 0x320000, 0x330000, 0x340000, granted,
                                            0x350000, 1, 4, 5, 256, 16, 8, 5, None, None) == rc


def test_binding_refuses_grants(pa):
    z = lambda *s, d=torch.int32: torch.zeros(*s, dtype=d)  # noqa: E731
    bf, i64 = torch.bfloat16, torch.int64
    q, pool = z(6, 4, 64, d=bf), z(3, 8, 2, 64, d=bf)
    for bad in (z(3), z(2, d=i64), z(4)[::2]):
        with pytest.raises(pa.PaError, match="granted"):
            pa.pa_plan_step(z(2), z(2), z(2), z(9), z(1), z(2, 3), z(3), z(7, d=i64), z(7), page_size=16, granted=bad)
        with pytest.raises(pa.PaError, match="granted"):
            pa.pa_tree_gqa(q, pool, pool, z(2, 3), z(2), z(3), z(6, d=i64), q, max_query=3, scale=1.0,
                           workspace=z(1 << 20, d=torch.uint8), granted=bad)
        with pytest.raises(pa.PaError, match="granted"):
            pa.pa_kv_compact(pool, pool, z(2, 3), z(2), z(3), z(2, 4), z(2), granted=bad, context_lens_out=z(2))


# ------------------------------------------------------------------------------------------ waits that give up

def _tree_kernel_source():
    with open(os.path.join(test_abi_host.ROOT, "paged_kv_attention_19_gb300", "csrc", "pa_tree.cuh")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    return text[text.index("tree_split_kernel("):text.index("tree_combine_kernel(")]


def test_waits_of_a_whole_warp_have_one_answer():
    """In the tree attention's kernel a wait that a thread ends for itself (mbar_wait) stands only in the branch of the elected
    issuing thread, which has no instruction in common with its warp's other lanes until its end; all others are the whole
    warp's, with the same answer in every lane.  (Lanes that disagree wait for one another without a limit: nothing to run.)"""
    text = _tree_kernel_source()
    a = text.index("if (elect_one()) {")
    depth, b = 0, text.index("{", a)
    while True:  # the branch's end
        depth += {"{": 1, "}": -1}.get(text[b], 0)
        b += 1
        if depth == 0:
            break
    alone, rest = text[a:b], text[:a] + text[b:]
    assert re.search(r"\bmbar_wait\(", alone) and not re.search(r"\bmbar_(try_)?wait(_lane)?\(|\bmbar_test\(", rest)
    assert not re.search(r"__syncwarp|_sync\(|warp_wait\(", alone)
    assert len(re.findall(r"\bwarp_wait\(", rest)) >= 10
    # an answer is looked at, but for copies that are only waited out before the end
    for line in rest.splitlines():
        if re.match(r"\s*warp_wait\(", line):
            assert re.search(r"(raw_full|full|q_full)\b", line), line


# ------------------------------------------------------------------------------------------ lengths

@pytest.mark.parametrize("fmt", ["", "_fp8", "_nvfp4"])
def test_tree_refuses_contexts_whose_last_tile_ends_past_31_bits(pa, fmt):
    scales = [0.5, 0.5] if fmt else []

    def call(longest, batch):
        return getattr(pa.lib, "pa_tree_gqa" + fmt)(
            0x100000, 0x200000, 0x300000, 0x400000, 0x410000, 0x420000, 0x430000, 0x500000, None, batch, 16, 8, 8, 2, 128, 256,
            10, 1 << 23, longest, 0.1, *scales, 0, 0, 0x700000, 1 << 30, None)

    for longest in (2 ** 31 - 1, 2 ** 31 - 63, 2 ** 31 - 128):
        assert call(longest, 2) == UNSUPPORTED
        assert pa.pa_tree_workspace_size(2, 8, 8, 2, 128, longest, 256) == 0
    assert call(2 ** 31 - 129, 0) == 0
    assert pa.pa_tree_workspace_size(2, 8, 8, 2, 128, 2 ** 31 - 129, 256) > 0
