"""Refusals of the streams' operators: every check that the host can make, made before any CUDA call (addresses here are never
touched)."""
import os
import re
import subprocess

import pytest
import torch

import stream_refs as S
import test_abi_host

pa = test_abi_host.pa  # the module fixture that builds and loads the library

INVALID, UNSUPPORTED, MISALIGNED, SMALL = -1, -2, -3, -4


def stream(pa, fmt="", **kw):
    a = dict(q=0x100000, k=0x200000, v=0x300000, bt=0x400000, lens=0x410000, qs=0x420000, granted=None, out=0x500000, lse=None,
             batch=2, T=16, mq=8, hq=8, hkv=2, D=128, p=16, pages=10, maxp=5, maxctx=80, scale=0.1, ksc=0.5, vsc=0.5, window=0,
             first=0, splits=0, ws=0x700000, wsb=1 << 30)
    a.update(kw)
    scales = [a["ksc"], a["vsc"]] if fmt else []
    return getattr(pa.lib, "pa_stream_gqa" + fmt)(
        a["q"], a["k"], a["v"], a["bt"], a["lens"], a["qs"], a["granted"], a["out"], a["lse"], a["batch"], a["T"], a["mq"],
        a["hq"], a["hkv"], a["D"], a["p"], a["pages"], a["maxp"], a["maxctx"], a["scale"], *scales, a["window"], a["first"],
        a["splits"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("fmt", ["", "_fp8", "_nvfp4"])
@pytest.mark.parametrize("kw,rc", [
    (dict(batch=0), 0), (dict(T=0), 0), (dict(batch=0, window=-5, first=3), 0), (dict(T=0, mq=1 << 30, hq=256), 0),
    (dict(batch=-1), INVALID), (dict(T=-1), INVALID), (dict(mq=0), INVALID), (dict(mq=-1), INVALID),
    (dict(mq=(1 << 30) + 1), UNSUPPORTED), (dict(hq=0), INVALID), (dict(hkv=0), INVALID), (dict(hkv=3), INVALID),
    (dict(hq=258), UNSUPPORTED), (dict(D=96), UNSUPPORTED), (dict(D=512), UNSUPPORTED), (dict(p=48), UNSUPPORTED),
    (dict(p=4), UNSUPPORTED), (dict(p=512), UNSUPPORTED), (dict(pages=0), INVALID), (dict(maxp=0), INVALID),
    (dict(maxctx=81), INVALID), (dict(maxctx=-1), INVALID), (dict(maxctx=2 ** 31 - 512, maxp=2 ** 27), UNSUPPORTED),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(splits=-1), INVALID),
    (dict(splits=4097), UNSUPPORTED), (dict(first=-1), INVALID), (dict(first=-1, window=9), INVALID), (dict(q=None), INVALID),
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(bt=None), INVALID), (dict(lens=None), INVALID), (dict(qs=None), INVALID),
    (dict(out=None), INVALID), (dict(ws=None), INVALID), (dict(q=0x100008), MISALIGNED), (dict(out=0x500008), MISALIGNED),
    (dict(lse=0x600002), MISALIGNED), (dict(granted=0x600002), MISALIGNED), (dict(qs=0x420002), MISALIGNED),
    (dict(ws=0x700008), MISALIGNED), (dict(wsb=64), SMALL)])
def test_stream_refuses(pa, fmt, kw, rc):
    assert stream(pa, fmt, **kw) == rc


def test_stream_refuses_scales_and_sizes(pa):
    for fmt in ("_fp8", "_nvfp4"):
        for bad in (0.0, -1.0, float("inf"), float("nan")):
            assert stream(pa, fmt, ksc=bad) == INVALID and stream(pa, fmt, vsc=bad) == INVALID
        assert stream(pa, fmt, scale=1e30, ksc=1e20) == INVALID and stream(pa, fmt, scale=1e30, ksc=1.0, T=0) == 0
    assert stream(pa, scale=3e38) == INVALID and stream(pa, scale=-3e38) == INVALID
    ws = pa.pa_stream_workspace_size
    assert ws(4, 8, 8, 2, 128, 1000, 16) >= 256 and ws(4, 100000, 8, 2, 128, 1000, 16) >= 256
    for bad in (dict(max_query=0), dict(max_query=(1 << 30) + 1), dict(num_kv_heads=3), dict(num_q_heads=258), dict(head_dim=96),
                dict(page_size=48), dict(num_splits=-1), dict(num_splits=5000), dict(max_context_len=2 ** 31 - 1)):
        a = dict(batch=4, max_query=8, num_q_heads=8, num_kv_heads=2, head_dim=128, max_context_len=1000, page_size=16)
        assert ws(**{**a, **bad}) == 0


def release(pa, **kw):
    a = dict(lens=0x100000, held=0x110000, ws=0x120000, ended=None, fl=0x130000, fc=0x140000, bt=0x150000, lo=0x160000, ho=0x170000,
             wo=0x180000, co=0x190000, bo=0x1a0000, batch=4, p=16, pages=10, maxp=5, window=32, first=4, status=None)
    a.update(kw)
    return pa.lib.pa_release_pages(a["lens"], a["held"], a["ws"], a["ended"], a["fl"], a["fc"], a["bt"], a["lo"], a["ho"], a["wo"],
                                   a["co"], a["bo"], a["batch"], a["p"], a["pages"], a["maxp"], a["window"], a["first"], a["status"],
                                   None)


@pytest.mark.parametrize("kw,rc", [
    (dict(batch=-1), INVALID), (dict(p=0), INVALID), (dict(pages=0), INVALID), (dict(maxp=0), INVALID), (dict(window=0), INVALID),
    (dict(window=-1), INVALID), (dict(first=-1), INVALID), (dict(batch=8193), UNSUPPORTED), (dict(maxp=1 << 20, p=1 << 12), UNSUPPORTED),
    (dict(maxp=1 << 20, batch=4096), UNSUPPORTED),
    (dict(lens=None), INVALID), (dict(held=None), INVALID), (dict(ws=None), INVALID), (dict(fl=None), INVALID), (dict(fc=None), INVALID),
    (dict(bt=None), INVALID), (dict(lo=None), INVALID), (dict(ho=None), INVALID), (dict(wo=None), INVALID), (dict(co=None), INVALID),
    (dict(bo=None), INVALID), (dict(lens=0x100002), MISALIGNED), (dict(ended=0x1b0001), MISALIGNED), (dict(status=0x1b0002), MISALIGNED),
    # an output over an input that is not its own, or over another output
    (dict(lo=0x110000), INVALID), (dict(lo=0x100004), INVALID), (dict(ho=0x100000), INVALID), (dict(wo=0x110000), INVALID),
    (dict(bo=0x150010), INVALID), (dict(bo=0x120000), INVALID), (dict(co=0x130004), INVALID), (dict(fl=0x150000), INVALID),
    (dict(ended=0x160000), INVALID), (dict(ended=0x130008), INVALID), (dict(status=0x190000), INVALID), (dict(wo=0x160000), INVALID)])
def test_release_refuses(pa, kw, rc):
    assert release(pa, **kw) == rc


def test_binding_refuses_tensors(pa):
    """Types, shapes, strides and devices are checked before anything is called."""
    z = lambda *s, d=torch.int32: torch.zeros(*s, dtype=d)  # noqa: E731
    bf = torch.bfloat16
    good = dict(q=z(6, 4, 64, d=bf), k_pool=z(3, 8, 2, 64, d=bf), v_pool=z(3, 8, 2, 64, d=bf), block_table=z(2, 3),
                context_lens=z(2), query_start=z(3), out=z(6, 4, 64, d=bf))
    ws = z(1 << 20, d=torch.uint8)

    def call(**kw):
        with pytest.raises(pa.PaError) as e:
            pa.pa_stream_gqa(**{**good, **kw}, max_query=3, scale=1.0, workspace=ws)
        assert e.value.status == pa.PA_ERR_INVALID_ARGUMENT
        return str(e.value)

    assert "not on a GPU" in call()
    assert "out" in call(out=z(6, 4, 64, d=torch.float16))
    assert "block_table" in call(block_table=z(2, 3, d=torch.int64))
    assert "query_start" in call(query_start=z(2))
    assert "granted" in call(granted=z(3))
    assert "v_pool" in call(v_pool=z(3, 8, 2, 32, d=bf))
    assert "q has" in call(q=z(6, 4, 128, d=bf)[:, :, ::2])
    assert "lse" in call(lse=z(6, 4, d=torch.float64))
    assert "first" in call(first=2 ** 31)
    with pytest.raises(pa.PaError, match="k_pool"):
        pa.pa_stream_gqa_nvfp4(**good, max_query=3, scale=1.0, k_scale=1.0, v_scale=1.0, workspace=ws)
    r = dict(context_lens=z(2), held_pages=z(2), window_start=z(2), free_list=z(9), free_count=z(1), block_table=z(2, 3))

    def give(**kw):
        with pytest.raises(pa.PaError) as e:
            pa.pa_release_pages(**{**r, **kw}, page_size=16, window=32)
        return str(e.value)

    assert "not on a GPU" in give()
    assert "held_pages has" in give(held_pages=z(3))
    assert "window_start has" in give(window_start=z(2, d=torch.int64))
    assert "free_count has" in give(free_count=z(2))
    assert "block_table_out" in give(block_table_out=z(2, 4))
    assert "ended" in give(ended=z(2, d=torch.bool))


def test_reference_of_the_release():
    """The plain release against a case done by hand: pages of 4 tokens, a window of 6, one token kept."""
    table = torch.tensor([[7, 3, 5, 9, -1], [1, -1, 2, 4, 0]]).numpy()
    got = S.release([13, 15], [4, 5], [0, 2], [8, 0, 0, 0, 0, 0, 0, 0, 0, 0], 1, table, 4, 10, 6, 1)
    # row 0: position 13 sees from 8 on, so page 1 goes; row 1: from 10 on, pages 0 and 1 lie behind, page 1 is gone
    assert got["table"].tolist() == [[7, -1, 5, 9, -1], [1, -1, 2, 4, 0]] and got["count"] == 2
    assert got["free_list"][:2].tolist() == [8, 3] and got["start"] == [2, 2] and got["bits"] == 0
    got = S.release([13, 15], [4, 5], [2, 2], [8] + [0] * 9, 1, got["table"], 4, 10, 6, 1, [0, 1])
    assert got["free_list"][:5].tolist() == [8, 1, 2, 4, 0] and got["lens"] == [13, 0] and got["held"] == [4, 0]


@pytest.mark.parametrize("threads,places,compiles", [(640, 20, True), (640, 16, False), (512, 16, True), (256, 7, False)])
def test_scan_has_a_place_for_each_warp(pa, tmp_path, threads, places, compiles):
    """A block of more warps than its array of partial sums has places is no program: the streams' kernels over codes have 20."""
    from paged_kv_attention_19_gb300 import build
    src = tmp_path / "scan.cu"
    src.write_text("#include \"pa_tree.cuh\"\n__global__ void f(long long *x) {\n  __shared__ long long part[%d];\n  long long before;\n"
                   "  *x = pa::tree_scan<%d>(1, &before, part);\n}\n" % (places, threads))
    r = subprocess.run([build.nvcc(), *build.ARCH, *build.NVCC_FLAGS, "-c", str(src), "-o", str(tmp_path / "scan.o")],
                       capture_output=True, text=True)
    assert (r.returncode == 0) == compiles, r.stderr
    assert compiles or "a place for each warp" in r.stderr


def kernel_source(name):
    return open(os.path.join(test_abi_host.ROOT, "paged_kv_attention_19_gb300", "csrc", name)).read()


@pytest.mark.parametrize("name", ["pa_stream.cuh", "pa_tree.cuh"])
def test_scores_wait_for_the_products_of_their_buffer(name):
    """The scores of an item are written over the weights of an earlier one, which its product reads from tensor memory.  Products
    with different accumulators are in no order of their own, so in every form of the kernel the wait stands before the scores."""
    text = kernel_source(name)
    begin = text[text.index("auto begin ="):]
    begin = begin[:begin.index("tc_mma_ss(")]
    waits = re.findall(r"if \(([^;]*?mbar_wait\(&pv_done\[b\], par\(c - (?:C::)?BACK\), status\))\) return false;", begin)
    assert len(waits) == 1
    condition = waits[0].split("!mbar_wait")[0]
    assert re.fullmatch(r"c >= (\(uint32_t\))?(C::)?BACK && ", condition), condition


def test_tensor_memory_loads_carry_their_wait():
    """A load's registers hold nothing before its wait, and to the compiler they are ready behind the statement: so the wait is in it."""
    loads = 0
    for path in sorted(os.listdir(os.path.join(test_abi_host.ROOT, "paged_kv_attention_19_gb300", "csrc"))):
        for statement in re.findall(r"\basm\b[^;(]*\((?:[^;\"]|\"[^\"]*\")*;", kernel_source(path)):
            if "tcgen05.ld." in statement:
                loads += 1
                assert statement.rfind("tcgen05.wait::ld.sync.aligned;") > statement.rfind("tcgen05.ld."), (path, statement[:90])
    assert loads >= 4
