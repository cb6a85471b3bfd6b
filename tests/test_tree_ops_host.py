"""Refusals of the tree-drafting operators: every check that the host can make, made before any CUDA call
(addresses here are never touched)."""
import pytest
import torch

import test_abi_host

pa = test_abi_host.pa  # the module fixture that builds and loads the library

INVALID, UNSUPPORTED, MISALIGNED, SMALL = -1, -2, -3, -4


def plan(pa, **kw):
    a = dict(lens=0x100000, news=0x110000, held=0x120000, fl=0x130000, fc=0x140000, par=None, bt=0x150000, lo=0x160000,
             ho=0x170000, co=0x180000, qs=0x190000, slots=0x1a0000, pos=0x1b0000, mask=None, batch=4, p=16, pages=10,
             maxp=5, tokens=64, status=None)
    a.update(kw)
    return pa.lib.pa_plan_step(a["lens"], a["news"], a["held"], a["fl"], a["fc"], a["par"], a["bt"], a["lo"], a["ho"],
                               a["co"], a["qs"], a["slots"], a["pos"], a["mask"], a["batch"], a["p"], a["pages"],
                               a["maxp"], a["tokens"], a["status"], None)


@pytest.mark.parametrize("kw,rc", [
    (dict(batch=-1), INVALID), (dict(p=0), INVALID), (dict(pages=0), INVALID), (dict(maxp=0), INVALID),
    (dict(tokens=-1), INVALID), (dict(batch=8193), UNSUPPORTED), (dict(maxp=1 << 20, p=1 << 12), UNSUPPORTED),
    (dict(lens=None), INVALID), (dict(news=None), INVALID), (dict(held=None), INVALID), (dict(fl=None), INVALID),
    (dict(fc=None), INVALID), (dict(bt=None), INVALID), (dict(lo=None), INVALID), (dict(ho=None), INVALID),
    (dict(co=None), INVALID), (dict(qs=None), INVALID), (dict(slots=None), INVALID), (dict(pos=None), INVALID),
    (dict(par=0x1c0000), INVALID), (dict(mask=0x1c0000), INVALID), (dict(lens=0x100002), MISALIGNED),
    (dict(slots=0x1a0004), MISALIGNED), (dict(status=0x1d0001), MISALIGNED),
    (dict(par=0x1c0000, mask=0x1d0004), MISALIGNED),
    # an output over an input that is not its own, or over another output
    (dict(lo=0x110000), INVALID), (dict(lo=0x100004), INVALID), (dict(ho=0x100000), INVALID), (dict(qs=0x150010), INVALID),
    (dict(pos=0x1a0000), INVALID), (dict(co=0x130004), INVALID), (dict(fl=0x150000), INVALID), (dict(status=0x190004), INVALID)])
def test_plan_refuses(pa, kw, rc):
    assert plan(pa, **kw) == rc


def rope(pa, fmt="", **kw):
    a = dict(q=0x100000, k=0x200000, v=0x300000, wq=0x400000, wk=0x410000, cs=0x420000, pos=0x430000, slots=0x440000,
             qo=0x500000, kp=0x600000, vp=0x700000, T=4, hq=8, hkv=2, D=128, qs=1024, ks=256, vs=256, rot=128, il=0,
             far=100, eps=1e-6, ksc=0.5, vsc=0.5, p=16, pages=8, status=None)
    a.update(kw)
    scales = [a["ksc"], a["vsc"]] if fmt else []
    return getattr(pa.lib, "pa_qk_norm_rope_write" + fmt)(
        a["q"], a["k"], a["v"], a["wq"], a["wk"], a["cs"], a["pos"], a["slots"], a["qo"], a["kp"], a["vp"], a["T"],
        a["hq"], a["hkv"], a["D"], a["qs"], a["ks"], a["vs"], a["rot"], a["il"], a["far"], a["eps"], *scales, a["p"],
        a["pages"], a["status"], None)


@pytest.mark.parametrize("fmt", ["", "_fp8", "_nvfp4"])
@pytest.mark.parametrize("kw,rc", [
    (dict(T=0), 0), (dict(T=-1), INVALID), (dict(hq=0), INVALID), (dict(hkv=0), INVALID), (dict(D=96), UNSUPPORTED),
    (dict(D=512), UNSUPPORTED), (dict(rot=0), INVALID), (dict(rot=256), INVALID), (dict(rot=24), UNSUPPORTED),
    (dict(far=0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=-1.0), INVALID), (dict(p=0), INVALID),
    (dict(pages=0), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(cs=None), INVALID), (dict(pos=None), INVALID), (dict(slots=None), INVALID), (dict(qo=None), INVALID),
    (dict(kp=None), INVALID), (dict(vp=None), INVALID), (dict(qs=1016), INVALID), (dict(ks=128), INVALID),
    (dict(qs=1028), MISALIGNED), (dict(q=0x100008), MISALIGNED), (dict(wq=0x400008), MISALIGNED),
    (dict(cs=0x420004), MISALIGNED), (dict(slots=0x440004), MISALIGNED), (dict(kp=0x600008), MISALIGNED),
    (dict(qo=0x100010), INVALID), (dict(qo=0x100000, qs=2048), INVALID), (dict(qo=0x200000), INVALID),
    (dict(vp=0x600010), INVALID), (dict(kp=0x300000), INVALID), (dict(vp=0x500000), INVALID),
    (dict(qo=0x420010), INVALID), (dict(cs=0x500000), INVALID), (dict(pos=0x600000), INVALID), (dict(slots=0x700008), INVALID),
    (dict(wq=0x500010), INVALID), (dict(wk=0x600010), INVALID), (dict(status=0x500004), INVALID)])
def test_rope_write_refuses(pa, fmt, kw, rc):
    assert rope(pa, fmt, **kw) == rc


@pytest.mark.parametrize("bad", [0.0, -1.0, float("inf"), float("nan")])
def test_rope_write_refuses_scales(pa, bad):
    for fmt in ("_fp8", "_nvfp4"):
        assert rope(pa, fmt, ksc=bad) == INVALID and rope(pa, fmt, vsc=bad) == INVALID


@pytest.mark.parametrize("bad", [1e-40, 1e-38, 2.0 ** -51, 2.0 ** 51, 3e38])
def test_rope_write_refuses_scales_out_of_range(pa, bad):
    for fmt in ("_fp8", "_nvfp4"):
        assert rope(pa, fmt, ksc=bad) == UNSUPPORTED and rope(pa, fmt, vsc=bad) == UNSUPPORTED
        assert rope(pa, fmt, T=0, ksc=2.0 ** -50, vsc=2.0 ** 50) == 0


def tree(pa, fmt="", **kw):
    a = dict(q=0x100000, k=0x200000, v=0x300000, bt=0x400000, lens=0x410000, qs=0x420000, mask=0x430000, out=0x500000,
             lse=None, batch=2, T=16, mq=8, hq=8, hkv=2, D=128, p=16, pages=10, maxp=5, maxctx=80, scale=0.1, ksc=0.5,
             vsc=0.5, window=0, splits=0, ws=0x700000, wsb=1 << 30)
    a.update(kw)
    scales = [a["ksc"], a["vsc"]] if fmt else []
    return getattr(pa.lib, "pa_tree_gqa" + fmt)(
        a["q"], a["k"], a["v"], a["bt"], a["lens"], a["qs"], a["mask"], a["out"], a["lse"], a["batch"], a["T"], a["mq"],
        a["hq"], a["hkv"], a["D"], a["p"], a["pages"], a["maxp"], a["maxctx"], a["scale"], *scales, a["window"],
        a["splits"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("fmt", ["", "_fp8", "_nvfp4"])
@pytest.mark.parametrize("kw,rc", [
    (dict(batch=0), 0), (dict(T=0), 0), (dict(batch=-1), INVALID), (dict(T=-1), INVALID), (dict(mq=0), INVALID),
    (dict(mq=65), UNSUPPORTED), (dict(hq=0), INVALID), (dict(hkv=3), INVALID), (dict(D=96), UNSUPPORTED),
    (dict(p=48), UNSUPPORTED), (dict(p=4), UNSUPPORTED), (dict(p=512), UNSUPPORTED), (dict(pages=0), INVALID),
    (dict(maxp=0), INVALID), (dict(maxctx=81), INVALID), (dict(maxctx=-1), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(splits=-1), INVALID), (dict(splits=4097), UNSUPPORTED), (dict(q=None), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(bt=None), INVALID), (dict(lens=None), INVALID), (dict(qs=None), INVALID),
    (dict(mask=None), INVALID), (dict(out=None), INVALID), (dict(ws=None), INVALID), (dict(q=0x100008), MISALIGNED),
    (dict(mask=0x430004), MISALIGNED), (dict(lse=0x600002), MISALIGNED), (dict(ws=0x700008), MISALIGNED),
    (dict(wsb=64), SMALL)])
def test_tree_refuses(pa, fmt, kw, rc):
    assert tree(pa, fmt, **kw) == rc


def test_tree_refuses_scales_and_sizes(pa):
    for fmt in ("_fp8", "_nvfp4"):
        for bad in (0.0, -1.0, float("inf"), float("nan")):
            assert tree(pa, fmt, ksc=bad) == INVALID and tree(pa, fmt, vsc=bad) == INVALID
    ws = pa.pa_tree_workspace_size
    assert ws(4, 8, 8, 2, 128, 1000, 16) >= 256
    for bad in (dict(max_query=65), dict(max_query=0), dict(num_kv_heads=3), dict(head_dim=96), dict(page_size=48)):
        a = dict(batch=4, max_query=8, num_q_heads=8, num_kv_heads=2, head_dim=128, max_context_len=1000, page_size=16)
        assert ws(**{**a, **bad}) == 0


def compact(pa, **kw):
    a = dict(k=0x100000, v=0x200000, bt=0x300000, lens=0x310000, qs=0x320000, acc=0x330000, num=0x340000, lo=0x350000,
             layers=1, batch=4, ma=5, tb=256, p=16, pages=8, maxp=5, status=None)
    a.update(kw)
    return pa.lib.pa_kv_compact(a["k"], a["v"], a["bt"], a["lens"], a["qs"], a["acc"], a["num"], a["lo"], a["layers"],
                                a["batch"], a["ma"], a["tb"], a["p"], a["pages"], a["maxp"], a["status"], None)


@pytest.mark.parametrize("kw,rc", [
    (dict(batch=0), 0), (dict(batch=-1), INVALID), (dict(layers=0), INVALID), (dict(ma=0), INVALID), (dict(tb=0), INVALID),
    (dict(p=0), INVALID), (dict(pages=0), INVALID), (dict(maxp=0), INVALID), (dict(tb=24), UNSUPPORTED),
    (dict(ma=65), UNSUPPORTED), (dict(batch=65536), UNSUPPORTED), (dict(maxp=1 << 20, p=1 << 12), UNSUPPORTED),
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(bt=None), INVALID), (dict(lens=None), INVALID),
    (dict(qs=None), INVALID), (dict(acc=None), INVALID), (dict(num=None), INVALID), (dict(lo=None), INVALID),
    (dict(k=0x100008), MISALIGNED), (dict(acc=0x330002), MISALIGNED), (dict(lo=0x310000), INVALID),
    (dict(lo=0x310004), INVALID), (dict(lo=0x320008), INVALID), (dict(v=0x100100), INVALID)])
def test_compact_refuses(pa, kw, rc):
    assert compact(pa, **kw) == rc


def test_binding_refuses_tensors(pa):
    """Types, shapes, strides and devices are checked before anything is called."""
    z = lambda *s, d=torch.int32: torch.zeros(*s, dtype=d)  # noqa: E731
    bf = torch.bfloat16
    good = dict(q=z(6, 4, 64, d=bf), k_pool=z(3, 8, 2, 64, d=bf), v_pool=z(3, 8, 2, 64, d=bf), block_table=z(2, 3),
                context_lens=z(2), query_start=z(3), tree_mask=z(6, d=torch.int64), out=z(6, 4, 64, d=bf))
    ws = z(1 << 20, d=torch.uint8)

    def call(**kw):
        with pytest.raises(pa.PaError) as e:
            pa.pa_tree_gqa(**{**good, **kw}, max_query=3, scale=1.0, workspace=ws)
        assert e.value.status == pa.PA_ERR_INVALID_ARGUMENT
        return str(e.value)

    assert "not on a GPU" in call()
    assert "out" in call(out=z(6, 4, 64, d=torch.float16))
    assert "block_table" in call(block_table=z(2, 3, d=torch.int64))
    assert "query_start" in call(query_start=z(2))
    assert "tree_mask" in call(tree_mask=z(12, d=torch.int64)[::2])
    assert "v_pool" in call(v_pool=z(3, 8, 2, 32, d=bf))
    assert "q has" in call(q=z(6, 4, 128, d=bf)[:, :, ::2])
    assert "lse" in call(lse=z(6, 4, d=torch.float64))
    q = z(5, 4, 64, d=bf)
    with pytest.raises(pa.PaError, match="k has to be"):
        pa.pa_qk_norm_rope_write(q, z(5, 2, 128, d=bf)[..., ::2], z(5, 2, 64, d=bf), None, None, z(9, 64, d=torch.float32),
                                 z(5), z(5, d=torch.int64), z(5, 4, 64, d=bf), good["k_pool"], good["v_pool"])
    with pytest.raises(pa.PaError, match="cos_sin"):
        pa.pa_qk_norm_rope_write(q, z(5, 2, 64, d=bf), z(5, 2, 64, d=bf), None, None, z(9, 64, d=torch.float64),
                                 z(5), z(5, d=torch.int64), z(5, 4, 64, d=bf), good["k_pool"], good["v_pool"])
    with pytest.raises(pa.PaError, match="slot_mapping"):
        pa.pa_plan_step(z(2), z(2), z(2), z(9), z(1), z(2, 3), z(3), z(7), z(7), page_size=16)
    with pytest.raises(pa.PaError, match="accepted"):
        pa.pa_kv_compact(good["k_pool"], good["v_pool"], z(2, 3), z(2), z(3), z(2, 4, d=torch.int64), z(2),
                         context_lens_out=z(2))
