"""Refusals of the attention calls, in the C ABI and in the Python binding: everything
here is rejected (or empty) on the host, before any HIP call."""
import ctypes
import os
import subprocess

import pytest
import torch

from conftest import ROOT
from fp4_block_scaled_x16_amd import api, attention
from test_abi import _err, lib  # noqa: F401 (lib: fixture)

FAKE, ODD = 0x10000, 0x10008
ARG, SHAPE, UNSUPPORTED = 1, 2, 3


def heads(**kw):
    return api.Heads(**dict(dict(x=FAKE, token_stride=1024, head_stride=128, heads=8), **kw))


def norm(**kw):
    return api.QKNormDesc(**dict(dict(q_weight=FAKE, k_weight=FAKE, weight_f32=0, eps=1e-6, table=FAKE, table_rows=64,
                                      rotary_dim=128, interleaved=0), **kw))


def cache(**kw):
    return api.KVCacheDesc(**dict(dict(
        format=api.MXFP8, heads=8, head_dim=128, page_size=16, pages=4, k_codes=FAKE, k_scales=FAKE, v_codes=FAKE,
        v_scales=FAKE, page_stride=16 * 8 * 128, head_stride=16 * 128, token_stride=128, scale_page_stride=16 * 8 * 4,
        scale_head_stride=64, scale_block_stride=16, amax=FAKE, target=448.0), **kw))


def by(s):
    return None if s is None else ctypes.byref(s)


def rope(lib, n=norm(), q=heads(), k=heads(), pos=FAKE, tokens=4, d=128, qo=heads(), ko=heads()):
    return lib.fp4_qk_norm_rope(by(n), by(q), by(k), pos, tokens, d, by(qo), by(ko), None)


def back(lib, n=norm(), q=heads(), k=heads(), pos=FAKE, tokens=4, d=128, dq=heads(), dk=heads(), qi=heads(), ki=heads(),
         wq=FAKE, wk=FAKE, ws=FAKE, size=1 << 30):
    return lib.fp4_qk_norm_rope_backward(by(n), by(q), by(k), pos, tokens, d, by(dq), by(dk), by(qi), by(ki), wq, wk, 0, ws,
                                         size, None)


def write(lib, c=cache(), k=heads(), v=heads(), slots=FAKE, tokens=4, n=None, pos=None, q=None, qo=None):
    return lib.fp4_kv_cache_write(by(c), by(k), by(v), slots, tokens, by(n), pos, by(q), by(qo), None)


def read(lib, c=cache(), slots=FAKE, n=4, k=FAKE, v=FAKE):
    return lib.fp4_kv_cache_read(by(c), slots, n, k, v, 0, None)


def decode(lib, c=cache(), q=heads(heads=16, token_stride=2048), table=FAKE, stride=4, width=4, lens=FAKE, n=3,
           scale=0.1, out=FAKE, out_type=1, lse=None, ws=None, size=0):
    return lib.fp4_attention_decode(by(c), by(q), table, stride, width, lens, n, scale, out, out_type, lse, ws, size, None)


BAD_HEADS = [(dict(heads=0), SHAPE), (dict(heads=-1), SHAPE), (dict(heads=1025), SHAPE), (dict(x=None), ARG), (dict(x=ODD), ARG),
             (dict(token_stride=-8), ARG), (dict(head_stride=132), ARG), (dict(token_stride=1028), ARG)]


@pytest.mark.parametrize("kw,status", BAD_HEADS)
def test_heads_are_rejected(lib, kw, status):
    bad = heads(**kw)
    assert rope(lib, q=bad) == status and _err(lib)
    assert rope(lib, ko=bad) == status
    assert back(lib, dk=bad) == status and back(lib, qi=bad) == status
    assert write(lib, k=bad) == status and write(lib, v=bad) == status
    assert decode(lib, q=bad) == status


def test_outputs_whose_rows_overlap(lib):
    for kw in (dict(head_stride=64), dict(token_stride=1016), dict(token_stride=0), dict(head_stride=0),
               dict(head_stride=504, token_stride=128)):
        assert rope(lib, qo=heads(**kw)) == ARG, kw
        assert back(lib, ki=heads(**kw)) == ARG, kw
        assert write(lib, n=norm(), pos=FAKE, q=heads(), qo=heads(**kw)) == ARG, kw
    # a single token's, and heads outermost: fine as far as they go (no tokens: nothing to run)
    assert rope(lib, tokens=0, qo=heads(token_stride=0)) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(q_weight=None), ARG), (dict(k_weight=None), ARG), (dict(q_weight=None, k_weight=None, table=None), ARG),
    (dict(q_weight=ODD), ARG), (dict(k_weight=ODD), ARG), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG),
    (dict(eps=float("inf")), ARG), (dict(table=ODD), ARG), (dict(rotary_dim=0), SHAPE), (dict(rotary_dim=24), SHAPE),
    (dict(rotary_dim=144), SHAPE), (dict(rotary_dim=-16), SHAPE), (dict(table_rows=0), SHAPE)])
def test_norms_are_rejected(lib, kw, status):
    bad = norm(**kw)
    assert rope(lib, n=bad) == status and _err(lib)
    assert back(lib, n=bad) == status
    assert write(lib, n=bad, pos=FAKE, q=heads(), qo=heads()) == status


def test_norm_calls_are_rejected(lib):
    assert rope(lib, n=None) == ARG and rope(lib, pos=None) == ARG
    assert rope(lib, d=96) == UNSUPPORTED and rope(lib, d=512) == UNSUPPORTED
    assert rope(lib, tokens=-1) == SHAPE and rope(lib, tokens=1 << 31) == SHAPE
    assert rope(lib, q=None) == ARG and rope(lib, qo=None) == ARG
    assert rope(lib, q=None, qo=None, k=None, ko=None) == ARG
    assert rope(lib, qo=heads(heads=4)) == SHAPE
    assert rope(lib, tokens=0) == 0
    assert back(lib, n=None) == ARG and back(lib, pos=None) == ARG
    assert back(lib, dq=None) == ARG and back(lib, qi=None) == ARG
    assert back(lib, dk=heads(heads=4)) == SHAPE
    assert back(lib, ws=None) == ARG and back(lib, ws=ODD) == ARG and back(lib, size=100) == ARG
    assert back(lib, wq=0x10002) == ARG
    assert back(lib, n=norm(q_weight=None, k_weight=None)) == ARG          # a weight's gradient without a norm
    assert back(lib, tokens=0, wq=None, wk=None, ws=None) == 0
    assert lib.fp4_qk_norm_workspace(96) == 0 and lib.fp4_qk_norm_workspace(128) > 0


@pytest.mark.parametrize("kw,status", [
    (dict(format=api.FP8_E5M2), UNSUPPORTED), (dict(format=4), UNSUPPORTED), (dict(format=-1), UNSUPPORTED),
    (dict(head_dim=96), UNSUPPORTED), (dict(heads=0), SHAPE), (dict(heads=2000), SHAPE), (dict(page_size=8), SHAPE),
    (dict(page_size=48), SHAPE), (dict(page_size=2048), SHAPE), (dict(page_size=-16), SHAPE), (dict(pages=0), SHAPE),
    (dict(pages=1 << 31), SHAPE), (dict(k_codes=None), ARG), (dict(v_scales=None), ARG), (dict(v_codes=ODD), ARG),
    (dict(k_scales=ODD), ARG), (dict(page_stride=0), ARG), (dict(token_stride=-128), ARG), (dict(head_stride=136), ARG),
    (dict(scale_block_stride=8), ARG), (dict(scale_page_stride=0), ARG), (dict(token_stride=112), ARG),
    (dict(token_stride=1 << 30), SHAPE), (dict(head_stride=1 << 40), SHAPE), (dict(scale_head_stride=1 << 30), SHAPE),
    (dict(format=api.NVFP4, amax=None), ARG), (dict(format=api.UE5M3, target=0.0), ARG),
    (dict(format=api.NVFP4, target=float("nan")), ARG)])
def test_caches_are_rejected(lib, kw, status):
    bad = cache(**kw)
    assert write(lib, c=bad) == status and _err(lib)
    assert read(lib, c=bad) == status
    assert decode(lib, c=bad) == status
    assert lib.fp4_attention_workspace(ctypes.byref(bad), 16, 4, 4) == 0


def test_cache_calls_are_rejected(lib):
    assert write(lib, c=None) == ARG and write(lib, k=None) == ARG and write(lib, v=None) == ARG
    assert write(lib, slots=None) == ARG and write(lib, tokens=-1) == SHAPE and write(lib, tokens=1 << 31) == SHAPE
    assert write(lib, k=heads(heads=4)) == SHAPE and write(lib, v=heads(heads=4)) == SHAPE
    assert write(lib, q=heads(), qo=heads()) == ARG                         # q needs a norm
    assert write(lib, n=norm(), pos=None) == ARG and write(lib, n=norm(), pos=FAKE, q=heads()) == ARG
    assert write(lib, tokens=0) == 0
    assert read(lib, c=None) == ARG and read(lib, slots=None) == ARG and read(lib, n=-1) == SHAPE
    assert read(lib, k=None, v=None) == ARG and read(lib, k=ODD) == ARG and read(lib, v=ODD) == ARG
    assert read(lib, n=0) == 0


def test_attention_is_rejected(lib):
    assert decode(lib, c=None) == ARG and decode(lib, q=None) == ARG
    assert decode(lib, q=heads(heads=12)) == SHAPE and decode(lib, n=-1) == SHAPE and decode(lib, n=1 << 31) == SHAPE
    assert decode(lib, n=1 << 28) == SHAPE                                  # more than 2^31 rows of the output
    assert decode(lib, table=None) == ARG and decode(lib, table=0x10002) == ARG and decode(lib, stride=-1) == ARG
    assert decode(lib, width=-1) == SHAPE and decode(lib, width=1 << 28) == SHAPE
    assert decode(lib, lens=None) == ARG and decode(lib, lens=0x10001) == ARG and decode(lib, lse=0x10002) == ARG
    assert decode(lib, scale=float("nan")) == ARG and decode(lib, scale=float("inf")) == ARG
    assert decode(lib, out=None) == ARG and decode(lib, out=ODD) == ARG and decode(lib, out_type=2) == ARG
    assert decode(lib, ws=ODD, size=64) == ARG and decode(lib, ws=FAKE, size=-1) == ARG
    assert decode(lib, n=0, table=None, lens=None, out=None) == 0
    assert lib.fp4_attention_workspace(None, 16, 4, 4) == 0
    assert lib.fp4_selftest_set_attention_splits(-1) == ARG and lib.fp4_selftest_set_attention_splits(513) == ARG


def test_struct_layouts_match_header(tmp_path):
    exe = tmp_path / "abi_layout"
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", "abi_layout_attention.c"), "-o", str(exe)], check=True)
    lines = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines()
    c = {k: int(v) for k, v in (line.split() for line in lines)}
    for name, cls in (("fp4_heads", api.Heads), ("fp4_qk_norm", api.QKNormDesc), ("fp4_kv_cache", api.KVCacheDesc)):
        assert ctypes.sizeof(cls) == c[name + ".__size__"], name
        for field, _ in cls._fields_:
            assert getattr(cls, field).offset == c["%s.%s" % (name, field)], (name, field)


# ------------------------------------------------------------- the binding --
BF = torch.bfloat16


def rows(t=4, h=8, d=128, dtype=BF):
    return torch.zeros((t, h, d), dtype=dtype)


def kv(fmt="mxfp8", **kw):
    return api.KVCache.empty(**dict(dict(pages=4, page_size=16, heads=8, head_dim=128, fmt=fmt, device="cpu"), **kw))


def test_binding_rejects_norms():
    w, t = torch.ones(128), torch.zeros((9, 64))
    for args in ((w, None), (None, None), (w, w.to(BF)), (w, torch.ones(64)), (torch.ones(256)[::2],) * 2,
                 (w.double(), w.double()), (w, w, t.double()), (w, w, torch.zeros((9, 63))), (w, w, t[:, ::2]), (w, w, t[0])):
        with pytest.raises(ValueError):
            api.QKNorm(*args)
    with pytest.raises(ValueError):
        api.QKNorm(w, w, t, style="pairs")


def test_binding_rejects_rows():
    n = api.QKNorm(torch.ones(128), torch.ones(128), torch.zeros((9, 64)))
    pos = torch.zeros(4, dtype=torch.int64)
    for q, k, p in ((rows(dtype=torch.float32), rows(), pos), (rows()[0], rows(), pos), (rows(), rows(3), pos),
                    (rows(), rows(d=64), pos), (rows(d=64), rows(d=64), pos), (rows(), rows(), None),
                    (rows(), rows(), pos.int()), (rows(), rows(), pos[:3]), (None, None, pos),
                    (rows(d=256)[..., ::2], rows(), pos)):
        with pytest.raises(ValueError):
            api.qk_norm_rope(n, q, k, p)
    with pytest.raises(ValueError):
        api.qk_norm_rope(n, rows(), rows(), pos, out=(rows(3), None))
    with pytest.raises(ValueError):
        api.qk_norm_rope_backward(n, rows(), rows(), pos, rows(), rows(h=4))
    with pytest.raises(ValueError):
        api.qk_norm_rope_backward(n, rows(), rows(), pos, rows(), rows(), weight_grads=torch.zeros(128))
    with pytest.raises(ValueError, match="GPU"):
        api.qk_norm_rope(n, rows(), rows(), pos)


def test_binding_rejects_caches():
    c = kv()
    for kw in (dict(fmt="fp8_e5m2"), dict(head_dim=96), dict(fmt="nvfp4"), dict(fmt="nvfp4", amax=torch.ones(1)),
               dict(fmt="ue5m3", amax=torch.ones(2, dtype=torch.float64))):
        with pytest.raises(ValueError):
            kv(**kw)
    kc, ks, vc, vs = c.k_codes, c.k_scales, c.v_codes, c.v_scales
    for args in ((kc[0], ks, vc, vs), (kc, ks, vc[:2], vs), (kc, ks[:, :, :2], vc, vs[:, :, :2]), (kc.int(), ks, vc.int(), vs),
                 (kc, ks, vc.transpose(1, 2).contiguous().transpose(1, 2), vs),
                 (kc.transpose(2, 3).contiguous().transpose(2, 3), ks, vc.transpose(2, 3).contiguous().transpose(2, 3), vs)):
        with pytest.raises(ValueError):
            api.KVCache("mxfp8", *args)
    assert kv("nvfp4", amax=torch.ones(2)).k_codes.shape == (4, 8, 16, 64)
    assert kv("fp8", head_dim=64).k_scales.shape == (4, 8, 1, 16)
    assert kv("ue5m3", head_dim=256, amax=torch.ones(2)).v_scales.shape == (4, 8, 16, 16)


def test_binding_rejects_writes_and_reads():
    c, slots = kv(), torch.zeros(4, dtype=torch.int64)
    n = api.QKNorm(torch.ones(128), torch.ones(128))
    for k, v, s, kw in ((rows(h=4), rows(), slots, {}), (rows(), rows(h=4), slots, {}), (rows(), rows(3), slots, {}),
                        (rows(), rows(), slots.int(), {}), (rows(), rows(), slots[:3], {}), (rows(), rows(), slots, dict(q=rows())),
                        (rows(), rows(), slots, dict(q=rows(3), norm=n)),
                        (rows(), rows(), slots, dict(q=rows(), norm=n, q_out=rows(h=4)))):
        with pytest.raises(ValueError):
            api.kv_cache_write(c, k, v, s, **kw)
    for s, dt in ((slots.int(), BF), (slots.view(2, 2), BF), (slots, torch.float16), (torch.zeros(8, dtype=torch.int64)[::2], BF)):
        with pytest.raises(ValueError):
            api.kv_cache_read(c, s, dt)


def test_binding_rejects_attention():
    c, t, n = kv(), torch.zeros((4, 3), dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    for q, table, lens, kw in ((rows(d=64), t, n, {}), (rows(), t.long(), n, {}), (rows(), t[:3], n, {}), (rows(), t[0], n, {}),
                               (rows(), t.t().contiguous().t(), n, {}), (rows(), t, n.long(), {}), (rows(), t, n[:3], {}),
                               (rows(), t, n, dict(out=rows(3))), (rows(), t, n, dict(out_dtype=torch.float16)),
                               (rows(), t, n, dict(out=rows(h=16)[:, ::2]))):
        with pytest.raises(ValueError):
            api.attention_decode(q, c, t if table is None else table, lens, **kw)


def test_layer_rejects():
    with pytest.raises(ValueError):
        attention.QuantizedAttention(torch.zeros((7 * 64, 128), dtype=BF), torch.zeros((128, 256), dtype=BF), 4, 2)
    with pytest.raises(ValueError):
        attention.QuantizedAttention(torch.zeros((8 * 96, 128), dtype=BF), torch.zeros((128, 384), dtype=BF), 4, 2)
    with pytest.raises(ValueError):
        attention.QuantizedAttention(torch.zeros((8 * 64, 128), dtype=BF), torch.zeros((128, 128), dtype=BF), 4, 2)
    with pytest.raises(ValueError):
        attention.QuantizedAttention(torch.zeros((7 * 64, 128), dtype=BF), torch.zeros((128, 192), dtype=BF), 3, 2)


def test_slots():
    t = torch.tensor([[4, 7, -1], [2, 0, 1]], dtype=torch.int32)
    s = lambda *p: attention.slots_of(t, torch.tensor(p), 16).tolist()        # noqa: E731
    assert s(0, 47) == [64, 31] and s(17, -1) == [113, -1] and s(32, 48) == [-1, -1]


def test_index_arrays_are_aligned_to_their_elements(lib):
    off = FAKE + 4
    assert rope(lib, pos=off) == ARG and back(lib, pos=off) == ARG
    assert write(lib, slots=off) == ARG and write(lib, n=norm(), pos=off) == ARG and read(lib, slots=off) == ARG
    bad = cache(format=api.NVFP4, amax=FAKE + 2)
    assert write(lib, c=bad) == ARG and read(lib, c=bad) == ARG and decode(lib, c=bad) == ARG


def test_contexts_end_at_2_30(lib):
    """Token numbers and what lies a few tiles behind them are 32 bits wide in the kernels."""
    assert decode(lib, width=1 << 26) == SHAPE and decode(lib, width=1 << 62) == SHAPE
    assert decode(lib, width=(1 << 26) - 1, n=0) == 0


def test_slots_without_pages():
    t = torch.empty((2, 0), dtype=torch.int32)
    assert attention.slots_of(t, torch.tensor([0, 5]), 16).tolist() == [-1, -1]
