"""The group-scaled and the cache library without a GPU: what the headers
declare, and what the host refuses before it touches the device."""
import ctypes
import os
import re

import pytest
import torch

import oracle as O
import rotated_w4a4_quantized_b200 as cr
from rotated_w4a4_quantized_b200 import workloads as wl
from tests import decoding_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, B, U = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x20000), ctypes.c_void_p(0x10008)
BIG = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def _built():
    from rotated_w4a4_quantized_b200 import build
    build.build()


def declared(name):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", name)).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(convrot_[a-z0-9_]+)\s*\(", text)))


def test_libraries_export_what_the_headers_declare():
    assert declared("convrot_w4g.h") == ["convrot_w4g_linear", "convrot_w4g_quantize_weight",
                                         "convrot_w4g_workspace_size"]
    assert declared("convrot_kv4.h") == [
        "convrot_kv4_append", "convrot_kv4_attention", "convrot_kv4_attention_workspace_size",
        "convrot_kv4_check_device_error", "convrot_kv4_plan", "convrot_kv4_read"]
    for lib, header in ((cr.lib_w4g(), "convrot_w4g.h"), (cr.lib_kv4(), "convrot_kv4.h")):
        for name in declared(header):
            assert hasattr(lib, name), name


def test_page_status_has_a_name():
    assert cr.lib().convrot_status_string(12).decode().startswith("CONVROT_ERR_PAGE")
    assert cr.STATUS[12] == "CONVROT_ERR_PAGE"


@pytest.mark.parametrize("attr,state,loader", [("LIB_W4G_PATH", "_lib_w4g", "lib_w4g"),
                                               ("LIB_KV4_PATH", "_lib_kv4", "lib_kv4")])
def test_missing_library_raises(monkeypatch, tmp_path, attr, state, loader):
    monkeypatch.setattr(cr, attr, str(tmp_path / "none.so"))
    monkeypatch.setattr(cr, state, None)
    with pytest.raises(RuntimeError, match="no fallback"):
        getattr(cr, loader)()


def test_missing_extension_raises(monkeypatch):
    import sys
    monkeypatch.setattr(cr, "_extension", None)
    monkeypatch.delattr(cr, "_decoding", raising=False)
    monkeypatch.setitem(sys.modules, cr.__name__ + "._decoding", None)
    with pytest.raises(RuntimeError, match="no fallback"):
        cr._native()


def test_extension_leaves_what_is_not_plainly_right_to_python():
    ext = cr._native()
    x = torch.zeros(2, 2)
    for f, n in ((ext.w4g_linear, 6), (ext.kv4_plan, 7), (ext.kv4_append, 5), (ext.kv4_read, 3), (ext.kv4_attention, 7)):
        for args in ([], [x] * n, [x] * (n - 1), [None] * n, [(x, x, x, x)] * n, [1] * n, [x] * (n - 2) + [64, 64],
                     [x, (x, x, x, x), x, x, x, 0.5, 64][:n], [-1] * n, [1 << 70] * n):
            assert f(*args) is None


def test_w4g_host_refusals():
    L = cr.lib_w4g()
    q = L.convrot_w4g_quantize_weight
    assert q(A, 4, 1024, 128, 64, B, B, None) == 2
    assert q(A, 4, 1024, 64, 256, B, B, None) == 2
    assert q(A, 4, 96, 0, 32, B, B, None) == 3            # K % 64
    assert q(A, 4, 64, 0, 128, B, B, None) == 3           # K % scale_group
    assert q(A, 4, 320, 256, 64, B, B, None) == 3         # K % group
    assert q(A, -1, 1024, 64, 64, B, B, None) == 3
    assert q(A, 4, 32768 + 64, 64, 64, B, B, None) == 3
    assert q(None, 0, 1024, 64, 64, None, None, None) == 0
    assert q(A, 4, 1024, 64, 64, B, None, None) == 1
    assert q(A, 4, 1024, 64, 64, B, U, None) == 4
    f = L.convrot_w4g_linear
    # a few short rows need no workspace; beyond, two bytes a channel of whole
    # 256-channel blocks and a factor for each, rows in sixteens (eights)
    assert cr.convrot_w4g_workspace_size(1, 16384) == 0 and cr.convrot_w4g_workspace_size(16, 1024) == 0
    assert cr.convrot_w4g_workspace_size(0, 1024) == 0
    assert cr.convrot_w4g_workspace_size(17, 1024) == 32 * 4 * 512 + 512
    assert cr.convrot_w4g_workspace_size(5, 4096) == 8 * 16 * 512 + 512
    assert cr.convrot_w4g_workspace_size(2, 16384 + 64) == 2 * 65 * 512 + 768
    ws = cr.convrot_w4g_workspace_size(40, 1024)
    assert f(A, B, B, None, 40, 8, 1024, 64, 64, A, ws - 1, B, None) == 5
    assert f(A, B, B, None, 40, 8, 1024, 64, 64, U, ws, B, None) == 5
    assert f(A, B, B, None, 40, 8, 1024, 64, 64, None, 0, B, None) == 1
    assert f(A, B, B, None, 40, 8, 1024, 32, 64, A, ws, B, None) == 2
    assert f(A, B, B, None, 4, BIG, 1024, 64, 64, A, ws, B, None) == 3
    assert f(A, B, B, None, 1 << 22, 8, 1024, 0, 64, None, 0, B, None) == 3
    assert f(A, B, B, None, -1, 8, 1024, 0, 64, None, 0, B, None) == 3
    assert f(A, B, B, U, 4, 8, 1024, 0, 64, None, 0, B, None) == 4
    assert f(A, B, None, None, 4, 8, 1024, 0, 64, None, 0, B, None) == 1
    assert f(None, None, None, None, 0, 8, 1024, 0, 64, None, 0, None, None) == 0
    assert f(None, None, None, None, 8, 0, 1024, 0, 64, None, 0, None, None) == 0


def cache(**over):
    v = dict(k_codes=A, k_scales=A, v_codes=A, v_scales=A, num_pages=4, kv_heads=2, page=16, head_dim=128, group=64)
    v.update(over)
    return cr._kv4_cache_arg(*(x.value if isinstance(x, ctypes.c_void_p) else x or 0 for x in v.values()))


BAD_CACHES = [(dict(group=128), 2), (dict(group=256), 3), (dict(head_dim=96), 3), (dict(head_dim=32), 3),
              (dict(page=24), 3), (dict(page=8), 3), (dict(page=512), 3), (dict(kv_heads=0), 3),
              (dict(kv_heads=1025), 3), (dict(num_pages=-1), 3), (dict(num_pages=1 << 27), 3),
              (dict(k_codes=None), 1), (dict(v_scales=None), 1), (dict(v_codes=U), 4)]


@pytest.mark.parametrize("over,status", BAD_CACHES)
def test_bad_caches_are_refused(over, status):
    L, c = cr.lib_kv4(), cache(**over)
    assert L.convrot_kv4_append(c, A, 256, A, 256, A, 3, None) == status
    assert L.convrot_kv4_read(c, A, 3, A, A, None) == status
    assert L.convrot_kv4_attention(c, A, 1024, 3, 8, A, 4, A, A, 2, 0.1, A, 1 << 30, A, None) == status


def test_kv4_host_refusals():
    L, c = cr.lib_kv4(), cache()
    f = L.convrot_kv4_append
    assert f(None, A, 256, A, 256, A, 3, None) == 1
    assert f(c, A, 255, A, 256, A, 3, None) == 3
    assert f(c, A, 256, A, 260, A, 3, None) == 3
    assert f(c, A, 256, A, 256, A, -1, None) == 3
    assert f(c, None, 256, None, 256, None, 0, None) == 0
    assert f(c, A, 256, A, 256, None, 3, None) == 1
    assert f(c, U, 256, A, 256, A, 3, None) == 4
    f = L.convrot_kv4_attention

    def attn(ldq=1024, T=3, heads=8, max_pages=4, B=2, scale=0.1, ws=A, n=1 << 30, out=A, q=A, table=A):
        return f(c, q, ldq, T, heads, table, max_pages, A, A, B, scale, ws, n, out, None)
    assert attn(heads=7) == 3 and attn(heads=1) == 3 and attn(heads=0) == 3
    assert attn(ldq=1023) == 3 and attn(ldq=1020) == 3
    assert attn(T=-1) == 3 and attn(B=8193) == 3 and attn(B=-1) == 3
    assert attn(max_pages=-1) == 3 and attn(max_pages=1 << 27) == 3
    assert attn(scale=float("nan")) == 3 and attn(scale=float("-inf")) == 3 and attn(scale=1e31) == 3
    assert attn(T=0, q=None, out=None) == 0 and attn(B=0) == 0
    assert attn(ws=None) == 1 and attn(out=None) == 1 and attn(table=None) == 1
    assert attn(n=100) == 5 and attn(ws=U) == 5
    assert attn(q=U) == 4 and attn(out=U) == 4
    f = L.convrot_kv4_plan

    def plan(cached=A, B=2, page=16, table=A, most=4, free=A, cap=4, tokens=4, slots=A, result=A):
        return f(cached, A, B, page, table, most, free, cap, A, tokens, A, A, slots, A, result, None)
    assert plan(B=-1) == 3 and plan(B=8193) == 3 and plan(page=48) == 3 and plan(most=-1) == 3
    assert plan(cap=-1) == 3 and plan(tokens=-1) == 3 and plan(tokens=1 << 31) == 3
    assert plan(cached=None) == 1 and plan(table=None) == 1 and plan(free=None) == 1 and plan(slots=None) == 1
    assert plan(cached=U) == 4 and plan(result=U) == 4


def test_attention_workspace_sizes():
    f = cr.convrot_kv4_attention_workspace_size
    assert f(0, 4, 8, 2, 128, 1000) == 0 and f(4, 0, 8, 2, 128, 1000) == 0
    assert f(4, 4, 7, 2, 128, 1000) == 0 and f(4, 4, 8, 2, 96, 1000) == 0
    one = f(1, 1, 4, 1, 128, 64)
    assert one > 0
    # bounded whatever the lengths, and large sizes do not overflow
    most = f(64, 64, 32, 8, 128, 131072)
    assert one < most < 64 << 20
    assert f((1 << 31) - 1, 8192, 65536, 1, 256, (1 << 31) - 1) < 64 << 20


def test_wrappers_refuse_host_tensors():
    x, qw = torch.zeros(1, 64, dtype=torch.bfloat16), torch.zeros(4, 32, dtype=torch.uint8)
    sg = torch.zeros(4, 1, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        cr.convrot_w4g_linear(x, qw, sg, None, 0, 64)
    with pytest.raises(ValueError, match="CUDA"):
        cr.convrot_w4g_quantize_weight(x, 0, 64)
    c = cr.convrot_kv4_new_cache(1, 1, 16, 64, "cpu")
    with pytest.raises(ValueError, match="CUDA"):
        cr.convrot_kv4_append(x.view(1, 1, 64), x.view(1, 1, 64), c, torch.zeros(1, dtype=torch.int64), 64)
    with pytest.raises(ValueError, match="CUDA"):
        cr.convrot_kv4_plan(torch.zeros(1).int(), torch.zeros(1).int(), torch.zeros(1, 1).int(), torch.zeros(1).int(),
                            torch.zeros(1).int(), 16, 1)


@pytest.mark.skipif(torch.cuda.is_available(), reason="a GPU is present")
def test_valid_calls_without_gpu_report_cuda_error():
    assert cr.lib_w4g().convrot_w4g_linear(A, B, B, None, 4, 8, 1024, 0, 64, None, 0, B, None) == 6
    assert cr.lib_kv4().convrot_kv4_read(cache(), A, 3, A, A, None) == 6


@pytest.mark.parametrize("group", [64, 256])
def test_the_restated_rotation_is_the_oracles(group):
    O.build()
    x = torch.randn(3, 512, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    got = ref.rotate(x.double(), group)
    assert torch.allclose(got, torch.from_numpy(O.rotate(wl.bf16_bits(x), group)), rtol=0, atol=1e-12)


def test_the_restated_quantiser_by_hand():
    y = torch.tensor([[7.0, -3.5, 0.5, 0.49, 0.0, -0.5, 2.5, 6.5]])
    c, s = ref.quantize_blocks(y, 8)
    assert s.tolist() == [[1.0]] and c.tolist() == [[7, -4, 1, 0, 0, -1, 3, 7]]
    c, s = ref.quantize_blocks(y * 2.0 ** -101, 8)
    assert s.tolist() == [[0.0]] and not c.any()


def test_the_restated_plan_by_hand():
    table, free = [[5, 0], [6, 7], [8, 0]], [1, 2, 3, 9, 9]
    got = ref.plan([16, 17, 3], [1, -1, 2], table, free, 2, 16, 4)
    # request 1 gives pages 6 and 7 back, request 0 takes the top one, 7
    assert got == dict(seq_lens=[17, 0, 5], cu_q=[0, 1, 1, 3], slots=[112, 131, 132, -1], positions=[16, 3, 4, -1],
                       result=[3, 1, 3, 0])
    assert table == [[5, 7], [6, 7], [8, 0]] and free == [1, 2, 6, 7, 9]
