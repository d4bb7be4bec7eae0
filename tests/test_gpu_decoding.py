"""The decoding operators together, as a server uses them: every step plans its
tokens, projects them with group-scaled weights, appends keys and values to the
cache, attends over it and projects the result.  Each operator is checked
against its own definition on what the one before it gave, with the gates of
their own tests, and a captured step replays."""
import os
import subprocess
import sys

import pytest
import torch

import rotated_w4a4_quantized_b200 as cr
from tests import decoding_ref as ref
from tests.test_gpu_guard_bytes import Guarded
from tests.test_gpu_kv4 import check as check_attention
from tests.test_gpu_w4g import check as check_linear

pytestmark = pytest.mark.gpu

HEADS, KV, D, HIDDEN, PAGE, GROUP = 4, 2, 64, 256, 16, 64


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from rotated_w4a4_quantized_b200 import build
    build.build()


class Layer:
    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        width = (HEADS + 2 * KV) * D
        self.wqkv = (torch.randn(width, HIDDEN, generator=g) * 0.1).to(torch.bfloat16).cuda()
        self.wo = (torch.randn(HIDDEN, HEADS * D, generator=g) * 0.1).to(torch.bfloat16).cuda()
        self.qkv = cr.convrot_w4g_quantize_weight(self.wqkv, GROUP, 32)
        self.out = cr.convrot_w4g_quantize_weight(self.wo, GROUP, 64)

    def __call__(self, x, cache, plan, table):
        qkv = cr.convrot_w4g_linear(x, *self.qkv, None, GROUP, 32)
        q = qkv[:, :HEADS * D].unflatten(1, (HEADS, D))
        k = qkv[:, HEADS * D:(HEADS + KV) * D].unflatten(1, (KV, D))
        v = qkv[:, (HEADS + KV) * D:].unflatten(1, (KV, D))
        cr.convrot_kv4_append(k, v, cache, plan.slots, GROUP)
        o = cr.convrot_kv4_attention(q, cache, table, plan.seq_lens, plan.cu_q, D ** -0.5, GROUP)
        return qkv, o, cr.convrot_w4g_linear(o.flatten(1), *self.out, None, GROUP, 64)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def test_steps_of_a_server():
    layer = Layer(1)
    cache = cr.convrot_kv4_new_cache(40, KV, PAGE, D, "cuda")
    table, free, count = i32([[-1] * 8] * 3), i32(list(range(40)) + [0] * 24), i32([40])
    lens, host_table, host_free, host_count = i32([0, 0, 0]), [[-1] * 8 for _ in range(3)], list(range(40)) + [0] * 24, 40
    host_lens = [0, 0, 0]
    g = torch.Generator().manual_seed(2)
    # prompts, single tokens, a finished request, its place taken, drafted tokens
    for new in ([20, 7, 1], [1, 1, 1], [1, -1, 4], [1, 33, 1], [3, 2, -1], [1, 1, 0]):
        T = sum(max(n, 0) for n in new)
        plan = cr.convrot_kv4_plan(lens, i32(new), table, free, count, PAGE, T)
        want = ref.plan(host_lens, new, host_table, host_free, host_count, PAGE, T)
        assert want["result"][3] == 0
        for name, value in want.items():
            assert getattr(plan, name).tolist() == value, name
        assert table.tolist() == host_table and free.tolist() == host_free
        host_lens, host_count = want["seq_lens"], want["result"][0]
        x = torch.randn(T, HIDDEN, generator=g).to(torch.bfloat16)
        qkv, o, y = layer(x.cuda(), cache, plan, table)
        assert cr.convrot_kv4_check_device_error() == 0
        check_linear(qkv, x, layer.qkv[0].cpu(), layer.qkv[1].cpu(), None, GROUP)
        host_cache = cr.Kv4Cache(*[t.cpu() for t in cache])
        # what lies in the cache is the definition of the projected rows
        rows = qkv[:, HEADS * D:].reshape(T * 2 * KV, D).contiguous()
        c, s = ref.quantize_blocks(cr.convrot_debug_rotate_f32(rows, GROUP).cpu(), D)
        c, s = c.reshape(T, 2, KV, D), s.reshape(T, 2, KV)
        for t, slot in enumerate(want["slots"]):
            for i in (0, 1):
                assert torch.equal(ref.unpack(host_cache[2 * i][slot // PAGE, :, slot % PAGE]), c[t, i])
                assert torch.equal(host_cache[2 * i + 1][slot // PAGE, :, slot % PAGE], s[t, i])
        q = qkv.cpu()[:, :HEADS * D].reshape(T, HEADS, D)
        check_attention(o, q, host_cache, table.cpu(), torch.tensor(host_lens), torch.tensor(want["cu_q"]), D ** -0.5, GROUP)
        check_linear(y, o.flatten(1).cpu(), layer.out[0].cpu(), layer.out[1].cpu(), None, GROUP)
        lens, count = plan.seq_lens, plan.free_count


def test_a_captured_step_replays():
    """One decoding step as a graph, lengths and pages fed back from step to
    step; beside it the same steps without a graph."""
    layer = Layer(3)

    def start():
        return dict(cache=cr.convrot_kv4_new_cache(20, KV, PAGE, D, "cuda"), table=i32([[-1] * 5] * 2),
                    free=i32(list(range(20))), count=i32([20]), lens=i32([0, 0]), new=i32([1, 1]),
                    x=torch.zeros(2, HIDDEN, dtype=torch.bfloat16, device="cuda"))

    def step(s):
        plan = cr.convrot_kv4_plan(s["lens"], s["new"], s["table"], s["free"], s["count"], PAGE, 2)
        y = layer(s["x"], s["cache"], plan, s["table"])[2]
        s["lens"].copy_(plan.seq_lens)
        s["count"].copy_(plan.free_count)
        return y
    warm = start()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(warm)
    torch.cuda.current_stream().wait_stream(side)
    one, two = start(), start()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step(one)
    g = torch.Generator().manual_seed(4)
    for _ in range(40):
        x = torch.randn(2, HIDDEN, generator=g).to(torch.bfloat16).cuda()
        one["x"].copy_(x)
        two["x"].copy_(x)
        graph.replay()
        assert torch.equal(y, step(two))
    assert one["lens"].tolist() == two["lens"].tolist() == [40, 40]
    assert torch.equal(one["table"], two["table"])
    assert cr.convrot_kv4_check_device_error() == 0


def test_native_and_python_calls_agree():
    """A stream given by name takes the Python path of the bindings."""
    s = torch.cuda.current_stream()
    g = torch.Generator().manual_seed(6)
    x = torch.randn(20, 256, generator=g).to(torch.bfloat16).cuda()
    qw, sg = cr.convrot_w4g_quantize_weight(torch.randn(128, 256, generator=g).to(torch.bfloat16).cuda(), 64, 64)
    b = torch.randn(128, generator=g).to(torch.bfloat16).cuda()
    for n in (1, 20):
        for bias in (None, b):
            assert torch.equal(cr.convrot_w4g_linear(x[:n], qw, sg, bias, 64, 64),
                               cr.convrot_w4g_linear(x[:n], qw, sg, bias, 64, 64, stream=s))
    k, v = (torch.randn(20, 2, 64, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    plans, caches = [], []
    for kw in ({}, {"stream": s}):
        table = i32([[-1, -1], [-1, -1]])
        p = cr.convrot_kv4_plan(i32([0, 0]), i32([17, 3]), table, i32([5, 4, 3, 2, 1, 0]), i32([6]), 16, 20, **kw)
        cache = cr.convrot_kv4_new_cache(6, 2, 16, 64, "cuda")
        cr.convrot_kv4_append(k, v, cache, p.slots, 64, **kw)
        kr, vr = cr.convrot_kv4_read(cache, p.slots, 64, **kw)
        o = cr.convrot_kv4_attention(x.unflatten(1, (4, 64)), cache, table, p.seq_lens, p.cu_q, 0.1, 64, **kw)
        plans.append((table, p.seq_lens, p.cu_q, p.slots, p.positions, p.result, p.free_count, p.status, kr, vr, o))
        caches.append(cache)
    for a, c in zip(plans[0] + tuple(caches[0]), plans[1] + tuple(caches[1])):
        assert torch.equal(a, c) and a.shape == c.shape


def test_overlapping_buffers_are_refused():
    """Results in the place of an operand would depend on which part of the GPU
    is first: every such call is refused and writes nothing."""
    def refused(f, *a, **k):
        with pytest.raises(cr.ConvRotError, match="OVERLAP"):
            f(*a, **k)
    cache = cr.convrot_kv4_new_cache(4, 2, 16, 64, "cuda")
    q = torch.randn(8, 4, 64).to(torch.bfloat16).cuda()
    before, i32 = q.clone(), lambda v: torch.tensor(v, dtype=torch.int32).cuda()
    table, lens, cu = i32([[0, 1, 2]]), i32([40]), i32([0, 8])
    refused(cr.convrot_kv4_attention, q, cache, table, lens, cu, 0.1, 64, out=q)
    room = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    out = room[4096:4096 + q.numel() * 2].view(torch.bfloat16).view(q.shape)
    refused(cr.convrot_kv4_attention, q, cache, table, lens, cu, 0.1, 64, workspace=room, out=out)
    slots = torch.arange(8).cuda()
    k = torch.empty(8, 2, 64, dtype=torch.bfloat16, device="cuda")
    refused(cr.convrot_kv4_read, cache, slots, 64, k=k, v=k)
    same = cr.Kv4Cache(cache.k_codes, cache.k_scales, cache.k_codes, cache.v_scales)
    refused(cr.convrot_kv4_append, q[:, :2], q[:, 2:], same, slots, 64)
    x = q.view(8, 256)
    weights = torch.zeros(256, 128, dtype=torch.uint8, device="cuda"), torch.zeros(256, 4, dtype=torch.bfloat16, device="cuda")
    refused(cr.convrot_w4g_linear, x, *weights, None, 64, 64, out=x)
    refused(cr.convrot_w4g_quantize_weight, x, 64, 64, qw=x.view(torch.uint8).view(-1)[:1024].view(8, 128))
    pages = torch.arange(12, dtype=torch.int32, device="cuda")
    refused(cr.convrot_kv4_plan, i32([3]), i32([1]), pages[:4].view(1, 4), pages, i32([8]), 16, 4)
    # columns of one buffer do not overlap
    both = torch.randn(8, 8, 64).to(torch.bfloat16).cuda()
    cr.convrot_kv4_append(both[:, :2], both[:, 2:4], cache, slots, 64)
    torch.cuda.synchronize()
    assert torch.equal(q, before) and torch.equal(pages, torch.arange(12, dtype=torch.int32, device="cuda"))


def test_the_first_calls_may_be_captured():
    """A process whose first calls are in a capture: nothing is set up in a
    way that a capture forbids."""
    code = """if True:
        import torch
        import rotated_w4a4_quantized_b200 as cr
        T, H, D = 8, 2, 128
        cache = cr.convrot_kv4_new_cache(20, H, 64, D, "cuda")
        k, q = (torch.randn(T, h, D, device="cuda").bfloat16() for h in (H, 4 * H))
        x = torch.randn(T, 1024, device="cuda").bfloat16()
        qw, sg = torch.full((512, 512), 0x21, dtype=torch.uint8, device="cuda"), torch.ones(512, 16, device="cuda").bfloat16()
        i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
        table, free, count = i32(*[0] * T * 4).view(T, 4), torch.arange(20, device="cuda").int(), i32(20)
        def step():
            p = cr.convrot_kv4_plan(i0, i1, table, free, count, 64, T)
            cr.convrot_kv4_append(k, k, cache, p.slots, 64)
            return (cr.convrot_kv4_attention(q, cache, table, p.seq_lens, p.cu_q, 0.1, 64),
                    *cr.convrot_kv4_read(cache, p.slots, 64), cr.convrot_w4g_linear(x, qw, sg, None, 64, 64))
        i0, i1 = i32(*[0] * T), i32(*[1] * T)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = step()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            assert torch.equal(a, b) and bool(a.float().abs().sum() > 0)
        print("captured")
    """
    run = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                         cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert run.returncode == 0 and "captured" in run.stdout, run.stderr[-2000:]


def test_writes_stay_inside_their_buffers():
    g = torch.Generator().manual_seed(5)

    def same(guards, plain):
        torch.cuda.synchronize()
        for a, b in zip(guards, plain):
            assert a.intact()
            assert torch.equal(a.t, b)

    w = torch.randn(37, 256, generator=g).to(torch.bfloat16).cuda()
    for group in (0, 64, 256):
        for sgroup in (32, 128):
            want = cr.convrot_w4g_quantize_weight(w, group, sgroup)
            qw, sg = Guarded((37, 128), torch.uint8), Guarded((37, 256 // sgroup), torch.bfloat16)
            cr.convrot_w4g_quantize_weight(w, group, sgroup, qw=qw.t, sg=sg.t)
            same((qw, sg), want)
            for M in (1, 4, 6, 16, 21, 80):
                x = torch.randn(M, 256, generator=g).to(torch.bfloat16).cuda()
                y = cr.convrot_w4g_linear(x, *want, None, group, sgroup)
                out = Guarded((M, 37), torch.bfloat16)
                ws = Guarded((max(16, cr.convrot_w4g_workspace_size(M, 256)),), torch.uint8, ws=True)
                cr.convrot_w4g_linear(x, *want, None, group, sgroup, workspace=ws.t, out=out.t)
                torch.cuda.synchronize()
                assert ws.intact()
                same((out,), (y,))
    for D_, heads, page in ((64, 3, 16), (128, 2, 64), (256, 1, 32)):
        shapes = ((5, heads, page, D_ // 2), torch.uint8), ((5, heads, page), torch.bfloat16)
        guards = [Guarded(s, d) for s, d in shapes * 2]
        cache = cr.Kv4Cache(*[a.t for a in guards])
        plain = cr.convrot_kv4_new_cache(5, heads, page, D_, "cuda")
        for t in cache:
            t.zero_()
        T = 5 * page
        k, v = (torch.randn(T, heads, D_, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
        slots = torch.randperm(T, generator=g).cuda()
        for c in (cache, plain):
            cr.convrot_kv4_append(k, v, c, slots, 64)
        same(guards, plain)
        ko, vo = (Guarded((T, heads, D_), torch.bfloat16) for _ in range(2))
        cr.convrot_kv4_read(cache, slots, 64, k=ko.t, v=vo.t)
        same((ko, vo), cr.convrot_kv4_read(plain, slots, 64))
        table = torch.arange(5).int().reshape(1, 5).cuda()
        for nq in (1, 2, 7):
            q = torch.randn(nq, 2 * heads, D_, generator=g).to(torch.bfloat16).cuda()
            args = (table, i32([T - 3]), i32([0, nq]), 0.1, 64)
            out = Guarded((nq, 2 * heads, D_), torch.bfloat16)
            ws = Guarded((cr.convrot_kv4_attention_workspace_size(nq, 1, 2 * heads, heads, D_, T),), torch.uint8, ws=True)
            cr.convrot_kv4_attention(q, cache, *args, workspace=ws.t, out=out.t)
            same((out,), (cr.convrot_kv4_attention(q, plain, *args),))
            assert ws.intact()
        same(guards, plain)
