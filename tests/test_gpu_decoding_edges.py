"""GPU tests of the decoding operators at their edges: rows that are not finite
in every form of the group-scaled layer, codes decided by the tie rule alone,
calls on two streams and from two threads at once.

Gates are those of test_gpu_w4g.py (products) and equality (codes, scales, the
same call twice)."""
import threading

import pytest
import torch

import rotated_w4a4_quantized_b200 as cr
from tests import decoding_ref as ref
from tests.test_gpu_kv4 import setup, to
from tests.test_gpu_w4g import check as check_linear, draw
from tests.tie_rows import exact_tie_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from rotated_w4a4_quantized_b200 import build
    build.build()


@pytest.mark.parametrize("group", [0, 64, 256])
@pytest.mark.parametrize("M,K", [(3, 512), (8, 512), (9, 512), (16, 4096), (20, 512), (2, 16896)])
def test_rows_that_are_not_finite(M, K, group):
    """Each form (up to 4, 8 and 16 tokens; numbers made by the product or
    before it): such a row gives NaN, the others what they gave without it."""
    x, qw, sg, b = draw(M, K, 50, 64, seed=M + K)
    clean = cr.convrot_w4g_linear(x.cuda(), qw.cuda(), sg.cuda(), b.cuda(), group, 64)
    bad = {0: float("nan"), M - 1: float("inf"), M // 2: float("-inf")}
    for row, v in bad.items():
        x[row, (37 * row + 7) % K] = v
    y = cr.convrot_w4g_linear(x.cuda(), qw.cuda(), sg.cuda(), b.cuda(), group, 64)
    good = [i for i in range(M) if i not in bad]
    assert torch.equal(y[good], clean[good])
    assert bool(y[list(bad)].isnan().all())
    if good:
        check_linear(y[good], x[good], qw, sg, b, group)


def as_bf16(bits):
    return torch.from_numpy(bits.astype("int32")).to(torch.int16).view(torch.bfloat16)


@pytest.mark.parametrize("D,group", [(64, 64), (128, 64), (256, 64), (256, 256)])
@pytest.mark.parametrize("T", [7, 30000])
def test_append_breaks_ties_away_from_zero(D, group, T):
    """Both spreads of a row over threads (few rows, many rows)."""
    heads = 4
    bits, _, s0, codes = exact_tie_rows(64 * heads, D, group, seed=D + group)
    rows, scales = as_bf16(bits).view(64, heads, D), torch.from_numpy(s0.copy()).to(torch.bfloat16).view(64, heads)
    codes = torch.from_numpy(codes.astype("int64")).view(64, heads, D)
    at = torch.arange(T) % 64
    k, v = rows[at].cuda(), (-rows[at]).cuda()
    pages = -(-T // 64)
    cache = cr.convrot_kv4_new_cache(pages, heads, 64, D, "cuda")
    slots = torch.randperm(pages * 64, generator=torch.Generator().manual_seed(1))[:T]
    cr.convrot_kv4_append(k, v, cache, slots.cuda(), group)
    kc, ks, vc, vs = (t.cpu() for t in cache)
    for sign, c, s in ((1, kc, ks), (-1, vc, vs)):
        assert torch.equal(ref.unpack(c[slots // 64, :, slots % 64]), sign * codes[at])
        assert torch.equal(s[slots // 64, :, slots % 64], scales[at])


@pytest.mark.parametrize("K,group,scale_group", [(64, 64, 64), (128, 64, 128)])
def test_weights_break_ties_away_from_zero(K, group, scale_group):
    bits, _, s0, codes = exact_tie_rows(500, K, group, seed=K)
    qw, sg = cr.convrot_w4g_quantize_weight(as_bf16(bits).cuda(), group, scale_group)
    assert torch.equal(ref.unpack(qw.cpu()), torch.from_numpy(codes.astype("int64")))
    assert torch.equal(sg.cpu()[:, 0], torch.from_numpy(s0.copy()).to(torch.bfloat16))


def calls(seed):
    """The calls of a step on operands of their own, and what they gave alone."""
    q, cache, table, lens, cu = setup([3000, 17, 900], [1, 2, 1], 8, 2, 128, 64, seed=seed)
    dev = (q.cuda(), to(cache), table.cuda(), lens.cuda(), cu.cuda())
    x, qw, sg, b = (t.cuda() for t in draw(21, 1024, 500, 64, seed=seed))
    slots = torch.arange(40, 60, device="cuda")

    def run():
        return (cr.convrot_kv4_attention(*dev, 0.1, 64), cr.convrot_w4g_linear(x, qw, sg, b, 64, 64),
                cr.convrot_w4g_linear(x[:3], qw, sg, b, 64, 64), *cr.convrot_kv4_read(dev[1], slots, 64))
    return run, run()


def test_two_streams_at_once():
    pairs = [calls(s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in pairs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (run, _) in enumerate(pairs):
            with torch.cuda.stream(streams[i]):
                got[i].append(run())
    torch.cuda.synchronize()
    for results, (_, want) in zip(got, pairs):
        assert all(torch.equal(a, b) for r in results for a, b in zip(r, want))


def test_two_threads_at_once():
    pairs = [calls(s) for s in (3, 4)]
    torch.cuda.synchronize()
    wrong, done = [], []

    def work(run, want):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got = run()
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want)):
                    wrong.append(1)
        done.append(1)
    threads = [threading.Thread(target=work, args=p) for p in pairs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(done) == 2 and not wrong


def test_two_graphs_on_one_workspace():
    """Two captured calls that share a workspace, replayed in turn."""
    a, b = (setup(lens, [1, 1], 8, 2, 128, 64, seed=5) for lens in ([5000, 700], [33, 4000]))
    ws = torch.empty(cr.convrot_kv4_attention_workspace_size(2, 2, 8, 2, 128, 128 * 64), dtype=torch.uint8, device="cuda")
    graphs, outs, wants = [], [], []
    for q, cache, table, lens, cu in (a, b):
        dev = (q.cuda(), to(cache), table.cuda(), lens.cuda(), cu.cuda())
        wants.append(cr.convrot_kv4_attention(*dev, 0.1, 64))
        out, g = torch.empty_like(wants[-1]), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            cr.convrot_kv4_attention(*dev, 0.1, 64, workspace=ws, out=out)
        graphs.append((g, dev))
        outs.append(out)
    for _ in range(5):
        for (g, _), out in zip(graphs, outs):
            out.zero_()
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, wants))
