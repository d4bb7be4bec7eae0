"""GPU tests of the group-scaled few-token layer (include/convrot_w4g.h).

Gates:
  - codes and scales of convrot_w4g_quantize_weight: equal, bit for bit, to
    the definition evaluated in fp32 on the GPU's own rotated values;
  - the product against float64:
      |y - t| <= 2^-8 |t| + 2^-17 L + Q,  L = the sum of |terms|:
    the final rounding to bf16 is off by half a step (2^-8 of the value); the
    fp32 sums over groups, blocks and parts take at most 2 x 128 roundings of
    2^-24 of L; Q is what the activations' numbers are off: half of 1 / 32000
    of the largest of 256 channels, and where they are rotated the fp32
    butterflies' 1e-5 of it (the gate of the other rotations), each times the
    weights' magnitudes.
"""
import pytest
import torch

import rotated_w4a4_quantized_b200 as cr
from tests import decoding_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from rotated_w4a4_quantized_b200 import build
    build.build()


def draw(M, K, N, scale_group, seed, bias=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g).to(torch.bfloat16)
    c = torch.randint(-7, 8, (N, K), generator=g)
    qw = ((c[:, 1::2] & 15) << 4 | (c[:, 0::2] & 15)).to(torch.uint8)
    sg = (torch.rand(N, K // scale_group, generator=g) * 0.02 + 0.001).to(torch.bfloat16)
    b = torch.randn(N, generator=g).to(torch.bfloat16) if bias else None
    return x, qw, sg, b


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def check(y, x, qw, sg, b, group=0):
    K = x.shape[1]
    xr = ref.rotate(x.double(), group)
    t, l1 = ref.linear(xr, qw, sg, b)
    w = (ref.unpack(qw).double() * sg.double().repeat_interleave(K // sg.shape[1], 1)).abs()
    pad = -K % 256
    top = torch.nn.functional.pad(xr.abs(), (0, pad)).unflatten(1, (-1, 256)).amax(-1)
    per_block = torch.nn.functional.pad(w, (0, pad)).unflatten(1, (-1, 256)).sum(-1)
    off = (0.5 / 32000 * (1 + 1e-3) + (1e-5 if group else 0.0)) * top @ per_block.T
    tol = 2.0 ** -8 * t.abs() + 2.0 ** -17 * l1 + off
    err = (y.cpu().double() - t).abs()
    assert bool((err <= tol).all()), f"{(err > tol).sum()} outputs off, worst {(err - tol).max()}"


@pytest.mark.parametrize("scale_group", [32, 64, 128])
@pytest.mark.parametrize("M,K,N", [
    (1, 128, 1), (1, 128, 16), (1, 256, 17), (2, 384, 149), (3, 1024, 1024), (8, 640, 300),
    (9, 1152, 260), (15, 2048, 2369), (16, 4096, 500), (17, 512, 70), (33, 256, 129), (5, 12288, 190),
    (16, 16384, 40), (8, 32768, 20), (1, 32768, 2000)])
def test_product_matches_float64(M, K, N, scale_group):
    x, qw, sg, b = draw(M, K, N, scale_group, seed=M + K + N, bias=N % 2 == 0)
    xc, qc, sc, bc = cuda(x, qw, sg, b)
    check(cr.convrot_w4g_linear(xc, qc, sc, bc, 0, scale_group), x, qw, sg, b)


@pytest.mark.parametrize("K,scale_group", [(64, 32), (64, 64), (192, 64), (320, 32), (960, 64)])
def test_short_and_odd_rows(K, scale_group):
    x, qw, sg, b = draw(4, K, 333, scale_group, seed=K)
    xc, qc, sc, bc = cuda(x, qw, sg, b)
    check(cr.convrot_w4g_linear(xc, qc, sc, bc, 0, scale_group), x, qw, sg, b)


def test_many_rows_of_weights():
    """More rows than one wave of CTAs holds."""
    x, qw, sg, b = draw(2, 128, 148 * 128 + 77, 64, seed=5)
    xc, qc, sc, bc = cuda(x, qw, sg, b)
    check(cr.convrot_w4g_linear(xc, qc, sc, bc, 0, 64), x, qw, sg, b)


@pytest.mark.parametrize("group", [64, 256])
@pytest.mark.parametrize("M,K,N,scale_group", [(1, 256, 40, 32), (1, 4096, 300, 64), (4, 1024, 77, 64),
                                               (7, 2816, 149, 128), (16, 4096, 200, 128), (40, 512, 65, 32),
                                               (3, 32768, 24, 64), (300, 256, 33, 64)])
def test_whole_layer_matches_float64(M, K, N, scale_group, group):
    x, qw, sg, b = draw(M, K, N, scale_group, seed=3 * M + K + N)
    check(cr.convrot_w4g_linear(*cuda(x, qw, sg, b), group, scale_group), x, qw, sg, b, group)


@pytest.mark.parametrize("M,K", [(1, 16384), (4, 4096), (16, 1024), (2, 8256)])
def test_prepared_and_own_numbers_agree(M, K):
    """The rows of a call whose CTAs make their own numbers, and of one with so
    many rows that they are prepared: the same to the last bit where as many
    tokens share a product."""
    x, qw, sg, b = draw(M, K, 100, 64, seed=K)
    y = cr.convrot_w4g_linear(*cuda(x, qw, sg, b), 64, 64)
    many = torch.cat([x] * (48 // M))
    assert cr.convrot_w4g_workspace_size(M, K) == 0 or K == 8256
    assert cr.convrot_w4g_workspace_size(len(many), K) > 0
    z = cr.convrot_w4g_linear(*cuda(many, qw, sg, b), 64, 64)
    for i in range(48 // M):
        if M == 16:
            assert torch.equal(z[i * M:(i + 1) * M], y)
        check(z[i * M:(i + 1) * M], x, qw, sg, b, 64)


def test_outliers_stay_in_their_block():
    """A channel 10^5 times the others costs precision in its 256 channels only,
    and weights of zero there leave none of it."""
    x, qw, sg, b = draw(3, 1024, 64, 64, seed=11)
    x[:, 300] = 1e5
    qw[:, 128:256] = 0
    check(cr.convrot_w4g_linear(*cuda(x, qw, sg, b), 0, 64), x, qw, sg, b)


@pytest.mark.parametrize("group", [0, 64, 256])
@pytest.mark.parametrize("scale_group", [32, 64, 128])
@pytest.mark.parametrize("N,K", [(1, 256), (5, 768), (33, 4096), (130, 1024)])
def test_quantized_weights_are_the_definition(N, K, scale_group, group):
    g = torch.Generator().manual_seed(N + K)
    w = (torch.randn(N, K, generator=g) * 0.02).to(torch.bfloat16)
    w[0, :K // 2] = 0
    if N > 4:
        w[1] = 0
        w[2] *= 2.0 ** -110      # scales below 2^-100 count as 0
        w[3] *= 2.0 ** 90
    wc = w.cuda()
    qw, sg = cr.convrot_w4g_quantize_weight(wc, group, scale_group)
    y = cr.convrot_debug_rotate_f32(wc, group).cpu() if group else w.float()
    c, s = ref.quantize_blocks(y, scale_group)
    assert torch.equal(sg.cpu(), s)
    assert torch.equal(ref.unpack(qw.cpu()), c)


def test_group_scales_beat_row_scales():
    """One channel in a hundred 20 times larger and no rotation to spread it:
    a scale for every 32 channels leaves less than half of a row scale's error
    (its blocks' largest values are smaller by far in most blocks)."""
    g = torch.Generator().manual_seed(1)
    w = torch.randn(64, 4096, generator=g) * 0.02
    w[:, torch.randperm(4096, generator=g)[:40]] *= 20
    w = w.to(torch.bfloat16)
    qw, sg = cr.convrot_w4g_quantize_weight(w.cuda(), 0, 32)
    mine = ref.unpack(qw.cpu()).double() * sg.cpu().double().repeat_interleave(32, 1)
    c, s = ref.quantize_blocks(w.float(), 4096)
    row = c.double() * s.double().repeat_interleave(4096, 1)
    assert (mine - w.double()).norm() < 0.5 * (row - w.double()).norm()


def test_rounds_once_at_the_end():
    """A product of 1 + 2^-7 and 1, times a scale of 1, plus a bias that cancels it."""
    x = torch.zeros(1, 64, dtype=torch.bfloat16)
    x[0, 3] = 1 + 2.0 ** -7
    qw = torch.zeros(16, 32, dtype=torch.uint8)
    qw[:, 1] = 0x70                                     # channel 3: 7
    sg = torch.ones(16, 1, dtype=torch.bfloat16)
    b = torch.full((16,), -7.0, dtype=torch.bfloat16)
    y = cr.convrot_w4g_linear(*cuda(x, qw, sg, b), 0, 64)
    assert torch.equal(y.cpu().float(), torch.full((1, 16), 7 * 2.0 ** -7))


def test_every_code_and_position():
    """One-hot rows read each weight back: 7 values a code, every channel."""
    K, N = 512, 20
    c = (torch.arange(N)[:, None] * 5 + torch.arange(K)[None, :] * 3) % 15 - 7
    qw = ((c[:, 1::2] & 15) << 4 | (c[:, 0::2] & 15)).to(torch.uint8).cuda()
    sg = torch.ones(N, K // 32, dtype=torch.bfloat16, device="cuda")
    eye = torch.eye(K, dtype=torch.bfloat16, device="cuda")
    y = cr.convrot_w4g_linear(eye, qw, sg, None, 0, 32)
    assert torch.equal(y.cpu().T.long(), c)


def test_nonfinite_activations_stay_in_their_row():
    x, qw, sg, b = draw(9, 256, 50, 64, seed=2)
    x[3, 7] = float("nan")
    x[8, 0] = float("inf")
    y = cr.convrot_w4g_linear(*cuda(x, qw, sg, b), 0, 64).cpu()
    clean = [i for i in range(9) if i not in (3, 8)]
    check(y[clean], x[clean], qw, sg, b)
    assert bool(y[3].isnan().all())


def test_empty_and_given_buffers():
    x, qw, sg, b = cuda(*draw(5, 256, 100, 64, seed=4))
    assert cr.convrot_w4g_linear(x[:0], qw, sg, b, 64, 64).shape == (0, 100)
    assert cr.convrot_w4g_linear(x, qw[:0], sg[:0], None, 64, 64).shape == (5, 0)
    want = cr.convrot_w4g_linear(x, qw, sg, b, 64, 64)
    out = torch.full((7, 100), 3.0, dtype=torch.bfloat16, device="cuda")
    got = cr.convrot_w4g_linear(x, qw, sg, b, 64, 64, out=out[:5])
    assert got.data_ptr() == out.data_ptr() and torch.equal(got, want)
    assert bool((out[5:] == 3.0).all())
    x = torch.cat([x] * 20)
    want = cr.convrot_w4g_linear(x, qw, sg, b, 64, 64)
    ws = torch.full((cr.convrot_w4g_workspace_size(100, 256),), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(cr.convrot_w4g_linear(x, qw, sg, b, 64, 64, workspace=ws), want)


def test_streams_and_captured_replays():
    x, qw, sg, b = cuda(*draw(3, 1024, 500, 64, seed=6))
    want = cr.convrot_w4g_linear(x, qw, sg, b, 256, 64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [cr.convrot_w4g_linear(x, qw, sg, b, 256, 64, stream=side) for _ in range(4)]
    with torch.cuda.stream(side):
        got.append(cr.convrot_w4g_linear(x, qw, sg, b, 256, 64))
    side.synchronize()
    assert all(torch.equal(y, want) for y in got)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cr.convrot_w4g_linear(x, qw, sg, b, 256, 64, out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_offsets_beyond_32_bits():
    """More than 2^32 bytes of codes: the last rows equal a small call's."""
    N, K = (1 << 32) // 16384 + 1000, 32768
    qw = torch.empty(N, K // 2, dtype=torch.uint8, device="cuda")
    sg = torch.full((N, K // 128), 0.01, dtype=torch.bfloat16, device="cuda")
    x, tail, tail_sg, _ = cuda(*draw(2, K, 900, 128, seed=8))
    qw[-900:] = tail
    sg[-900:] = tail_sg
    y = cr.convrot_w4g_linear(x, qw, sg, None, 64, 128)[:, -900:]
    z = cr.convrot_w4g_linear(x, tail, tail_sg, None, 64, 128)
    # (another number of rows a CTA: other parts of K, sums in another order)
    t, l1 = ref.linear(ref.rotate(x.cpu().double(), 64), tail.cpu(), tail_sg.cpu(), None)
    assert bool(((y - z).cpu().double().abs() <= 2.0 ** -7 * t.abs() + 2.0 ** -16 * l1).all())


def test_refusals_on_the_device():
    x, qw, sg, b = cuda(*draw(2, 256, 64, 64, seed=7))
    with pytest.raises(cr.ConvRotError, match="GROUP"):
        cr.convrot_w4g_linear(x, qw, sg, b, 32, 64)
    with pytest.raises(cr.ConvRotError, match="GROUP"):
        cr.convrot_w4g_linear(x, qw, sg, b, 64, 16)
    with pytest.raises(ValueError, match="sg has shape"):
        cr.convrot_w4g_linear(x, qw, sg, b, 64, 32)
    with pytest.raises(ValueError, match="contiguous"):
        cr.convrot_w4g_linear(x.T.contiguous().T, qw, sg, b, 64, 64)
    with pytest.raises(ValueError, match="workspace holds"):
        cr.convrot_w4g_linear(torch.cat([x] * 40), qw, sg, b, 64, 64, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        cr.convrot_w4g_linear(x, qw, sg.float(), b, 64, 64)
