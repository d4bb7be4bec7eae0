"""GPU tests of the attention over the INT4 cache where its softmax reference,
or the reference of its values' weights, moves: histories so long that every
warp takes several tiles, scores and scales of values far apart, keys that a
query must not see.

Gate, per row, against float64 (p: softmax weights of the row, s_j: scales of
its values, A: root of a sum of squares over channels):
  |o - t|_2 <= (1 + 2^-6) |sum_j p_j |v_j| (d_j + E)|_2     scores
               + (2^-11 + 2^-16) |sum_j p_j |v_j||_2         weights, sums
               + 2^-8 |t|_2                                  the result's rounding
               + sqrt(D) (8 5 2^-23 sum_j p_j s_j + 7 2^-29 n max_j p_j s_j)
with d_j = expm1 of what score j may be off (decoding_ref.attention adds that
up) and E = sum_j p_j d_j for the softmax's sum; (1 + 2^-6) takes their second
order.  A weight is rounded to f16 (2^-11); one below the f16 range is off by at
most half a step, 2^-25, where the row's largest weight so far is at least
2^6 / 2^0.1, so by less than 2^-29 of the largest p_j s_j, times a code of 7, for
each of n keys.  The offset of 8 that the codes carry comes and goes in fp32.
Nothing here depends on a key that the row does not see.
"""
import math

import pytest
import torch

import rotated_w4a4_quantized_b200 as cr
from tests import decoding_ref as ref

pytestmark = pytest.mark.gpu

PAGE = 16


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from rotated_w4a4_quantized_b200 import build
    build.build()


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert cr.convrot_kv4_check_device_error() == 0


def pack(c):
    return ((c[..., 1::2] & 15) << 4 | (c[..., 0::2] & 15)).to(torch.uint8)


def paged(rows, page, order):
    """[H, n, ...] -> [pages, H, page, ...], the n rows in pages `order`."""
    H, n = rows.shape[:2]
    pages = len(order)
    out = torch.zeros(H, pages * page, *rows.shape[2:], dtype=rows.dtype)
    out[:, :n] = rows
    out = out.unflatten(1, (pages, page)).transpose(0, 1)
    placed = torch.empty_like(out)
    placed[order] = out
    return placed.contiguous()


class Shaped:
    """One history of n tokens whose scores are chosen: the rotated query is 8
    in channel 0 and 0 elsewhere, the keys are +-7 there, so that with a scale of
    1/8 a key's score is +-7 times its scale.  scores [H, n] in units of log2,
    scales [H, n] of the values, codes [H, n, D] of the values."""

    def __init__(self, scores, scales, codes, page=PAGE, seed=0):
        H, n, D = codes.shape
        kc = torch.zeros(H, n, D, dtype=torch.int64)
        kc[:, :, 0] = 7 * torch.sign(scores).long()
        self.ks = (scores.abs() * math.log(2) / 7).to(torch.bfloat16)
        self.vs = scales.to(torch.bfloat16)
        self.kc, self.vc, self.n, self.D, self.H, self.page = kc, codes, n, D, H, page
        pages = -(-n // page)
        self.order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))
        self.cache = cr.Kv4Cache(*[paged(t, page, self.order).cuda() for t in (pack(kc), self.ks, pack(codes), self.vs)])
        self.scale, self.group = 0.125, 64

    def queries(self, T, G):
        """bf16 [T, H G, D]: rotated, channel 0 is 8."""
        e = torch.zeros(self.D, dtype=torch.float64)
        e[0] = 8.0
        q = ref.rotate(e, self.group).to(torch.bfloat16)
        assert torch.equal(ref.rotate(q.double(), self.group), e)
        return q.expand(T, self.H * G, self.D).contiguous()

    def run(self, q, requests, lens=None, table=None, cu=None):
        i32 = dict(dtype=torch.int32, device="cuda")
        new = q.shape[0] // requests
        table = self.order.int() if table is None else table
        lens = torch.full((requests,), self.n, **i32) if lens is None else lens
        cu = torch.arange(0, q.shape[0] + 1, new, **i32) if cu is None else cu
        return cr.convrot_kv4_attention(q.cuda(), self.cache, table.cuda().expand(requests, -1).contiguous(), lens, cu,
                                        self.scale, self.group).cpu()

    def row(self, q, h, seen):
        """(t, allowance) of one query (bf16 [D]) of shared head h."""
        kk = self.kc[h, seen].double() * self.ks[h, seen].double()[:, None]
        sv = self.vs[h, seen].double()
        vv = self.vc[h, seen].double() * sv[:, None]
        qr = ref.rotate(q.double(), self.group)
        s = kk @ qr * self.scale
        p = torch.softmax(s, 0)
        t = ref.rotate(p @ vv, self.group)
        l1 = kk.abs() @ (qr.abs() * 2.0 ** -17 + qr.abs().max() * (2.0 ** -16 + 1e-5)) * abs(self.scale)
        d = torch.expm1(l1 + s.abs() * 2.0 ** -22 + 2.0 ** -22)
        E = float(p @ d)
        terms = p @ vv.abs()
        allow = ((1 + 2.0 ** -6) * ((p * (d + E)) @ vv.abs()).norm() + (2.0 ** -11 + 2.0 ** -16) * terms.norm()
                 + 2.0 ** -8 * t.norm()
                 + self.D ** 0.5 * (8 * 5 * 2.0 ** -23 * (p @ sv) + 7 * 2.0 ** -29 * len(s) * (p * sv).max()))
        return t, float(allow)


def check_rows(out, want, what=""):
    """Every row of out [T, D] against (t, allowance)."""
    t, allow = want
    err = (out.double() - t).norm(dim=-1)
    assert bool((err <= allow).all()), f"{what}: {int((err > allow).sum())} of {len(err)} rows off, worst {float(err.max())}, allowed {allow}"


def long_history(D, n=9000, heads=8, seed=1):
    """Scores and values of 8 heads and 9000 tokens: for 8 requests more than
    four tiles a warp."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(-7, 8, (heads, n, D), generator=g)
    scales = (torch.rand(heads, n, generator=g) + 0.5) * 0.4
    scores = torch.randn(heads, n, generator=g) * 2
    return scores, scales, codes


# heads that share a head -> rows of a block: 4, 4, 8 and (but for D = 256) 16
FORMS = [(64, 1), (64, 8), (64, 16), (128, 4), (128, 6), (128, 16), (256, 2), (256, 8)]


def check_long(a, G, requests=8):
    q = a.queries(requests, G)
    out = a.run(q, requests)
    everything = torch.ones(a.n, dtype=torch.bool)
    for h in range(a.H):
        want = a.row(q[0, 0], h, everything)
        check_rows(out[:, h * G:(h + 1) * G].reshape(-1, a.D), want, f"head {h}")


@pytest.mark.parametrize("D,G", FORMS)
def test_several_tiles_a_warp(D, G):
    check_long(Shaped(*long_history(D)), G)


@pytest.mark.parametrize("D,G", FORMS)
def test_reference_moves_while_some_keys_underflow(D, G):
    """In head h, the keys h and h + 8 of every 16 are 2^-200 of the others, so
    that the lanes that hold them have no softmax sum of their own; then a key
    2^9 above all before it moves the reference."""
    scores, scales, codes = long_history(D)
    j = torch.arange(scores.shape[1])
    tile = j // 64
    scores[:] = 0.0
    codes[:] = 7
    late = ((tile // 4) % 4 == 3) & (j % 64 == 33)     # one key a tile, every fourth round of tiles
    for h in range(8):
        scores[h, j % 8 == h] = -200.0
    scores[:, late] = 9.5
    codes[:, late] = -7
    check_long(Shaped(scores, scales, codes), G)


@pytest.mark.parametrize("D,G", FORMS)
def test_value_scales_rise_and_fall(D, G):
    """The values' scales move by 2^24 up and down along the history, the
    scores against them, so that keys of all scales count."""
    scores, scales, codes = long_history(D)
    tile = torch.arange(scores.shape[1]) // 64
    for h in range(8):
        wave = 12 * torch.sin(tile / (5.0 + 3 * h))
        scales[h] *= 2.0 ** wave.round()
        if h & 1:
            scores[h] -= wave
    check_long(Shaped(scores, scales, codes), G)


@pytest.mark.parametrize("ratio", [2.0 ** 24, 2.0 ** 40, 2.0 ** 100])
@pytest.mark.parametrize("D,G", FORMS)
def test_a_hidden_value_of_any_scale_changes_nothing(D, G, ratio):
    """The newest of three tokens has a value far above the others; the two
    queries before it must not see it."""
    g = torch.Generator().manual_seed(D + G)
    for n in (3, 40, 64, 700):
        codes = torch.randint(-7, 8, (2, n, D), generator=g)
        scales = (torch.rand(2, n, generator=g) + 0.5) * 0.4
        scores = torch.randn(2, n, generator=g)
        scales[:, -1] *= ratio
        a = Shaped(scores, scales, codes)
        q = a.queries(3, G)
        out = a.run(q, 1)
        for i in range(3):
            seen = torch.arange(n) <= n - 3 + i
            for h in range(2):
                check_rows(out[i, h * G:(h + 1) * G], a.row(q[i, h * G], h, seen), f"n {n}, query {i}, head {h}")


@pytest.mark.parametrize("D,G", FORMS)
@pytest.mark.parametrize("n,where", [(64, 5), (1500, 3), (9000, 70), (9000, 4500)])
def test_a_large_value_of_no_weight_changes_nothing(D, G, n, where):
    """A value 2^60 times the others whose softmax weight is 2^-110 of theirs."""
    scores, scales, codes = long_history(D, n)
    scores *= 0.5
    scales[:, where] *= 2.0 ** 60
    scores[:, where] = -110.0
    check_long(Shaped(scores, scales, codes), G)


@pytest.mark.parametrize("D,G", FORMS)
@pytest.mark.parametrize("n,where", [(64, 60), (1500, 1400), (9000, 70), (9000, 4500), (9000, 8999)])
def test_a_small_value_of_all_the_weight_is_the_result(D, G, n, where):
    """A value 2^-60 times the others, with 2^110 times their softmax weight: it
    is the result, not what is left of the others."""
    scores, scales, codes = long_history(D, n)
    scores *= 0.5
    scales[:, where] *= 2.0 ** -60
    scores[:, where] = 110.0
    check_long(Shaped(scores, scales, codes), G)


@pytest.mark.parametrize("D,G", FORMS)
@pytest.mark.parametrize("n", [50, 9000])
def test_values_of_zero(D, G, n):
    """Scales of zero: of the keys that weigh most, and of all of them."""
    scores, scales, codes = long_history(D, n)
    scales[:4, ::3] = 0.0
    scores[:4, ::3] += 30.0
    scales[4:] = 0.0
    check_long(Shaped(scores, scales, codes), G)


@pytest.mark.parametrize("D,G", FORMS)
@pytest.mark.parametrize("scale", [2.0 ** -98, 2.0 ** 60, 2.0 ** 118])
def test_values_of_extreme_scales(D, G, scale):
    """The sums over many keys of the largest and the smallest values."""
    scores, scales, codes = long_history(D)
    scales[:] = (scales * scale)
    codes = codes.abs()
    check_long(Shaped(scores, scales, codes), G)


@pytest.mark.parametrize("D,G", [(64, 1), (128, 4), (128, 16), (256, 8)])
def test_missing_pages_in_later_tiles(D, G):
    """Pages outside the cache in the later tiles of the warps: their keys are
    as if they were not there."""
    a = Shaped(*long_history(D))
    table = a.order.int().clone()
    missing = torch.arange(len(table)) % 37 == 29
    table[missing] = torch.where(torch.arange(int(missing.sum())) % 2 == 0, -3, len(table) + 5).int()
    q = a.queries(8, G)
    out = a.run(q, 8, table=table)
    assert cr.convrot_kv4_check_device_error() == 12
    seen = ~missing.repeat_interleave(PAGE)[:a.n]
    for h in range(a.H):
        check_rows(out[:, h * G:(h + 1) * G].reshape(-1, D), a.row(q[0, 0], h, seen), f"head {h}")


@pytest.mark.parametrize("D,G", [(64, 2), (128, 4), (256, 2)])
def test_a_prompt_among_long_histories(D, G):
    """130 new tokens of one request between single tokens of others."""
    a = Shaped(*long_history(D, 6000, heads=2))
    new = [1, 130, 1, 0, 1]
    lens, i32 = [6000, 5000, 17, 40, 6000], dict(dtype=torch.int32, device="cuda")
    q = a.queries(sum(new), G)
    out = a.run(q, 5, lens=torch.tensor(lens, **i32), cu=torch.tensor([0, 1, 131, 132, 132, 133], **i32))
    j = torch.arange(a.n)
    for row, (b, i) in enumerate((b, i) for b, n in enumerate(new) for i in range(n)):
        if b == 1 and i % 43:
            continue
        for h in range(2):
            check_rows(out[row, h * G:(h + 1) * G], a.row(q[0, 0], h, j <= lens[b] - new[b] + i), f"request {b}, query {i}")


@pytest.mark.parametrize("left", [-2.0 ** -100, -1.0, float("nan"), float("-inf"), 1e38])
@pytest.mark.parametrize("D,G", FORMS)
def test_what_lies_behind_the_end_hides_no_larger_scale(D, G, left):
    """The scales of the last tile's values are far above all before them; beside
    them, behind the request's end, lies whatever the memory held."""
    scores, scales, codes = long_history(D)
    n = scores.shape[1]
    assert n % 64 == 40
    scales[:, n - 40:] *= 2.0 ** 14
    a = Shaped(scores, scales, codes)
    a.cache.v_scales[a.order[-1], :, n % PAGE:] = left
    a.cache.k_scales[a.order[-1], :, n % PAGE:] = left
    check_long(a, G)
