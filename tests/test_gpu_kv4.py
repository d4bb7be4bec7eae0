"""GPU tests of the INT4 cache of keys and values (include/convrot_kv4.h).

Gates:
  - append: codes and scales equal, bit for bit, to the definition evaluated
    in fp32 on the GPU's own rotated rows; nothing else in the cache changes;
  - read: (codes s) R^T rounded once to bf16: exact, so bit-equal;
  - plan: whole numbers, equal to a list-by-list restatement;
  - attention, per row: |o - t|_2 <= e |A|_2 + 2^-8 |t|_2, where A_d = sum_j
    p_j |v_jd| bounds the terms of every rotated output value, the rotation
    back keeps 2-norms, the output's rounding is off by 2^-8 of each value, and
      e = expm1(2 ds) + 2^-11 + 2^-16:
    each weight p_j is off by at most the factor exp(2 ds) for scores off by
    ds (decoding_ref.attention adds ds up: 16-bit queries, fp32 rotation, exp2), its product with the value's scale is rounded to f16 (2^-11), and
    the fp32 sums and joins of parts stay below 2^-16; two small terms for the
    offset that the values' codes carry and for weights below the f16 range.
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


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert cr.convrot_kv4_check_device_error() == 0


def make_cache(pages, heads, page, D, seed, scale=0.4):
    g = torch.Generator().manual_seed(seed)
    c = torch.randint(-7, 8, (2, pages, heads, page, D), generator=g)
    codes = ((c[..., 1::2] & 15) << 4 | (c[..., 0::2] & 15)).to(torch.uint8)
    s = ((torch.rand(2, pages, heads, page, generator=g) + 0.5) * scale).to(torch.bfloat16)
    return cr.Kv4Cache(codes[0], s[0], codes[1], s[1])


def to(cache):
    return cr.Kv4Cache(*[t.cuda() for t in cache])


# ---------------------------------------------------------------- append, read

@pytest.mark.parametrize("D,group", [(64, 64), (128, 64), (256, 64), (256, 256)])
@pytest.mark.parametrize("T,heads,page", [(1, 1, 16), (5, 3, 16), (33, 8, 32), (300, 2, 64), (70, 5, 256)])
def test_append_is_the_definition_and_read_is_exact(T, heads, page, D, group):
    g = torch.Generator().manual_seed(T + D + page)
    k, v = (torch.randn(T, heads, D, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    k[0, 0] = 0
    if T > 4:
        v[1] *= 1000.0
        v[2] *= 2.0 ** -120
    pages = -(-T // page) + 2
    slots = torch.randperm(pages * page, generator=g)[:T]
    if T > 4:
        slots[3] = -1
    before = make_cache(pages, heads, page, D, seed=T)
    cache = to(before)
    cr.convrot_kv4_append(k, v, cache, slots.cuda(), group)
    after = [t.cpu() for t in cache]
    want = [t.clone() for t in before]
    for x, codes, scales in ((k, want[0], want[1]), (v, want[2], want[3])):
        y = cr.convrot_debug_rotate_f32(x.reshape(T * heads, D), group).cpu()
        c, s = ref.quantize_blocks(y, D)
        c, s = c.reshape(T, heads, D), s.reshape(T, heads)
        packed = ((c[..., 1::2] & 15) << 4 | (c[..., 0::2] & 15)).to(torch.uint8)
        for t in range(T):
            if slots[t] >= 0:
                codes[slots[t] // page, :, slots[t] % page] = packed[t]
                scales[slots[t] // page, :, slots[t] % page] = s[t]
    for a, w in zip(after, want):
        assert torch.equal(a, w)
    kr, vr = cr.convrot_kv4_read(cache, slots.cuda(), group)
    for got, codes, scales in ((kr, want[0], want[1]), (vr, want[2], want[3])):
        at = slots.clamp(min=0)
        y = ref.unpack(codes[at // page, :, at % page]).double() * scales[at // page, :, at % page].double()[..., None]
        y = ref.rotate(y, group).float().to(torch.bfloat16)
        y[slots < 0] = 0
        assert torch.equal(got.cpu(), y)


def test_append_takes_columns_of_a_fused_projection():
    g = torch.Generator().manual_seed(3)
    T, heads, D = 9, 4, 128
    qkv = torch.randn(T, 6 * heads * D + 8, generator=g).to(torch.bfloat16).cuda()
    k = qkv[:, 4 * heads * D:5 * heads * D].unflatten(1, (heads, D))
    v = qkv[:, 5 * heads * D:6 * heads * D].unflatten(1, (heads, D))
    slots = torch.arange(T).cuda() + 7
    one, two = (to(make_cache(3, heads, 16, D, seed=1)) for _ in range(2))
    cr.convrot_kv4_append(k, v, one, slots, 64)
    cr.convrot_kv4_append(k.contiguous(), v.contiguous(), two, slots, 64)
    assert all(torch.equal(a, b) for a, b in zip(one, two))


@pytest.mark.parametrize("heads,D,group", [(8, 64, 64), (5, 128, 64), (3, 256, 64), (3, 256, 256)])
def test_append_of_many_rows_is_the_append_of_few(heads, D, group):
    """A call of many rows spreads a row over fewer threads than a call of
    few: the bits are the same."""
    T, page = 4000000 // (heads * D) | 1, 64
    g = torch.Generator(device="cuda").manual_seed(D + heads)
    kv = torch.empty(T, 2 * heads * D + 8, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    kv[T // 2, :heads * D] = 0
    kv[T // 3, 7] = float("inf")
    k, v = kv[:, :heads * D].unflatten(1, (heads, D)), kv[:, heads * D:2 * heads * D].unflatten(1, (heads, D))
    pages = T // page + 3
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T]
    slots[5::97] = -1
    one, two = (to(make_cache(1, heads, page, D, seed=1)) for _ in range(2))
    one, two = (cr.Kv4Cache(*[t.expand(pages, *t.shape[1:]).contiguous() for t in c]) for c in (one, two))
    cr.convrot_kv4_append(k, v, one, slots, group)
    step = -(-T // 14) * 2                     # (slots begin on 16 bytes)
    for t in range(0, T, step):
        cr.convrot_kv4_append(k[t:t + step], v[t:t + step], two, slots[t:t + step], group)
    for a, b in zip(one, two):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_append_keeps_nonfinite_rows_to_themselves():
    k = torch.randn(3, 2, 64).to(torch.bfloat16).cuda()
    v = k.clone()
    k[1, 0, 5] = float("nan")
    k[2, 1, 5] = float("inf")
    cache = cr.convrot_kv4_new_cache(1, 2, 16, 64, "cuda")
    cr.convrot_kv4_append(k, v, cache, torch.arange(3).cuda(), 64)
    finite = cache.k_scales[0].isfinite()
    bad = [(0, 1), (1, 2)]
    assert [(h, t) for h in range(2) for t in range(3) if not finite[h, t]] == bad
    assert bool(cache.v_scales.isfinite().all())


def test_slots_outside_the_cache_are_skipped_and_reported():
    k = torch.randn(3, 2, 64).to(torch.bfloat16).cuda()
    before = make_cache(2, 2, 16, 64, seed=9)
    cache = to(before)
    slots = torch.tensor([32, 4, 1 << 40]).cuda()          # 2 pages of 16: 0 .. 31
    cr.convrot_kv4_append(k, k, cache, slots, 64)
    assert cr.convrot_kv4_check_device_error() == 12
    keep = torch.arange(16) != 4
    assert torch.equal(cache.k_codes.cpu()[0][:, keep], before.k_codes[0][:, keep])
    assert torch.equal(cache.k_codes.cpu()[1], before.k_codes[1])
    kr, vr = cr.convrot_kv4_read(cache, slots, 64)
    assert cr.convrot_kv4_check_device_error() == 12
    assert not kr[0].any() and not vr[2].any() and kr[1].any()


# ---------------------------------------------------------------- plan

def run_plan(cached, new, table, free, count, page, max_tokens):
    i32 = dict(dtype=torch.int32, device="cuda")
    tab, fr = torch.tensor(table, **i32).reshape(len(cached), len(table[0]) if table else 2), torch.tensor(free, **i32)
    args = (torch.tensor(cached, **i32), torch.tensor(new, **i32), tab, fr, torch.tensor([count], **i32), page, max_tokens)
    p = cr.convrot_kv4_plan(*args)
    again = cr.convrot_kv4_plan(*args)
    got = {n: getattr(p, n).tolist() for n in ("seq_lens", "cu_q", "slots", "positions", "result")}
    assert got == {n: getattr(again, n).tolist() for n in got}, "a second call on the same inputs differs"
    assert p.free_count.tolist() == got["result"][:1] and p.status.tolist() == got["result"][3:]
    return got, tab.tolist(), fr.tolist()


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("B,page,most,new_most,pad", [(1, 16, 4, 1, 0), (3, 16, 9, 40, 3), (64, 16, 20, 1, 0),
                                                      (200, 32, 12, 90, 17), (1500, 64, 5, 60, 1),
                                                      (8192, 16, 2, 3, 100), (5, 256, 40, 4000, 5)])
def test_plan_matches_lists(B, page, most, new_most, pad, seed):
    g = torch.Generator().manual_seed(seed * 100 + B)
    new = torch.randint(-1, new_most + 1, (B,), generator=g).tolist()
    cached = [int(torch.randint(0, most * page - max(n, 0) + 1, (1,), generator=g)) if n <= most * page else 0 for n in new]
    ids = torch.randperm(B * most + 4000, generator=g).tolist()
    table = [ids[b * most:(b + 1) * most] for b in range(B)]
    count = sum(-(-max(n, 0) // page) + 1 for n in new)
    free = (ids[B * most:] * (count // 4000 + 2))[:count] + [-7] * (B * most)
    tokens = sum(max(n, 0) for n in new) + pad
    want_table, want_free = [list(r) for r in table], list(free)
    want = ref.plan(cached, new, want_table, want_free, count, page, tokens)
    got, got_table, got_free = run_plan(cached, new, table, free, count, page, tokens)
    assert got == want and got_table == want_table and got_free == want_free


PLANS = [
    # status, cached, new, table width, free pages, count, page, max_tokens
    (1, [16, 3], [1, 14], 3, [8], 1, 16, 20),
    (0, [16, 3], [1, 13], 3, [8], 1, 16, 20),
    (2, [16, 48], [1, 1], 3, [8, 9], 2, 16, 20),
    (2, [16, 0], [1, 2 ** 31 - 1], 3, [8, 9], 2, 16, 20),
    (3, [16, 3], [5, 6], 3, [8, 9], 2, 16, 10),
    (4, [-1, 3], [5, 6], 3, [8, 9], 2, 16, 20),
    (4, [49, 3], [-1, 6], 3, [8, 9], 2, 16, 20),
    (4, [1, 3], [1, 6], 3, [8, 9], 3, 16, 20),
    (4, [1, 3], [1, 6], 3, [8, 9], -1, 16, 20),
    (4, [33, 3], [-1, 6], 3, [8, 9, 0], 2, 16, 20),       # three pages come back, room for one
    (0, [33, 3], [-1, 6], 3, [8, 9, 0, 0, 0], 2, 16, 20),
    (0, [0, 0], [0, 0], 3, [8, 9], 2, 16, 0),
    (0, [0, 0], [-1, -1], 3, [], 0, 16, 4),
    (0, [33, 20], [-1, 20], 3, [0] * 5, 0, 16, 20),       # only returned pages to take
]


@pytest.mark.parametrize("case", PLANS)
def test_plan_edges_and_refusals_change_nothing(case):
    status, cached, new, most, free, count, page, tokens = case
    table = [[10 * b + j for j in range(most)] for b in range(2)]
    want_table, want_free = [list(r) for r in table], list(free)
    want = ref.plan(cached, new, want_table, want_free, count, page, tokens)
    got, got_table, got_free = run_plan(cached, new, table, free, count, page, tokens)
    assert want["result"][3] == status
    assert got == want and got_table == want_table and got_free == want_free


def test_plan_without_requests():
    got, _, _ = run_plan([], [], [], [5, 6], 2, 16, 3)
    assert got == dict(seq_lens=[], cu_q=[0], slots=[-1] * 3, positions=[-1] * 3, result=[2, 0, 0, 0])


# ---------------------------------------------------------------- attention

def setup(lens, new, heads, kv_heads, D, page, seed, spread=1.5, extra=0):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    most = max(1, max(-(-n // page) for n in lens)) + extra
    cache = make_cache(B * most + 1, kv_heads, page, D, seed)
    table = torch.randperm(B * most + 1, generator=g)[:B * most].reshape(B, most).int()
    for b, n in enumerate(lens):
        table[b, -(-n // page):] = -1                      # entries that are never read
    cu = torch.tensor([0] + new).cumsum(0).int()
    q = (torch.randn(int(cu[-1]), heads, D, generator=g) * spread).to(torch.bfloat16)
    return q, cache, table, torch.tensor(lens).int(), cu


def run_attention(q, cache, table, lens, cu, scale, group, **kw):
    return cr.convrot_kv4_attention(q.cuda(), to(cache), table.cuda(), lens.cuda(), cu.cuda(), scale, group, **kw)


def check(out, q, cache, table, lens, cu, scale, group, dead=()):
    t, allow = ref.attention(q, cache, table, lens, cu, scale, group, dead)
    err = (out.cpu().double() - t).norm(dim=-1)
    assert bool((err <= allow).all()), f"{int((err > allow).sum())} rows off, worst {(err - allow).max()} of {allow.max()}"


@pytest.mark.parametrize("D,group", [(64, 64), (128, 64), (256, 64), (256, 256)])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (4, 1), (6, 2), (16, 1), (14, 2)])
def test_decode_shapes(D, group, heads, kv_heads):
    lens = [1, 15, 16, 17, 63, 64, 65, 200]
    a = setup(lens, [1] * 8, heads, kv_heads, D, 16, seed=D + heads)
    check(run_attention(*a, D ** -0.5, group), *a, D ** -0.5, group)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_pages_end_inside_tiles(page):
    lens = [page - 1, page, page + 1, 2 * page + 7, 1000, 5]
    a = setup(lens, [1] * 6, 8, 2, 128, page, seed=page, extra=2)
    check(run_attention(*a, 128 ** -0.5, 64), *a, 128 ** -0.5, 64)


@pytest.mark.parametrize("D,group", [(64, 64), (128, 64), (256, 256)])
@pytest.mark.parametrize("new", [[2, 2, 2], [5, 1, 3], [7, 0, 40], [33, 33, 33], [0, 0, 1], [1, 70, 0]])
def test_several_new_tokens(new, D, group):
    lens = [130, 64, 71]
    lens = [max(n, m) for n, m in zip(lens, new)]
    a = setup(lens, new, 6, 2, D, 32, seed=sum(new))
    check(run_attention(*a, D ** -0.5, group), *a, D ** -0.5, group)


def test_long_histories_are_split_and_joined():
    lens = [9000, 1, 3333]
    a = setup(lens, [1, 1, 2], 4, 2, 64, 64, seed=8)
    check(run_attention(*a, 0.125, 64), *a, 0.125, 64)


def test_many_requests():
    lens = [(37 * b) % 190 for b in range(300)]
    a = setup(lens, [1] * 300, 2, 1, 64, 16, seed=8)
    check(run_attention(*a, 0.125, 64), *a, 0.125, 64)


def test_rows_that_see_nothing_are_zero():
    """No cached token, more queries than tokens, and a length of zero."""
    a = setup([0, 3, 20], [1, 5, 2], 4, 2, 128, 16, seed=2)
    out = run_attention(*a, 0.1, 64)
    assert not out[0].any() and not out[1:3].any() and out[3:].any()
    check(out, *a, 0.1, 64)


def test_hidden_keys_may_hold_anything():
    """Scales that are NaN or infinite behind the end of a request, and in keys
    that only a later query sees."""
    q, cache, table, lens, cu = setup([21, 40], [1, 3], 4, 2, 128, 16, seed=3)
    clean = run_attention(q, cache, table, lens, cu, 0.1, 64)
    for s in (cache.k_scales, cache.v_scales):
        s[table[0, 1], :, 5:] = float("nan")
        s[table[1, 2], :, 8:] = float("inf")
        s[table[1, 2], 0, 7] = float("nan")                # position 39: the last query's own
    out = run_attention(q, cache, table, lens, cu, 0.1, 64)
    keep = torch.ones(4, 4, dtype=torch.bool)
    keep[3, :2] = False
    assert torch.equal(out.cpu()[keep], clean.cpu()[keep])
    assert bool(out[3, :2].isnan().all())


def test_large_scores_stay_finite():
    """One key wins by far: scores of thousands, queries over eight decades."""
    q, cache, table, lens, cu = setup([100, 100, 100], [1, 1, 1], 2, 1, 128, 16, seed=4)
    q[0] *= 1000
    q[1] *= 1e-30
    q[2, :, ::7] *= 1e6
    for scale in (0.1, -0.1, 0.0):
        a = (q, cache, table, lens, cu)
        out = run_attention(*a, scale, 64)
        assert bool(out.isfinite().all())
    check(run_attention(q[1:2], cache, table[1:2], lens[1:2], cu[:2], 0.1, 64), q[1:2], cache, table[1:2], lens[1:2], cu[:2], 0.1, 64)


def test_large_and_small_value_scales():
    q, cache, table, lens, cu = setup([300], [1], 4, 1, 128, 16, seed=5)
    cache.v_scales[:, :, ::2] *= 2.0 ** 60
    cache.v_scales[:, :, 1::2] *= 2.0 ** -60
    a = (q, cache, table, lens, cu)
    check(run_attention(*a, 0.05, 64), *a, 0.05, 64)


def test_pages_outside_the_cache_are_hidden_and_reported():
    q, cache, table, lens, cu = setup([100, 50], [1, 2], 4, 2, 64, 16, seed=6)
    table[0, 2] = 1 << 20
    table[1, 0] = -5
    out = run_attention(q, cache, table, lens, cu, 0.125, 64)
    assert cr.convrot_kv4_check_device_error() == 12
    check(out, q, cache, table, lens, cu, 0.125, 64, dead=[(0, 2), (1, 0)])


def test_lengths_beyond_the_table_and_queries_beyond_q_are_cut():
    """Device data that contradict the shapes stay inside the buffers."""
    q, cache, table, lens, cu = setup([32, 32], [1, 1], 2, 1, 64, 16, seed=7)
    want = run_attention(q, cache, table, lens, cu, 0.125, 64)
    out = run_attention(q, cache, table, torch.tensor([1 << 30, 32]).int(), torch.tensor([0, 1, 50]).int(), 0.125, 64)
    assert torch.equal(out[:1], want[:1])
    out = run_attention(q, cache, table, torch.tensor([-4, 32]).int(), torch.tensor([-9, 0, 1]).int(), 0.125, 64)
    assert out.shape == want.shape


def test_rows_behind_the_last_request_are_left():
    q, cache, table, lens, cu = setup([40, 9], [1, 1], 4, 2, 128, 16, seed=9)
    pad = torch.cat([q, torch.full((5, 4, 128), float("nan"), dtype=torch.bfloat16)])
    out = torch.full((7, 4, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    got = run_attention(pad, cache, table, lens, cu, 0.1, 64, out=out)
    # (the number of rows, padding included, chooses the height of the row
    # blocks, so the sums' order may be another than without padding)
    check(got[:2], q, cache, table, lens, cu, 0.1, 64)
    assert bool((got[2:] == 3.0).all())


def test_queries_as_columns_of_a_fused_projection():
    q, cache, table, lens, cu = setup([40, 9, 30], [1, 2, 1], 4, 2, 128, 16, seed=10)
    wide = torch.randn(4, 4 * 128 + 512).to(torch.bfloat16)
    wide[:, :512] = q.reshape(4, 512)
    out = cr.convrot_kv4_attention(wide.cuda()[:, :512].unflatten(1, (4, 128)), to(cache), table.cuda(), lens.cuda(),
                                   cu.cuda(), 0.1, 64)
    assert torch.equal(out, run_attention(q, cache, table, lens, cu, 0.1, 64))


def test_workspace_needs_no_initialisation_and_can_be_shared_in_order():
    a = setup([5000, 700, 33], [1, 1, 1], 8, 2, 128, 64, seed=11)
    size = cr.convrot_kv4_attention_workspace_size(3, 3, 8, 2, 128, a[2].shape[1] * 64)
    want = run_attention(*a, 0.1, 64)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        assert torch.equal(run_attention(*a, 0.1, 64, workspace=ws), want)
    with pytest.raises(ValueError, match="workspace holds"):
        run_attention(*a, 0.1, 64, workspace=ws[:-256])


def test_attention_on_another_stream_and_captured():
    q, cache, table, lens, cu = setup([3000, 200], [1, 1], 8, 2, 128, 64, seed=12)
    dev = (q.cuda(), to(cache), table.cuda(), lens.cuda(), cu.cuda())
    want = cr.convrot_kv4_attention(*dev, 0.1, 64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [cr.convrot_kv4_attention(*dev, 0.1, 64, stream=side) for _ in range(4)]
    side.synchronize()
    assert all(torch.equal(o, want) for o in got)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cr.convrot_kv4_attention(*dev, 0.1, 64, out=out)
    # a replay sees new lengths
    for n in (3000, 17, 2999):
        dev[3][0] = n
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, cr.convrot_kv4_attention(*dev, 0.1, 64))


def test_offsets_beyond_32_bits():
    """Rows whose codes lie more than 2^32 bytes into the cache."""
    heads, page, D = 8, 128, 128
    pages = (1 << 32) // (heads * page * D // 2) + 40
    cache = cr.Kv4Cache(*[torch.empty(pages, heads, page, *w, dtype=d, device="cuda")
                          for w, d in (((D // 2,), torch.uint8), ((), torch.bfloat16)) * 2])
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(300, heads, D, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    small = cr.convrot_kv4_new_cache(3, heads, page, D, "cuda")
    t = torch.arange(300).cuda()
    table = torch.tensor([[pages - 1, pages - 30, pages - 2]]).int().cuda()
    slots = table[0].long()[t // page] * page + t % page
    cr.convrot_kv4_append(k, v, cache, slots, 64)
    cr.convrot_kv4_append(k, v, small, t, 64)
    for a, b in zip(cr.convrot_kv4_read(cache, slots, 64), cr.convrot_kv4_read(small, t, 64)):
        assert torch.equal(a, b)
    q = torch.randn(1, 32, D, generator=g).to(torch.bfloat16).cuda()
    lens, cu = torch.tensor([300]).int().cuda(), torch.tensor([0, 1]).int().cuda()
    far = cr.convrot_kv4_attention(q, cache, table, lens, cu, 0.1, 64)
    near = cr.convrot_kv4_attention(q, small, torch.tensor([[0, 1, 2]]).int().cuda(), lens, cu, 0.1, 64)
    assert torch.equal(far, near)


def test_empty_calls():
    q, cache, table, lens, cu = setup([5], [1], 2, 1, 64, 16, seed=13)
    assert run_attention(q[:0], cache, table, lens, cu, 0.1, 64).shape == (0, 2, 64)
    assert run_attention(q, cache, table[:0], lens[:0], cu[:1], 0.1, 64).shape == (1, 2, 64)
    none = torch.empty(1, 0, dtype=torch.int32)
    out = run_attention(q, cache, none, torch.zeros(1).int(), cu, 0.1, 64)
    assert not out.any()
    k = torch.empty(0, 1, 64, dtype=torch.bfloat16, device="cuda")
    cr.convrot_kv4_append(k, k, to(cache), torch.empty(0, dtype=torch.int64, device="cuda"), 64)


# ---------------------------------------------------------------- refusals

def test_refusals():
    q, cache, table, lens, cu = (x if isinstance(x, tuple) else x.cuda() for x in setup([5], [1], 2, 1, 64, 16, seed=14))
    cache = to(cache)
    with pytest.raises(cr.ConvRotError, match="SHAPE"):
        cr.convrot_kv4_attention(q, cache, table, lens, cu, 0.1, 256)
    with pytest.raises(cr.ConvRotError, match="GROUP"):
        cr.convrot_kv4_attention(q, cache, table, lens, cu, 0.1, 32)
    with pytest.raises(cr.ConvRotError, match="SHAPE"):
        cr.convrot_kv4_attention(q, cache, table, lens, cu, float("inf"), 64)
    with pytest.raises(ValueError, match="cu_q"):
        cr.convrot_kv4_attention(q, cache, table, lens, cu[:1], 0.1, 64)
    with pytest.raises(ValueError, match="dense within a token"):
        cr.convrot_kv4_attention(q.transpose(1, 2).contiguous().transpose(1, 2), cache, table, lens, cu, 0.1, 64)
    two = cr.convrot_kv4_new_cache(2, 2, 16, 64, "cuda")
    with pytest.raises(cr.ConvRotError, match="SHAPE"):
        cr.convrot_kv4_attention(torch.zeros(1, 3, 64, dtype=torch.bfloat16, device="cuda"), two, table, lens, cu, 0.1, 64)
    odd = cr.convrot_kv4_new_cache(2, 1, 24, 64, "cuda")
    with pytest.raises(cr.ConvRotError, match="SHAPE"):
        cr.convrot_kv4_attention(q, odd, table, lens, cu, 0.1, 64)
    with pytest.raises(cr.ConvRotError, match="SHAPE"):
        cr.convrot_kv4_plan(lens, lens, table, lens, lens, 24, 4)
    wide = torch.zeros(2, 70, dtype=torch.bfloat16, device="cuda")[:, :64].unflatten(1, (1, 64))
    with pytest.raises(cr.ConvRotError, match="SHAPE"):       # 70 values between tokens: not a multiple of 8
        cr.convrot_kv4_append(wide, wide, cache, torch.zeros(2, dtype=torch.int64, device="cuda"), 64)
