"""GPU tests: lengths, tables, slots and counters that are parts of longer
arrays, at every offset within 16 bytes, give what arrays of their own give,
in the native and in the Python path of the bindings (a stream given)."""
import pytest
import torch

import rotated_w4a4_quantized_b200 as cr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from rotated_w4a4_quantized_b200 import build
    build.build()


def shifted(t, offset):
    """`t` as a part of a longer array that begins `offset` elements earlier."""
    room = torch.full((t.numel() + offset + 3,), -99, dtype=t.dtype, device="cuda")
    part = room[offset:offset + t.numel()].view(t.shape)
    part.copy_(t)
    return part


@pytest.mark.parametrize("named", [False, True])
@pytest.mark.parametrize("offset", [0, 1, 2, 3])
def test_parts_of_longer_arrays(offset, named):
    kw = {"stream": torch.cuda.current_stream()} if named else {}
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")   # noqa: E731
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(20, 2, 64, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    q = torch.randn(20, 4, 64, generator=g).to(torch.bfloat16).cuda()
    results = []
    for part in (lambda t: t, lambda t: shifted(t, offset)):
        cached, new, table = part(i32([3, 0, 16])), part(i32([2, 17, 1])), part(i32([[6, -1], [-1, -1], [7, -1]]))
        free, count = part(i32([5, 4, 3, 2, 1, 0])), part(i32([6]))
        p = cr.convrot_kv4_plan(cached, new, table, free, count, 16, 20, **kw)
        lens, cu, slots = part(p.seq_lens), part(p.cu_q), part(p.slots)
        cache = cr.convrot_kv4_new_cache(8, 2, 16, 64, "cuda")
        cr.convrot_kv4_append(k, v, cache, slots, 64, **kw)
        kr, vr = cr.convrot_kv4_read(cache, slots, 64, **kw)
        o = cr.convrot_kv4_attention(q, cache, table, lens, cu, 0.1, 64, **kw)
        results.append([table, free, p.seq_lens, p.cu_q, p.slots, p.positions, p.result, *cache, kr, vr, o])
    assert results[0][6].tolist() == [3, 3, 20, 0]
    for a, b in zip(*results):
        assert torch.equal(a, b)
    assert cr.convrot_kv4_check_device_error() == 0


def test_a_step_of_some_of_the_requests():
    """The second half of a server's requests: slices of its state."""
    i32 = dict(dtype=torch.int32, device="cuda")
    lens, new, table = torch.tensor([9, 8, 31, 16, 5], **i32), torch.ones(5, **i32), torch.arange(10, **i32).view(5, 2)
    p = cr.convrot_kv4_plan(lens[3:], new[3:], table[3:], torch.arange(20, 30, **i32), torch.tensor([7, 10], **i32)[1:], 16, 2)
    assert p.slots.tolist() == [29 * 16, 8 * 16 + 5] and p.seq_lens.tolist() == [17, 6] and p.result.tolist() == [9, 1, 2, 0]
    assert table[3].tolist() == [6, 29]
    cache = cr.convrot_kv4_new_cache(30, 1, 16, 64, "cuda")
    k = torch.randn(3, 1, 64, device="cuda").bfloat16()
    slots = torch.tensor([5, 6, 7], device="cuda")
    cr.convrot_kv4_append(k[1:], k[1:], cache, slots[1:], 64)
    one, _ = cr.convrot_kv4_read(cache, slots[2:], 64)
    both, _ = cr.convrot_kv4_read(cache, slots[1:], 64)
    assert torch.equal(one[0], both[1]) and bool(one.any())


def test_a_captured_plan_of_a_slice_reads_the_lengths_of_its_replay():
    i32 = dict(dtype=torch.int32, device="cuda")
    lens, table = torch.tensor([9, 3, 5], **i32), torch.arange(3, **i32).view(3, 1)
    args = (torch.ones(2, **i32), table[1:], torch.arange(4, **i32), torch.tensor([4], **i32), 16, 2)
    cr.convrot_kv4_plan(lens[1:], *args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p = cr.convrot_kv4_plan(lens[1:], *args)
    for a, b in ((3, 5), (7, 1)):
        lens[1:] = torch.tensor([a, b], **i32)
        graph.replay()
        torch.cuda.synchronize()
        assert p.seq_lens.tolist() == [a + 1, b + 1] and p.positions.tolist() == [a, b]
