"""The cache library's whole-number arrays without a GPU: they may begin
anywhere that their type allows (parts of longer arrays), not only on 16 bytes."""
import ctypes

import pytest

import rotated_w4a4_quantized_b200 as cr
from tests.test_abi_decoding import A, cache

ALIGN = 4
ODD = ctypes.c_void_p(0x10002)


@pytest.fixture(scope="module", autouse=True)
def _built():
    from rotated_w4a4_quantized_b200 import build
    build.build()


def at(offset):
    return ctypes.c_void_p(0x10000 + offset)


def append(slots):
    return cr.lib_kv4().convrot_kv4_append(cache(), A, 256, A, 256, slots, 3, None)


def read(slots):
    return cr.lib_kv4().convrot_kv4_read(cache(), slots, 3, A, A, None)


def attention(table=A, lens=A, cu=A):
    return cr.lib_kv4().convrot_kv4_attention(cache(), A, 1024, 3, 8, table, 4, lens, cu, 2, 0.1, A, 1 << 30, A, None)


def plan(**over):
    v = dict(cached=A, new=A, table=A, free=A, count=A, lens=A, cu=A, slots=A, positions=A, result=A)
    v.update(over)
    return cr.lib_kv4().convrot_kv4_plan(v["cached"], v["new"], 2, 16, v["table"], 4, v["free"], 4, v["count"], 4, v["lens"],
                                         v["cu"], v["slots"], v["positions"], v["result"], None)


# (a call whose arguments are all right goes on to look its pointers up: these
# are no device memory, or there is no device)

def test_slots_begin_on_8_bytes():
    for f in (append, read, lambda p: plan(slots=p)):
        assert f(at(8)) != ALIGN and f(at(0)) != ALIGN
        assert f(at(4)) == ALIGN and f(ODD) == ALIGN


@pytest.mark.parametrize("name", ["table", "lens", "cu"])
def test_attention_takes_parts_of_arrays(name):
    for offset in (4, 8, 12):
        assert attention(**{name: at(offset)}) != ALIGN
    assert attention(**{name: ODD}) == ALIGN


@pytest.mark.parametrize("name", ["new", "table", "free", "count", "lens", "cu", "positions"])
def test_plan_takes_parts_of_arrays(name):
    for offset in (4, 8, 12):
        assert plan(**{name: at(offset)}) != ALIGN
    assert plan(**{name: ODD}) == ALIGN


@pytest.mark.parametrize("name", ["cached", "result"])
def test_the_plans_lengths_and_result_begin_on_16_bytes(name):
    assert plan(**{name: at(8)}) == ALIGN and plan(**{name: at(16)}) != ALIGN
