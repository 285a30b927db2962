"""Every kernel instance that some size reaches has a parity case (no GPU needed): after a change of the
rules that choose them, this says which instance lost its test."""
import math
import random

import pytest

from tests import operator_tiles as S
from tests.test_gpu_operators import FFN, MATMUL


@pytest.fixture(scope="module")
def choice():
    from fp8_moe_layer_b200 import build
    build.build()
    from fp8_moe_layer_b200 import ops
    return S.Choice(ops.LIB)


def sizes(n, *ranges):
    """Sizes spread over the logarithm of each range, with at most the work of a long prompt."""
    rng = random.Random(0)
    while n:
        v = []
        for lo, hi, step in ranges:
            x = math.exp(rng.uniform(math.log(lo), math.log(hi)))
            v.append(min(hi, max(lo, round(x / step) * step)))
        if math.prod(v) <= 8192 * 7168 * 4096:
            n -= 1
            yield v


@pytest.mark.parametrize("op", ["matmul", "ffn"])
def test_every_instance_has_a_parity_case(choice, op):
    rule, cases = ((choice.matmul, MATMUL + S.MATMUL) if op == "matmul"
                   else (choice.ffn, FFN + S.FFN))
    covered = set().union(*(rule(*c) for c in cases))
    last = (16, 28672, 16) if op == "matmul" else (16, 14336, 16)
    reached = set().union(*(rule(*c) for c in sizes(20000, (1, 8192, 1), (16, 14336, 16), last)))
    assert len(reached) > 10 and reached <= covered, sorted(reached - covered)


def test_the_cases_of_long_prompts_run_on_pairs(choice):
    assert choice.matmul(8192, 7168, 4096) == {"int8 pair"}
    assert choice.ffn(8192, 7168, 2048) == {"gated pair", "down pair", "gradient of the activation pair",
                                            "three products pair"}
