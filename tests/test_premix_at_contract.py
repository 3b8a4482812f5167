"""Which kernel premix_fwd_qkv_at takes is part of its contract (the bits of
premix_fwd_qkv, or of the kernel for few tokens): the header states the rule that
the code applies, and past it the bits are those of premix_fwd_qkv."""
import os
import re

import pytest

import synthetic as S
from helpers import to_dev

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def constants():
    src = open(os.path.join(ROOT, "transformer_attention_iha_gb300", "csrc", "premix_tc.cu")).read()
    return [int(re.search(rf"{n} = (\d+)", src).group(1)) for n in ("kFewRows", "kFewCtas")]


def test_the_header_states_the_rule_that_the_code_applies():
    rows, ctas = constants()
    text = " ".join(open(os.path.join(ROOT, "include", "iha.h")).read().replace("*", " ").split())
    m = re.search(r"3 B N ceil\(H P / (\d+)\) <= (\d+) \((\d+) tokens of 20 -> 80 heads, "
                  r"(\d+) of 8 -> 16\)", text)
    assert m and [int(x) for x in m.groups()] == [rows, ctas, ctas // 3 // -(-80 // rows),
                                                  ctas // 3 // -(-16 // rows)]
    assert "to 64 bf16 tokens" not in text


@pytest.mark.gpu
@pytest.mark.parametrize("H,P,d", [(20, 4, 128), (8, 2, 64), (32, 4, 64), (5, 3, 128)])
def test_past_the_rule_the_bits_are_those_of_premix_fwd_qkv(H, P, d):
    import torch
    import transformer_attention_iha_gb300 as T
    rows, ctas = constants()
    n = ctas // 3 // -(-H * P // rows) + 1
    xs = [to_dev(S.normal((1, n, H, d), 510, t)) for t in range(3)]
    ws = [to_dev(S.premix_weight(H, P, 511, t)) for t in range(3)]
    pos = torch.arange(n, dtype=torch.int32, device="cuda")[None]
    a = T.premix_fwd_qkv(xs, ws, P, rope=True)
    b = T.premix_fwd_qkv_at(xs, ws, P, pos)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
