"""Inputs of AttentionInputs that its kernels, which take addresses alone, would
misread: refused before anything is enqueued.  No GPU, no call launches."""
import pytest
import torch

from gather_matmul_b200 import build
from gather_matmul_b200.layers import AttentionInputs

F16, BF16 = torch.float16, torch.bfloat16
HQ, HK, DIM, K, S, R = 2, 1, 64, 128, 2, 8
WIDTHS = [HQ * DIM, HK * DIM, HK * DIM]


@pytest.fixture(scope="module", autouse=True)
def library():
    build.build()


def stacks(dtype=BF16, n=3):
    return [torch.zeros(S, R, K, dtype=dtype) for _ in range(n)], [torch.zeros(S, w, R, dtype=dtype) for w in WIDTHS]


def layer(A, B):
    W = torch.zeros(sum(WIDTHS), K).to(torch.float8_e4m3fn)
    return AttentionInputs(W, torch.ones(2, 1), A, B, HQ, HK, DIM, torch.ones(DIM // 2, dtype=torch.float64),
                           max_tokens=8)


def test_stacks_of_several_types_are_refused():
    A, B = stacks()
    for i in range(3):
        with pytest.raises(TypeError):
            layer(A, [b.half() if j == i else b for j, b in enumerate(B)])
        if i:
            with pytest.raises(TypeError):
                layer([a.half() if j == i else a for j, a in enumerate(A)], B)
    layer(A, B)
    layer(A[:1], B)


def test_number_of_stacks():
    A, B = stacks()
    with pytest.raises(ValueError):
        layer(A[:2], B)


def test_stacks_that_are_not_contiguous_are_refused():
    A, B = stacks()
    with pytest.raises(ValueError):
        layer([A[0], torch.zeros(1, R, K, dtype=BF16).expand(S, R, K), A[2]], B)   # one adapter's memory
    fused = torch.zeros(S, sum(WIDTHS), R, dtype=BF16)
    with pytest.raises(ValueError):
        layer(A, list(fused.split(WIDTHS, 1)))
    with pytest.raises(ValueError):
        layer(A, [B[0], B[1], torch.zeros(S, WIDTHS[2], R, dtype=BF16, device="meta")])


def test_inputs_of_another_type_or_device_are_refused():
    A, B = stacks(F16)
    idx, pos = torch.zeros(4, dtype=torch.int32), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(TypeError, match="as the LoRA stacks"):
        layer(A, B)(torch.zeros(4, K, dtype=BF16), idx, pos, torch.zeros(4, sum(WIDTHS), dtype=BF16))
    with pytest.raises(ValueError, match="idx must be on"):
        layer(A, B)(torch.zeros(4, K, dtype=F16), torch.empty(4, dtype=torch.int32, device="meta"), pos,
                    torch.zeros(4, sum(WIDTHS), dtype=F16))
    with pytest.raises(ValueError, match="current CUDA device"):
        layer(A, B)(torch.zeros(4, K, dtype=F16), idx, pos, torch.zeros(4, sum(WIDTHS), dtype=F16))
