"""Sizes that an int of the C calls cannot hold are refused by the binding, not
cut down to their low 32 bits.  No memory stands behind these tensors, and no
call here launches."""
import pytest
import torch

from gather_matmul_b200 import _lib, build, ops

BF16, FP8 = torch.bfloat16, torch.float8_e4m3fn
PAST = 1 << 32          # as an int: 0


@pytest.fixture(scope="module", autouse=True)
def library():
    build.build()


def meta(*shape, dtype):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("T,K", [(1, PAST + 128), (PAST + 1, 16), (1 << 31, 16), (1, 1 << 31)])
def test_quantize_refuses_sides_past_an_int(T, K):
    x, q = meta(T, K, dtype=BF16), meta(T, K, dtype=FP8)
    with pytest.raises(ValueError, match="2\\^31"):
        ops.quantize_fp8(x, q, meta(T, -(-K // 128), dtype=torch.float32))


@pytest.mark.parametrize("rows", [PAST + 1, PAST + 128, -PAST + 1])
def test_quantize_refuses_block_rows_past_an_int(rows):
    """As an int the first is one row to a scale, for which `scale` is too short."""
    x, q = meta(5, 256, dtype=BF16), meta(5, 256, dtype=FP8)
    with pytest.raises(ops.LoraError) as e:
        ops.quantize_fp8(x, q, meta(1 if rows > 0 else 0, 2, dtype=torch.float32), block_rows=rows)
    assert e.value.status == _lib.LORA_ERR_UNSUPPORTED


@pytest.mark.parametrize("T,N,K", [(PAST + 1, 64, 128), (4, PAST + 64, 128), (4, 64, PAST + 128)])
def test_products_refuse_sides_past_an_int(T, N, K):
    KB, NB, f = -(-K // 128), -(-N // 128), torch.float32
    W, ws, y = meta(N, K, dtype=FP8), meta(NB, KB, dtype=f), meta(T, N, dtype=BF16)
    with pytest.raises(ValueError, match="2\\^31"):
        ops.matmul_fp8(meta(T, K, dtype=FP8), meta(T, KB, dtype=f), W, ws, y)
    with pytest.raises(ValueError, match="2\\^31"):
        ops.linear_fp8(meta(T, K, dtype=BF16), W, ws, y, meta(1 << 20, dtype=torch.uint8))


def test_workspace_and_frequencies_past_an_int():
    for T, K in [(PAST + 4, 128), (4, PAST + 128)]:
        with pytest.raises(ops.LoraError):
            ops.linear_fp8_workspace(T, K, device="meta")
    for rot in (PAST + 64, -PAST + 64, 1 << 30):
        with pytest.raises(ops.LoraError):
            ops.rope_frequencies(rot, device="meta")
    assert ops.linear_fp8_workspace(4, 128, device="meta").numel() == 768
    assert ops.rope_frequencies(64, device="cpu")[0].numel() == 32


def test_rotation_refuses_numbers_past_an_int():
    x, f = meta(4, 512, dtype=BF16), meta(32, dtype=torch.float64)
    pos = meta(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="2\\^31"):
        ops.rope(meta(PAST + 4, 512, dtype=BF16), meta(PAST + 4, 512, dtype=BF16), [8], 64,
                 meta(PAST + 4, dtype=torch.int64), f)
    with pytest.raises(ops.LoraError):
        ops.rope(x, x, [8], 64, pos, meta((PAST >> 1) + 32, dtype=torch.float64))
    with pytest.raises(ValueError):
        ops.rope(x, x, [8], PAST + 64, pos, f)
    with pytest.raises(ValueError):
        ops.rope(x, x, [PAST + 8], 64, pos, f)
    for heads, dim, off in [([8], -PAST + 64, None), ([-PAST + 8], 64, None), ([PAST + 8], 64, [-PAST * 64]),
                            ([0], 64, None), ([8], 0, None)]:
        with pytest.raises(ops.LoraError) as e:
            ops.rope(x, x, heads, dim, pos, f, x_col_off=off, y_col_off=off)
        assert e.value.status == _lib.LORA_ERR_INVALID_ARG
