"""GPU tests of the operators around a LoRA-wrapped projection: calls whose
memory layout, size or values are unusual, each against its formula in 64 bits.
Tolerances as in test_base_ops.py."""
import pytest
import torch

from gather_matmul_b200 import ops
from test_base_ops import BF16, TYPES, gen, rotated

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [1, 2])
@pytest.mark.parametrize("norm", [False, True], ids=["rope", "norm"])
def test_rope_in_place_into_a_narrower_view(dtype, T, norm):
    """The q and k columns of a fused projection as y, the whole of it as x:
    the same memory in views of other widths, whatever the number of rows."""
    heads, dim, g = [4, 2], 64, gen(61)
    n = sum(heads) * dim
    qkv = torch.randn(T, n + 2 * dim, generator=g, device="cuda").to(dtype)
    x, pos = qkv.clone(), torch.randint(0, 4096, (T,), generator=g, device="cuda")
    f, m = ops.rope_frequencies(dim)
    w = [(1 + 0.3 * torch.randn(dim, generator=g, device="cuda")).to(dtype) for _ in heads]
    if norm:
        ops.norm_rope(qkv, w, qkv[:, :n], heads, dim, pos, f, attn_scale=m)
    else:
        ops.rope(qkv, qkv[:, :n], heads, dim, pos, f, attn_scale=m)
    c = 0
    for (r, tol), h in zip(rotated(x, heads, dim, pos, f, m, False, [0, 4 * dim], w if norm else None, 1e-6), heads):
        assert ((qkv[:, c:c + h * dim].double().view(T, h, dim) - r).abs() <= tol).all()
        c += h * dim
    assert torch.equal(qkv[:, n:], x[:, n:])


def test_rope_of_one_row_still_refuses_shared_memory():
    row = torch.randn(1, 512, generator=gen(62), device="cuda").to(BF16)
    f, pos = ops.rope_frequencies(64)[0], torch.zeros(1, dtype=torch.int64, device="cuda")
    before = row.clone()
    with pytest.raises(ops.LoraError):
        ops.rope(row, row[:, 8:], [2], 64, pos, f)              # 8 columns further
    with pytest.raises(ops.LoraError):
        ops.rope(row, row, [2, 2], 64, pos, f, x_col_off=[0, 128], y_col_off=[128, 0])   # slices swapped
    torch.cuda.synchronize()
    assert torch.equal(row, before)
