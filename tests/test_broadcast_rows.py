"""Operands of the block norms and of the gated linear recurrence whose rows are one broadcast row, with one batch row
and with several."""
import pytest
import torch

from state_space_model_mamba_amd import block_norm, recurrence


def test_row_strides_of_one_batch_row():
    x = torch.zeros(3, 7, 48)
    sb, sl = block_norm.row_strides(x[:1, :1, :16].expand(1, 7, 16), "s")
    assert sl == 0 and sb > 0 and sb % 8 == 0   # 0, 0 would be a contiguous tensor
    assert block_norm.row_strides(x[:, :1, :16].expand(3, 7, 16), "s") == (7 * 48, 0)
    with pytest.raises(ValueError, match="broadcast"):
        block_norm.row_strides(x[:1, :1, :16].expand(2, 7, 16), "s")


@pytest.mark.gpu
@pytest.mark.parametrize("batch", [1, 3])
def test_a_broadcast_row_gives_the_bits_of_its_copies(batch):
    L, D = 70, 64
    rn = lambda *s: torch.randn(s, generator=gen).bfloat16().cuda()  # noqa: E731
    gen = torch.Generator().manual_seed(batch)
    x, dy, one = rn(batch, L, D), rn(batch, L, D), rn(batch, 1, D)
    row = one.expand(batch, L, D)
    copy = row.clone(memory_format=torch.contiguous_format)
    w = 1 + 0.1 * rn(D).float()
    same = lambda a, b: all(torch.equal(a[k], b[k]) for k in a if a[k] is not None)  # noqa: E731
    for a, b in zip(block_norm.add_norm_fwd(row, x, w), block_norm.add_norm_fwd(copy, x, w)):
        assert torch.equal(a, b)
    assert same(block_norm.add_norm_bwd(row, x, w, 1.0, dy, None), block_norm.add_norm_bwd(copy, x, w, 1.0, dy, None))
    for p, q in (((x, row), (x, copy)), ((row, x), (copy, x))):
        assert torch.equal(block_norm.gated_norm_fwd(*p, w, groups=2), block_norm.gated_norm_fwd(*q, w, groups=2))
        assert same(block_norm.gated_norm_bwd(*p, w, None, 1.0, dy, groups=2), block_norm.gated_norm_bwd(*q, w, None, 1.0, dy, groups=2))
        assert torch.equal(recurrence.linrec_fwd(*p)["y"], recurrence.linrec_fwd(*q)["y"])
        assert same(recurrence.linrec_bwd(*p, None, None, dy), recurrence.linrec_bwd(*q, None, None, dy))
    pool = [torch.zeros((batch, D), device="cuda") for _ in range(2)]
    ys = [recurrence.linrec_step(x[:, :60], t[:, :60], s) for t, s in zip((row, copy), pool)]
    assert torch.equal(*ys) and torch.equal(*pool)
