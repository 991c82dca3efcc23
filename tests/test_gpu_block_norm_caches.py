"""The norms' backward past the caches, by what a call moves: a float32 residual's gradients beside bf16 operands, and
operands without a gate.  Rows are alone but for the sums over them, so parts of the rows, which stay below the caches'
size, give the same bits."""
import pytest
import torch

from state_space_model_mamba_amd import block_norm as bn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["add with a float32 residual", "add without a residual", "gated without a gate"])
def test_more_than_the_caches_hold(kind):
    # 16384 x 2048: 604, 335 and 201 MB; the last stays below
    L, D, parts = 16384, 2048, 4
    gen = torch.Generator(device="cuda").manual_seed(1)
    rn = lambda: torch.randn((1, L, D), generator=gen, device="cuda")  # noqa: E731
    x, dy, r, dr = rn().bfloat16(), rn().bfloat16(), rn(), rn()
    w = 1 + 0.1 * torch.randn((D,), generator=gen, device="cuda")

    def call(at):
        if kind.startswith("gated"):
            return bn.gated_norm_bwd(x[:, at], None, w, None, 1.0, dy[:, at], groups=2)
        if kind.endswith("without a residual"):
            return bn.add_norm_bwd(x[:, at], None, w, 1.0, dy[:, at], dy[:, at])
        return bn.add_norm_bwd(x[:, at], r[:, at], w, 1.0, dy[:, at], dr[:, at])

    print(f"[case] {kind}", flush=True)
    whole, sums = call(slice(0, L)), torch.zeros(D, dtype=torch.float64, device="cuda")
    for lo in range(0, L, L // parts):
        at = slice(lo, lo + L // parts)
        part = call(at)
        assert torch.equal(part["dx"], whole["dx"][:, at])
        assert whole.get("dresidual") is None or torch.equal(part["dresidual"], whole["dresidual"][:, at])
        sums += part["dweight"]
    # a block adds at most 64 rows in float32, each sum is rounded once more: of the terms' size, which the norm of L random
    # terms is sqrt(L) below at most
    assert float((whole["dweight"] - sums).norm() / sums.norm()) < (64 + 2) * 2.0 ** -24 * L ** 0.5
