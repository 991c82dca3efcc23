"""add_norm_fwd with y in x's place and the new residual in the old one's, as include/block_norm.h allows: the bits of
the call with outputs of their own, also where a block takes many tokens and has asked for the next one's operands."""
import ctypes

import pytest
import torch

from state_space_model_mamba_amd import block_norm as bn

pytestmark = pytest.mark.gpu
IO = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.mark.parametrize("io,res", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("L,D", [(1, 64), (70, 1000), (2 * 65536 + 70, 136), (2 * 32768 + 77, 520), (8192 + 100, 8192), (4096 + 100, 16384)])
def test_in_place(L, D, io, res):
    gen = torch.Generator(device="cuda").manual_seed(L)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, r, w = rn(1, L, D).to(IO[io]), rn(1, L, D).to(IO[res]), 1 + 0.1 * rn(D)
    print(f"[case] {io}/{res} {L} x {D}", flush=True)
    ref = bn.add_norm_fwd(x, r, w)
    shape = bn.make_shape(1, L, D, io_dtype=bn._io(IO[io]), residual_dtype=bn._io(IO[res]))
    ptr = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    rc = bn.load_library().add_norm_fwd(ctypes.byref(shape), ptr(x), ptr(r), ptr(w), None, None, ptr(x), ptr(r), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0 and torch.equal(x, ref[0]) and torch.equal(r, ref[1])
