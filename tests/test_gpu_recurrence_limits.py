"""The gated linear recurrence at the documented number of rows: more chunks than one launch can have threads for
(2^32).  The operands are broadcast over the batch, so every batch row has to give the bits of the first, and that one
those of a call of its own rows."""
import pytest
import torch

from state_space_model_mamba_amd import recurrence as rec

pytestmark = pytest.mark.gpu


def test_more_rows_than_one_launch_has_threads_for():
    B, L, C = (1 << 16) + 1, 1 << 14, 8   # 2^30 rows and some: 2^23 chunks of 512 threads forward, 2^24 backward
    assert B * L < 2 ** 31 - 4096
    gen = torch.Generator().manual_seed(0)
    x, g, dy = (torch.randn((1, L, C), generator=gen).bfloat16().cuda() for _ in range(3))
    kw = dict(gate="sigmoid", input_scale="complement")
    one = rec.linrec_fwd(x, g, want_final_states=True, want_chunk_states=True, **kw)
    few = rec.linrec_bwd(x, g, None, None, dy, chunk_states=one["chunk_states"], want_d_initial_states=False, **kw)
    wide = lambda t: t.expand(B, L, C)  # noqa: E731

    def same(got, ref, label):
        print(f"[case] {label}", flush=True)
        for lo in range(0, B, 8192):
            part = got[lo:lo + 8192]
            assert torch.equal(part, ref.expand(part.shape)), f"{label}, batch rows from {lo}"

    print("[case] forward", flush=True)
    r = rec.linrec_fwd(wide(x), wide(g), want_final_states=True, want_chunk_states=True, **kw)
    torch.cuda.synchronize()
    same(r["y"], one["y"], "y")
    same(r["final_states"], one["final_states"], "final_states")
    states = r["chunk_states"]
    same(states.view(B, L // 64, C), one["chunk_states"][None], "chunk_states")
    del r
    print("[case] backward", flush=True)
    b = rec.linrec_bwd(wide(x), wide(g), None, None, wide(dy).contiguous(), chunk_states=states, want_d_initial_states=False, **kw)
    torch.cuda.synchronize()
    same(b["dx"], few["dx"], "dx")
    same(b["dg"], few["dg"], "dg")
    del b, states
    torch.cuda.empty_cache()
