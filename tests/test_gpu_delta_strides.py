"""GPU checks of the gated delta rule on rows so wide that a chunk of them spans
far more than 32 bits of bytes: the same bits as from rows side by side.  (Only
the slices that the operator reads are written; the rest of a wide row is never
touched.)"""
import pytest
import torch

from state_space_model_mamba_amd import delta
from tests.test_gpu_delta import GRADS, args, cuda, make

pytestmark = pytest.mark.gpu

WIDEST = 1 << 26   # the widest row stride, in elements


@pytest.mark.parametrize("io,H,P,G,N", [("bf16", 2, 32, 1, 64), ("bf16", 2, 72, 2, 128), ("f32", 2, 32, 1, 64), ("f32", 2, 24, 1, 16)])
def test_the_widest_rows_of_q_k_and_v(io, H, P, G, N):
    L = 70
    print(f"[case] rows of {WIDEST} elements {io} H={H} P={P} G={G} N={N}", flush=True)
    d = cuda(make(1, L, H, P, G, N, io, seed=71))
    wide = torch.empty((1, L, WIDEST), dtype=d["q"].dtype, device="cuda")
    at, s = 0, dict(d)
    for name, heads, width in (("v", H, P), ("k", G, N), ("q", G, N)):
        part = wide[..., at:at + heads * width]
        part.copy_(d[name].flatten(2))
        s[name] = part.unflatten(-1, (heads, width))
        at += heads * width
    a, b = delta.delta_fwd(*args(d), want_final_states=True), delta.delta_fwd(*args(s), want_final_states=True)
    ga, gb = delta.delta_bwd(*args(d), d["do"]), delta.delta_bwd(*args(s), d["do"])
    torch.cuda.synchronize()
    assert torch.equal(a["o"], b["o"]) and torch.equal(a["final_states"], b["final_states"])
    for k in GRADS:
        assert torch.equal(ga[k], gb[k]), k


def test_rows_of_many_heads():
    """16660 float32 heads of 1024 values, each with a key of its own: a chunk of v, dout and dv is 4.4 GB.  The last
    heads by themselves give the same bits."""
    H, P, N, L, last = 16660, 1024, 4, 64, 3
    assert 63 * H * P * 4 >= 1 << 32 and H * P <= WIDEST
    gen = torch.Generator(device="cuda").manual_seed(72)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    q, k, v, do = rn(1, L, H, N) / 2, rn(1, L, H, N) / 2, rn(1, L, H, P), rn(1, L, H, P)
    g, beta = -torch.rand((1, L, H), generator=gen, device="cuda") / 4, torch.rand((1, L, H), generator=gen, device="cuda")
    cut = lambda x: x[:, :, -last:].contiguous()  # noqa: E731
    few = [cut(x) for x in (q, k, v, g, beta)]
    o = delta.delta_fwd(q, k, v, g, beta)["o"]
    r = delta.delta_bwd(q, k, v, g, beta, do, want_d_initial_states=False)
    fo, fr = delta.delta_fwd(*few)["o"], delta.delta_bwd(*few, cut(do), want_d_initial_states=False)
    torch.cuda.synchronize()
    assert torch.equal(cut(o), fo)
    for name in ("dq", "dk", "dv", "dg", "dbeta"):
        assert torch.equal(cut(r[name]), fr[name]), name
