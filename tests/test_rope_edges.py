"""Norm and rotation at the edges of its shapes: a side without heads."""
import pytest
import torch

from backward_adapter_gb300 import rope


@pytest.mark.gpu
@pytest.mark.parametrize("S", [0, 5, 3000])
@pytest.mark.parametrize("side", ["q", "k"])
def test_a_side_without_heads_has_a_weight_gradient_of_zero(side, S):
    """The sum over no rows is written like any other, into memory that holds something else."""
    D = 64
    g = torch.Generator(device="cuda").manual_seed(S)
    x, dx = (torch.randn((2, 4, S, D), generator=g, device="cuda") for _ in range(2))
    none = torch.empty((2, 0, S, D), device="cuda")
    f, w = rope.rope_inv_freq(D, device="cuda")[0], torch.rand(D, device="cuda")
    args = (dx, none, x, none) if side == "k" else (none, dx, none, x)
    at, other = (3, 2) if side == "k" else (2, 3)
    got = rope.qk_norm_rope_bwd(*args, f, q_weight=w, k_weight=w, dq_weight=torch.full((D,), 7.0, device="cuda"),
                                dk_weight=torch.full((D,), 7.0, device="cuda"))
    assert torch.equal(got[at], torch.zeros(D, device="cuda"))
    want = rope.qk_norm_rope_bwd(dx, dx, x, x, f, q_weight=w, k_weight=w)
    assert torch.equal(got[0 if side == "k" else 1], want[0])
    # with other heads beside them the same n terms are added in another order: each sum is off by at most (n + 64) 2^-24 of
    # the sum of magnitudes (see test_rope), a term's being that of its rotated pair times |x| r
    n, m = 8 * S, torch.hypot(dx[..., :32].double(), dx[..., 32:].double()).repeat(1, 1, 1, 2)
    size = (m * x.double().abs() * (x.double().square().mean(-1, keepdim=True) + 1e-6).rsqrt()).sum((0, 1, 2))
    assert bool(((got[other].double() - want[other].double()).abs() <= 2 * (n + 64) * 2.0 ** -24 * size).all())
