"""Seeded inputs of the gated delta rule's tests."""
import torch

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def unit(g, *shape, device="cpu"):
    v = torch.randn(*shape, generator=g, device=device)
    return v / v.norm(dim=-1, keepdim=True)


def direction(g, batch, L, H, P, G, N, dtype, device="cpu", decay=0.3, alike=0.3):
    """Queries and keys of length one with a common part (``alike``), decays up
    to ``decay`` a token, beta in (0, 1), a few of them 0."""
    common = unit(g, N, device=device)

    def near(*shape):
        v = unit(g, *shape, device=device) + alike * common
        return (v / v.norm(dim=-1, keepdim=True)).to(DT[dtype]).contiguous()

    def rand(*shape):
        return torch.rand(*shape, generator=g, device=device)
    beta = rand(batch, L, H)
    return dict(q=near(batch, L, G, N), k=near(batch, L, G, N),
                v=torch.randn(batch, L, H, P, generator=g, device=device).to(DT[dtype]),
                g=-decay * rand(batch, L, H) ** 3, beta=torch.where(rand(batch, L, H) < 0.05, torch.zeros_like(beta), beta))
