"""The norm, the 8-bit checkpoint and the relative position bias together with triangle attention,
as a pair block uses them: norm_linear makes q, k, v and the pair bias from z, the relative position
bias is added to the pair bias, the attention reads both, and the gradients come back to z, the
norm's parameters, the projection and the table.  Against the same block in FP64 torch autograd."""
import pytest
import torch

import triangle_attention_biomolecular_b200 as T

H, D, C = 4, 32, 128


def inputs(N, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return {
        "z": r(1, N, N, C).to(torch.bfloat16),
        "w": 1 + 0.2 * r(C),
        "b": 0.1 * r(C),
        "proj": (r(3 * H * D + 8, C) / C ** 0.5).to(torch.bfloat16),
        "table": 0.5 * r(34, H),
    }, r(1, N, N, H, D).to(torch.bfloat16), torch.cumsum(1 + (torch.rand(N, generator=g) < 0.1).int(), 0).int(), \
        (torch.arange(N) * 2 // N).int()


def block(p, up, pos, grp, checkpoint, orientation="start"):
    N = pos.shape[0]
    qkvb = T.norm_linear(p["z"], p["w"], p["b"], p["proj"], checkpoint=checkpoint)
    q, k, v = (qkvb[..., x * H * D:(x + 1) * H * D].unflatten(-1, (H, D)) for x in range(3))
    base = qkvb[..., 3 * H * D:3 * H * D + H].permute(0, 3, 1, 2)
    bias = T.relative_position_bias(p["table"], T.relpos_edges_clipped(16), pos, group_q=grp, base=base)
    mask = torch.zeros(1, N, N, device="cuda")
    mask[..., N - 3:] = -1e9
    out = T.triangle_attention(q, k, v, bias, mask, orientation=orientation)
    out.backward(up)
    return out


def block64(p, up, pos, grp, orientation="start"):
    N = pos.shape[0]
    h = torch.nn.functional.layer_norm(p["z"], (C,), p["w"], p["b"], 1e-5)
    qkvb = h @ p["proj"].t()
    q, k, v = (qkvb[..., x * H * D:(x + 1) * H * D].unflatten(-1, (H, D)) for x in range(3))
    if orientation == "end":
        q, k, v = (t.transpose(1, 2) for t in (q, k, v))
    delta = (pos[None, :] - pos[:, None]).clamp(-16, 16).long() + 16
    bucket = torch.where(grp[:, None] == grp[None, :], delta, 33)
    bias = qkvb[..., 3 * H * D:3 * H * D + H].permute(0, 3, 1, 2) + p["table"][bucket].permute(2, 0, 1)
    s = torch.einsum("bijhd,bikhd->bhijk", q, k) / D ** 0.5 + bias[:, :, None]
    s[..., N - 3:] = float("-inf")
    out = torch.einsum("bhijk,bikhd->bijhd", s.softmax(-1), v)
    if orientation == "end":
        out = out.transpose(1, 2)
    out.backward(up)
    return out


# BF16 stands between the steps (q, k, v, bias and their gradients, dz): half a step is 2^-8 at
# most and 2^-9 / sqrt(3) = 1.1e-3 rms; some four to eight of them in a chain, and the attention's
# own gradients, which are good to 2e-2, bound a gradient's relative error by 2e-2, the output's by
# 1e-2.  The 8-bit z adds to dz, dw and dproj at most 4 / 127 / sqrt(3) = 0.018 rms, dz twice.
@pytest.mark.gpu
@pytest.mark.parametrize("N,orientation", [(24, "start"), (61, "start"), (40, "end")])
def test_block_against_fp64(N, orientation):
    p0, up, pos, grp = inputs(N)
    p64 = {n: t.double().requires_grad_() for n, t in p0.items()}
    ref = block64(p64, up.double(), pos, grp, orientation)
    rel = lambda a, b: ((a.double().cpu() - b).norm() / b.norm()).item()  # noqa: E731
    outs = []
    for checkpoint, gate in ((None, 2e-2), ("int8", 6e-2)):
        p = {n: t.cuda().requires_grad_() for n, t in p0.items()}
        out = block(p, up.cuda(), pos.cuda(), grp.cuda(), checkpoint, orientation)
        outs.append(out.detach())
        assert rel(out.detach(), ref.detach()) <= 1e-2
        for n in p:
            assert p[n].grad.dtype == p0[n].dtype
            assert rel(p[n].grad, p64[n].grad) <= (gate if n in ("z", "w", "proj") else 2e-2), (checkpoint, n)
        again = {n: t.cuda().requires_grad_() for n, t in p0.items()}
        block(again, up.cuda(), pos.cuda(), grp.cuda(), checkpoint, orientation)
        for n in ("z", "w", "b", "table"):
            assert torch.equal(p[n].grad, again[n].grad), n  # repeatable through the whole block
    assert torch.equal(*outs)  # the checkpoint changes no output
