"""Norms and workspaces of clipping over and beside the gradients."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_norms_and_workspaces_over_and_beside_gradients():
    import bit_nf4_quantized_04_b200 as q
    g = torch.randn(4, 512, generator=torch.Generator().manual_seed(3)).cuda()
    want, norm = q.clip_grad_norm([g], 0.5, n=4)
    # the norms, the gradient, the output and the workspace side by side in one buffer
    flat = torch.zeros(4 + 2048 + 2048 + 4096, device="cuda")
    g2, out = flat[4:2052].view(4, 512), flat[2052:4100].view(4, 512)
    g2.copy_(g)
    got, n2 = q.clip_grad_norm([g2], 0.5, n=4, out=[out], norm=flat[:4], ws=flat[4100:].view(torch.uint8))
    assert torch.equal(got[0], want[0]) and torch.equal(n2, norm) and torch.equal(g2, g)
    for kw in (dict(norm=flat[4:8]), dict(norm=flat[2052:2056]), dict(ws=flat[2052:]), dict(norm=flat[4100:4104], ws=flat[4100:])):
        with pytest.raises(q.Qnf4Error, match="overlaps"):
            q.clip_grad_norm([g2], 0.5, n=4, out=[out], **kw)
    with pytest.raises(q.Qnf4Error, match="overlaps"):
        q.grad_norm([g2], n=4, norm=flat[2048:2052])
    q.check()
    assert torch.equal(g2, g) and torch.equal(out, want[0])
