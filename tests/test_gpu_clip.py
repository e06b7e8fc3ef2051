"""Gradient norms and clipping over lists of tensors, per adapter, against float64.

Tolerances (relative, half a step per rounding, u = 2^-24 for fp32): a norm is one rounding of
a float64 root, u (the float64 sum's own error is below 1e-12 here). The factor takes the
norm's rounding, those of the addition and the division, and the product its own: 4 u; a bf16
output adds half a step of bf16, 2^-8.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = 2.0 ** -8


def _grads(shapes, dtypes, std, seed, n):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, *s, generator=g, device="cuda") * std * (1 + i)).to(dt)
            for i, (s, dt) in enumerate(zip(shapes, dtypes))]


def _reference(grads, n, max_norm):
    sq = torch.zeros(n, dtype=torch.float64, device="cuda")
    for t in grads:
        if t.numel():
            sq += t.reshape(n, -1).double().square().sum(1)
    norm = sq.sqrt()
    m = torch.tensor(max_norm, dtype=torch.float32).double().item()
    c = (m / (norm + 1e-6)).clamp(max=1.0)
    return norm, [t.double().reshape(n, -1) * c[:, None] for t in grads]


def _check(q, grads, n, max_norm, out=None):
    keep = [t.clone() for t in grads]
    norm, want = _reference(keep, n, max_norm)
    got, gn = q.clip_grad_norm(grads, max_norm, n=n, out=out)
    only = q.grad_norm(keep, n=n)
    q.check()
    assert gn.dtype == torch.float32 and gn.shape == (n,)
    assert torch.equal(gn, only)
    assert bool(((gn.double() - norm).abs() <= 1.01 * U * norm).all())
    for g, w, k in zip(got, want, keep):
        assert g.dtype == k.dtype and g.shape == k.shape
        tol = 4.01 * U + (BF if g.dtype == torch.bfloat16 else 0.0)
        assert bool(((g.double().reshape(n, -1) - w).abs() <= tol * w.abs()).all())
    return got, gn


F, H = torch.float32, torch.bfloat16


@pytest.mark.parametrize("n", [1, 3])
@pytest.mark.parametrize("shapes,dtypes", [
    ([(1,)], [F]), ([(1,)], [H]),
    ([(7,), (4095,), (4097,), (3, 5)], [F, H, H, F]),
    ([(16, 448), (1000, 5), (64, 4096)], [F, F, F]),
    ([(8, 4096), (11008, 8)], [H, H]),
    ([(0,), (33,), (0, 4), (8192,)], [F, H, H, F]),
])
@pytest.mark.parametrize("max_norm", [0.3, 1e9, 0.0])
def test_norm_and_clip_match_float64(shapes, dtypes, n, max_norm):
    import bit_nf4_quantized_04_b200 as q
    grads = _grads(shapes, dtypes, 0.01, 5, n)
    keep = [t.clone() for t in grads]
    _check(q, grads, n, max_norm)
    assert all(torch.equal(a, b) for a, b in zip(grads, keep))  # the inputs are left
    got, _ = _check(q, grads, n, max_norm, out=grads)           # and in place
    assert all(a is b for a, b in zip(got, grads))


def test_more_tensors_than_one_launch_holds():
    import bit_nf4_quantized_04_b200 as q
    shapes = [(5 + i % 61,) for i in range(1100)]
    grads = _grads(shapes, [F if i % 3 else H for i in range(1100)], 0.001, 6, 2)
    _check(q, grads, 2, 0.5)


def test_unaligned_views_and_their_neighbours():
    # views that start at an odd element, in and out at different offsets: element by element,
    # and nothing beside them is written
    import bit_nf4_quantized_04_b200 as q
    for dt in (F, H):
        src = torch.randn(3 * 5000 + 64, device="cuda").to(dt)
        dst = torch.full_like(src, 7.0)
        for off_in, off_out in ((1, 1), (3, 6), (2, 5), (0, 1)):
            g = src[off_in:off_in + 15000].view(3, 5000)
            o = dst[off_out:off_out + 15000].view(3, 5000)
            _check(q, [g], 3, 1.0, out=[o])
            assert bool((dst[:off_out] == 7.0).all()) and bool((dst[off_out + 15000:] == 7.0).all())
            dst.fill_(7.0)


def test_each_adapter_has_its_own_factor():
    # adapter 0 holds an infinity, 1 a NaN, 2 is small enough to be left, 3 is clipped
    import bit_nf4_quantized_04_b200 as q
    g = torch.full((4, 1000), 0.5, device="cuda")
    g[2] = 1e-4
    g[0, 17] = float("inf")
    g[1, 999] = float("nan")
    b = torch.full((4, 8), 0.25, device="cuda", dtype=H)
    b[2] = 0
    (o, ob), norm = q.clip_grad_norm([g, b], 1.0, n=4)
    q.check()
    assert norm[0].item() == float("inf") and bool(norm[1].isnan())
    assert bool(o[0, 17].isnan()) and bool((o[0, :17] == 0).all()) and bool((ob[0] == 0).all())
    assert bool(o[1].isnan().all()) and bool(ob[1].isnan().all())
    assert torch.equal(o[2], g[2]) and torch.equal(ob[2], b[2])
    want = (1000 * 0.25 + 8 * 0.0625) ** 0.5
    assert abs(norm[3].item() - want) <= 1.01 * U * want
    assert abs(o[3, 0].item() - 0.5 / want) <= 5 * U


def test_squares_beyond_fp32_range():
    import bit_nf4_quantized_04_b200 as q
    for v in (1e30, 1e-30):
        g = torch.full((100,), v, device="cuda")
        want = g[0].double().item() * 10.0
        n = q.grad_norm([g])
        q.check()
        assert abs(n.item() - want) <= 1.01 * U * want


def test_same_bits_every_time_and_in_a_graph():
    # two captured graphs with a workspace of their own each, replayed in turn on new values
    import bit_nf4_quantized_04_b200 as q
    grads = _grads([(16, 4096), (4096, 16), (333,)], [F, F, H], 0.02, 8, 2)
    out = [torch.empty_like(t) for t in grads]
    norm = torch.empty(2, device="cuda")
    q.clip_grad_norm(grads, 0.3, n=2, out=out, norm=norm)
    first = [t.clone() for t in out] + [norm.clone()]
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g1):
        q.clip_grad_norm(grads, 0.3, n=2, out=out, norm=norm)
    with torch.cuda.graph(g2):
        q.clip_grad_norm(grads, 0.3, n=2, out=out, norm=norm)
    for g in (g1, g2, g1):
        for t in out:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip([*out, norm], first))
    for t in grads:
        t.mul_(2)
    g2.replay()
    torch.cuda.synchronize()
    assert torch.equal(norm, 2 * first[-1])  # a power of two scales the norm exactly


def test_another_stream():
    import bit_nf4_quantized_04_b200 as q
    grads = _grads([(64, 4096)], [F], 0.02, 9, 1)
    want = q.grad_norm(grads)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = q.grad_norm(grads)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_refusals_of_the_binding():
    import bit_nf4_quantized_04_b200 as q
    g = torch.ones(4, 6, device="cuda")
    with pytest.raises(TypeError):
        q.grad_norm([g.half()])
    with pytest.raises(ValueError):
        q.grad_norm([g.t()])
    with pytest.raises(ValueError):
        q.grad_norm([g, g.cpu()])
    with pytest.raises(ValueError):
        q.grad_norm([])
    with pytest.raises(q.Qnf4Error, match="ERR_SHAPE"):
        q.grad_norm([g], n=5)
    with pytest.raises(q.Qnf4Error, match="outputs .* overlap"):
        q.clip_grad_norm([g, g.clone()], 1.0, out=[g, g])
    with pytest.raises(ValueError):
        q.clip_grad_norm([g], 1.0, out=[g.bfloat16()])
    for bad in (-1.0, float("inf"), float("nan")):
        with pytest.raises(q.Qnf4Error, match="ERR_ARG"):
            q.clip_grad_norm([g], bad)
    with pytest.raises(ValueError):
        q.grad_norm([g], ws=torch.empty(8, dtype=torch.uint8, device="cuda"))


def test_dist_path_clips_in_place():
    import bit_nf4_quantized_04_b200 as q
    from bit_nf4_quantized_04_b200 import dist
    grads = _grads([(8, 512), (512, 8)], [F, H], 0.02, 12, 3)
    want, norm = q.clip_grad_norm([t.clone() for t in grads], 0.4, n=3)
    got = dist.allreduce_clip_adapter_grads(grads, 0.4, 3)
    assert torch.equal(got, norm) and all(torch.equal(a, b) for a, b in zip(grads, want))


def test_an_output_that_is_another_gradient_is_refused():
    """Scaling into each other's buffers would read what another part has already written."""
    import bit_nf4_quantized_04_b200 as q
    a, b = torch.ones(4, 6, device="cuda"), torch.ones(4, 6, device="cuda")
    with pytest.raises(q.Qnf4Error, match="overlaps gradient"):
        q.clip_grad_norm([a, b], 1.0, out=[b, a])
    with pytest.raises(q.Qnf4Error, match="overlaps gradient"):
        q.clip_grad_norm([a, b], 1.0, out=[torch.empty_like(a), a])
    flat = torch.ones(40, device="cuda")
    with pytest.raises(q.Qnf4Error, match="overlaps gradient"):
        q.clip_grad_norm([flat[:16], b], 1.0, out=[flat[8:24], torch.empty_like(b)])
    with pytest.raises(q.Qnf4Error, match="outputs .* overlap"):
        q.clip_grad_norm([a, b], 1.0, out=[flat[:24].view(4, 6), flat[16:].view(4, 6)])
    out, _ = q.clip_grad_norm([a, b], 1.0, out=[a.view(4, 6), torch.empty_like(b)])  # its own buffer, as a view
    assert out[0].data_ptr() == a.data_ptr() and torch.equal(a, out[1])
