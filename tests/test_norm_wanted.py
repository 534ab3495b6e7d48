"""The PyTorch operator of the norm and rotation keeps and works out what is wanted, and no more."""
import pytest
import torch

from place_partial_rope_gb300 import binding, torch_op

DEV = "cuda"


def test_meta_kernels():
    torch_op.register()
    ops = getattr(torch.ops, torch_op.NAMESPACE)
    meta = dict(device="meta")
    q, k, w = torch.empty((2, 3, 4, 8), **meta), torch.empty((2, 3, 1, 8), **meta), torch.empty(8, **meta)
    for keep in (True, False):
        got = ops.norm_rotary(q, k, w, w, None, None, norm_slice=[0, 8], keep_rstd=keep)
        assert [t.numel() for t in got] == [192, 48, 24 * keep, 6 * keep]
    r = torch.empty((2, 3, 4), **meta)
    for wanted in ([True, True], [False, True], [True, False], [False, False]):
        got = ops.norm_rotary_backward(q, k, q, k, w, w, r, r[..., :1], None, None, norm_slice=[0, 8], weight_grads=wanted)
        assert [t.numel() for t in got] == [192, 48, 8 * wanted[0], 8 * wanted[1]]


@pytest.mark.gpu
@pytest.mark.parametrize("wanted", [(True, False), (False, True), (False, False)])
def test_weights_without_a_gradient(wanted, monkeypatch):
    """Their gradients are not asked of the kernels, and the others are those of a call that wants all."""
    g = torch.Generator().manual_seed(2)
    rows = [torch.randn((2, 5, h, 64), generator=g).to(DEV) for h in (4, 2)]
    weights = [torch.randn(64, generator=g).to(DEV) for _ in range(2)]
    tables = [torch.randn((1, 5, 1, 32), generator=g).to(DEV) for _ in range(2)]
    asked, plain = [], binding.rope_partial_norm_bwd

    def bwd(*args, dq_weight=None, dk_weight=None, **kw):
        asked.append((dq_weight is not None, dk_weight is not None))
        plain(*args, dq_weight=dq_weight, dk_weight=dk_weight, **kw)

    monkeypatch.setattr(binding, "rope_partial_norm_bwd", bwd)
    grads = []
    for want in ((True, True), wanted):
        x = [t.clone().requires_grad_() for t in rows]
        w = [t.clone().requires_grad_(need) for t, need in zip(weights, want)]
        a, b = torch_op.norm_rotary(*x, *w, *tables, partial_slice=[0, 32])
        ((a * a).sum() + (b * 3).sum()).backward()
        grads.append([t.grad for t in x + w])
    assert asked == [(True, True), wanted]
    for full, got, need in zip(*grads, (True, True, *wanted)):
        assert torch.equal(full, got) if need else got is None


@pytest.mark.gpu
def test_without_gradients_nothing_is_kept(monkeypatch):
    kept, plain = [], binding.rope_partial_norm_fwd

    def fwd(*args, q_rstd=None, k_rstd=None, **kw):
        kept.append((q_rstd is not None, k_rstd is not None))
        plain(*args, q_rstd=q_rstd, k_rstd=k_rstd, **kw)

    monkeypatch.setattr(binding, "rope_partial_norm_fwd", fwd)
    q, k = torch.randn((2, 5, 4, 64), device=DEV), torch.randn((2, 5, 2, 64), device=DEV)
    want = torch_op.norm_rotary(q.requires_grad_(), k, None, None, None, None)
    with torch.no_grad():
        got = torch_op.norm_rotary(q, k, None, None, None, None)
    alone = torch_op.norm_rotary(q.detach(), None, None, None, None, None)
    assert kept == [(True, True), (False, False), (False, False)] and alone[1] is None
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(alone[0], want[0])
