"""The norm and rotation where their inputs or their work are at an edge:
frequencies that are no numbers, second derivatives, and CTAs that walk over
many tiles of tokens."""
import pytest
import torch

from tests import _rows

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
EPS = 1e-6


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _bf16(g, *shape, std=2.0):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(torch.bfloat16)


@pytest.mark.parametrize("d,R,inter", [(128, 128, False), (64, 32, True), (128, 48, False)])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_frequencies_that_are_no_finite_numbers(fa_mod, cuda_device, d, R, inter, bad):
    """Their pair is NaN at every position, 0 among them, as position times
    frequency is; nothing else changes.  The gradient of the pair is NaN too, and with
    a norm, whose mean runs over the row, that of the whole row."""
    g = _gen(R)
    q, k, gq, gk = (_bf16(g, 50, h, d) for h in (4, 2, 4, 2))
    pos = torch.arange(50, dtype=torch.int32, device=DEV)
    inv = _rows.inv_freq(R).to(DEV)
    w = torch.rand(d, generator=g, device=DEV) + 0.5
    wrong = inv.clone()
    wrong[3] = bad
    i, j = (int(x[3]) for x in _rows.pairs(R, inter))
    hit = torch.zeros(d, dtype=torch.bool, device=DEV)
    hit[i] = hit[j] = True
    for weights in ((), (w, w)):
        want = fa_mod.qk_norm_rope(q, k, pos, inv, *weights, interleaved=inter)
        got = fa_mod.qk_norm_rope(q, k, pos, wrong, *weights, interleaved=inter)
        for a, b in zip(got, want):
            assert torch.isnan(a[..., hit]).all() and torch.equal(a[..., ~hit], b[..., ~hit])
    want = fa_mod.qk_norm_rope_bwd(q, k, gq, gk, pos, inv, interleaved=inter)
    got = fa_mod.qk_norm_rope_bwd(q, k, gq, gk, pos, wrong, interleaved=inter)
    for a, b in zip(got[:2], want[:2]):
        assert torch.isnan(a[..., hit]).all() and torch.equal(a[..., ~hit], b[..., ~hit])
    got = fa_mod.qk_norm_rope_bwd(q, k, gq, gk, pos, wrong, w, w, interleaved=inter)
    assert torch.isnan(got[0]).all() and torch.isnan(got[1]).all()
    assert torch.isnan(got[2][hit]).all() and torch.isfinite(got[2][~hit]).all()

    pages = torch.zeros(4, 2, 16, d, dtype=torch.bfloat16, device=DEV)
    table = torch.arange(4, dtype=torch.int32, device=DEV)[None]
    zero = torch.zeros_like(pos)
    kp, vp = pages.clone(), pages.clone()
    oq = fa_mod.append_paged(q, k, k, kp, vp, table, pos, wrong, w, w, batch_idx=zero, interleaved=inter)
    rq, rk = fa_mod.qk_norm_rope(q, k, pos, wrong, w, w, interleaved=inter)
    rows = kp.transpose(1, 2).reshape(64, 2, d)[:50]
    for a, b in ((oq, rq), (rows, rk)):
        assert torch.isnan(a[..., hit]).all() and torch.equal(a[..., ~hit], b[..., ~hit])
    assert fa_mod.get_device_error() == 0


def test_second_derivatives_are_refused(fa_mod, cuda_device):
    """A loss on the gradients themselves: their graph is not there, and leaving its
    share out without a word would be a wrong gradient."""
    from io_aware_exact_35_b200 import autograd
    g = _gen(3)
    q, k = (_bf16(g, 20, h, 64).requires_grad_() for h in (4, 2))
    w = torch.rand(64, generator=g, device=DEV).requires_grad_()
    pos, inv = torch.arange(20, dtype=torch.int32, device=DEV), _rows.inv_freq(64).to(DEV)
    oq, ok = autograd.qk_norm_rope(q, k, pos, inv, w, w)
    first = torch.autograd.grad(oq.float().square().sum() + ok.float().sum(), (q, k, w), create_graph=True)
    plain = fa_mod.qk_norm_rope_bwd(q.detach(), k.detach(), (2 * oq.detach().float()).bfloat16(), torch.ones_like(k),
                                    pos, inv, w.detach(), w.detach())
    assert torch.equal(first[0], plain[0]) and torch.equal(first[1], plain[1])
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (first[0].float().square().sum() + q.float().sum()).backward()
