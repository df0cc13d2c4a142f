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


# ---------------------------------------------------------------- many tiles a CTA
def _tiles_case(seed, T, H, Hkv, d, inter, R, positive):
    """Token-major slices of one projection.  positive: one sign everywhere, so that
    the sums of the weights' gradients lose none of their size to cancellation."""
    g = _gen(seed)
    qkv, up = _bf16(g, T, H + 2 * Hkv, d), _bf16(g, T, H + Hkv, d)
    if positive:
        qkv, up = qkv.abs() + 0.25, up.abs() + 0.25
    pos = torch.randint(-10 ** 6, 10 ** 6, (T,), generator=g, device=DEV, dtype=torch.int32)
    if positive:  # no turn: the products keep their sign
        pos.zero_()
    w = [torch.rand(d, generator=g, device=DEV) + 0.5 for _ in range(2)]
    return qkv, up, pos, _rows.inv_freq(R).to(DEV), w


CASES = [(19001, 8, 3, 128, False, 128), (19003, 5, 2, 64, True, 32), (40011, 2, 1, 64, False, 64),
         (20011, 3, 4, 128, True, 128), (19001, 16, 2, 128, False, 48)]
"""The passes run on at most 592 CTAs of 128 threads, and d / 16 threads take a token
or a share of its heads: at most 16 (d = 128) or 32 (d = 64) tokens a tile, so that
each CTA walks over two tiles or more, the last one ragged."""


@pytest.mark.parametrize("T,H,Hkv,d,inter,R", CASES)
def test_forward_over_many_tiles(fa_mod, cuda_device, T, H, Hkv, d, inter, R):
    qkv, _, pos, inv, w = _tiles_case(T + H, T, H, Hkv, d, inter, R, False)
    q, k = qkv[:, :H], qkv[:, H:H + Hkv]
    got = fa_mod.qk_norm_rope(q, k, pos, inv, *w, interleaved=inter)
    a = _rows.angles(pos, inv, 3)
    for x, o, wt, n in zip((q, k), got, w, "qk"):
        _rows.within(o, _rows.forward(x, wt, a, R, inter, EPS), _rows.forward_bound(x, wt, a, R, inter, EPS), n)
    assert fa_mod.get_device_error() == 0


@pytest.mark.parametrize("positive", [False, True])
@pytest.mark.parametrize("T,H,Hkv,d,inter,R", CASES)
def test_backward_over_many_tiles(fa_mod, cuda_device, T, H, Hkv, d, inter, R, positive):
    """The weights' gradients within a bound that a missing tile does not meet."""
    qkv, up, pos, inv, w = _tiles_case(T - H, T, H, Hkv, d, inter, R, positive)
    q, k, gq, gk = qkv[:, :H], qkv[:, H:H + Hkv], up[:, :H], up[:, H:]
    got = fa_mod.qk_norm_rope_bwd(q, k, gq, gk, pos, inv, *w, interleaved=inter)
    assert fa_mod.get_device_error() == 0
    a = _rows.angles(pos, inv, 3)
    for i, (x, gr, wt, n) in enumerate(zip((q, k), (gq, gk), w, "qk")):
        dx, dw, bx, _ = _rows.backward(x, wt, gr, a, R, inter, EPS)
        _rows.within(got[i], dx, bx, "d" + n)
        # The terms of the sum and their sizes.  A term is right to 2 F32 of its size.
        # It then passes through the sums of its thread, of the threads with the same
        # columns in its warp (8 at most: 3), of 4 warps, and of the CTAs' partials, of
        # which a thread takes every 32nd (19 of 592) and 32 threads meet (5): as many
        # roundings of 2^-24 as there are sums behind it.  The 592 CTAs are shared
        # between q and k by their heads, and a tensor's rows spread over its CTAs'
        # groups as evenly as whole tiles and heads allow: twice the average.
        xh = x.double() * _rows.normed(x, wt, EPS)[1]
        dy = _rows.rotate(gr.double(), -a, R, inter)
        size = gr.double().abs()
        ii, jj = _rows.pairs(R, inter)
        both = size[..., ii] + size[..., jj]
        size[..., ii] = size[..., jj] = both
        heads = x.shape[1]
        groups = 592 * heads // (H + Hkv) * (128 // (d // 16))
        depth = 2 * -(-T * heads // groups) + 3 + 4 + 19 + 5
        bound = (2 * _rows.F32 + depth * 2.0 ** -24) * (size * xh.abs()).sum((0, 1))
        _rows.within(got[2 + i], dw, bound, f"d{n}_weight")
        # what the bound is worth: a lost tile takes away a token's heads at least
        for t in (0, T // 2, T - 1):
            assert ((dy[t] * xh[t]).sum(0).abs() > bound).any()


@pytest.mark.parametrize("T,H,Hkv,d,inter,R", CASES)
def test_append_over_many_tiles(fa_mod, cuda_device, T, H, Hkv, d, inter, R):
    """Keys and values of tokens in any order, some of them padding, against the
    64-bit rows at their places; places of no token stay as they were."""
    qkv, _, pos, inv, w = _tiles_case(T * 2 + H, T, H, Hkv, d, inter, R, False)
    q, k, v = qkv.split([H, Hkv, Hkv], 1)
    page, cols = 16, -(-T // (3 * 16)) + 1
    g = _gen(T)
    P = 3 * cols
    table = torch.randperm(P, generator=g, device=DEV).to(torch.int32).reshape(3, cols)
    at = torch.randperm(3 * cols * page, generator=g, device=DEV)[:T]
    seq, place = (at // (cols * page)).to(torch.int32), (at % (cols * page)).to(torch.int32)
    pad = torch.rand(T, generator=g, device=DEV) < 0.05
    place[pad] = -1
    kp = torch.full((P, Hkv, page, d), 7.0, dtype=torch.bfloat16, device=DEV)
    vp = kp.clone()
    out = torch.full((T, H, d), 7.0, dtype=torch.bfloat16, device=DEV)
    fa_mod.append_paged(q, k, v, kp, vp, table, pos, inv, *w, batch_idx=seq, cache_positions=place, interleaved=inter,
                        q_out=out)
    assert fa_mod.get_device_error() == 0
    a = _rows.angles(pos, inv, 3)
    keep = ~pad
    rows = table[seq[keep].long(), place[keep].long() // page].long() * page + place[keep].long() % page
    flat = lambda pool: pool.transpose(1, 2).reshape(P * page, Hkv, d)
    _rows.within(out[keep], _rows.forward(q, w[0], a, R, inter, EPS)[keep],
                 _rows.forward_bound(q, w[0], a, R, inter, EPS)[keep], "q")
    _rows.within(flat(kp)[rows], _rows.forward(k, w[1], a, R, inter, EPS)[keep],
                 _rows.forward_bound(k, w[1], a, R, inter, EPS)[keep], "k")
    assert torch.equal(flat(vp)[rows], v[keep])
    rest = torch.ones(P * page, dtype=torch.bool, device=DEV)
    rest[rows] = False
    assert (out[pad] == 7).all() and (flat(kp)[rest] == 7).all() and (flat(vp)[rest] == 7).all()
