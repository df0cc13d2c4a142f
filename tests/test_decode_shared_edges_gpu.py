"""fa.decode_shared where its inputs or its work are at an edge: groups that
overlap, values that are no numbers, maxima that move inside a CTA, rings that
wrap and batches of many sequences."""
import numpy as np
import pytest
import torch

from tests.test_decode_shared_gpu import DEV, Case, _run

pytestmark = pytest.mark.gpu


def _owner(cu, B):
    """The group of each batch entry: a group that runs backwards or leaves the
    batch has none, and no group begins before the end of an earlier one."""
    owner, end = [None] * B, 0
    for g, (a, b) in enumerate(zip(cu, cu[1:])):
        if 0 <= a <= b <= B:
            for i in range(max(a, end), b):
                owner[i] = g
            end = max(end, b)
    return owner


@pytest.mark.parametrize("cu,B,H,Hkv,d", [
    ([0, 5, 3, 8], 9, 8, 2, 64),                 # 3 and 4 in two groups, 8 in none
    ([0, 100, 20, 128], 128, 8, 2, 128),         # row tiles of the overlap beyond those of disjoint groups
    ([0, 100, 0, 100], 110, 4, 4, 64),           # the same entries twice
    ([5, -1, 3, 20], 9, 8, 2, 64),               # no group is left
    ([2, 9, 1, 4, 2, 7], 9, 40, 1, 64),          # back and forth
    ([2 * g for g in range(34)] + [10, 90, 20, 91], 95, 8, 2, 64),  # behind the first 32 groups
])
def test_groups_that_overlap(fa_mod, cuda_device, cu, B, H, Hkv, d):
    G = len(cu) - 1
    c = Case(B + G, H, Hkv, d, 16, [0] * G, [90 + 61 * g % 700 for g in range(G)], [(23 * b) % 50 for b in range(B)])
    c.cu = torch.tensor(cu, dtype=torch.int32)
    c.group = _owner(cu, B)
    o, lse = fa_mod.decode_shared(*c.dev(), cu_batch=c.cu.to(DEV))
    assert fa_mod.get_device_error() == 1
    c.check(o, lse)
    again = fa_mod.decode_shared(*c.dev(), cu_batch=c.cu.to(DEV))
    assert fa_mod.get_device_error() == 1
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("B,H,Hkv,d,plen,lens", [
    (5, 8, 2, 64, 100, [0, 3, 40, 700, 9]),            # one key tile, 128 rows a CTA
    (5, 8, 2, 128, 2500, [0] * 5),                     # the prefix alone, several tiles
    (5, 8, 8, 128, 0, [1, 3, 40, 700, 16]),            # own keys alone
    (160, 8, 4, 64, 1300, [b % 60 for b in range(160)]),   # 256 rows a CTA, one warp a row in the merge
])
def test_values_that_are_no_numbers(fa_mod, cuda_device, B, H, Hkv, d, plen, lens):
    """A query with a NaN gives NaN and no other row does; so do a NaN key for the
    queries over it, and a NaN value in its column alone.  (A row all of whose scores
    are NaN is not a row without keys, whose answer is 0.)"""
    c = Case(B + H, H, Hkv, d, 16, [B], [plen], lens)
    args, cu = c.dev(), c.cu.to(DEV)
    o, lse = fa_mod.decode_shared(*args, cu_batch=cu)
    args[0][3, 1, 5] = float("nan")
    args[0][B - 1, H - 1] = float("nan")
    on, ln = fa_mod.decode_shared(*args, cu_batch=cu)
    hit = torch.zeros(B, H, dtype=torch.bool, device=DEV)
    hit[3, 1] = hit[B - 1, H - 1] = True
    assert torch.isnan(on[hit]).all() and torch.isnan(ln[hit]).all()
    assert torch.equal(on[~hit], o[~hit]) and torch.equal(ln[~hit], lse[~hit])

    # key 2 of the prefix, else of sequence 3; key/value head 1
    args = c.dev()
    page = int(c.ptable[0, 0]) if plen else int(c.table[3, 0])
    r = H // Hkv
    hit = torch.zeros(B, H, dtype=torch.bool, device=DEV)
    hit[slice(None) if plen else 3, r:2 * r] = True
    args[1][page, 1, 2, 7] = float("nan")
    on, ln = fa_mod.decode_shared(*args, cu_batch=cu)
    assert torch.isnan(on[hit]).all() and torch.isnan(ln[hit]).all()
    assert torch.equal(on[~hit], o[~hit]) and torch.equal(ln[~hit], lse[~hit])
    args = c.dev()
    args[2][page, 1, 2, 7] = float("nan")
    on, ln = fa_mod.decode_shared(*args, cu_batch=cu)
    assert torch.isnan(on[hit][:, 7]).all() and torch.equal(ln, lse)
    on[hit, 7] = o[hit, 7]
    assert torch.equal(on, o)
    assert fa_mod.get_device_error() == 0


# ---------------------------------------------------------------- many key tiles a CTA
def _towards_the_queries(c, seed, jumps):
    """Queries about one direction, and keys of no direction but at `jumps`: key
    `at` of a list then scores `height` (log2 units) above those before it, so that
    with 8 to 16 the maximum moves by more than is let stand while what came before keeps
    its weight: hundreds of keys at 2^-10 against one.  Lists: prefixes, then own keys."""
    g = torch.Generator().manual_seed(seed)
    way = torch.randint(0, 2, (c.d,), generator=g) * 2.0 - 1
    c.q = (way + 0.2 * torch.randn(c.q.shape, generator=g)).to(torch.bfloat16)
    unit = np.log(2.0) / np.sqrt(c.d)  # of the direction for one log2 unit of the score
    for i, ((k, v), marks) in enumerate(zip(c.keys, jumps)):
        k.copy_((0.02 * torch.randn(k.shape, generator=g)).to(torch.bfloat16))
        for at, height in marks:
            k[at] = (height * unit * way).to(torch.bfloat16)
        table, row = (c.ptable, i) if i < len(c.plens) else (c.table, i - len(c.plens))
        for j in range(-(-k.shape[0] // c.page)):
            m = min(c.page, k.shape[0] - j * c.page)
            c.kp[int(table[row, j]), :, :m] = k[j * c.page:j * c.page + m].transpose(0, 1)


# The prefix CTAs of these shapes are 148 for one split (37 heads x 4 groups), the
# device's SMs, so that a split more would be a second round: every CTA takes all
# key tiles of its group's prefix.
@pytest.mark.parametrize("page", [1, 4, 16, 256])
@pytest.mark.parametrize("H,per", [(148, 33), (37, 3)])  # 132 rows a group: 256 a CTA; 3 rows: 128
@pytest.mark.parametrize("d", [64, 128])
def test_every_key_tile_in_one_split(fa_mod, cuda_device, page, H, per, d):
    """The ring of key tiles wraps several times, by TMA and row by row, and the
    running maximum moves inside a CTA, early, late, twice and at the very end."""
    plens = [900, 1301, 640, 70]
    B = 4 * per
    c = Case(page + H, H, 37, d, page, [per] * 4, plens, [(5 * b) % 40 for b in range(B)])
    marks = [[(300, 10), (700, 20)], [(130, 9), (1300, 19)], [(639, 10)], [(69, 12)]] + [[]] * B
    _towards_the_queries(c, page, marks)
    size = fa_mod.lib().fa_decode_shared_workspace_size
    got = size(B, H, 37, 4, page, c.ptable.shape[1], 0, d)
    assert got == 4 * B * H * d + 8 * B * H + (-4 * B * H * d) % 256 + (-8 * B * H) % 256, "more than one split"
    o, lse = _run(fa_mod, c)
    c.check(o, lse, only=[0, 1, per - 1, per, 2 * per, 3 * per - 1, 4 * per - 1])


@pytest.mark.parametrize("H,Hkv,d,page", [(8, 2, 128, 16), (4, 4, 64, 16), (24, 2, 128, 4), (20, 1, 64, 64)])
def test_the_maximum_moves_along_own_keys(fa_mod, cuda_device, H, Hkv, d, page):
    """Long own parts, of which a warp takes many steps of 16 keys: the maximum
    moves inside a warp's stretch and what was summed before keeps its weight."""
    lens = [20000, 0, 17, 9000, 640]
    c = Case(H + page, H, Hkv, d, page, [2, 1], [200, 0], lens)
    marks = [[(150, 10)], [], [(4000, 9), (4100, 18), (12345, 27)], [], [(16, 10)], [(20, 10), (8990, 20)], [(639, 12)]]
    _towards_the_queries(c, H, marks)
    o, lse = _run(fa_mod, c)
    c.check(o, lse)


@pytest.mark.parametrize("B,L", [(700, 9000), (1100, 6000)])
def test_splits_chosen_for_many_sequences(fa_mod, cuda_device, B, L):
    """The number of prefix splits is chosen from the lengths of more sequences than
    a CTA has threads; lengths that fill it, and few, give the same answers."""
    c = Case(B, 2, 1, 64, 16, [B - 1], [L], [(29 * b) % 128 for b in range(B)])
    some = [0, 1, 511, 512, 513, 640, B - 2, B - 1]
    o, lse = _run(fa_mod, c)
    c.check(o, lse, only=some)
    again = _run(fa_mod, c)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    c.keys[1:] = [(k[:0], v[:0]) if b % 100 else (k, v) for b, (k, v) in enumerate(c.keys[1:])]
    c.lens = [k.shape[0] for k, _ in c.keys[1:]]
    o, lse = _run(fa_mod, c)
    c.check(o, lse, only=some)
