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
