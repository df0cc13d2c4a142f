"""Every call of the native binding that takes a workspace refuses one that is no
contiguous memory of its device, before any launch."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def _calls(fa_mod):
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)
    q = torch.ones(3, 4, 64, dtype=torch.bfloat16, device=DEV)
    k = torch.ones(3, 2, 64, dtype=torch.bfloat16, device=DEV)
    w, inv = torch.ones(64, device=DEV), torch.ones(32, device=DEV)
    pool = torch.ones(9, 2, 16, 64, dtype=torch.bfloat16, device=DEV)
    table = torch.full((4, 3), -1, dtype=torch.int32, device=DEV)
    lens, refs = ints(0, 0, 0, 0), torch.zeros(9, dtype=torch.int32, device=DEV)
    prefix, own = ints(0, 1, 2)[None], ints(3, 4, 5)[:, None]
    return {
        "qk_norm_rope_bwd": lambda **kw: fa_mod.qk_norm_rope_bwd(q, k, q, k, ints(0, 1, 2), inv, w, w, **kw),
        "qk_norm_rope_bwd without weights": lambda **kw: fa_mod.qk_norm_rope_bwd(q, k, q, k, ints(0, 1, 2), inv, **kw),
        "pages_reserve": lambda **kw: fa_mod.pages_reserve(table, refs, ints(0), ints(20), 16, **kw),
        "pages_fork": lambda **kw: fa_mod.pages_fork([pool], table, lens, refs, ints(0), ints(1), 16, **kw),
        "pages_compact": lambda **kw: fa_mod.pages_compact([pool], table, refs, **kw),
        "decode_shared": lambda **kw: fa_mod.decode_shared(q, pool, pool, prefix, ints(40), own, ints(1, 2, 3), **kw),
    }


@pytest.mark.parametrize("name", ["qk_norm_rope_bwd", "qk_norm_rope_bwd without weights", "pages_reserve", "pages_fork",
                                  "pages_compact", "decode_shared"])
def test_refusals(fa_mod, cuda_device, name):
    call = _calls(fa_mod)[name]
    with pytest.raises(ValueError, match="workspace must be on cuda:0, got cpu"):
        call(workspace=torch.empty(1 << 24, dtype=torch.uint8))
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        call(workspace=torch.empty(1, dtype=torch.uint8, device=DEV).expand(1 << 24))
    call(workspace=torch.empty(1 << 22, dtype=torch.float32, device=DEV))  # any type will do
    assert fa_mod.get_device_error() == 0
