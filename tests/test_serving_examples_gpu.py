"""The serving examples that users are given do what they say: their text is run."""
import os
import re

import pytest
import torch

from tests._parity import check_lse, check_o

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
GUIDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


@pytest.mark.parametrize("prompt_len", [37, 48])
def test_loop_and_samples_of_one_prompt(fa_mod, cuda_device, prompt_len):
    """A prompt in row 2, samples of it in rows 3 to 6 and another request in row 0:
    steps of the loop, with the shared decode equal to decode_paged over the samples' rows."""
    with open(GUIDE) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    loop = next(b for b in blocks if "pages_reserve" in b)
    fork, decode = re.split(r"(?=^full = )", next(b for b in blocks if "pages_fork" in b), flags=re.M)
    g = torch.Generator(device=DEV).manual_seed(prompt_len)
    H, Hkv, d, page_size, P = 8, 2, 64, 16, 90
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)
    names = dict(torch=torch, fa=fa_mod, page_size=page_size, prompt_len=prompt_len, parent=2, first=3, last=7,
                 most_own_pages=4, parents=ints(2, 2, 2, 2), children=ints(3, 4, 5, 6), inv_freq=torch.rand(32, device=DEV),
                 wq=torch.ones(d, device=DEV), wk=torch.ones(d, device=DEV), kpages=rnd(P, Hkv, page_size, d),
                 vpages=rnd(P, Hkv, page_size, d), table=torch.full((7, 12), -1, dtype=torch.int32, device=DEV),
                 lens=torch.zeros(7, dtype=torch.int32, device=DEV), refs=torch.zeros(P, dtype=torch.int32, device=DEV))
    names["pools"] = [names["kpages"], names["vpages"]]
    assert fa_mod.pages_reserve(names["table"], names["refs"], ints(0, 2), ints(5, prompt_len), page_size).all()
    names["lens"].copy_(ints(5, 0, prompt_len, 0, 0, 0, 0))
    exec(fork, names)
    assert names["made"].all() and (names["lens"][3:] == prompt_len).all()
    for step in range(20):
        names["q"], names["k"], names["v"] = rnd(7, H, d), rnd(7, Hkv, d), rnd(7, Hkv, d)
        exec(loop, names)
        assert names["granted"].all()
        want = names["o"][3:].clone(), names["lse"][3:].clone()
        exec(decode, names)
        # both round p and the output to bf16: half a step each on either side
        check_o(names["o"], want[0].double().cpu().numpy())
        check_lse(names["lse"], want[1].double().cpu().numpy())
    assert names["lens"].tolist() == [25, 20] + [prompt_len + 20] * 5
    assert fa_mod.get_device_error() == 0
