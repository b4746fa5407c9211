"""The README's example of trained experts runs as it stands, and its two ways agree:
the steps round g and u, the experts' rows and gh to bf16 between them, the one call does not.
Both are off from the exact result by a few roundings of 2^-8 each (at most seven in a
row), as norms over the whole; and the codes that differ stand for values 2^-7 apart."""
import os
import re

import pytest
import torch

import moe_decode_ffn_gb300 as m

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_trained_experts_of_the_readme():
    text = open(os.path.join(ROOT, "README.md")).read()
    found = [b for b in re.findall(r"```python\n(.*?)```", text, re.S) if "si_moe_experts(" in b]
    assert len(found) == 1
    m.build()
    torch.manual_seed(3)
    names = {"torch": torch, "m": m}
    exec(found[0], names)
    one = names["y"], names["gx"], names["gw"], names["ggate_up"], names["gdown"]
    for a, b in zip(one, (names["y2"], *names["steps"])):
        assert a.shape == b.shape and a.dtype == b.dtype and bool(torch.isfinite(a).all())
        a, b = a.detach().double(), b.detach().double()
        assert float((a - b).norm()) <= (2 * 7 * 2.0 ** -8 + 2.0 ** -7) * float(b.norm())
