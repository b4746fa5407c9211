"""The README's recipe for a checkpoint's scales gives the tiles of the format."""
import os
import re

import numpy as np
import pytest
import torch

from oracle import mxfp4 as X

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def recipe():
    text = open(os.path.join(ROOT, "README.md")).read()
    found = [b for b in re.findall(r"```python\n(.*?)```", text, re.S) if "def scale_tiles" in b]
    assert len(found) == 1
    names = {"torch": torch}
    exec(re.search(r"def scale_tiles.*?(?=\n\S)", found[0] + "\nend", re.S).group(0), names)
    return names["scale_tiles"]


@pytest.mark.parametrize("E,rows,cols", [(1, 1, 32), (2, 128, 128), (3, 256, 384), (2, 130, 160), (1, 767, 2080)])
def test_scale_tiles_of_the_readme(E, rows, cols):
    s = np.random.default_rng(rows).integers(0, 255, (E, rows, cols // 32), dtype=np.uint8)
    got = recipe()(torch.from_numpy(s))
    assert np.array_equal(got.numpy(), np.stack([X.tile(q) for q in s]))
