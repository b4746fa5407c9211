"""Launches whose static and dynamic shared memory together pass 48 KB while the
dynamic part alone does not: each size as the first of its process, so that no
larger call has raised the kernel's limit before."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def alone(code):
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


# the second launch of a long sort: 64 (E + 1) dynamic bytes beside 4176 static ones
@pytest.mark.parametrize("E", [701, 702, 766, 767, 768])
def test_long_sort_first_in_its_process(E):
    alone(f"""
import torch, moe_decode_ffn_gb300 as m
from oracle import mxfp4 as X
ids = torch.randint(-1, {E} + 2, (4097, 1), generator=torch.Generator().manual_seed({E}), dtype=torch.int32)
got = m.si_moe_sort(ids.cuda(), {E})
assert all((a.cpu().numpy() == b).all() for a, b in zip(got, X.sort(ids.numpy(), {E})))
print("same")
""")


def test_long_sort_grows_and_shrinks():
    """Several sizes in one process, the limit raised in between."""
    alone("""
import torch, moe_decode_ffn_gb300 as m
from oracle import mxfp4 as X
for E in (3, 702, 767, 1024, 702, 850, 5):
    ids = torch.randint(0, E, (700, 6), generator=torch.Generator().manual_seed(E), dtype=torch.int32)
    got = m.si_moe_sort(ids.cuda(), E)
    assert all((a.cpu().numpy() == b).all() for a, b in zip(got, X.sort(ids.numpy(), E)))
print("same")
""")


def test_experts_of_a_long_batch_first_in_their_process():
    """The expert FFN sorts with the same kernel: one call equals its two halves."""
    alone("""
import torch, moe_decode_ffn_gb300 as m
E, H, I, T, k = 740, 64, 32, 2050, 2
g = torch.Generator(device="cuda").manual_seed(1)
draw = lambda *s: torch.randn(*s, generator=g, device="cuda")
experts = m.Mxfp4Experts.quantize(draw(E, I, H), draw(E, I, H), draw(E, H, I))
x = draw(T, H).to(torch.bfloat16)
ids = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
w = torch.rand(T, k, generator=g, device="cuda")
y = m.si_moe_ffn_mxfp4(experts, x, ids, w)
h = [m.si_moe_ffn_mxfp4(experts, x[a:b], ids[a:b], w[a:b]) for a, b in ((0, 1025), (1025, T))]
assert torch.equal(y, torch.cat(h))
print("same")
""")


def test_norm_of_rows_that_fill_the_default():
    """4 dynamic bytes a value beside 32 static ones."""
    alone("""
import torch, moe_decode_ffn_gb300 as m
n = 12288
g = torch.Generator().manual_seed(2)
a, b = (torch.randn(n, generator=g).to(torch.bfloat16) for _ in range(2))
s, y, _ = m.si_add_rmsnorm3(a.cuda(), b.cuda(), None, torch.ones(n, dtype=torch.bfloat16, device="cuda"))
want = (a.float() + b.float()).to(torch.bfloat16)
assert torch.equal(s.cpu(), want)
print("same")
""")
