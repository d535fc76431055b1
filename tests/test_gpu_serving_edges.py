"""GPU tests of the serving operators where a call differs from the ordinary one: another call's
workspace, scores at fp32's end, policies past a cache's capacity, layers that rotate.  Tolerances
are the bounds of oracle/serving.py unless a test derives its own."""
import numpy as np
import pytest
import torch

from intra_spatial_pipelining_gb300 import sgp
from oracle import serving as S
from tests.test_gpu_serving import D, NAN, Prefix, bf16, f64, ints, within

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------------------
# prefix attention
# ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("nq,nkv,cap,sizes", [
    (64, 8, 1024, (375, 374, 93, 5, 1)), (16, 1, 1281, (512, 300, 2)), (5, 5, 257, (300, 299, 150, 31)),
    (12, 4, 130, (512, 200, 1))])
def test_prefix_attention_in_the_workspace_of_a_larger_call(nq, nkv, cap, sizes):
    """One workspace, sized for the first of `sizes` sequences and for a capacity of `cap`, serves the
    smaller calls, and none writes behind the size that its own arguments ask for."""
    dims = sgp.make_heads(nq, nkv)
    size = sgp.sgp_prefix_attention_workspace_bytes
    room = size(dims, sizes[0], cap, 2)
    buf = torch.empty(room + 65536, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(nq + cap)
    for T in sizes:
        for c in (cap, cap // 2):
            # a few long sequences and the others short: every chunk count, little to check
            own = [c if t < 3 else int(rng.integers(0, 9)) for t in range(T)]
            x = Prefix(T + c, T, nq, nkv, [70, 3], own, [t % 3 - 1 for t in range(T)], cap=c)
            need = size(dims, T, c, 2)
            assert need <= room
            for n in (room, need):
                buf.fill_(165)
                buf[:64] = 0
                x.ws = buf[:n]
                x.o.fill_(NAN)
                x.run()
                x.check()
                assert (buf[need:] == 165).all()
