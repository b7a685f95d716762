"""Rows of queries and keys at the ends of what qknorm_fwd and qknorm_bwd take: magnitudes far
from one.  References and bounds as in test_gpu_qknorm.py."""
import pytest
import torch

from tests.test_gpu_qknorm import close, make, reference
from xlstm_mlstm_matrix_amd import binding as B

pytestmark = pytest.mark.gpu


def cu(c):
    return {n: None if t is None else t.cuda() for n, t in c.items()}


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("shift,eps", [(50, 1e-6), (56, 0.0), (-30, 0.0), (-44, 0.0)])
@pytest.mark.parametrize("shape,n", [((2, 7, 3, 2, 64), 16), ((1, 9, 2, 1, 33), 5)], ids=str)
def test_rows_of_any_magnitude(io, norm, shift, eps, shape, n):
    """Rows of 2^shift: their squares, and one over them, are ordinary float32 numbers, the
    third power of one over their norm is not."""
    c = make(io, *shape, n, norm, 100, seed=shift)
    c["q"], c["k"] = c["q"] * 2.0 ** shift, c["k"] * 2.0 ** shift
    y, dx, dw = reference(c, norm, eps, "half", 1.25)
    g = cu(c)
    kw = dict(norm=norm, eps=eps, inv_freq=g["f"], positions=g["pos"], amplitude=1.25)
    got = B.qknorm_fwd(g["q"], g["k"], g["wq"], g["wk"], **kw) \
        + B.qknorm_bwd(g["q"], g["k"], g["dyq"], g["dyk"], g["wq"], g["wk"], **kw)
    torch.cuda.synchronize()
    for name, x, (ref, tol) in zip(("yq", "yk", "dq", "dk", "dwq", "dwk"), got, y + dx + dw):
        close(x, ref, tol, "f32" if name[:2] == "dw" else io, f"{io} {norm} 2^{shift} {name}")
