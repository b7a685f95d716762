"""linattn_step on states of all the sizes that its kernels are chosen by: those
that the cache holds and those streamed past it, in place, from one tensor into
another, and from the zero state.  Float64 on the device; bounds as in
test_gpu_linattn's test_step."""
import pytest
import torch

from xlstm_mlstm_matrix_amd import binding as B

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
U = 2.0 ** -24


@pytest.mark.parametrize("dk,dv", [(256, 512), (240, 272), (112, 208), (128, 128), (64, 112)], ids=str)
@pytest.mark.parametrize("mb", [150, 250, 400])   # of 2^20 bytes: streamed never, from a tensor into another, always
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_step_of_large_states(io, mb, dk, dv):
    H = 5
    Bn = (mb << 20) // (H * dk * dv * 4)
    r = torch.Generator(device="cuda").manual_seed(dk + dv)
    q, k = (torch.randn((Bn, H, dk), generator=r, device="cuda").to(DT[io]) for _ in range(2))
    v = torch.randn((Bn, H, dv), generator=r, device="cuda").to(DT[io])
    S = torch.randn((Bn, H, dk, dv), generator=r, device="cuda")
    g = torch.linspace(-2.0, 0.0, H, device="cuda")
    print(f"[linattn] step {io} {Bn} x {H} x {dk} x {dv}", flush=True)
    o, S1 = B.linattn_step(q, k, v, g, S, scale=0.1, inplace=False)
    S2 = S.clone()
    o2, S2 = B.linattn_step(q, k, v, g, S2, scale=0.1)
    z, Z = B.linattn_step(q, k, v, g, scale=0.1)
    torch.cuda.synchronize()
    # o's sum over rows is split otherwise in the streaming kernel
    assert torch.equal(S1, S2)
    gam = torch.exp(g.double())[:, None, None]
    for b in range(0, Bn, 64):     # 64 sequences at a time: float64 copies of 1 GB
        n = slice(b, b + 64)
        kv = k[n].double()[..., None] * v[n].double()[..., None, :]
        for x, Sx, S0 in ((o, S1, S[n].double()), (o2, S2, S[n].double()), (z, Z, torch.zeros((), device="cuda", dtype=torch.float64))):
            ref, A = gam * S0 + kv, gam * S0.abs() + kv.abs()
            assert bool(((Sx[n].double() - ref).abs() <= 16 * U * A).all())
            ro = (q[n].double()[..., None, :] @ ref)[..., 0, :] * 0.1
            Ao = (q[n].double().abs()[..., None, :] @ A)[..., 0, :] * 0.1
            assert bool(((x[n].double() - ro).abs() <= HALF[io] * 1.01 * ro.abs() + (dk + 64) * U * Ao).all())
