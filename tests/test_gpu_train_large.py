"""Tensors of more than 2^31 elements: the rows at the far end against 64 bits (and against the same rows in
a small call, which must agree bit for bit where a row's result depends on that row alone)."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_grouped_fp32_gb300 import moe as m
    yield m
    torch.cuda.empty_cache()


def rand(*shape, dtype=BF16, seed=0):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda", dtype=dtype)


def test_grouped_mm_rows_past_2_31_elements(moe):
    M, K, N = 70000, 64, 32768  # 2.3 G outputs
    a, b = rand(M, K), rand(3, K, N, seed=1)
    offs = torch.tensor([0, 10, 20, M], dtype=torch.int32, device="cuda")
    out = moe.grouped_mm(a, b, offs)
    ref = a[-5:].double() @ b[2].double()
    mag = a[-5:].double().abs() @ b[2].double().abs()
    assert ((out[-5:].double() - ref).abs() <= K * 2.0 ** -23 * mag + 2.0 ** -8 * ref.abs()).all()


def test_wgrad_of_experts_past_2_31_elements(moe):
    E, K, N = 40, 8192, 8192  # 2.7 G outputs
    a, g = rand(E, K), rand(E, N, seed=1)
    offs = torch.arange(E + 1, dtype=torch.int32, device="cuda")
    out = moe.grouped_mm_wgrad(a, g, offs, out_dtype=BF16)
    for e in (0, E - 2, E - 1):
        want = a[e].float()[:, None] * g[e].float()[None]  # one product each: exact in fp32
        assert torch.equal(out[e], want.bfloat16())


def test_swiglu_past_2_31_elements(moe):
    M, f = 80000, 14336  # 2.3 G pre-activations
    gu, dh = rand(M, 2 * f), rand(M, f, seed=1)
    w = torch.rand(M, device="cuda")
    small = [t[-9:].clone() for t in (gu, dh, w)]
    assert torch.equal(moe.swiglu(gu, w)[-9:], moe.swiglu(small[0], small[2]))
    for a, b in zip(moe.swiglu_backward(gu, dh, w), moe.swiglu_backward(small[0], small[1], small[2])):
        assert a is b or torch.equal(a[-9:], b)


def test_block_norm_past_2_31_elements(moe):
    T, d = 540000, 4096  # 2.2 G values
    x, h, w = rand(T, d), rand(T, d, seed=1), torch.rand(d, device="cuda")
    xs, hs = x[-7:].clone(), h[-7:].clone()
    for a, b in zip(moe.block_norm(x, w, h, w), moe.block_norm(xs, w, hs, w)):
        assert torch.equal(a[-7:], b)
    ga = moe.block_norm_backward(x, dy=x, dn=h, w_pre=w, h=h, w_post=w)
    gb = moe.block_norm_backward(xs, dy=xs, dn=hs, w_pre=w, h=hs, w_post=w)
    assert torch.equal(ga["x"][-7:], gb["x"]) and torch.equal(ga["h"][-7:], gb["h"])


def test_adamw_past_2_31_elements(moe):
    n = (1 << 31) + 777
    p, g = rand(n), rand(n, seed=1)
    m, v, ms, vs = moe.adamw_state(p, 8)
    ps, gs = p[-777:].clone(), g[-777:].clone()
    tail = (n - 777) % 256
    assert tail == 0  # the last 777 elements are whole blocks and a rest, as they are alone
    small = moe.adamw_state(ps, 8)
    moe.adamw_step([p], [g], [m], [v], lr=1e-2, m_scales=[ms], v_scales=[vs])
    moe.adamw_step([ps], [gs], [small[0]], [small[1]], lr=1e-2, m_scales=[small[2]], v_scales=[small[3]])
    assert torch.equal(p[-777:], ps)
    assert torch.equal(m[-777:].view(torch.uint8), small[0].view(torch.uint8))
    assert torch.equal(vs[-4:], small[3])
