"""The exit norm's activations and their derivatives element by element, far into their tails (norm_group_gated, include/norm.h).

Weights of 0 make the normed value the bias alone, so that dgate = dy bias act'(gate) with a gate behind the norm, and of one row
dbias = dy act'(bias) without a gate.  Bars, relative to each value: in fp32 the logistic function is off by 1.75 2^-22 (expf one ulp, a sum's rounding,
a division of two ulps), the sigmoid's derivative by two of them and two products: 2^-20; silu's s (1 + z (1 - s)) by z times
s's error as well, up to z = 17, where s becomes 1: 2^-16; in bf16 the rounding, 2^-8, and the approximations' 2^-15
(an exponent of up to 116 rounded in fp32, twice)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

def bar(act, dtype, rounded=True):
    if dtype == torch.float32:
        return 2.0 ** -20 if act == "sigmoid" else 2.0 ** -16
    return 2.0 ** -15 + (2.0 ** -8 if rounded else 0.0)


def slopes(act, z):
    s = 1 / (1 + np.exp(-z))
    c = 1 / (1 + np.exp(z))  # 1 - s without its cancellation
    return s * c if act == "sigmoid" else s * (1 + z * c)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("act,ends", [("sigmoid", (-80, 80)), ("silu", (0, 80))])  # silu's own slope crosses 0 at -1.28
@pytest.mark.parametrize("w", [64, 75, 2048])
def test_derivatives_in_the_tails(w, act, ends, dtype):
    from state_space_model_mamba_gb300 import norm
    r = np.random.default_rng(w)
    zeros = torch.zeros(w, device="cuda")
    x, dy = (torch.from_numpy(r.standard_normal((1, w)).astype(np.float32)).cuda().to(dtype) for _ in range(2))
    z = torch.linspace(*ends, w, device="cuda")[None].to(dtype)
    n64 = [t.double().cpu().numpy() for t in (dy, z)]
    ref = n64[0] * slopes(act, n64[1])
    g = norm.group_norm_gated_backward(dy, x, zeros, bias=zeros + 1, gate=z, activation=act)["dgate"]
    assert np.abs(g.double().cpu().numpy() / ref - 1).max() <= bar(act, dtype)
    b = z[0].float()
    g = norm.group_norm_gated_backward(dy, x, zeros, bias=b, activation=act)["dbias"]  # fp32 whatever the inputs' type
    ref = n64[0][0] * slopes(act, b.double().cpu().numpy())
    assert np.abs(g.double().cpu().numpy() / ref - 1).max() <= bar(act, dtype, False)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_gates_at_the_ends_of_the_type(act, first, dtype):
    """Gates of -+3e38 and +-100: outputs and gradients stay finite, and are 0 where the activation and its slope are."""
    from state_space_model_mamba_gb300 import norm
    g = torch.Generator(device="cuda").manual_seed(3)
    x, dy = (torch.randn(4, 128, generator=g, device="cuda").to(dtype) for _ in range(2))
    z = torch.tensor([-3e38, 3e38 if act == "sigmoid" else 1e4, -100.0, 100.0], device="cuda")[:, None].expand(4, 128).to(dtype).contiguous()
    w = torch.ones(128, device="cuda")
    y = norm.group_norm_gated(x, w, gate=z, groups=2, activation=act, gate_first=first)
    out = norm.group_norm_gated_backward(dy, x, w, gate=z, groups=2, activation=act, gate_first=first)
    for t in (y, out["dx"], out["dgate"], out["dweight"]):
        assert torch.isfinite(t.float()).all()
    assert not y[0].any() and not out["dgate"][0].any() and not out["dx"][0].any()
    if act == "sigmoid":
        assert not out["dgate"][1].any()  # 1 - sigmoid is 0 in fp32
