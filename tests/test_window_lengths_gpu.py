"""Window attention of one token and of batches in which nobody is present, in every form: o = v, lse the score and no gradient of
q and k beyond what fp32 sums of 64 terms of size 1 differ by; zeros throughout."""
import numpy as np
import pytest
import window_util as wu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bf16,simt", [(False, False), (True, False), (True, True)])
@pytest.mark.parametrize("valid", [None, [1, 0, 1], [0, 0, 0]])
@pytest.mark.parametrize("W,sinks", [(1, 0), (7, 2)])
def test_one_token(W, sinks, valid, bf16, simt):
    from state_space_model_mamba_gb300 import window
    T = torch.bfloat16 if bf16 else torch.float32
    x = wu.draw(3, 1, 4, 2, 64, 5, bf16)
    d = {n: torch.from_numpy(a).cuda().to(T) for n, a in x.items()}
    vl = None if valid is None else torch.tensor(valid, dtype=torch.int32, device="cuda")
    o, lse = window.window_forward(d["q"], d["k"], d["v"], W, sinks, valid_len=vl, simt=simt)
    g = window.window_backward(d["q"], d["k"], d["v"], o, lse, d["do"], W, sinks, valid_len=vl, simt=simt)
    on = np.ones(3) if valid is None else np.array(valid)
    at = on[:, None, None, None]
    assert np.array_equal(o.float().cpu().numpy(), np.repeat(x["v"], 2, 2) * at)
    s = (x["q"].astype(float) * np.repeat(x["k"], 2, 2)).sum(-1).transpose(0, 2, 1) / 8 * on[:, None, None]
    assert np.abs(lse.double().cpu().numpy() - s).max() < 1e-5
    assert g["dq"].float().abs().max() < 64 * 2 ** -22 and g["dk"].float().abs().max() < 64 * 2 ** -22
    ref = x["do"].reshape(3, 1, 2, 2, 64).astype(float).sum(3) * at
    dv = g["dv"].double().cpu().numpy()
    assert np.abs(dv - ref).max() <= (2.0 ** -8 if bf16 else 2.0 ** -20) * max(np.abs(ref).max(), 1e-30)
    absent = torch.tensor(on == 0, device="cuda")
    for t in (g["dq"], g["dk"], g["dv"]):
        assert not t[absent].any()


@pytest.mark.parametrize("bf16,simt", [(False, False), (True, False), (True, True)])
def test_nobody_is_present(bf16, simt):
    from state_space_model_mamba_gb300 import window
    T = torch.bfloat16 if bf16 else torch.float32
    d = {n: torch.full((2, 300, h, 64), float("nan"), device="cuda", dtype=T) for n, h in (("q", 4), ("k", 2), ("v", 2), ("do", 4))}
    vl = torch.zeros(2, dtype=torch.int32, device="cuda")
    o, lse = window.window_forward(d["q"], d["k"], d["v"], 50, 3, valid_len=vl, simt=simt, check_status=True)
    g = window.window_backward(d["q"], d["k"], d["v"], o, lse, d["do"], 50, 3, valid_len=vl, simt=simt, check_status=True)
    for t in (o, lse, *g.values()):
        assert torch.equal(t, torch.zeros_like(t))
