"""Channel-major quantisation of fewer than four channels, over sequences of
whole tiles and ragged ones: tokens of zeros, of the smallest numbers and the
largest, and with a NaN or an infinity in each place, among ordinary ones.  Bits
of the token-major call, and for the special tokens what the definition says."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [1, 2, 3])
@pytest.mark.parametrize("B,L", [(1, 16), (1, 64), (2, 256), (3, 77), (1, 1001), (300, 33)])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_special_tokens(B, L, K, io):
    import torch
    import selective_state_space_80_amd as mamba
    dt = torch.float32 if io == "f32" else torch.bfloat16
    inf, nan = float("inf"), float("nan")
    y = torch.randn((B * L, K), generator=torch.Generator().manual_seed(K * L)).to(dt)
    n = torch.arange(B * L)
    tiny, least = torch.finfo(dt).smallest_normal, torch.finfo(dt).min
    y[n % 13 == 1] = 0.0
    y[n % 13 == 2] = -0.0
    y[n % 13 == 3] = tiny
    y[n % 13 == 4] *= 1e-39  # denormals
    y[n % 13 == 6] = least
    for k in range(K):
        y[n % 13 == 7 + k, k] = nan
        y[n % 13 == 10 + k, k] = inf if k % 2 else -inf
    q, s = mamba.quantize_int8(y.view(B, L, K).transpose(1, 2).contiguous().cuda(), channel_major=True)
    q2, s2 = mamba.quantize_int8(y.view(B, L, K).cuda())
    assert torch.equal(q, q2) and torch.equal(s.view(torch.int32), s2.view(torch.int32))
    q, s = q.cpu().view(B * L, K), s.cpu().view(-1)
    zero, odd = (y == 0).all(-1), ~torch.isfinite(y).all(-1)
    assert (s[zero] == 0).all() and not q[zero].any()
    assert torch.isnan(s[odd]).all() and not q[odd].any()
    assert (q[n % 13 == 3] == 127).all() and (q[n % 13 == 6] == -127).all()
    fine = ~odd & ~zero
    top = y.double().abs().amax(-1)
    assert torch.equal(s[fine], (top[fine] / 127.0).float())
    v = y.double()[fine] * 127.0 / top[fine, None]
    assert ((q[fine].double() - v).abs() <= 0.5 + 1e-12).all()
