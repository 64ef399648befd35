"""The workspace a caller gives to the binding: its size counts in bytes whatever
its type, and memory that the call's GPU does not own is refused before any call."""
import pytest

import selective_state_space_80_amd as mamba


def test_workspace_is_checked_before_the_call():
    import torch
    gpu = torch.device("cuda", 0)  # nothing is put on it
    host = torch.empty(4096, dtype=torch.uint8)
    with pytest.raises(ValueError, match="workspace is on cpu"):
        mamba._workspace(host, 16, gpu)
    with pytest.raises(ValueError, match="contiguous"):
        mamba._workspace(host[::2], 16, host.device)
    for dt, size in ((torch.uint8, 1), (torch.bfloat16, 2), (torch.float32, 4)):
        given = torch.empty(100, dtype=dt)
        kept, count = mamba._workspace(given, 16, host.device)
        assert kept is given and count == 100 * size
    made, count = mamba._workspace(None, 33, host.device)
    assert made.device == host.device and count == made.numel() * made.element_size() >= 33


@pytest.mark.gpu
def test_calls_take_a_workspace_of_any_type():
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    M, D = 700, 300
    dy, h, w = rand(M, D), rand(M, D), rand(D)
    need = mamba.rms_norm_bwd_workspace_size(M, D)
    want = mamba.rms_norm_bwd(dy, h, w)
    for dt in (torch.uint8, torch.float32, torch.int64):
        ws = torch.empty(-(-need // dt.itemsize), dtype=dt, device="cuda")
        got = mamba.rms_norm_bwd(dy, h, w, workspace=ws)
        assert all(torch.equal(got[k], want[k]) for k in want), dt
    B, D, L, N = 1, 64, 500, 16
    x, dt_, Bm, Cm = rand(B, D, L), 0.1 * rand(B, D, L), rand(B, L, N), rand(B, L, N)
    A = -torch.rand((D, N), generator=g, device="cuda") - 0.1
    need = mamba.selective_scan_fwd_workspace_size(B, D, L, N)
    y = mamba.selective_scan_fwd(x, dt_, A, Bm, Cm)
    assert torch.equal(mamba.selective_scan_fwd(x, dt_, A, Bm, Cm, workspace=torch.empty(-(-need // 4), device="cuda")), y)
    for call in (lambda ws: mamba.rms_norm_bwd(dy, h, w, workspace=ws),
                 lambda ws: mamba.selective_scan_fwd(x, dt_, A, Bm, Cm, workspace=ws),
                 lambda ws: mamba.selective_scan_bwd(x, dt_, A, Bm, Cm, y, workspace=ws)):
        with pytest.raises(ValueError):
            call(torch.empty(1 << 22, dtype=torch.uint8))  # host memory
