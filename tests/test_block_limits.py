"""Limits of the block operators' entry points on the CPU: refusals that happen before any HIP
call, what is accepted as far as the next check, and the words of the errors."""
import pytest

from mlstm_matrix_memory_amd import binding as b
from test_block_abi import P, _far, _scan_bwd, refused


def test_more_threads_than_the_parameter_sums_take():
    """The backward's sums over the pieces run 1024 threads for every 64 channels and each of N + 2
    gradients; past 2^32 of them nothing of the call is launched."""
    b.load_library()
    D, N = 1 << 23, 64
    names = ("x", "dtp", "A", "Bm", "Cm", "skip", "bias", "z", "h0", "dy", "dh", "gx", "gdt", "gz", "gB", "gC", "gA", "gD",
             "gb", "gh", "ws")
    far = _far({k: P[i] for i, k in enumerate(names)})
    wide = {k: D for k in ("xs", "dts", "zs", "ds", "gxs", "gdts", "gzs")}
    narrow = {k: N for k in ("bs", "cs", "gBs", "gCs")}
    status = _scan_bwd(b.load_library(), B=1, S=1, rows=1, D=D, N=N, n=1 << 45, **wide, **narrow, **far)
    refused(status, "more threads than one launch takes", b.MLSTM_ERR_UNSUPPORTED)


@pytest.mark.parametrize("name,call", [
    ("x", lambda pkg, h, f: pkg.mlstm_rms_norm_fwd(h, f)),
    ("x", lambda pkg, h, f: pkg.mlstm_rms_norm_quant(h, f)),
    ("residual", lambda pkg, h, f: pkg.mlstm_rms_norm_fwd(h.float(), f, residual=h)),
    ("residual_out", lambda pkg, h, f: pkg.mlstm_rms_norm_fwd(h.float(), f, residual_out=h)),
    ("r", lambda pkg, h, f: pkg.mlstm_rms_norm_bwd(h, f, h.float())),
    ("dy", lambda pkg, h, f: pkg.mlstm_rms_norm_bwd(h.float(), f, h)),
    ("x", lambda pkg, h, f: pkg.ssm_conv_fwd(h, f)),
    ("x", lambda pkg, h, f: pkg.ssm_conv_step(h, f, f)),
    ("x", lambda pkg, h, f: pkg.ssm_conv_bwd(h, f, h)),
    ("x", lambda pkg, h, f: pkg.ssm_scan_fwd(h, h, f, h, h)),
    ("x", lambda pkg, h, f: pkg.ssm_step(h, h, f, h, h, f)),
    ("x", lambda pkg, h, f: pkg.ssm_scan_bwd(h, h, f, h, h, h)),
])
def test_dtype_errors_name_their_tensor(name, call, monkeypatch):
    import torch
    import mlstm_matrix_memory_amd as pkg
    monkeypatch.setattr(b, "_gpu", lambda t, _: t.device)
    with pytest.raises(TypeError, match=f"^{name} must be float32 or bfloat16, got torch.float16"):
        call(pkg, torch.zeros(2, 3, 8, dtype=torch.float16), torch.ones(8))


def test_max_len_is_any_bound_of_the_lengths():
    """A caller may keep one bound for batches of any size: above the rows that there are it counts as these."""
    import torch
    x, start = torch.zeros(16, 8), torch.tensor([0, 5, 16], dtype=torch.int32)
    assert b._batch(x, start, 4096, x.device) == (2, 16, 16)
    assert b._batch(x, start, 11, x.device) == (2, 11, 16)
    with pytest.raises(ValueError, match="max_len"):
        b._batch(x, start, None, x.device)
