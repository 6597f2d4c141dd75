"""Values at the border of what the balance loss (mx_moe_balance,
mx_moe_balance_bwd) takes: what is not finite shows, and only where it belongs."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E", [1, 5, 8, 60, 128])
@pytest.mark.parametrize("T", [40, 700])                  # one part a sequence, and several
def test_infinite_logits_show(gpu_lib, T, E, dtype):
    """A logit of +inf makes its token's softmax NaN (inf - inf), so the loss and
    the means of its sequence and the token's gradient are, and no others."""
    gen = torch.Generator().manual_seed(T + E)
    k = min(2, E)
    z = torch.randn((T, E), generator=gen).to(dtype).cuda()
    idx = gpu_lib.mx_moe_route(z, k)[0]
    seg = torch.tensor([0, T // 4, T // 2, T - 3], dtype=torch.int32, device="cuda")
    dl, dm = torch.randn(3, generator=gen).cuda(), torch.randn((3, E), generator=gen).cuda()
    add = torch.randn((T, E), generator=gen).to(dtype).cuda()

    def run(logits, bias=None):
        loss, counts, mean = gpu_lib.mx_moe_balance(logits, idx, bias=bias, segments=seg)
        dz = gpu_lib.mx_moe_balance_bwd(logits, counts, k, dloss=dl, dmean_prob=dm, bias=bias, segments=seg, add=add)
        return loss, counts, mean, dz

    want = run(z)
    bad = z.clone()
    rows = [T // 4 + 1, T // 2 - 1]                        # both of the second sequence
    bad[rows[0], E // 2] = float("inf")
    bad[rows[1]] = float("inf")
    bad[T - 1, 0] = float("inf")                           # behind the last sequence: takes no part
    loss, counts, mean, dz = run(bad)
    assert torch.isnan(loss[1]) and torch.isnan(mean[1]).all() and torch.isnan(dz[rows]).all()
    assert torch.equal(counts, want[1])
    assert torch.equal(loss[[0, 2]], want[0][[0, 2]]) and torch.equal(mean[[0, 2]], want[2][[0, 2]])
    rest = np.setdiff1d(np.arange(T), rows)
    assert torch.equal(dz[rest], want[3][rest])
    # shut by its key (inf - inf is NaN): as if it were not there
    if E > 1:
        b = torch.zeros(E, device="cuda")
        b[0] = float("-inf")
        shut = z.clone()
        shut[:, 0] = float("inf")
        assert all(torch.equal(x, y) for x, y in zip(run(shut, b), run(z, b)))
