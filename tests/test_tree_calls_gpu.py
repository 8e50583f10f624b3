"""Calls of the draft-tree and eviction operators that their documentation allows
and that test_tree_gpu.py does not make: one workspace for trees of every size,
arguments that are the same tensor, values at the ends of the types' ranges, every
kernel in the range-checked build."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import kv_compression_b200 as kvc  # noqa: E402
from test_tree_gpu import Batch, ok  # noqa: E402

pytestmark = pytest.mark.gpu


# B, H, dtype, d_c, d_r: the CUDA-core kernel's wish falls with T in the first four (to nothing in the second)
@pytest.mark.parametrize("B,H,dtype,d_c,d_r", [(8, 4, "bf16", 256, 32), (64, 16, "bf16", 256, 32), (8, 6, "bf16", 256, 32),
                                               (32, 16, "f32", 128, 32), (3, 16, "bf16", 512, 64), (40, 128, "bf16", 512, 64)])
def test_one_workspace_serves_every_smaller_tree(B, H, dtype, d_c, d_r):
    plan = kvc.Plan(B, H, d_c, d_r, dtype, 4096)
    sizes = [plan.tree_workspace(T).numel() for T in range(1, 65)]
    assert sizes == sorted(sizes)
    ws = plan.tree_workspace(64)
    for T in (1, 2, 7, 16, 33):
        x = Batch(H, T, [90 + 7 * b for b in range(B)], page=64, dtype=dtype, d_c=d_c, d_r=d_r, seed=T)
        out, lse = x.decode(plan, ws=ws)
        mass = x.mass(plan, lse, None, 1.0, ws=ws)
        ok(plan)
        want, z = x.decode(plan)
        assert torch.equal(out, want) and torch.equal(lse, z)
        assert torch.equal(mass, x.mass(plan, lse, None, 1.0))
    with pytest.raises(kvc.LcaError) as e:                   # still a refusal where it is too small
        x.decode(plan, ws=ws[:256])
    assert e.value.status == kvc.LCA_ERR_INVALID_ARG


@pytest.mark.parametrize("lens,budget", [([5000, 300, 131072, 0, 40000, 512, 513, 9000], 512), ([900, 65, 64, 3], 64),
                                         ([70000, -1, 99999999, 65000], 60000)])
def test_kept_lens_in_place(lens, budget):
    """The lengths become those that are kept in the tensor they come from; the same rows are kept."""
    B, stride = len(lens), max(n for n in lens if n < 10 ** 7)
    s = torch.rand(B, stride, generator=torch.Generator(device="cuda").manual_seed(budget), device="cuda")
    plan = kvc.Plan(B, 1, 64, 16, "f32", stride)
    want, kept = (torch.full((B, budget), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    lengths, kl = torch.tensor(lens, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    bad = any(n < 0 or n > stride for n in lens)
    plan.evict_select(s, lengths, 3, 16, want, kl)
    assert plan.device_error() == (kvc.LCA_ERR_DEVICE_INPUT if bad else kvc.LCA_OK)
    assert kl.tolist() == [min(n, budget) if 0 <= n <= stride else 0 for n in lens]
    for _ in range(20):
        n = lengths.clone()
        kept.fill_(-7)
        plan.evict_select(s, n, 3, 16, kept, n)
        assert plan.device_error() == (kvc.LCA_ERR_DEVICE_INPUT if bad else kvc.LCA_OK)
        assert torch.equal(n, kl) and torch.equal(kept, want)
