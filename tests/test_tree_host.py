"""The draft-tree and eviction operators without a GPU: refusals that come before
any CUDA call, the mask helper, and pins of the 64-bit reference that the GPU
tests compare with."""
import ctypes
import os
import re

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import kv_compression_b200 as kvc  # noqa: E402
import tree_reference as ref  # noqa: E402
from kv_compression_b200 import build as kbuild  # noqa: E402
from oracle import oracle as orc  # noqa: E402


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kvc.load_library()


def test_null_plan_refused_before_any_cuda_call(lib):
    one = ctypes.c_void_p(4096)
    assert lib.lca_tree_workspace(None, 1) == -1
    cache = (one, one, 1, 64, one, 1)
    assert lib.lca_tree_decode(None, one, one, 1, *cache, one, None, None, one, None, one, 1 << 30, None) == 1
    assert lib.lca_attn_mass(None, one, one, 1, *cache, one, None, None, one, None, 1.0, one, 64, one, 1 << 30,
                             None) == 1
    assert lib.lca_evict_select(None, one, 64, one, 0, 0, 1, one, one, None) == 1
    assert lib.lca_cache_compact(None, *cache, one, 1, one, None, None, 0, None) == 1


@pytest.mark.parametrize("T", [1, 2, 5, 63, 64])
def test_tree_mask_is_self_and_ancestors(T):
    rng = np.random.default_rng(T)
    parents = np.stack([np.array([rng.integers(-1, i) if i else -1 for i in range(T)]) for _ in range(3)]
                       + [np.arange(T) - 1, np.full(T, -1)])
    got = kvc.tree_mask(torch.from_numpy(parents)).numpy().view(np.uint64)
    assert np.array_equal(got, ref.words_of(parents))


def test_tree_mask_refuses_what_is_no_tree():
    for bad in ([[0]], [[-1, 1]], [[-2]], [[-1] * 65]):
        with pytest.raises(kvc.LcaError):
            kvc.tree_mask(torch.tensor(bad))


def _batch(B, T, H, d_c, d_r, lens, drafts, words, seed):
    r = np.random.default_rng(seed)
    c = [r.standard_normal((n + d, d_c)) for n, d in zip(lens, drafts)]
    k = [r.standard_normal((n + d, d_r)) for n, d in zip(lens, drafts)]
    s = 1.5 / np.sqrt(d_c + d_r)
    return ref.Tree(r.standard_normal((B, T, H, d_c)) * s, r.standard_normal((B, T, H, d_r)) * s, c, k, lens, drafts,
                    words)


def test_reference_of_one_node_is_dense_attention():
    t = _batch(2, 1, 3, 16, 8, [20, 20], [1, 1], ref.chain_words(2, 1), 1)
    out, lse, _, _ = t.attend(0, 0)
    want = orc.mla(t.q_c[:, 0].astype(np.float32), t.q_r[:, 0].astype(np.float32),
                   np.stack(t.c).astype(np.float32), np.stack(t.k).astype(np.float32))
    assert np.allclose(out[:, 0], want, rtol=0, atol=1e-5)


def test_reference_of_a_path_is_dense_attention_of_its_prefix():
    """In a tree each node attends as the last token of its own path would."""
    parents = np.array([[-1, 0, 0, 2, 1]])
    t = _batch(1, 5, 2, 16, 8, [7], [5], ref.words_of(parents), 2)
    out, lse, _, _ = t.attend(0, 0)
    path = [0, 2, 3]                                     # node 3
    rows = list(range(7)) + [7 + j for j in path]
    one = ref.Tree(t.q_c[:, 3:4], t.q_r[:, 3:4], [t.c[0][rows]], [t.k[0][rows]], [len(rows) - 1], [1],
                   ref.chain_words(1, 1))
    o, z, _, _ = one.attend(0, 0)
    assert np.allclose(o[0, 0], out[0, 3], rtol=1e-13) and np.allclose(z[0, 0], lse[0, 3], rtol=1e-13)


def test_reference_mass_of_a_row_is_one():
    t = _batch(2, 4, 3, 16, 8, [9, 0], [4, 3], ref.words_of(np.array([[-1, 0, 0, -1]] * 2)), 3)
    _, lse, _, _ = t.attend(0, 0)
    m = t.mass(lse, None, 1.0)
    assert np.allclose([x.sum() for x, _ in m], [4 * 3, 3 * 3])
    lse[0, 1] = np.inf                                   # a rejected node adds nothing
    assert np.allclose(t.mass(lse, None, 1.0)[0][0].sum(), 3 * 3)


def test_reference_select_by_hand():
    s = np.array([5, 1, 2, 2, np.nan, 2, -1, 0.0, -0.0, 9], dtype=np.float32)
    assert list(ref.select(s, 10, 1, 1, 4)) == [0, 2, 3, 9]
    assert list(ref.select(s, 10, 0, 0, 7)) == [0, 1, 2, 3, 5, 7, 9]
    assert list(ref.select(s, 10, 0, 0, 9)) == [0, 1, 2, 3, 5, 6, 7, 8, 9]
    assert list(ref.select(s, 3, 1, 1, 4)) == [0, 1, 2]
    assert list(ref.select(s, 10, 2, 2, 4)) == [0, 1, 8, 9]


def test_every_kernel_of_these_operators_checks_its_indexes():
    """The range-checked build is of use where a kernel has checks: by itself, or in the lookups of pool rows and
    sums that it calls."""
    csrc = os.path.join(os.path.dirname(kbuild.__file__), "csrc")
    found = []
    for name in ("tree_common.cuh", "tree_simt_kernel.cuh", "tree_tc_kernel.cuh", "mass_tc_kernel.cuh", "evict_kernel.cuh"):
        with open(os.path.join(csrc, name)) as f:
            text = f.read()
        for body in re.split(r"\b__global__\b", text)[1:]:
            found.append(re.search(r"(lca_\w+_kernel)\(", body).group(1))
            assert re.search(r"LCA_CHECK\(|tree_row\(|mass_store\(", body[:body.index("\n}\n")]), found[-1]
        for helper in ("tree_row", "mass_store"):
            if re.search(r"__forceinline__ \w+ " + helper + r"\(", text):
                assert "LCA_CHECK(" in text.split(" " + helper + "(", 1)[1].split("\n}\n")[0], helper
    assert len(found) == 10
