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
import tree_reference as ref  # noqa: E402
from kv_compression_b200 import build as kbuild  # noqa: E402
from test_tree_gpu import UP_BF16, Batch, check_mass, check_tree, ok  # noqa: E402

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


def _masked_by_keys(H, dtype, value, **kw):
    """A batch whose tokens named here have a key that makes their logits value / 2: the first 200 of a sequence (a
    whole tile), all that are cached, those in the middle and at the end; and the indexes of the others."""
    x = Batch(H, 3, [300, 130, 700, 140], page=64, seed=51, dtype=dtype, **kw)
    x.q_r[..., 0] = 0.5
    cut = [np.arange(200), np.arange(130), np.arange(390, 700), np.array([0, 128, 139])]
    rest = []
    for b, m in enumerate(cut):
        rows = torch.from_numpy(x.rows_of[b][m]).cuda()
        x.k[rows, 0] = value
        rest.append(np.setdiff1d(np.arange(x.lens[b] + 3), m))
    return x, cut, rest


def _without(x, rest):
    """The definition over the other tokens alone."""
    t = x.tree()
    for b, r in enumerate(rest):
        t.lens[b] = int((r < x.lens[b]).sum())
        t.c[b], t.k[b] = t.c[b][r], t.k[b][r]
    return t


def _check_masked(x, cut, rest, plan, tc):
    out, lse = x.decode(plan)
    ok(plan)
    t = _without(x, rest)
    want, wz, eo, ez = t.attend(UP_BF16 if tc else 0.0, UP_BF16 if x.dtype == "bf16" else 2.0 ** -24)
    got, gz = out.double().cpu().numpy(), lse.double().cpu().numpy()
    right = bool(np.all(np.abs(got - want) <= eo)), bool(np.all(np.abs(gz - wz) <= ez))
    assert right == (True, True)
    s = x.mass(plan, lse, None, 1.0).double().cpu().numpy()
    ok(plan)
    for b, (m, e) in enumerate(t.mass(gz, None, 1.0)):
        assert np.all(s[b, cut[b]] == 0)
        assert np.all(np.abs(s[b, rest[b]] - m) <= e)


KINDS = [(16, "bf16", False), (128, "bf16", False), (16, "bf16", True), (1, "bf16", True), (4, "f32", False), (1, "f32", False)]


@pytest.mark.parametrize("H,dtype,force", KINDS)
def test_tokens_with_logits_of_minus_infinity(H, dtype, force):
    kw = {} if dtype == "bf16" else dict(d_c=64, d_r=16)
    x, cut, rest = _masked_by_keys(H, dtype, float("-inf"), **kw)
    plan = x.plan()
    plan.set(kvc.OPT_FORCE_SIMT, int(force))
    _check_masked(x, cut, rest, plan, dtype == "bf16" and not force)
    for b in range(x.B):                                     # every row so: as if nothing were seen
        x.k[torch.from_numpy(x.rows_of[b]).cuda(), 0] = float("-inf")
    out, lse = x.decode(plan)
    ok(plan)
    assert bool((out == 0).all()) and bool((lse == float("-inf")).all())
    assert bool((x.mass(plan, lse, None, 1.0)[:, :133] == 0).all())


@pytest.mark.parametrize("value", [-3e38, -1e30, -1e20, -1e15, -1e10, -1e9, -1e6, -1e4])
@pytest.mark.parametrize("H,dtype,force", KINDS)
def test_tokens_masked_by_a_large_negative_logit(H, dtype, force, value):
    """Half of `value` lies so far below the other logits (a few units) that its weight is 0 in fp32."""
    kw = {} if dtype == "bf16" else dict(d_c=64, d_r=16)
    x, cut, rest = _masked_by_keys(H, dtype, value, **kw)
    plan = x.plan()
    plan.set(kvc.OPT_FORCE_SIMT, int(force))
    _check_masked(x, cut, rest, plan, dtype == "bf16" and not force)


@pytest.mark.parametrize("H", [16, 128])
def test_logits_that_the_tensor_cores_kernel_counts_as_minus_infinity(H):
    x, _, _ = _masked_by_keys(H, "bf16", 0.0)
    for b in range(x.B):
        x.k[torch.from_numpy(x.rows_of[b]).cuda(), 0] = -1e10
    plan = x.plan()
    out, lse = x.decode(plan)
    ok(plan)
    assert bool((out == 0).all()) and bool((lse == float("-inf")).all())


NOT_FINITE = [(which, v) for which in "ck" for v in (float("nan"), float("inf"), float("-inf"))]


@pytest.mark.parametrize("where", ["drafted", "cached"])
@pytest.mark.parametrize("lens", [[40] * 6, [126, 127, 300, 255, 128, 0]], ids=["one_tile", "tiles"])
@pytest.mark.parametrize("H,dtype,force", KINDS)
def test_rows_that_are_not_finite(H, dtype, force, lens, where):
    """Every head of every node that sees such a row, by the logit that it makes: NaN and +inf make all NaN, -inf is a
    weight of 0 and leaves NaN in the dims of C_KV that are not finite (a drafted row: may leave it everywhere)."""
    kw = {} if dtype == "bf16" else dict(d_c=64, d_r=16)
    lens = [max(n, 1) for n in lens] if where == "cached" else lens
    x = Batch(H, 4, lens, page=64, seed=52, dtype=dtype, **kw)
    x.set_words(ref.words_of(np.tile([-1, -1, 1, 0], (6, 1))))           # nodes 1 and 2 see node 1
    at = [n + 1 if where == "drafted" else n // 2 for n in lens]
    for b, (which, v) in enumerate(NOT_FINITE):
        (x.c if which == "c" else x.k)[int(x.rows_of[b][at[b]]), 5] = v
    feel = (1, 2) if where == "drafted" else (0, 1, 2, 3)
    plan = x.plan()
    plan.set(kvc.OPT_FORCE_SIMT, int(force))
    out, lse = x.decode(plan)
    ok(plan)
    tc = dtype == "bf16" and not force
    t = _without(x, [np.setdiff1d(np.arange(n + 4), a) if where == "cached" else np.arange(n + 4) for n, a in zip(lens, at)])
    if where == "drafted":                                   # the definition without node 1's row
        for b in range(6):
            t.c[b][at[b]] = t.k[b][at[b]] = 0.0
        t.words = t.words & ~np.uint64(2)
    want, wz, eo, ez = t.attend(UP_BF16 if tc else 0.0, UP_BF16 if dtype == "bf16" else 2.0 ** -24)
    got, gz = out.double().cpu().numpy(), lse.double().cpu().numpy()
    q = {"c": x.q_c[..., 5].double().cpu().numpy(), "k": x.q_r[..., 5].double().cpu().numpy()}
    kinds = set()
    for b, (which, v) in enumerate(NOT_FINITE):
        for i in range(4):
            for h in range(H):
                o, z = got[b, i, h], gz[b, i, h]
                near = np.abs(o - want[b, i, h]) <= eo[b, i, h] + 1e-30
                same = z == wz[b, i, h] or abs(z - wz[b, i, h]) <= ez[b, i, h]
                logit = v * q[which][b, i, h]
                if i not in feel:
                    kinds.add("other")
                    assert near.all() and same, (b, i, h)
                elif not logit < 0:
                    kinds.add("all")
                    assert np.isnan(o).all() and np.isnan(z), (b, i, h)
                elif which == "k":
                    kinds.add("key")
                    assert near.all() and same, (b, i, h)
                else:
                    kinds.add("dim")
                    may = where == "drafted"
                    assert np.isnan(o[5]) and (near | (np.arange(x.d_c) == 5) | (may & np.isnan(o))).all(), (b, i, h)
                    assert same or (may and np.isnan(z)), (b, i, h)
    assert {"all", "key", "dim"} <= kinds


@pytest.mark.parametrize("H", [16, 128])
def test_truncation_is_made_up_for_on_average(H):
    """Full rows of random products: the tensor core's truncation, 4e-7 to 6e-7 of a logit, less the factor's 3.6e-7.  The
    bound of 2^-22 = 2.4e-7 of the logits at work (the weights' mean of them; 2^-21 beside it for the exponential, the
    sums and the logarithm) holds neither without the factor nor with a wrong one.  The mean over the rows is compared:
    the rest of a row's error is as often up as down."""
    x = Batch(H, 1, [1000, 777, 1023, 900, 640, 810, 1001, 512], seed=53, scale=8.0)
    plan = x.plan()
    out, lse = x.decode(plan)
    ok(plan)
    t = x.tree()
    at_work, want = np.zeros((x.B, H)), np.zeros((x.B, H))
    for b in range(x.B):
        logits, _, _ = t.logits(b, 0)
        m = logits.max(1, keepdims=True)
        e = np.exp(logits - m)
        want[b] = m[:, 0] + np.log(e.sum(1))
        at_work[b] = (e * logits).sum(1) / e.sum(1)
    assert at_work.mean() > 15
    bound = 2.0 ** -22 * at_work.mean() + 2.0 ** -21
    assert abs((lse[:, 0].double().cpu().numpy() - want).mean()) <= bound
    z = torch.from_numpy(want).float().cuda()[:, None].contiguous()      # (rounded to nearest: as often up as down)
    s = x.mass(plan, z, None, 1.0).double().cpu().numpy()
    total = sum(s[b, :n + 1].sum() for b, n in enumerate(x.lens))
    assert abs(total / (x.B * H) - 1) <= bound


@pytest.mark.parametrize("H", [16, 128])
def test_logits_formed_exactly(H):
    """One product a logit, of whole numbers: nothing is cut off, and lse is off by the factor's 3 2^-23 and at most six
    roundings (the factor's constant, the product, M, ln 2, the sum, the last product), the weight by those in its
    exponent."""
    x = Batch(H, 1, [0] * 12, seed=54)
    x.q_c.zero_()
    x.q_r.zero_()
    x.k.zero_()
    value = torch.tensor([1, 2, 3, 5, 10, 20, 31, 60, -1, -7, -33, -60], dtype=torch.float32)
    x.q_r[..., 7] = 1.0
    for b in range(12):
        x.k[int(x.rows_of[b][0]), 7] = float(value[b])
    plan = x.plan()
    out, lse = x.decode(plan)
    ok(plan)
    want = value.double()[:, None].expand(12, H)
    most = (3 * 2.0 ** -23 + 6 * 2.0 ** -24) * want.abs()
    assert bool(((lse[:, 0].double().cpu() - want).abs() <= most).all())
    for b in range(12):
        assert bool((out[b] == x.c[int(x.rows_of[b][0])]).all())         # a weight of 1
    s = x.mass(plan, want.float().cuda()[:, None].contiguous(), None, 1.0)[:, 0].double().cpu()
    # H weights of 1 and what the exponent's error makes of them; 2^-20 for the exponential and the sum
    assert bool(((s - H).abs() <= H * (most[:, 0] * 1.001 + 2.0 ** -20)).all())


@pytest.fixture(scope="module")
def checked():
    return kbuild.build_checked()


@pytest.mark.parametrize("H,T,lens,dtype,kw,opts", [
    (16, 4, [700, 0, 300], "bf16", {}, {kvc.OPT_NUM_CTAS: 3}),                                  # several units a CTA
    (16, 2, [100 + 3 * b for b in range(50)], "bf16", {}, {}),
    (128, 9, [4000, 130], "bf16", {}, {}),
    (128, 9, [400, 130, 77], "bf16", {}, {kvc.OPT_NUM_CTAS: 5}),
    (16, 16, [9000], "bf16", {}, {}),
    (16, 5, [900, 65], "bf16", {}, {kvc.OPT_FORCE_SIMT: 1}),
    (3, 1, [900, 65], "bf16", {}, {kvc.OPT_FORCE_SIMT: 1}),
    (2, 30, [900, 65], "f32", dict(d_c=64, d_r=16), {}),
    (6, 12, [2000, 1], "bf16", dict(d_c=256, d_r=32), {}),
])
def test_checked_build_of_trees_and_weights(checked, H, T, lens, dtype, kw, opts):
    """No check fires, and the same bits come out as from the ordinary build."""
    x = Batch(H, T, lens, page=64, dtype=dtype, seed=55, **kw)
    got = []
    for lib in (None, checked):
        plan = x.plan(lib_path=lib)
        for k, v in opts.items():
            plan.set(k, v)
        out, lse = x.decode(plan)
        s = x.mass(plan, lse, torch.ones(x.B, x.cap, device="cuda"), 0.5)
        ok(plan)
        got.append((out, lse, s))
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("lens,budget", [([3000, 64, 65, 0, 2049], 64), ([131072, 40000], 16384), ([50000], 49999), ([500000], 70)])
def test_checked_build_of_choice_and_compaction(checked, lens, budget):
    x = Batch(1, 1, lens, page=64, seed=56, d_c=64, d_r=8)
    s0 = torch.rand(x.B, x.cap, device="cuda")
    n_src, got = torch.tensor(lens, dtype=torch.int32, device="cuda"), []
    for lib in (None, checked):
        plan = x.plan(lib_path=lib)
        c, k, s, kl = x.c.clone(), x.k.clone(), s0.clone(), n_src.clone()
        kept = torch.full((x.B, budget), -7, dtype=torch.int32, device="cuda")
        plan.evict_select(s, kl, 4, 8, kept, kl)
        plan.cache_compact(c, k, x.page, x.dtable, kept, kl, scores=s)
        ok(plan)
        got.append((kept, kl, c.view(torch.int16), k.view(torch.int16), s))
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_mask_words_from_parents_on_either_side():
    """Made from parents on the CPU the words need no wait; a graph of the other calls takes them as they then are."""
    x = Batch(16, 5, [200, 60], page=64, seed=57)
    parents = [torch.tensor([[-1, 0, 0, 1, 3], [-1, -1, 1, 1, 0]]), torch.tensor([[-1, 0, 1, 2, 3], [-1, 0, 0, 2, -1]])]
    plan, ws = x.plan(), x.plan().tree_workspace(5)
    x.mask = kvc.tree_mask(parents[0]).cuda()
    assert torch.equal(x.mask, kvc.tree_mask(parents[0].cuda()))
    out, z = torch.zeros_like(x.q_c), torch.zeros(2, 5, 16, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan.tree_decode(x.q_c, x.q_r, x.c, x.k, x.page, x.dtable, x.dlens, out, z, mask=x.mask, workspace=ws)
    for p in parents:
        x.mask.copy_(kvc.tree_mask(p))
        g.replay()
        torch.cuda.synchronize()
        want, wz = x.decode(plan)
        assert torch.equal(out, want) and torch.equal(z, wz)
    ok(plan)


@pytest.mark.parametrize("H,dtype,page", [(16, "bf16", 64), (128, "bf16", 0), (4, "f32", 64)])
def test_a_whole_step_captured(H, dtype, page):
    """Copies, another stream's work, attention, weights, commit, choice and compaction in one graph, behind one
    another; replayed with other contents it does what the calls do one by one."""
    T, kw = 4, {} if dtype == "bf16" else dict(d_c=64, d_r=16)
    x = Batch(H, T, [300, 5000, 129], page=page, seed=58, dtype=dtype, extra=20, **kw)
    x.c.nan_to_num_(0.0)
    x.k.nan_to_num_(0.0)
    plan, budget = x.plan(), 128
    host = [x.q_c.cpu().pin_memory(), (x.q_c * -0.5).cpu().pin_memory()]
    src = torch.stack([torch.tensor([n + 1, n + 3]) for n in x.lens]).int().cuda()
    two = torch.full((3,), 2, dtype=torch.int32, device="cuda")

    class State:
        def __init__(self):
            self.c, self.k, self.q = x.c.clone(), x.k.clone(), torch.zeros_like(x.q_c)
            self.lens, self.scores = x.dlens.clone(), torch.rand(3, x.cap, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
            self.out, self.lse = torch.zeros_like(x.q_c), torch.zeros(3, T, H, device="cuda")
            self.kept = torch.zeros(3, budget, dtype=torch.int32, device="cuda")
            self.ws = plan.tree_workspace(T)
            self.side = torch.cuda.Stream()

        def reset(self):
            for a, b in ((self.c, x.c), (self.k, x.k), (self.lens, x.dlens)):
                a.copy_(b)
            self.scores.copy_(State().scores)

        def step(self, q):
            here = torch.cuda.current_stream()
            self.side.wait_stream(here)
            with torch.cuda.stream(self.side):               # something else that the attention waits for
                self.scores.mul_(0.5)
            self.q.copy_(q, non_blocking=True)
            here.wait_stream(self.side)
            plan.tree_decode(self.q, x.q_r, self.c, self.k, x.page, x.dtable, self.lens, self.out, self.lse, mask=x.mask, workspace=self.ws)
            self.side.wait_stream(here)
            with torch.cuda.stream(self.side):
                self.scores.add_(0.25)
            here.wait_stream(self.side)
            plan.attn_mass(self.q, x.q_r, self.c, self.k, x.page, x.dtable, self.lens, self.lse, self.scores, prev=self.scores,
                           decay=0.75, mask=x.mask, workspace=self.ws)
            plan.cache_compact(self.c, self.k, x.page, x.dtable, src, two, dst0=self.lens, scores=self.scores)
            self.lens.add_(2)
            plan.evict_select(self.scores, self.lens, 4, 16, self.kept, self.lens)
            plan.cache_compact(self.c, self.k, x.page, x.dtable, self.kept, self.lens, scores=self.scores)

        def all(self):
            torch.cuda.synchronize()
            ok(plan)
            bits = torch.int16 if x.dt == torch.bfloat16 else torch.int32
            return [t.clone() for t in (self.out, self.lse, self.scores, self.kept, self.lens, self.c.view(bits), self.k.view(bits))]

    a, b = State(), State()
    want = []
    for q in host:
        a.reset()
        a.step(q)
        want.append(a.all())
    pinned = host[0].clone().pin_memory()
    g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        b.step(pinned)
    for q, w in ((host[0], want[0]), (host[1], want[1]), (host[0], want[0])):
        torch.cuda.synchronize()
        pinned.copy_(q)
        b.reset()
        g.replay()
        for got, expected in zip(b.all(), w):
            assert torch.equal(got, expected)


@pytest.mark.parametrize("force", [False, True], ids=["auto", "simt"])
@pytest.mark.parametrize("B,H,T", [(65535, 1, 1), (2, 4096, 3), (1, 4096, 64)])
def test_the_largest_batches_and_head_counts(B, H, T, force):
    """As many sequences, and as many heads, as the calls take: a few tokens each, against plain torch in 64 bits.
    Bounds as in tree_reference.py, with the batch's largest sum |q k|; the logits stay below 20."""
    g = torch.Generator(device="cuda").manual_seed(B + T)
    cap = T + 3
    r = torch.Generator().manual_seed(B + T)
    lens = torch.randint(0, 4, (B,), generator=r).int().cuda()
    c = torch.randn(B * cap, 512, generator=g, device="cuda").clamp(-6, 6).bfloat16()
    k = torch.randn(B * cap, 64, generator=g, device="cuda").bfloat16()
    q_c = (torch.randn(B, T, H, 512, generator=g, device="cuda") * 0.08).bfloat16()
    q_r = (torch.randn(B, T, H, 64, generator=g, device="cuda") * 0.08).bfloat16()
    plan = kvc.Plan(B, H, 512, 64, "bf16", cap)
    plan.set(kvc.OPT_FORCE_SIMT, int(force))
    out, lse = torch.zeros_like(q_c), torch.zeros(B, T, H, device="cuda")
    s = torch.full((B, cap), -77.0, device="cuda")
    plan.tree_decode(q_c, q_r, c, k, cap, None, lens, out, lse)
    plan.attn_mass(q_c, q_r, c, k, cap, None, lens, lse, s)
    ok(plan)
    pos, node = torch.arange(cap, device="cuda"), torch.arange(T, device="cuda")
    for b0 in range(0, B, 8192):
        b1 = min(B, b0 + 8192)
        C, K = c.view(B, cap, 512)[b0:b1].double(), k.view(B, cap, 64)[b0:b1].double()
        n = lens[b0:b1, None, None].long()
        sees = pos[None, None, :] <= n + node[None, :, None]               # a chain, [b, T, cap]
        mass = torch.zeros(b1 - b0, cap, dtype=torch.float64, device="cuda")
        for i in range(T):
            x = q_c[b0:b1, i].double() @ C.transpose(1, 2) + q_r[b0:b1, i].double() @ K.transpose(1, 2)
            x = x.masked_fill(~sees[:, i, None, :], -float("inf"))
            z = torch.logsumexp(x, 2)
            p = torch.exp(x - z[..., None])
            want = p @ C
            ex = 576 * 2.0 ** -23 * float((q_c[b0:b1, i].double().abs() @ C.abs().transpose(1, 2)
                                           + q_r[b0:b1, i].double().abs() @ K.abs().transpose(1, 2)).max())
            assert float((lse[b0:b1, i] - z).abs().max()) <= ex + 2.0 ** -20 * 21
            most = (2 * ex + 2.0 ** -18 + 2.0 ** -8) * (p @ C.abs()) + 2.0 ** -8 * want.abs()
            assert bool(((out[b0:b1, i].double() - want).abs() <= most).all())
            mass += torch.exp(x - lse[b0:b1, i].double()[..., None]).sum(1)
        valid = pos[None, :] < lens[b0:b1, None] + T
        err = (s[b0:b1].double() - mass).abs()
        assert bool((err[valid] <= (ex + 2.0 ** -18 + (T * H + 32) * 2.0 ** -23) * mass[valid] + 1e-30).all())
        assert bool((s[b0:b1][~valid] == -77.0).all())


@pytest.mark.parametrize("H,dtype", [(16, "bf16"), (4, "f32")])
def test_sequences_that_share_their_first_pages(H, dtype):
    """A common prompt: two pages listed by all three sequences.  Attention and weights read them; an eviction that
    keeps them where they are may move the rows behind."""
    kw = {} if dtype == "bf16" else dict(d_c=64, d_r=16)
    x = Batch(H, 3, [300, 200, 450], page=64, seed=59, dtype=dtype, **kw)
    x.table[1:, :2] = x.table[0, :2]
    x.dtable.copy_(torch.from_numpy(x.table))
    x.rows_of = [x.rows(b, np.arange(n + 3)) for b, n in enumerate(x.lens)]
    plan = x.plan()
    out, lse = x.decode(plan)
    check_tree(x, out, lse, tc=dtype == "bf16")
    s = x.mass(plan, lse, None, 1.0)
    check_mass(x, s, lse, None, 1.0)
    kept, kl = torch.zeros(3, 160, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    plan.evict_select(s, x.dlens, 128, 8, kept, kl)
    before = [x.c[torch.from_numpy(x.rows_of[b]).cuda()].clone() for b in range(3)]
    plan.cache_compact(x.c, x.k, 64, x.dtable, kept, kl, scores=s)
    ok(plan)
    for b in range(3):
        now = x.c[torch.from_numpy(x.rows_of[b][:160]).cuda()]
        assert torch.equal(now, before[b][kept[b].long()])


@pytest.mark.parametrize("H,dtype,force", KINDS)
def test_what_belongs_to_no_drafted_token_is_not_felt(H, dtype, force):
    """Queries, mask words and lse of nodes past a sequence's own, and old sums past its cached tokens, may hold anything."""
    kw = {} if dtype == "bf16" else dict(d_c=64, d_r=16)
    drafts = [3, 7, 0, 1, 8]
    x = Batch(H, 8, [300, 127, 64, 0, 513], drafts, page=64, seed=60, dtype=dtype, **kw)
    plan = x.plan()
    plan.set(kvc.OPT_FORCE_SIMT, int(force))
    prev = torch.rand(5, x.cap, device="cuda")
    out, lse = x.decode(plan)
    s = x.mass(plan, lse, prev, 0.5)
    for b, d in enumerate(drafts):
        x.q_c[b, d:], x.q_r[b, d:] = float("nan"), float("inf")
        x.mask[b, d:] = -1
        lse[b, d:] = float("nan")
        prev[b, x.lens[b]:] = float("nan")
    again, z = x.decode(plan)
    assert torch.equal(again, out)
    assert all(torch.equal(z[b, :d], lse[b, :d]) for b, d in enumerate(drafts))
    assert torch.equal(x.mass(plan, lse, prev, 0.5), s)
    ok(plan)
