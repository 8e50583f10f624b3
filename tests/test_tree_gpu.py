"""The draft-tree attention, the accumulated attention weights, the choice of an
eviction and the compaction on the GPU, each against its definition in 64 bits
(tree_reference.py, with bounds derived there), and a run of them together."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import kv_compression_b200 as kvc  # noqa: E402
import tree_reference as ref  # noqa: E402
from gpu_helpers import Guarded  # noqa: E402
from kv_compression_b200 import build as kbuild  # noqa: E402

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
UP_BF16 = 2.0 ** -8


class Batch:
    """Seeded inputs on the device.  Rows of no token are NaN; table entries past a sequence's pages are -1."""

    def __init__(self, H, T, lens, drafts=None, page=0, parents="random", dtype="bf16", d_c=512, d_r=64, seed=0,
                 scale=2.5, extra=0, null_mask=False, null_drafts=False):
        self.H, self.T, self.B = H, T, len(lens)
        self.lens, self.drafts = list(lens), list(drafts) if drafts is not None else [T] * len(lens)
        self.d_c, self.d_r, self.dtype = d_c, d_r, dtype
        B, dt = self.B, BF16 if dtype == "bf16" else F32
        self.dt = dt
        r = np.random.default_rng(seed)
        self.rng = r
        used = [n + d for n, d in zip(self.lens, self.drafts)]
        self.cap = max(max(used), 1) + extra
        if page:
            per = -(-self.cap // page)
            need = [-(-u // page) for u in used]
            order = r.permutation(sum(need) + 3).astype(np.int32)
            table, at = np.full((B, per), -1, np.int32), 0
            for b, k in enumerate(need):
                table[b, :k] = order[at:at + k]
                at += k
            self.table, self.page, rows = table, page, len(order) * page
        else:
            self.table, self.page, rows = None, self.cap, B * self.cap
        self.rows_of = [self.rows(b, np.arange(used[b])) for b in range(B)]
        c, k = np.full((rows, d_c), np.nan, np.float32), np.full((rows, d_r), np.nan, np.float32)
        for b in range(B):
            c[self.rows_of[b]] = r.standard_normal((used[b], d_c), dtype=np.float32)
            k[self.rows_of[b]] = r.standard_normal((used[b], d_r), dtype=np.float32)
        s = scale / np.sqrt(d_c + d_r)
        self.c, self.k = torch.from_numpy(c).to(dt).cuda(), torch.from_numpy(k).to(dt).cuda()
        self.q_c = torch.from_numpy(r.standard_normal((B, T, H, d_c), dtype=np.float32) * np.float32(s)).to(dt).cuda()
        self.q_r = torch.from_numpy(r.standard_normal((B, T, H, d_r), dtype=np.float32) * np.float32(s)).to(dt).cuda()
        if isinstance(parents, str) and parents == "random":
            parents = np.stack([[r.integers(-1, i) if i else -1 for i in range(T)] for _ in range(B)])
        self.words = ref.chain_words(B, T) if null_mask else ref.words_of(np.asarray(parents)) if parents is not None else None
        self.mask = None if null_mask else torch.from_numpy(self.words.view(np.int64)).cuda() if self.words is not None else None
        self.dtable = None if self.table is None else torch.from_numpy(self.table).cuda()
        self.dlens = torch.tensor(self.lens, dtype=torch.int32).cuda()
        self.ddrafts = None if null_drafts else torch.tensor(self.drafts, dtype=torch.int32).cuda()

    def set_words(self, words):
        self.words = words
        self.mask = torch.from_numpy(words.view(np.int64)).cuda()

    def rows(self, b, pos):
        pos = np.asarray(pos)
        if self.table is None:
            return b * self.page + pos
        return self.table[b, pos // self.page].astype(np.int64) * self.page + pos % self.page

    def tree(self):
        c, k = self.c.double().cpu().numpy(), self.k.double().cpu().numpy()
        return ref.Tree(self.q_c.double().cpu().numpy(), self.q_r.double().cpu().numpy(),
                        [c[x] for x in self.rows_of], [k[x] for x in self.rows_of], self.lens, self.drafts, self.words)

    def plan(self, **kw):
        return kvc.Plan(self.B, self.H, self.d_c, self.d_r, self.dtype, self.cap, **kw)

    def decode(self, plan, lse=True, ws=None, stream=None):
        fill = -77.0
        out = Guarded((self.B, self.T, self.H, self.d_c), self.dt, fill, -3.0)
        z = Guarded((self.B, self.T, self.H), F32, fill, -3.0) if lse else None
        plan.tree_decode(self.q_c, self.q_r, self.c, self.k, self.page, self.dtable, self.dlens, out.t,
                         z.t if lse else None, mask=self.mask, draft_lens=self.ddrafts, workspace=ws, stream=stream)
        torch.cuda.synchronize()
        out.check()
        if lse:
            z.check()
        return out.t, z.t if lse else None

    def mass(self, plan, lse, prev, decay, stride=None, ws=None):
        stride = stride or self.cap
        s = Guarded((self.B, stride), F32, -77.0, -3.0)
        plan.attn_mass(self.q_c, self.q_r, self.c, self.k, self.page, self.dtable, self.dlens, lse, s.t, prev=prev,
                       decay=decay, mask=self.mask, draft_lens=self.ddrafts, workspace=ws)
        torch.cuda.synchronize()
        s.check()
        return s.t


def ok(plan):
    st = plan.device_error()
    assert st == kvc.LCA_OK, f"device error {st} at site {plan.device_error_site():#x}"


def check_tree(x: Batch, out, lse, tc: bool):
    """Every written element within its bound; rows of nodes past a sequence's own untouched."""
    up = UP_BF16 if tc else 0.0
    uo = UP_BF16 if x.dtype == "bf16" else 2.0 ** -24
    want, wz, eo, ez = x.tree().attend(up, uo)
    got, gz = out.double().cpu().numpy(), lse.double().cpu().numpy() if lse is not None else None
    for b in range(x.B):
        d = x.drafts[b]
        assert np.all(got[b, d:] == -77.0), "rows past the drafted tokens were written"
        err = np.abs(got[b, :d] - want[b, :d])
        assert (err / (eo[b, :d] + 1e-30)).max(initial=0) <= 1, b
        if gz is not None:
            assert np.all(gz[b, d:] == -77.0)
            fine = np.isfinite(wz[b, :d])
            assert np.array_equal(gz[b, :d][~fine], wz[b, :d][~fine])
            assert np.all(np.abs(gz[b, :d] - wz[b, :d])[fine] <= ez[b, :d][fine])


def check_mass(x: Batch, scores, lse, prev, decay):
    got = scores.double().cpu().numpy()
    res = x.tree().mass(lse.double().cpu().numpy(), None if prev is None else prev.double().cpu().numpy(), decay)
    for b, (s, e) in enumerate(res):
        m = len(s)
        assert np.all(got[b, m:] == -77.0), "positions past the sequence were written"
        err = np.abs(got[b, :m] - s)
        assert (err / (e + 1e-30)).max(initial=0) <= 1, b


# (H, T, lens, drafts, page, dtype, d_c, d_r)
SMALL = [
    (16, 1, [1], [1], 0, "bf16", 512, 64),
    (16, 1, [0, 127, 128, 300], None, 0, "bf16", 512, 64),
    (16, 4, [130, 0, 63, 1000, 252], [4, 3, 0, 1, 4], 64, "bf16", 512, 64),
    (8, 7, [500, 77], None, 192, "bf16", 512, 64),
    (24, 5, [129, 640], [5, 2], 128, "bf16", 512, 64),
    (5, 3, [200, 3], None, 64, "bf16", 512, 64),
    (128, 2, [700, 65], None, 64, "bf16", 512, 64),
    (128, 9, [300], [8], 0, "bf16", 512, 64),
    (16, 64, [100, 5], [64, 33], 64, "bf16", 512, 64),
    (1, 1, [2000], None, 64, "bf16", 512, 64),
    (4, 7, [1001, 313, 0], [7, 6, 5], 0, "f32", 64, 16),
    (3, 2, [40, 333], None, 64, "f32", 64, 16),
    (2, 33, [90], None, 0, "f32", 512, 64),
    (6, 4, [100, 511], None, 128, "bf16", 128, 32),
    (1, 3, [50], None, 0, "bf16", 1024, 256),
    (2, 5, [77, 1], None, 0, "f32", 8, 8),
    (6, 12, [300, 0, 65], [12, 7, 1], 64, "bf16", 256, 32),
    (16, 4, [129, 64], None, 0, "f32", 40, 24),
    (4, 5, [70], None, 0, "f32", 512, 128),
    (10, 1, [33, 200], None, 64, "bf16", 640, 64),
    (3, 11, [90], None, 0, "f32", 1024, 256),
]
IDS = ["H{}_T{}_n{}_d{}_p{}_{}_{}_{}".format(a, b, "-".join(map(str, c)), "" if d is None else "-".join(map(str, d)), e, f, g, h)
       for a, b, c, d, e, f, g, h in SMALL]


def small(case, seed=0, **kw):
    H, T, lens, drafts, page, dtype, d_c, d_r = case
    return Batch(H, T, lens, drafts, page, dtype=dtype, d_c=d_c, d_r=d_r, seed=seed, **kw)


def is_tc(x, plan_opts=()):
    return x.dtype == "bf16" and x.d_c == 512 and x.d_r == 64 and kvc.OPT_FORCE_SIMT not in plan_opts


@pytest.mark.parametrize("force", [False, True], ids=["auto", "simt"])
@pytest.mark.parametrize("case", SMALL, ids=IDS)
def test_tree_decode_matches_definition(case, force):
    x = small(case, seed=len(case[2]) + case[0])
    plan = x.plan()
    if force:
        plan.set(kvc.OPT_FORCE_SIMT, 1)
    out, lse = x.decode(plan)
    ok(plan)
    check_tree(x, out, lse, tc=is_tc(x) and not force)
    again, z = x.decode(plan, lse=False)                    # the same bits again, without lse
    assert torch.equal(again, out)


@pytest.mark.parametrize("force", [False, True], ids=["auto", "simt"])
@pytest.mark.parametrize("case", SMALL, ids=IDS)
def test_attn_mass_matches_definition(case, force):
    x = small(case, seed=len(case[2]) + case[0], extra=3)
    plan = x.plan()
    if force:
        plan.set(kvc.OPT_FORCE_SIMT, 1)
    _, lse = x.decode(plan)
    prev = torch.rand(x.B, x.cap, device="cuda") * x.H
    got = x.mass(plan, lse, prev, 0.75)
    ok(plan)
    check_mass(x, got, lse, prev, 0.75)
    lse2 = lse.clone()
    lse2[:, 0] = float("inf")                               # the first node was rejected
    a = x.mass(plan, lse2, None, 1.0)
    check_mass(x, a, lse2, None, 1.0)
    assert torch.equal(a, x.mass(plan, lse2, None, 1.0))
    nan = torch.full_like(prev, float("nan"))               # prev is not read where decay is 0
    assert torch.equal(a, x.mass(plan, lse2, nan, 0.0))


def test_mass_in_place():
    x = Batch(16, 3, [300, 150], page=64, seed=4, extra=10)
    plan = x.plan()
    _, lse = x.decode(plan)
    prev = torch.rand(x.B, x.cap, device="cuda")
    want = x.mass(plan, lse, prev, 0.5)
    s = prev.clone()
    plan.attn_mass(x.q_c, x.q_r, x.c, x.k, x.page, x.dtable, x.dlens, lse, s, prev=s, decay=0.5, mask=x.mask,
                   draft_lens=x.ddrafts)
    for b in range(x.B):
        m = x.lens[b] + x.drafts[b]
        assert torch.equal(s[b, :m], want[b, :m]) and torch.equal(s[b, m:], prev[b, m:])


@pytest.mark.parametrize("dtype,H", [("bf16", 16), ("bf16", 128), ("f32", 4)])
def test_chain_and_all_drafts_are_the_defaults(dtype, H):
    kw = dict(dtype=dtype, **(dict(d_c=64, d_r=16) if dtype == "f32" else {}))
    a = Batch(H, 6, [200, 50], seed=3, parents=np.tile(np.arange(6) - 1, (2, 1)), **kw)
    b = Batch(H, 6, [200, 50], seed=3, null_mask=True, null_drafts=True, **kw)
    pa, pb = a.plan(), b.plan()
    oa, za = a.decode(pa)
    ob, zb = b.decode(pb)
    assert torch.equal(oa, ob) and torch.equal(za, zb)
    check_tree(b, ob, zb, tc=dtype == "bf16")


@pytest.mark.parametrize("force", [False, True], ids=["auto", "simt"])
@pytest.mark.parametrize("dtype,H", [("bf16", 16), ("bf16", 128), ("f32", 4)])
def test_rows_that_see_nothing_and_masked_garbage(dtype, H, force):
    """Nodes with empty words over an empty cache give 0 and -inf; rows that hold infinities or NaN are felt by the
    nodes that see them alone."""
    kw = dict(dtype=dtype, **(dict(d_c=64, d_r=16) if dtype == "f32" else {}))
    for lens in ([0, 0, 70], [126, 127, 300]):
        x = Batch(H, 5, lens, seed=5, **kw)
        words = ref.words_of(np.tile([-1, -1, 0, 1, -1], (3, 1)))
        words[:, 4] = 0                                      # node 4 sees no drafted token
        x.set_words(words)
        bad = {0: (float("nan"), "c"), 1: (float("inf"), "c"), 2: (float("-inf"), "k")}
        for b, (v, which) in bad.items():                    # node 1's row is broken: nodes 1 and 3 see it
            (x.c if which == "c" else x.k)[int(x.rows_of[b][lens[b] + 1]), 3] = v
        plan = x.plan()
        if force:
            plan.set(kvc.OPT_FORCE_SIMT, 1)
        out, lse = x.decode(plan)
        ok(plan)
        t = x.tree()
        for b in range(3):
            t.c[b][lens[b] + 1] = 0.0                        # not seen by the nodes compared
            t.k[b][lens[b] + 1] = 0.0
        want, wz, eo, ez = t.attend(UP_BF16 if dtype == "bf16" else 0.0, UP_BF16 if dtype == "bf16" else 2.0 ** -24)
        got, gz = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for i in (0, 2, 4):
            assert np.all(np.abs(got[:, i] - want[:, i]) <= eo[:, i] + 1e-30)
            fine = np.isfinite(wz[:, i])
            assert np.array_equal(gz[:, i][~fine], wz[:, i][~fine])
            assert np.all(np.abs(gz[:, i][fine] - wz[:, i][fine]) <= ez[:, i][fine])
        for b, (v, which) in bad.items():
            if which == "c":
                assert np.isnan(got[b, [1, 3]][..., 3]).all() or np.isinf(v)
                assert not np.isfinite(got[b, [1, 3]][..., 3]).any()
        # the weights of the others do not feel it either
        lse[:, [1, 3]] = float("inf")
        s = x.mass(plan, lse, None, 1.0).cpu().numpy()
        z = lse.double().cpu().numpy()
        for b, (m, e) in enumerate(t.mass(z, None, 1.0)):
            assert np.all(np.abs(s[b, :len(m)] - m) <= e + 1e-30)


def test_infinite_weights_rows_of_no_token_not_felt():
    """Pool rows of no token hold NaN throughout these tests; here the spare rows hold infinities too."""
    x = Batch(16, 2, [100, 129], page=64, seed=6)
    for t in (x.c, x.k):
        t[torch.isnan(t)] = float("inf")
    plan = x.plan()
    out, lse = x.decode(plan)
    ok(plan)
    check_tree(x, out, lse, tc=True)


@pytest.mark.parametrize("force", [False, True], ids=["auto", "simt"])
def test_rising_and_falling_logits(force):
    """Logits that rise from tile to tile by far more than an exponential's range, and fall."""
    for sign in (1.0, -1.0):
        x = Batch(16, 3, [900, 400], page=64, seed=7)
        for b in range(2):
            ramp = torch.linspace(0, 30, len(x.rows_of[b]), device="cuda")
            rows = torch.from_numpy(x.rows_of[b]).cuda()
            x.c[rows, 0] = (sign * ramp).to(BF16)
        x.q_c[..., 0] = 12.0
        plan = x.plan()
        if force:
            plan.set(kvc.OPT_FORCE_SIMT, 1)
        out, lse = x.decode(plan)
        ok(plan)
        check_tree(x, out, lse, tc=not force)


def test_the_longest_sequence():
    """2^31 - 4097 positions over a few pages that the table lists again and again: the drafted token, the last of
    them, has a logit of 60 where the others have none above 1, so it has all but e^(22 + 1 - 60) of the weight.  Both
    bounds are a unit of fp32 and that share."""
    cap = 2 ** 31 - 1 - 4096
    pages = -(-cap // 64)
    c = torch.rand(16 * 64, 8, device="cuda") / 8
    k = torch.zeros(16 * 64, 8, device="cuda")
    table = (torch.arange(pages, dtype=torch.int32, device="cuda") % 15)[None].contiguous()
    table[0, -1] = 15
    last = 15 * 64 + (cap - 1) % 64
    c[last] = 60.0 / 8
    q_c, q_r = torch.ones(1, 1, 1, 8, device="cuda"), torch.zeros(1, 1, 1, 8, device="cuda")
    out, lse = torch.empty(1, 1, 1, 8, device="cuda"), torch.empty(1, 1, 1, device="cuda")
    plan = kvc.Plan(1, 1, 8, 8, "f32", cap)
    plan.tree_decode(q_c, q_r, c, k, 64, table, torch.tensor([cap - 1], dtype=torch.int32).cuda(), out, lse)
    ok(plan)
    assert float((out - 7.5).abs().max()) <= 7.5 * (2.0 ** -22 + np.exp(-37.0))
    assert abs(float(lse) - 60.0) <= 60 * 2.0 ** -22


@pytest.mark.parametrize("H,T,lens,page", [(16, 8, [5000, 9000, 1200], 64), (128, 3, [4000, 2500], 128),
                                           (16, 1, [20000], 0), (32, 5, [3000] * 9, 64)])
def test_longer_contexts(H, T, lens, page):
    x = Batch(H, T, lens, page=page, seed=8)
    plan = x.plan()
    out, lse = x.decode(plan)
    ok(plan)
    check_tree(x, out, lse, tc=True)
    prev = torch.rand(x.B, x.cap, device="cuda")
    check_mass(x, x.mass(plan, lse, prev, 1.0), lse, prev, 1.0)


@pytest.mark.parametrize("B,H,T,most", [(40, 16, 3, 300), (150, 16, 2, 140), (33, 128, 3, 200), (40, 128, 9, 150), (70, 8, 3, 400),
                                        (1200, 16, 1, 150), (950, 16, 4, 140)])
def test_many_sequences(B, H, T, most):
    """More sequences than lanes of a warp; more row blocks than the schedule splits; some without drafted tokens."""
    r = np.random.default_rng(B)
    lens = [int(r.integers(0, most)) for _ in range(B)]
    drafts = [int(r.integers(0, T + 1)) for _ in range(B)]
    drafts[3] = T
    x = Batch(H, T, lens, drafts, page=64, seed=B)
    plan = x.plan()
    out, lse = x.decode(plan)
    ok(plan)
    prev = torch.rand(x.B, x.cap, device="cuda")
    s = x.mass(plan, lse, prev, 0.5)
    ok(plan)
    some = [0, 1, 3, 31, 32, B - 1]                          # the definition in 64 bits for a few of them
    y = x.tree()
    for a in ("lens", "drafts", "c", "k"):
        setattr(y, a, [getattr(y, a)[b] for b in some])
    y.q_c, y.q_r, y.words, y.B = y.q_c[some], y.q_r[some], y.words[some], len(some)
    z = Batch.__new__(Batch)
    z.B, z.drafts, z.dtype, z.tree = len(some), y.drafts, "bf16", lambda: y
    check_tree(z, out[some], lse[some], tc=True)
    check_mass(z, s[some], lse[some], prev[some], 0.5)
    simt = x.plan()                                          # and all of them against the other kernels
    simt.set(kvc.OPT_FORCE_SIMT, 1)
    o2, z2 = x.decode(simt)
    assert float((out.float() - o2.float()).abs().max()) <= 0.05
    assert torch.allclose(lse, z2, rtol=0, atol=2e-4)
    s2 = x.mass(simt, lse, prev, 0.5)
    assert torch.allclose(s, s2, rtol=2e-4, atol=1e-5)


@pytest.mark.parametrize("ctas", [1, 2, 7])
@pytest.mark.parametrize("H,T", [(16, 1), (16, 2), (16, 4), (128, 2)])
def test_few_ctas(H, T, ctas):
    x = Batch(H, T, [700, 0, 300], page=64, seed=31)
    plan = x.plan()
    plan.set(kvc.OPT_NUM_CTAS, ctas)
    out, lse = x.decode(plan)
    ok(plan)
    check_tree(x, out, lse, tc=True)
    check_mass(x, x.mass(plan, lse, None, 1.0), lse, None, 1.0)


def test_nothing_drafted_at_all():
    for lens in ([0, 0], [300, 40]):
        x = Batch(16, 2, lens, [0, 0], page=64, seed=32, extra=3)
        plan = x.plan()
        out, lse = x.decode(plan)
        assert bool((out == -77.0).all()) and bool((lse == -77.0).all())
        prev = torch.rand(x.B, x.cap, device="cuda")
        check_mass(x, x.mass(plan, lse, prev, 0.5), lse, prev, 0.5)
        ok(plan)


@pytest.mark.parametrize("H,T", [(16, 1), (16, 2), (16, 4), (24, 4), (128, 2)])
def test_a_wait_that_runs_out_is_reported(H, T):
    """The load that every CTA's first wait is for is left out: the bounded waits end, the error is reported, and the
    next call of the same plan is right."""
    x = Batch(H, T, [700, 130], page=64, seed=33)
    plan = x.plan()
    good, z = x.decode(plan)
    s = x.mass(plan, z, None, 1.0)
    plan.set(kvc.OPT_WAIT_TIMEOUT_NS, 20_000_000)
    plan.set(kvc.OPT_DEBUG_SKIP_LOAD, 1)
    x.decode(plan)
    assert plan.device_error() == kvc.LCA_ERR_DEVICE_TIMEOUT
    x.mass(plan, z, None, 1.0)
    assert plan.device_error() == kvc.LCA_ERR_DEVICE_TIMEOUT
    plan.set(kvc.OPT_DEBUG_SKIP_LOAD, 0)
    plan.set(kvc.OPT_WAIT_TIMEOUT_NS, 2_000_000_000)
    out, lse = x.decode(plan)
    assert torch.equal(out, good) and torch.equal(lse, z)
    assert torch.equal(x.mass(plan, z, None, 1.0), s)
    ok(plan)


def test_three_dimensional_and_strided_caches():
    """[B, capacity, d] caches are taken as they are; a strided one is refused rather than copied."""
    x = Batch(16, 2, [50, 90], seed=34)
    plan = x.plan()
    out, lse = x.decode(plan)
    c, k = x.c.view(2, x.cap, 512), x.k.view(2, x.cap, 64)
    got = torch.full_like(out, -77.0)
    plan.tree_decode(x.q_c, x.q_r, c, k, x.cap, None, x.dlens, got, mask=x.mask, draft_lens=x.ddrafts)
    assert torch.equal(got, out)
    wide = torch.zeros(2, x.cap, 600, dtype=BF16, device="cuda")[..., :512]
    with pytest.raises(kvc.LcaError):
        plan.tree_decode(x.q_c, x.q_r, wide, k, x.cap, None, x.dlens, got)
    with pytest.raises(kvc.LcaError):
        plan.cache_compact(wide, k, x.cap, None, torch.zeros(2, 1, dtype=torch.int32, device="cuda"),
                           torch.ones(2, dtype=torch.int32, device="cuda"))


def test_three_dimensional_caches_have_to_fit_the_page_size():
    x = Batch(16, 2, [50, 90], seed=35)
    plan = x.plan()
    out, _ = x.decode(plan)
    c, k = x.c.view(2, x.cap, 512), x.k.view(2, x.cap, 64)
    for page in (x.cap - 1, x.cap // 2):
        with pytest.raises(kvc.LcaError):
            plan.tree_decode(x.q_c, x.q_r, c, k, page, None, x.dlens, out, mask=x.mask)


@pytest.mark.parametrize("dtype,H", [("bf16", 16), ("f32", 4)])
def test_bad_lengths_and_pages_are_reported(dtype, H):
    kw = dict(dtype=dtype, **(dict(d_c=64, d_r=16) if dtype == "f32" else {}))
    x = Batch(H, 4, [200, 100, 300], page=64, seed=9, **kw)
    plan = x.plan()
    good, z = x.decode(plan)
    lens, drafts, table = x.dlens.clone(), x.ddrafts.clone(), x.dtable.clone()
    for which, value in (("lens", -1), ("lens", x.cap - 3), ("lens", 2 ** 31 - 1), ("drafts", 5), ("drafts", -1)):
        (x.dlens if which == "lens" else x.ddrafts)[1] = value
        out, lse = x.decode(plan)
        assert plan.device_error() == kvc.LCA_ERR_DEVICE_INPUT
        assert bool(torch.isnan(out[1]).all()) and bool(torch.isnan(lse[1]).all())
        assert torch.equal(out[[0, 2]], good[[0, 2]]) and torch.equal(lse[[0, 2]], z[[0, 2]])
        s = x.mass(plan, z, None, 1.0)
        assert plan.device_error() == kvc.LCA_ERR_DEVICE_INPUT
        assert bool((s[1] == -77.0).all())
        x.dlens.copy_(lens)
        x.ddrafts.copy_(drafts)
    for value in (-1, 10 ** 6):                              # page 0 is read instead
        x.dtable[2, 1] = value
        out, lse = x.decode(plan)
        assert plan.device_error() == kvc.LCA_ERR_DEVICE_INPUT
        assert torch.equal(out[:2], good[:2])
        x.mass(plan, z, None, 1.0)
        assert plan.device_error() == kvc.LCA_ERR_DEVICE_INPUT
        x.dtable.copy_(table)
    assert torch.equal(x.decode(plan)[0], good)
    ok(plan)


def test_refusals():
    x = Batch(16, 4, [200, 100], page=64, seed=10)
    plan = x.plan()
    ws = plan.tree_workspace(4)
    out = torch.empty(2, 4, 16, 512, dtype=BF16, device="cuda")
    lse = torch.empty(2, 4, 16, device="cuda")
    sc = torch.zeros(2, x.cap, device="cuda")

    def tree(status, **kw):
        a = dict(q_c=x.q_c, q_r=x.q_r, c_pool=x.c, k_pool=x.k, page_size=64, block_table=x.dtable, seq_lens=x.dlens,
                 out=out, lse=lse, mask=x.mask, draft_lens=x.ddrafts, workspace=ws)
        a.update(kw)
        with pytest.raises(kvc.LcaError) as e:
            plan.tree_decode(**a)
        assert e.value.status == status, e.value

    INV, ALIGN, UNSUP = 1, 3, 2
    tree(INV, q_c=x.q_c.float())
    tree(INV, q_c=x.q_c[:, ::2])
    tree(INV, q_r=x.q_r.transpose(1, 2).contiguous().transpose(1, 2))
    tree(INV, out=out.float())
    tree(INV, lse=lse.double())
    tree(INV, seq_lens=x.dlens.long())
    tree(INV, draft_lens=x.ddrafts[:1])
    tree(INV, mask=x.mask.int())
    tree(INV, block_table=x.dtable[:1])
    tree(INV, page_size=32)
    tree(INV, page_size=0)
    tree(INV, block_table=None, page_size=10 ** 6)           # fewer pages than sequences
    tree(INV, workspace=ws[:128])
    tree(INV, c_pool=x.c.cpu())
    big = torch.empty(ws.numel() + 256, dtype=torch.uint8, device="cuda")
    tree(ALIGN, workspace=big[8:])
    flat = torch.empty(2 * 4 * 16 * 512 + 8, dtype=BF16, device="cuda")
    tree(ALIGN, out=flat[1:1 + 2 * 4 * 16 * 512].view(2, 4, 16, 512))
    long = torch.zeros(2, 65, 16, 512, dtype=BF16, device="cuda")
    tree(INV, q_c=long, q_r=torch.zeros(2, 65, 16, 64, dtype=BF16, device="cuda"), out=torch.empty_like(long),
         lse=None, mask=None)
    plan.set(kvc.OPT_KERNEL, 3)                              # the two-CTA decode kernel has no such form
    tree(UNSUP)
    plan.set(kvc.OPT_KERNEL, 0)
    with pytest.raises(kvc.LcaError):
        plan.tree_workspace(65)
    with pytest.raises(kvc.LcaError):
        plan.attn_mass(x.q_c, x.q_r, x.c, x.k, 64, x.dtable, x.dlens, lse, sc.double(), workspace=ws)
    kept, kl = torch.zeros(2, 8, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    for sink, recent in ((-1, 0), (0, -1), (9, 0), (5, 4)):
        with pytest.raises(kvc.LcaError):
            plan.evict_select(sc, x.dlens, sink, recent, kept, kl)
    with pytest.raises(kvc.LcaError):
        plan.evict_select(sc, x.dlens.long(), 0, 0, kept, kl)
    with pytest.raises(kvc.LcaError):
        plan.cache_compact(x.c, x.k, 64, x.dtable, kept.long(), kl)
    torch.cuda.synchronize()
    ok(plan)


def _select_plan(B, L):
    return kvc.Plan(B, 1, 64, 16, "f32", L)


@pytest.mark.parametrize("lens,stride,sink,recent,budget,kind", [
    ([1000, 37, 64, 0, 65], 1000, 4, 16, 64, "normal"),
    ([5000, 4999], 5003, 0, 0, 1, "normal"),
    ([5000, 4097], 5000, 64, 128, 192, "normal"),            # nothing but the protected rows
    ([3000, 2049], 3000, 1, 0, 2048, "ties"),
    ([4096, 1025], 4100, 0, 7, 500, "equal"),
    ([2500], 2500, 3, 5, 600, "odd"),
    ([70000, 33000, 131072], 131072, 64, 4096, 16384, "normal"),
    ([131072], 131072, 0, 0, 131071, "ties"),
])
def test_select_matches_definition(lens, stride, sink, recent, budget, kind):
    B = len(lens)
    r = np.random.default_rng(sum(lens))
    s = np.exp(2 * r.standard_normal((B, stride))).astype(np.float32)
    if kind == "ties":
        s = np.floor(s * 2) / 2
    if kind == "equal":
        s[:] = 0.25
    if kind == "odd":                                        # signs, zeros of both, infinities, NaN, subnormals
        s = r.choice(np.array([-1.5, 0.0, -0.0, 1e-42, np.inf, -np.inf, np.nan, 3.0, 1e30], np.float32), (B, stride))
    plan = _select_plan(B, stride)
    kept = Guarded((B, budget), torch.int32, -7, -123456789)
    kl = Guarded((B,), torch.int32, -7, -123456789)
    x = torch.from_numpy(s).cuda()
    for b, n in enumerate(lens):
        x[b, n:] = float("nan")                              # not read
    plan.evict_select(x, torch.tensor(lens, dtype=torch.int32).cuda(), sink, recent, kept.t, kl.t)
    torch.cuda.synchronize()
    ok(plan)
    kept.check()
    kl.check()
    got = kept.t.cpu().numpy()
    for b, n in enumerate(lens):
        want = ref.select(s[b], n, sink, recent, budget)
        assert int(kl.t[b]) == len(want)
        assert np.array_equal(got[b, :len(want)], want), b
        assert np.all(got[b, len(want):] == -7)


@pytest.mark.parametrize("n", [20_000_000, 40_000_000])
def test_select_of_very_long_sequences(n):
    """Runs of thousands of rows a thread, where a row's place among the threads is no longer one multiplication."""
    sink, recent, budget = 7, 1000, 30_001
    g = torch.Generator(device="cuda").manual_seed(n)
    s = torch.randint(0, 1 << 22, (1, n), generator=g, device="cuda").float()      # about 10 rows of each sum
    kept = Guarded((1, budget), torch.int32, -7, -123456789)
    kl = torch.zeros(1, dtype=torch.int32, device="cuda")
    plan = kvc.Plan(1, 1, 8, 8, "f32", n)
    plan.evict_select(s, torch.tensor([n], dtype=torch.int32).cuda(), sink, recent, kept.t, kl)
    ok(plan)
    top = torch.sort(s[0, sink:n - recent], descending=True, stable=True).indices[:budget - sink - recent] + sink
    place = torch.cat([torch.arange(sink, device="cuda"), torch.arange(n - recent, n, device="cuda")])
    assert int(kl) == budget
    assert torch.equal(kept.t[0].long(), torch.sort(torch.cat([top, place])).values)
    kept.check()


def test_select_bad_length():
    plan = _select_plan(3, 100)
    x = torch.rand(3, 100, device="cuda")
    kept = torch.full((3, 10), -7, dtype=torch.int32, device="cuda")
    kl = torch.full((3,), -7, dtype=torch.int32, device="cuda")
    plan.evict_select(x, torch.tensor([50, 101, -1], dtype=torch.int32).cuda(), 1, 1, kept, kl)
    assert plan.device_error() == kvc.LCA_ERR_DEVICE_INPUT
    assert kl.tolist() == [10, 0, 0] and bool((kept[1:] == -7).all())


def _compact_reference(x: Batch, src, dst0, c, k, s):
    c, k, s = c.copy(), k.copy(), s.copy() if s is not None else None
    c0, k0, s0 = c.copy(), k.copy(), s.copy() if s is not None else None
    for b, rows in enumerate(src):
        for j, t in enumerate(rows):
            to, at = int(x.rows(b, dst0[b] + j)), int(x.rows(b, t))
            c[to], k[to] = c0[at], k0[at]
            if s is not None:
                s[b, dst0[b] + j] = s0[b, t]
    return c, k, s


def _bits(t):
    return t.view(torch.int16 if t.dtype == BF16 else torch.int32).cpu().numpy()


@pytest.mark.parametrize("lens,page,keep,commit,dtype,d_c,d_r", [
    ([1000, 700, 64, 1], 64, [300, 700, 0, 1], False, "bf16", 512, 64),
    ([5000, 3001], 128, [2500, 1], False, "bf16", 512, 64),
    ([900, 300], 0, [450, 299], False, "bf16", 512, 64),
    ([1001, 500], 0, [300, 200], False, "f32", 64, 16),
    ([700, 600, 500], 192, [350, 1, 499], False, "bf16", 128, 32),
    ([300], 64, [150], False, "f32", 1024, 256),
    ([200], 0, [100], False, "bf16", 8, 8),
    ([130, 63, 0, 500], 64, [5, 1, 16, 0], True, "bf16", 512, 64),
    ([70000], 64, [35000], False, "bf16", 512, 64),
])
@pytest.mark.parametrize("sums", [True, False], ids=["sums", "nosums"])
def test_compact_matches_definition(lens, page, keep, commit, dtype, d_c, d_r, sums):
    T = 16 if commit else 1
    x = Batch(1, T, lens, page=page, dtype=dtype, d_c=d_c, d_r=d_r, seed=12)
    r = np.random.default_rng(1)
    dst0 = list(lens) if commit else [0] * x.B
    src = []
    for b, m in enumerate(keep):
        pool = np.arange(lens[b], lens[b] + T) if commit else np.arange(lens[b])
        src.append(np.sort(r.choice(pool, m, replace=False)))
    if not commit and keep[0] > 10:
        src[0][:7] = np.arange(7)                            # rows at their place
        src[0] = np.unique(src[0])
    most = max(max(len(s) for s in src), 1) + 2
    arr = np.full((x.B, most), -5, np.int32)
    for b, s in enumerate(src):
        arr[b, :len(s)] = s
    sc = torch.rand(x.B, x.cap, device="cuda") if sums else None
    c, k = _bits(x.c), _bits(x.k)
    want = _compact_reference(x, src, dst0, c, k, sc.cpu().numpy() if sums else None)
    plan = x.plan()
    plan.cache_compact(x.c, x.k, x.page, x.dtable, torch.from_numpy(arr).cuda(),
                       torch.tensor([len(s) for s in src], dtype=torch.int32).cuda(),
                       dst0=torch.tensor(dst0, dtype=torch.int32).cuda() if commit else None, scores=sc)
    torch.cuda.synchronize()
    ok(plan)
    assert np.array_equal(_bits(x.c), want[0]) and np.array_equal(_bits(x.k), want[1])
    if sums:
        assert np.array_equal(sc.cpu().numpy(), want[2])


@pytest.mark.parametrize("lens,page,first,keep,dtype,d_c,d_r", [
    ([6000, 4000, 40, 5000], 64, [0, 100, 3, 0], [1100, 3899, 7, 0], "bf16", 512, 64),
    ([6000, 1500], 0, [3500, 0], [1300, 1499], "bf16", 512, 64),          # all from behind; nearly all from within
    ([9000], 192, [64], [2000], "bf16", 128, 32),
    ([5000, 5000], 0, [0, 1], [1500, 1200], "f32", 64, 16),
    ([4000], 64, [0], [2000], "f32", 1024, 256),
    ([30000] * 3, 64, [4, 0, 9], [7500, 29000, 5], "bf16", 512, 64),
])
@pytest.mark.parametrize("again", [1, 3])
def test_compact_of_long_lists(lens, page, first, keep, dtype, d_c, d_r, again):
    """Lists of several tiles, from any first row, with rows from within and from behind the destination; also one
    call behind another (the rows closed up, then taken out of each other's results)."""
    x = Batch(1, 1, lens, page=page, dtype=dtype, d_c=d_c, d_r=d_r, seed=44)
    r = np.random.default_rng(2)
    sc = torch.rand(x.B, x.cap, device="cuda")
    c, k, s = _bits(x.c), _bits(x.k), sc.cpu().numpy()
    plan = x.plan()
    for turn in range(again):
        src = [np.sort(r.choice(np.arange(first[b], lens[b]), keep[b] // (turn + 1), replace=False)) for b in range(x.B)]
        arr = np.full((x.B, max(len(a) for a in src) + 1), -5, np.int32)
        for b, a in enumerate(src):
            arr[b, :len(a)] = a
        c, k, s = _compact_reference(x, src, first, c, k, s)
        plan.cache_compact(x.c, x.k, x.page, x.dtable, torch.from_numpy(arr).cuda(),
                           torch.tensor([len(a) for a in src], dtype=torch.int32).cuda(),
                           dst0=torch.tensor(first, dtype=torch.int32).cuda(), scores=sc)
    ok(plan)
    assert np.array_equal(_bits(x.c), c) and np.array_equal(_bits(x.k), k) and np.array_equal(sc.cpu().numpy(), s)


@pytest.mark.parametrize("kind", ["random", "falling", "far", "page"])
def test_compact_long_bad_lists_stay_in_their_rows(kind):
    """Whatever a list holds, only the rows it may name as destinations of its own sequence change."""
    x = Batch(1, 1, [5000, 5000, 5000], page=64, seed=45)
    m, r = 1200, np.random.default_rng(3)
    src = np.tile(np.sort(r.choice(5000, m, replace=False)).astype(np.int32), (3, 1))
    if kind == "random":
        src[1] = r.integers(-2 ** 31, 2 ** 31 - 1, m)
    elif kind == "falling":
        src[1] = src[1, ::-1]
    elif kind == "far":
        src[1, 300:] = 10 ** 9
    table = x.dtable.clone()
    if kind == "page":
        table[1, 40:] = 10 ** 6
    c0 = _bits(x.c).copy()
    want, _, _ = _compact_reference(x, [src[0], [], src[2]], [0, 0, 0], c0, _bits(x.k), None)
    plan = x.plan()
    plan.cache_compact(x.c, x.k, 64, table, torch.from_numpy(src).cuda(), torch.full((3,), m, dtype=torch.int32).cuda())
    assert plan.device_error() == kvc.LCA_ERR_DEVICE_INPUT
    got = _bits(x.c)
    free = np.ones(len(c0), bool)
    free[x.rows(1, np.arange(m))] = False
    assert np.array_equal(got[free], want[free])


def test_compact_bad_lists_are_reported_and_harmless():
    x = Batch(1, 1, [300, 300, 300], page=64, seed=13)
    plan = x.plan()
    src = torch.tensor([[5, 9, 20], [5, 4, 9], [1, 2, 10 ** 6]], dtype=torch.int32).cuda()
    n = torch.tensor([3, 3, 3], dtype=torch.int32).cuda()
    c0 = _bits(x.c).copy()
    plan.cache_compact(x.c, x.k, 64, x.dtable, src, n)
    assert plan.device_error() == kvc.LCA_ERR_DEVICE_INPUT
    want = c0.copy()
    for b, moves in enumerate(([(0, 5), (1, 9), (2, 20)], [(0, 5), (2, 9)], [(0, 1), (1, 2)])):
        for to, at in moves:
            want[x.rows(b, to)] = c0[x.rows(b, at)]
    assert np.array_equal(_bits(x.c), want)
    for bad_n, bad_d in ((4, 0), (-1, 0), (1, -1), (1, 301)):
        before = _bits(x.c).copy()
        plan.cache_compact(x.c, x.k, 64, x.dtable, src[:1].repeat(3, 1).contiguous(),
                           torch.tensor([0, bad_n, 0], dtype=torch.int32).cuda(),
                           dst0=torch.tensor([0, bad_d, 0], dtype=torch.int32).cuda())
        assert plan.device_error() == kvc.LCA_ERR_DEVICE_INPUT
        assert np.array_equal(_bits(x.c), before)
    # a destination page out of range is not written (page 0 belongs to someone)
    before = _bits(x.c).copy()
    table = x.dtable.clone()
    table[0, 0] = -1
    plan.cache_compact(x.c, x.k, 64, table, torch.tensor([[100], [0], [0]], dtype=torch.int32).cuda(),
                       torch.tensor([1, 0, 0], dtype=torch.int32).cuda())
    assert plan.device_error() == kvc.LCA_ERR_DEVICE_INPUT
    assert np.array_equal(_bits(x.c), before)


@pytest.mark.parametrize("at,value", [(101, 100), (50, 60), (3, -1)])
def test_compact_reports_a_bad_entry_among_rows_at_their_place(at, value):
    x = Batch(1, 1, [300, 300], page=64, seed=43)
    plan = x.plan()
    src = np.tile(np.arange(200, dtype=np.int32), (2, 1))
    src[:, 199] = 250
    src[1, at] = value
    c0 = _bits(x.c).copy()
    plan.cache_compact(x.c, x.k, 64, x.dtable, torch.from_numpy(src).cuda(), torch.tensor([200, 200], dtype=torch.int32).cuda())
    assert plan.device_error() == kvc.LCA_ERR_DEVICE_INPUT
    want = c0.copy()
    for b in range(2):
        want[x.rows(b, 199)] = c0[x.rows(b, 250)]
    if value == 60:                                          # a good entry by itself; those after it break the order
        got = _bits(x.c)
        assert np.array_equal(got[x.rows(0, np.arange(300))], want[x.rows(0, np.arange(300))])
    else:
        assert np.array_equal(_bits(x.c), want)


def test_checked_build():
    """The range-checked debug build over the small cases: no check fails, the same bounds hold."""
    lib = kbuild.build_checked()
    for case in SMALL:
        x = small(case, seed=21)
        plan = x.plan(lib_path=lib)
        out, lse = x.decode(plan)
        ok(plan)
        check_tree(x, out, lse, tc=is_tc(x))
        check_mass(x, x.mass(plan, lse, None, 1.0), lse, None, 1.0)
        ok(plan)


@pytest.mark.parametrize("H,dtype", [(16, "bf16"), (128, "bf16"), (4, "f32")])
def test_graph_and_two_streams(H, dtype):
    """Captured and replayed with new contents; two graphs of one plan, each with its workspace, at once."""
    kw = dict(dtype=dtype, **(dict(d_c=64, d_r=16) if dtype == "f32" else {}))
    x = Batch(H, 6, [3000, 900], page=64, seed=14, **kw)
    y = Batch(H, 6, [3000, 900], page=64, seed=15, **kw)
    plan = x.plan()
    want = [b.decode(plan) for b in (x, y)]
    mass = [b.mass(plan, z, None, 1.0) for b, (_, z) in zip((x, y), want)]
    graphs, res = [], []
    for b in (x, y):
        ws = plan.tree_workspace(6)
        out, z = torch.zeros_like(want[0][0]), torch.zeros_like(want[0][1])
        s = torch.full_like(mass[0], -77.0)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            plan.tree_decode(b.q_c, b.q_r, b.c, b.k, b.page, b.dtable, b.dlens, out, z, mask=b.mask,
                             draft_lens=b.ddrafts, workspace=ws)
            plan.attn_mass(b.q_c, b.q_r, b.c, b.k, b.page, b.dtable, b.dlens, z, s, mask=b.mask,
                           draft_lens=b.ddrafts, workspace=ws)
        graphs.append((g, ws))
        res.append((out, z, s))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for o, z, s in res:
            o.zero_()
            z.zero_()
            s.fill_(-77.0)
        torch.cuda.synchronize()
        for st, (g, _) in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for (o, z, s), (wo, wz), wm in zip(res, want, mass):
            assert torch.equal(o, wo) and torch.equal(z, wz) and torch.equal(s, wm)
    ok(plan)
    # a call on a stream that is not the current one
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    o, z = x.decode(plan, stream=st)
    assert torch.equal(o, want[0][0]) and torch.equal(z, want[0][1])
    # lengths changed under the graph
    x.dlens.copy_(torch.tensor([100, 899], dtype=torch.int32))
    x.lens, x.rows_of = [100, 899], [x.rows(0, np.arange(106)), x.rows(1, np.arange(905))]
    graphs[0][0].replay()
    torch.cuda.synchronize()
    check_tree(x, res[0][0], res[0][1], tc=dtype == "bf16")


@pytest.mark.parametrize("H,dtype,page", [(16, "bf16", 64), (4, "f32", 0)])
def test_speculate_commit_score_evict_together(H, dtype, page):
    """Steps as a server would run them: draft a tree, attend, accept a path, add its weights up, commit it; when the
    cache is over its budget, choose and compact; then go on.  Each step against the definitions, on a CPU copy of
    the cache that is moved by the same lists."""
    T, budget, sink, recent = 6, 160, 4, 32
    kw = dict(dtype=dtype, **(dict(d_c=64, d_r=16) if dtype == "f32" else {}))
    x = Batch(H, T, [150, 90, 157], page=page, seed=16, extra=40, **kw)
    if page:                                                 # every sequence owns pages for its whole capacity
        per = -(-x.cap // page)
        x.table = np.random.default_rng(2).permutation(3 * per).astype(np.int32).reshape(3, per)
        rows = 3 * per * page
        x.dtable = torch.from_numpy(x.table).cuda()
    else:
        rows = 3 * x.cap
    x.c = torch.randn(rows, x.d_c, device="cuda").to(x.dt)
    x.k = torch.randn(rows, x.d_r, device="cuda").to(x.dt)
    plan = x.plan()
    ws = plan.tree_workspace(T)
    scores = torch.zeros(3, x.cap, device="cuda")
    r = np.random.default_rng(17)
    lens = np.array(x.lens)
    for step in range(6):
        x.lens = list(map(int, lens))
        x.dlens.copy_(torch.tensor(x.lens, dtype=torch.int32))
        x.rows_of = [x.rows(b, np.arange(n + T)) for b, n in enumerate(x.lens)]
        parents = np.stack([[r.integers(-1, i) if i else -1 for i in range(T)] for _ in range(3)])
        x.words = ref.words_of(parents)
        x.mask = kvc.tree_mask(torch.from_numpy(parents).cuda())
        x.q_c = (torch.randn_like(x.q_c.float()) * 2.5 / np.sqrt(x.d_c + x.d_r)).to(x.dt)
        for b, n in enumerate(x.lens):                       # the drafted tokens' latents
            at = torch.from_numpy(x.rows(b, np.arange(n, n + T))).cuda()
            x.c[at], x.k[at] = torch.randn(T, x.d_c, device="cuda").to(x.dt), torch.randn(T, x.d_r, device="cuda").to(x.dt)
        out, lse = x.decode(plan, ws=ws)
        check_tree(x, out, lse, tc=dtype == "bf16")
        path = []                                            # accepted: a leaf's path
        for b in range(3):
            i, p = int(r.integers(0, T)), []
            while i >= 0:
                p.append(i)
                i = int(parents[b, i])
            path.append(sorted(p))
        for b, p in enumerate(path):
            reject = [i for i in range(T) if i not in p]
            lse[b, reject] = float("inf")
        prev = scores.clone()
        plan.attn_mass(x.q_c, x.q_r, x.c, x.k, x.page, x.dtable, x.dlens, lse, scores, prev=scores, decay=0.5,
                       mask=x.mask, draft_lens=x.ddrafts, workspace=ws)
        got = scores.double().cpu().numpy()
        for b, (s, e) in enumerate(x.tree().mass(lse.double().cpu().numpy(), prev.double().cpu().numpy(), 0.5)):
            assert np.all(np.abs(got[b, :len(s)] - s) <= e + 1e-30)
        most = max(map(len, path))
        src = np.zeros((3, most), np.int32)
        for b, p in enumerate(path):
            src[b, :len(p)] = [x.lens[b] + i for i in p]
        want = _compact_reference(x, [src[b, :len(p)] for b, p in enumerate(path)], x.lens, _bits(x.c), _bits(x.k),
                                  scores.cpu().numpy())
        n_src = torch.tensor([len(p) for p in path], dtype=torch.int32).cuda()
        plan.cache_compact(x.c, x.k, x.page, x.dtable, torch.from_numpy(src).cuda(), n_src, dst0=x.dlens, scores=scores)
        assert np.array_equal(_bits(x.c), want[0]) and np.array_equal(scores.cpu().numpy(), want[2])
        new = x.dlens + n_src
        lens = new.cpu().numpy()
        kept = torch.zeros(3, budget, dtype=torch.int32, device="cuda")
        kl = torch.zeros(3, dtype=torch.int32, device="cuda")
        plan.evict_select(scores, new, sink, recent, kept, kl)
        sc = scores.cpu().numpy()
        keep = [ref.select(sc[b], int(lens[b]), sink, recent, budget) for b in range(3)]
        for b in range(3):
            assert np.array_equal(kept[b, :len(keep[b])].cpu().numpy(), keep[b])
        want = _compact_reference(x, keep, [0] * 3, _bits(x.c), _bits(x.k), sc)
        plan.cache_compact(x.c, x.k, x.page, x.dtable, kept, kl, scores=scores)
        assert np.array_equal(_bits(x.c), want[0]) and np.array_equal(_bits(x.k), want[1])
        assert np.array_equal(scores.cpu().numpy(), want[2])
        lens = kl.cpu().numpy()
    assert lens.max() == budget
    ok(plan)
