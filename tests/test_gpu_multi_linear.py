"""GPU tests of the many-adapter linear layer (forward, backward, the plan of a
batch) against the formulas in fp64, token by token with its own adapter.

Tolerances, element by element, with u = 2^-24 (half a step of fp32):
  A sum of k bf16 products on the tensor cores is taken 16 products at a time;
  each step may cut up to a whole step of fp32, 2 u, of the running sum, which
  never exceeds S = sum |a||b|; parts of K and the final sums add a few more:
  E(k) = (k / 16 + 32) 2 u S.  Sums on CUDA cores (one rounding of half a step a
  term) are below that.
  T, U: E(K).   T and U enter the W' product to 16 bits: 2^-16 |s T||L2| more.
  Y, dX: E(K) of the base sum, E(r) of the adapter's, and T's own error through L2.
  dL: three parts (24 bits): E(3 tokens), U's own error, 2^-23 of the products.
  bf16 outputs: one rounding, 2^-8 of the value, more."""
import numpy as np
import pytest
import torch

from oracle import nf4

import bit_nf4_quantized_blockwise_b200 as q
import synth
from _helpers import OTHER_CODEBOOKS, oracle_quantized

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def E(k, S):
    return (k / 16 + 32) * 2 * U * S


def ids_of(kind, M, n, none, seed):
    rng = np.random.default_rng(seed)
    if kind == "each":
        a = np.arange(M) % n
    elif kind == "runs":  # contiguous, ragged, in no order of adapters
        cuts = np.sort(rng.choice(np.arange(1, max(M, 2)), size=min(n, M) - 1, replace=False)) if M > 1 else []
        a = rng.permutation(n)[np.searchsorted(cuts, np.arange(M), side="right")]
    else:
        a = rng.integers(0, n, M)
    a = np.where(rng.random(M) < none, -1, a)
    return a.astype(np.int32)


class Case:
    def __init__(self, M, h, o, n, r, kind="runs", none=0.0, seed=0, codebook=None, dq=True, scale=None):
        g = torch.Generator().manual_seed(seed + 17)
        self.M, self.h, self.o, self.n, self.r = M, h, o, n, r
        cb = nf4.nf4_codebook() if codebook is None else codebook
        W_t = synth.weight_t(o, h, seed=seed)
        self.ids = ids_of(kind, M, n, none, seed)
        self.X = synth.activations(M, h, seed=seed, tag="X")
        self.dY = synth.activations(M, o, seed=seed, tag="dY")
        self.L1 = (torch.randn(n, h, r, generator=g) * 0.05).bfloat16()
        self.L2 = (torch.randn(n, r, o, generator=g) * 0.05).bfloat16()
        self.s = torch.rand(n, generator=g) + 0.25 if scale is None else scale
        if dq:
            cp, _, e, sc, mu = oracle_quantized(W_t, cb)
            wb = nf4.dequant(cp, e, sc, mu, cb)
            self.W = nf4.bf16_bits_to_f32(wb).reshape(o, h).astype(np.float64)
        self.Wq = q.quantize_weight(W_t.cuda(), cb, double_quant=dq)
        if not dq:
            self.W = q.qlora_dequant(self.Wq).double().cpu().numpy()

    def device(self):
        bank = q.AdapterBank(self.L1.cuda(), self.L2.cuda(), self.s.cuda())
        plan = q.qlora_adapter_plan(torch.from_numpy(self.ids).cuda(), self.n)
        return bank, plan

    def f64(self):
        return [t.double().numpy() for t in (self.X, self.dY, self.L1, self.L2, self.s)]

    def forward(self):
        """(Y, bound, T, bound)"""
        X, _, L1, L2, s = self.f64()
        Y, bY = X @ self.W.T, E(self.h, np.abs(X) @ np.abs(self.W).T)
        T, bT = np.zeros((self.M, self.r)), np.zeros((self.M, self.r))
        for a in range(self.n):
            at = np.nonzero(self.ids == a)[0]
            T[at] = X[at] @ L1[a]
            bT[at] = E(self.h, np.abs(X[at]) @ np.abs(L1[a]))
            S = s[a] * (np.abs(T[at]) @ np.abs(L2[a]))
            Y[at] += s[a] * (T[at] @ L2[a])
            bY[at] += E(2 * self.r, S) + 2.0 ** -16 * S + s[a] * (bT[at] @ np.abs(L2[a]))
        return Y, bY, T, bT

    def backward(self):
        """(dX, bound, dL1, bound, dL2, bound)"""
        X, dY, L1, L2, s = self.f64()
        _, _, T, bT = self.forward()
        dX, bX = dY @ self.W, E(self.o, np.abs(dY) @ np.abs(self.W))
        d1, b1 = np.zeros(L1.shape), np.zeros(L1.shape)
        d2, b2 = np.zeros(L2.shape), np.zeros(L2.shape)
        for a in range(self.n):
            at = np.nonzero(self.ids == a)[0]
            if not at.size:
                continue
            Ua = dY[at] @ L2[a].T
            bU = E(self.o, np.abs(dY[at]) @ np.abs(L2[a]).T)
            S = s[a] * (np.abs(Ua) @ np.abs(L1[a]).T)
            dX[at] += s[a] * (Ua @ L1[a].T)
            bX[at] += E(2 * self.r, S) + 2.0 ** -16 * S + s[a] * (bU @ np.abs(L1[a]).T)
            d1[a], d2[a] = s[a] * X[at].T @ Ua, s[a] * T[at].T @ dY[at]
            S1, S2 = s[a] * np.abs(X[at]).T @ np.abs(Ua), s[a] * np.abs(T[at]).T @ np.abs(dY[at])
            k = 3 * (at.size + 128)
            b1[a] = E(k, S1) + 2.0 ** -22 * S1 + s[a] * np.abs(X[at]).T @ bU
            b2[a] = E(k, S2) + 2.0 ** -22 * S2 + s[a] * bT[at].T @ np.abs(dY[at])
        return dX, bX, d1, b1, d2, b2


def near(got, want, bound):
    got = got.double().cpu().numpy()
    if got.dtype != np.float64 or got.shape != want.shape:
        raise AssertionError((got.shape, want.shape))
    off = np.abs(got - want) - bound
    assert np.all(np.isfinite(got)) and np.all(off <= 1e-30), (float(np.max(off)), np.unravel_index(np.argmax(off), off.shape))


def rounded(want, bound, dtype):
    return bound + (2.0 ** -8 * np.abs(want) + 2.0 ** -8 * bound if dtype == torch.bfloat16 else 0.0)


def check(c, dtype=torch.float32, saved=True):
    bank, plan = c.device()
    X, dY = c.X.cuda(), c.dY.cuda()
    Y, T = q.qlora_multi_linear_fwd(c.Wq, X, bank, plan, y_dtype=dtype)
    dX, d1, d2 = q.qlora_multi_linear_bwd(c.Wq, X, dY, bank, plan, T_saved=T if saved else None, dx_dtype=dtype)
    torch.cuda.synchronize()
    q.qlora_check_status()
    wY, bY, wT, bT = c.forward()
    near(T, wT, bT)
    assert Y.dtype == dtype and dX.dtype == dtype
    near(Y, wY, rounded(wY, bY, dtype))
    wX, bX, w1, b1, w2, b2 = c.backward()
    near(dX, wX, rounded(wX, bX, dtype))
    near(d1, w1, b1)
    near(d2, w2, b2)


# ---------------------------------------------------------------- the plan

@pytest.mark.parametrize("M,n", [(1, 1), (1, 7), (31, 3), (256, 1), (257, 5), (1000, 1000), (5000, 40), (4096, 2500)])
@pytest.mark.parametrize("kind,none", [("each", 0.0), ("runs", 0.0), ("runs", 0.3), ("mixed", 0.1), ("mixed", 1.0)])
def test_plan_groups_tokens_stably(M, n, kind, none):
    ids = ids_of(kind, M, n, none, seed=M + n)
    if M > 2:
        ids[M // 2] = n + 5  # out of range: none
    plan = q.qlora_adapter_plan(torch.from_numpy(ids).cuda(), n)
    b = plan.buffer.cpu().numpy()
    own = np.where((ids >= 0) & (ids < n), ids, -1)
    order = []
    for a in own.tolist():
        if a not in order:
            order.append(a) if M < 300 else None
            if M >= 300:
                break
    if M >= 300:
        _, at = np.unique(own, return_index=True)
        order = own[np.sort(at)].tolist()
    want = np.concatenate([np.nonzero(own == a)[0] for a in order])
    pad = lambda k: (4 * k + 255) // 256 * 256  # noqa: E731
    head = b[:16].view(np.int32)
    perm = b[256:256 + 4 * M].view(np.int32)
    assert np.array_equal(perm, want)
    assert head[0] == len([a for a in order if a >= 0]) and head[1] == int(np.array_equal(want, np.arange(M)))
    owner = b[256 + pad(M):256 + pad(M) + 4 * M].view(np.int32)
    assert np.array_equal(owner, own)


# ---------------------------------------------------------------- the layer

@pytest.mark.parametrize("M", [1, 2, 9, 17, 33, 64, 200, 257, 513])
@pytest.mark.parametrize("kind", ["runs", "mixed"])
def test_token_counts(M, kind):
    check(Case(M, 512, 384, 5, 16, kind=kind, none=0.2, seed=M))


@pytest.mark.parametrize("h,o", [(128, 128), (256, 576), (576, 256), (1024, 320), (320, 1024)])
def test_ragged_feature_tiles(h, o):
    check(Case(150, h, o, 3, 24, seed=h + o))


@pytest.mark.parametrize("r", [8, 16, 24, 40, 64, 72, 128, 136, 200, 256])
def test_ranks(r):
    check(Case(140, 256, 512, 4, r, kind="mixed", none=0.1, seed=r), saved=False)


@pytest.mark.parametrize("M", [1, 8, 16, 17, 32])
@pytest.mark.parametrize("h,o,r", [(64, 256, 8), (192, 256, 72), (128, 1152, 256), (2048, 128, 64), (4096, 320, 16)])
def test_decode_shapes(M, h, o, r):
    check(Case(M, h, o, 5, r, kind="mixed", none=0.2, seed=M + r))


@pytest.mark.parametrize("M,h,o,n", [(34, 64, 256, 2), (260, 2048, 128, 3), (40, 4096, 64, 40), (1025, 64, 512, 2),
                                     (256, 512, 9728, 2)])
def test_narrow_and_wide_layers(M, h, o, n):
    check(Case(M, h, o, n, 8, kind="mixed", none=0.1, seed=M + h))


@pytest.mark.parametrize("M,n,kind", [(300, 300, "each"), (700, 90, "mixed"), (1300, 1, "runs"), (1290, 6, "runs"),
                                      (64, 200, "mixed"), (16, 16, "each"), (32, 5, "mixed")])
def test_group_sizes(M, n, kind):
    check(Case(M, 384, 512, n, 16, kind=kind, none=0.05, seed=M + n))


@pytest.mark.parametrize("M", [8, 40, 600])
def test_bf16_outputs(M):
    check(Case(M, 512, 768, 4, 64, kind="mixed", none=0.1, seed=M), dtype=torch.bfloat16)


def test_deep_and_wide():
    check(Case(530, 2048, 1536, 7, 64, seed=3))
    check(Case(2100, 1024, 4096, 3, 32, kind="mixed", seed=4))


@pytest.mark.parametrize("M", [4, 20, 130])
def test_no_adapter_at_all(M):
    c = Case(M, 256, 384, 3, 8, none=1.1, seed=M)
    assert np.all(c.ids == -1)
    check(c)


@pytest.mark.parametrize("M", [16, 100])
@pytest.mark.parametrize("cb", list(OTHER_CODEBOOKS))
def test_other_codebooks(cb, M):
    check(Case(M, 256, 320, 3, 16, seed=9, codebook=OTHER_CODEBOOKS[cb]))


@pytest.mark.parametrize("M", [5, 90])
def test_single_level_constants(M):
    check(Case(M, 320, 192, 3, 16, seed=9, dq=False))


def test_one_adapter_matches_the_single_adapter_layer():
    c = Case(300, 512, 768, 1, 64, seed=2, scale=torch.tensor([0.25]))
    bank, plan = c.device()
    X, dY = c.X.cuda(), c.dY.cuda()
    Y, T = q.qlora_multi_linear_fwd(c.Wq, X, bank, plan)
    Z, S = q.qlora_linear_fwd(c.Wq, X, bank.L1[0], bank.L2[0], 0.25)
    _, bY, _, bT = c.forward()
    near(Y, Z.double().cpu().numpy(), 2 * bY)
    near(T, S.double().cpu().numpy(), 2 * bT)


# ---------------------------------------------------------------- isolation

def _bad(c, what, value):
    if what == "X":
        c.X[c.M // 2, 3] = value
    elif what == "dY":
        c.dY[c.M // 2, 5] = value
    elif what == "L1":
        c.L1[1, 7, 2] = value
    else:
        c.L2[1, 2, 9] = value


@pytest.mark.parametrize("M,kind", [(12, "mixed"), (30, "each"), (150, "mixed"), (400, "runs")])
@pytest.mark.parametrize("what", ["X", "dY", "L1", "L2"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_nonfinite_values_stay_with_their_token_and_adapter(M, kind, what, value):
    """One bad value in one token or one adapter: everything that does not depend on it is what it
    is without it."""
    c = Case(M, 256, 320, 3, 16, kind=kind, none=0.1, seed=M)
    wY, bY, wT, bT = c.forward()
    wX, bX, w1, b1, w2, b2 = c.backward()
    _bad(c, what, value)
    bank, plan = c.device()
    X, dY = c.X.cuda(), c.dY.cuda()
    Y, T = q.qlora_multi_linear_fwd(c.Wq, X, bank, plan)
    dX, d1, d2 = q.qlora_multi_linear_bwd(c.Wq, X, dY, bank, plan, T_saved=T)
    torch.cuda.synchronize()
    q.qlora_check_status()
    bad_row = c.M // 2
    rows = np.ones(M, bool)      # tokens that must be as before
    if what in ("X", "dY"):
        rows[bad_row] = False
        bad_adapter = int(c.ids[bad_row])
    else:
        rows = c.ids != 1
        bad_adapter = 1
    ads = np.array([a != bad_adapter for a in range(c.n)])
    if what != "dY":
        near(Y[rows], wY[rows], bY[rows])
        near(T[rows], wT[rows], bT[rows])
    if what != "X":
        near(dX[rows], wX[rows], bX[rows])
    near(d1[ads], w1[ads], b1[ads])
    near(d2[ads], w2[ads], b2[ads])
    if what == "X":
        assert not torch.isfinite(Y[bad_row]).any()
    if what == "dY":
        assert not torch.isfinite(dX[bad_row]).any()


@pytest.mark.parametrize("M", [20, 300, 1300])
def test_a_batch_of_nan_ends_and_keeps_to_itself(M):
    """All of X and dY NaN but for the tokens of adapter 2, which are as before."""
    c = Case(M, 256, 320, 3, 16, kind="mixed", none=0.1, seed=M)
    mine = c.ids == 2
    wY, bY, wT, bT = c.forward()
    wX, bX, w1, b1, w2, b2 = c.backward()
    c.X[torch.from_numpy(~mine)] = float("nan")
    c.dY[torch.from_numpy(~mine)] = float("nan")
    bank, plan = c.device()
    X, dY = c.X.cuda(), c.dY.cuda()
    Y, T = q.qlora_multi_linear_fwd(c.Wq, X, bank, plan)
    dX, d1, d2 = q.qlora_multi_linear_bwd(c.Wq, X, dY, bank, plan, T_saved=T)
    torch.cuda.synchronize()
    q.qlora_check_status()
    near(Y[mine], wY[mine], bY[mine])
    near(dX[mine], wX[mine], bX[mine])
    near(d1[2:], w1[2:], b1[2:])
    near(d2[2:], w2[2:], b2[2:])
    assert torch.isnan(Y[~mine]).all() and torch.isnan(dX[~mine]).all()


@pytest.mark.parametrize("M", [20, 300])
def test_an_adapter_of_nan_keeps_to_its_tokens(M):
    c = Case(M, 256, 320, 3, 16, kind="mixed", none=0.1, seed=M)
    mine = c.ids != 1
    wY, bY, _, _ = c.forward()
    wX, bX, _, _, _, _ = c.backward()
    c.L1[1] = float("nan")
    c.L2[1] = float("inf")
    bank, plan = c.device()
    X, dY = c.X.cuda(), c.dY.cuda()
    Y, _ = q.qlora_multi_linear_fwd(c.Wq, X, bank, plan, y_dtype=torch.bfloat16)
    dX, _, _ = q.qlora_multi_linear_bwd(c.Wq, X, dY, bank, plan, dx_dtype=torch.bfloat16)
    near(Y[mine], wY[mine], rounded(wY, bY, torch.bfloat16)[mine])
    near(dX[mine], wX[mine], rounded(wX, bX, torch.bfloat16)[mine])
    assert not torch.isfinite(Y[~mine]).any() and not torch.isfinite(dX[~mine]).any()


@pytest.mark.parametrize("M,h,o", [(70, 5184, 256), (330, 256, 10304)])
def test_wide_rows_out_of_order(M, h, o):
    """Rows of a little more than one and two pieces of the sorting copies."""
    check(Case(M, h, o, 5, 16, kind="mixed", none=0.1, seed=M))


def test_large_bank_with_few_of_its_adapters_in_the_batch():
    c = Case(70, 128, 128, 3000, 8, kind="mixed", seed=4)
    c.ids = np.where(c.ids % 3 == 0, 2999, c.ids % 5).astype(np.int32)
    check(c)


# ---------------------------------------------------------------- how it is called

def test_results_repeat_bit_for_bit():
    c = Case(700, 512, 640, 6, 64, kind="mixed", seed=1)
    bank, plan = c.device()
    X, dY = c.X.cuda(), c.dY.cuda()
    outs = [q.qlora_multi_linear_fwd(c.Wq, X, bank, plan) + q.qlora_multi_linear_bwd(c.Wq, X, dY, bank, plan)
            for _ in range(3)]
    for other in outs[1:]:
        for a, b in zip(outs[0], other):
            assert torch.equal(a, b)


@pytest.mark.parametrize("M", [6, 24, 300])
def test_other_stream_given_outputs_and_reused_workspace(M):
    c = Case(M, 256, 512, 4, 16, kind="mixed", none=0.1, seed=M)
    wY, bY, wT, bT = c.forward()
    wX, bX, w1, b1, w2, b2 = c.backward()
    L = q.lib()
    ws = torch.full((max(L.qlora_multi_linear_fwd_workspace_size(512, 256, M, 4, 16),
                         L.qlora_multi_linear_bwd_workspace_size(512, 256, M, 4, 16)),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        bank, plan = c.device()
        X, dY = c.X.cuda(), c.dY.cuda()
        Y = torch.full((M, 512), float("nan"), device="cuda")
        T = torch.full((M, 16), float("nan"), device="cuda")
        dX = torch.full((M, 256), float("nan"), device="cuda")
        d1 = torch.full((4, 256, 16), float("nan"), device="cuda")
        d2 = torch.full((4, 16, 512), float("nan"), device="cuda")
        for _ in range(2):
            q.qlora_multi_linear_fwd(c.Wq, X, bank, plan, Y=Y, T_save=T, ws=ws)
            q.qlora_multi_linear_bwd(c.Wq, X, dY, bank, plan, T_saved=T, dX=dX, dL1=d1, dL2=d2, ws=ws)
    torch.cuda.current_stream().wait_stream(st)
    near(Y, wY, bY)
    near(T, wT, bT)
    near(dX, wX, bX)
    near(d1, w1, b1)
    near(d2, w2, b2)


@pytest.mark.parametrize("M", [7, 28, 300])
def test_captured_batch_replays_with_new_tokens_and_adapters(M):
    c = Case(M, 256, 384, 4, 16, kind="mixed", seed=5)
    d = Case(M, 256, 384, 4, 16, kind="runs", none=0.3, seed=5)
    d.X = synth.activations(M, 256, seed=77, tag="X")
    ids, X = torch.from_numpy(c.ids).cuda(), c.X.cuda()
    dY = c.dY.cuda()
    bank, plan = c.device()

    def work():
        q.qlora_adapter_plan(ids, 4, plan=plan)
        Y, T = q.qlora_multi_linear_fwd(c.Wq, X, bank, plan)
        return (Y, T) + q.qlora_multi_linear_bwd(c.Wq, X, dY, bank, plan, T_saved=T)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        work()
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for case in (c, d, c):
        ids.copy_(torch.from_numpy(case.ids))
        X.copy_(case.X)
        graph.replay()
        torch.cuda.synchronize()
        wY, bY, wT, bT = case.forward()
        wX, bX, w1, b1, w2, b2 = case.backward()
        for got, want, bound in zip(out, (wY, wT, wX, w1, w2), (bY, bT, bX, b1, b2)):
            near(got, want, bound)


def test_gradients_match_differences():
    """d<Y, dY> along a random direction of X, L1[a] and L2[a], by central differences of the fp64 forward."""
    c = Case(40, 128, 256, 3, 8, kind="mixed", none=0.1, seed=8)
    bank, plan = c.device()
    X, dY = c.X.cuda(), c.dY.cuda()
    dX, d1, d2 = (t.double().cpu().numpy() for t in q.qlora_multi_linear_bwd(c.Wq, X, dY, bank, plan))
    Xd, dYd, L1, L2, s = c.f64()

    def loss(X, L1, L2):
        Y = X @ c.W.T
        for a in range(c.n):
            at = c.ids == a
            Y[at] += s[a] * (X[at] @ L1[a]) @ L2[a]
        return float(np.sum(Y * dYd))
    rng = np.random.default_rng(0)
    for k, (x, g) in enumerate(((Xd, dX), (L1, d1), (L2, d2))):
        v = rng.standard_normal(x.shape)
        e = 1e-4
        args = [[Xd, L1, L2], [Xd, L1, L2]]
        args[0][k], args[1][k] = x + e * v, x - e * v
        # the loss is bilinear in X and each factor: the difference is exact up to fp64
        diff = (loss(*args[0]) - loss(*args[1])) / (2 * e)
        assert abs(float(np.sum(g * v)) - diff) <= 1e-4 * np.sqrt(np.sum(g * g) * np.sum(v * v)) + 1e-6


def test_training_several_adapters_as_used():
    """Forward, backward and the many-tensor AdamW step in a row: each adapter moves as it does when it
    is trained alone with its own tokens by the same kernels, and one without tokens stays."""
    c = Case(90, 256, 384, 4, 16, kind="mixed", seed=12)
    c.ids[c.ids == 3] = 0   # adapter 3 has no tokens
    X, dY = c.X.cuda(), c.dY.cuda()
    masters = [t.float().cuda() for t in (c.L1, c.L2)]

    def train(ids, steps=3):
        p = [m.clone() for m in masters]
        copies = [m.bfloat16() for m in masters]
        bank = q.AdapterBank(copies[0], copies[1], c.s.cuda())
        opt = q.MultiAdamW([x[a] for x in p for a in range(4)], copies=[x[a] for x in copies for a in range(4)])
        opt.cfg.max_grad_norm = None
        for _ in range(steps):
            plan = q.qlora_adapter_plan(torch.from_numpy(ids).cuda(), 4)
            _, T = q.qlora_multi_linear_fwd(c.Wq, X, bank, plan)
            _, g1, g2 = q.qlora_multi_linear_bwd(c.Wq, X, dY, bank, plan, T_saved=T)
            there = np.isin(np.arange(4), ids)
            opt.step([g[a] if there[a] else None for g in (g1, g2) for a in range(4)])
        return p
    together = train(c.ids)
    for a in range(3):
        alone = train(np.where(c.ids == a, a, -1).astype(np.int32))
        for x, y in zip(together, alone):
            # sums of other lengths round differently; three steps of lr 2e-4 move by 6e-4 at most
            assert float((x[a] - y[a]).abs().max()) <= 2e-5
            assert not torch.equal(x[a], masters[0][a] if x is together[0] else masters[1][a])
    for x, m in zip(together, masters):
        assert torch.equal(x[3], m[3])
