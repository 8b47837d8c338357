"""Attention, forward and backward, against softmax attention in 64 bits.

Two bounds per output. (1) Per element, the worst case: P enters its product rounded to bf16 (2^-8 of each
probability), so O is within 2^-8 sum_j P_j |V_j| of it, plus half a step of O itself; dV likewise with |dO|. dS is
rounded to bf16 (2^-8 |dS|) and carries delta, formed from the bf16 O: P times 2^-8 sum |dO| |O|. The 32-bit part (S
and dP of at most 128 products, exp2, sums) is below 2^-11 of a term: 128 * 2^-24 of sum |q| |k| scale, at most 2^5
here, is 2^-12. (2) Over the whole tensor: roundings are independent, so the errors' squares add up; the 2-norm of the
difference is held to that of 2^-8 times each term, sqrt(3) above what uniform roundings give. One key too many or too
few in a row breaks this bound at any length here.
"""
import math

import pytest
import torch

import bit_nf4_quantized_03_b200 as q
from tests.gpu_util import ensure_built

pytestmark = pytest.mark.gpu
H = 2.0 ** -8          # half a bf16 step
F = 2.0 ** -11         # the 32-bit part, relative to a term
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def visible(nq, nk, causal, window):
    i = torch.arange(nq, device="cuda")[:, None] + (nk - nq)
    j = torch.arange(nk, device="cuda")[None]
    ok = torch.ones(nq, nk, dtype=torch.bool, device="cuda")
    if causal:
        ok &= j <= i
    if window:
        ok &= j > i - window
    return ok


class Problem:
    def __init__(self, q_lens, k_lens, hq, hkv, d, causal=False, window=0, seed=0, scale=None, spare=0, lead=0):
        """spare, lead: tokens behind the last sequence and before the first one, in none of them."""
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.q_lens, self.k_lens, self.hq, self.hkv, self.d = list(q_lens), list(k_lens), hq, hkv, d
        self.causal, self.window, self.lead = causal, window, lead
        self.scale = d ** -0.5 if scale is None else scale
        tq, tk = sum(q_lens) + spare + lead, sum(k_lens) + spare + lead
        self.Q, self.K, self.V = (2 * rnd(tq, hq, d)).to(BF), rnd(tk, hkv, d).to(BF), rnd(tk, hkv, d).to(BF)
        self.dO = rnd(tq, hq, d).to(BF)
        cum = lambda l: torch.tensor([lead + sum(l[:i]) for i in range(len(l) + 1)], dtype=torch.int32, device="cuda")  # noqa: E731
        self.cu_q, self.cu_k = cum(q_lens), cum(k_lens)
        self.how = dict(causal=causal, window=window, scale=scale, cu_q=self.cu_q, cu_k=self.cu_k)

    def parts(self):
        a = b = self.lead
        for nq, nk in zip(self.q_lens, self.k_lens):
            yield slice(a, a + nq), slice(b, b + nk), nq, nk
            a, b = a + nq, b + nk

    def forward(self):
        O = torch.full_like(self.Q, 7.0)
        lse = torch.full(self.Q.shape[:2], 7.0, device="cuda")
        q.qlora_attention_fwd(self.Q, self.K, self.V, O, lse, **self.how)
        q.qlora_check_device_error()
        return O, lse

    def backward(self, O, lse):
        g = [torch.full_like(t, 7.0) for t in (self.Q, self.K, self.V)]
        q.qlora_attention_bwd(self.Q, self.K, self.V, O, self.dO, lse, *g, **self.how)
        q.qlora_check_device_error()
        return g

    def reference(self, with_grads=True):
        """{name: (value, worst case, root of the squares)} in 64 bits; tokens in no sequence keep the filling."""
        dev, f8 = "cuda", torch.float64
        group = self.hq // self.hkv
        shapes = {"O": self.Q.shape, "dQ": self.Q.shape, "dK": self.K.shape, "dV": self.V.shape}
        out = {n: [torch.full(s, 7.0, dtype=f8, device=dev), *(torch.zeros(s, dtype=f8, device=dev) for _ in range(2))]
               for n, s in shapes.items()}
        lse_all = torch.full(self.Q.shape[:2], 7.0, dtype=f8, device=dev)
        lse_tol = torch.zeros_like(lse_all)
        for sq, sk, nq, nk in self.parts():
            ok = visible(nq, nk, self.causal, self.window)
            for kh in range(self.hkv):
                K, V = self.K[sk, kh].double(), self.V[sk, kh].double()
                acc = [torch.zeros(nk, self.d, dtype=f8, device=dev) for _ in range(6)]     # dK, dV: value, worst, squares
                for h in range(kh * group, (kh + 1) * group):
                    Q, dO = self.Q[sq, h].double(), self.dO[sq, h].double()
                    S = (Q @ K.T * self.scale).masked_fill(~ok, -math.inf)
                    lse = torch.logsumexp(S, 1) if nk else torch.full((nq,), -math.inf, dtype=f8, device=dev)
                    P = torch.exp(S - torch.where(lse == -math.inf, 0.0, lse)[:, None])
                    O = P @ V
                    lse_all[sq, h] = lse
                    sizes = (Q.abs() @ K.abs().T * self.scale).amax(1) if nk else torch.zeros(nq, dtype=f8, device=dev)
                    lse_tol[sq, h] = 2.0 ** -17 * sizes + 2.0 ** -18 * (1 + torch.where(lse == -math.inf, 0.0, lse.abs()))
                    for i, t in enumerate((O, (H + F) * (P @ V.abs()) + H * O.abs(), H * H * (P ** 2 @ V ** 2 + O ** 2))):
                        out["O"][i][sq, h] = t
                    if not with_grads:
                        continue
                    dP = dO @ V.T
                    delta = (dO * O).sum(1, keepdim=True)
                    dS = P * (dP - delta)
                    noise = (dO.abs() * O.abs()).sum(1, keepdim=True)           # delta's sizes
                    fine = dO.abs() @ V.abs().T                                 # dP's sizes
                    E = (H + F) * dS.abs() + P * (H * noise + F * (fine + noise))
                    E2 = H * H * (dS ** 2 + P ** 2 * (dO ** 2 * O ** 2).sum(1, keepdim=True)) + (F * P * (fine + noise)) ** 2
                    c = self.scale
                    dQ = c * dS @ K
                    for i, t in enumerate((dQ, c * E @ K.abs() + H * dQ.abs(), c * c * E2 @ K ** 2 + (H * dQ) ** 2)):
                        out["dQ"][i][sq, h] = t
                    for i, t in enumerate((c * dS.T @ Q, c * E.T @ Q.abs(), c * c * E2.T @ Q ** 2,
                                           P.T @ dO, (H + F) * (P.T @ dO.abs()), H * H * (P ** 2).T @ dO ** 2)):
                        acc[i] += t
                for name, at in (("dK", 0), ("dV", 3)):
                    v, worst, sq2 = acc[at:at + 3]
                    for i, t in enumerate((v, worst + H * v.abs(), sq2 + (H * v) ** 2)):
                        out[name][i][sk, kh] = t
        return {n: (v, w, s.sqrt()) for n, (v, w, s) in out.items()}, lse_all, lse_tol


def close(got, ref, name):
    value, worst, root = ref
    assert torch.isfinite(got).all(), name
    d = (got.double() - value).abs()
    bad = d > worst + 1e-30
    assert not bad.any(), (name, int(bad.sum()), float((d / (worst + 1e-30)).max()), bad.nonzero()[:4].tolist())
    total, allow = float(d.norm()), float(root.norm())
    assert total <= allow + 1e-30, (name, total, allow)


def check(p, grads=True):
    ref, lse_ref, lse_tol = p.reference(grads)
    O, lse = p.forward()
    close(O, ref["O"], "O")
    empty = lse_ref == -math.inf
    assert (lse[empty] == -math.inf).all()
    d = (lse.double() - lse_ref)[~empty].abs()
    assert (d <= lse_tol[~empty]).all(), float((d / lse_tol[~empty]).max())
    if not grads:
        return
    got = p.backward(O, lse)
    for name, t in zip(("dQ", "dK", "dV"), got):
        close(t, ref[name], name)
    again = p.backward(*p.forward())
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("n", [1, 2, 64, 100, 128, 129, 257, 520])
def test_one_sequence(n, d, causal):
    check(Problem([n], [n], 2, 2, d, causal, seed=n))


@pytest.mark.parametrize("d", [8, 40, 72, 80, 96, 120])
def test_head_dims(d):
    check(Problem([70, 200], [70, 200], 2, 1, d, True, seed=d))


@pytest.mark.parametrize("hq,hkv", [(3, 1), (4, 2), (7, 1), (12, 4), (16, 1), (33, 1), (64, 1), (64, 2)])
@pytest.mark.parametrize("d", [128, 64])
def test_shared_key_heads(hq, hkv, d):
    check(Problem([5, 90], [5, 90], hq, hkv, d, True, seed=hq))


@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 1), (True, 17), (True, 128), (True, 1000)])
def test_ragged_sequences(causal, window):
    # none, one and many tokens; fewer keys than queries leaves rows empty under a causal mask; more keys continue one
    q_lens = [0, 1, 130, 5, 300, 64, 0, 33]
    k_lens = [4, 1, 130, 200, 170, 0, 0, 400]
    check(Problem(q_lens, k_lens, 4, 2, 64, causal, window, seed=window))


@pytest.mark.parametrize("window", [1, 63, 64, 65, 129, 300])
def test_window_over_many_tiles(window):
    check(Problem([700, 37], [700, 260], 3, 3, 128, True, window, seed=window))


@pytest.mark.parametrize("k_lens", [[5000], [257, 4096, 1, 900], [64] * 40])
@pytest.mark.parametrize("new", [1, 3, 16])
@pytest.mark.parametrize("hq,hkv,d", [(8, 1, 128), (8, 8, 64), (14, 2, 128)])
def test_few_queries_on_long_keys(k_lens, new, hq, hkv, d):
    check(Problem([new] * len(k_lens), k_lens, hq, hkv, d, True, seed=new), grads=len(k_lens) == 4)


def test_many_sequences():
    lens = [(i * 7) % 19 for i in range(150)]
    check(Problem(lens, lens, 2, 1, 64, True, seed=3))


def test_large_and_small_logits():
    # rows whose maximum grows over the tiles, and a scale that makes the softmax one-hot
    p = Problem([300], [300], 2, 2, 128, True, seed=5, scale=0.02)
    check(p)
    p = Problem([300], [300], 2, 2, 64, False, seed=6, scale=0.9)
    p.K[:150] *= 0.1
    p.K[290:] *= 4
    ref, lse_ref, _ = p.reference(False)
    O, lse = p.forward()
    # S reaches 2^9 here: 64 * 2^-24 of sum |q| |k| scale (below 2^11) is 2^-7 in the exponent
    assert ((O.double() - ref["O"][0]).abs() <= ref["O"][1] + 2.0 ** -7 * ref["O"][1] / H).all()
    assert torch.isfinite(lse).all() and float((lse.double() - lse_ref).abs().max()) <= 2.0 ** -7 + 2.0 ** -14


def test_values_outside_a_sequence_do_not_reach_it():
    # NaN and infinity behind the last sequence, before the first, and in a whole neighbouring sequence
    for d, hq, hkv in ((128, 2, 2), (64, 6, 2)):
        p = Problem([40, 90, 129], [200, 33, 129], hq, hkv, d, True, seed=11, spare=70, lead=3)
        ref, lse_ref, _ = p.reference()
        O, lse = p.forward()
        g = p.backward(O, lse)
        dirty = Problem([40, 90, 129], [200, 33, 129], hq, hkv, d, True, seed=11, spare=70, lead=3)
        bad = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda").to(BF)
        for t, lo, hi in ((dirty.Q, 43, 133), (dirty.dO, 43, 133), (dirty.K, 203, 236), (dirty.V, 203, 236)):
            n = t.shape[0]
            where = torch.cat([torch.arange(3), torch.arange(lo, hi), torch.arange(n - 70, n)]).cuda()
            t[where] = bad[torch.arange(where.numel(), device="cuda") % 3][:, None, None]
        O2, lse2 = dirty.forward()
        g2 = dirty.backward(O2, lse2)
        for a, b, lo, hi in ((O, O2, 43, 133), (lse, lse2, 43, 133), (g[0], g2[0], 43, 133), (g[1], g2[1], 203, 236),
                             (g[2], g2[2], 203, 236)):
            keep = torch.ones(a.shape[0], dtype=torch.bool, device="cuda")
            keep[lo:hi] = False
            assert torch.equal(a[keep], b[keep])
        # tokens in no sequence are left as they were
        for t in (O, lse, *g, O2, lse2, *g2):
            assert (t[:3] == 7).all() and (t[-70:] == 7).all()


def test_equal_sequences_without_offsets():
    p = Problem([96] * 3, [130] * 3, 4, 2, 64, True, seed=2)
    O, lse = p.forward()
    O2, lse2 = torch.empty_like(O), torch.empty_like(lse)
    q.qlora_attention_fwd(p.Q, p.K, p.V, O2, lse2, batch=3, causal=True)
    assert torch.equal(O, O2) and torch.equal(lse, lse2)
    g = p.backward(O, lse)
    g2 = [torch.empty_like(t) for t in g]
    q.qlora_attention_bwd(p.Q, p.K, p.V, O, p.dO, lse, *g2, batch=3, causal=True)
    assert all(torch.equal(a, b) for a, b in zip(g, g2))
    # lse is not required
    O3 = torch.empty_like(O)
    q.qlora_attention_fwd(p.Q, p.K, p.V, O3, batch=3, causal=True)
    assert torch.equal(O, O3)


def test_parts_of_wider_matrices():
    # q, k and v as columns of one projection's output, and their gradients as columns of another
    hq, hkv, d, n = 4, 2, 64, 150
    p = Problem([n], [n], hq, hkv, d, True, seed=8)
    O, lse = p.forward()
    g = p.backward(O, lse)
    wide = torch.full((n, (hq + 2 * hkv) * d + 8), 3.0, dtype=BF, device="cuda")
    grad = torch.full_like(wide, 5.0)
    cut = lambda m, a, h: m[:, a * d:(a + h) * d].unflatten(1, (h, d))  # noqa: E731
    views = [(cut(m, 0, hq), cut(m, hq, hkv), cut(m, hq + hkv, hkv)) for m in (wide, grad)]
    for v, t in zip(views[0], (p.Q, p.K, p.V)):
        v.copy_(t)
    Ow = torch.full((n, hq * d + 16), 9.0, dtype=BF, device="cuda")
    dOw = torch.zeros_like(Ow)
    cut(dOw, 0, hq).copy_(p.dO)
    lse2 = torch.empty_like(lse)
    q.qlora_attention_fwd(*views[0], cut(Ow, 0, hq), lse2, causal=True)
    q.qlora_attention_bwd(*views[0], cut(Ow, 0, hq), cut(dOw, 0, hq), lse2, *views[1], causal=True)
    q.qlora_check_device_error()
    assert torch.equal(cut(Ow, 0, hq), O) and torch.equal(lse2, lse)
    assert all(torch.equal(a, b) for a, b in zip(views[1], g))
    assert (Ow[:, hq * d:] == 9).all() and (grad[:, -8:] == 5).all() and (wide[:, -8:] == 3).all()


def test_no_tokens_on_one_side():
    p = Problem([5], [0], 2, 1, 64)
    O, lse = p.forward()
    assert (O == 0).all() and (lse == -math.inf).all()
    dQ, dK, dV = p.backward(O, lse)
    assert (dQ == 0).all()
    p = Problem([0], [5], 2, 1, 64)
    O, lse = p.forward()
    dQ, dK, dV = p.backward(O, lse)
    assert (dK == 0).all() and (dV == 0).all()


def test_bad_offsets_are_clamped():
    # offsets outside the tensors, or descending ones: no access outside, the error word stays clean
    p = Problem([40, 40], [40, 40], 2, 2, 64, True, seed=4)
    for cu in ([-5, 40, 1 << 30], [0, 90, 20], [1 << 30, -1, 7]):
        t = torch.tensor(cu, dtype=torch.int32, device="cuda")
        O, lse = torch.zeros_like(p.Q), torch.zeros(80, 2, device="cuda")
        q.qlora_attention_fwd(p.Q, p.K, p.V, O, lse, causal=True, cu_q=t, cu_k=t)
        g = [torch.zeros_like(x) for x in (p.Q, p.K, p.V)]
        q.qlora_attention_bwd(p.Q, p.K, p.V, O, p.dO, lse, *g, causal=True, cu_q=t, cu_k=t)
        q.qlora_check_device_error()


def test_captured_replayed_and_on_another_stream():
    p = Problem([200, 77], [200, 77], 4, 2, 128, True, seed=9)
    O, lse = p.forward()
    want = [O, lse, *p.backward(O, lse)]
    got = [torch.zeros_like(t) for t in want]
    ws = torch.empty(q.qlora_attention_bwd_workspace_bytes(277, 4), dtype=torch.uint8, device="cuda")

    def step(stream=None):
        q.qlora_attention_fwd(p.Q, p.K, p.V, got[0], got[1], **p.how, stream=stream)
        q.qlora_attention_bwd(p.Q, p.K, p.V, got[0], p.dO, got[1], *got[2:], **p.how, ws=ws, stream=stream)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    step(s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    q.qlora_check_device_error()


def test_reference_gradients_match_differences():
    # the formulas that the tests above use, against central differences of softmax attention in 64 bits
    p = Problem([6, 4], [6, 9], 2, 1, 8, True, 3, seed=1)
    ref, _, _ = p.reference()

    def loss():
        return float((p.reference(False)[0]["O"][0] * p.dO.double()).sum())

    for name, key in (("Q", "dQ"), ("K", "dK"), ("V", "dV")):
        base = getattr(p, name).double()
        step = 1e-5 * torch.randn(base.shape, dtype=torch.float64, device="cuda")
        setattr(p, name, base + step)
        up = loss()
        setattr(p, name, base - step)
        down = loss()
        setattr(p, name, base)
        want = float((ref[key][0] * step).sum())
        assert abs((up - down) / 2 - want) <= 1e-6 * float((ref[key][0].abs() * step.abs()).sum()), name


# --------------------------------------------- few rows: work shared evenly, cut tiles joined --
@pytest.mark.parametrize("q_lens,k_lens,hq,hkv,d", [
    ([1], [20000], 1, 1, 128),                       # one tile, cut into more pieces than the joining threads' groups
    ([1], [9000], 6, 2, 40),
    ([1] * 5, [12000, 1, 64, 65, 513], 4, 1, 72),    # most blocks on one sequence, the short ones whole
    ([100], [3000], 2, 2, 128),                      # tiles of many rows, cut
    ([60, 3, 0, 90], [700, 2500, 90, 91], 4, 2, 64),
    ([1] * 70, [1 + (i * 211) % 900 for i in range(70)], 8, 4, 64),    # more sequences than a warp reads at once
    ([2] * 40 + [75], [300] * 40 + [75], 2, 1, 64),  # one sequence of many tiles among short ones
    ([i % 2 for i in range(1300)], [(i * 37) % 70 for i in range(1299)] + [3000], 1, 1, 8),    # 41 sequences a lane
    ([0, 0, 1, 0], [500, 0, 0, 70], 2, 1, 64),       # the one row sees nothing
])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 400)])
def test_few_rows(q_lens, k_lens, hq, hkv, d, causal, window):
    check(Problem(q_lens, k_lens, hq, hkv, d, causal, window, seed=len(q_lens)), grads=False)


def test_few_rows_without_offsets():
    p = Problem([2] * 3, [1500] * 3, 4, 2, 64, True, seed=2)
    O, lse = p.forward()
    O2, lse2 = torch.empty_like(O), torch.empty_like(lse)
    q.qlora_attention_fwd(p.Q, p.K, p.V, O2, lse2, batch=3, causal=True)
    assert torch.equal(O, O2) and torch.equal(lse, lse2)


def test_few_rows_with_values_outside():
    # a cache with room behind its last key, and a neighbour's keys, that hold anything
    args = ([1, 1, 3], [2000, 700, 1100], 8, 2, 128, True)
    p, dirty = Problem(*args, seed=4, spare=100), Problem(*args, seed=4, spare=100)
    bad = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda").to(BF)
    for t in (dirty.K, dirty.V):
        for lo, hi in ((2000, 2700), (3800, 3900)):
            t[lo:hi] = bad[torch.arange(t[lo:hi].numel(), device="cuda") % 3].view_as(t[lo:hi])
    (O, lse), (O2, lse2) = p.forward(), dirty.forward()
    keep = [0, 2, 3, 4]
    assert torch.equal(O[keep], O2[keep]) and torch.equal(lse[keep], lse2[keep])
    assert (O2[5:] == 7).all() and (lse2[5:] == 7).all()


@pytest.mark.parametrize("n,k", [(1, 3000), (1, 30), (300, 300)])
def test_not_a_number_is_not_hidden(n, k):
    # inputs of a sequence that are not finite are outside the promise; what they give is not a plausible number
    p = Problem([n], [k], 40, 40, 64, False, seed=6)
    p.K[k // 2, 1] = float("nan")
    O, lse = p.forward()
    assert O[:, 1].isnan().all() and lse[:, 1].isnan().all()
    assert O[:, 0].isfinite().all() and lse[:, 2:].isfinite().all()


def test_few_rows_on_two_streams_and_replayed():
    ps = [Problem([1] * 4, [3000, 900, 1, 250], 8, 2, 128, True, seed=s) for s in (1, 2)]
    want = [p.forward() for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    got = [tuple(torch.zeros_like(t) for t in w) for w in want]

    def run(i, **kw):
        q.qlora_attention_fwd(ps[i].Q, ps[i].K, ps[i].V, *got[i], **ps[i].how, **kw)

    torch.cuda.synchronize()
    for _ in range(20):                              # each call has a workspace of its own
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                run(i)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for w, g in zip(want, got) for a, b in zip(w, g))
    graphs = [torch.cuda.CUDAGraph() for _ in ps]
    for i, graph in enumerate(graphs):
        with torch.cuda.graph(graph):
            run(i)
    for g in got:
        for t in g:
            t.zero_()
    torch.cuda.synchronize()
    for s, graph in zip(streams, graphs):
        with torch.cuda.stream(s):
            graph.replay()
            graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for w, g in zip(want, got) for a, b in zip(w, g))
    q.qlora_check_device_error()


def test_few_rows_with_a_given_workspace():
    p = Problem([1] * 3, [2000, 100, 700], 4, 1, 128, True, seed=3)
    O, lse = p.forward()
    need = int(q.lib().qlora_attention_fwd_workspace_bytes(q._attention(p.Q, p.K, p.V, O, lse, None, True, 0, None,
                                                                       p.cu_q, p.cu_k)))
    assert need > 0
    ws = torch.full((need + 256,), 0xAB, dtype=torch.uint8, device="cuda")
    O2, lse2 = torch.zeros_like(O), torch.zeros_like(lse)
    q.qlora_attention_fwd(p.Q, p.K, p.V, O2, lse2, **p.how, ws=ws[:need])
    assert torch.equal(O, O2) and torch.equal(lse, lse2)
    assert (ws[need:] == 0xAB).all()
    with pytest.raises(q.QloraError):
        q.qlora_attention_fwd(p.Q, p.K, p.V, O2, lse2, **p.how, ws=ws[:need - 16])


def test_a_cache_beyond_32_bits():
    # 2.2e9 elements of keys and as many of values; the second sequence lies behind the 2^31st
    n, tail, heads, d = 270000, 300, 64, 128
    p = Problem([2], [tail], heads, heads, d, True, seed=12)
    ref, lse_ref, lse_tol = p.reference()
    K, V = (torch.zeros(n + tail, heads, d, dtype=BF, device="cuda") for _ in range(2))
    K[n:], V[n:] = p.K, p.V
    assert K[n].data_ptr() - K.data_ptr() > 1 << 32
    Q, dO = torch.cat((p.Q[:1], p.Q)), torch.cat((torch.zeros_like(p.dO[:1]), p.dO))
    how = dict(causal=True, cu_q=torch.tensor([0, 1, 3], dtype=torch.int32, device="cuda"),
               cu_k=torch.tensor([0, n, n + tail], dtype=torch.int32, device="cuda"))
    O, lse = torch.full_like(Q, 7.0), torch.full((3, heads), 7.0, device="cuda")
    q.qlora_attention_fwd(Q, K, V, O, lse, **how)
    q.qlora_check_device_error()
    close(O[1:], ref["O"], "O")
    assert ((lse[1:].double() - lse_ref).abs() <= lse_tol).all()
    # the first one's keys and values are zero: every probability is 1 / n, a sum of n ones in 32 bits and its logarithm
    assert (O[0] == 0).all() and ((lse[0] - math.log(n)).abs() <= 2.0 ** -18 * (1 + math.log(n))).all()
    g = [torch.full_like(t, 7.0) for t in (Q, K, V)]
    q.qlora_attention_bwd(Q, K, V, O, dO, lse, *g, **how)
    q.qlora_check_device_error()
    close(g[0][1:], ref["dQ"], "dQ")
    close(g[1][n:], ref["dK"], "dK")
    close(g[2][n:], ref["dV"], "dV")
    assert (g[0][0] == 0).all() and not g[1][:n].any() and not g[2][:n].any()


# ------------------------------------------- rows enough for two tiles per block on every SM --
def takes_two_tiles(p):
    tokens, n, most = p.Q.shape[0], len(p.q_lens), 128 // (p.hq // p.hkv)
    tiles = min(tokens, tokens // (2 * most) + n)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return -(-tokens // n) * (p.hq // p.hkv) > 128 and tiles * p.hkv >= sms


@pytest.mark.parametrize("hq,hkv,d", [(40, 40, 128), (40, 40, 64), (36, 12, 128), (40, 40, 24), (64, 16, 80)])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 1), (True, 100), (True, 1000)])
def test_many_rows(hq, hkv, d, causal, window):
    # none, one and many tokens; fewer keys than queries, and more; a last tile of one row
    p = Problem([300, 1, 700, 129, 0, 513], [300, 64, 650, 400, 9, 513], hq, hkv, d, causal, window, seed=hq + window)
    assert takes_two_tiles(p)
    check(p, grads=False)


@pytest.mark.parametrize("n", [257, 512, 640])
def test_many_rows_of_equal_sequences(n):
    p = Problem([n] * 2, [n] * 2, 50, 50, 128, True, seed=n)
    assert takes_two_tiles(p)
    O, lse = p.forward()
    ref, lse_ref, lse_tol = p.reference(False)
    close(O, ref["O"], "O")
    assert ((lse.double() - lse_ref).abs() <= lse_tol).all()
    O2, lse2 = torch.empty_like(O), torch.empty_like(lse)
    q.qlora_attention_fwd(p.Q, p.K, p.V, O2, lse2, batch=2, causal=True)
    assert torch.equal(O, O2) and torch.equal(lse, lse2)


def test_many_rows_with_values_outside():
    args = ([300, 400, 260], [300, 410, 260], 48, 24, 64, True)
    p, dirty = Problem(*args, seed=4, spare=90, lead=5), Problem(*args, seed=4, spare=90, lead=5)
    assert takes_two_tiles(p)
    bad = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda").to(BF)
    for t, spots in ((dirty.Q, ((0, 5), (305, 705), (965, 1055))), (dirty.K, ((0, 5), (305, 715), (975, 1065))),
                     (dirty.V, ((0, 5), (305, 715), (975, 1065)))):
        for lo, hi in spots:
            t[lo:hi] = bad[torch.arange(t[lo:hi].numel(), device="cuda") % 3].view_as(t[lo:hi])
    (O, lse), (O2, lse2) = p.forward(), dirty.forward()
    for at in (slice(5, 305), slice(705, 965)):
        assert torch.equal(O[at], O2[at]) and torch.equal(lse[at], lse2[at])
    for at in (slice(0, 5), slice(965, 1055)):
        assert (O2[at] == 7).all() and (lse2[at] == 7).all()


def test_many_rows_do_not_hide_what_is_not_a_number_and_grow():
    # a reference maximum that is raised tile after tile, and keys that are not finite
    p = Problem([600], [600], 60, 60, 64, False, seed=8, scale=0.05)
    assert takes_two_tiles(p)
    p.K *= (1 + torch.arange(600, device="cuda") // 64)[:, None, None].to(BF)
    ref, lse_ref, _ = p.reference(False)
    O, lse = p.forward()
    # 64 * 2^-24 of sum |q| |k| scale (below 2^7 here) is 2^-11 in the exponent
    assert ((O.double() - ref["O"][0]).abs() <= ref["O"][1] + 2.0 ** -11 * ref["O"][1] / H).all()
    assert float((lse.double() - lse_ref).abs().max()) <= 2.0 ** -11 + 2.0 ** -14
    p.K[300, 1] = float("nan")
    O, lse = p.forward()
    assert O[:, 1].isnan().all() and lse[:, 1].isnan().all() and O[:, 2:].isfinite().all()


@pytest.mark.parametrize("hq,hkv,d", [(40, 40, 128), (36, 12, 128), (40, 40, 64), (64, 16, 80)])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 100)])
def test_many_tiles_backward(hq, hkv, d, causal, window):
    # several tiles of each kernel for every block, empty ones among them
    check(Problem([300, 1, 700, 129, 0, 513], [300, 64, 650, 400, 9, 513], hq, hkv, d, causal, window, seed=d + window))


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("causal", [False, True])
def test_backward_does_not_hide_what_is_not_a_number(d, causal):
    # one query at a time, at neighbouring places of a step, has a lse (then a Q) that is not a number: nothing that its
    # probabilities enter is a plausible number, and no other head or key notices
    n = 40
    for i in (0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 31, 32, 39):
        p = Problem([n], [n], 2, 2, d, causal, seed=7)
        O, lse = p.forward()
        lse[i, 1] = float("nan")
        dQ, dK, dV = p.backward(O, lse)
        seen = i + 1 if causal else n
        assert dQ[i, 1].isnan().all(), i
        for name, t in (("dK", dK), ("dV", dV)):
            assert t[:seen, 1].isnan().all(), (name, i)
            assert t[seen:, 1].isfinite().all() and t[:, 0].isfinite().all(), (name, i)
        rest = [j for j in range(n) if j != i]
        assert dQ[rest, 1].isfinite().all() and dQ[:, 0].isfinite().all()
    p = Problem([n], [n], 2, 2, d, causal, seed=7)
    p.Q[8, 0] = float("nan")
    dQ, dK, dV = p.backward(*p.forward())
    for t in (dQ[8:9], dK[:9 if causal else n], dV[:9 if causal else n]):
        assert t[:, 0].isnan().all() and t[:, 1].isfinite().all()


@pytest.mark.parametrize("causal", [True, False])
def test_many_empty_sequences(causal):
    # 200 samples among 40,000 sequences, nearly all of them empty: the grids' bounds count a tile more for each
    n, each, hq, hkv, d = 40000, 100, 64, 64, 8
    ends = torch.arange(0, n, n // 200)
    lens = torch.zeros(n, dtype=torch.int64)
    lens[ends] = each
    cu = torch.zeros(n + 1, dtype=torch.int32)
    cu[1:] = lens.cumsum(0)
    p = Problem([each] * 200, [each] * 200, hq, hkv, d, causal, seed=14)
    want = [*p.forward()]
    want += p.backward(*want)
    p.how = dict(p.how, cu_q=cu.cuda(), cu_k=cu.cuda())
    got = p.backward(*want[:2])
    assert all(torch.equal(a, b) for a, b in zip(want[2:], got))
    # the forward's tiles follow the mean length here, so its steps may differ: one and the same bound holds
    ref = p.forward()
    assert float((ref[0].double() - want[0].double()).norm()) <= 2 * H * float(want[0].double().norm())
    # and all of them behind the last sample, or before the first
    for where in (slice(0, 200), slice(n - 200, n)):
        lens.zero_()
        lens[where] = each
        cu[1:] = lens.cumsum(0)
        p.how = dict(p.how, cu_q=cu.cuda(), cu_k=cu.cuda())
        g = p.backward(*want[:2])
        assert all(torch.equal(a, b) for a, b in zip(want[2:], g))


def test_a_tile_that_takes_seconds():
    # backward: one sequence whose keys meet 290 million rows of queries (2.25 million steps of one tile), short ones behind
    # it. The warp that hands out tiles is two ahead and has to wait for the long one's end. Queries are zero, so that the
    # probabilities are 1 / keys, and only a few gradients are not.
    nq, nk, more, heads, d = 4_500_000, 128, 600, 64, 8
    tq, tk = nq + more, nk + more
    g = torch.Generator(device="cuda")
    g.manual_seed(15)
    Q, O = (torch.zeros(tq, heads, d, dtype=BF, device="cuda") for _ in range(2))
    K, V = (torch.randn(tk, 1, d, generator=g, device="cuda").to(BF) for _ in range(2))
    lse = torch.zeros(tq, heads, device="cuda")
    lse[:nq] = math.log(nk)
    dO = torch.zeros_like(Q)
    dO[nq - 3:] = torch.randn(more + 3, heads, d, generator=g, device="cuda").to(BF)
    ends = torch.arange(more + 1, dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    how = dict(cu_q=torch.cat((zero, nq + ends)), cu_k=torch.cat((zero, nk + ends)))
    dK, dV = torch.full_like(K, 7.0), torch.full_like(V, 7.0)
    dQ = torch.full_like(Q, 7.0)
    q.qlora_attention_bwd(Q, K, V, O, dO, lse, dQ, dK, dV, **how)
    q.qlora_check_device_error()
    f = dO[nq - 3:].double()
    # P is 1/128 and 1 up to the 32-bit exponential, its bf16 rounding exact: dV is a sum of dO's, rounded once
    for at, of, n in ((slice(0, nk), f[:3].flatten(0, 1), nk), (slice(nk, tk), f[3:], 1)):
        want = of.sum(0).expand(nk, d) / n if n > 1 else of.sum(1)
        size = of.abs().sum(0).expand(nk, d) / n if n > 1 else of.abs().sum(1)
        assert ((dV[at, 0].double() - want).abs() <= H * want.abs() + (H + F) * size).all()
    assert (dK == 0).all()
    # dS = P dO V^T with delta 0; dQ = scale dS K
    for at, of, keys in ((slice(nq - 3, nq), f[:3], slice(0, nk)), (slice(nq, tq), f[3:], None)):
        Kf, Vf = K[:, 0].double(), V[:, 0].double()
        if keys is not None:
            dS, E, Kk = of @ Vf[keys].T / nk, of.abs() @ Vf[keys].abs().T / nk, Kf[keys]
            want, size = dS @ Kk, E @ Kk.abs()
        else:
            dS, E = (of * Vf[nk:, None]).sum(-1, keepdim=True), (of * Vf[nk:, None]).abs().sum(-1, keepdim=True)
            want, size = dS * Kf[nk:, None], E * Kf[nk:, None].abs()
        c = d ** -0.5
        assert ((dQ[at].double() - c * want).abs() <= H * c * want.abs() + (H + F) * c * size).all()
    assert not dQ[:nq - 3].any()


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (4, 4, 64)])
@pytest.mark.parametrize("new", [1, 3])
def test_a_cache_with_room_behind_its_keys(hq, hkv, d, new):
    # the layout that the header names: every slot two sequences, its keys and the room behind them, which holds NaN
    slots, capacity = 5, 700
    lens = [300, 3, 700, 64, 129]
    p = Problem([x for _ in range(slots) for x in (new, 0)], [x for n in lens for x in (n, capacity - n)], hq, hkv, d, True,
                seed=21)
    for s, n in enumerate(lens):
        for t in (p.K, p.V):
            t[s * capacity + n:(s + 1) * capacity] = float("nan")
    check(p)
    if new == 1:        # the offsets as the README makes them
        starts = torch.arange(slots, device="cuda") * capacity
        cu_k = torch.stack((starts, starts + torch.tensor(lens, device="cuda")), 1).flatten()
        cu_k = torch.cat((cu_k, cu_k.new_tensor([slots * capacity]))).int()
        cu_q = (torch.arange(2 * slots + 1, device="cuda") + 1).div(2, rounding_mode="floor").int()
        assert torch.equal(cu_q, p.cu_q) and torch.equal(cu_k, p.cu_k)


@pytest.mark.parametrize("q_lens,k_lens,hq,hkv,d,window", [
    ([1] * 63 + [2048], [100 + 40 * i for i in range(63)] + [2048], 4, 4, 64, 0),     # a prompt among single new tokens
    ([2048] + [1] * 63, [2500] + [700] * 63, 8, 2, 128, 300),
    ([1, 5] * 8, [900] * 16, 8, 2, 128, 0),                                           # one and five new tokens in turn
    ([2] * 20 + [1000] + [0] * 30, [64] * 20 + [1000] + [5] * 30, 2, 1, 64, 0),
])
def test_prompts_among_new_tokens(q_lens, k_lens, hq, hkv, d, window):
    check(Problem(q_lens, k_lens, hq, hkv, d, True, window, seed=len(q_lens)))
