"""The operators of a decoder layer in a row, as a training step and a generation step use them: residual norms, NF4
linear layers with adapters, rotary embedding, attention, SiLU gate; forward and backward against autograd through the
formulas in 64 bits on the dequantized weights.

Bounds. Every operator rounds its outputs to bf16 (2^-8 of a value at most) and works in 32 bits inside; the linear
layers' weights are bf16 values on both sides. A step's forward has 12 such outputs in a row (h, q, turned q, P, O, o, h,
gate, s, down, r, h), its backward as many again (dS among them), each an error of at most 2^-8 of its tensor's norm.
Roundings are independent, so the errors' squares add up: behind n of them a tensor is off by at most sqrt(n) 2^-8 of its
norm where the maps between keep relative errors. Norms and residual additions do, products with random matrices enlarge
signal and error alike, and the logits are below 1, so that the softmax's slopes are too; differences (dP - delta, the
norms' backward) leave down to a quarter of what enters them, errors do not cancel: four times that is allowed. A
missing term, a wrong sign or a wrong turn moves a tensor by more than half its norm."""
import pytest
import torch

import bit_nf4_quantized_03_b200 as q
from bit_nf4_quantized_03_b200 import synth
from tests.gpu_util import ensure_built, gpu_quantize

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
HALF = 2.0 ** -8
D, HQ, HKV, HD, FF, R, ALPHA, WINDOW = 256, 8, 2, 32, 384, 16, 16.0, 90
SCALE = 0.02                                            # of the logits: below 1 here


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


class Linear:
    def __init__(self, n, k, layer):
        self.n, self.k = n, k
        self.qw = gpu_quantize(synth.weight(n, k, layer=layer), q.QLORA_SCALE_DQ_FP8)
        self.A, self.B = (t.cuda() for t in synth.lora_pair(R, k, n, layer=layer))
        W = torch.empty(n, k, dtype=BF, device="cuda")
        q.qlora_nf4_dequantize(self.qw, W)
        self.W = W.double()
        self.ref = [t.double().requires_grad_() for t in (self.A, self.B)]

    def fwd(self, X):
        m = X.shape[0]
        self.X, self.U = X, torch.empty(m, R, device="cuda")
        Y = torch.empty(m, self.n, dtype=BF, device="cuda")
        self.ws = torch.empty(q.qlora_linear_workspace_bytes(m, self.n, self.k, R), dtype=torch.uint8, device="cuda")
        return q.qlora_linear_fwd(self.qw, X, self.A, self.B, R, ALPHA, Y, q.QLORA_DTYPE_BF16, self.U, self.ws)

    def bwd(self, dY, dX=None):
        """Gradient of the input, added to dX if that is given."""
        flags = 0 if dX is None else q.QLORA_BWD_ACCUMULATE_DX
        dX = torch.empty_like(self.X) if dX is None else dX
        self.dA, self.dB = torch.empty(R, self.k, device="cuda"), torch.empty(self.n, R, device="cuda")
        q.qlora_linear_bwd(self.qw, self.X, dY, self.A, self.B, R, ALPHA, self.U, dX, q.QLORA_DTYPE_BF16, self.dA,
                           self.dB, flags, self.ws)
        return dX

    def plain(self, x):
        return x @ self.W.T + ALPHA / R * (x @ self.ref[0].T) @ self.ref[1].T


class Layer:
    def __init__(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.near_one = lambda n: 1 + 0.2 * torch.randn(n, generator=g, device="cuda")
        self.q, self.k, self.v = (Linear(h * HD, D, 10 * seed + i) for i, h in enumerate((HQ, HKV, HKV)))
        self.o, self.gate, self.up = (Linear(*s, 10 * seed + 3 + i) for i, s in enumerate(((D, HQ * HD), (FF, D), (FF, D))))
        self.down = Linear(D, FF, 10 * seed + 6)
        self.w1, self.w2, self.w3, self.post, self.res = (self.near_one(D) for _ in range(5))
        self.ref = {n: getattr(self, n).double().requires_grad_() for n in ("w1", "w2", "w3", "post", "res")}
        self.rot = q.qlora_rotary_init(HD, base=10000.0)

    # ------------------------------------------------------------------ the framework's operators
    def forward(self, x, pos, cu, cache=None, cu_k=None):
        """cache: (K, V, rows): keys and values are put there, and all of the cache's are read."""
        m = x.shape[0]
        new = lambda *s: torch.empty(*s, dtype=BF, device="cuda")  # noqa: E731
        self.x, self.pos, self.cu = x, pos, cu
        _, h = q.qlora_norm_residual_fwd(x, None, None, None, self.w1, None, new(m, D))
        Q, K, V = (f.fwd(h).view(m, -1, HD) for f in (self.q, self.k, self.v))
        self.Q, self.K, self.V = new(m, HQ, HD), new(m, HKV, HD), V
        q.qlora_rotary_apply(self.rot, pos, Q, self.Q, K, self.K)
        self.O, self.lse = new(m, HQ, HD), torch.empty(m, HQ, device="cuda")
        keys, values = self.K, self.V
        if cache is not None:
            cache[0][cache[2]], cache[1][cache[2]] = self.K, self.V
            keys, values = cache[:2]
        self.how = dict(causal=True, window=WINDOW, scale=SCALE, cu_q=cu, cu_k=cu if cu_k is None else cu_k)
        q.qlora_attention_fwd(self.Q, keys, values, self.O, self.lse, **self.how)
        self.a = self.o.fwd(self.O.view(m, -1))
        # a norm behind the block and a weighted residual, as some models have them
        self.r, h = q.qlora_norm_residual_fwd(x, self.a, self.post, self.res, self.w2, new(m, D), new(m, D))
        self.g, self.u = self.gate.fwd(h), self.up.fwd(h)
        self.s = new(m, FF)
        q.qlora_silu_gate_fwd(self.g, self.u, self.s)
        self.f = self.down.fwd(self.s)
        self.r2, self.h3 = q.qlora_norm_residual_fwd(self.r, self.f, None, None, self.w3, new(m, D), new(m, D))
        return self.r2, self.h3

    def backward(self, dr2, dh3):
        new = torch.empty_like
        vec = lambda: torch.empty(D, device="cuda")  # noqa: E731
        self.d = {n: vec() for n in self.ref}
        dr, df = new(self.r), new(self.f)
        q.qlora_norm_residual_bwd(dr2, dh3, self.r2, self.f, None, None, self.w3, dr, df, dw_pre=self.d["w3"])
        ds, dg, du = self.down.bwd(df), new(self.g), new(self.u)
        q.qlora_silu_gate_bwd(ds, self.g, self.u, dg, du)
        dh = self.up.bwd(du, self.gate.bwd(dg))
        dx, da = new(self.x), new(self.a)
        q.qlora_norm_residual_bwd(dr, dh, self.r, self.a, self.post, self.res, self.w2, dx, da, self.d["post"],
                                  self.d["res"], self.d["w2"])
        dO = self.o.bwd(da).view_as(self.O)
        dQ, dK, dV = new(self.Q), new(self.K), new(self.V)
        q.qlora_attention_bwd(self.Q, self.K, self.V, self.O, dO, self.lse, dQ, dK, dV, **self.how)
        q.qlora_rotary_apply(self.rot, self.pos, dQ, dQ, dK, dK, transpose=True)
        dh = self.v.bwd(dV.flatten(1), self.k.bwd(dK.flatten(1), self.q.bwd(dQ.flatten(1))))
        out = new(self.x)
        q.qlora_norm_residual_bwd(dx, dh, self.x, None, None, None, self.w1, out, dw_pre=self.d["w1"])
        return out

    # ------------------------------------------------------------------ the formulas
    def plain(self, x, pos, lens):
        p = self.ref
        rms = lambda t, w: t / (t.square().mean(-1, keepdim=True) + 1e-5).sqrt() * w  # noqa: E731
        m = x.shape[0]
        h = rms(x, p["w1"])
        Q, K, V = (f.plain(h).view(m, -1, HD) for f in (self.q, self.k, self.v))
        angle = pos.double()[:, None] * 10000.0 ** (-torch.arange(0, HD, 2, device="cuda", dtype=torch.float64) / HD)
        c, s = angle.cos()[:, None], angle.sin()[:, None]

        def turn(t):
            a, b = t.chunk(2, -1)
            return torch.cat((a * c - b * s, b * c + a * s), -1)

        Q, K = turn(Q), turn(K).repeat_interleave(HQ // HKV, 1)
        V = V.repeat_interleave(HQ // HKV, 1)
        outs, at = [], 0
        for n in lens:
            sl = slice(at, at + n)
            S = torch.einsum("ihd,jhd->hij", Q[sl], K[sl]) * SCALE
            i = torch.arange(n, device="cuda")
            ok = (i[None] <= i[:, None]) & (i[None] > i[:, None] - WINDOW)
            outs.append(torch.einsum("hij,jhd->ihd", S.masked_fill(~ok, -float("inf")).softmax(-1), V[sl]))
            at += n
        a = self.o.plain(torch.cat(outs).flatten(1))
        r = x + p["res"] * rms(a, p["post"])
        h = rms(r, p["w2"])
        f = self.down.plain(torch.nn.functional.silu(self.gate.plain(h)) * self.up.plain(h))
        r2 = r + f
        return r2, rms(r2, p["w3"])


def off(got, ref, roundings, name):
    rel = float((got.double() - ref.detach()).norm() / ref.detach().norm())
    assert torch.isfinite(got).all() and rel <= 4 * roundings ** 0.5 * HALF, (name, rel, 4 * roundings ** 0.5 * HALF)


LENS = [130, 1, 64, 77, 28]


def _inputs(m, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(m, D, generator=g, device="cuda").to(BF) for _ in range(3)]


def _offsets(lens):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")


def test_training_step_of_two_layers():
    layers = [Layer(1), Layer(2)]
    m = sum(LENS)
    x, dr, dh = _inputs(m, 3)
    pos = torch.cat([torch.arange(n, device="cuda", dtype=torch.int32) for n in LENS])
    cu = _offsets(LENS)
    r1, _ = layers[0].forward(x, pos, cu)
    r2, h2 = layers[1].forward(r1, pos, cu)
    dmid = layers[1].backward(dr, dh)
    dx = layers[0].backward(dmid, torch.zeros_like(dh))
    q.qlora_check_device_error()
    xr = x.double().requires_grad_()
    p1, _ = layers[0].plain(xr, pos, LENS)
    p2, ph2 = layers[1].plain(p1, pos, LENS)
    ((p2 * dr.double()).sum() + (ph2 * dh.double()).sum()).backward()
    off(r2, p2, 24, "r")
    off(h2, ph2, 24, "h")
    off(dx, xr.grad, 48, "dx")
    for i, layer in enumerate(layers):
        for n in layer.ref:
            if i == 0 and n == "w3":                    # its norm's output is not used
                assert (layer.d[n] == 0).all()
                continue
            off(layer.d[n], layer.ref[n].grad, 48, (i, n))
        for n in ("q", "k", "v", "o", "gate", "up", "down"):
            f = getattr(layer, n)
            off(f.dA, f.ref[0].grad, 48, (i, n, "A"))
            off(f.dB, f.ref[1].grad, 48, (i, n, "B"))


def test_generation_step_continues_a_prefill():
    # the tokens one at a time against a cache give what the whole sequences give, and the same again from a graph
    layer, m = Layer(4), sum(LENS)
    x = _inputs(m, 5)[0]
    pos = torch.cat([torch.arange(n, device="cuda", dtype=torch.int32) for n in LENS])
    cu, b = _offsets(LENS), len(LENS)
    want, want_h = (t.clone() for t in layer.forward(x, pos, cu))
    K, V = layer.K.clone(), layer.V.clone()
    last = cu[1:].long() - 1
    K[last], V[last] = float("nan"), float("nan")       # the step brings these itself
    step = torch.arange(b + 1, dtype=torch.int32, device="cuda")
    xs, ps = x[last].clone(), pos[last].clone()
    run = lambda: layer.forward(xs, ps, step, cache=(K, V, last), cu_k=cu)  # noqa: E731
    r, h = run()
    q.qlora_check_device_error()
    ref, ref_h = layer.plain(x.double(), pos, LENS)
    off(r, ref[last], 12, "r")
    off(h, ref_h[last], 12, "h")
    off(want, ref, 12, "whole r")
    off(want_h, ref_h, 12, "whole h")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r2, h2 = run()
    for t in (r2, h2):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(r, r2) and torch.equal(h, h2)
    q.qlora_check_device_error()


def test_workspaces_belong_to_the_stream_of_their_call(monkeypatch):
    # the calls that allocate one, on the default stream by its address, on a side stream by its address and as an object
    side = torch.cuda.Stream()
    x = torch.randn(40, 2, 64, device="cuda").to(BF)
    lse = torch.zeros(40, 2, device="cuda")
    keys = torch.randn(3000, 2, 64, device="cuda").to(BF)
    g = [torch.empty_like(x) for _ in range(3)]
    rows, w = torch.randn(40, 128, device="cuda").to(BF), torch.ones(128, device="cuda")
    O, dx, dw = torch.empty_like(x), torch.empty_like(rows), torch.empty_like(w)
    O1 = torch.empty_like(x[:1])
    seen, empty = [], torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: (seen.append(torch.cuda.current_stream().cuda_stream), empty(*a, **k))[1])
    for stream, at in ((None, 0), (0, 0), (torch.cuda.default_stream(), 0), (side.cuda_stream, side.cuda_stream),
                       (side, side.cuda_stream)):
        side.wait_stream(torch.cuda.current_stream())
        seen.clear()
        q.qlora_attention_fwd(x, x, x, O, lse, causal=True, stream=stream)
        q.qlora_attention_bwd(x, x, x, O, x, lse, *g, causal=True, stream=stream)
        q.qlora_attention_fwd(x[:1], keys, keys, O1, stream=stream)
        q.qlora_norm_residual_bwd(None, rows, rows, None, None, None, w, dx, dw_pre=dw, stream=stream)
        assert seen == [at] * 3, stream
        torch.cuda.synchronize()
    q.qlora_check_device_error()
