"""Norms around the residual add against the formulas in 64 bits.

Bounds. A row's sums have positive or mixed terms, at most 64 roundings deep: 2^-18 of the sum of sizes; a value made
of a few such factors and terms is within 2^-16 of the sum of its terms' sizes. bf16 outputs add half a step, 2^-8 of
the value. Weight gradients add at most 56 rows per block and 8 runs of 19 blocks in 32 bits: again below 2^-16 of the
sum of the terms' sizes.
"""
import pytest
import torch

import bit_nf4_quantized_03_b200 as q
from tests.gpu_util import ensure_built

pytestmark = pytest.mark.gpu
EPS, SCALE = 1e-5, 0.37
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


class Case:
    def __init__(self, m, cols, residual, post, gate, pre, dt, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.dt, self.shape = dt, (m, cols)
        x = rnd(m, cols) * 2
        x[:, ::97] *= 30
        self.x = x.to(dt)
        self.y = rnd(m, cols).to(torch.bfloat16) if residual else None
        self.w_post = 1 + 0.3 * rnd(cols) if post else None
        self.gate = 0.5 + 0.3 * rnd(cols) if gate else None
        self.w_pre = 1 + 0.3 * rnd(cols) if pre else None
        self.dr = rnd(m, cols).to(dt)
        self.dh = rnd(m, cols).to(torch.bfloat16) if pre else None

    def vectors(self):
        return self.w_post, self.gate, self.w_pre


def _d(t):
    return None if t is None else t.double()


def _fwd_ref(c):
    """r and h in 64 bits, each with the sum of its terms' sizes."""
    x, y, wp, g, w = _d(c.x), _d(c.y), _d(c.w_post), _d(c.gate), _d(c.w_pre)
    r, size = x, x.abs()
    if y is not None:
        t = y if wp is None else y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * wp
        t = SCALE * (t if g is None else t * g)
        r, size = x + t, size + t.abs()
    if w is None:
        return r, size, None, None
    rho = torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS)
    return r, size, r * rho * w, size * rho * w.abs()


def _bwd_ref(c, r, dr):
    """Gradients from the formulas in 64 bits and the sizes of their terms: {name: (value, size)}."""
    r, y, wp, g, w, dh = _d(r), _d(c.y), _d(c.w_post), _d(c.gate), _d(c.w_pre), _d(c.dh)
    d = torch.zeros_like(r) if dr is None else _d(dr)
    size = d.abs()
    out = {}
    if w is not None:
        rho = torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS)
        u = dh * w
        d = d + rho * u - r * rho ** 3 * (u * r).mean(-1, keepdim=True)
        size = size + rho * u.abs() + r.abs() * rho ** 3 * (u * r).abs().mean(-1, keepdim=True)
        out["dw_pre"] = ((dh * r * rho).sum(0), (dh * r * rho).abs().sum(0))
    out["dx"] = (d, size)
    if y is not None:
        e, es = SCALE * d, SCALE * size
        eta = torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) if wp is not None else 1.0
        t = y if wp is None else y * eta * wp
        if g is not None:
            out["dgate"] = ((e * t).sum(0), (es * t.abs()).sum(0))
            e, es = e * g, es * g.abs()
        if wp is not None:
            out["dw_post"] = ((e * y * eta).sum(0), (es * y.abs() * eta).sum(0))
            e, es = e * wp, es * wp.abs()
            es = eta * es + y.abs() * eta ** 3 * (es * y.abs()).mean(-1, keepdim=True)
            e = eta * e - y * eta ** 3 * (e * y).mean(-1, keepdim=True)
        out["dy"] = (e, es)
    return out


def _close(got, ref, size, name):
    assert torch.isfinite(got).all(), name
    d = (got.double() - ref).abs()
    allow = ref.abs() * HALF[got.dtype] + size * 2.0 ** -16 + 1e-37
    assert (d <= allow).all(), (name, float((d / allow).max()))


def _run_fwd(c, store_r=True):
    r = torch.empty(c.shape, dtype=c.dt, device="cuda") if c.y is not None and store_r else None
    h = torch.empty(c.shape, dtype=torch.bfloat16, device="cuda") if c.w_pre is not None else None
    q.qlora_norm_residual_fwd(c.x, c.y, *c.vectors(), r, h, scale=SCALE, eps=EPS)
    q.qlora_check_device_error()
    return r, h


def _run_bwd(c, r, dr, weights=True, flags=0, start=None):
    new = lambda t: None if t is None or not weights else (torch.empty_like(t) if start is None else torch.full_like(t, start))  # noqa: E731
    dx = torch.empty(c.shape, dtype=c.dt, device="cuda")
    dy = torch.empty(c.shape, dtype=torch.bfloat16, device="cuda") if c.y is not None else None
    dw = [new(t) for t in c.vectors()]
    q.qlora_norm_residual_bwd(dr, c.dh, r, c.y, *c.vectors(), dx, dy, *dw, scale=SCALE, eps=EPS, flags=flags)
    q.qlora_check_device_error()
    return {"dx": dx, "dy": dy, "dw_post": dw[0], "dgate": dw[1], "dw_pre": dw[2]}


KINDS = [(True, True, True, True), (True, False, False, True), (True, True, False, True), (True, False, True, False),
         (False, False, False, True)]
SHAPES = [(1, 8), (3, 64), (5, 328), (300, 1416), (7, 4096), (2, 4104), (311, 8192), (4, 8200), (3, 16384)]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m,cols", SHAPES)
def test_norm_forward_and_backward(m, cols, kind, dt):
    c = Case(m, cols, *kind, dt, seed=m + cols)
    r, h = _run_fwd(c)
    rr, rs, hr, hs = _fwd_ref(c)
    if r is not None:
        _close(r, rr, rs, "r")
    if h is not None:
        _close(h, hr, hs, "h")
    saved = c.x if r is None else r
    for dr in (c.dr, None) if c.w_pre is not None else (c.dr,):
        got = _run_bwd(c, saved, dr)
        for name, (ref, size) in _bwd_ref(c, saved, dr).items():
            _close(got[name], ref, size, name)
        again = _run_bwd(c, saved, dr)
        frozen = _run_bwd(c, saved, dr, weights=False)
        for name, t in got.items():
            assert t is None or torch.equal(t, again[name]), name
        # without weight gradients the row sums may be split over the threads in another way: another order of the same
        # 32-bit terms, so the same bounds, not the same bits
        for name in ("dx", "dy"):
            if frozen[name] is not None:
                ref, size = _bwd_ref(c, saved, dr)[name]
                _close(frozen[name], ref, size, name)


def test_norm_gradients_match_differences():
    # the formulas above against central differences of the forward's definition, in 64 bits
    c = Case(3, 40, True, True, True, True, torch.float32, seed=9)
    r0 = _fwd_ref(c)[0]
    grads = _bwd_ref(c, r0, c.dr)

    def loss():
        r, _, h, _ = _fwd_ref(c)
        return float((r * c.dr.double()).sum() + (h * c.dh.double()).sum())

    for name, key in (("x", "dx"), ("y", "dy"), ("w_post", "dw_post"), ("gate", "dgate"), ("w_pre", "dw_pre")):
        base = getattr(c, name).double()
        step = torch.randn(base.shape, device="cuda", dtype=torch.float64) * 1e-4
        setattr(c, name, base + step)
        up = loss()
        setattr(c, name, base - step)
        down = loss()
        setattr(c, name, base)
        want = float((grads[key][0] * step).sum())
        # third-order term: the step is 1e-4 of values of order one
        assert abs((up - down) / 2 - want) <= 1e-5 * float((grads[key][1] * step.abs()).sum()), name


def test_norm_accumulates_and_works_in_place():
    c = Case(130, 512, True, True, True, True, torch.bfloat16, seed=4)
    r, h = _run_fwd(c)
    got = _run_bwd(c, r, c.dr)
    more = _run_bwd(c, r, c.dr, flags=q.QLORA_BWD_ACCUMULATE_GRADS, start=2.0)
    for name in ("dw_post", "dgate", "dw_pre"):
        # the sum starts from 2: one more rounding of a value of that size
        assert ((more[name] - got[name] - 2.0).abs() <= 2.0 ** -22 * (got[name].abs() + 2.0)).all()
    x, y = c.x.clone(), c.y.clone()
    q.qlora_norm_residual_fwd(x, y, *c.vectors(), x, y, scale=SCALE, eps=EPS)
    assert torch.equal(x, r) and torch.equal(y, h)
    dr, dh = c.dr.clone(), c.dh.clone()
    q.qlora_norm_residual_bwd(dr, dh, r, c.y, *c.vectors(), dr, dh, scale=SCALE, eps=EPS)
    assert torch.equal(dr, got["dx"]) and torch.equal(dh, got["dy"])
    # the sum formed but not stored gives the same norm
    assert torch.equal(_run_fwd(c, store_r=False)[1], h)


def test_norm_no_rows_and_zero_rows_of_values():
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w, dw = torch.ones(64, device="cuda"), torch.full((64,), 7.0, device="cuda")
    q.qlora_norm_residual_fwd(e, None, None, None, w, None, e)
    q.qlora_norm_residual_bwd(None, e, e, None, None, None, w, e, dw_pre=dw, flags=q.QLORA_BWD_ACCUMULATE_GRADS)
    assert (dw == 7).all()
    q.qlora_norm_residual_bwd(None, e, e, None, None, None, w, e, dw_pre=dw)
    assert (dw == 0).all()
    # a row of zeros: rho = 1 / sqrt(eps), everything finite
    c = Case(2, 64, True, True, False, True, torch.float32)
    c.x.zero_()
    c.y.zero_()
    r, h = _run_fwd(c)
    assert (r == 0).all() and (h == 0).all()
    for t in _run_bwd(c, r, c.dr).values():
        assert t is None or torch.isfinite(t).all()
    q.qlora_check_device_error()


def test_norm_captured_and_replayed_on_another_stream():
    c = Case(50, 4096, True, False, False, True, torch.bfloat16, seed=6)
    r, h = torch.empty_like(c.x), torch.empty_like(c.y)
    dx, dw = torch.empty_like(c.x), torch.empty_like(c.w_pre)
    ws = torch.empty(q.qlora_norm_residual_workspace_bytes(50, 4096), dtype=torch.uint8, device="cuda")

    def step():
        q.qlora_norm_residual_fwd(c.x, c.y, None, None, c.w_pre, r, h, scale=SCALE, eps=EPS)
        q.qlora_norm_residual_bwd(c.dr, c.dh, r, c.y, None, None, c.w_pre, dx, dw_pre=dw, scale=SCALE, eps=EPS, ws=ws)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (r, h, dx, dw)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (r, h, dx, dw):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (r, h, dx, dw)))
    q.qlora_check_device_error()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m,cols", [(2500, 8), (1300, 328), (2100, 4096), (1000, 6144), (950, 8192), (640, 12288), (500, 16384)])
def test_norm_many_rows(m, cols, kind, dt):
    # several rows for every group of threads, in rings of one to four rows
    test_norm_forward_and_backward(m, cols, kind, dt)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,cols", [(2100, 4096), (950, 8192), (500, 16384)])
def test_norm_many_rows_in_place(m, cols, dt):
    # r over x, h over y, dx over dr and dy over dh, while the next rows are on their way; and what may be left out
    c = Case(m, cols, True, True, True, True, dt, seed=cols)
    r, h = _run_fwd(c)
    x, y = c.x.clone(), c.y.clone()
    q.qlora_norm_residual_fwd(x, y, *c.vectors(), x, y, scale=SCALE, eps=EPS)
    assert torch.equal(x, r) and torch.equal(y, h)
    for weights in (True, False):
        got = _run_bwd(c, r, c.dr, weights)
        dr, dh = c.dr.clone(), c.dh.clone()
        dw = [torch.empty_like(t) if weights else None for t in c.vectors()]
        q.qlora_norm_residual_bwd(dr, dh, r, c.y, *c.vectors(), dr, dh, *dw, scale=SCALE, eps=EPS)
        assert torch.equal(dr, got["dx"]) and torch.equal(dh, got["dy"])
        assert not weights or all(torch.equal(a, got[n]) for a, n in zip(dw, ("dw_post", "dgate", "dw_pre")))
        # no dy, and one weight gradient of three
        dx, dg = torch.empty_like(r), torch.empty_like(c.gate) if weights else None
        q.qlora_norm_residual_bwd(c.dr, c.dh, r, c.y, *c.vectors(), dx, None, None, dg, scale=SCALE, eps=EPS)
        assert torch.equal(dx, got["dx"]) and (not weights or torch.equal(dg, got["dgate"]))
    q.qlora_check_device_error()
