"""Rotary positions against the definition in 64 bits.

Bound per element: half a bf16 step of the value (2^-8 of it), and for the 32-bit part 2^-20 of the pair's size times
the magnitude: the angle's remainder is rounded once (2^-24 of at most one turn, 2^-21.3 rad), sine and cosine and the
two products and their sum add a few 2^-24 each.
"""
import math

import pytest
import torch

import bit_nf4_quantized_03_b200 as q
from tests.gpu_util import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _table(rot):
    return torch.tensor([rot.turns[i] for i in range(rot.rot_dim // 2)], dtype=torch.float64, device="cuda")


def _ref(rot, pos, x, transpose=False):
    """(value, size of the pair) of the turned x in 64 bits."""
    a = pos.double()[:, None] * _table(rot) * (2 * math.pi) * (-1 if transpose else 1)
    c, s = (rot.magnitude * a.cos())[:, None], (rot.magnitude * a.sin())[:, None]
    y, size = x.double().clone(), x.double().abs() * 0
    n = rot.rot_dim
    u, v = (slice(0, n // 2), slice(n // 2, n)) if rot.layout == q.QLORA_ROTARY_HALF else (slice(0, n, 2), slice(1, n, 2))
    xd = x.double()
    y[..., u] = xd[..., u] * c - xd[..., v] * s
    y[..., v] = xd[..., v] * c + xd[..., u] * s
    size[..., u] = size[..., v] = (xd[..., u].abs() + xd[..., v].abs()) * rot.magnitude
    return y, size


def _close(got, ref, size):
    d = (got.double() - ref).abs()
    allow = ref.abs() * 2.0 ** -8 + size * 2.0 ** -20 + 1e-38
    assert torch.isfinite(got).all()
    assert (d <= allow).all(), float((d / allow).max())


def _bf(*shape, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot", [(8, 8), (64, 64), (128, 128), (128, 64), (80, 24), (96, 80), (128, 40), (256, 256), (256, 16)])
@pytest.mark.parametrize("m,hq,hk", [(1, 1, 0), (3, 5, 2), (257, 8, 8)])
def test_rotary_matches_definition(layout, d, rot, m, hq, hk):
    r = q.qlora_rotary_init(d, rot, layout, magnitude=1.1)
    pos = torch.randint(0, 1 << 17, (m,), device="cuda", dtype=torch.int32)
    x = _bf(m, hq, d)
    k = _bf(m, hk, d, seed=1) if hk else None
    for transpose in (False, True):
        y, ky = torch.empty_like(x), (None if k is None else torch.empty_like(k))
        q.qlora_rotary_apply(r, pos, x, y, k, ky, transpose=transpose)
        q.qlora_check_device_error()
        _close(y, *_ref(r, pos, x, transpose))
        assert torch.equal(y[..., rot:], x[..., rot:])
        if k is not None:
            _close(ky, *_ref(r, pos, k, transpose))
        # in place: the same bits
        x2, k2 = x.clone(), (None if k is None else k.clone())
        q.qlora_rotary_apply(r, pos, x2, k=k2, transpose=transpose)
        assert torch.equal(x2, y) and (k is None or torch.equal(k2, ky))


@pytest.mark.parametrize("scaling,kw", [("linear", dict(factor=4.0)),
                                        ("bands", dict(factor=8.0, low=1.0, high=4.0, original_length=8192.0)),
                                        ("yarn", dict(factor=4.0, low=1.0, high=32.0, original_length=4096.0, magnitude=1.14))])
def test_rotary_scaled_at_far_positions(scaling, kw):
    # any int32 position: the far ends, and one step next to them
    pos = torch.tensor([0, 1, 131071, (1 << 31) - 1, (1 << 31) - 2, -1, -(1 << 31)], device="cuda", dtype=torch.int32)
    r = q.qlora_rotary_init(128, 128, base=500000.0, scaling=scaling, **kw)
    x = _bf(7, 4, 128)
    y, _ = q.qlora_rotary_apply(r, pos, x, torch.empty_like(x))
    q.qlora_check_device_error()
    _close(y, *_ref(r, pos, x))


def test_rotary_strided_parts_of_one_matrix():
    # q and k as columns of one [m, (hq + 2 hk) d] projection, turned in place; v beside them is left alone
    m, hq, hk, d = 37, 6, 2, 64
    qkv = _bf(m, (hq + 2 * hk) * d)
    before = qkv.clone()
    qv = qkv[:, :hq * d].view(m, hq, d)
    kv = qkv[:, hq * d:(hq + hk) * d].view(m, hk, d)
    pos = torch.arange(m, device="cuda", dtype=torch.int32)
    r = q.qlora_rotary_init(d, d)
    q.qlora_rotary_apply(r, pos, qv, k=kv)
    q.qlora_check_device_error()
    _close(qv, *_ref(r, pos, before[:, :hq * d].view(m, hq, d)))
    _close(kv, *_ref(r, pos, before[:, hq * d:(hq + hk) * d].view(m, hk, d)))
    assert torch.equal(qkv[:, (hq + hk) * d:], before[:, (hq + hk) * d:])
    with pytest.raises(ValueError):
        q.qlora_rotary_apply(r, pos, qv.transpose(0, 1)[:, :m].contiguous().transpose(0, 1))


def test_rotary_transpose_is_the_gradient():
    # <g, R x> = <R^T g, x>, and a difference quotient of it along x (R is linear, so the quotient is exact in 64 bits)
    r = q.qlora_rotary_init(64, 48, "interleaved", magnitude=0.9)
    pos = torch.tensor([5, 70000], device="cuda", dtype=torch.int32)
    x, g = _bf(2, 3, 64), _bf(2, 3, 64, seed=2)
    gx, _ = q.qlora_rotary_apply(r, pos, g, torch.empty_like(g), transpose=True)
    step = _bf(2, 3, 64, seed=3).double()
    change = ((_ref(r, pos, x.double() + step)[0] - _ref(r, pos, x.double() - step)[0]) / 2 * g.double()).sum()
    # each of the 384 products carries half a bf16 step of gx
    allow = float((gx.double().abs() * step.abs()).sum()) * 2.0 ** -7
    assert abs(float(change - (gx.double() * step).sum())) <= allow


def test_rotary_empty_and_other_stream():
    r = q.qlora_rotary_init(64)
    x = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    q.qlora_rotary_apply(r, torch.empty(0, dtype=torch.int32, device="cuda"), x)
    x, pos = _bf(16, 2, 64), torch.arange(16, device="cuda", dtype=torch.int32)
    want, _ = q.qlora_rotary_apply(r, pos, x, torch.empty_like(x))
    got = torch.empty_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    q.qlora_rotary_apply(r, pos, x, got, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
    q.qlora_check_device_error()


def heads_per_thread(m, hq, hk, d, rot, in_place):
    """The run of heads that a thread takes, by the launch's rule."""
    pairs = 8 if rot % 16 == 0 else 4
    groups = rot // (2 * pairs) + (0 if in_place else -(-(d - rot) // 16))
    blocks = -(-m // (256 // groups))
    want = torch.cuda.get_device_properties(0).multi_processor_count // 3
    run = 8
    while run > 1 and blocks * (-(-hq // run) + -(-hk // run)) < want:
        run //= 2
    return run


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot", [(128, 128), (128, 64), (128, 40), (96, 80), (80, 24), (256, 128)])
@pytest.mark.parametrize("m,hq,hk", [(2100, 28, 1), (2100, 13, 5), (2100, 32, 32), (2051, 9, 0)])
def test_rotary_of_many_tokens(layout, d, rot, m, hq, hk):
    # threads with runs of eight heads, in two batches of four: whole runs, runs of one to five heads, heads of q and of k
    assert heads_per_thread(m, hq, hk, d, rot, False) == 8 == heads_per_thread(m, hq, hk, d, rot, True)
    r = q.qlora_rotary_init(d, rot, layout, magnitude=0.8)
    g = torch.Generator(device="cuda")
    g.manual_seed(m + hq)
    pos = torch.randint(-5, 1 << 17, (m,), generator=g, device="cuda", dtype=torch.int32)
    # eight elements of other things between the tokens, which stay
    wide = _bf(m, hq * d + 8, seed=4)
    x = wide[:, :hq * d].view(m, hq, d)
    k = _bf(m, hk, d, seed=1) if hk else None
    for transpose in (False, True):
        out = torch.full_like(wide, 3.0)
        y, ky = out[:, :hq * d].view(m, hq, d), (None if k is None else torch.empty_like(k))
        q.qlora_rotary_apply(r, pos, x, y, k, ky, transpose=transpose)
        q.qlora_check_device_error()
        assert (out[:, hq * d:] == 3).all()
        for got, of in ((y, x), (ky, k)):
            if of is not None:
                _close(got, *_ref(r, pos, of, transpose))
                assert torch.equal(got[..., rot:], of[..., rot:])
        x2, k2 = wide.clone()[:, :hq * d].view(m, hq, d), (None if k is None else k.clone())
        q.qlora_rotary_apply(r, pos, x2, k=k2, transpose=transpose)
        assert torch.equal(x2, y) and (k is None or torch.equal(k2, ky))


@pytest.mark.parametrize("m,hq,hk,run", [(150, 28, 1, 2), (260, 28, 1, 4), (40, 13, 5, 1)])
def test_rotary_of_runs_in_between(m, hq, hk, run):
    assert heads_per_thread(m, hq, hk, 128, 128, True) == run
    r = q.qlora_rotary_init(128)
    pos = torch.arange(m, device="cuda", dtype=torch.int32)
    x, k = _bf(m, hq, 128), _bf(m, hk, 128, seed=1)
    y, ky = torch.empty_like(x), torch.empty_like(k)
    q.qlora_rotary_apply(r, pos, x, y, k, ky)
    _close(y, *_ref(r, pos, x))
    _close(ky, *_ref(r, pos, k))
    q.qlora_check_device_error()
