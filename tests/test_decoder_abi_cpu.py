"""Host-only checks of the decoder-layer operators (no GPU): the rotary table against its definition, and every
refusal, before anything is launched. Addresses are made up: a call that is refused reads none of them."""
import ctypes
import math

import pytest
import torch

import bit_nf4_quantized_03_b200 as q

P = [1 << (20 + i) for i in range(20)]


@pytest.fixture(scope="module")
def L():
    from bit_nf4_quantized_03_b200 import build
    build.build()
    return q.lib()


# ------------------------------------------------------------------ rotary --
@pytest.mark.parametrize("rot,base", [(8, 10000.0), (128, 10000.0), (80, 500000.0), (256, 1e6)])
def test_rotary_table_unscaled_and_linear(L, rot, base):
    plain = q.qlora_rotary_init(256, rot, base=base)
    slow = q.qlora_rotary_init(256, rot, "interleaved", base, "linear", factor=4.0)
    for i in range(rot // 2):
        want = math.exp(-2.0 * i / rot * math.log(base)) / (2 * math.pi)
        assert plain.turns[i] == pytest.approx(want, rel=1e-13)
        assert slow.turns[i] == pytest.approx(want / 4.0, rel=1e-13)
    assert all(plain.turns[i] == 0.0 for i in range(rot // 2, 128))


def test_rotary_table_bands_and_yarn(L):
    d, base, n, factor = 128, 10000.0, 8192.0, 8.0
    bands = q.qlora_rotary_init(d, d, base=base, scaling="bands", factor=factor, low=1.0, high=4.0, original_length=n)
    yarn = q.qlora_rotary_init(d, d, base=base, scaling="yarn", factor=factor, low=1.0, high=32.0, original_length=n,
                               magnitude=1.2)
    assert yarn.magnitude == pytest.approx(1.2)
    first = math.floor(d * math.log(n / (32 * 2 * math.pi)) / (2 * math.log(base)))
    last = math.ceil(d * math.log(n / (1 * 2 * math.pi)) / (2 * math.log(base)))
    seen = set()
    for i in range(d // 2):
        f = base ** (-2 * i / d)
        wave = 2 * math.pi / f
        if wave <= n / 4.0:
            want, kind = f, "kept"
        elif wave >= n / 1.0:
            want, kind = f / factor, "scaled"
        else:
            k = (n / wave - 1.0) / 3.0
            want, kind = f * k + f / factor * (1 - k), "between"
        seen.add(kind)
        assert bands.turns[i] == pytest.approx(want / (2 * math.pi), rel=1e-12)
        ramp = min(1.0, max(0.0, (i - first) / (last - first)))
        assert yarn.turns[i] == pytest.approx((f / factor * ramp + f * (1 - ramp)) / (2 * math.pi), rel=1e-12)
    assert seen == {"kept", "scaled", "between"}


def test_rotary_init_refusals(L):
    ok = dict(head_dim=128, rot_dim=64, layout=0, scaling=0, base=1e4, factor=1.0, low=1.0, high=4.0,
              original_length=8192.0, magnitude=1.0)
    rot = q.Rotary()

    def call(**kw):
        a = {**ok, **kw}
        cfg = q.RotaryConfig(*[a[f] for f, _ in q.RotaryConfig._fields_])
        return L.qlora_rotary_init(ctypes.byref(cfg), ctypes.byref(rot))

    assert call() == 0
    assert L.qlora_rotary_init(None, ctypes.byref(rot)) == 1
    for bad in (dict(layout=2), dict(scaling=4), dict(scaling=-1), dict(rot_dim=136), dict(rot_dim=0), dict(head_dim=0),
                dict(base=1.0), dict(base=float("inf")), dict(base=float("nan")), dict(magnitude=float("nan")),
                dict(scaling=1, factor=0.0), dict(scaling=1, factor=float("nan")), dict(scaling=2, low=0.0),
                dict(scaling=2, low=4.0), dict(scaling=3, original_length=0.0), dict(scaling=3, high=float("inf"))):
        assert call(**bad) == 1, bad
    for bad in (dict(rot_dim=12), dict(head_dim=132, rot_dim=64), dict(head_dim=264)):
        assert call(**bad) == 2, bad
    with pytest.raises(ValueError):
        q.qlora_rotary_init(128, layout="spiral")
    with pytest.raises(ValueError):
        q.qlora_rotary_init(128, scaling="more")


def test_rotary_apply_refusals(L):
    rot = q.qlora_rotary_init(128, 64)

    def call(r=rot, pos=P[0], m=4, x=P[1], ldx=512, hq=4, y=P[2], ldy=512, k=P[3], ldk=256, hk=2, ky=P[4], ldky=256):
        return L.qlora_rotary_apply(None if r is None else ctypes.byref(r), pos, m, x, ldx, hq, y, ldy, k, ldk, hk, ky,
                                    ldky, 0, None)

    assert call(m=0) == 0
    assert call(m=0, x=None, y=None, pos=None, k=None, hk=0) == 0
    for bad in (dict(r=None), dict(r=q.Rotary()), dict(m=-1), dict(hq=0), dict(hk=0), dict(k=None), dict(pos=None),
                dict(pos=P[0] | 2), dict(x=None), dict(x=P[1] | 8), dict(y=None), dict(ky=None), dict(k=P[3] | 4),
                dict(ldx=504), dict(ldy=8), dict(ldk=248), dict(ldky=0), dict(y=P[1], ldy=520)):
        assert call(**bad) == 1, bad
    for bad in (dict(ldx=513), dict(ldy=516), dict(ldk=260), dict(ldky=257), dict(m=1 << 31),
                dict(hq=40000, ldx=40000 * 128, ldy=40000 * 128)):
        assert call(**bad) == 2, bad


# -------------------------------------------------------------------- norm --
def test_norm_fwd_refusals(L):
    def call(n=(4, 64, 0, 1e-5, 1.0), x=P[0], y=P[1], wp=P[2], g=P[3], w=P[4], r=P[5], h=P[6]):
        s = None if n is None else ctypes.byref(q.Norm(*n))
        return L.qlora_norm_residual_fwd(s, x, y, wp, g, w, r, h, None)

    assert call(n=(0, 64, 0, 1e-5, 1.0)) == 0
    for bad in (dict(n=None), dict(n=(-1, 64, 0, 1e-5, 1.0)), dict(n=(4, 0, 0, 1e-5, 1.0)), dict(n=(4, 64, 2, 1e-5, 1.0)),
                dict(n=(4, 64, 0, -1.0, 1.0)), dict(n=(4, 64, 0, float("nan"), 1.0)),
                dict(n=(4, 64, 0, 1e-5, float("inf"))), dict(x=None), dict(w=None), dict(h=None),
                dict(w=None, h=None, r=None), dict(y=None), dict(y=None, wp=None, g=None), dict(x=P[0] | 8),
                dict(h=P[6] | 2), dict(g=P[3] | 4)):
        assert call(**bad) == 1, bad
    for bad in (dict(n=(4, 60, 0, 1e-5, 1.0)), dict(n=(4, 16392, 0, 1e-5, 1.0)), dict(n=(1 << 31, 64, 0, 1e-5, 1.0))):
        assert call(**bad) == 2, bad


def test_norm_bwd_refusals(L):
    need = q.qlora_norm_residual_workspace_bytes(4, 64)
    assert need == 4 * 2 * 64 * 4          # two column sums per row's block
    assert q.qlora_norm_residual_workspace_bytes(0, 64) == 0
    assert q.qlora_norm_residual_workspace_bytes(4, 60) == 0

    def call(n=(4, 64, 1, 1e-5, 1.0), dr=P[0], dh=P[1], r=P[2], y=P[3], wp=P[4], g=P[5], w=P[6], dx=P[7], dy=P[8],
             dwp=P[9], dg=P[10], dw=P[11], flags=0, ws=P[12], ws_bytes=need):
        s = None if n is None else ctypes.byref(q.Norm(*n))
        return L.qlora_norm_residual_bwd(s, dr, dh, r, y, wp, g, w, dx, dy, dwp, dg, dw, flags, ws, ws_bytes, None)

    assert call(n=(0, 64, 1, 1e-5, 1.0), dwp=None, dg=None, dw=None) == 0
    assert call(n=(0, 64, 1, 1e-5, 1.0), flags=1) == 0
    for bad in (dict(n=None), dict(flags=2), dict(flags=4), dict(dr=None, dh=None, w=None, dw=None), dict(dh=None),
                dict(w=None), dict(w=None, dh=None), dict(wp=None), dict(g=None), dict(y=None), dict(r=None),
                dict(dx=None), dict(dx=P[7] | 4), dict(dw=P[11] | 8),
                dict(y=None, wp=None, g=None, dwp=None, dg=None)):
        assert call(**bad) == 1, bad
    assert call(n=(4, 68, 1, 1e-5, 1.0)) == 2
    for bad in (dict(ws=None), dict(ws=P[12] | 8), dict(ws_bytes=need - 1)):
        assert call(**bad) == 4, bad


def test_binding_refuses_cpu_tensors_and_wrong_shapes(L):
    rot = q.qlora_rotary_init(64)
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        q.qlora_rotary_apply(rot, torch.zeros(3, dtype=torch.int32), x)
    with pytest.raises(ValueError):
        q.qlora_rotary_apply(rot, torch.zeros(3, dtype=torch.int32), torch.zeros(3, 2, 128, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        q.qlora_norm_residual_fwd(torch.zeros(3, 64), None, None, None, torch.ones(64), None, None)
    with pytest.raises(ValueError):
        q.qlora_norm_residual_fwd(torch.zeros(3, 64, dtype=torch.float16), None, None, None, None, None, None)


class _Fake:
    """A tensor as far as the device check looks at it."""

    def __init__(self, index):
        self.index = index

    def get_device(self):
        return self.index


def test_calls_run_on_the_device_of_their_tensors(monkeypatch):
    now, seen = [0], []

    class On:
        def __init__(self, i):
            self.i = i

        def __enter__(self):
            self.before, now[0] = now[0], self.i

        def __exit__(self, *exc):
            now[0] = self.before

    class Lib:
        @staticmethod
        def entry(*args):
            seen.append((now[0], args))
            return args[0]

        @staticmethod
        def qlora_status_string(status):
            return b"refused"

    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", On)
    monkeypatch.setattr(q, "lib", lambda: Lib)
    monkeypatch.setattr(q, "_raw_stream", lambda i: 1000 + i)
    assert q._device(_Fake(3), None, _Fake(3)) == 3
    q._run("entry", 3, (0, 7), None)                 # another device than the current one: its stream, and back
    q._run("entry", 0, (0, 7), None)
    q._run("entry", 0, (0, 7), 55)
    assert seen == [(3, (0, 7, 1003)), (0, (0, 7, 1000)), (0, (0, 7, 55))] and now[0] == 0
    with pytest.raises(q.QloraError):
        q._run("entry", 3, (0 + 2, 7), None)
    assert now[0] == 0
    with pytest.raises(ValueError):
        q._device(_Fake(0), _Fake(1))
    with pytest.raises(ValueError):
        q._device(_Fake(0), _Fake(-1))               # a CPU tensor


def test_a_workspace_is_allocated_on_the_stream_of_its_call(monkeypatch):
    # memory from another stream's pool could be handed out again there while the call still runs
    now, seen = ["current"], []

    class On:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            self.before, now[0] = now[0], self.s

        def __exit__(self, *exc):
            now[0] = self.before

    empty = torch.empty
    monkeypatch.setattr(torch.cuda, "stream", On)
    # as torch has it: address 0 is no stream of anybody's, so a new one is made
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda at, device=None: f"external {at}" if at else "new")
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    monkeypatch.setattr(torch, "empty", lambda *a, **k: (seen.append(now[0]), empty(*a, **k))[1])
    like = torch.zeros(1)
    for stream in (None, 0, 77, "side"):
        ws, n = q._workspace(None, 64, like, stream)
        assert n == 64 and ws.numel() == 64
    assert seen == ["current", "default", "external 77", "side"]
    assert q._workspace(None, 0, like, 0) == (None, 0) and q._workspace(ws, 64, like, 0)[0] is ws
    assert len(seen) == 4


# --------------------------------------------------------------- attention --
def _attn(**kw):
    a = dict(batch=2, heads_q=4, heads_kv=2, head_dim=64, causal=1, window=0, scale=0.125, reserved=0, tokens_q=8,
             tokens_k=10, ld_q=256, ld_k=128, ld_v=128, ld_o=256, cu_q=P[10], cu_k=P[11])
    a.update(kw)
    return q.Attention(*[a[f] for f, _ in q.Attention._fields_])


_BAD_ATTENTION = (dict(batch=0), dict(heads_q=0), dict(heads_kv=0), dict(heads_q=5, ld_q=320, ld_o=320), dict(head_dim=0),
                  dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
                  dict(window=-1), dict(window=4, causal=0), dict(cu_q=None), dict(cu_k=None),
                  dict(cu_q=P[10] | 2), dict(tokens_q=-1), dict(tokens_k=-1), dict(ld_q=248), dict(ld_k=120),
                  dict(ld_v=0), dict(ld_o=255), dict(cu_q=None, cu_k=None, tokens_q=9))
_UNSUPPORTED_ATTENTION = (dict(head_dim=60, ld_q=256), dict(head_dim=136, ld_q=544, ld_k=272, ld_v=272, ld_o=544),
                          dict(heads_q=130, heads_kv=2, ld_q=130 * 64, ld_o=130 * 64), dict(ld_q=257), dict(ld_k=132),
                          dict(ld_v=129), dict(ld_o=260), dict(tokens_q=(1 << 30) + 1), dict(tokens_k=(1 << 30) + 1),
                          dict(tokens_k=1 << 27), dict(ld_q=1 << 40))


def test_attention_fwd_refusals(L):
    def call(a=None, Q=P[0], K=P[1], V=P[2], O=P[3], lse=P[4]):
        return L.qlora_attention_fwd(ctypes.byref(_attn() if a is None else a), Q, K, V, O, lse, None, 0, None)

    assert L.qlora_attention_fwd(None, P[0], P[1], P[2], P[3], None, None, 0, None) == 1
    assert call(_attn(tokens_q=0), Q=None, O=None) == 0
    for bad in _BAD_ATTENTION:
        assert call(_attn(**bad)) == 1, bad
    for bad in _UNSUPPORTED_ATTENTION:
        assert call(_attn(**bad)) == 2, bad
    for bad in (dict(Q=None), dict(K=None), dict(V=None), dict(O=None), dict(Q=P[0] | 8), dict(K=P[1] | 2),
                dict(V=P[2] | 4), dict(O=P[3] | 8), dict(lse=P[4] | 4)):
        assert call(**bad) == 1, bad


def test_attention_fwd_workspace(L):
    def need(**kw):
        return L.qlora_attention_fwd_workspace_bytes(ctypes.byref(_attn(**kw)))

    # one row per key head and sequence, cut tiles' results of 592 places; longer rows take more, long sequences none
    few = dict(tokens_q=2, tokens_k=10000, cu_q=P[10])
    assert need(**few) == 2 * 296 * (2 * 64 + 2 * 2) * 4
    assert need(tokens_q=2, tokens_k=100) == 0 == need(tokens_q=0, tokens_k=10000)
    assert need(tokens_q=100, tokens_k=10000) == 2 * 296 * 100 * 66 * 4
    assert need(tokens_q=20000, tokens_k=20000) == 0
    assert need(head_dim=0) == 0 == need(tokens_k=-1) and L.qlora_attention_fwd_workspace_bytes(None) == 0
    n = need(**few)
    for ws, size in ((None, n), (None, 0), (P[9] | 8, n), (P[9], n - 1)):
        assert L.qlora_attention_fwd(ctypes.byref(_attn(**few)), P[0], P[1], P[2], P[3], P[4], ws, size, None) == 4


def test_attention_bwd_refusals(L):
    need = q.qlora_attention_bwd_workspace_bytes(8, 4)
    assert need == 8 * 4 * 4 + 16 and q.qlora_attention_bwd_workspace_bytes(-1, 4) == 0

    def call(a=None, Q=P[0], K=P[1], V=P[2], O=P[3], dO=P[4], lse=P[5], dQ=P[6], dK=P[7], dV=P[8], ws=P[9], n=need):
        return L.qlora_attention_bwd(ctypes.byref(_attn() if a is None else a), Q, K, V, O, dO, lse, dQ, dK, dV, ws, n,
                                     None)

    assert L.qlora_attention_bwd(None, *P[:10], need, None) == 1
    assert call(_attn(tokens_q=0, tokens_k=0), Q=None, K=None, V=None, O=None, dO=None, lse=None, dQ=None, dK=None,
                dV=None, ws=None, n=0) == 0
    for bad in _BAD_ATTENTION:
        assert call(_attn(**bad)) == 1, bad
    for bad in _UNSUPPORTED_ATTENTION:
        assert call(_attn(**bad)) == 2, bad
    for name in ("Q", "K", "V", "O", "dO", "lse", "dQ", "dK", "dV"):
        assert call(**{name: None}) == 1, name
        assert call(**{name: P[12] | 8}) == 1, name
    for bad in (dict(ws=None), dict(ws=P[9] | 8), dict(n=need - 1)):
        assert call(**bad) == 4, bad


def test_attention_binding_refusals(L):
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        q.qlora_attention_fwd(x, x, x, x)                                   # CPU tensors
    with pytest.raises(ValueError):
        q.qlora_attention_fwd(x.view(4, 128), x, x, x)
    with pytest.raises(ValueError):
        q.qlora_attention_bwd(x, x, x, x, x, None, x, x, x)


def test_attention_takes_a_million_sequences(L):
    # more are refused: some warps walk over them one by one while others wait, and that wait has a limit
    many = dict(tokens_q=0, tokens_k=0, heads_q=1, heads_kv=1, ld_q=64, ld_k=64, ld_v=64, ld_o=64)
    for batch, want in ((1 << 20, 0), ((1 << 20) + 1, 2)):
        a = ctypes.byref(_attn(batch=batch, **many))
        assert L.qlora_attention_fwd(a, None, None, None, None, None, None, 0, None) == want
        assert L.qlora_attention_bwd(a, *[None] * 10, 0, None) == want


def test_attention_bwd_counts_rows_of_a_key_head_in_32_bits(L):
    # the masks of a key are intervals of query rows (token * heads per key head): 2^31 of them do not fit
    wide = dict(heads_q=64, heads_kv=1, head_dim=8, ld_q=512, ld_o=512, ld_k=8, ld_v=8, tokens_k=8)
    most = ((1 << 31) - 1 - (128 << 6)) // 64
    for tokens, want in ((most, 1), (most + 1, 2), (1 << 26, 2)):
        a = ctypes.byref(_attn(tokens_q=tokens, **wide))
        assert L.qlora_attention_bwd(a, *[None] * 10, 0, None) == want, tokens         # 1: the pointers, looked at after
        assert L.qlora_attention_fwd(a, None, P[0], P[1], None, None, None, 0, None) == 1


def test_binding_refuses_what_does_not_fit_32_bits(L):
    # the low 32 bits of each of these are a valid value
    big, bf = 1 << 32, torch.bfloat16
    meta = lambda *s, t=bf: torch.empty(*s, dtype=t, device="meta")  # noqa: E731
    x = meta(4, 2, 64)
    for kw in (dict(window=big, causal=True), dict(window=big + 5, causal=True), dict(window=5 - big, causal=True),
               dict(batch=big + 1), dict(batch=1 - big)):
        with pytest.raises(ValueError, match="32 bits"):
            q.qlora_attention_fwd(x, x, x, x, **kw)
        with pytest.raises(ValueError, match="32 bits"):
            q.qlora_attention_bwd(x, x, x, x, x, meta(4, 2, t=torch.float32), x, x, x, **kw)
    for shape in ((1, 1, big + 64), (1, big + 2, 8)):
        with pytest.raises(ValueError, match="32 bits"):
            q.qlora_attention_fwd(*[meta(*shape)] * 4)
    with pytest.raises(ValueError, match="32 bits"):
        q.qlora_rotary_init(big + 64)
    with pytest.raises(ValueError, match="32 bits"):
        q.qlora_rotary_init(64, rot_dim=big + 64)
    with pytest.raises(ValueError, match="32 bits"):
        q.qlora_rotary_apply(q.qlora_rotary_init(8), meta(1, t=torch.int32), meta(1, big + 1, 8))
    wide, vec = meta(1, big + 64), meta(big + 64, t=torch.float32)
    with pytest.raises(ValueError, match="32 bits"):
        q.qlora_norm_residual_fwd(wide, None, None, None, vec, None, wide)
    with pytest.raises(ValueError, match="32 bits"):
        q.qlora_norm_residual_bwd(None, wide, wide, None, None, None, vec, wide)
    with pytest.raises(ValueError, match="32 bits"):
        q.qlora_norm_residual_bwd(None, x[0], x[0], None, None, None, meta(64, t=torch.float32), x[0], flags=big)
    with pytest.raises(ValueError, match="32 bits"):
        q.qlora_norm_residual_workspace_bytes(4, big + 64)
    with pytest.raises(ValueError, match="32 bits"):
        q.qlora_attention_bwd_workspace_bytes(4, big + 2)
