"""Host side of the cache-row, expansion, prefill and tree decode entry points
(argument checks before CUDA is touched, the binding's refusals) and pins of
their float64 oracles against independent computations."""
import ctypes
import math
import types

import numpy as np
import pytest
import torch

from mla_latent_kv_05_gb300 import _build, binding
from oracle import expanded, fp4_codec, fp8_codec, mla_oracle, row_codec
from tests.test_binding_cpu import FakeLib, FakeTensor

FORMATS = ["bf16", "fp8", "fp4", "fp8_v41", "fp4_v41"]
Z = ctypes.c_void_p(0)
F = ctypes.c_void_p(0x10000)
SCALE = ctypes.c_float(0.1)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return binding.load()


def off(n):
    return ctypes.c_void_p(0x10000 + n)


@pytest.mark.parametrize("fmt", FORMATS)
def test_row_entries_validate_on_the_host(lib, fmt):
    def app(c=F, cs=512, r=F, rs=64, cache=F, bt=F, sl=F, cu=F, b=2, n=3, pages=4, page=64, mp=2, ws=F, wsb=256):
        return getattr(lib, "mla_cache_append_" + fmt)(c, cs, r, rs, cache, bt, sl, cu, b, n, pages, page, mp, ws, wsb, Z)

    def gat(cache=F, bt=F, sl=F, cu=F, b=2, n=3, pages=4, page=64, mp=2, out=F, ws=F, wsb=256):
        return getattr(lib, "mla_cache_gather_" + fmt)(cache, bt, sl, cu, b, n, pages, page, mp, out, ws, wsb, Z)

    for name in ("c", "r", "cache", "bt", "sl", "cu", "ws"):
        assert app(**{name: Z}) == -1, name
    for name in ("cache", "bt", "sl", "cu", "out", "ws"):
        assert gat(**{name: Z}) == -1, name
    for fn in (app, gat):
        assert fn(b=-1) == -1 and fn(n=-1) == -1 and fn(pages=0) == -1 and fn(mp=0) == -1
        assert fn(page=32) == -2 and fn(b=(1 << 16) + 1) == -2 and fn(pages=1 << 25) == -2 and fn(n=1 << 30) == -2
        assert fn(cache=off(8)) == -1 and fn(ws=off(128)) == -1 and fn(cu=off(2)) == -1
        assert fn(wsb=32) == -3
        assert fn(b=0) == 0 and fn(n=0) == 0
    assert app(cs=0) == -1 and app(cs=513) == -1 and app(rs=68) == -1
    assert app(c=off(8)) == -1 and app(r=off(4)) == -1 and gat(out=off(8)) == -1


def test_expand_validates_on_the_host(lib):
    def call(x=F, st=512, uk=F, uv=F, n=3, h=128, dv=128, k=F, v=F, ws=F, wsb=256):
        return lib.mla_expand_kv(x, st, uk, uv, n, h, dv, k, v, ws, wsb, Z)

    for name in ("x", "uk", "uv", "k", "v", "ws"):
        assert call(**{name: Z}) == -1, name
    assert call(n=-1) == -1 and call(h=64) == -2 and call(dv=64) == -2 and call(n=(1 << 24) + 1) == -2
    assert call(st=504) == -1 and call(st=516) == -1                 # rows overlap; not 16 bytes
    assert call(x=off(8)) == -1 and call(k=off(16)) == -1 and call(ws=off(64)) == -1 and call(wsb=8) == -3
    assert call(n=0) == 0


def test_prefill_validates_on_the_host(lib):
    ok = (16384, 128, 8192, 64, 16384, 128, 64, 16384, 128)

    def call(qn=F, qr=F, kn=F, kr=F, v=F, st=ok, cq=F, ck=F, b=2, nq=5, nk=9, h=128, causal=1, scale=0.1, out=F,
             lse=F, ws=F, wsb=1 << 20):
        s = None if st is None else (ctypes.c_size_t * 9)(*st)
        return lib.mla_prefill_bf16(qn, qr, kn, kr, v, s, cq, ck, b, nq, nk, h, causal, ctypes.c_float(scale), out, lse,
                                    ws, wsb, Z)

    for name in ("qn", "qr", "kn", "kr", "v", "cq", "ck", "out", "lse", "ws"):
        assert call(**{name: Z}) == -1, name
    assert call(st=None) == -1
    for i in range(9):
        for bad in (0, 12, 1 << 39):
            assert call(st=ok[:i] + (bad,) + ok[i + 1:]) == -1, (i, bad)
    assert call(b=-1) == -1 and call(nq=-1) == -1 and call(nk=-1) == -1
    assert call(scale=0.0) == -1 and call(scale=math.nan) == -1 and call(scale=math.inf) == -1
    assert call(h=64) == -2 and call(b=(1 << 16) + 1) == -2 and call(nq=(1 << 24) + 1) == -2
    assert call(qn=off(8)) == -1 and call(out=off(16)) == -1 and call(ws=off(64)) == -1
    assert call(wsb=64) == -3
    assert call(b=0) == 0 and call(nq=0) == 0
    n = ctypes.c_size_t(0)
    assert lib.mla_workspace_size_prefill(-1, 4, ctypes.byref(n)) == -1
    assert lib.mla_workspace_size_prefill(1, (1 << 24) + 1, ctypes.byref(n)) == -2
    assert lib.mla_workspace_size_prefill(3, 1000, ctypes.byref(n)) == 0
    tiles = sum(-(-x // 256) for x in (998, 1, 1))                    # the most tiles three sequences of 1000 queries make
    assert n.value >= 64 + 32 * tiles


@pytest.mark.parametrize("fmt", FORMATS)
def test_tree_entries_validate_on_the_host(lib, fmt):
    def call(q=F, qr=F, cache=F, bt=F, sl=F, par=F, nn=Z, b=2, t=3, h=128, pages=4, page=64, mp=2, scale=0.1, out=F,
             lse=F, ws=F, wsb=1 << 30):
        return getattr(lib, "mla_decode_tree_" + fmt)(q, qr, cache, bt, sl, par, nn, b, t, h, pages, page, mp,
                                                      ctypes.c_float(scale), out, lse, ws, wsb, Z)

    for name in ("q", "qr", "cache", "bt", "sl", "par", "out", "lse", "ws"):
        assert call(**{name: Z}) == -1, name
    assert call(b=-1) == -1 and call(t=0) == -1 and call(mp=0) == -1 and call(scale=-1.0) == -1
    assert call(t=65) == -2 and call(h=64) == -2 and call(page=16) == -2 and call(b=1025, t=64) == -2
    assert call(b=1024, t=64, mp=1 << 14) == -2                       # 2^30 pages over the rows
    assert call(q=off(16)) == -1 and call(out=off(16)) == -1 and call(par=off(2)) == -1 and call(nn=off(1)) == -1
    assert call(b=0) == 0
    n = ctypes.c_size_t(0)
    assert lib.mla_workspace_size_tree(1, 65, 128, 64, ctypes.byref(n)) == -2
    assert lib.mla_workspace_size_tree(1, 0, 128, 64, ctypes.byref(n)) == -1
    assert lib.mla_workspace_size_tree(1, 4, 64, 64, ctypes.byref(n)) == -2


# ------------------------------------------------------------------ the binding
STREAM = types.SimpleNamespace(cuda_stream=0x77)


class Rows(FakeTensor):
    def __init__(self, shape, strides=None, dev=0):
        super().__init__(shape, dev)
        self._strides = strides or [int(np.prod(shape[d + 1:])) for d in range(len(shape))]

    def stride(self, d):
        return self._strides[d]


@pytest.fixture
def fake(monkeypatch):
    fl = FakeLib()
    monkeypatch.setattr(binding, "load", lambda *a, **k: fl)
    monkeypatch.setattr(binding, "_check", lambda *a, **k: None)
    monkeypatch.setattr(binding, "_check_rows", lambda *a, **k: None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return fl


def values(args):
    return [a.value if hasattr(a, "value") else a for a in args]


@pytest.mark.parametrize("fmt", FORMATS)
def test_row_wrappers_marshal(fake, fmt):
    w = binding._ROW_WIDTH[fmt]
    c, r, cache = Rows((7, 512), (1152, 1)), Rows((7, 64), (576, 1)), FakeTensor((9, 64, w))
    bt, sl, cu, ws, out = FakeTensor((3, 5)), FakeTensor((3,)), FakeTensor((4,)), FakeTensor((256,)), FakeTensor((7, 576))
    assert getattr(binding, "mla_cache_append_" + fmt)(c, r, cache, bt, sl, cu, workspace=ws, stream=STREAM) is cache
    assert getattr(binding, "mla_cache_gather_" + fmt)(cache, bt, sl, cu, 7, out=out, workspace=ws, stream=STREAM) is out
    (n1, a1), (n2, a2) = fake.calls
    p = lambda t: t.data_ptr()  # noqa: E731
    assert (n1, n2) == ("mla_cache_append_" + fmt, "mla_cache_gather_" + fmt)
    assert values(a1) == [p(c), 1152, p(r), 576, p(cache), p(bt), p(sl), p(cu), 3, 7, 9, 64, 5, p(ws), 256, 0x77]
    assert values(a2) == [p(cache), p(bt), p(sl), p(cu), 3, 7, 9, 64, 5, p(out), p(ws), 256, 0x77]
    with pytest.raises(ValueError, match="c_kv"):
        getattr(binding, "mla_cache_append_" + fmt)(Rows((7, 512), dev=1), r, cache, bt, sl, cu, workspace=ws, stream=STREAM)
    with pytest.raises(ValueError, match="kv_cache must be"):
        getattr(binding, "mla_cache_gather_" + fmt)(FakeTensor((9, 64, w + 1)), bt, sl, cu, 7, out=out, workspace=ws)
    with pytest.raises(ValueError, match="n_rows"):
        getattr(binding, "mla_cache_gather_" + fmt)(cache, bt, sl, cu, -1, out=out, workspace=ws)
    assert len(fake.calls) == 2


def test_expand_and_prefill_wrappers_marshal(fake):
    lat, uk, uv = Rows((7, 512), (576, 1)), FakeTensor((128, 128, 512)), FakeTensor((128, 128, 512))
    k, v, ws = FakeTensor((7, 128, 128)), FakeTensor((7, 128, 128)), FakeTensor((4096,))
    assert binding.mla_expand_kv(lat, uk, uv, k_nope=k, v=v, workspace=ws, stream=STREAM) == (k, v)
    qn, qr = Rows((5, 128, 128), (24576, 192, 1)), Rows((5, 128, 64), (24576, 192, 1))
    kn, kr, vv = Rows((1, 128, 128), (3, 128, 1)), Rows((1, 64), (5, 1)), Rows((1, 128, 128))
    cq, ck, out, lse = FakeTensor((4,)), FakeTensor((4,)), FakeTensor((5, 128, 128)), FakeTensor((5, 128))
    assert binding.mla_prefill_bf16(qn, qr, kn, kr, vv, cq, ck, 0.5, causal=False, out=out, lse=lse, workspace=ws,
                                    stream=STREAM) == (out, lse)
    (n1, a1), (n2, a2) = fake.calls
    p = lambda t: t.data_ptr()  # noqa: E731
    assert n1 == "mla_expand_kv" and n2 == "mla_prefill_bf16"
    assert values(a1) == [p(lat), 576, p(uk), p(uv), 7, 128, 128, p(k), p(v), p(ws), 4096, 0x77]
    assert values(a2[:5]) == [p(qn), p(qr), p(kn), p(kr), p(vv)]
    # a dimension of one entry gets the contiguous stride, whatever the view says
    assert list(a2[5]) == [24576, 192, 24576, 192, 16384, 128, 64, 16384, 128]
    assert values(a2[6:]) == [p(cq), p(ck), 3, 5, 1, 128, 0, 0.5, p(out), p(lse), p(ws), 4096, 0x77]
    with pytest.raises(ValueError, match="k_rope"):
        binding.mla_prefill_bf16(qn, qr, kn, Rows((1, 64), dev=1), vv, cq, ck, 0.5, out=out, lse=lse, workspace=ws)
    assert len(fake.calls) == 2


@pytest.mark.parametrize("fmt", FORMATS)
def test_tree_wrappers_marshal(fake, fmt):
    q, qr, cache = FakeTensor((3, 6, 128, 512)), FakeTensor((3, 6, 128, 64)), FakeTensor((9, 64, binding._ROW_WIDTH[fmt]))
    bt, sl, par, nn, ws = FakeTensor((3, 5)), FakeTensor((3,)), FakeTensor((3, 6)), FakeTensor((3,)), FakeTensor((999,))
    out, lse = FakeTensor((3, 6, 128, 512)), FakeTensor((3, 6, 128))
    fn = getattr(binding, "mla_decode_tree_" + fmt)
    assert fn(q, qr, cache, bt, sl, par, 0.25, n_nodes=nn, out=out, lse=lse, workspace=ws, stream=STREAM) == (out, lse)
    fn(q, qr, cache, bt, sl, par, 0.25, out=out, lse=lse, workspace=ws, stream=STREAM)
    p = lambda t: t.data_ptr()  # noqa: E731
    (n1, a1), (_, a2) = fake.calls
    assert n1 == "mla_decode_tree_" + fmt
    tail = [3, 6, 128, 9, 64, 5, 0.25, p(out), p(lse), p(ws), 999, 0x77]
    assert values(a1) == [p(x) for x in (q, qr, cache, bt, sl, par, nn)] + tail
    assert values(a2) == [p(x) for x in (q, qr, cache, bt, sl, par)] + [None] + tail
    with pytest.raises(ValueError, match="parents"):
        fn(q, qr, cache, bt, sl, FakeTensor((3, 6), 1), 0.25, out=out, lse=lse, workspace=ws)
    assert len(fake.calls) == 2


def test_row_checks_refuse_what_the_kernels_cannot_read():
    bad = torch.zeros((4, 512), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        binding._check_rows(bad, "x", (512,))
    with pytest.raises(TypeError, match="tensor"):
        binding._check_rows(np.zeros((4, 512)), "x", (512,))

    class Cuda:                                            # a tensor's metadata, said to be on a GPU
        def __init__(self, t):
            self.t = t

        def __getattr__(self, n):
            return True if n == "is_cuda" else getattr(self.t, n)

    def refuses(t, match, tail=(512,), rows=None, kind=ValueError):
        real = binding.torch.Tensor
        try:
            binding.torch.Tensor = Cuda
            with pytest.raises(kind, match=match):
                binding._check_rows(Cuda(t), "x", tail, rows)
        finally:
            binding.torch.Tensor = real

    base = torch.zeros(1 << 16, dtype=torch.bfloat16)
    shift = (-(base.data_ptr() // 2)) % 8                  # the first 16-byte boundary
    ok = base[shift:shift + 8 * 600].view(8, 600)[:, :512]
    refuses(ok.float(), "bfloat16", kind=TypeError)
    refuses(ok, "shape", (448,))
    refuses(ok, "shape", (512,), 7)
    refuses(base[shift + 4:shift + 4 + 4096].view(8, 512), "16 bytes")
    refuses(base[shift:shift + 8 * 516].view(8, 516)[:, :512], "16 bytes")
    refuses(base[shift:shift + 4096].view(512, 8).T, "last dimension")
    refuses(base[shift:shift + 512].expand(8, 512), "16 bytes")   # a broadcast row


# ------------------------------------------------------------------ the oracles
def test_row_encoder_against_torch_casts_and_a_scale_search():
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((40, 576)) * np.exp2(rng.integers(-30, 30, (40, 1)))).astype(np.float32)
    x = torch.from_numpy(x).to(torch.bfloat16).double().numpy()
    x[3, :64] = 0
    for kind, group, top in (("fp8", 32, 448.0), ("fp4", 16, 6.0)):
        codes, scales = row_codec.encode_groups(x, kind)
        k = scales.astype(int) - 127
        g = x.reshape(40, -1, group)
        amax = np.abs(g).max(-1)
        nz = amax > 0
        assert (k[~nz] == 0).all()
        assert (amax <= top * np.exp2(k.astype(float)))[nz].all() and (amax > top * np.exp2(k - 1.0))[nz].all()
        scaled = g / np.exp2(k.astype(float))[..., None]
        if kind == "fp8":
            want = torch.from_numpy(scaled).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
            np.testing.assert_array_equal(codes.reshape(want.shape), want)
        else:
            back = fp4_codec.e2m1_to_float64(codes).reshape(scaled.shape)
            grid = np.concatenate([row_codec.E2M1, -row_codec.E2M1])
            best = np.abs(scaled[..., None] - grid).min(-1)
            np.testing.assert_array_equal(np.abs(scaled - back), best)      # nearest
            mid = (row_codec.E2M1[:-1] + row_codec.E2M1[1:]) / 2
            np.testing.assert_array_equal(row_codec.float64_to_e2m1(mid) % 2, 0)   # ties to even


@pytest.mark.parametrize("fmt,decode,width", [("fp8", fp8_codec.dequant_rows, 594), ("fp4", fp4_codec.dequant_rows, 324),
                                              ("fp8_v41", fp8_codec.dequant_rows_v41, 528),
                                              ("fp4_v41", fp4_codec.dequant_rows_v41, 288)])
def test_encoded_rows_decode_to_themselves(fmt, decode, width):
    # decoded values encode to the same values: the codes are exact under their scale
    rng = np.random.default_rng(4)
    c, r = rng.standard_normal((9, 512)), rng.standard_normal((9, 64))
    raw = row_codec.encode_rows(c, r, fmt)
    assert raw.shape == (9, width) and raw.dtype == np.uint8
    v = decode(raw)
    again = decode(row_codec.encode_rows(v[:, :512], v[:, 512:], fmt))
    np.testing.assert_array_equal(v, again)
    latent = 448 if fmt.endswith("v41") else 512
    step = 2.0 ** -4 if fmt.startswith("fp8") else 2.0 ** -2       # half a step of the format, relative, or of its smallest
    src = np.concatenate([c, r], -1)
    cols = np.r_[0:latent, 512:576]
    group = 32 if fmt.startswith("fp8") else 16
    top = np.abs(src[:, cols]).reshape(9, -1, group).max(-1).repeat(group, 1)
    err = np.abs(v[:, cols] - src[:, cols])
    assert (err <= step * np.abs(src[:, cols]) + top * (2.0 ** -17 if group == 32 else 2.0 ** -3)).all()


def test_non_finite_groups_take_the_nan_scale():
    x = np.ones((1, 576))
    x[0, 40] = np.inf
    codes, scales = row_codec.encode_groups(x, "fp8")
    assert scales[0, 1] == 255 and (codes[0, 32:64] == 0).all() and (np.delete(scales[0], 1) != 255).all()


@pytest.mark.parametrize("causal", [True, False])
def test_expanded_oracle_against_torch_softmax(causal):
    g = torch.Generator().manual_seed(5)
    nq, nk = [3, 7], [5, 4]
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    qn, qr, kn, kr, v = r(10, 2, 8), r(10, 2, 4), r(9, 2, 8), r(9, 4), r(9, 2, 6)
    out, lse, mag = expanded.prefill(*(t.numpy() for t in (qn, qr, kn, kr, v)), [0, 3, 10], [0, 5, 9], 0.3, causal, [0, 1])
    q0 = k0 = 0
    for n, m in zip(nq, nk):
        for h in range(2):
            s = 0.3 * (torch.cat([qn[q0:q0 + n, h], qr[q0:q0 + n, h]], -1) @ torch.cat([kn[k0:k0 + m, h], kr[k0:k0 + m]], -1).T)
            if causal:
                s = s.masked_fill(~torch.ones((n, m), dtype=torch.bool).tril(m - n), -math.inf)
            seen = torch.isfinite(s).any(-1)
            p = torch.softmax(s, -1).nan_to_num(0.0)
            np.testing.assert_allclose(out[q0:q0 + n, h], (p @ v[k0:k0 + m, h]).numpy(), atol=1e-12)
            np.testing.assert_allclose(lse[q0:q0 + n, h][seen], torch.logsumexp(s, -1)[seen].numpy(), atol=1e-12)
            assert np.isneginf(lse[q0:q0 + n, h][~seen]).all() and (out[q0:q0 + n, h][~seen] == 0).all()
            assert causal or bool(seen.all())
        q0, k0 = q0 + n, k0 + m


def test_expanded_oracle_is_the_unabsorbed_decode():
    rng = np.random.default_rng(6)
    c, kr = rng.standard_normal((11, 512)), rng.standard_normal((11, 64))
    wk, wv = rng.standard_normal((3, 16, 512)) / 20, rng.standard_normal((3, 16, 512)) / 20
    qn, qr = rng.standard_normal((3, 16)), rng.standard_normal((3, 64))
    want, wl = mla_oracle.attend_unabsorbed(qn, qr, c, kr, wk, wv, 0.1)
    k, v = np.einsum("nc,hdc->nhd", c, wk), np.einsum("nc,hdc->nhd", c, wv)
    out, lse, _ = expanded.prefill(qn[None], qr[None], k, kr, v, [0, 1], [0, 11], 0.1, True, [0, 1, 2])
    np.testing.assert_allclose(out[0], want, atol=1e-12)
    np.testing.assert_allclose(lse[0], wl, atol=1e-12)


def test_tree_visibility_is_reachability():
    parents = [-1, 0, 0, 2, -1, 4, 3]
    a = np.eye(7, dtype=int)
    for i, p in enumerate(parents):
        if p >= 0:
            a[i, p] = 1
    reach = np.linalg.matrix_power(a, 7) > 0
    for i in range(7):
        see = expanded.tree_sees(parents, 7, i, 5)
        np.testing.assert_array_equal(see[:5], np.arange(5))
        np.testing.assert_array_equal(see[5:] - 5, np.nonzero(reach[i])[0])
    assert expanded.tree_sees(parents, 3, 4, 5).size == 0
    np.testing.assert_array_equal(expanded.tree_sees([-1, 0, 1, 2], 4, 3, 6), np.arange(10))   # a chain: causal
