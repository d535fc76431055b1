"""Rotation, 8-bit caches and their attention without a GPU: struct layouts, every refusal that the host
makes before it touches the device, the binding's checks, workspace sizes, the oracle against other ways
to the same numbers, and the arithmetic that the integer codes rest on."""
import ctypes
import math
import os
import subprocess
from fractions import Fraction as F

import numpy as np
import pytest
import torch

from intra_spatial_pipelining_gb300 import build, sgp
from oracle import kvq as Q
from oracle import layer as O
from oracle import serving as S
from tests.test_serving_devices_cpu import BF, F32, I32, U8, Fake, env  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
E = sgp.SGP_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    build.build()
    return sgp.lib()


@pytest.fixture(scope="module")
def mem():
    """Host memory whose address stands in for device pointers: nothing is launched."""
    buf = ctypes.create_string_buffer(1 << 16)
    return buf, (ctypes.addressof(buf) + 255) & ~255


def test_struct_layouts_match_the_header(lib, tmp_path):
    structs = [sgp.sgp_rope, sgp.sgp_kvq]
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "sgp.h"', "int main(void){"]
    for st in structs:
        n = st.__name__
        lines.append(f'printf("{n} %zu\\n", sizeof({n}));')
        lines += [f'printf("{n}.{f} %zu\\n", offsetof({n}, {f}));' for f, _ in st._fields_]
    names = ("SGP_ROPE_HALF", "SGP_ROPE_INTERLEAVED", "SGP_ROPE_PLAIN", "SGP_ROPE_LINEAR", "SGP_ROPE_BY_TURNS",
             "SGP_ROPE_BY_INDEX", "SGP_KVQ_E4M3", "SGP_KVQ_INT8")
    lines += [f'printf("{n} %d\\n", {n});' for n in names]
    src = tmp_path / "abi.c"
    src.write_text("\n".join(lines + ["return 0;}"]))
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "abi")], check=True)
    out = dict(l.split() for l in subprocess.run([str(tmp_path / "abi")], capture_output=True, text=True,
                                                 check=True).stdout.splitlines())
    for st in structs:
        n = st.__name__
        assert int(out[n]) == ctypes.sizeof(st), n
        for f, _ in st._fields_:
            assert int(out[f"{n}.{f}"]) == getattr(st, f).offset, f"{n}.{f}"
    assert [int(out[n]) for n in names] == [0, 1, 0, 1, 2, 3, 0, 1]      # the order of the binding's names


# ---------------------------------------------------------------------------------------
# rotation
# ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("scaling", ["none", "linear", "turns", "index"])
@pytest.mark.parametrize("rot,theta,factor,context,low,high", [
    (64, 150000.0, 32.0, 4096.0, 1.0, 32.0), (16, 10000.0, 4.0, 8192.0, 1.0, 4.0), (48, 1.5, 0.5, 100.0, 0.01, 90.0)])
def test_rope_frequencies(lib, scaling, rot, theta, factor, context, low, high):
    r = sgp.make_rope(rot, theta, layout="interleaved", scaling=scaling, factor=factor, context=context,
                      turns_low=low, turns_high=high, amplitude=1.5)
    want = Q.frequencies(rot, theta, scaling, factor, context, low, high)
    np.testing.assert_allclose(list(r.freq)[:rot // 2], want, rtol=1e-13)
    assert not any(list(r.freq)[rot // 2:]) and (r.rot_dim, r.layout, r.amplitude) == (rot, 1, 1.5)
    if scaling != "none":
        plain = Q.frequencies(rot, theta)
        assert (np.minimum(plain, plain / factor) - 1e-15 <= want).all() and (want <= np.maximum(plain, plain / factor) + 1e-15).all()


def test_rope_init_refuses_bad_arguments(lib):
    r = sgp.sgp_rope()
    ok = dict(rope=ctypes.byref(r), rot=64, layout=0, theta=1e4, scaling=3, factor=2.0, context=100.0, low=1.0, high=2.0,
              amplitude=1.0)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.sgp_rope_init(a["rope"], a["rot"], a["layout"], a["theta"], a["scaling"], a["factor"], a["context"],
                                 a["low"], a["high"], a["amplitude"])
    assert call() == 0
    nan, inf = math.nan, math.inf
    for kw in (dict(rope=None), dict(rot=0), dict(rot=8), dict(rot=24), dict(rot=80), dict(rot=-16), dict(layout=2),
               dict(layout=-1), dict(theta=1.0), dict(theta=nan), dict(theta=inf), dict(scaling=4), dict(scaling=-1),
               dict(factor=0.0), dict(factor=nan), dict(factor=inf), dict(context=0.0), dict(context=nan), dict(low=0.0),
               dict(low=2.0), dict(high=1.0), dict(high=nan), dict(high=inf), dict(amplitude=nan), dict(amplitude=inf)):
        assert call(**kw) == E, kw
        assert lib.sgp_last_error().decode()
    # what a scaling does not use is not read
    assert call(scaling=0, factor=nan, context=nan, low=nan, high=nan) == 0
    assert call(scaling=1, context=nan, low=nan, high=nan) == 0
    for kw in (dict(layout="rows"), dict(scaling="ntk")):
        with pytest.raises(ValueError):
            sgp.make_rope(**kw)


ROPE = dict(nq=4, nkv=2, gq=0, gk=0, eps=0.0, pos=0, q=0, ldq=256, qo=8192, ldqo=256, k=16384, ldk=128, ko=20480, ldko=128,
            T=4, ws=0, nbytes=64, rot=64, layout=0, amp=1.0, freq=1.0)


def test_qk_rope_refuses_bad_arguments(lib, mem):
    base = mem[1]

    def call(**kw):
        a = dict(ROPE, **kw)
        d = sgp.make_heads(a["nq"], a["nkv"], a.get("d", 64))
        r = sgp.sgp_rope(a["rot"], a["layout"], a["amp"])
        r.freq[3] = a["freq"]
        at = lambda x: None if x is None else base + x
        return lib.sgp_qk_rope(ctypes.byref(d), ctypes.byref(r) if not a.get("none") else None, at(a["gq"]), at(a["gk"]), a["eps"],
                               at(a["pos"]), at(a["q"]), a["ldq"], at(a["qo"]), a["ldqo"], at(a["k"]), a["ldk"], at(a["ko"]),
                               a["ldko"], a["T"], at(a["ws"]), a["nbytes"], None)
    nan = math.nan
    for kw in (dict(d=128), dict(nkv=0), dict(nq=3), dict(nq=34), dict(none=True), dict(rot=20), dict(rot=128), dict(layout=2),
               dict(amp=nan), dict(freq=nan), dict(freq=math.inf), dict(eps=-1.0), dict(eps=nan), dict(T=0), dict(T=(1 << 20) + 1),
               dict(gq=8), dict(gk=2), dict(pos=None), dict(pos=2), dict(q=8), dict(q=None), dict(qo=None), dict(qo=8200),
               dict(k=None), dict(ko=None), dict(k=16392), dict(ko=20488), dict(q=None, qo=None, k=None, ko=None),
               dict(ldq=255), dict(ldq=260), dict(ldq=248), dict(ldqo=(1 << 41)), dict(ldk=120), dict(ldko=132),
               dict(ws=None), dict(ws=64), dict(nbytes=63),
               # results that overlap inputs or each other without being the same rows
               dict(qo=16), dict(qo=512), dict(q=8192, ldq=264), dict(ko=16), dict(ko=8192), dict(ko=16384 + 16),
               dict(ko=16384, ldko=136), dict(qo=16384)):
        assert call(**kw) == E, kw
    # rows of one stride may interleave: k_out into the gaps of q_out's rows
    assert call(ldqo=384, qo=32768, ko=32768 + 512, ldko=384, T=4, ws=None) == E      # (the workspace is what is refused)
    assert b"workspace" in lib.sgp_last_error()
    assert call(ldqo=384, qo=32768, ko=32768 + 496, ldko=384, T=4, ws=None) == E
    assert b"overlap" in lib.sgp_last_error()
    assert call(q=32768, ldq=384, qo=32768, ldqo=384, k=32768 + 512, ldk=384, ko=32768 + 512, ldko=384, ws=None) == E
    assert b"workspace" in lib.sgp_last_error()


def test_qk_rope_append_refuses_bad_arguments(lib, mem):
    base = mem[1]
    ok = dict(ROPE, kc=24576, vc=28672, cap=4, n=4, seq=0, slot=0, v=16384 + 2048, ldv=128)

    def call(**kw):
        a = dict(ok, **kw)
        d = sgp.make_heads(a["nq"], a["nkv"])
        r = sgp.sgp_rope(a["rot"], a["layout"], a["amp"])
        at = lambda x: None if x is None else base + x
        c = sgp.sgp_layer(k_cache=at(a["kc"]), v_cache=at(a["vc"]), kv_cap=a["cap"])
        return lib.sgp_qk_rope_append(ctypes.byref(d), ctypes.byref(r), at(a["gq"]), at(a["gk"]), a["eps"], at(a["pos"]),
                                      at(a["q"]), a["ldq"], at(a["qo"]), a["ldqo"], at(a["k"]), a["ldk"], at(a["v"]), a["ldv"],
                                      None if a.get("none") else ctypes.byref(c), a["n"], at(a["seq"]), at(a["slot"]), a["T"],
                                      at(a["ws"]), a["nbytes"], None)
    for kw in (dict(none=True), dict(kc=None), dict(kc=24584), dict(vc=None), dict(vc=28680), dict(cap=0), dict(cap=1 << 30),
               dict(cap=1 << 20, n=1 << 11), dict(n=0), dict(n=-1), dict(slot=None), dict(slot=2), dict(seq=2), dict(k=8),
               dict(v=8), dict(ldv=120), dict(q=24576), dict(qo=28672), dict(k=28672), dict(v=24576), dict(vc=24576 + 2048),
               dict(qo=16384), dict(qo=16384 + 2048), dict(q=None), dict(qo=None), dict(T=0), dict(ws=None)):
        assert call(**kw) == E, kw
    # without v its cache is not read; keys in place; no queries
    for kw in (dict(v=None, vc=None, ws=None), dict(k=None, ws=None), dict(q=None, qo=None, ws=None), dict(seq=None, ws=None)):
        assert call(**kw) == E and b"workspace" in lib.sgp_last_error(), kw


def test_rotation_against_the_layers():
    """The oracle's rotation is the decode layer's, at any layout a permutation of it, and keeps lengths."""
    rng = np.random.default_rng(1)
    x, pos = rng.standard_normal((5, 3, 64)), [0, 1, 77, -9, 30000]
    y, err = Q.rope(x, pos, Q.frequencies(64, 150000.0))
    want = np.stack([O.rope(x[t], p, 150000.0) for t, p in enumerate(pos)])
    np.testing.assert_allclose(y, want, atol=1e-9)
    perm = np.arange(64).reshape(2, 32).T.reshape(-1)          # pair by pair
    z, _ = Q.rope(x[..., perm], pos, Q.frequencies(64, 150000.0), layout="interleaved")
    np.testing.assert_allclose(z, y[..., perm], atol=1e-12)
    np.testing.assert_allclose((y ** 2).sum(2), (x ** 2).sum(2))
    w, e = Q.rope(x, pos, Q.frequencies(32, 1e4), amplitude=2.0)
    assert np.array_equal(w[..., 32:], x[..., 32:]) and not e[..., 32:].any()
    np.testing.assert_allclose((w[..., :32] ** 2).sum(2), 4 * (x[..., :32] ** 2).sum(2))
    assert (err[..., 0] >= S.UBF * np.abs(y[..., 0])).all()


# ---------------------------------------------------------------------------------------
# caches in 8 bits
# ---------------------------------------------------------------------------------------
def _kvq(base, k=0, v=8192, ks=16384, vs=17408, cap=32, block=16, fmt=0):
    at = lambda x: None if x is None else base + x
    return sgp.sgp_kvq(at(k), at(v), at(ks), at(vs), cap, block, fmt)


BAD_KVQ = (dict(k=None), dict(v=None), dict(k=8), dict(v=8200), dict(ks=None), dict(vs=None), dict(ks=16386), dict(vs=2),
           dict(cap=0), dict(cap=8), dict(cap=72), dict(cap=-16), dict(block=0), dict(block=8), dict(block=24), dict(block=256),
           dict(fmt=2), dict(fmt=-1), dict(cap=1 << 29))


def test_kvq_fold_refuses_bad_arguments(lib, mem):
    base = mem[1]
    src, rest = (20480, 24576), (28672, 36864)                # 4 sequences x 1 head x 8 and x 16 rows

    def call(nkv=1, kvq=None, a=src, acap=8, b=rest, bcap=16, n=60000, h=60032, no=60064, ho=60096, T=4, ws=0, nbytes=64, none=None):
        d, c = sgp.make_heads(nkv, nkv), _kvq(base, **(kvq or {}))
        at = lambda x: None if x is None else base + x
        f = sgp.sgp_layer(k_cache=at(a[0]), v_cache=at(a[1]), kv_cap=acap)
        r = sgp.sgp_layer(k_cache=at(b[0]), v_cache=at(b[1]), kv_cap=bcap)
        p = [None if none == i else ctypes.byref(x) for i, x in enumerate((d, f, c, r))]
        return lib.sgp_kvq_fold(*p, at(n), at(h), at(no), at(ho), T, at(ws), nbytes, None)
    for bad in BAD_KVQ:
        if bad != dict(cap=-16):
            assert call(kvq=bad) == E, bad
    for kw in (dict(none=0), dict(none=1), dict(none=2), dict(none=3), dict(nkv=0), dict(T=0), dict(T=513), dict(a=(None, 0)),
               dict(a=(20480 + 16, 24576)), dict(b=(28680, 36864)), dict(acap=0), dict(bcap=0), dict(n=None), dict(h=None),
               dict(no=None), dict(ho=None), dict(n=60001), dict(h=60000), dict(no=60096), dict(no=60000), dict(ho=60032),
               dict(no=60032), dict(ho=60000), dict(no=60004), dict(ws=None), dict(ws=16), dict(nbytes=63),
               # no room for what may be left, in place with another capacity, caches that share bytes
               dict(acap=32, bcap=14, a=(40960, 49152 + 8192)), dict(acap=8, bcap=7), dict(b=src, bcap=16), dict(b=(20480, 36864), bcap=8),
               dict(b=(28672, 24576)), dict(b=(28672, 28672)), dict(a=(0, 24576)), dict(a=(20480, 8192)), dict(b=(28672, 16384)),
               dict(kvq=dict(v=1024)), dict(kvq=dict(vs=16384)), dict(kvq=dict(ks=4096)), dict(kvq=dict(k=20480)),
               dict(a=(20480, 20480), b=(20480, 20480), bcap=8)):
        assert call(**kw) == E, kw
    # in place, lengths too; and from one cache as both keys and values into others
    for kw in (dict(b=src, bcap=8, no=60000, ho=60032), dict(a=(20480, 20480)), dict(acap=8, bcap=8)):
        assert call(ws=None, **kw) == E and b"workspace" in lib.sgp_last_error(), kw


def test_kvq_attention_refuses_bad_arguments(lib, mem):
    base = mem[1]
    need = sgp.sgp_kvq_attention_workspace_bytes(sgp.make_heads(16, 2), 4)

    def call(nq=16, nkv=2, d=64, kvq=None, h=0, k=0, v=4096, cap=8, window=0, n=0, q=0, o=32768, lse=0, T=4, ws=0,
             nbytes=need, cache=True, none=None):
        dims, c = sgp.make_heads(nq, nkv, d), _kvq(base, **(kvq or {}))
        at = lambda x: None if x is None else base + x
        t = sgp.sgp_layer(k_cache=at(k), v_cache=at(v), kv_cap=cap, window=window)
        return lib.sgp_kvq_attention(None if none == 0 else ctypes.byref(dims), None if none == 1 else ctypes.byref(c), at(h),
                                     ctypes.byref(t) if cache else None, at(n), at(q), at(o), at(lse), T, at(ws), nbytes, None)
    for bad in BAD_KVQ:
        assert call(kvq=bad) == E, bad
    for kw in (dict(none=0), dict(none=1), dict(d=128), dict(nkv=0), dict(nq=0), dict(nq=17), dict(nq=34), dict(T=0), dict(T=513),
               dict(h=None), dict(h=2), dict(k=None), dict(k=8), dict(v=None), dict(cap=0), dict(window=-1), dict(n=None),
               dict(n=1), dict(q=None), dict(q=8), dict(o=None), dict(o=16), dict(o=8), dict(lse=2), dict(ws=None), dict(ws=128),
               dict(nbytes=need - 1), dict(nbytes=0), dict(cap=1 << 28)):
        assert call(**kw) == E, kw
        assert lib.sgp_last_error().decode()
    # a sequence's positions are counted in 32 bits
    assert call(nq=1, nkv=1, T=1, kvq=dict(cap=1 << 30), cap=1 << 30) == E and b"2^31" in lib.sgp_last_error()
    assert call(nq=1, nkv=1, T=1, kvq=dict(cap=1 << 30), cap=(1 << 30) - 1, ws=None) == E and b"workspace" in lib.sgp_last_error()
    for kw in (dict(cache=False, n=None), dict(lse=None), dict(o=0), dict(window=5)):
        assert call(nbytes=0, **kw) == E and b"workspace" in lib.sgp_last_error(), kw
    size = sgp.sgp_kvq_attention_workspace_bytes
    for nq, nkv in ((16, 2), (1, 1), (64, 8), (2048, 128)):
        row = [size(sgp.make_heads(nq, nkv), T) for T in range(1, 513)]
        assert all(a <= b for a, b in zip(row, row[1:])) and row[0] > 0
    for args in ((sgp.make_heads(16, 2), 0), (sgp.make_heads(16, 2), 513), (sgp.make_heads(16, 2, 128), 4), (sgp.make_heads(17, 2), 4)):
        assert size(*args) == 0


def test_codes_against_torch():
    t = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(Q.E4M3, t, equal_nan=True)
    rng = np.random.default_rng(0)
    x = torch.from_numpy(rng.standard_normal((256, 64)) * 2.0 ** rng.integers(-8, 9, (256, 1))).bfloat16()
    for block in (16, 32, 64, 128):
        y = x.float().view(-1, block * 64)
        amax = y.abs().amax(1, keepdim=True)
        c, s = Q.quantise(x.double().numpy(), block, "int8")
        scale = amax / torch.full_like(amax, 127.0)
        assert np.array_equal(s.astype(np.float32), scale[:, 0].numpy())
        assert np.array_equal(c.view(np.int8).reshape(-1), (y / scale).round().to(torch.int8).numpy().reshape(-1))
        c, s = Q.quantise(x.double().numpy(), block, "e4m3")
        assert (s == 2.0 ** np.ceil(np.log2(amax[:, 0].double().numpy() / 448))).all()
        got = (y / torch.from_numpy(s).float()[:, None]).to(torch.float8_e4m3fn)
        assert np.array_equal(c.reshape(-1), got.view(torch.uint8).numpy().reshape(-1))
        # a value is off by half a step of its code
        v = Q.values(c, s, block, "e4m3")
        step = np.maximum(np.abs(x.double().numpy()) * 2.0 ** -4, np.repeat(s, block)[:, None] * 2.0 ** -10)
        assert (np.abs(v - x.double().numpy()) <= step).all()
        c, s = Q.quantise(x.double().numpy(), block, "int8")
        assert (np.abs(Q.values(c, s, block, "int8") - x.double().numpy()) <= np.repeat(s, block)[:, None] * 0.5001).all()
    x[3, 5] = math.inf
    for fmt in ("e4m3", "int8"):
        c, s = Q.quantise(x.double().numpy(), 64, fmt)
        assert math.isnan(s[0]) and not c[:64].any() and np.isfinite(s[1:]).all()


def test_attention_oracle():
    """Against softmax written out for one head, with positions hidden."""
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((3, 64)), rng.standard_normal((70, 64)), rng.standard_normal((70, 64))
    o, lse, eo, el = Q.attention(q, k, v, np.full(48, 0.25), 10, 48)
    for h in range(3):
        e = [math.exp(q[h] @ k[p] / 8) for p in range(10, 70)]
        np.testing.assert_allclose(o[h], sum(w * v[p + 10] for p, w in enumerate(e)) / sum(e))
        np.testing.assert_allclose(lse[h], math.log(sum(e)))
    assert (eo > 0).all() and (eo < 0.05).all() and (el < 1e-4).all()
    o, lse, eo, el = Q.attention(q, k[:0], v[:0], np.zeros(0), 0, 0)
    assert not o.any() and (lse == -math.inf).all()


def _rn(x):
    """A positive fraction rounded to 24 significant bits, halves to even."""
    if x == 0:
        return F(0)
    e = x.numerator.bit_length() - x.denominator.bit_length()
    e -= F(2) ** e > x
    unit = F(2) ** (e - 23)
    return F(round(x / unit)) * unit


def test_one_correction_gives_every_integer_code():
    """The kernel takes z = x * (1 / s), corrects it once by its exact remainder and rounds to an integer;
    the definition rounds the fp32 quotient x / s.  The same for every pair of significands that bf16
    numbers x and amax have (s = amax / 127 in fp32) and every quotient from 1/8 up; below it both are 0.
    Exponents shift both alike."""
    missed = 0
    for ma in range(128, 256):
        s = _rn(F(ma, 127))
        inv = _rn(1 / s)
        for mx in range(128, 256):
            for ex in range(10):
                x = F(mx, 2 ** ex)
                if x > ma or x / s < F(1, 8):
                    continue
                want = round(_rn(x / s))
                z = _rn(x * inv)
                missed += round(z) != want
                r = x - z * s
                r = _rn(r) if r >= 0 else -_rn(-r)
                assert round(_rn(z + r * inv)) == want, (ma, mx, ex)
    assert missed > 0                                         # without the correction some are not


# ---------------------------------------------------------------------------------------
# the binding, with fakes for devices and tensors
# ---------------------------------------------------------------------------------------
F8 = torch.float8_e4m3fn


def calls(current, dev_cache, dev_codes, dev_rest):
    def on(dev, make):
        current[0] = dev
        out = make(lambda dtype, *shape: Fake(dtype, *shape, dev=dev))
        current[0] = 0
        return out
    d, r = sgp.make_heads(4, 2), sgp.sgp_rope(64, 0, 1.0)
    cache = on(dev_cache, lambda t: sgp.make_cache(t(BF, 3, 2, 10, 64), t(BF, 3, 2, 10, 64)))
    rest = on(dev_rest, lambda t: sgp.make_cache(t(BF, 3, 2, 16, 64), t(BF, 3, 2, 16, 64)))
    codes = on(dev_codes, lambda t: sgp.make_kvq(t(F8, 3, 2, 64, 64), t(F8, 3, 2, 64, 64), t(F32, 3, 2, 4), t(F32, 3, 2, 4)))
    n, q, k, ws = Fake(I32, 3), Fake(BF, 3, 256), Fake(BF, 3, 128), Fake(U8, 1 << 22)
    o, lse, g = Fake(BF, 3, 4, 64), Fake(F32, 3, 4), Fake(BF, 64)
    return {
        "sgp_qk_rope": lambda: sgp.sgp_qk_rope(d, r, g, g, 1e-5, n, q, q, k, k, 3, ws),
        "sgp_qk_rope_append": lambda: sgp.sgp_qk_rope_append(d, r, g, None, 1e-5, n, q, q, k, k, cache, 3, n, n, 3, ws),
        "sgp_kvq_fold": lambda: sgp.sgp_kvq_fold(d, cache, codes, rest, n, n, n, n, 3, ws),
        "sgp_kvq_attention": lambda: sgp.sgp_kvq_attention(d, codes, n, rest, n, o, o, lse, 3, ws)}


def test_everything_on_the_current_device_is_called(env):  # noqa: F811
    lib, current = env
    for name, call in calls(current, 0, 0, 0).items():
        call()
        assert lib.calls[-1] == name


@pytest.mark.parametrize("name,devices", [
    ("sgp_qk_rope_append", (1, 0, 0)), ("sgp_kvq_fold", (1, 0, 0)), ("sgp_kvq_fold", (0, 1, 0)), ("sgp_kvq_fold", (0, 0, 1)),
    ("sgp_kvq_attention", (0, 1, 0)), ("sgp_kvq_attention", (0, 0, 1))])
def test_structures_of_another_device_are_refused(env, name, devices):  # noqa: F811
    lib, current = env
    with pytest.raises(ValueError, match="device"):
        calls(current, *devices)[name]()
    assert not lib.calls


def test_the_binding_checks_rows_and_arrays(env):  # noqa: F811
    lib, current = env
    d, r = sgp.make_heads(4, 2), sgp.sgp_rope(64, 0, 1.0)
    n, q, k, ws = Fake(I32, 3), Fake(BF, 3, 256), Fake(BF, 3, 128), Fake(U8, 64)
    ok = dict(gq=None, pos=n, q=q, qo=q, k=k, ko=k, T=3, ws=ws)

    def call(**kw):
        a = dict(ok, **kw)
        return sgp.sgp_qk_rope(d, r, a["gq"], None, 0.0, a["pos"], a["q"], a["qo"], a["k"], a["ko"], a["T"], a["ws"])
    call()
    for kw in (dict(gq=Fake(BF, 32)), dict(gq=Fake(F32, 64)), dict(pos=Fake(torch.int64, 3)), dict(pos=Fake(I32, 2)),
               dict(q=Fake(BF, 3, 128)), dict(q=Fake(BF, 2, 256)), dict(qo=Fake(F32, 3, 256)), dict(k=Fake(BF, 3, 2, 64)),
               dict(ko=Fake(BF, 3, 128, dev=1)), dict(T=4), dict(ws=Fake(U8, 63)), dict(ws=Fake(F32, 64))):
        with pytest.raises(ValueError):
            call(**kw)
    assert len(lib.calls) == 1
    codes, scale = Fake(F8, 3, 2, 64, 64), Fake(F32, 3, 2, 4)
    for args in ((Fake(U8, 3, 2, 64, 64),) * 2 + (scale, scale), (codes, Fake(F8, 3, 2, 32, 64), scale, scale),
                 (codes, codes, scale, Fake(F32, 3, 2, 2)), (codes, codes, Fake(F32, 3, 2, 5), Fake(F32, 3, 2, 5)),
                 (codes, codes, Fake(F32, 2, 2, 4), Fake(F32, 2, 2, 4)), (codes, codes, Fake(F32, 3, 8), Fake(F32, 3, 8)),
                 (codes, codes, Fake(torch.float64, 3, 2, 4), Fake(torch.float64, 3, 2, 4)),
                 (codes, Fake(torch.int8, 3, 2, 64, 64), scale, scale), (Fake(F8, 3, 2, 64), Fake(F8, 3, 2, 64), scale, scale)):
        with pytest.raises(ValueError):
            sgp.make_kvq(*args)
    c = sgp.make_kvq(codes, codes, scale, scale)
    assert (c.cap, c.block, c.format) == (64, 16, 0)
    assert sgp.make_kvq(Fake(torch.int8, 1, 1, 128, 64), Fake(torch.int8, 1, 1, 128, 64), Fake(F32, 1, 1, 1), Fake(F32, 1, 1, 1)).block == 128
