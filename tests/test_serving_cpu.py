"""The serving operators without a GPU: struct layouts, every refusal that the host makes before
it touches the device, the binding's checks, and the workspace sizes."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from intra_spatial_pipelining_gb300 import build, sgp, synth
from oracle import serving as S

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
    base = (ctypes.addressof(buf) + 255) & ~255
    return buf, base


def test_struct_layouts_match_the_header(lib, tmp_path):
    structs = [sgp.sgp_prefix, sgp.sgp_evict, sgp.sgp_lora]
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "sgp.h"', "int main(void){"]
    for st in structs:
        n = st.__name__
        lines.append(f'printf("{n} %zu\\n", sizeof({n}));')
        lines += [f'printf("{n}.{f} %zu\\n", offsetof({n}, {f}));' for f, _ in st._fields_]
    src = tmp_path / "abi.c"
    src.write_text("\n".join(lines + ["return 0;}"]))
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "abi")],
                   check=True)
    out = dict(l.split() for l in subprocess.run([str(tmp_path / "abi")], capture_output=True,
                                                 text=True, check=True).stdout.splitlines())
    for st in structs:
        n = st.__name__
        assert int(out[n]) == ctypes.sizeof(st), n
        for f, _ in st._fields_:
            assert int(out[f"{n}.{f}"]) == getattr(st, f).offset, f"{n}.{f}"


def _cache(base, cap=100, window=0, k=0, v=8192):
    return sgp.sgp_layer(k_cache=base + k, v_cache=base + v, kv_cap=cap, window=window)


def test_prefix_attention_refuses_bad_arguments(lib, mem):
    base = mem[1]
    ok = dict(nq=16, nkv=2, d=64, cache=_cache(base), n=2, pcap=50, pk=base, pv=base, plen=base,
              of=base, kv_len=base, q=base, o=base + 16384, lse=base, T=4, ws=base, nbytes=1 << 40)

    def call(**kw):
        a = dict(ok, **kw)
        d = sgp.make_heads(a["nq"], a["nkv"], a["d"])
        pre = sgp.sgp_prefix(a["pk"], a["pv"], a["plen"], a["of"], a["n"], a["pcap"])
        return lib.sgp_prefix_attention(ctypes.byref(d), ctypes.byref(a["cache"]) if a["cache"] else None,
                                        ctypes.byref(pre), a["kv_len"], a["q"], a["o"], a["lse"],
                                        a["T"], a["ws"], a["nbytes"], None)
    bad = [dict(d=128), dict(nkv=0), dict(nq=0), dict(nq=17), dict(nq=34, nkv=2), dict(nkv=1025, nq=1025),
           dict(T=0), dict(T=513), dict(cache=None), dict(cache=_cache(0, k=0)),
           dict(cache=_cache(base, k=8)), dict(cache=_cache(base, v=8)), dict(cache=_cache(base, cap=0)),
           dict(cache=_cache(base, window=-1)), dict(cache=_cache(base, cap=1 << 29)),
           dict(n=-1), dict(n=513), dict(pk=None), dict(pv=base + 8), dict(plen=None), dict(of=None),
           dict(of=base + 2), dict(pcap=0), dict(pcap=1 << 30), dict(kv_len=None), dict(q=None),
           dict(q=base + 8), dict(o=None), dict(o=base + 16), dict(lse=base + 2), dict(ws=None),
           dict(ws=base + 16), dict(nbytes=0)]
    for kw in bad:
        assert call(**kw) == E, kw
        assert lib.sgp_last_error().decode()
    d = sgp.make_heads(16, 2)
    assert call(nbytes=sgp.sgp_prefix_attention_workspace_bytes(d, 4, 100, 2) - 1) == E
    # fewer prefixes never need more
    sizes = [sgp.sgp_prefix_attention_workspace_bytes(d, 64, 100, n) for n in (0, 1, 2, 64, 512)]
    assert sizes == sorted(sizes) and sizes[-1] == sizes[-2]
    for args in ((d, 0, 100, 1), (d, 513, 100, 1), (d, 4, 0, 1), (d, 4, 100, -1), (d, 4, 100, 513),
                 (sgp.make_heads(16, 2, 128), 4, 100, 1)):
        assert sgp.sgp_prefix_attention_workspace_bytes(*args) == 0


def test_attention_weights_refuses_bad_arguments(lib, mem):
    base = mem[1]

    def call(nq=16, nkv=2, cache=_cache(base), kv_len=base, q=base, lse=base, acc=base, T=4, ws=base,
             nbytes=64):
        d = sgp.make_heads(nq, nkv)
        return lib.sgp_attention_weights(ctypes.byref(d), ctypes.byref(cache), kv_len, q, lse, acc, T,
                                         ws, nbytes, None)
    for kw in (dict(nq=15), dict(T=0), dict(T=513), dict(cache=_cache(base, window=5)),
               dict(cache=_cache(base, k=16)),
               dict(cache=_cache(base, cap=0)), dict(cache=_cache(0)), dict(kv_len=None), dict(q=None),
               dict(q=base + 8), dict(lse=None), dict(acc=None), dict(acc=base + 2), dict(ws=None),
               dict(ws=base + 64), dict(nbytes=63)):
        assert call(**kw) == E, kw


def test_kv_evict_refuses_bad_arguments(lib, mem):
    base = mem[1]
    src = _cache(base, cap=20, k=0, v=20480)             # 4 x 2 x 20 rows of 128 bytes
    dst = _cache(base, cap=10, k=40960, v=51200)
    acc, acc_out = base + 62000, base + 64000

    def call(nkv=2, a=src, b=dst, budget=8, sink=1, recent=2, kv=base, kv_out=base, w=acc, wo=acc_out,
             kept=base, T=4, ws=base, nbytes=1 << 30, policy=True):
        d, e = sgp.make_heads(nkv, nkv), sgp.make_evict(budget, sink, recent)
        return lib.sgp_kv_evict(ctypes.byref(d), ctypes.byref(a), ctypes.byref(b),
                                ctypes.byref(e) if policy else None, kv, kv_out, w, wo, kept, T, ws,
                                nbytes, None)
    far = _cache(base, cap=20, k=4096, v=20480)
    for kw in (dict(policy=False), dict(budget=0), dict(budget=11), dict(sink=-1), dict(recent=-1),
               dict(sink=4, recent=5), dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), dict(T=0), dict(T=513),
               dict(kv=None), dict(kv_out=None), dict(w=None), dict(wo=None), dict(kept=base + 2),
               dict(ws=None), dict(nbytes=0), dict(a=_cache(0)), dict(b=_cache(base, cap=0)),
               dict(b=far), dict(b=src, wo=acc_out),                    # overlap; in place without acc
               dict(b=_cache(base, cap=19, k=0, v=20480), wo=acc),      # in place, another capacity
               dict(b=_cache(base, cap=10, k=40960, v=45000 - 45000 % 16)),  # the target's k and v
               dict(wo=acc + 4), dict(nkv=0), dict(kv_out=base + 4),
               dict(a=_cache(base, cap=20, k=16, v=20480)), dict(b=_cache(base, cap=10, k=40960, v=51216))):
        assert call(**kw) == E, kw
    d = sgp.make_heads(2, 2)
    assert sgp.sgp_kv_evict_workspace_bytes(d, 4, 8) > 4 * 2 * 8 * 4
    assert sgp.sgp_kv_evict_workspace_bytes(d, 4, 0) == 0
    assert sgp.sgp_kv_evict_workspace_bytes(d, 513, 8) == 0


def test_lora_apply_refuses_bad_arguments(lib, mem):
    base = mem[1]

    def call(n=3, i=64, o=96, r=16, a=base, b=base, scale=None, rank=None, of=base, x=base, ldx=64,
             y=base + 4096, ldy=96, z=base + 8192, ldz=96, T=4, ws=base, nbytes=64):
        p = sgp.sgp_lora(a, b, scale, rank, n, i, o, r)
        return lib.sgp_lora_apply(ctypes.byref(p), of, x, ldx, y, ldy, z, ldz, T, ws, nbytes, None)
    for kw in (dict(n=0), dict(n=4097), dict(i=48), dict(i=0), dict(o=33), dict(r=0), dict(r=12),
               dict(r=136), dict(a=None), dict(b=base + 8), dict(scale=base + 2), dict(rank=base + 1),
               dict(of=None), dict(x=None), dict(y=base + 2), dict(z=None), dict(ldx=63), dict(ldx=68),
               dict(ldy=88), dict(ldz=1 << 41), dict(T=0), dict(T=513), dict(ws=base + 8),
               dict(nbytes=32), dict(z=base + 4096 + 32), dict(z=base + 4096, ldz=104),
               dict(z=base, x=base + 128)):
        assert call(**kw) == E, kw
    assert lib.sgp_lora_apply(None, base, base, 64, base, 96, base, 96, 4, base, 64, None) == E


def test_workspace_views(lib, mem):
    d = sgp.make_dims(synth.SHAPE_GPTOSS)
    T, n = 64, sgp.sgp_workspace_bytes(d, 64, 8192)
    view = sgp.sgp_layer_dump()
    r = lib.sgp_workspace_views(ctypes.byref(d), T, 8192, mem[1], n, ctypes.byref(view))
    assert r == sgp.SGP_OK
    rows = {"a": d.hidden, "q": 4096, "o": 4096, "h": d.hidden, "u": d.hidden}
    spans = sorted((getattr(view, k), getattr(view, k) + T * w * 2) for k, w in rows.items())
    assert spans[0][0] > mem[1] and spans[-1][1] <= mem[1] + n
    assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:]))
    assert view.logits is None and view.y is None
    for args in ((0, 8192, mem[1], n), (513, 8192, mem[1], n), (T, 0, mem[1], n), (T, 8192, None, n),
                 (T, 8192, mem[1], n - 1)):
        assert lib.sgp_workspace_views(ctypes.byref(d), *args, ctypes.byref(view)) == E
    assert lib.sgp_workspace_views(ctypes.byref(d), T, 8192, mem[1], n, None) == E


def test_binding_refuses_what_the_abi_cannot_see(lib):
    """Types, sizes, layouts and devices, before any pointer is passed on."""
    f = torch.zeros(2, 2, 8, 64)
    with pytest.raises(ValueError):
        sgp.make_cache(f, f)                                   # not bf16
    with pytest.raises(ValueError):
        sgp.make_cache(f.bfloat16(), f.bfloat16()[:, :, :4])   # shapes differ
    with pytest.raises(ValueError):
        sgp.make_lora(torch.zeros(2, 16, 64), torch.zeros(2, 96, 8))
    with pytest.raises(ValueError):
        sgp.make_cache(f.bfloat16(), f.bfloat16())             # not on a GPU


def test_oracle_against_a_second_formulation():
    """The bounds' oracle itself: softmax over the joined positions, a window, an empty row."""
    rng = np.random.default_rng(3)
    q, k, v = (rng.standard_normal(s) for s in ((4, 64), (9, 64), (9, 64)))
    o, lse, eo, el = S.attention(q, k, v, 2)
    for h in range(4):
        e = [np.exp(np.dot(q[h], k[p]) / 8.0) for p in range(2, 9)]
        assert abs(lse[h] - np.log(sum(e))) < 1e-12
        assert np.allclose(o[h], sum(w * v[p] for w, p in zip(e, range(2, 9))) / sum(e), atol=1e-12)
    assert (eo > 0).all() and (el > 0).all()
    o, lse, _, _ = S.attention(q, k, v, 9)
    assert not o.any() and np.isneginf(lse).all()
    add, _ = S.attention_weights(q[None], k[None, None], [9], S.attention(q, k, v, 0)[1][None])
    assert np.allclose(add.sum(), 4.0)
    nan = float("nan")
    assert S.evict(np.array([0, nan, 3, 3, -0.0, 3, 9, 0]), 8, 5, 1, 1).tolist() == [0, 2, 3, 6, 7]
    assert S.evict(np.array([0, nan, -np.inf, nan]), 4, 3, 0, 1).tolist() == [0, 2, 3]
    assert S.evict(np.zeros(6), 6, 3, 0, 0).tolist() == [0, 1, 2]
    assert S.evict(np.zeros(3), 3, 5, 0, 0).tolist() == [0, 1, 2]
    x, y = rng.standard_normal((2, 64)), rng.standard_normal((2, 32))
    a, b = rng.standard_normal((1, 8, 64)), rng.standard_normal((1, 32, 8))
    out, err = S.lora(x, y, a, b, [2.0], [3], [0, -1])
    assert np.allclose(out[0], y[0] + 2 * sum(b[0, :, r] * (a[0, r] @ x[0]) for r in range(3)))
    assert (out[1] == y[1]).all() and not err[1].any()
