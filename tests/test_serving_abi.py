"""ttt_attention_paged, ttt_add_rms_norm, ttt_gated_delta_packed and ttt_gated_delta_decode refuse bad arguments on the host, before anything is enqueued
(no GPU: every call below fails validation), and report their workspaces."""
import pytest

import chunked_weight_sequence_amd as ttt

OK, E_NULL, E_SHAPE, E_DTYPE, E_ALIGN, E_WS, E_UNSUP, E_LAUNCH, E_ALIAS = range(9)
A = 0x7F0000000000          # fake, 16-byte aligned device addresses (never dereferenced)
MB = 1 << 20
F32, BF16 = 0, 1
INF, NAN = float("inf"), float("nan")


def norm(**kw):
    a = dict(X=A, xs=2560, R=A + 64 * MB, rs=2560, dt=BF16, w=A + 128 * MB, eps=1e-6, S=A + 192 * MB, ss=2560,
             Y=A + 256 * MB, ys=2560, sc=None, group=0, N=1000, D=2560)
    a.update(kw)
    return ttt.lib().ttt_add_rms_norm(a["X"], a["xs"], a["R"], a["rs"], a["dt"], a["w"], a["eps"], a["S"], a["ss"],
                                      a["Y"], a["ys"], a["sc"], a["group"], a["N"], a["D"], None)


SC = A + 320 * MB


@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), E_DTYPE), (dict(X=None), E_NULL), (dict(Y=None), E_NULL), (dict(N=0), E_SHAPE),
    (dict(N=(1 << 30) + 1), E_SHAPE), (dict(D=0), E_SHAPE), (dict(D=2556), E_SHAPE),
    (dict(D=16392, xs=16392, rs=16392, ss=16392, ys=16392), E_SHAPE), (dict(eps=-1.0), E_SHAPE),
    (dict(eps=NAN), E_SHAPE), (dict(eps=INF), E_SHAPE), (dict(xs=2552), E_SHAPE), (dict(rs=2564), E_SHAPE),
    (dict(ss=0), E_SHAPE), (dict(ys=-2560), E_SHAPE), (dict(ys=(1 << 31) + 8), E_SHAPE),
    (dict(group=128), E_SHAPE),                                              # without scales
    (dict(sc=SC, group=8), E_SHAPE), (dict(sc=SC, group=1024), E_SHAPE), (dict(sc=SC, group=96), E_SHAPE),
    (dict(sc=SC, group=-128), E_SHAPE), (dict(sc=SC, group=512, D=2304), E_SHAPE), (dict(sc=SC, ys=2564), E_SHAPE),
    (dict(X=A + 8), E_ALIGN), (dict(w=A + 128 * MB + 4), E_ALIGN), (dict(Y=A + 256 * MB + 8), E_ALIGN),
    (dict(sc=SC + 4), E_ALIGN),
    (dict(S=A + 16), E_ALIAS), (dict(S=A, ss=2568), E_ALIAS), (dict(Y=A + 64 * MB + 5120), E_ALIAS),
    (dict(Y=A + 192 * MB), E_ALIAS), (dict(S=A, Y=A), E_ALIAS), (dict(sc=SC, Y=A), E_ALIAS),
    (dict(sc=A + 256 * MB), E_ALIAS), (dict(sc=A + 64 * MB), E_ALIAS), (dict(S=A + 128 * MB), E_ALIAS),
])
def test_norm_rejects_bad_arguments(kw, code):
    assert norm(**kw) == code


def step(**kw):
    a = dict(Q=A, qs=2048, K=A + 64 * MB, ks=2048, V=A + 128 * MB, vs=4096, dt=BF16, g=A + 192 * MB,
             b=A + 193 * MB, O=A + 256 * MB, os=4096, si=A + 1024 * MB, so=A + 4096 * MB, sl=A + 320 * MB,
             n=100, S=64, Hk=16, Hv=32, dk=128, dv=128, scale=0.1, norm=1, eps=1e-6)
    a.update(kw)
    return ttt.lib().ttt_gated_delta_decode(
        a["Q"], a["qs"], a["K"], a["ks"], a["V"], a["vs"], a["dt"], a["g"], a["b"], a["O"], a["os"], a["si"],
        a["so"], a["sl"], a["n"], a["S"], a["Hk"], a["Hv"], a["dk"], a["dv"], a["scale"], a["norm"], a["eps"], None)


DELTA = [
    (dict(dt=7), E_DTYPE), (dict(dt=F32), E_UNSUP), (dict(Q=None), E_NULL), (dict(K=None), E_NULL),
    (dict(V=None), E_NULL), (dict(g=None), E_NULL), (dict(b=None), E_NULL), (dict(O=None), E_NULL),
    (dict(S=0), E_SHAPE), (dict(Hk=0), E_SHAPE), (dict(Hv=0), E_SHAPE), (dict(Hk=5), E_SHAPE),
    (dict(dk=0), E_SHAPE), (dict(dv=-64), E_SHAPE), (dict(dk=96), E_UNSUP), (dict(dv=32, vs=1024, os=1024), E_UNSUP),
    (dict(dv=576, vs=32 * 576, os=32 * 576), E_UNSUP), (dict(scale=NAN), E_SHAPE), (dict(eps=-1e-6), E_SHAPE),
    (dict(eps=INF), E_SHAPE), (dict(qs=2040), E_SHAPE), (dict(ks=2052), E_SHAPE), (dict(vs=4088), E_SHAPE),
    (dict(os=(1 << 31) + 8), E_SHAPE), (dict(n=0), E_SHAPE), (dict(n=1 << 31), E_SHAPE),
    (dict(Q=A + 2), E_ALIGN), (dict(g=A + 192 * MB + 4), E_ALIGN), (dict(si=A + 1024 * MB + 8), E_ALIGN),
    (dict(sl=A + 320 * MB + 4), E_ALIGN), (dict(O=A + 128 * MB), E_ALIAS), (dict(O=A), E_ALIAS),
    (dict(so=A + 1024 * MB + 64), E_ALIAS), (dict(so=A + 256 * MB), E_ALIAS), (dict(so=A + 192 * MB), E_ALIAS),
    (dict(O=A + 1024 * MB), E_ALIAS), (dict(sl=A + 4096 * MB), E_ALIAS),
]


@pytest.mark.parametrize("kw,code", DELTA + [
    (dict(sl=None, n=63), E_SHAPE), (dict(S=1 << 20, Hk=8, Hv=8), E_SHAPE)])
def test_step_rejects_bad_arguments(kw, code):
    assert step(**kw) == code


def delta(**kw):
    a = dict(Q=A, qs=2048, K=A + 64 * MB, ks=2048, V=A + 128 * MB, vs=4096, dt=BF16, g=A + 192 * MB,
             b=A + 193 * MB, O=A + 256 * MB, os=4096, si=A + 1024 * MB, so=A + 4096 * MB, sl=A + 320 * MB,
             n=100, cu=A + 321 * MB, S=64, N=1000, Hk=16, Hv=32, dk=128, dv=128, scale=0.1, norm=1, eps=1e-6,
             ws=A + 8192 * MB, wsb=None)
    a.update(kw)
    need = ttt.lib().ttt_gated_delta_packed_workspace(a["S"], a["N"], a["Hk"], a["Hv"], a["dk"], a["dv"])
    a["wsb"] = need if a["wsb"] is None else a["wsb"]
    return ttt.lib().ttt_gated_delta_packed(
        a["Q"], a["qs"], a["K"], a["ks"], a["V"], a["vs"], a["dt"], a["g"], a["b"], a["O"], a["os"], a["si"],
        a["so"], a["sl"], a["n"], a["cu"], a["S"], a["N"], a["Hk"], a["Hv"], a["dk"], a["dv"], a["scale"],
        a["norm"], a["eps"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", DELTA + [
    (dict(cu=None), E_NULL), (dict(N=0), E_SHAPE), (dict(N=(1 << 26) + 1), E_SHAPE), (dict(sl=None, n=63), E_SHAPE),
    (dict(N=1 << 25), E_SHAPE), (dict(qs=(1 << 23) + 8), E_SHAPE), (dict(os=(1 << 23) + 8), E_SHAPE),
    (dict(ws=None), E_WS), (dict(wsb=100), E_WS), (dict(cu=A + 321 * MB + 4), E_ALIGN), (dict(ws=A + 8192 * MB + 8), E_ALIGN),
    (dict(cu=A + 256 * MB), E_ALIAS), (dict(ws=A), E_ALIAS), (dict(ws=A + 1024 * MB), E_ALIAS), (dict(ws=A + 256 * MB), E_ALIAS)])
def test_packed_delta_rejects_bad_arguments(kw, code):
    assert delta(**kw) == code


def test_packed_delta_workspace():
    W = ttt.lib().ttt_gated_delta_packed_workspace
    assert W(0, 64, 1, 1, 64, 64) == 0 and W(1, 64, 1, 1, 96, 64) == 0 and W(1, 64, 1, 1, 64, 32) == 0
    assert W(1, 64, 2, 2, 64, 64) == 2 * W(1, 64, 1, 1, 64, 64) > 0
    assert W(1, 32768, 32, 32, 128, 128) <= 513 * 32 * 25600


def paged(**kw):
    a = dict(Q=A, qs=None, Kc=A + 64 * MB, Vc=A + 96 * MB, dt=BF16, O=A + 128 * MB, os=None, lse=A + 192 * MB,
             cu=A + 200 * MB, tab=A + 208 * MB, mp=64, page=16, np=512, lens=A + 216 * MB, n=8, Nq=300, Hq=16, Hkv=4,
             dh=64, scale=0.1, window=0, ws=A + 512 * MB, wsb=None)
    a.update(kw)
    for k in ("qs", "os"):
        a[k] = a["Hq"] * a["dh"] if a[k] is None else a[k]
    need = ttt.lib().ttt_attention_paged_workspace(a["n"], a["Nq"], a["mp"], a["page"], a["Hq"], a["Hkv"], a["dh"])
    a["wsb"] = need if a["wsb"] is None else a["wsb"]
    return ttt.lib().ttt_attention_paged(
        a["Q"], a["qs"], a["Kc"], a["Vc"], a["dt"], a["O"], a["os"], a["lse"], a["cu"], a["tab"], a["mp"], a["page"],
        a["np"], a["lens"], a["n"], a["Nq"], a["Hq"], a["Hkv"], a["dh"], a["scale"], a["window"], a["ws"], a["wsb"],
        None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), E_DTYPE), (dict(dt=F32), E_UNSUP), (dict(Q=None), E_NULL), (dict(Kc=None), E_NULL),
    (dict(Vc=None), E_NULL), (dict(O=None), E_NULL), (dict(cu=None), E_NULL), (dict(tab=None), E_NULL),
    (dict(lens=None), E_NULL), (dict(n=0), E_SHAPE), (dict(n=(1 << 20) + 1), E_SHAPE), (dict(Nq=0), E_SHAPE),
    (dict(Nq=(1 << 26) + 1), E_SHAPE), (dict(Hq=15), E_SHAPE), (dict(Hkv=0), E_SHAPE), (dict(mp=0), E_SHAPE),
    (dict(mp=1 << 27), E_SHAPE), (dict(np=0), E_SHAPE), (dict(np=1 << 30, page=128), E_SHAPE),
    (dict(window=-1), E_SHAPE), (dict(window=(1 << 30) + 1), E_SHAPE), (dict(scale=0.0), E_SHAPE),
    (dict(scale=INF), E_SHAPE), (dict(Nq=1 << 26, Hq=32, Hkv=4), E_SHAPE), (dict(dh=96), E_UNSUP),
    (dict(page=24), E_UNSUP), (dict(page=8), E_UNSUP), (dict(page=1 << 17), E_UNSUP), (dict(qs=1016), E_SHAPE),
    (dict(os=1028), E_SHAPE), (dict(Q=A + 2), E_ALIGN), (dict(tab=A + 208 * MB + 4), E_ALIGN),
    (dict(O=A), E_ALIAS), (dict(O=A + 64 * MB), E_ALIAS), (dict(lse=A + 128 * MB), E_ALIAS),
    (dict(lse=A + 216 * MB), E_ALIAS), (dict(O=A + 96 * MB + 1024), E_ALIAS),
])
def test_paged_rejects_bad_arguments(kw, code):
    assert paged(**kw) == code


def test_paged_workspace():
    L = ttt.lib().ttt_attention_paged_workspace
    assert L(0, 16, 4, 16, 8, 8, 64) == 0 and L(1, 16, 4, 24, 8, 8, 64) == 0 and L(1, 16, 4, 16, 8, 8, 96) == 0
    assert L(1, 32768, 512, 64, 32, 8, 128) == 0      # row tiles enough
    need = L(1, 64, 512, 64, 32, 8, 128)              # few rows, many keys: partial results of each piece
    assert need > 0 and need % (64 * 32 * 130 * 4) == 0
    big = dict(n=1, Nq=64, mp=512, page=64, Hq=32, Hkv=8, dh=128)
    assert paged(**big, wsb=need - 1) == E_WS and paged(**big, ws=None) == E_WS
    assert paged(**big, ws=A) == E_ALIAS
