"""Host-side argument checks of the entry points around long caches (several axes, 4-bit caches, gathered
weights, eviction): every call is refused, or has nothing to do, before any launch (no GPU)."""
import ctypes

import pytest

from paged_kv_decode_21_gb300 import build as pkd_build

FAKE = ctypes.c_void_p(1 << 20)          # aligned, never dereferenced on the failing paths
ODD = ctypes.c_void_p((1 << 20) + 2)
F = ctypes.c_float


@pytest.fixture(scope="module")
def L():
    pkd_build.build()
    from paged_kv_decode_21_gb300 import ops
    return ops.lib()


@pytest.mark.parametrize("kind", ["fp16", "fp8", "int4"])
def test_append(L, kind):
    def call(q=FAKE, k=FAKE, v=FAKE, qs=1024, ks=256, vs=256, tab=FAKE, ax=FAKE, st=FAKE, pos=FAKE, bt=FAKE, cl=FAKE,
             qo=FAKE, os_=1024, kc=FAKE, vc=FAKE, T=4, B=2, A=3, Hq=8, Hkv=2, D=128, R=128, il=0, MP=64, BS=16, NB=4,
             MB=2, s=1.0, s2=1.0, err=None):
        a = (q, k, v, qs, ks, vs, tab, ax, st, pos, bt, cl, qo, os_, kc, vc, T, B, A, Hq, Hkv, D, R, il, MP, BS, NB, MB)
        if kind == "fp16":
            return L.paged_kv_append_rope_axes(*a, err, None)
        fn = L.paged_kv_append_rope_axes_fp8 if kind == "fp8" else L.paged_kv_append_rope_int4
        return fn(*a, F(s), F(s2), err, None)
    assert call(T=0) == 0 and call(B=0) == 0
    assert call(T=-1) == 2 and call(B=-1) == 2 and call(Hkv=0) == 2 and call(BS=0) == 2 and call(NB=0) == 2
    assert call(D=120) == 2 and call(D=528, ks=2000, vs=2000, qs=9000, os_=9000) == 2
    assert call(R=8) == 2 and call(R=144) == 2 and call(MP=0) == 2
    assert call(A=0) == 2 and call(A=9) == 3
    assert call(st=None, T=5) == 2
    assert call(qs=1016) == 2 and call(ks=248) == 2 and call(os_=0) == 2
    assert call(qs=1028) == 4 and call(ks=260) == 4
    for name in ("k", "v", "bt", "cl", "kc", "vc", "q", "qo", "tab", "ax", "pos"):
        if kind == "int4" and name in ("ax", "pos"):
            continue
        assert call(**{name: None}) == 1, name
        assert call(**{name: ODD}) == 4, name
    assert call(st=ODD) == 4 and call(err=ODD) == 4 and call(ax=ctypes.c_void_p((1 << 20) + 8)) == 4
    if kind != "fp16":
        for bad in (0.0, -1.0, float("inf"), float("nan")):
            assert call(s=bad) == 2 and call(s2=bad) == 2
    if kind == "int4":
        assert call(ax=None) == 3                              # three axes, and nothing says which pair goes by which
        assert call(pos=None) == 1 and call(ax=None, pos=None, A=1, k=None) == 1
        assert call(D=256, ks=512, vs=512, qs=2048, os_=2048) == 3 and call(D=32, R=32) == 3
        assert call(R=48) == 3 and call(BS=8) == 3


def test_read(L):
    def call(kc=FAKE, vc=FAKE, bt=FAKE, sl=FAKE, st=FAKE, ko=FAKE, vo=FAKE, ks=256, vs=256, T=4, B=2, Hkv=2, D=128,
             BS=16, NB=4, MB=2, s=1.0, s2=1.0, err=None):
        return L.paged_kv_read_int4(kc, vc, bt, sl, st, ko, vo, ks, vs, T, B, Hkv, D, BS, NB, MB, F(s), F(s2), err, None)
    assert call(T=0) == 0 and call(B=0) == 0
    assert call(T=-1) == 2 and call(B=-1) == 2 and call(Hkv=0) == 2 and call(NB=0) == 2 and call(MB=0) == 2
    assert call(D=96) == 3 and call(BS=8) == 3 and call(st=None, T=5) == 2
    assert call(ks=248) == 2 and call(vs=0) == 2 and call(ks=260) == 4 and call(s=0.0) == 2 and call(s2=float("nan")) == 2
    for name in ("kc", "vc", "bt", "sl", "ko", "vo"):
        assert call(**{name: None}) == 1 and call(**{name: ODD}) == 4, name
    assert call(st=ODD) == 4 and call(err=ODD) == 4


def test_decode(L):
    def call(p=None, B=2, QL=1, Hq=8, Hkv=2, D=128, BS=16, NB=64, MB=64, mc=1000, scale=0.1, ks=1.0, vs=1.0, P=0,
             ws=FAKE, wsb=1 << 30, err=None):
        ptrs = [FAKE] * 6
        for i, x in (p or {}).items():
            ptrs[i] = x
        return L.paged_decode_attention_int4(*ptrs, B, QL, Hq, Hkv, D, BS, NB, MB, mc, F(scale), F(ks), F(vs), P, ws,
                                             wsb, err, None)
    assert call(B=0) == 0
    assert call(B=-1) == 2 and call(QL=0) == 2 and call(Hq=7) == 2 and call(mc=-1) == 2 and call(mc=1025) == 2
    assert call(Hq=18) == 3 and call(D=96) == 3 and call(BS=8) == 3
    assert call(scale=float("inf")) == 2 and call(ks=0.0) == 2 and call(vs=float("nan")) == 2
    assert call(P=48) == 2 and call(P=-2) == 2 and call(P=16) == 2 and call(QL=1 << 29) == 2
    assert call(mc=(1 << 30) + 1, MB=1 << 27) == 2
    for i in range(6):
        assert call(p={i: None}) == 1 and call(p={i: ODD}) == 4, i
    assert call(err=ODD) == 4
    size = L.paged_decode_int4_workspace_size(2, 1, 8, 2, 128, 16, 1000, 0)
    assert size > 0 and call(ws=None) == 5 and call(wsb=size - 1) == 5 and call(ws=ctypes.c_void_p((1 << 20) + 16)) == 4
    assert L.paged_decode_int4_workspace_size(2, 1, 8, 2, 128, 16, 1000, -1) == 0
    assert L.paged_decode_int4_workspace_size(2, 1, 8, 2, 128, 16, 100, 0) == 0       # nothing splits
    assert L.paged_decode_int4_workspace_size(2, 0, 8, 2, 128, 16, 1000, 0) == 0
    assert L.paged_decode_int4_workspace_size(2, 1, 8, 2, 96, 16, 1000, 0) == 0


def test_weights(L):
    def call(p=None, B=2, QL=1, Hq=8, Hkv=2, D=128, BS=16, NB=64, MB=64, mc=1000, scale=0.1, ks=1.0, decay=1.0, kind=0,
             ws=FAKE, wsb=1 << 30, err=None):
        ptrs = [FAKE] * 6
        for i, x in (p or {}).items():
            ptrs[i] = x
        return L.paged_kv_attention_weights(*ptrs, B, QL, Hq, Hkv, D, BS, NB, MB, mc, F(scale), F(ks), F(decay), kind, ws,
                                            wsb, err, None)
    assert call(B=0) == 0 and call(mc=0) == 0
    assert call(B=-1) == 2 and call(QL=0) == 2 and call(Hq=7) == 2 and call(mc=-1) == 2 and call(mc=1025) == 2
    assert call(NB=0) == 2 and call(MB=0) == 2 and call(mc=(1 << 30) + 1, MB=1 << 27) == 2 and call(QL=1 << 29) == 2
    assert call(Hq=18) == 3 and call(D=96) == 3 and call(BS=8) == 3 and call(kind=3) == 2 and call(kind=-1) == 2
    assert call(scale=float("nan")) == 2 and call(ks=0.0) == 2
    for bad in (-0.5, 1.5, float("nan")):
        assert call(decay=bad) == 2
    for i in range(6):
        assert call(p={i: ODD}) == 4, i
        if i != 4:                                             # start_lens may be left out
            assert call(p={i: None}) == 1, i
    assert call(p={4: None}, ws=None) == 5
    assert call(err=ODD) == 4
    size = L.paged_kv_attention_weights_workspace_size(2, 1, 8, 2, 128, 16, 1000)
    assert size > 0 and call(ws=None) == 5 and call(wsb=size - 1) == 5 and call(ws=ctypes.c_void_p((1 << 20) + 16)) == 4
    assert L.paged_kv_attention_weights_workspace_size(0, 1, 8, 2, 128, 16, 1000) == 0
    assert L.paged_kv_attention_weights_workspace_size(2, 1, 8, 2, 96, 16, 1000) == 0


def test_select(L):
    def call(p=None, B=2, Hkv=2, BS=16, NB=64, MB=8, mc=100, K=8, sink=1, rec=2, err=None):
        ptrs = [FAKE] * 5
        for i, x in (p or {}).items():
            ptrs[i] = x
        return L.paged_kv_token_select(*ptrs, B, Hkv, BS, NB, MB, mc, K, sink, rec, err, None)
    assert call(B=0) == 0
    assert call(B=-1) == 2 and call(Hkv=0) == 2 and call(BS=0) == 2 and call(NB=0) == 2 and call(MB=0) == 2
    assert call(mc=129) == 2 and call(K=0) == 2 and call(sink=-1) == 2 and call(rec=-1) == 2 and call(sink=7) == 2
    assert call(B=1 << 30, Hkv=4) == 2
    for i in range(5):
        assert call(p={i: None}) == 1 and call(p={i: ODD}) == 4, i
    assert call(err=ODD) == 4


def test_compact(L):
    def call(p=None, B=2, Hkv=2, D=128, BS=16, NB=64, MB=8, K=8, MN=2, kind=0, err=None):
        ptrs = [FAKE] * 8
        for i, x in (p or {}).items():
            ptrs[i] = x
        return L.paged_kv_compact(*ptrs, B, Hkv, D, BS, NB, MB, K, MN, kind, err, None)
    assert call(B=0) == 0
    assert call(B=-1) == 2 and call(Hkv=0) == 2 and call(NB=0) == 2 and call(MB=0) == 2 and call(K=0) == 2 and call(MN=0) == 2
    assert call(D=96) == 3 and call(BS=8) == 3 and call(kind=3) == 2 and call(kind=-1) == 2
    for i in range(8):
        assert call(p={i: ODD}) == 4, i
        if i != 2:                                             # weights may be left out
            assert call(p={i: None}) == 1, i
    assert call(p={2: None, 3: None}) == 1 and call(err=ODD) == 4


def test_counts_past_32_bits_are_refused(L):
    big = (1 << 30) + 1
    sel = lambda K=8, mc=100, MB=1 << 27: L.paged_kv_token_select(*[FAKE] * 5, 2, 2, 16, 64, MB, mc, K, 0, 0, None, None)  # noqa: E731
    assert sel(K=big) == 2 and sel(mc=big) == 2
    assert L.paged_kv_compact(*[FAKE] * 8, 2, 2, 128, 16, 64, 8, big, 2, 0, None, None) == 2
