"""Host-side argument checks of the serving-step entry points (no GPU: every call is refused, or has
nothing to do, before any launch)."""
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


@pytest.mark.parametrize("fp8", [False, True])
def test_append_rope(L, fp8):
    def call(q=FAKE, k=FAKE, v=FAKE, qs=1024, ks=256, vs=256, tab=FAKE, st=FAKE, pos=None, bt=FAKE, cl=FAKE, qo=FAKE,
             os_=1024, kc=FAKE, vc=FAKE, T=4, B=2, Hq=8, Hkv=2, D=128, R=128, il=0, MP=64, BS=16, NB=4, MB=2, s=1.0,
             err=None):
        a = (q, k, v, qs, ks, vs, tab, st, pos, bt, cl, qo, os_, kc, vc, T, B, Hq, Hkv, D, R, il, MP, BS, NB, MB)
        return L.paged_kv_append_rope_fp8(*a, F(s), F(1.0), err, None) if fp8 else L.paged_kv_append_rope(*a, err, None)
    assert call(T=0) == 0 and call(B=0) == 0
    assert call(T=-1) == 2 and call(B=-1) == 2 and call(Hkv=0) == 2 and call(BS=0) == 2 and call(NB=0) == 2
    assert call(D=120) == 2 and call(D=528, ks=2000, vs=2000, qs=9000, os_=9000) == 2    # a multiple of 16, up to 512
    assert call(R=8) == 2 and call(R=144) == 2 and call(MP=0) == 2
    assert call(st=None, T=5) == 2                                    # runs of one length need a whole number
    assert call(qs=1016) == 2 and call(ks=248) == 2 and call(os_=0) == 2   # a token's heads do not fit
    assert call(qs=1028) == 4 and call(ks=260) == 4                   # 16-byte steps
    assert call(qs=2048) == 2                                         # in place, rows would meet other tokens'
    for name in ("k", "v", "bt", "cl", "kc", "vc", "q", "qo", "tab"):
        assert call(**{name: None}) == 1, name
        assert call(**{name: ODD}) == 4, name
    assert call(st=ODD) == 4 and call(pos=ODD) == 4 and call(err=ODD) == 4
    if fp8:
        assert call(s=0.0) == 2 and call(s=float("inf")) == 2


@pytest.mark.parametrize("fp8", [False, True])
def test_prefix(L, fp8):
    def call(p=None, B=4, QL=1, Y=2, Hq=8, Hkv=2, D=128, BS=16, NB=64, MP=8, MB=8, mp=100, mc=100, scale=0.1, ks=1.0,
             ws=FAKE, wsb=1 << 30, err=None):
        ptrs = [FAKE] * 9
        for i, x in (p or {}).items():
            ptrs[i] = x
        a = (*ptrs, B, QL, Y, Hq, Hkv, D, BS, NB, MP, MB, mp, mc, F(scale))
        if fp8:
            return L.paged_decode_attention_prefix_fp8(*a, F(ks), F(1.0), ws, wsb, err, None)
        return L.paged_decode_attention_prefix(*a, ws, wsb, err, None)
    assert call(B=0) == 0
    assert call(B=-1) == 2 and call(QL=0) == 2 and call(Y=-1) == 2 and call(mp=-1) == 2
    assert call(mp=129) == 2 and call(mc=129) == 2 and call(MP=0) == 2
    assert call(mp=(1 << 30) + 1, MP=1 << 27) == 2 and call(mc=(1 << 30) + 1, MB=1 << 27) == 2
    assert call(QL=1 << 29) == 2                                      # rows past 32 bits
    assert call(Hq=7) == 2 and call(Hq=18) == 3 and call(D=96) == 3 and call(BS=8) == 3
    assert call(scale=float("nan")) == 2
    for i in range(9):
        assert call(p={i: None}) == 1, i
        assert call(p={i: ODD}) == 4, i
    assert call(err=ODD) == 4
    assert call(ws=None) == 5 and call(wsb=100) == 5 and call(ws=ctypes.c_void_p((1 << 20) + 16)) == 4
    if fp8:
        assert call(ks=-1.0) == 2
    size = L.paged_decode_prefix_workspace_size(4, 1, 8, 2, 128, 16, 2, 100, 100)
    assert size > 0 and call(wsb=size // 4) == 5
    assert L.paged_decode_prefix_workspace_size(4, 1, 8, 2, 128, 16, 0, 0, 0) == 0
    assert L.paged_decode_prefix_workspace_size(4, 0, 8, 2, 128, 16, 2, 100, 100) == 0
    assert L.paged_decode_prefix_workspace_size(4, 1, 8, 2, 128, 16, 2, (1 << 30) + 1, 100) == 0
    assert L.paged_decode_prefix_workspace_size(4, 1 << 29, 8, 2, 128, 16, 2, 100, 100) == 0
    # groups past the batch's sequences are empty: they cost no workspace, and their number no overflow
    assert (L.paged_decode_prefix_workspace_size(4, 1, 8, 2, 128, 16, 0x7fffffff, 100, 100)
            == L.paged_decode_prefix_workspace_size(4, 1, 8, 2, 128, 16, 4, 100, 100))


def test_bounds(L):
    def call(k=FAKE, bt=FAKE, cl=FAKE, st=None, bo=FAKE, B=2, Hkv=2, D=128, BS=16, NB=64, MB=8, mt=100, f8=0, err=None):
        return L.paged_kv_block_bounds(k, bt, cl, st, bo, B, Hkv, D, BS, NB, MB, mt, f8, err, None)
    assert call(B=0) == 0 and call(mt=0) == 0
    assert call(mt=-1) == 2 and call(B=-1) == 2 and call(MB=0) == 2 and call(D=96) == 3 and call(BS=8) == 3
    for name in ("k", "bt", "cl", "bo"):
        assert call(**{name: None}) == 1 and call(**{name: ODD}) == 4, name
    assert call(st=ODD) == 4 and call(err=ODD) == 4


def test_select(L):
    def call(p=None, B=2, Hq=8, Hkv=2, D=128, BS=16, NB=64, MB=8, mc=100, K=4, sink=1, rec=1, f8=0, err=None):
        ptrs = [FAKE] * 6
        for i, x in (p or {}).items():
            ptrs[i] = x
        return L.paged_kv_block_select(*ptrs, B, Hq, Hkv, D, BS, NB, MB, mc, K, sink, rec, f8, err, None)
    assert call(B=0) == 0
    assert call(K=0) == 2 and call(sink=-1) == 2 and call(sink=3, rec=2) == 2 and call(mc=129) == 2 and call(Hq=7) == 2
    assert call(Hq=18) == 3 and call(D=96) == 3 and call(BS=8) == 3
    assert call(MB=50000, mc=49152 * 16 + 1) == 3
    for i in range(6):
        assert call(p={i: None}) == 1 and call(p={i: ODD}) == 4, i
    assert call(err=ODD) == 4


@pytest.mark.parametrize("fp8", [False, True])
def test_blocks(L, fp8):
    def call(p=None, B=2, Hq=8, Hkv=2, D=128, BS=16, NB=64, MB=8, K=64, scale=0.1, ks=1.0, ws=FAKE, wsb=1 << 30, err=None):
        ptrs = [FAKE] * 8
        for i, x in (p or {}).items():
            ptrs[i] = x
        a = (*ptrs, B, Hq, Hkv, D, BS, NB, MB, K, F(scale))
        if fp8:
            return L.paged_decode_attention_blocks_fp8(*a, F(ks), F(1.0), ws, wsb, err, None)
        return L.paged_decode_attention_blocks(*a, ws, wsb, err, None)
    assert call(B=0) == 0
    assert call(K=0) == 2 and call(MB=0) == 2 and call(Hq=7) == 2 and call(scale=float("inf")) == 2
    assert call(K=1 << 28) == 2 and call(K=(1 << 26) + 1) == 2
    assert call(Hq=18) == 3 and call(D=96) == 3 and call(BS=8) == 3
    for i in range(8):
        assert call(p={i: None}) == 1 and call(p={i: ODD}) == 4, i
    assert call(err=ODD) == 4
    if fp8:
        assert call(ks=0.0) == 2
    size = L.paged_decode_blocks_workspace_size(2, 8, 2, 128, 16, 64)
    assert size > 0 and call(ws=None) == 5 and call(wsb=size // 4) == 5
    assert L.paged_decode_blocks_workspace_size(2, 8, 2, 128, 16, 4) == 0    # nothing splits
    assert L.paged_decode_blocks_workspace_size(2, 8, 2, 96, 16, 64) == 0
