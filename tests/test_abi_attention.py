"""CPU-side checks of apex4_rope and the kv4 calls: every refusal happens on the host, before any
HIP call and before a pointer is used; and of the host implementation that the GPU tests use."""
import numpy as np
import pytest

import attention_ref as ref
from w4a4_group_quantized_amd import apex4

OK, INVALID, UNSUPPORTED, ALIGN, WORKSPACE = 0, 1, 2, 3, 4
A, B, C, D, E, F = (0x10000 * i for i in range(1, 7))      # fake aligned device addresses: never dereferenced
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(apex4.LIB_PATH):
        pytest.skip("libapex4.so not built (run __graft_entry__.build())")
    return apex4.lib()


def rope(L, x=A, type=1, T=4, H=8, dim=128, ldx=1024, pos=B, freqs=C, R=128, inter=0, scale=1.0, y=D, ldy=1024):
    return L.apex4_rope(x, type, T, H, dim, ldx, pos, freqs, R, inter, scale, y, ldy, None)


def test_rope_refusals(L):
    for bad in (dict(T=-1), dict(T=2 ** 24 + 1), dict(H=0), dict(H=1025, ldx=2 ** 20, ldy=2 ** 20), dict(dim=0),
                dict(dim=72), dict(dim=1040, H=1, ldx=2048, ldy=2048), dict(R=0), dict(R=8), dict(R=24), dict(R=144),
                dict(ldx=1016), dict(ldy=1016), dict(ldx=2 ** 32), dict(scale=INF), dict(scale=NAN), dict(x=None),
                dict(y=None), dict(pos=None), dict(freqs=None)):
        assert rope(L, **bad) == INVALID, bad
    assert rope(L, type=3) == UNSUPPORTED
    for bad in (dict(x=A + 8), dict(y=D + 4), dict(pos=B + 4), dict(freqs=C + 4), dict(ldx=1028), dict(ldy=1025)):
        assert rope(L, **bad) == ALIGN, bad
    assert rope(L, T=0, x=None, y=None, pos=None, freqs=None) == OK
    assert rope(L, T=0, R=8) == INVALID


def append(L, q=A, k=B, v=C, type=1, T=4, Hq=8, Hkv=2, dim=128, ldq=1024, ldk=256, ldv=256, pos=D, freqs=E, R=128,
           inter=0, scale=1.0, slots=F, pages=9, page=64, kc=A, ks=B, vc=C, vs=D, qo=E):
    return L.apex4_kv4_append(q, k, v, type, T, Hq, Hkv, dim, ldq, ldk, ldv, pos, freqs, R, inter, scale, slots, pages,
                              page, kc, ks, vc, vs, qo, None)


PLAIN = dict(q=None, Hq=0, qo=None, pos=None, freqs=None, R=0)


def test_append_refusals(L):
    for bad in (dict(T=-1), dict(T=2 ** 24 + 1), dict(Hq=-1), dict(Hq=1025, ldq=2 ** 20), dict(Hkv=0), dict(Hkv=1025),
                dict(pages=0), dict(pages=2 ** 31), dict(page=0), dict(dim=0), dict(R=8), dict(R=144), dict(R=20),
                dict(ldq=1000), dict(ldk=248), dict(ldv=248), dict(scale=INF), dict(k=None), dict(v=None),
                dict(slots=None), dict(kc=None), dict(ks=None), dict(vc=None), dict(vs=None), dict(q=None),
                dict(qo=None), dict(pos=None), dict(freqs=None), dict(Hq=0), dict(R=0),
                dict(PLAIN, q=A), dict(PLAIN, qo=A), dict(PLAIN, pos=D), dict(PLAIN, R=64), dict(PLAIN, Hq=8, q=A, qo=A)):
        assert append(L, **bad) == INVALID, bad
    for bad in (dict(type=0), dict(type=3), dict(dim=96), dict(dim=512), dict(page=8), dict(page=48), dict(page=2048)):
        assert append(L, **bad) == UNSUPPORTED, bad
    for bad in (dict(q=A + 8), dict(k=B + 2), dict(v=C + 8), dict(qo=E + 8), dict(slots=F + 4), dict(pos=D + 4),
                dict(freqs=E + 2), dict(kc=A + 8), dict(ks=B + 4), dict(vc=C + 1), dict(vs=D + 8), dict(ldq=1028),
                dict(ldk=260), dict(ldv=257)):
        assert append(L, **bad) == ALIGN, bad
    assert append(L, T=0, k=None) == OK
    assert append(L, T=0, k=None, **PLAIN) == OK


def read(L, kc=A, ks=B, vc=C, vs=D, pages=9, page=64, Hkv=2, dim=128, slots=E, T=5, type=0, k=A, v=B):
    return L.apex4_kv4_read(kc, ks, vc, vs, pages, page, Hkv, dim, slots, T, type, k, v, None)


def test_read_refusals(L):
    for bad in (dict(T=-1), dict(T=2 ** 24 + 1), dict(T=2 ** 24, Hkv=512), dict(pages=0), dict(Hkv=0), dict(slots=None),
                dict(kc=None), dict(ks=None), dict(vc=None), dict(vs=None), dict(k=None), dict(v=None)):
        assert read(L, **bad) == INVALID, bad
    for bad in (dict(type=3), dict(type=-1), dict(dim=32), dict(page=24)):
        assert read(L, **bad) == UNSUPPORTED, bad
    for bad in (dict(kc=A + 8), dict(ks=B + 4), dict(vc=C + 8), dict(vs=D + 4), dict(slots=E + 4), dict(k=A + 8),
                dict(v=B + 4)):
        assert read(L, **bad) == ALIGN, bad
    assert read(L, T=0, slots=None, k=None, v=None) == OK


def attend(L, q=A, type=1, T=8, b=4, Hq=8, Hkv=2, dim=128, ldq=1024, cu=B, lens=C, table=D, cols=10, kc=A, ks=B, vc=C,
           vs=D, pages=9, page=64, scale=0.1, causal=1, window=0, max_q=4, max_kv=640, o=E, lse=None, ws=F, n=None):
    need = L.apex4_kv4_attention_workspace_size(T, b, Hq, Hkv, dim, max_q, max_kv)
    return L.apex4_kv4_attention(q, type, T, b, Hq, Hkv, dim, ldq, cu, lens, table, cols, kc, ks, vc, vs, pages, page,
                                 scale, causal, window, max_q, max_kv, o, lse, ws, need if n is None else n, None)


def test_attention_refusals(L):
    for bad in (dict(T=-1), dict(T=2 ** 24 + 1), dict(T=2 ** 24, Hq=1024, ldq=2 ** 20), dict(b=-1), dict(b=65537),
                dict(Hq=0), dict(Hq=1025, Hkv=1025, ldq=2 ** 20), dict(Hkv=0), dict(Hkv=3), dict(dim=0), dict(ldq=1016),
                dict(cols=0), dict(cols=2 ** 30), dict(pages=0), dict(pages=2 ** 31), dict(page=0), dict(scale=INF),
                dict(scale=NAN), dict(window=-1), dict(window=4, causal=0), dict(max_q=0), dict(max_kv=0), dict(cu=None),
                dict(q=None), dict(lens=None), dict(table=None), dict(o=None), dict(kc=None), dict(ks=None),
                dict(vc=None), dict(vs=None)):
        assert attend(L, **bad) == INVALID, bad
    for bad in (dict(type=0), dict(type=3), dict(dim=80), dict(page=8), dict(page=96)):
        assert attend(L, **bad) == UNSUPPORTED, bad
    for bad in (dict(q=A + 8), dict(o=E + 8), dict(lse=F + 2), dict(cu=B + 2), dict(lens=C + 1), dict(table=D + 2),
                dict(kc=A + 8), dict(ks=B + 8), dict(vc=C + 4), dict(vs=D + 4), dict(ldq=1028), dict(ws=F + 8)):
        assert attend(L, **bad) == ALIGN, bad
    assert attend(L, T=0, q=None) == OK and attend(L, T=0, b=0, q=None, cu=None) == OK
    assert attend(L, b=0, q=None) == OK
    for bad in ((0, 4, 8, 2, 128, 4, 640), (8, 0, 8, 2, 128, 4, 640), (8, 4, 8, 3, 128, 4, 640),
                (8, 4, 8, 2, 100, 4, 640), (8, 4, 8, 2, 128, 0, 640), (8, 4, 8, 2, 128, 4, -1)):
        assert L.apex4_kv4_attention_workspace_size(*bad) == 0, bad


def test_cache_layout_by_hand():
    """One page of 16 tokens, one head of 64 numbers: nibbles at places worked out by hand."""
    c = ref.Cache(1, 1, 16, 64)
    c.kc[:], c.vc[:] = -8, -8                           # nibble 0
    c.kc[0, 0, 3, 10] = 7                               # token 3, number 10: byte 5, low half
    c.kc[0, 0, 3, 11] = -3                              # and its high half
    c.vc[0, 0, 6, 21] = 5                               # token 6 = 4 * 1 + 2; number 21 = 5 + 16: high half, r 5, v 0
    c.vc[0, 0, 6, 37] = -7                              # number 37 = 5 + 32: low half, v 1
    k, _, v, _ = c.arrays()
    assert k.shape == (1, 1, 16, 32) and v.shape == (1, 1, 1, 512)
    assert k[0, 0, 3, 5] == 15 | 5 << 4 and np.count_nonzero(k) == 1
    assert v[0, 0, 0, (16 + 5) * 8 + 2] == 13 << 4 and v[0, 0, 0, (16 + 5) * 8 + 4 + 2] == 1
    assert np.count_nonzero(v) == 2
    for page, dim in ((16, 64), (32, 128), (64, 256)):
        c = ref.Cache(3, 2, page, dim, seed=page)
        back = ref.Cache.of(*c.arrays())
        assert (back.kc == c.kc).all() and (back.vc == c.vc).all()


def test_codes_by_hand():
    x = np.zeros((4, 64), np.float32)
    x[0, :4] = [7, -7, 2.5, -0.5]                       # scale 1; ties to even
    x[1, 0], x[1, 1] = np.inf, 1
    x[2, 5] = np.nan
    c, s = ref.codes(x)
    assert s[0] == 1 and list(c[0, :4]) == [7, -7, 2, 0] and s[3] == 0 and not c[3].any()
    assert np.isnan(s[1]) and np.isnan(s[2]) and not c[1:3].any()


def test_attention_by_hand():
    """Two tokens whose scores differ by ln 3: weights 1/4 and 3/4; one that only sees itself."""
    c = ref.Cache(1, 1, 16, 64)
    c.kc[:], c.ks[:], c.vs[:] = 0, 1, 1
    c.kc[0, 0, 1, 0] = 1
    c.vc[:] = 0
    c.vc[0, 0, 0, 0], c.vc[0, 0, 1, 0] = 4, 8 - 1
    q = np.zeros((2, 1, 64))
    q[:, 0, 0] = np.log(3.0)
    o, lse, *_ = ref.attention(q, "float16", c, np.zeros((1, 1), np.int32), [2], np.array([0, 2]), scale=1.0)
    assert np.allclose(o[:, 0, 0], [4, 4 / 4 + 7 * 3 / 4]) and np.allclose(lse[:, 0], [0, np.log(4.0)])
