"""CPU-side checks of apex4_route, apex4_experts_w4a4 and the e4m3 calls: every
refusal happens on the host, before any HIP call and before a pointer is used."""
import numpy as np
import pytest

import layers_ref as ref
from w4a4_group_quantized_amd import apex4

OK, INVALID, UNSUPPORTED, ALIGN, WORKSPACE = 0, 1, 2, 3, 4
A, B, C, D = 0x10000, 0x20000, 0x30000, 0x40000      # fake aligned device addresses: never dereferenced


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(apex4.LIB_PATH):
        pytest.skip("libapex4.so not built (run __graft_entry__.build())")
    return apex4.lib()


def route(L, logits=A, type=0, M=4, E=64, score=0, bias=None, n_group=1, keep=1, top=1, k=4, renorm=1, scale=1.0,
          ids=B, gates=C):
    return L.apex4_route(logits, type, M, E, score, bias, n_group, keep, top, k, renorm, scale, ids, gates, None)


def test_route_refusals(L):
    for bad in (dict(M=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=65), dict(k=5, E=4), dict(n_group=0),
                dict(n_group=3), dict(n_group=65, E=130), dict(n_group=4, keep=0), dict(n_group=4, keep=5),
                dict(n_group=16, keep=1, k=5), dict(top=0), dict(top=3), dict(score=2), dict(scale=float("inf")),
                dict(scale=float("nan")), dict(logits=None), dict(ids=None), dict(gates=None), dict(M=2 ** 26 + 1)):
        assert route(L, **bad) == INVALID, bad
    assert route(L, type=3) == UNSUPPORTED
    for bad in (dict(logits=A + 2), dict(logits=A + 1, type=1), dict(bias=A + 2), dict(ids=B + 2), dict(gates=C + 1)):
        assert route(L, **bad) == ALIGN, bad
    assert route(L, M=0, logits=None, ids=None, gates=None) == OK
    assert route(L, M=0, k=0) == INVALID             # arguments are checked for no rows too


def experts(L, x=A, ids=B, gates=C, M=4, k=2, E=8, H=256, I=128, group=128, gu=A, sgu=B, dn=A, sdn=B, y=D, y32=None,
            ws=0x100000, nbytes=None):
    n = L.apex4_experts_workspace_size(M, k, E, H, I, group) if nbytes is None else nbytes
    return L.apex4_experts_w4a4(x, ids, gates, M, k, E, H, I, group, gu, sgu, dn, sdn, y, y32, ws, n, None)


def test_experts_refusals(L):
    for bad in (dict(M=-1), dict(k=0), dict(k=65), dict(E=0), dict(E=1025), dict(H=0), dict(H=192), dict(I=64),
                dict(I=-128), dict(group=0), dict(M=2 ** 30), dict(H=2 ** 17, I=2 ** 15), dict(x=None),
                dict(ids=None), dict(gates=None), dict(gu=None), dict(sgu=None), dict(dn=None), dict(sdn=None),
                dict(y=None)):
        assert experts(L, **bad) == INVALID, bad
    assert experts(L, group=64) == UNSUPPORTED
    need = L.apex4_experts_workspace_size(4, 2, 8, 256, 128, 128)
    assert need > 0
    assert experts(L, nbytes=need - 1) == WORKSPACE
    assert experts(L, ws=None) == WORKSPACE
    for bad in (dict(x=A + 8), dict(ids=B + 2), dict(gates=C + 2), dict(gu=A + 8), dict(sgu=B + 2), dict(dn=A + 4),
                dict(sdn=B + 1), dict(y=D + 2), dict(y32=D + 2), dict(ws=0x100000 + 16)):
        assert experts(L, **bad) == ALIGN, bad
    assert experts(L, M=0, x=None, ws=None) == OK
    for bad in ((0, 2, 8, 256, 128, 128), (4, 2, 8, 200, 128, 128), (4, 2, 8, 256, 128, 64), (-4, 2, 8, 256, 128, 128)):
        assert L.apex4_experts_workspace_size(*bad) == 0


def test_e4m3_refusals(L):
    for f in (L.apex4_quantize_e4m3, L.apex4_pack_weight_e4m3):
        assert f(A, 1, -1, 256, B, C, None) == INVALID
        assert f(A, 1, 4, 0, B, C, None) == INVALID
        assert f(A, 1, 4, 200, B, C, None) == INVALID
        assert f(A, 1, 2 ** 26, 256, B, C, None) == INVALID          # 2^34 elements
        assert f(A, 0, 4, 256, B, C, None) == UNSUPPORTED            # fp32
        assert f(None, 1, 4, 256, B, C, None) == INVALID
        assert f(A, 1, 4, 256, None, C, None) == INVALID
        assert f(A, 1, 4, 256, B, None, None) == INVALID
        assert f(A + 8, 1, 4, 256, B, C, None) == ALIGN
        assert f(A, 2, 4, 256, B + 4, C, None) == ALIGN
        assert f(None, 1, 0, 256, None, None, None) == OK

    def gemm(qa=A, sa=B, qw=A, sw=B, M=8, N=40, K=256, t=1, y=C, y32=None, ws=None, n=None):
        n = L.apex4_gemm_e4m3_workspace_size(M, N, K) if n is None else n
        return L.apex4_gemm_e4m3(qa, sa, qw, sw, M, N, K, t, y, y32, ws or (D if n else None), n, None)

    for bad in (dict(M=-1), dict(N=-1), dict(K=0), dict(K=100), dict(K=2 ** 23), dict(N=2 ** 27), dict(qa=None),
                dict(sa=None), dict(qw=None), dict(sw=None), dict(y=None)):
        assert gemm(**bad) == INVALID, bad
    assert gemm(t=0) == UNSUPPORTED
    for bad in (dict(qa=A + 8), dict(sa=B + 2), dict(qw=A + 4), dict(sw=B + 1), dict(y=C + 1), dict(y32=C + 2)):
        assert gemm(**bad) == ALIGN, bad
    assert gemm(M=0, qa=None) == OK and gemm(N=0, qw=None) == OK

    def linear(x=A, t=1, qw=A, sw=B, M=80, N=40, K=256, y=C, y32=None, ws=0x100000, n=None):
        n = L.apex4_linear_e4m3_workspace_size(M, N, K) if n is None else n
        return L.apex4_linear_e4m3(x, t, qw, sw, M, N, K, y, y32, ws, n, None)

    need = L.apex4_linear_e4m3_workspace_size(80, 40, 256)
    assert need >= 80 * 256 + 80 * 2 * 4
    # the smallest calls are one launch without a workspace
    assert L.apex4_linear_e4m3_workspace_size(1, 4096, 4096) == 0
    assert L.apex4_linear_e4m3_workspace_size(16, 40, 1024) == 0
    assert L.apex4_linear_e4m3_workspace_size(17, 40, 256) > 0
    assert L.apex4_linear_e4m3_workspace_size(16, 40, 1152) > 0
    assert linear(M=8, ws=None, x=None) == INVALID
    assert linear(n=need - 1) == WORKSPACE and linear(ws=None) == WORKSPACE
    for bad in (dict(M=-1), dict(K=130), dict(x=None), dict(qw=None), dict(sw=None), dict(y=None)):
        assert linear(**bad) == INVALID, bad
    assert linear(t=0) == UNSUPPORTED
    for bad in (dict(x=A + 2), dict(ws=0x100000 + 128), dict(y=C + 1)):
        assert linear(**bad) == ALIGN, bad
    assert linear(M=0, x=None, ws=None, n=0) == OK


def test_binding_refuses_host_tensors_and_wrong_types():
    torch = pytest.importorskip("torch")
    x = torch.zeros((4, 256))
    for call in (lambda: apex4.route(x, 2), lambda: apex4.quantize_e4m3(x), lambda: apex4.pack_weight_e4m3(x),
                 lambda: apex4.linear_e4m3(x, x, x), lambda: apex4.experts(x, x, x, x, x, x, x)):
        with pytest.raises(ValueError):
            call()


def test_plain_implementations_agree_with_each_other():
    """The reference's pieces on cases worked by hand."""
    assert ref.e4m3_round(np.array([448.0, 17, 19, 2.0 ** -10, 3 * 2.0 ** -10, -0.3])).tolist() == \
        [448.0, 16.0, 20.0, 0.0, 2.0 ** -8, -0.3125]
    v = ref.e4m3_decode(np.arange(256))
    ok = ~np.isnan(v)
    assert ok.sum() == 254 and v[0x7E] == 448 and v[1] == 2.0 ** -9 and v[0x38] == 1.0
    assert np.array_equal(ref.e4m3_round(v[ok]), v[ok])
    ids, g = ref.route(np.array([[0.0, 1.0, 1.0, -np.inf]]), 3, renormalize=False)
    assert ids.tolist() == [[1, 2, 0]] and abs(g[0, 0] - np.e / (1 + 2 * np.e)) < 1e-15
    q, s = ref.int4(np.array([[7.0, 0.5, 1.5, -7.0] + [0.0] * 124], dtype=np.float16))
    assert s[0, 0] == 1.0 and q[0, :4].tolist() == [7, 0, 2, -7]
    assert ref.pack(np.array([[1, -1, 7, -8]])).tolist() == [[0xF1, 0x87]]


def test_sizes_past_the_launch_limits_are_refused(L):
    assert route(L, M=(1 << 25) + 1) == INVALID
    M, N = 1 << 20, 1 << 17
    assert L.apex4_gemm_e4m3_workspace_size(M, N, 128) == 0
    assert L.apex4_linear_e4m3_workspace_size(M, N, 128) == 0
    assert L.apex4_gemm_e4m3(None, None, None, None, M, N, 128, 1, None, None, None, 0, None) == INVALID
    assert L.apex4_linear_e4m3(None, 1, None, None, M, N, 128, None, None, None, 0, None) == INVALID
