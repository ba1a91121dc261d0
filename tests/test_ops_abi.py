"""Host-side checks of the LayerNorm, paged-attention and mixture-of-experts
entry points on the CPU: every call here must fail validation, or be one that
launches nothing (no rows, a size query)."""
import ctypes

import pytest
import torch

import associative_algebra_block_amd as aa

G = 1 << 32          # distinct, aligned addresses that nothing reads
BAD, SHAPE, UNSUP, OK = aa.AA_ERR_INVALID_ARG, aa.AA_ERR_SHAPE, aa.AA_ERR_UNSUPPORTED, aa.AA_OK
BF16, F32 = aa.AA_BF16, aa.AA_F32


@pytest.fixture(scope="module")
def lib():
    return aa.load()


def call(lib, name, args, **changed):
    a = dict(args)
    unknown = set(changed) - set(a)
    assert not unknown, unknown
    a.update(changed)
    status = getattr(lib, name)(*a.values())
    assert status == OK or aa.aa_last_error().startswith(name), aa.aa_last_error()
    return status


NORM = dict(X=G, delta=2 * G, gamma=3 * G, beta=4 * G, S=5 * G, Y=6 * G, mean=7 * G, rstd=8 * G, M=4, d=768, eps=1e-5,
            xt=F32, dt=BF16, yt=BF16, stream=None)


@pytest.mark.parametrize("status,changed", [
    (BAD, dict(M=-1)), (BAD, dict(d=0)), (BAD, dict(d=-3)), (UNSUP, dict(d=16385)), (UNSUP, dict(M=1 << 31)),
    (BAD, dict(eps=-1e-5)), (BAD, dict(eps=float("nan"))), (BAD, dict(eps=float("inf"))),
    (BAD, dict(xt=2)), (BAD, dict(dt=-1)), (BAD, dict(yt=7)),
    (BAD, dict(X=None)), (BAD, dict(Y=None)), (BAD, dict(X=G + 8)), (BAD, dict(Y=6 * G + 2)), (BAD, dict(gamma=3 * G + 4)),
    (BAD, dict(S=None)), (BAD, dict(delta=None)), (BAD, dict(mean=None)), (BAD, dict(rstd=None)),
    (BAD, dict(Y=G)), (BAD, dict(Y=5 * G + 16)), (BAD, dict(S=G + 16)), (BAD, dict(Y=2 * G + 4 * 768 * 2 - 16)),
    (BAD, dict(mean=8 * G)), (BAD, dict(rstd=3 * G + 768 * 4 - 16)),
    (OK, dict(M=0)), (OK, dict(M=0, X=None, Y=None)),
])
def test_layernorm_forward(lib, status, changed):
    assert call(lib, "aa_layernorm_fwd", NORM, **changed) == status


BWD = dict(X=G, dY=2 * G, gamma=3 * G, mean=4 * G, rstd=5 * G, dS=6 * G, dX=7 * G, dgamma=8 * G, dbeta=9 * G, M=4,
           d=768, xt=F32, yt=BF16, ws=10 * G, nbytes=1 << 20, stream=None)


@pytest.mark.parametrize("status,changed", [
    (BAD, dict(M=-1)), (BAD, dict(d=0)), (UNSUP, dict(d=1 << 40)), (UNSUP, dict(M=1 << 40)), (BAD, dict(xt=2)),
    (BAD, dict(yt=2)), (BAD, dict(X=None)), (BAD, dict(dY=None)), (BAD, dict(mean=None)), (BAD, dict(rstd=None)),
    (BAD, dict(dX=None)), (BAD, dict(dgamma=8 * G + 4)), (BAD, dict(nbytes=768 * 8 - 1)), (BAD, dict(ws=None)),
    (BAD, dict(ws=10 * G + 8)), (BAD, dict(dX=G)), (BAD, dict(dX=2 * G)), (BAD, dict(dX=6 * G + 16)),
    (BAD, dict(dgamma=9 * G)), (BAD, dict(ws=7 * G + 16)), (BAD, dict(dgamma=3 * G)),
])
def test_layernorm_backward(lib, status, changed):
    assert call(lib, "aa_layernorm_bwd", BWD, **changed) == status


def test_layernorm_workspace(lib):
    n = ctypes.c_size_t(5)
    assert lib.aa_layernorm_bwd_workspace(4, 768, ctypes.byref(n)) == OK and n.value >= 2 * 768 * 4
    assert lib.aa_layernorm_bwd_workspace(4, 768, None) == OK
    assert lib.aa_layernorm_bwd_workspace(0, 768, ctypes.byref(n)) == OK and n.value == 0
    assert lib.aa_layernorm_bwd_workspace(-1, 768, None) == BAD
    assert lib.aa_layernorm_bwd_workspace(1, 0, None) == BAD


CACHE = dict(n_pages=100, page=64, hkv=8, dim=128)
APPEND = dict(K=G, V=2 * G, ldk=1024, ldv=1024, dt=F32, kp=3 * G, vp=4 * G, **CACHE, table=5 * G, n_seqs=3, max_pages=10,
              seq=None, pos=6 * G, n=3, stream=None)


@pytest.mark.parametrize("status,changed", [
    (BAD, dict(dt=3)), (BAD, dict(n_pages=0)), (BAD, dict(hkv=0)), (BAD, dict(dim=0)), (BAD, dict(n_seqs=-1)),
    (BAD, dict(max_pages=0)), (UNSUP, dict(page=8)), (UNSUP, dict(page=48)), (UNSUP, dict(page=8192)),
    (UNSUP, dict(dim=20)), (UNSUP, dict(dim=264)), (UNSUP, dict(hkv=1025, dim=8, ldk=8200, ldv=8200)),
    (UNSUP, dict(n_pages=1 << 31)), (BAD, dict(n=-1)), (UNSUP, dict(n=1 << 31, seq=7 * G)), (SHAPE, dict(n=4)),
    (SHAPE, dict(ldk=1023)), (SHAPE, dict(ldv=0)), (UNSUP, dict(ldv=1 << 31)),
    (BAD, dict(K=None)), (BAD, dict(V=None)), (BAD, dict(K=G + 2)), (BAD, dict(kp=None)), (BAD, dict(vp=4 * G + 8)),
    (BAD, dict(table=None)), (BAD, dict(table=5 * G + 2)), (BAD, dict(pos=None)), (BAD, dict(seq=7 * G + 1)),
    (BAD, dict(kp=4 * G)), (BAD, dict(kp=G)), (BAD, dict(vp=5 * G)), (BAD, dict(vp=6 * G)), (BAD, dict(seq=3 * G)),
    (OK, dict(n=0)), (OK, dict(n=0, K=None, V=None, n_seqs=0)),
])
def test_kv_append(lib, status, changed):
    assert call(lib, "aa_kv_append", APPEND, **changed) == status


ATTN = dict(Q=G, ldq=4096, qt=BF16, kp=3 * G, vp=4 * G, n_pages=100, page=64, heads=32, hkv=8, dim=128, table=5 * G,
            n_seqs=3, max_pages=1000, lengths=6 * G, scale=0.1, O=7 * G, ot=BF16, ws=8 * G, nbytes=1 << 30, stream=None)


@pytest.mark.parametrize("status,changed", [
    (BAD, dict(qt=2)), (BAD, dict(ot=2)), (BAD, dict(heads=0)), (SHAPE, dict(heads=30)), (SHAPE, dict(ldq=4095)),
    (UNSUP, dict(page=24)), (UNSUP, dict(dim=12, ldq=1 << 20)), (UNSUP, dict(n_seqs=1 << 20)),
    (BAD, dict(scale=float("nan"))), (BAD, dict(scale=float("inf"))), (BAD, dict(Q=None)), (BAD, dict(Q=G + 1)),
    (BAD, dict(kp=None)), (BAD, dict(vp=None)), (BAD, dict(table=None)), (BAD, dict(lengths=None)),
    (BAD, dict(lengths=6 * G + 2)), (BAD, dict(O=None)), (BAD, dict(O=7 * G + 8)), (BAD, dict(nbytes=16)),
    (BAD, dict(ws=None)), (BAD, dict(ws=8 * G + 4)), (BAD, dict(O=G)), (BAD, dict(O=3 * G)), (BAD, dict(ws=7 * G)),
    (BAD, dict(ws=4 * G)), (OK, dict(n_seqs=0)), (OK, dict(n_seqs=0, Q=None, O=None, ws=None, nbytes=0)),
])
def test_attn_decode(lib, status, changed):
    assert call(lib, "aa_attn_decode", ATTN, **changed) == status


@pytest.mark.parametrize("scale", [1.8e38, -1.8e38, 3.4e38])
def test_attn_scales_beyond_the_kernels_base(lib, scale):
    """Scores are taken to base 2: a scale whose product with log2 e is infinite
    is refused."""
    assert call(lib, "aa_attn_decode", ATTN, scale=scale) == BAD
    assert call(lib, "aa_attn_decode", ATTN, scale=scale / 2, n_seqs=0) == OK


def test_attn_workspace(lib):
    n = ctypes.c_size_t(0)
    f = lib.aa_attn_decode_workspace
    assert f(1, 32, 8, 128, 64, 2048, ctypes.byref(n)) == OK and n.value % (32 * (128 + 2) * 4) == 0 and n.value > 0
    assert f(512, 32, 8, 128, 64, 2048, ctypes.byref(n)) == OK and n.value == 0      # rows enough: not split
    assert f(0, 32, 8, 128, 64, 2048, ctypes.byref(n)) == OK and n.value == 0
    assert f(1, 32, 8, 128, 64, 2048, None) == OK
    assert f(1, 31, 8, 128, 64, 2048, None) == SHAPE
    assert f(1, 32, 8, 100, 64, 2048, None) == UNSUP
    assert f(-1, 32, 8, 128, 64, 2048, None) == BAD


@pytest.fixture(scope="module")
def moe():
    up = aa.aa_plan_create("Qq", 4, 128, 256)
    down = aa.aa_plan_create("Qq", 4, 256, 128)
    return up, down, dict(up=up.handle, down=down.handle, X=G, Wr=2 * G, E=16, k=4, norm=1, Wg=3 * G, Wu=4 * G, Wd=5 * G,
                          Y=6 * G, experts=7 * G, weights=8 * G, M=3, pos=0, types=None, ws=9 * G, nbytes=1 << 24,
                          stream=None)


@pytest.mark.parametrize("status,changed", [
    (BAD, dict(up=None)), (BAD, dict(down=None)), (BAD, dict(E=0)), (BAD, dict(k=0)), (SHAPE, dict(k=17)),
    (UNSUP, dict(E=513)), (UNSUP, dict(E=100, k=65)), (BAD, dict(M=-1)), (UNSUP, dict(M=20000)),
    (UNSUP, dict(M=1 << 40)), (BAD, dict(pos=-1)), (BAD, dict(types=10 * G)), (BAD, dict(X=None)), (BAD, dict(Wr=None)),
    (BAD, dict(Wg=None)), (BAD, dict(Wu=3 * G + 8)), (BAD, dict(Wd=None)), (BAD, dict(Y=None)), (BAD, dict(Y=6 * G + 4)),
    (BAD, dict(experts=7 * G + 2)), (BAD, dict(weights=8 * G + 1)), (BAD, dict(ws=None)), (BAD, dict(nbytes=100)),
    (BAD, dict(Y=G)), (BAD, dict(Y=3 * G + 15 * 128 * 256 * 2)), (BAD, dict(ws=6 * G)), (BAD, dict(experts=8 * G)),
    (BAD, dict(weights=9 * G)), (OK, dict(M=0)), (OK, dict(M=0, X=None, Y=None, ws=None, nbytes=0)),
])
def test_moe(lib, moe, status, changed):
    assert call(lib, "aa_moe_ffn_fwd", moe[2], **changed) == status


def test_moe_plans(lib, moe):
    base = moe[2]
    n = ctypes.c_size_t(0)

    def status(up, down):
        got = call(lib, "aa_moe_ffn_fwd", base, up=up.handle, down=down.handle)
        assert lib.aa_moe_ffn_workspace(up.handle, down.handle, 16, 4, 3, ctypes.byref(n)) == got
        return got

    c = aa.aa_plan_create
    assert status(c("Qq", 4, 128, 256), c("Qq", 2, 256, 128)) == SHAPE
    assert status(c("Qq", 4, 128, 256), c("Q2xQ2", 4, 256, 128)) == SHAPE
    assert status(c("Qq", 4, 128, 256), c("Qq", 4, 128, 128)) == SHAPE
    assert status(c("Qq", 4, 128, 256), c("Qq", 4, 256, 128, "pos_mod", 8)) == SHAPE
    assert status(c("Qq", 4, 128, 256, "pos_mod", 0, "f32", "f32"), c("Qq", 4, 256, 128)) == UNSUP
    assert status(c("Qq", 4, 128, 256), c("Qq", 4, 256, 128, "pos_mod", 0, "f32", "f32")) == UNSUP
    assert status(c("Qq", 4, 128, 256, "block_rows"), c("Qq", 4, 256, 128, "block_rows")) == UNSUP
    assert status(c("Qq", 4, 80, 48), c("Qq", 4, 48, 80)) == UNSUP                  # layout 2
    e = [(0, 1), (1, 0)]
    assert status(aa.aa_plan_create_digraph(2, e, 64, 64), aa.aa_plan_create_digraph(2, e, 64, 64)) == UNSUP
    up, down = c("Qq", 4, 128, 256, "explicit"), c("Qq", 4, 256, 128, "explicit")
    assert call(lib, "aa_moe_ffn_fwd", base, up=up.handle, down=down.handle) == BAD     # no types
    assert call(lib, "aa_moe_ffn_fwd", base, up=up.handle, down=down.handle, types=10 * G + 2) == BAD
    assert lib.aa_moe_ffn_workspace(moe[0].handle, moe[1].handle, 16, 4, 3, ctypes.byref(n)) == OK
    assert n.value >= 3 * (16 * 8 + 4 * 256 * 4 + 4 * 8)
    assert lib.aa_moe_ffn_workspace(moe[0].handle, moe[1].handle, 16, 4, 0, ctypes.byref(n)) == OK and n.value == 0


def test_binding_takes_device_tensors_only():
    x = torch.zeros(2, 8)
    i = torch.zeros(2, dtype=torch.int32)
    k, v = torch.zeros(1, 1, 16, 8, dtype=torch.bfloat16), torch.zeros(1, 1, 8, 16, dtype=torch.bfloat16)
    up, down = aa.aa_plan_create("Qq", 2, 32, 32), aa.aa_plan_create("Qq", 2, 32, 32)
    for f in (lambda: aa.aa_layernorm_fwd(x, None, None, x), lambda: aa.aa_layernorm_bwd(x, x, None, x, x, x),
              lambda: aa.aa_kv_append(x, x, k, v, i.view(2, 1), i),
              lambda: aa.aa_attn_decode(x, k, v, i.view(2, 1), i, x.view(2, 1, 8), 1.0),
              lambda: aa.aa_moe_ffn_fwd(up, down, x, x, x, x, x, x, 1)):
        with pytest.raises(ValueError, match="device tensor"):
            f()
    with pytest.raises(TypeError):
        aa.aa_layernorm_fwd(1234, None, None, 1234)


def test_missing_binding_fails_loudly(monkeypatch):
    """Without the extension module the operators' calls raise: there is no
    other path."""
    import sys
    monkeypatch.setattr(aa, "_MARSHAL", None)
    monkeypatch.delattr(aa, "_aa_binding", raising=False)
    monkeypatch.setitem(sys.modules, "associative_algebra_block_amd._aa_binding", None)
    with pytest.raises(RuntimeError, match="is not built"):
        aa.aa_layernorm_fwd(torch.zeros(1, 1), None, None, torch.zeros(1, 1))
