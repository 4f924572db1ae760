"""Host-side argument checks of the 8-bit inference entry points.  CPU only:
no call here reaches a kernel."""
import ctypes

import pytest

from expanded_rank_matrix_b200 import externd as X

P = ctypes.c_void_p(1 << 20)         # never dereferenced
MIS4 = ctypes.c_void_p((1 << 20) + 2)
MIS16 = ctypes.c_void_p((1 << 20) + 8)


@pytest.fixture(scope="module")
def lib():
    from expanded_rank_matrix_b200 import build
    build.build()
    return X.load()


def test_quantize_rows_arguments(lib):
    ok = dict(X=P, type=X.BF16, ldx=64, rows=4, n=64, Q=P, ldq=64, scale=P)

    def call(**kw):
        a = {**ok, **kw}
        return lib.externd_quantize_rows(a["X"], a["type"], a["ldx"], a["rows"], a["n"], a["Q"],
                                         a["ldq"], a["scale"], None)
    for bad in (dict(X=None), dict(Q=None), dict(scale=None), dict(type=X.I8), dict(type=-1),
                dict(type=4), dict(ldx=63), dict(ldq=63), dict(ldq=72), dict(n=0), dict(n=-1),
                dict(n=X.I8_MAX_INNER + 1, ldx=1 << 20, ldq=1 << 20), dict(rows=-1),
                dict(rows=(1 << 30) + 1), dict(Q=MIS16), dict(scale=MIS4),
                dict(X=ctypes.c_void_p((1 << 20) + 1)), dict(X=MIS4, type=X.F32)):
        assert call(**bad) == X.ERR_INVALID_ARG, bad
    assert call(rows=0) == X.OK
    assert call(rows=0, X=None, Q=None, scale=None) == X.OK


def test_matmul_arguments(lib):
    ok = dict(X=P, xtype=X.I8, ldx=64, xs=P, W=P, ldw=64, ws=P, b=None, rows=4, n=64, m=8, Y=P,
              ytype=X.F32, ldy=8)

    def call(**kw):
        a = {**ok, **kw}
        return lib.externd_matmul_i8(a["X"], a["xtype"], a["ldx"], a["xs"], a["W"], a["ldw"],
                                     a["ws"], a["b"], a["rows"], a["n"], a["m"], a["Y"],
                                     a["ytype"], a["ldy"], None)
    for bad in (dict(X=None), dict(W=None), dict(ws=None), dict(Y=None), dict(xs=None),
                dict(xtype=7), dict(ytype=X.I8), dict(ldx=63), dict(ldx=72), dict(ldw=72),
                dict(ldw=48), dict(ldy=7), dict(n=0), dict(m=0), dict(rows=-1),
                dict(m=X.I8_MAX_OUT + 1, ldy=1 << 25), dict(X=MIS16), dict(W=MIS16),
                dict(ws=MIS4), dict(b=MIS4), dict(xs=MIS4), dict(Y=MIS4),
                dict(Y=ctypes.c_void_p((1 << 20) + 1), ytype=X.BF16),
                dict(n=X.I8_MAX_INNER + 1, ldx=1 << 20, ldw=1 << 20)):
        assert call(**bad) == X.ERR_INVALID_ARG, bad
    assert call(rows=0) == X.OK
    assert call(rows=0, W=None) == X.ERR_INVALID_ARG


def test_pack_and_apply_arguments(lib):
    pack = [P, P, P, 8, 64, 16, P, P, P, None]

    def with_(args, i, v):
        return args[:i] + [v] + args[i + 1:]
    for i in (0, 1, 2, 6, 7, 8):
        assert lib.externd_pack_codes(*with_(pack, i, None)) == X.ERR_INVALID_ARG
        assert lib.externd_pack_codes(*with_(pack, i, MIS4)) == X.ERR_INVALID_ARG
    for i in (6, 7):
        assert lib.externd_pack_codes(*with_(pack, i, MIS16)) == X.ERR_INVALID_ARG
    for i, v in ((3, 0), (4, 0), (5, 0), (3, X.I8_MAX_OUT + 1), (4, X.I8_MAX_INNER + 1),
                 (5, X.I8_MAX_INNER + 1)):
        assert lib.externd_pack_codes(*with_(pack, i, v)) == X.ERR_INVALID_ARG
    app = [P, P, P, P, 8, 64, 16, P, X.F32, 64, None, 4, P, X.F32, 8, None]
    for i in (0, 1, 2, 3, 7, 12):
        assert lib.externd_ternary_apply_i8(*with_(app, i, None)) == X.ERR_INVALID_ARG, i
    for i, v in ((0, MIS16), (1, MIS16), (2, MIS4), (3, MIS4), (4, 0), (5, 0), (6, 0), (8, 9),
                 (9, 63), (11, -1), (13, X.I8), (14, 7), (8, X.I8),
                 (6, X.I8_MAX_INNER + 1)):
        assert lib.externd_ternary_apply_i8(*with_(app, i, v)) == X.ERR_INVALID_ARG, i
    assert lib.externd_ternary_apply_i8(*with_(app, 11, 0)) == X.OK


def test_code_words():
    assert X.code_words(1) == 8 and X.code_words(128) == 8 and X.code_words(129) == 16
    assert X.code_words(2560) == 160
    assert X.code_words(0) == 0 and X.code_words(X.I8_MAX_OUT + 1) == 0


def test_wait_budget_must_not_be_negative(lib):
    mm = [P, X.I8, 64, P, P, 64, P, None, 0, 64, 8, P, X.F32, 8]
    assert lib.externd_matmul_i8_ex(*mm, -1, None) == X.ERR_INVALID_ARG
    assert lib.externd_matmul_i8_ex(*mm, 1, None) == X.OK
    app = [P, P, P, P, 8, 64, 16, P, X.F32, 64, None, 0, P, X.F32, 8]
    assert lib.externd_ternary_apply_i8_ex(*app, -1, None) == X.ERR_INVALID_ARG
    assert lib.externd_ternary_apply_i8_ex(*app, 1, None) == X.OK
