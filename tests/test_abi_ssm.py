"""Refusals of the selective state space scan and of the group norm at the C
ABI: bad host arguments come back with the documented status before anything
is launched (no GPU needed; accepted calls reach the launch and fail there)."""
import ctypes

import pytest
import torch

import causal_depthwise_short_conv1d_amd as S
from tests.test_abi import BASE, EALIAS, EALIGN, EARG, ELAUNCH, ENULL, ESHAPE, ESTRIDE, GB, OK, addr, no_gpu
from tests.test_abi_gdr import status

INF = float("inf")


@pytest.fixture(scope="module")
def lib():
    return S.load_library()


def fwd(lib, **kw):
    no_gpu()
    a = dict(x=addr(1), xs=(512, 64, 1), dt=addr(2), ds=(8, 1, 0), f32=0, a=addr(3), as_=(1, 0, 0), b=addr(4), bs=(256, 128, 1),
             c=addr(5), cs=(256, 128, 1), d=addr(6), dd=(1, 0), z=addr(7), zs=(512, 64, 1), bias=addr(8), db=(1, 0), sp=1,
             lo=-INF, hi_=INF, st=addr(9), ss=(8 * 64 * 128, 64 * 128, 128, 1), lines=4, ci=addr(10), hi=addr(11), qsl=addr(12),
             batch=2, T=10, H=8, G=2, P=64, N=128, pad=-1, o=addr(13), os=(512, 64, 1), ws=None, wb=0)
    a.update(kw)
    return status(lib, "ssm_fwd_varlen", a["x"], *a["xs"], a["dt"], *a["ds"], a["f32"], a["a"], *a["as_"], a["b"], *a["bs"],
                  a["c"], *a["cs"], a["d"], *a["dd"], a["z"], *a["zs"], a["bias"], *a["db"], a["sp"], a["lo"], a["hi_"],
                  a["st"], *a["ss"], a["lines"], a["ci"], a["hi"], a["qsl"], a["batch"], a["T"], a["H"], a["G"], a["P"], a["N"],
                  a["pad"], a["o"], *a["os"], a["ws"], a["wb"], None)


def test_fwd_accepted(lib):
    assert fwd(lib) == ELAUNCH
    assert fwd(lib, st=None, hi=None, lines=0) == ELAUNCH
    assert fwd(lib, d=None, z=None, bias=None) == ELAUNCH
    assert fwd(lib, f32=1) == ELAUNCH
    assert fwd(lib, bs=(0, 0, 0), xs=(0, 0, 0)) == ELAUNCH      # one row for every token: read only
    assert fwd(lib, x=ctypes.c_void_p(BASE + GB + 2)) == ELAUNCH
    assert fwd(lib, P=37, N=3, ss=(8 * 37 * 3, 37 * 3, 3, 1)) == ELAUNCH
    assert fwd(lib, as_=(64 * 128, 128, 1), ds=(512, 64, 1), db=(64, 1), dd=(64, 1)) == ELAUNCH
    assert fwd(lib, lo=0.0, hi_=0.0) == ELAUNCH


def test_fwd_empty_is_a_noop(lib):
    assert fwd(lib, T=0, x=None, qsl=None) == OK
    assert fwd(lib, batch=0, x=None) == OK


def test_fwd_nulls(lib):
    for x in ("x", "dt", "a", "b", "c", "o", "qsl"):
        assert fwd(lib, **{x: None}) == ENULL, x
    assert fwd(lib, st=None) == ENULL                           # has_initial_state needs a state


def test_fwd_sizes(lib):
    for kw in (dict(batch=-1), dict(T=-1), dict(T=1 << 31), dict(T=(1 << 31) - 256), dict(H=0), dict(G=0), dict(G=3), dict(P=0),
               dict(N=0), dict(N=257, ss=(1 << 30, 1 << 24, 257, 1)), dict(lines=0), dict(ci=None, lines=1), dict(lines=-1),
               dict(batch=1 << 30)):
        assert fwd(lib, **kw) == ESHAPE, kw
    for kw in (dict(lo=1.0, hi_=0.5), dict(lo=float("nan")), dict(hi_=float("nan"))):
        assert fwd(lib, **kw) == EARG, kw


def test_fwd_strides(lib):
    for x in ("xs", "bs", "cs", "zs", "os", "ds", "as_"):
        assert fwd(lib, **{x: (512, -64, 1)}) == ESTRIDE, x
    for x in ("dd", "db"):
        assert fwd(lib, **{x: (-1, 0)}) == ESTRIDE, x
    assert fwd(lib, os=(512, 32, 1)) == ESTRIDE                 # heads of out overlap
    assert fwd(lib, os=(0, 64, 1)) == ESTRIDE
    assert fwd(lib, ss=(0, 64 * 128, 128, 1)) == ESTRIDE        # lines overlap
    assert fwd(lib, ss=(8 * 64 * 128, 64 * 128, 127, 1)) == ESTRIDE


def test_fwd_alignment_and_overlap(lib):
    for x in ("x", "b", "c", "z", "o", "dt"):
        assert fwd(lib, **{x: ctypes.c_void_p(BASE + 20 * GB + 1)}) == EALIGN, x
    for x in ("a", "d", "bias", "st", "ci", "qsl"):
        assert fwd(lib, **{x: ctypes.c_void_p(BASE + 20 * GB + 2)}) == EALIGN, x
    assert fwd(lib, f32=1, dt=ctypes.c_void_p(BASE + 20 * GB + 2)) == EALIGN
    for x in range(1, 10):
        assert fwd(lib, o=addr(x)) == EALIAS, x
    for x in range(1, 9):
        assert fwd(lib, st=addr(x)) == EALIAS, x


def test_fwd_workspace(lib):
    f = lib.ssm_fwd_workspace_bytes
    need = f(2, 2000, 8, 2, 64, 128, 0)
    assert need > 0
    assert fwd(lib, T=2000, ws=addr(14), wb=need) == ELAUNCH
    assert fwd(lib, T=2000, ws=addr(14), wb=need - 1) == ESHAPE
    assert fwd(lib, T=2000, ws=ctypes.c_void_p(BASE + 14 * GB + 8), wb=need) == EALIGN
    for x in (*range(1, 10), 13):
        assert fwd(lib, T=2000, ws=addr(x), wb=need) == EALIAS, x
    assert f(2, 600, 8, 2, 64, 128, 0) == 0                     # short sequences
    assert f(100, 1 << 20, 64, 8, 64, 128, 0) == 0              # many of them
    assert f(1, 2000, 8, 2, 64, 129, 0) == 0                    # more states than the chunked kernel has
    channels = dict(H=2, G=2, as_=(64 * 16, 16, 1), ds=(128, 64, 1), db=(64, 1), dd=(64, 1), N=16, xs=(128, 64, 1), zs=(128, 64, 1),
                    os=(128, 64, 1), ss=(2 * 64 * 16, 64 * 16, 16, 1))
    need = f(2, 2000, 2, 2, 64, 16, 1)
    assert need > 0
    assert fwd(lib, T=2000, ws=addr(14), wb=need, **channels) == ELAUNCH
    assert fwd(lib, T=2000, ws=addr(14), wb=need - 1, **channels) == ESHAPE
    assert f(2, 2000, 4, 2, 64, 16, 1) == 0                     # heads that share groups
    assert f(2, 2000, 2, 2, 64, 65, 1) == 0
    for bad in ((0, 2000, 8, 2, 64, 128, 0), (2, 0, 8, 2, 64, 128, 0), (2, 2000, 0, 2, 64, 128, 0), (2, 2000, 8, 3, 64, 128, 0),
                (2, 2000, 8, 0, 64, 128, 0), (2, 2000, 8, 2, 0, 128, 0), (2, 2000, 8, 2, 64, 0, 0), (1, 1 << 31, 8, 2, 64, 128, 0)):
        assert f(*bad) == 0


def update(lib, **kw):
    no_gpu()
    a = dict(x=addr(1), xs=(2048, 512, 64, 1), dt=addr(2), ds=(32, 8, 1, 0), f32=0, a=addr(3), as_=(1, 0, 0), b=addr(4),
             bs=(1024, 256, 128, 1), c=addr(5), cs=(1024, 256, 128, 1), d=addr(6), dd=(1, 0), z=addr(7), zs=(2048, 512, 64, 1),
             bias=addr(8), db=(1, 0), sp=1, lo=-INF, hi_=INF, st=addr(9), ss=(8 * 64 * 128, 64 * 128, 128, 1), lines=16,
             ci=addr(10), cis=(4, 1), steps=4, acc=addr(11), osi=addr(12), osis=(4, 1), batch=2, seqlen=4, H=8, G=2, P=64, N=128,
             pad=-1, o=addr(13), os=(2048, 512, 64, 1))
    a.update(kw)
    return status(lib, "ssm_update", a["x"], *a["xs"], a["dt"], *a["ds"], a["f32"], a["a"], *a["as_"], a["b"], *a["bs"], a["c"],
                  *a["cs"], a["d"], *a["dd"], a["z"], *a["zs"], a["bias"], *a["db"], a["sp"], a["lo"], a["hi_"], a["st"],
                  *a["ss"], a["lines"], a["ci"], *a["cis"], a["steps"], a["acc"], a["osi"], *a["osis"], a["batch"],
                  a["seqlen"], a["H"], a["G"], a["P"], a["N"], a["pad"], a["o"], *a["os"], None)


def test_update_refusals(lib):
    assert update(lib) == ELAUNCH
    assert update(lib, acc=None, osi=None, ci=None, d=None, z=None, bias=None) == ELAUNCH
    assert update(lib, batch=0, x=None) == OK
    assert update(lib, seqlen=0, x=None) == OK
    for x in ("x", "dt", "a", "b", "c", "st", "o", "ci"):       # ci: num_accepted_tokens needs it
        assert update(lib, **{x: None}) == ENULL, x
    for kw in (dict(batch=-1), dict(seqlen=-1), dict(steps=0), dict(lines=0), dict(ci=None, acc=None, lines=1), dict(G=3),
               dict(N=300, ss=(1 << 30, 1 << 20, 300, 1))):
        assert update(lib, **kw) == ESHAPE, kw
    for kw in (dict(cis=(-1, 0)), dict(osis=(4, -1)), dict(xs=(-1, 512, 64, 1)), dict(os=(2048, 512, 63, 1)),
               dict(ss=(1, 64 * 128, 128, 1))):
        assert update(lib, **kw) == ESTRIDE, kw
    for x in ("acc", "osi", "ci"):
        assert update(lib, **{x: ctypes.c_void_p(BASE + 20 * GB + 1)}) == EALIGN, x
    assert update(lib, lo=2.0, hi_=1.0) == EARG
    for x in range(1, 10):
        assert update(lib, o=addr(x)) == EALIAS, x


def norm(lib, **kw):
    no_gpu()
    a = dict(x=addr(1), xs=(1024, 128, 1), z=addr(2), zs=(1024, 128, 1), w=addr(3), ws=128, b=addr(4), bs=0, f32=0, rows=10, G=8,
             n=128, kind=0, act=1, first=0, eps=1e-5, o=addr(5), os=(1024, 128, 1))
    a.update(kw)
    return lib.sconv_group_norm(a["x"], *a["xs"], a["z"], *a["zs"], a["w"], a["ws"], a["b"], a["bs"], a["f32"], a["rows"], a["G"],
                                a["n"], a["kind"], a["act"], a["first"], a["eps"], a["o"], *a["os"], None)


def test_norm_refusals(lib):
    assert norm(lib) == ELAUNCH
    assert norm(lib, z=None, w=None, b=None) == ELAUNCH
    assert norm(lib, first=1, kind=1, act=2, f32=1) == ELAUNCH
    assert norm(lib, o=addr(1)) == ELAUNCH                      # in place of x, or of z
    assert norm(lib, o=addr(2)) == ELAUNCH
    assert norm(lib, xs=(0, 0, 0)) == ELAUNCH
    for x in ("rows", "G", "n"):
        assert norm(lib, **{x: 0, "x": None}) == OK, x
        assert norm(lib, **{x: -1}) == ESHAPE, x
    assert norm(lib, rows=1 << 40) == ESHAPE
    for x in ("x", "o"):
        assert norm(lib, **{x: None}) == ENULL, x
    for kw in (dict(xs=(-1, 128, 1)), dict(zs=(1024, 128, -1)), dict(ws=-1), dict(bs=-1), dict(os=(1024, 64, 1)), dict(os=(0, 128, 1)),
               dict(os=(-1024, 128, 1))):
        assert norm(lib, **kw) == ESTRIDE, kw
    for kw in (dict(kind=2), dict(act=3), dict(act=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=INF), dict(z=None, first=1)):
        assert norm(lib, **kw) == EARG, kw
    for x in ("x", "z", "w", "b", "o"):
        assert norm(lib, **{x: ctypes.c_void_p(BASE + 20 * GB + 1)}) == EALIGN, x
    assert norm(lib, f32=1, w=ctypes.c_void_p(BASE + 20 * GB + 2)) == EALIGN
    assert norm(lib, o=addr(1), os=(2048, 128, 1)) == EALIAS    # x, but not its elements
    assert norm(lib, o=ctypes.c_void_p(BASE + GB + 2)) == EALIAS
    for x in (3, 4):
        assert norm(lib, o=addr(x)) == EALIAS, x


def test_binding_refusals():
    bf = torch.bfloat16
    qsl = torch.tensor([0, 3], dtype=torch.int32)
    head = dict(x=torch.zeros(3, 4, 8, dtype=bf), dt=torch.zeros(3, 4), A=torch.zeros(4), B=torch.zeros(3, 2, 16, dtype=bf),
                C=torch.zeros(3, 2, 16, dtype=bf), state=torch.zeros(2, 4, 8, 16))
    chan = dict(x=torch.zeros(3, 32, dtype=bf), dt=torch.zeros(3, 32), A=torch.zeros(32, 16), B=torch.zeros(3, 16, dtype=bf),
                C=torch.zeros(3, 16, dtype=bf), state=torch.zeros(2, 32, 16))
    for good in (head, chan):
        with pytest.raises(ValueError, match="GPU tensor"):
            S.ssm_fwd_varlen(query_start_loc=qsl, **good)
        with pytest.raises(ValueError, match="GPU tensor"):
            S.ssm_update(**good)
        x = good["x"]
        for bad in (dict(x=x[:2]), dict(dt=good["dt"][:, :3]), dict(A=good["A"][:3]), dict(B=good["B"][:2]), dict(C=good["C"][..., :5]),
                    dict(state=good["state"][:, :3]), dict(state=good["state"][..., :5]), dict(out=x[:1]), dict(z=x[:1]),
                    dict(D=torch.zeros(3)), dict(dt_bias=torch.zeros(3)), dict(A=torch.zeros(2, 2, 2)), dict(x=x[0])):
            with pytest.raises(ValueError):
                S.ssm_fwd_varlen(query_start_loc=qsl, **{**good, **bad})
            with pytest.raises(ValueError):
                S.ssm_update(**{**good, **bad})
        with pytest.raises(ValueError, match="num_accepted_tokens"):
            S.ssm_update(**good, num_accepted_tokens=qsl)
        with pytest.raises(ValueError, match="output_state_indices"):
            S.ssm_update(**good, output_state_indices=qsl)
        with pytest.raises(ValueError, match="state is required"):
            S.ssm_update(**{**good, "state": None})
    with pytest.raises(ValueError):
        S.ssm_fwd_varlen(query_start_loc=qsl, **{**head, "B": torch.zeros(3, 3, 16, dtype=bf), "C": torch.zeros(3, 3, 16, dtype=bf)})
    x = torch.zeros(3, 32, dtype=bf)
    with pytest.raises(ValueError, match="GPU tensor"):
        S.sconv_group_norm(x)
    for bad in (dict(group_size=5), dict(group_size=0), dict(weight=torch.zeros(5, dtype=bf)), dict(bias=torch.zeros(5, dtype=bf)),
                dict(z=x[:2]), dict(out=x[:2]), dict(norm="batch"), dict(activation="relu"), dict(gate_first=True), dict(x=x[0]),
                dict(x=x.view(3, 4, 8), group_size=4)):
        with pytest.raises(ValueError):
            S.sconv_group_norm(**{"x": x, **bad})
