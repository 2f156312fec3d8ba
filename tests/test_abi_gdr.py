"""Refusals of the gated delta rule and of draft verification at the C ABI:
bad host arguments come back with the documented status before anything is
launched (no GPU needed; accepted calls reach the launch and fail there)."""
import ctypes

import pytest
import torch

import causal_depthwise_short_conv1d_amd as S
from tests.test_abi import BASE, EALIAS, EALIGN, EARG, ELAUNCH, ENULL, ESHAPE, ESTRIDE, GB, OK, addr, no_gpu


@pytest.fixture(scope="module")
def lib():
    return S.load_library()


def status(lib, name, *args):
    """What a call returns, packed into words or not."""
    rc = getattr(lib, name)(*args)
    words = (ctypes.c_uint64 * len(args))()
    for i, (a, t) in enumerate(zip(args, getattr(lib, name).argtypes)):
        v = t(a) if not isinstance(a, ctypes.c_void_p) else a
        ctypes.memmove(ctypes.addressof(words) + 8 * i, ctypes.byref(v), ctypes.sizeof(v))
    packed = getattr(lib, name + "_packed")
    assert packed(bytes(words)) == rc
    assert packed(None) == ENULL
    return rc


def fwd(lib, **kw):
    no_gpu()
    a = dict(q=addr(1), qs=(256, 64, 1), k=addr(2), ks=(256, 64, 1), v=addr(3), vs=(512, 64, 1),
             g=addr(4), gs=(8, 1), b=addr(5), bs=(8, 1), al=None, dt=None, st=addr(6),
             ss=(8 * 64 * 64, 64 * 64, 64, 1), lines=4, ci=addr(7), hi=addr(8), qsl=addr(9), batch=2, T=10, hk=4,
             hv=8, dk=64, dv=64, scale=1.0, l2=1, pad=-1, o=addr(10), os=(512, 64, 1), ws=None, wb=0)
    a.update(kw)
    return status(lib, "gdr_fwd_varlen", a["q"], *a["qs"], a["k"], *a["ks"], a["v"], *a["vs"], a["g"], *a["gs"], a["b"],
                              *a["bs"], a["al"], a["dt"], a["st"], *a["ss"], a["lines"], a["ci"], a["hi"], a["qsl"],
                              a["batch"], a["T"], a["hk"], a["hv"], a["dk"], a["dv"], a["scale"], a["l2"], a["pad"],
                              a["o"], *a["os"], a["ws"], a["wb"], None)


def test_fwd_workspace(lib):
    need = lib.gdr_fwd_workspace_bytes(2, 1000, 4, 8, 64, 64, 1)
    assert need > 0
    assert fwd(lib, T=1000, ws=addr(11), wb=need) == ELAUNCH
    assert fwd(lib, T=1000, ws=addr(11), wb=need - 1) == ESHAPE
    assert fwd(lib, T=1000, ws=ctypes.c_void_p(BASE + 11 * GB + 8), wb=need) == EALIGN
    for x in (1, 2, 3, 4, 5, 6, 10):
        assert fwd(lib, T=1000, ws=addr(x), wb=need) == EALIAS, x
    assert lib.gdr_fwd_workspace_bytes(2, 128, 4, 8, 64, 64, 1) == 0            # short sequences: one kernel
    assert lib.gdr_fwd_workspace_bytes(2, 129, 4, 8, 64, 64, 1) > 0
    assert lib.gdr_fwd_workspace_bytes(8, 2048, 4, 32, 64, 64, 1) == 0          # more heads: longer ones
    assert lib.gdr_fwd_workspace_bytes(8, 2049, 4, 32, 64, 64, 1) > 0
    assert lib.gdr_fwd_workspace_bytes(2000, 10, 4, 8, 64, 64, 1) == 0          # many heads: one kernel
    assert lib.gdr_fwd_workspace_bytes(2000, 64000, 4, 8, 64, 64, 0) == 0       # short sequences, by elements
    assert lib.gdr_fwd_workspace_bytes(2000, 64001, 4, 8, 64, 64, 0) > 0
    # more threads than a launch can have: the prepared chunks', the walk's
    assert lib.gdr_fwd_workspace_bytes(1, 1 << 26, 1, 8, 64, 64, 1) > 0
    assert lib.gdr_fwd_workspace_bytes(1, 1 << 26, 8, 8, 64, 64, 1) == 0
    assert lib.gdr_fwd_workspace_bytes(1 << 20, 1 << 26, 1, 1, 64, 64, 0) > 0
    assert lib.gdr_fwd_workspace_bytes(1 << 20, 1 << 26, 1, 16, 64, 64, 0) == 0
    for bad in ((0, 1000, 4, 8, 64, 64, 1), (2, 0, 4, 8, 64, 64, 1), (2, 1000, 0, 8, 64, 64, 1),
                (2, 1000, 4, 8, 129, 64, 1), (2, 1000, 4, 8, 64, 0, 1), (2, 1000, 3, 8, 64, 64, 1),
                ((1 << 31) - 1, 1 << 30, 1, (1 << 31) - 1, 64, (1 << 31) - 1, 0)):
        assert lib.gdr_fwd_workspace_bytes(*bad) == 0


def test_fwd_accepted(lib):
    assert fwd(lib) == ELAUNCH
    assert fwd(lib, st=None, hi=None, lines=0) == ELAUNCH
    assert fwd(lib, al=addr(11), dt=addr(12)) == ELAUNCH
    assert fwd(lib, qs=(0, 0, 0)) == ELAUNCH                    # one query for every token: read only
    assert fwd(lib, q=ctypes.c_void_p(BASE + GB + 2)) == ELAUNCH
    assert fwd(lib, dk=37, dv=3, ss=(8 * 37 * 3, 37 * 3, 37, 1)) == ELAUNCH


def test_fwd_empty_is_a_noop(lib):
    assert fwd(lib, T=0, q=None, qsl=None) == OK
    assert fwd(lib, batch=0, q=None) == OK


def test_fwd_nulls(lib):
    for x in ("q", "k", "v", "g", "b", "o", "qsl"):
        assert fwd(lib, **{x: None}) == ENULL, x
    assert fwd(lib, st=None) == ENULL                           # has_initial_state needs a state
    assert fwd(lib, al=addr(11)) == ENULL
    assert fwd(lib, dt=addr(11)) == ENULL


def test_fwd_sizes(lib):
    for kw in (dict(batch=-1), dict(T=-1), dict(T=1 << 31), dict(T=(1 << 31) - 256), dict(hk=0), dict(hv=0), dict(hk=3), dict(dk=0), dict(dv=0),
               dict(dk=257, ss=(1 << 30, 1 << 24, 257, 1)), dict(lines=0), dict(ci=None, lines=1), dict(lines=-1),
               dict(batch=1 << 30)):
        assert fwd(lib, **kw) == ESHAPE, kw
    assert fwd(lib, scale=float("nan")) == EARG
    assert fwd(lib, scale=float("inf")) == EARG


def test_fwd_strides(lib):
    for x in ("qs", "ks", "vs", "os"):
        assert fwd(lib, **{x: (512, -64, 1)}) == ESTRIDE, x
    assert fwd(lib, gs=(-8, 1)) == ESTRIDE
    assert fwd(lib, os=(512, 32, 1)) == ESTRIDE                 # heads of out overlap
    assert fwd(lib, os=(0, 64, 1)) == ESTRIDE
    assert fwd(lib, ss=(0, 64 * 64, 64, 1)) == ESTRIDE          # lines overlap
    assert fwd(lib, ss=(8 * 64 * 64, 64 * 64, 63, 1)) == ESTRIDE


def test_fwd_alignment_and_overlap(lib):
    for x in ("q", "k", "v", "o"):
        assert fwd(lib, **{x: ctypes.c_void_p(BASE + 20 * GB + 1)}) == EALIGN, x
    for x in ("g", "b", "st", "ci", "qsl"):
        assert fwd(lib, **{x: ctypes.c_void_p(BASE + 20 * GB + 2)}) == EALIGN, x
    for x in (1, 2, 3, 4, 5, 6):
        assert fwd(lib, o=addr(x)) == EALIAS, x
    for x in (1, 2, 3, 4, 5):
        assert fwd(lib, st=addr(x)) == EALIAS, x


def update(lib, **kw):
    no_gpu()
    a = dict(q=addr(1), qs=(1024, 256, 64, 1), k=addr(2), ks=(1024, 256, 64, 1), v=addr(3), vs=(2048, 512, 64, 1),
             g=addr(4), gs=(32, 8, 1), b=addr(5), bs=(32, 8, 1), al=None, dt=None, st=addr(6),
             ss=(8 * 64 * 64, 64 * 64, 64, 1), lines=16, ci=addr(7), cs=(4, 1), steps=4, acc=addr(8), osi=addr(9),
             osis=(4, 1), batch=2, seqlen=4, hk=4, hv=8, dk=64, dv=64, scale=1.0, l2=0, pad=-1, o=addr(10),
             os=(2048, 512, 64, 1))
    a.update(kw)
    return status(lib, "gdr_update", a["q"], *a["qs"], a["k"], *a["ks"], a["v"], *a["vs"], a["g"], *a["gs"], a["b"], *a["bs"],
                          a["al"], a["dt"], a["st"], *a["ss"], a["lines"], a["ci"], *a["cs"], a["steps"], a["acc"],
                          a["osi"], *a["osis"], a["batch"], a["seqlen"], a["hk"], a["hv"], a["dk"], a["dv"],
                          a["scale"], a["l2"], a["pad"], a["o"], *a["os"], None)


def test_update_refusals(lib):
    assert update(lib) == ELAUNCH
    assert update(lib, acc=None, osi=None, ci=None) == ELAUNCH
    assert update(lib, batch=0, q=None) == OK
    assert update(lib, seqlen=0, q=None) == OK
    for x in ("q", "k", "v", "g", "b", "st", "o", "ci"):        # ci: num_accepted_tokens needs it
        assert update(lib, **{x: None}) == ENULL, x
    for kw in (dict(batch=-1), dict(seqlen=-1), dict(steps=0), dict(lines=0), dict(ci=None, acc=None, lines=1),
               dict(hk=3), dict(dk=300, ss=(1 << 30, 1 << 20, 300, 1))):
        assert update(lib, **kw) == ESHAPE, kw
    for kw in (dict(cs=(-1, 0)), dict(osis=(4, -1)), dict(qs=(-1, 256, 64, 1)), dict(os=(2048, 512, 63, 1)),
               dict(ss=(1, 64 * 64, 64, 1))):
        assert update(lib, **kw) == ESTRIDE, kw
    for x in ("acc", "osi", "ci"):
        assert update(lib, **{x: ctypes.c_void_p(BASE + 20 * GB + 1)}) == EALIGN, x
    assert update(lib, o=addr(3)) == EALIAS                     # out may not be v
    assert update(lib, o=addr(6)) == EALIAS


def verify(lib, **kw):
    no_gpu()
    a = dict(t=addr(1), s=addr(2), p=addr(3), ps=1000, q=addr(4), qs=1000, ua=addr(5), us=addr(6), batch=3, nd=7,
             V=1000, most=4, o=addr(7), os=5, n=addr(8), ws=addr(9), wb=None)
    a.update(kw)
    wb = lib.sconv_verify_workspace_bytes(a["batch"], a["V"]) if a["wb"] is None else a["wb"]
    return lib.sconv_verify_drafts(a["t"], a["s"], a["p"], a["ps"], a["q"], a["qs"], a["ua"], a["us"], a["batch"],
                                   a["nd"], a["V"], a["most"], a["o"], a["os"], a["n"], a["ws"], wb, None)


def test_verify_refusals(lib):
    assert verify(lib) == ELAUNCH
    assert verify(lib, q=None) == ELAUNCH
    assert verify(lib, nd=0, t=None, ua=None, most=0, os=1) == ELAUNCH
    assert verify(lib, ps=0, qs=0) == ELAUNCH                   # one row for all: read only
    assert verify(lib, batch=0, p=None) == OK
    for x in ("t", "s", "p", "ua", "us", "o", "n", "ws"):
        assert verify(lib, **{x: None}) == ENULL, x
    for kw in (dict(batch=-1, wb=0), dict(nd=-1), dict(V=0, wb=99), dict(V=-1, wb=99), dict(most=-1), dict(wb=8),
               dict(V=(1 << 30) + 1, ps=1 << 31, qs=1 << 31), dict(most=(1 << 31) - 1)):
        assert verify(lib, **kw) == ESHAPE, kw
    for kw in (dict(ps=-1), dict(qs=-1), dict(os=4)):
        assert verify(lib, **kw) == ESTRIDE, kw
    for x in ("t", "s", "p", "q", "ua", "us", "o", "n"):
        assert verify(lib, **{x: ctypes.c_void_p(BASE + 20 * GB + 2)}) == EALIGN, x
    assert verify(lib, ws=ctypes.c_void_p(BASE + 20 * GB + 4)) == EALIGN
    for x in (1, 2, 3, 4, 5, 6):
        assert verify(lib, o=addr(x)) == EALIAS, x
    assert verify(lib, n=addr(7)) == EALIAS
    assert verify(lib, ws=addr(3)) == EALIAS


def test_workspace_bytes(lib):
    f = lib.sconv_verify_workspace_bytes
    assert f(0, 1000) == 0 and f(3, 0) == 0 and f(-1, 5) == 0
    assert f(1, 1) == 16 + 8 and f(2, 1024) == 32 + 8
    assert f(1 << 20, 1 << 20) % 8 == 0 and f(1 << 20, 1 << 20) > 1 << 24


def test_binding_refusals():
    q = torch.zeros(3, 2, 16, dtype=torch.bfloat16)
    v = torch.zeros(3, 4, 8, dtype=torch.bfloat16)
    g = torch.zeros(3, 4)
    st = torch.zeros(2, 4, 8, 16)
    qsl = torch.tensor([0, 3], dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU tensor"):
        S.gdr_fwd_varlen(q, q, v, g, g, st, qsl)
    for bad in (dict(k=q[:, :1]), dict(v=v[:2]), dict(v=v[:, :3]), dict(g=g[:2]), dict(beta=g[:, :2]),
                dict(state=st[:, :2]), dict(out=v[:1]), dict(A_log=g[0]), dict(q=q[0])):
        a = dict(q=q, k=q, v=v, g=g, beta=g, state=st)
        a.update(bad)
        with pytest.raises(ValueError):
            S.gdr_fwd_varlen(a.pop("q"), a.pop("k"), a.pop("v"), a.pop("g"), a.pop("beta"), a.pop("state"), qsl, **a)
        with pytest.raises(ValueError):
            a = dict(q=q, k=q, v=v, g=g, beta=g, state=st)
            a.update(bad)
            S.gdr_update(a.pop("q"), a.pop("k"), a.pop("v"), a.pop("g"), a.pop("beta"), a.pop("state"), **a)
    with pytest.raises(ValueError, match="num_accepted_tokens"):
        S.gdr_update(q, q, v, g, g, st, num_accepted_tokens=qsl)
    with pytest.raises(ValueError, match="output_state_indices"):
        S.gdr_update(q, q, v, g, g, st, output_state_indices=qsl)
    p = torch.zeros(4, 10)
    x = torch.zeros(3, dtype=torch.int32)
    u = torch.zeros(3)
    with pytest.raises(ValueError, match="GPU tensor"):
        S.sconv_verify_drafts(x, qsl, p, None, u, u, 3)
    for bad in (dict(target_probs=p[:3]), dict(draft_probs=p[:2]), dict(draft_probs=p[:3, :5]),
                dict(target_probs=torch.zeros(10, 4).t()), dict(tokens=torch.zeros(1, 3, dtype=torch.int32))):
        a = dict(draft_tokens=x, draft_start_loc=qsl, target_probs=p, draft_probs=None, accept_uniform=u,
                 sample_uniform=u, max_drafts=3)
        a.update(bad)
        with pytest.raises(ValueError):
            S.sconv_verify_drafts(**a)
