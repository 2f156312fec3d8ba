"""GPU parity of draft verification: tokens and counts equal those of the
64-bit definition."""
import pytest
import torch

import causal_depthwise_short_conv1d_amd as S
from tests import gdr_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


def draw(counts, V, seed, with_q=True, sparse=False, agree=0.7):
    gen = torch.Generator().manual_seed(seed)
    nd, rows = sum(counts), sum(counts) + len(counts)
    logits = torch.randn(rows, V, generator=gen) * 2
    if sparse:
        logits[torch.rand(rows, V, generator=gen) < 0.9] = float("-inf")
        logits[:, V // 2] = 0.0
    p = torch.softmax(logits, -1)
    own = torch.cat([torch.arange(c) + sum(counts[:i]) + i for i, c in enumerate(counts)] or [torch.zeros(0)]).long()
    q = torch.softmax(logits[own] * agree + torch.randn(nd, V, generator=gen) * (1 - agree), -1)
    tok = torch.multinomial(q, 1, generator=gen)[:, 0].to(torch.int32) if nd else torch.zeros(0, dtype=torch.int32)
    start = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32)
    return dict(tokens=tok, start=start, p=p, q=q if with_q else None, ua=torch.rand(nd, generator=gen),
                us=torch.rand(len(counts), generator=gen))


def put(t):
    return None if t is None else t.to(DEV)


def check(d, most, view=None):
    want = R.verify(d["tokens"], d["start"], d["p"], d["q"], d["ua"], d["us"], most)
    p, q = put(d["p"]), put(d["q"])
    if view:
        p, q = view(p), None if q is None else view(q)
    got = S.sconv_verify_drafts(put(d["tokens"]), put(d["start"]), p, q, put(d["ua"]), put(d["us"]), most)
    torch.cuda.synchronize()
    assert torch.equal(got[1].cpu(), want[1])
    assert torch.equal(got[0].cpu(), want[0])
    return want


@pytest.mark.parametrize("V", [1, 2, 63, 64, 65, 255, 256, 257, 1000, 1023, 1024, 1025, 4097, 32000, 100003])
@pytest.mark.parametrize("with_q", [True, False])
def test_vocabularies(V, with_q):
    check(draw([3, 0, 1, 4], V, V, with_q), 4)


@pytest.mark.parametrize("counts", [[0], [1], [0, 0, 0], [5] * 33, [1, 0, 7, 2] * 20])
@pytest.mark.parametrize("sparse", [False, True])
def test_batches(counts, sparse):
    check(draw(counts, 777, len(counts), sparse=sparse), max(counts))


def test_long_draft_lists_and_clamped_ones():
    d = draw([130, 70, 3], 200, 3, agree=1.0)
    d["q"] = torch.cat([d["p"][:130], d["p"][131:201], d["p"][202:205]]) * 0.999    # nearly all stand
    d["ua"] *= 1.0
    want = check(d, 130)
    assert want[1].max() > 65                          # past the first ballot
    check(d, 100)                                      # drafts behind max_drafts are not looked at
    check(d, 0)


def test_rows_without_mass_and_odd_values():
    d = draw([2, 2, 2, 2, 1, 1], 500, 4)
    d["p"][:3] = 0                                     # no mass: refused, index 0
    d["q"][2] = d["p"][3] * 2                          # nothing is left of p - q: drawn from p
    d["ua"][2] = 0.9
    d["p"][6, 5:400] = float("nan")                    # NaN and negative entries have no mass
    d["p"][7, :50] = -1.0
    d["us"][3], d["us"][4], d["us"][5] = 0.0, 1.0, 0.99999994
    d["tokens"][8] = 500                               # outside the vocabulary
    d["tokens"][9] = -3
    check(d, 2)
    d["q"] = None
    check(d, 2)


def test_greedy_rows():
    """One-hot targets: drafts stand while they are the target's token."""
    V, counts = 3000, [4, 4, 4]
    d = draw(counts, V, 5, with_q=False)
    best = d["p"].argmax(-1)
    d["p"] = torch.nn.functional.one_hot(best, V).float()
    rows = best.view(3, 5)
    d["tokens"] = rows[:, :4].reshape(-1).to(torch.int32).clone()
    d["tokens"][6] = (d["tokens"][6] + 1) % V
    want = check(d, 4)
    assert want[1].tolist() == [5, 3, 5]
    assert want[0][1].tolist() == rows[1, :3].tolist() + [-1, -1]


def test_pitched_rows():
    def view(t):
        b = torch.full((t.shape[0], t.shape[1] + 5), 9.0, device=DEV)
        b[:, 3:3 + t.shape[1]] = t
        return b[:, 3:3 + t.shape[1]]
    check(draw([2, 3], 1537, 6), 3, view)


def test_rows_past_32_bits():
    """Row offsets above 2^31 elements."""
    V, rows = 1 << 20, 2100
    p = torch.zeros(rows, V, device=DEV)
    p[-1, 12345] = 0.25
    p[-1, V - 1] = 0.75
    nd = rows - 1
    start = torch.tensor([0, nd], dtype=torch.int32, device=DEV)
    tok = torch.zeros(nd, dtype=torch.int32, device=DEV)
    p[:, 0] = 1.0
    p[-1, 0] = 0.0
    u = torch.zeros(nd, device=DEV)
    for us, want in ((0.1, 12345), (0.3, V - 1)):
        t, a = S.sconv_verify_drafts(tok, start, p, None, u, torch.tensor([us], device=DEV), nd)
        assert a.item() == rows and t[0, -1].item() == want


def test_graph_replays_and_two_at_once():
    a, b = draw([3] * 9, 5000, 7), draw([2, 0, 3] * 3, 5000, 8)
    for d in (a, b):
        for x in d:
            d[x] = put(d[x])

    def call(d):
        return S.sconv_verify_drafts(d["tokens"], d["start"], d["p"], d["q"], d["ua"], d["us"], 3)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(3):                                 # two streams at once, each with its own workspace
        with torch.cuda.stream(s1):
            got.append((call(a), a))
        with torch.cuda.stream(s2):
            got.append((call(b), b))
    torch.cuda.synchronize()
    graphs = []
    for d in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r = call(d)
        graphs.append((g, r, d))
    for r, d in got:
        w = R.verify(*(d[x].cpu() for x in ("tokens", "start", "p", "q", "ua", "us")), 3)
        assert torch.equal(r[0].cpu(), w[0]) and torch.equal(r[1].cpu(), w[1])
    for i in range(3):
        for g, r, d in graphs:
            d["us"].copy_(torch.rand(9, generator=torch.Generator().manual_seed(i)))
            g.replay()
        torch.cuda.synchronize()
        for g, r, d in graphs:
            w = R.verify(*(d[x].cpu() for x in ("tokens", "start", "p", "q", "ua", "us")), 3)
            assert torch.equal(r[0].cpu(), w[0]) and torch.equal(r[1].cpu(), w[1]), i
