"""Pins the 64-bit references of the gated delta rule and of draft verification
on the CPU: against the chunked closed form, by splitting a sequence, and by
the distribution that rejection sampling keeps."""
import numpy as np
import pytest
import torch

from tests import gdr_ref as R


def chunked(q, k, v, g, beta, S, chunk):
    """One sequence by chunks: T = (I + A)^-1, U = T (beta v - beta e^G K S^T)."""
    n = q.shape[0]
    out = torch.zeros(v.shape, dtype=R.F64)
    for a in range(0, n, chunk):
        s = slice(a, min(n, a + chunk))
        m = s.stop - a
        for h in range(v.shape[1]):
            K, Q, V, b = k[s, h], q[s, h], v[s, h], beta[s, h]
            G = g[s, h].cumsum(0)
            D = torch.exp(G[:, None] - G[None]).tril()
            A = (b[:, None] * D * (K @ K.T)).tril(-1)
            T = torch.linalg.inv(torch.eye(m, dtype=R.F64) + A)
            U = T @ (b[:, None] * (V - torch.exp(G)[:, None] * (K @ S[h].T)))
            out[s, h] = torch.exp(G)[:, None] * (Q @ S[h].T) + (D * (Q @ K.T)) @ U
            S[h] = torch.exp(G[-1]) * S[h] + U.T @ (torch.exp(G[-1] - G)[:, None] * K)
    return out, S


@pytest.mark.parametrize("n,chunk,raw", [(1, 64, True), (37, 16, True), (130, 64, False)])
def test_recurrence_is_the_chunked_form(n, chunk, raw):
    d = R.draw_inputs((n,), 2, 4, 24, 12, seed=n, raw=raw)
    S0 = torch.randn(3, 4, 12, 24)
    out, _, st, _, _ = R.fwd(**d, state=S0, qsl=[0, n], cache_indices=[1], has_init=[True], scale=0.3, l2norm=True,
                             c=1, f=1)
    q, k = R.norm_qk(d["q"], d["k"], 0.3, True, 4)
    g, b = R.gates(d["g"], d["beta"], d["A_log"], d["dt_bias"])
    o2, S2 = chunked(q, k, d["v"].double(), g, b, S0[1].double().clone(), chunk)
    # 64-bit sums of some hundred terms: 1e-12 leaves a factor of a hundred
    assert torch.allclose(out, o2, rtol=1e-12, atol=1e-12)
    assert torch.allclose(st[1], S2, rtol=1e-12, atol=1e-12)
    assert torch.equal(st[0], S0[0].double()) and torch.equal(st[2], S0[2].double())


def test_a_split_sequence_and_decode_continue_the_state():
    d = R.draw_inputs((9,), 1, 2, 16, 8, seed=5)
    S0 = torch.zeros(1, 2, 8, 16)
    whole = R.fwd(**d, state=S0, qsl=[0, 9], cache_indices=None, has_init=None, scale=1.0, l2norm=True, c=1, f=1)
    part = {x: (d[x][:4] if x in ("q", "k", "v", "g", "beta") else d[x]) for x in d}
    rest = {x: (d[x][4:].unsqueeze(0) if x in ("q", "k", "v", "g", "beta") else d[x]) for x in d}
    a = R.fwd(**part, state=S0, qsl=[0, 4], cache_indices=None, has_init=None, scale=1.0, l2norm=True, c=1, f=1)
    b = R.update(**rest, state=a[2], cache_indices=None, accepted=None, osi=None, scale=1.0, l2norm=True)
    assert torch.allclose(torch.cat([a[0], b[0][0]]), whole[0], rtol=1e-12, atol=1e-13)
    assert torch.allclose(b[2], whole[2], rtol=1e-12, atol=1e-13)


def test_verification_keeps_the_target_distribution():
    """Whatever the draft's distribution, the first token is distributed as the target's."""
    V, N = 5, 20000
    gen = torch.Generator().manual_seed(1)
    p = torch.tensor([0.4, 0.1, 0.0, 0.3, 0.2])
    q = torch.tensor([0.1, 0.5, 0.2, 0.2, 0.0])
    draft = torch.multinomial(q, N, replacement=True, generator=gen).to(torch.int32)
    rows = p.expand(2 * N, V)
    tok, acc = R.verify(draft, torch.arange(N + 1), rows, q.expand(N, V), torch.rand(N, generator=gen),
                        torch.rand(N, generator=gen), 1)
    freq = np.bincount(tok[:, 0].numpy(), minlength=V) / N
    # five standard deviations of a frequency over 20000 draws: 5 * sqrt(.25 / 20000) = 0.018
    assert np.abs(freq - p.numpy()).max() < 0.018
    assert freq[2] == 0 and abs((acc == 2).float().mean().item() - torch.minimum(p, q).sum().item()) < 0.018
