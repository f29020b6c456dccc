"""CPU pins of the plain definitions the serving operators are tested against,
and the host-side refusals of those operators."""
import numpy as np
import pytest
import torch

import plain_serving as plain


@pytest.fixture(scope="module")
def sv():
    from speculative_decoding_verification_vocab_gb300 import _build
    _build.build()
    import speculative_decoding_verification_vocab_gb300 as m
    m.load_library()
    return m


def test_verification_keeps_the_targets_law():
    """Drafts from p, uniforms on a dense grid: the first emitted token follows
    q, within the grid's step; a walk that swaps the rows does not."""
    q = np.array([[0.5, 0.25, 0.125, 0.125]] * 2, np.float32)
    p = np.array([[0.125, 0.125, 0.5, 0.25]], np.float32)
    G = 64
    u = (np.arange(G, dtype=np.float32) + 0.5) / G

    def law(q, p):
        mass = np.zeros(4)
        for d in range(4):
            for a in u:
                for s in u:
                    t, _, st = plain.verify_one(q, p, np.array([d]), np.array([a]), s)
                    assert st == 0
                    mass[t[0]] += p[0, d] / (G * G)
        return mass
    assert np.abs(law(q, p) - q[0]).max() < 2 / G
    wrong = np.concatenate([p, p])
    assert np.abs(law(wrong, q[:1]) - q[0]).max() > 0.1


def test_one_hot_equals_a_point_mass():
    rng = np.random.default_rng(0)
    for _ in range(50):
        q = rng.dirichlet(np.ones(9), 4).astype(np.float32)
        d = rng.integers(0, 9, 3)
        p = np.zeros((3, 9), np.float32)
        p[np.arange(3), d] = 1
        ua, us = rng.random(3, np.float32) * 0.3, np.float32(rng.random())
        assert plain.verify_one(q, None, d, ua, us) == plain.verify_one(q, p, d, ua, us)


def test_draw_is_the_inverse_cdf():
    rng = np.random.default_rng(1)
    for _ in range(200):
        w = rng.random(50).astype(np.float32)
        u = np.float32(rng.random())
        c = np.cumsum(w.astype(np.float64))
        near = np.abs(c - u * c[-1]).min() < 1e-12
        assert near or plain._draw(w, u) == int((c <= np.float64(u) * c[-1]).sum())


def test_verify_probs_host_checks(sv):
    """Bad arguments are refused before any CUDA call (no GPU here)."""
    f = sv.load_library().sv_verify_chain_probs
    x = 4096  # never looked at: the refusals below come first

    def call(ldq=10, p=None, ldp=10, dt=0, d=x, n=None, ua=x, us=x, B=1, N=2, V=10, t=x, a=x, s=x,
             q=x):
        return f(q, ldq, p, ldp, dt, d, n, ua, us, B, N, V, t, a, s, None)
    assert call(B=-1) == 1 and call(N=-1) == 1 and call(V=0) == 1
    assert call(dt=2) == 1 and b"SV_F32" in sv.load_library().sv_last_error()
    assert call(ldq=9) == 1 and call(p=x, ldp=9) == 1
    assert b"stride" in sv.load_library().sv_last_error()
    assert call(ldq=2 ** 61) == 1
    assert call(V=(1 << 22) + 1, ldq=1 << 23) == 2 and call(N=1025) == 2
    assert call(q=None) == 1 and call(us=None) == 1 and call(d=None) == 1 and call(ua=None) == 1
    assert call(t=None) == 1 and call(a=None) == 1 and call(s=None) == 1
    assert b"null" in sv.load_library().sv_last_error()
    assert call(q=x + 2) == 1 and call(us=x + 1) == 1
    assert b"misaligned" in sv.load_library().sv_last_error()
    assert call(B=0, q=None, us=None) == 0


def test_verify_probs_binding_refusals(sv):
    q, p = torch.zeros(2, 3, 8), torch.zeros(2, 2, 8)
    d, ua, us = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2), torch.zeros(2)
    o = (torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
         torch.zeros(2, dtype=torch.int32))

    def call(q=q, p=p, d=d, n=None, ua=ua, us=us, o=o):
        with pytest.raises(ValueError):
            sv.sv_verify_chain_probs(q, p, d, n, ua, us, *o)
    call(p=p.bfloat16())                                   # another type than q
    call(p=torch.zeros(2, 3, 8))                           # another shape
    call(q=torch.zeros(2, 8, 3).transpose(1, 2))           # columns apart
    call(q=torch.zeros(4, 3, 8)[::2])                      # sequences apart
    call(d=d.long()), call(ua=ua.double()), call(us=us[:1])
    call(n=torch.zeros(3, dtype=torch.int32))
    call(d=torch.zeros(2, 4, dtype=torch.int32)[:, ::2])
    call()                                                 # pageable host memory
