"""The references of the learner's block operators, pinned (CPU): the
generator against its published answers, the codes against the format."""

import numpy as np
import torch

import block_refs as B


def test_philox_known_answers():
    f = 0xFFFFFFFF
    cases = [((0, 0, 0, 0), (0, 0), "6627e8d5 e169c58d bc57ac4c 9b00dbd8"),
             ((f, f, f, f), (f, f), "408f276d 41c83b0e a20bc7c6 6d5451fd"),
             ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
              "d16cfe09 94fdcceb 5001e420 24126ea1")]
    for counter, key, want in cases:
        got = B.philox([np.array([c]) for c in counter], key)
        assert " ".join("%08x" % int(w[0]) for w in got) == want


def test_keep_factors_of_pieces_are_the_wholes():
    whole = B.keep_factors(9, 50, 0.3, 12345678901234, site=7, first_row=2 ** 32 - 4)
    assert torch.equal(B.keep_factors(4, 50, 0.3, 12345678901234, 7, 2 ** 32 + 1), whole[5:])
    assert torch.equal(B.keep_factors(9, 13, 0.3, 12345678901234, 7, 2 ** 32 - 4), whole[:, :13])
    assert abs(float((whole == 0).double().mean()) - 0.3) < 0.1
    assert set(whole.unique().tolist()) == {0.0, 65536 / (65536 - 19661)}
    assert not bool(B.keep_factors(2, 9, 1.0, 1).any()) and bool((B.keep_factors(2, 9, 0.0, 1) == 1).all())


def test_codes():
    x = torch.randn(130, 200, generator=torch.Generator().manual_seed(0))
    x[3] = 0
    q, s = B.blocks(x)
    assert q.shape == (130, 256) and s.shape == (2, 130) and float(s[0, 3]) == 1.0 and not bool(q[:, 200:].any())
    back = (B.values(q).view(130, 2, 128) * s.double().t()[:, :, None]).view(130, 256)[:, :200]
    assert bool(((back - x.double()).abs() <= 2.0 ** -4 * x.double().abs() + 2.0 ** -10 * x.abs().max()).all())
    q, s = B.tiles(x)
    assert q.shape == (130, 256) and s.shape == (2, 2)
    assert float(s[1, 1]) == float(torch.tensor(float(x[128:, 128:].abs().max())) / 448)
    p, mag = B.product(q, s[[0]].t().expand(2, 130).contiguous(), q, s)
    assert p.shape == (130, 130) and bool((p.abs() <= mag * (1 + 1e-12)).all())
