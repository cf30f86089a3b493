"""quant_ref.near, by which attention over held rows is judged, tells kernels that drop bits
from those that do not: the definition with fewer bits of P or Q, on the CPU."""
import pytest
import torch

import quant_ref as ref


def cut(x, pieces):
    """The first bf16 pieces of fp32 numbers, cut off after 8 bits each."""
    x, got = x.float(), torch.zeros_like(x, dtype=torch.float32)
    for _ in range(pieces):
        y = (x - got).view(torch.int32) & -65536
        got = got + y.view(torch.float32)
    return got.double()


def one(t, d, bits, p_of=lambda p: p, q_of=lambda q: q, dtype=torch.float32, seed=0):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((48, d), generator=g).to(dtype)
    k, v = (torch.randn((t, d), generator=g) for _ in range(2))
    k[:, ::41] = 3 * k[:, ::41] + 6
    k, v = (ref.stands(x.to(dtype), bits) for x in (k, v))

    def out(q, p_of):
        x = q @ k.T * d ** -0.5
        p = torch.exp(x - x.amax(-1, keepdim=True))
        return p_of(p) @ v / p.sum(-1, keepdim=True)
    return out(q_of(q.float()).double(), p_of).to(dtype), out(q.double(), lambda p: p)


SIZES = [(4000, 128), (2500, 128), (2700, 80), (1000, 256), (60, 64)]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("t,d", SIZES)
def test_fp32_with_fewer_pieces_is_far(t, d, bits):
    assert ref.near(*one(t, d, bits)) is None
    assert ref.near(*one(t, d, bits, p_of=lambda p: cut(p, 3), q_of=lambda q: cut(q, 3))) is None
    for n in (1, 2):
        assert ref.near(*one(t, d, bits, p_of=lambda p: cut(p, n))) is not None
        assert ref.near(*one(t, d, bits, q_of=lambda q: cut(q, n))) is not None


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("t,d", SIZES)
def test_bf16_with_one_term_is_far(t, d, bits):
    bf16 = torch.bfloat16
    assert ref.near(*one(t, d, bits, dtype=bf16)) is None
    two = lambda p: p.to(bf16).double() + (p - p.to(bf16).double()).to(bf16).double()  # noqa: E731
    assert ref.near(*one(t, d, bits, p_of=two, dtype=bf16)) is None
    assert ref.near(*one(t, d, bits, p_of=lambda p: p.to(bf16).double(), dtype=bf16)) is not None
    assert ref.near(*one(t, d, bits, p_of=lambda p: p.to(torch.float16).double(), dtype=bf16)) is not None
