"""orpo_head_logits_q where the result is known to the last bit.

Weights and rows of h that are small integers: every product and every partial sum is an integer below 2^24, exact in
fp32 in any order and whether adds round or truncate, so the logits have to be equal to the integers' own product.
One missing, doubled or misplaced product shows, at any d.  And weights on a tie: one-hot rows of h read single
weights out, which have to be scale q + bias rounded once.  A single row of h out of a wider buffer gives
the bits that it gives alone."""

from fractions import Fraction

import pytest
import torch

import orpo_preference_loss_gb300 as orpo
from gpu_helpers import dev, status_tensor

pytestmark = pytest.mark.gpu


def run(h, q, bits, group, out=None):
    st = status_tensor()
    out = torch.full((h.shape[0], q[0].shape[0]), float("nan"), device=dev()) if out is None else out
    orpo.orpo_head_logits_q(h, *q, bits, group, 0.0, out, st)
    assert int(st.item()) == 0
    return out


@pytest.mark.parametrize("M,d,V,bits,group", [
    (1, 256, 4096, 4, 64), (1, 2560, 40000, 4, 64), (3, 3840, 20000, 4, 32), (13, 3840, 20000, 4, 32),
    (16, 16384, 700, 4, 64), (20, 4096, 20000, 4, 128), (24, 3232, 9633, 4, 32), (33, 768, 4871, 4, 96),
    (64, 4096, 20000, 4, 128), (64, 16384, 333, 4, 64), (130, 1568, 2000, 4, 32), (8, 2048, 32000, 8, 32),
    (40, 4096, 5000, 8, 64), (3, 5376, 3000, 8, 64), (5, 8200, 500, 4, 8), (11, 4104, 500, 8, 24)])
def test_integers_are_exact(M, d, V, bits, group):
    """Weights q - 8 (8 bits: q - 128 of q in 120 .. 135), rows of h in -2 .. 2: sums stay below 16384 * 16 < 2^24."""
    g = torch.Generator("cuda").manual_seed(d + M)
    w = torch.randint(-8, 8, (V, d), generator=g, device=dev(), dtype=torch.int16)
    h = torch.randint(-2, 3, (M, d), generator=g, device=dev(), dtype=torch.int16)
    if bits == 4:
        u = (w + 8).to(torch.uint8)
        wq, bias = u[:, 0::2] | (u[:, 1::2] << 4), -8.0
    else:
        wq, bias = (w + 128).to(torch.uint8), -128.0
    sc = torch.ones((V, d // group), device=dev()).bfloat16()
    q = (wq.contiguous(), sc, torch.full_like(sc, bias))
    want = (h.double() @ w.double().T).float()
    hb = h.bfloat16()
    first = run(hb, q, bits, group)
    assert torch.equal(first, want)
    # small scales take another form of the dequantisation
    small = (q[0], sc * 2.0 ** -9, q[2] * 2.0 ** -9)
    assert torch.equal(run(hb, small, bits, group) * 512, want)
    for _ in range(10):
        assert torch.equal(run(hb, q, bits, group), want)


def bf16_once(x: Fraction) -> float:
    """x > 0 rounded to 8 significant bits, ties to even."""
    e = 0
    while x >= 256:
        x, e = x / 2, e + 1
    while x < 128:
        x, e = x * 2, e - 1
    n = x.numerator // x.denominator
    rest = x - n
    if rest > Fraction(1, 2) or (rest == Fraction(1, 2) and n % 2 == 1):
        n += 1
    return float(n) * 2.0 ** e


@pytest.mark.parametrize("offset", [0, 4, 8])
@pytest.mark.parametrize("bits,group", [(4, 32), (4, 8), (8, 32), (8, 16)])
@pytest.mark.parametrize("magnitude", [0, -12])
def test_weights_are_rounded_once(bits, group, offset, magnitude):
    """Products of scale and q that lie halfway between two bf16 values, with biases far below: which way they round is
    the bias's sign, on every kernel of the entry point (aligned weights and groups of 32 take another than the rest)."""
    if bits == 8 and offset == 4:
        pytest.skip("8-bit weights start on 8 bytes")
    d, ties = 64, [(77, 5), (35, 11), (55, 7), (91, 11), (111, 7), (43, 9)]  # scale (times 2^-7) and q: odd 9-bit products
    ties = [(s, q) for s, q in ties if 256 < s * q < 512 and s * q % 2 == 1]
    assert len(ties) >= 4
    V = 2 * len(ties)
    raw = torch.zeros((V, d), dtype=torch.uint8)
    sc = torch.zeros((V, d // group))
    bi = torch.zeros((V, d // group))
    want = torch.zeros((d, V))
    unit, tiny = Fraction(2) ** (magnitude - 7), Fraction(2) ** (magnitude - 40)
    for i in range(V):
        s, q = ties[i // 2]
        sign = 1 if i % 2 == 0 else -1
        raw[i], sc[i], bi[i] = q, float(s * unit), float(sign * tiny)
        want[:, i] = bf16_once(s * q * unit + sign * tiny)
    packed = raw[:, 0::2] | (raw[:, 1::2] << 4) if bits == 4 else raw
    flat = torch.zeros(packed.numel() + 16, dtype=torch.uint8, device=dev())
    wq = flat[offset:offset + packed.numel()].view(packed.shape)
    wq.copy_(packed)
    h = torch.eye(d, device=dev()).bfloat16()
    got = run(h, (wq, sc.to(dev()).bfloat16(), bi.to(dev()).bfloat16()), bits, group)
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("pitch", [65, 67, 70, 1000])
def test_the_pitch_of_a_single_row_does_not_matter(pitch):
    g = torch.Generator("cuda").manual_seed(pitch)
    wq = torch.randint(0, 256, (300, 32), generator=g, device=dev(), dtype=torch.uint8)
    sc = torch.ones((300, 2), device=dev()).bfloat16()
    h = torch.randn((1, 64), generator=g, device=dev()).bfloat16()
    wide = torch.zeros((1, pitch), device=dev()).bfloat16()
    wide[:, :64] = h
    assert wide[:, :64].stride(0) == pitch
    assert torch.equal(run(wide[:, :64], (wq, sc, sc), 4, 32), run(h, (wq, sc, sc), 4, 32))
