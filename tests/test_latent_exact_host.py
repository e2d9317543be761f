"""What the cases of tests/latent_exact.py tell apart: P as the sum of two 16-bit values is within their tolerance, P as one
value, or with the second's sign or place wrong, is not (a model in 64 bits, on the CPU)."""

import pytest

import latent_exact as X

FORMS = {"two": lambda hi, lo: hi + lo, "one": lambda hi, lo: hi, "subtracted": lambda hi, lo: hi - lo,
         "shifted": lambda hi, lo: hi + lo.roll(1, dims=1)}


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("H, r, lens, new", X.CASES)
def test_the_second_value_shows(H, r, lens, new, dt):
    c = X.chunk(H, r, lens, new, dt)
    want, tol = X.attention(c, 2)
    off = {n: ((X.modelled(c, f) - want).abs() / tol.clamp(min=1e-30)).max() for n, f in FORMS.items()}
    assert off["two"] <= 1
    for n in ("one", "subtracted", "shifted"):
        assert off[n] > 2, n
    loose = X.attention(c, 1)[1]
    assert bool(((X.modelled(c, FORMS["one"]) - want).abs() <= loose).all())
