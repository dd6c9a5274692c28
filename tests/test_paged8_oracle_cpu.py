"""Pins of the 8-bit cache's oracle, and planted mistakes that they must catch (no GPU needed)."""
import numpy as np
import pytest

from oracle import paged8

torch = pytest.importorskip("torch")


def _check_codes():
    assert paged8.VALUES[0x38] == 1.0 and paged8.VALUES[0x77] == 240.0 and paged8.VALUES[0x7E] == 448.0
    assert paged8.VALUES[1] == 2.0 ** -9 and np.isnan(paged8.VALUES[0x7F]) and paged8.VALUES[0xB8] == -1.0
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(every, paged8.VALUES, equal_nan=True)
    x = np.concatenate([np.random.default_rng(0).standard_normal(4000) * 60, np.linspace(-0.05, 0.05, 4001), [np.nan, 0.0, -0.0]])
    x = np.clip(x, -240, 240)
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(paged8.encode(np.float64(np.float32(x))), want)
    # ties: 17 lies between 16 and 18, 19 between 18 and 20
    assert paged8.VALUES[paged8.encode([17.0, 19.0])].tolist() == [16.0, 20.0]


def _check_scales():
    for dtype in ("bf16", "fp16"):
        for top, e in ((1.0, -7), (255.9, 0), (256.0, 1), (0.99, -8)):
            assert paged8.exponent(np.array([-top, 0.1, np.nan, np.inf]), dtype) == e
        assert paged8.exponent(np.zeros(3), dtype) == paged8.LOW[dtype]
        assert paged8.exponent(np.array([1e38]), dtype) == {"bf16": 119, "fp16": 8}[dtype]
    tdt = {"bf16": torch.bfloat16, "fp16": torch.float16}
    for dtype in ("bf16", "fp16"):  # what any code stands for at the ends of the range is a number of the type
        for e in (paged8.LOW[dtype], 0, paged8.HIGH[dtype]):
            # codes reach 240, or 256 where it has room above
            v = paged8.VALUES[:0x79 if e < paged8.HIGH[dtype] else 0x78] * 2.0 ** e
            assert np.array_equal(torch.from_numpy(v).to(tdt[dtype]).double().numpy(), v)


def _check_append():
    rng = np.random.default_rng(1)
    codes = paged8.quantise(rng.standard_normal((4, 16, 2, 8)), -6, "bf16")
    scales = np.full((4, 2, 2), 121, dtype=np.uint8)
    x = rng.standard_normal((7, 2, 8)) * 40
    table = np.array([[2, 0], [3, 1]])
    got, s = paged8.append8(codes, scales, x, [0, 5, 7], table, [15, 17], "bf16")
    v, old = paged8.values(got, s), paged8.values(codes, scales)
    # sequence 0: entries 10 .. 14 of page 2 behind two older ones of their block;
    # sequence 1: entry 15 of page 3 and entry 0 of page 1
    for n, (page, slot) in enumerate([(2, 10), (2, 11), (2, 12), (2, 13), (2, 14), (3, 15), (1, 0)]):
        assert (np.abs(v[page, slot] - x[n]) <= np.abs(x[n]) / 16 + 2.0 ** -9).all()
    assert (np.abs(v[2, 8:10] - old[2, 8:10]) <= np.abs(old[2, 8:10]) / 16 + 2.0 ** -9).all()
    assert (np.abs(v[3, 8:15] - old[3, 8:15]) <= np.abs(old[3, 8:15]) / 16 + 2.0 ** -9).all()
    keep = np.ones(codes.shape[:2], dtype=bool)
    keep[2, 8:15] = keep[3, 8:] = keep[1, 0] = False
    assert (got[keep] == codes[keep]).all() and (s[2, 1] >= 121).all() and (s[0] == 121).all() and (s[2, 0] == 121).all()
    # the smallest scale that holds the block, no larger
    top = np.abs(v[1, 0]).max(axis=-1)
    assert ((top >= 2.0 ** (s[1, 0].astype(int) - 127) * 128 * 15 / 16) & (top <= 2.0 ** (s[1, 0].astype(int) - 127) * 256)).all()
    back = paged8.read8(got, s, [0, 3, 4], table, [9, 15])
    assert np.array_equal(back, np.stack([v[2, 9], v[2, 10], v[2, 11], v[3, 15]]))


def _check_norm():
    x = np.random.default_rng(2).standard_normal((3, 4, 64)) * 7
    y = paged8.norm(x, np.full(64, 2.0), 0.0)
    assert np.allclose((y * y).mean(-1), 4.0) and np.allclose(y / x, (y / x)[..., :1])
    assert np.allclose(paged8.norm(np.zeros(8), np.ones(8), 1e-6), 0)
    assert np.allclose(paged8.norm(np.ones(8), np.ones(8), 3.0), 0.5)


CHECKS = [_check_codes, _check_scales, _check_append, _check_norm]


@pytest.mark.parametrize("check", CHECKS)
def test_oracle_pins(check):
    check()


_ENCODE, _EXPONENT, _BLOCK, _NORM = paged8.encode, paged8.exponent, paged8.append_block, paged8.norm


@pytest.mark.parametrize("name,wrong,check", [
    ("encode", lambda x: _ENCODE(np.asarray(x) * (1 + 2.0 ** -6)), _check_codes),                       # not the nearest
    ("encode", lambda x: np.where(np.isnan(x), 0, _ENCODE(x)).astype(np.uint8), _check_codes),          # NaN lost
    ("exponent", lambda x, d: _EXPONENT(x, d) + 1, _check_scales),                                      # a bit wasted
    ("exponent", lambda x, d: _EXPONENT(np.nan_to_num(x, nan=0, posinf=1e9), d), _check_scales),        # infinities count
    ("append_block", lambda c, s, n, b, d: _BLOCK(c, s, n, 0, d), _check_append),                       # over the older ones
    ("append_block", lambda c, s, n, b, d: (_BLOCK(c, s, n, b, d)[0], int(s)), _check_append),          # the scale not written
    ("norm", lambda x, w, e: _NORM(x, w, e) * (1 if w is None else w), _check_norm),                    # weighted twice
    ("norm", lambda x, w, e: _NORM(x, w, 0.0), _check_norm),                                            # eps forgotten
])
def test_planted_mistakes_fail_a_pin(monkeypatch, name, wrong, check):
    monkeypatch.setattr(paged8, name, wrong)
    with pytest.raises((AssertionError, IndexError, ValueError)):
        with np.errstate(all="ignore"):
            check()
