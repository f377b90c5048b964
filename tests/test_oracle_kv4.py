"""The fp64 oracle of the 4-bit cache against closed forms (CPU)."""
import numpy as np
import pytest

from oracle import kv4


def test_levels_of_an_even_grid_are_exact():
    # 0..15 twice over: s = 1, z = 0, codes = the values
    x = np.tile(np.arange(16.0), 2)
    n, s, z = kv4.quantise_group(x)
    assert s == 1.0 and z == 0.0 and n.tolist() == x.astype(int).tolist()
    # shifted and scaled by powers of two
    n, s, z = kv4.quantise_group(x * 0.25 - 2)
    assert s == 0.25 and z == -2.0 and n.tolist() == x.astype(int).tolist()


def test_ties_go_to_the_even_code():
    x = np.zeros(32)
    x[1] = 15.0
    x[2:17] = np.arange(15) + 0.5
    n, s, _ = kv4.quantise_group(x)
    assert s == 1.0
    assert n[2:17].tolist() == [0, 2, 2, 4, 4, 6, 6, 8, 8, 10, 10, 12, 12, 14, 14]


def test_scale_rounds_to_bf16_and_codes_clamp():
    x = np.zeros(32)
    x[0] = 1.0                                           # 1/15 = 0x3D888889: rounds to bf16 0x3D89
    n, s, _ = kv4.quantise_group(x)
    assert s == float(np.array([0x3D89 << 16], dtype=np.uint32).view(np.float32)[0])
    assert n[0] == 15 and n[1:].max() == 0


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf, 2.0 ** 127])
def test_what_the_format_does_not_hold_is_nan(bad):
    x = np.ones(32)
    x[5] = bad
    n, s, z = kv4.quantise_group(x)
    assert n.max() == 0 and np.isnan(s) and np.isnan(z)


def test_constant_and_tiny_groups():
    n, s, z = kv4.quantise_group(np.full(32, -3.5))
    assert s == 0.0 and z == -3.5 and n.max() == 0
    x = np.zeros(32)
    x[0] = 2.0 ** -98                                    # /15 is below 2^-100
    n, s, z = kv4.quantise_group(x)
    assert s == 0.0 and n.max() == 0


def test_error_is_within_half_a_step():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((20, 128))
    n, s, z = kv4.quantise_rows(x)
    # half a step, and what the scale's rounding (2^-9 of it) leaves at the top code
    assert np.all(np.abs(kv4.values(n, s, z) - x) <= np.repeat(s, 32, -1) * (0.5 + 15 * 2.0 ** -8))


def test_decode_mask_cap_and_bias():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((2, 128)), rng.standard_normal((9, 128)), rng.standard_normal((9, 128))
    pos = np.arange(9)
    v2 = v.copy()
    v2[3] = np.nan                                       # not seen: sinks 0, 1 and the last 4
    out, p = kv4.decode(q, k, v2, 0.1, pos, 8, window=4, n_sink=2)
    assert np.all(p[:, [2, 3, 4]] == 0) and np.allclose(p.sum(1), 1) and np.isfinite(out).all()
    # a huge cap is no cap; a steep bias leaves the nearest key
    a = kv4.decode(q, k, v, 0.1, pos, 8)[0]
    assert np.allclose(kv4.decode(q, k, v, 0.1, pos, 8, softcap=1e6)[0], a, atol=1e-6)
    near = kv4.decode(q, k, v, 0.1, pos, 8, slopes=np.array([1e3, 1e3]))[1]
    assert np.allclose(near[:, 8], 1)


def test_prefill_masks():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((6, 128)), rng.standard_normal((10, 128)), rng.standard_normal((10, 128))
    out, lse = kv4.prefill(q, k, v, 0.1)
    # the last row is a decode step
    assert np.allclose(out[-1], kv4.decode(q[-1:], k, v, 0.1, np.arange(10), 9)[0][0])
    # a prefix of everything: every row sees all keys
    full, _ = kv4.prefill(q, k, v, 0.1, prefix=10)
    assert np.allclose(full[0], kv4.decode(q[:1], k, v, 0.1, np.arange(10), 9)[0][0])
    # a document that starts behind the row: nothing is seen
    none, lse = kv4.prefill(q, k, v, 0.1, doc_start=np.full(6, 10))
    assert np.all(none == 0) and np.all(lse == -np.inf)
    # more queries than keys: the first rows come before the first key
    short, lse = kv4.prefill(q, k[:4], v[:4], 0.1)
    assert np.all(short[:2] == 0) and np.all(lse[:2] == -np.inf) and np.isfinite(lse[2:]).all()
