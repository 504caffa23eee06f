"""The attention side's oracle pins must catch plausible mistakes.

Each case plants one mistake in the source of ``oracle/attention_oracle.py`` (in memory, on
the CPU, never in the tree) and runs the pins of ``tests/test_attention_oracle.py``, and
those below, against the result; mistakes that all pins pass are holes in them."""
import importlib.util
import os
import types

import numpy as np
import pytest

from oracle import attention_oracle as AO

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = open(os.path.join(ROOT, "oracle", "attention_oracle.py")).read()

# name -> (text in the oracle, replacement)
MUTATIONS = {
    "e4m3_half_up": ("return np.rint(r / step) * step", "return np.floor(r / step + 0.5) * step"),
    "e4m3_no_subnormals": ("2.0 ** -20))), -6.0)", "2.0 ** -20))), -20.0)"),
    "fp8_other_largest": ("m / np.float32(448.0)", "m / np.float32(240.0)"),
    "fp8_signed_max": ("m = np.abs(row).max()", "m = row.max()"),
    "tiny_rows_kept": ("if float(m) < SMALLEST:", "if float(m) < 0.0:"),
    "nan_rows_kept": ("        if not np.isfinite(row).all():\n            scale[i] = np.nan\n            continue\n", ""),
    "bf16_infinity_kept": ("if np.isfinite(v).all():", "if not np.isnan(v).any():"),
    "bf16_truncated": ("((b + 0x7FFF + ((b >> 16) & 1)) >> 16 << 16)", "(b >> 16 << 16)"),
    "opq_sign": ("np.where(neg[0] != 0, -1.0, 1.0)", "np.where(neg[0] != 0, 1.0, -1.0)"),
    "opq_levels_power": ("(q / 15.0) ** (1.0 / alpha_f32(alpha))", "(q / 15.0) ** alpha_f32(alpha)"),
    "opq_levels_unrounded": ("return bf16_bits_to_f32(f64_to_bf16_bits(g)).astype(np.float64)", "return g"),
    "turn_sign": ("y[t, :, a] = x[t, :, a] * c - x[t, :, b] * s", "y[t, :, a] = x[t, :, a] * c + x[t, :, b] * s"),
    "turn_back_is_forward": ("s = -s if backward else s", "s = s"),
    "one_axis": ("positions[t][axis[i]]", "positions[t][axis[0]]"),
    "pairs_of_layouts": ('(i, i + pairs) if layout == "half"', '(2 * i, 2 * i + 1) if layout == "half"'),
    "frequencies_yarn_swapped": ("f * keep + f / factor * (1 - keep)", "f * (1 - keep) + f / factor * keep"),
    "frequencies_ntk_exponent": ("factor ** (rot / (rot - 2))", "factor ** (rot / (rot + 2))"),
    "amplitude": ("1.0 + 0.1 * math.log(factor)", "1.0 + 0.1 * math.log2(factor)"),
    "mask_transposed": ("if seen[t, j]]", "if seen[j, t]]"),
    "prefix_one_short": ("list(range(length)) + ", "list(range(length - 1)) + "),
    "scale_forgotten": ("s = scale * (k @ q[t, h])", "s = k @ q[t, h]"),
    "lse_without_maximum": ("lse[t, h] = m + math.log(l)", "lse[t, h] = math.log(l)"),
    "weights_not_normalised": ("out[t, h] = (e / l) @ v", "out[t, h] = e @ v"),
}


def _mutated(old, new):
    assert SOURCE.count(old) >= 1, f"not in the oracle: {old}"
    m = types.ModuleType("oracle.mutated")
    m.__package__ = "oracle"
    exec(compile(SOURCE.replace(old, new), "attention_oracle (mutated)", "exec"), m.__dict__)
    return m


def _pins(oracle):
    """Every pin, as callables on one oracle."""
    path = os.path.join(ROOT, "tests", "test_attention_oracle.py")
    spec = importlib.util.spec_from_file_location("pins_of_the_attention_oracle", path)
    pins = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(pins)
    pins.AO = oracle
    yield pins.test_e4m3_rounding_equals_torch_for_every_neighbourhood
    yield pins.test_cache_rows_by_hand
    yield pins.test_rotary_oracle_is_a_turn
    yield pins.test_attention_oracle_equals_torch
    for kw in (dict(scaling="ntk", factor=4.0), dict(scaling="yarn", factor=16.0, original_len=4096.0)):
        yield lambda kw=kw: pins.test_frequencies(128, kw)
    yield lambda: _levels_by_hand(oracle)
    yield lambda: _signs_and_rounding_by_hand(oracle)


def _levels_by_hand(oracle):
    """alpha 1/2: level q is (q / 15)^2; 1/9 and 16/225 as their nearest bfloat16."""
    g = oracle.opq_levels(0.5)
    assert list(g[[0, 15]]) == [0.0, 1.0]
    assert g[5] == 228 / 2048 and g[4] == 146 / 2048          # 227.6 and 145.6 of 2^-11


def _signs_and_rounding_by_hand(oracle):
    row = np.zeros((1, 64), np.float32)
    row[0, :4] = [-2.0, 1.0, -1.0, 1.0 + 2.0 ** -8 + 2.0 ** -20]
    codes, scale = oracle.cache_rows(row, "opq4", alpha=1.0)   # 15 |x| / 2: 15, 7.5 up to 8, 8
    assert scale[0] == 2.0 and codes[0, 0] == -1.0 and codes[0, 1] == -codes[0, 2] == 137 / 256   # 136.5 of 2^-8
    codes, _ = oracle.cache_rows(row, "bf16")
    assert codes[0, 3] == 1.0 + 2.0 ** -7                      # just past the tie
    codes, scale = oracle.cache_rows(row, "fp8")
    assert scale[0] == np.float32(2.0) / np.float32(448.0) and codes[0, 0] == -448.0
    row[0, 5] = 3.4e38                                         # past the largest bfloat16
    codes, scale = oracle.cache_rows(row, "bf16")
    assert np.isnan(scale[0]) and not codes.any()


def test_the_pins_hold_for_the_oracle():
    for pin in _pins(AO):
        pin()


@pytest.mark.parametrize("name", MUTATIONS)
def test_a_planted_mistake_fails_a_pin(name):
    oracle, failed = _mutated(*MUTATIONS[name]), 0
    for pin in _pins(oracle):
        try:
            pin()
        except (AssertionError, ValueError, FloatingPointError):
            failed += 1
    assert failed, f"{name}: every pin passes"
