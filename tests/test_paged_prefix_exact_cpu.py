"""The criterion that the prefix kernel is held to in test_paged_prefix_exact_gpu.py: its arithmetic written out passes, and
what could go wrong in it does not."""
import numpy as np
import pytest

from oracle import codec, paged as op
from prefix_cases import CLIMBS, FAULTS, MOST, attention, climbing, rescaled


def _refused(got, ref):
    return op.not_nearest(got.astype(np.float16).astype(np.float64), ref) > MOST


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("name", CLIMBS)
def test_faults_of_rescaling_are_refused(name, d):
    climb = CLIMBS[name]
    moves = sum(c >= 13 for c in climb) + (name == "of 5 and 8")
    for seed in range(3):
        q, k, v = climbing(climb, d, 6, seed)
        q, k, v = q.astype(np.float64), op.restore(*k), op.restore(*v)
        ref = attention(q, k, v, 1 / np.sqrt(d))
        assert np.median(np.abs(ref)) > 2.0 ** -8
        assert not _refused(rescaled(q, k, v, 1 / np.sqrt(d)), ref)
        for fault in FAULTS:
            if "rescale" in fault and not moves:
                continue
            if fault == "no remainders of weights" and "40" in name:
                continue                                     # the tiles that count have few weights that are no fp16
            assert _refused(rescaled(q, k, v, 1 / np.sqrt(d), fault), ref), fault


@pytest.mark.parametrize("d", [64, 128])
def test_rounded_operands_are_refused(d):
    """Keys, values or weights rounded to fp16 once, against values of any kind."""
    for seed in range(3):
        rng = np.random.default_rng(seed)
        k, v = (codec.quantize_g64((rng.normal(size=(700, d)) * (0.5 + rng.random(d))).astype(np.float16)) for _ in range(2))
        q = (1.3 * rng.normal(size=(6, d))).astype(np.float16).astype(np.float64)
        k, v = op.restore(*k), op.restore(*v)
        half = lambda x: x.astype(np.float16).astype(np.float64)
        scale = 1 / np.sqrt(d)
        ref = attention(q, k, v, scale)
        assert not _refused(rescaled(q, k, v, scale), ref)
        assert _refused(rescaled(q, half(k), v, scale), ref)
        assert _refused(rescaled(q, k, v, scale, "no remainders of weights"), ref)
        assert _refused(rescaled(q, k, v, scale, "no remainders of values"), ref)
