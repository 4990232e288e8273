"""YaRN's pair range where it lies far outside the 32 pairs: rope_table and a rotation plan against the
definition, whose whole numbers have no border (CPU only)."""

from fractions import Fraction

import numpy as np
import pytest

import compressed_sparse_attention_kv_gb300 as cskv
from oracle import rope


@pytest.fixture(scope="module", autouse=True)
def built():
    from compressed_sparse_attention_kv_gb300 import build
    build.build()


FAR = [(1.0 + 1e-8, rope.YARN_V4),                                                     # both ends beyond 2^31
       (1.0 + 1e-8, dict(factor=16.0, original=1e-3, beta_fast=32.0, beta_slow=1.0)),     # below -2^31
       (1.0 + 1e-7, rope.YARN_V4),                                                     # one end beyond
       (1.0 + 2.0 ** -52, dict(factor=4.0, original=1e300, beta_fast=1e-3, beta_slow=1e300)),
       (160000.0, dict(factor=16.0, original=1e300, beta_fast=32.0, beta_slow=1.0)),
       (160000.0, rope.YARN_V4)]


@pytest.mark.parametrize("theta,yarn", FAR)
def test_speeds_with_a_range_far_outside(theta, yarn):
    f = rope.inv_freq(theta, yarn=yarn)
    pos = np.array([0, 1, 2, 1000])
    want = rope.table(pos, theta, yarn=yarn)
    # float32 of angles up to 1,000 in double precision, a few of their ulps apart
    assert np.max(np.abs(cskv.rope_table(pos, theta, yarn=yarn).astype(np.float64) - want)) <= 2.0 ** -23
    plan = cskv.RopePlan(theta, yarn=yarn)
    for k in range(32):
        w = plan.struct.speed[k]
        turns = float(Fraction((w[0] << 64) | (w[1] << 32) | w[2], 1 << 96))
        assert abs(turns * 2 * np.pi - f[k]) <= 1e-14 * f[k] + 1e-28


def test_an_endless_original_length_keeps_every_speed():
    """The pairs that turn often enough over it are all of them, whatever the beta."""
    for beta in (1e-3, 32.0, 1e300):
        y = dict(factor=16.0, original=float("inf"), beta_fast=beta, beta_slow=beta)
        assert np.array_equal(cskv.rope_table([5, 77], yarn=y), cskv.rope_table([5, 77]))
