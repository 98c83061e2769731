"""The paged key-value cache operators at their edges, on the GPU against the
fp64 oracle; tolerances are those of tests/test_gpu_kv.py where none is derived
beside the test."""
import pytest

from tests.test_gpu_kv import S, Setup, _check_attend, _fill_and_attend  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("softcap", [50.0, 65.0, 1e3, 1e4, 1e6, 1e30, 3e38])
@pytest.mark.parametrize("dtype,new,d", [("f16", 1, 128), ("bf16", 1, 64), ("f16", 60, 128), ("bf16", 60, 80)])
def test_softcap_far_above_the_scores(S, softcap, dtype, new, d):
    """c(s) keeps the bits of a small s whatever the softcap, in both kernels."""
    s = Setup(S, [300], [new], 4, 4, d, 1, dtype, seed=21)
    _, q, out = _fill_and_attend(S, s, softcap=softcap)
    _check_attend(s, q, out, softcap=softcap)
    s.close()


@pytest.mark.parametrize("new", [1, 60])
@pytest.mark.parametrize("softcap", [2.0, 1e-3, 1e-30, 1e-42])
def test_softcap_below_the_scores(S, new, softcap):
    s = Setup(S, [300], [new], 4, 4, 64, 1, "f16", seed=22)
    _, q, out = _fill_and_attend(S, s, softcap=softcap)
    _check_attend(s, q, out, softcap=softcap)
    s.close()


@pytest.mark.parametrize("new", [1, 60])
def test_softcap_around_large_scores(S, new):
    """Scores from far below softcap to near it (q . k scale of about +-150)."""
    s = Setup(S, [300], [new], 4, 4, 64, 1, "f16", seed=22)
    _, q, out = _fill_and_attend(S, s, softcap=100.0, scale=64 ** -0.5 * 16)
    _check_attend(s, q, out, softcap=100.0, scale=64 ** -0.5 * 16)
    s.close()
