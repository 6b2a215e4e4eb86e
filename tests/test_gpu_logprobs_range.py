"""ddt_token_logprobs where logits divided by the temperature are large: small temperatures, and
logits with a large common offset.  Differences to the largest logit are exact in fp32 there or
carry one rounding, so the results keep their precision."""
import math

import numpy as np
import pytest
import torch

from tests import _serving as S
from tests.test_gpu_logprobs import BF, F32, _logits, _run
from tree_speculative_decoding_02_gb300 import synth

pytestmark = pytest.mark.gpu


def _check(r, logits, token, T, top_n):
    """The relative error of Z is at most 2 * 2^-22 (a term's exponential and that of its thread's
    reference), 2^-24 a rounding for (100 + V / 4096) additions on a term's way, 4 * 2^-24 |u| for its
    exponent u = (x - m) / T, whose mean over p is at most log V, and 2^-24 for the correction of the
    references.  log p adds 6 roundings of its own size.  The entropy is log Z minus the mean of u:
    its terms carry Z's error times |u| and up to 16 log2 for the way over a thread's reference, in the
    numerator and in Z."""
    V, u24 = logits.shape[2], S.U
    lp, en, ids, tl = S.logprobs_ref(S.f64(logits), None, token.numpy(), top_n, float(np.float32(T)))
    ez = 2.0 ** -21 + (101 + V / 4096 + 4 * math.log(V)) * u24

    def near(got, want):
        got = got.double().numpy()
        same = got == want
        with np.errstate(invalid="ignore"):
            err = np.abs(got - want)
            tol = ez + 6 * u24 * np.abs(want)
        assert (same | (err <= tol)).all(), np.where(same, 0, err / tol).max()
    assert (r["status"] == 0).all()
    near(r["logprob"], lp)
    near(r["top_logprob"], tl)
    np.testing.assert_array_equal(r["top_token"].numpy(), ids)
    err = np.abs(r["entropy"].double().numpy() - en)
    tol = ez * (1 + 2 * (en + 16 * math.log(2))) + 6 * u24 * en
    assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [1003, 40001])
@pytest.mark.parametrize("T", [0.02, 1e-3, 1e-5, 1e-7, 1e-20, 1e-37, 30.0])
def test_small_temperatures(dtype, V, T):
    logits = _logits(52, 1, 9, V, dtype)
    top = logits[0, 3:6].max(-1, keepdim=True).values
    logits[0, 3:6, ::7] = top                                   # many tokens share the largest logit
    logits[0, 6] -= 20.0                                        # all negative
    token = logits[0].float().argmax(-1).to(torch.int32)[None]
    token[0, 7:] = 5
    r = _run(logits, token, top_n=8, temperature=T)
    _check(r, logits, token, T, 8)


@pytest.mark.parametrize("offset", [3e3, -3e4, 1e6, -1e7, 2e30])
@pytest.mark.parametrize("V", [4099, 151936])
def test_a_common_offset(offset, V):
    """fp32 logits far from zero, masked entries among them; at 2e30 all that are not masked are equal."""
    g = synth.gen(53, 90)
    logits = (synth.normal((1, 6, V), 3.0, g=g, dtype=F32) + offset)
    logits[0, 1, ::3] = -math.inf
    logits[0, 2, 5:] = torch.finfo(F32).min
    logits[0, 3, :V // 2] = offset - 2e4 if abs(offset) < 1e20 else offset   # the row's start far below its rest
    logits[0, 4, V // 2:] = 0.0 if offset < 0 else offset                    # references that leave the far range
    token = logits[0].argmax(-1).to(torch.int32)[None]
    token[0, 5] = V - 1
    r = _run(logits, token, top_n=4)
    _check(r, logits, token, 1.0, 4)
