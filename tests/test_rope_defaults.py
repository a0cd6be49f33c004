"""What make_rope fills in for each scaling, and YaRN with its customary parameters on the GPU."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import decode_attention_13_b200 as gtq  # noqa: E402


@pytest.mark.parametrize("factor", [1.0, 4.0, 40.0])
def test_yarn_is_32_turns_and_a_magnitude(factor):
    c = gtq.make_rope(128, 1e6, scaling=gtq.ROPE_YARN, factor=factor, original_context=32768)
    assert (c.low_freq, c.high_freq) == (1.0, 32.0)
    assert c.magnitude == 0.1 * math.log(factor) + 1.0


def test_the_others_keep_theirs():
    for scaling in (gtq.ROPE_PLAIN, gtq.ROPE_LINEAR, gtq.ROPE_LLAMA3):
        c = gtq.make_rope(128, 1e6, scaling=scaling, factor=8.0, original_context=8192)
        assert (c.low_freq, c.high_freq, c.magnitude) == (1.0, 4.0, 1.0)


def test_what_is_given_stands():
    c = gtq.make_rope(128, 1e6, scaling=gtq.ROPE_YARN, factor=4.0, original_context=32768, low_freq=2.0, high_freq=16.0,
                      magnitude=1.0)
    assert (c.low_freq, c.high_freq, c.magnitude) == (2.0, 16.0, 1.0)


@pytest.mark.parametrize("factor", [0.0, -1.0])
def test_a_factor_that_the_library_refuses_gets_there(factor):
    assert gtq.make_rope(128, 1e6, scaling=gtq.ROPE_YARN, factor=factor, original_context=32768).factor == factor


@pytest.mark.gpu
@pytest.mark.parametrize("pairing", [gtq.PAIRING_HALF, gtq.PAIRING_INTERLEAVED])
@pytest.mark.parametrize("backward", [False, True])
def test_yarn_with_its_customary_parameters(pairing, backward):
    from tests.test_gpu_rope import check, frequencies, reference

    d, theta, factor, context = 128, 1e6, 4.0, 32768.0
    cfg = gtq.make_rope(d, theta, rope_pairing=pairing, dtype=gtq.DTYPE_FP32, scaling=gtq.ROPE_YARN, factor=factor,
                        original_context=context, backward=backward)
    x = torch.randn((2, 3, 21, d), generator=torch.Generator().manual_seed(5)).cuda()
    pos = np.random.default_rng(6).integers(0, 131072, (2, 21))
    y = torch.empty_like(x)
    gtq.gtq_rope(cfg, x, y, positions=torch.from_numpy(pos).cuda())
    freq = frequencies(d, theta, gtq.ROPE_YARN, factor, context, 1.0, 32.0)
    ref, size = reference(x.cpu().numpy(), pos, freq, d, pairing == gtq.PAIRING_HALF, 0.1 * math.log(factor) + 1.0, backward)
    check(y, ref, size, torch.float32)
