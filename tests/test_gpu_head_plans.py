"""The head's products under every plan: whole tiles, equal runs of a tile's stages,
runs with rests that are laid end to end, and all stages end to end, by lone CTAs and
by pairs. The shapes below come to the plans that the other tests' shapes do not."""
import pytest

import test_gpu_head as H

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K,N,act,bias,residual", [
    (5, 2196, 6827, "silu", 1, 1),     # lone CTAs, runs with rests
    (7, 2200, 6816, "gelu", 1, 1),     # the same, rows of 16-byte vectors
    (814, 1493, 5042, "silu", 1, 0),   # pairs, all stages end to end
    (816, 1496, 5048, "none", 0, 1),
])
def test_forward(M, K, N, act, bias, residual):
    H.test_forward(M, K, N, act, bias, residual)


@pytest.mark.parametrize("M,K,N,act", [
    (5, 19713, 825, "silu"),      # dx by lone CTAs, end to end
    (6, 6437, 1803, "none"),      # dx by lone CTAs, runs with rests
    (287, 10407, 1679, "gelu"),   # dx by pairs, end to end
    (781, 19659, 9, "none"),      # dW by lone CTAs, end to end
    (1943, 6438, 8, "silu"),      # dW by lone CTAs, runs with rests
    (1365, 19568, 196, "none"),   # dW by pairs, end to end
    (1156, 261, 68, "gelu"),      # dW by pairs, runs
    (2198, 130, 6543, "none"),    # dW by pairs, runs with rests
])
def test_backward(M, K, N, act):
    H.test_backward(M, K, N, act)
