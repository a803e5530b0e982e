"""The gated scan's launch rules and forms that other sizes do not reach: more pairs of sequence and
channel block than clusters of two hold, one CTA for a sequence of several tiles, and 8 tokens a
thread (one bf16 sequence of 1024 tokens or more) on gates at their ends."""
import pytest
import torch

from kimi_delta_attention_17_gb300 import build
from tests.test_gpu_gated_scan import TYPES, check, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()


# At 152 SMs. bf16: 64 channels a block, 4 CTAs per SM forward and 3 backward; mixed: 32 channels, 3 and 2; fp32: 32
# channels, 4 and 3.
@pytest.mark.parametrize("types,B,T,D", [
    ("bf16", 40, 301, 640),    # 400 pairs: over the 304 (228) clusters of two, 4 CTAs each
    ("bf16", 70, 150, 1280),   # 1400 pairs: one CTA each, three tiles
    ("mixed", 30, 530, 320),   # 300 pairs: over 228 (152), 4 CTAs each
    ("mixed", 72, 300, 512),   # 1152 pairs: one CTA each, three tiles
    ("f32", 40, 290, 320),     # 400 pairs: over 304 (228)
    ("f32", 90, 150, 512)])    # 1440 pairs: one CTA each
def test_more_pairs_than_clusters(types, B, T, D):
    check(make(B, T, D, types, "logsigmoid", seed=B), "logsigmoid", "complement")


@pytest.mark.parametrize("types", list(TYPES))
def test_one_cta_for_uneven_packed_sequences(types):
    """One sequence of many means among short ones, empty ones beside it."""
    cu = [0, 3, 3, 1400] + [1400 + 9 * i for i in range(1, 60)]
    check(make(1, cu[-1], 264, types, "log", seed=1, N=len(cu) - 1), "log", "norm", cu=cu)


@pytest.mark.parametrize("write", ["plain", "complement", "norm"])
def test_long_bf16_chain_with_extreme_log_gates(write):
    v = make(1, 2600, 72, "bf16")
    lowest = torch.finfo(torch.bfloat16).min
    v["g"][0, ::97] = -float("inf")
    v["g"][0, 3::211] = lowest
    v["g"][0, 500:1400] = 0.0
    v["g"][0, 1500:, :4] = -1e-6
    v["g"][0, 420, :] = -100.0
    check(v, "log", write)


@pytest.mark.parametrize("gate", ["logsigmoid", "bounded"])
@pytest.mark.parametrize("write", ["plain", "complement", "norm"])
def test_long_bf16_chain_with_extreme_logits(gate, write):
    v = make(1, 1500, 72, "bf16", gate)
    for i, z in enumerate((float("inf"), -float("inf"), 88.0, -88.0, 20.0, -20.0, 3e38, -3e38, 0.0)):
        v["g"][0, 10 + i::137] = z
    check(v, gate, write)
