"""config.json's rope_scaling blocks in the head norm and rotation's
configuration: what a block asks for is applied or refused, never dropped."""

import math

import pytest

from llama_decoder_layer_gb300 import binding as lb

YARN = {"rope_type": "yarn", "factor": 4.0, "original_max_position_embeddings": 32768}
LLAMA3 = {"rope_type": "llama3", "factor": 8.0, "low_freq_factor": 1.0, "high_freq_factor": 4.0,
          "original_max_position_embeddings": 8192}


def config(block, **kw):
    return lb.QkNormRopeConfig(8, 2, 64, rope_scaling=block, **kw).c()


@pytest.mark.parametrize("block", [
    {**YARN, "mscale": 1.0}, {**YARN, "mscale": 0.707, "mscale_all_dim": 0.707}, {**YARN, "mscale_all_dim": 1.0},
    {**YARN, "truncate": False}, {**LLAMA3, "mscale": 1.0}, {"rope_type": "default", "mrope_section": [16, 24, 24]},
    {"rope_type": "linear", "factor": 2.0, "long_factor": [1.0]}, {**YARN, "rope_theta": 1e6},
    {"rope_type": "linear"}, {"type": "linear", "factor": None}, {k: v for k, v in YARN.items() if k != "factor"},
    {k: v for k, v in LLAMA3.items() if k != "factor"}, {"rope_type": "dynamic", "factor": 2.0}])
def test_a_block_that_asks_for_more_is_refused(block):
    with pytest.raises(lb.LlamaError):
        config(block)


def test_what_a_block_says_is_taken():
    c = config(YARN)
    assert (c.rope_scaling, c.rs_factor, c.rs_low_freq_factor, c.rs_high_freq_factor, c.rs_original_max_pos) == \
        (3, 4.0, 1.0, 32.0, 32768)
    assert abs(c.rs_attention_factor - (0.1 * math.log(4.0) + 1.0)) < 1e-6
    # keys that are there but say nothing, or what is done anyway
    for extra in ({"mscale": None, "beta_fast": None, "attention_factor": None}, {"truncate": True},
                  {"rope_theta": 10000.0}, {"type": "yarn"}):
        d = config({**YARN, **extra})
        assert bytes(d) == bytes(c), extra
    d = config({**YARN, "beta_fast": 16, "beta_slow": 2, "attention_factor": 1.25})
    assert (d.rs_low_freq_factor, d.rs_high_freq_factor, d.rs_attention_factor) == (2.0, 16.0, 1.25)
    c = config(LLAMA3)
    assert (c.rope_scaling, c.rs_factor, c.rs_low_freq_factor, c.rs_high_freq_factor, c.rs_original_max_pos) == \
        (1, 8.0, 1.0, 4.0, 8192)
    assert config({"type": "linear", "factor": 2.0}).rs_factor == 2.0
    assert config(None).rope_scaling == config({}).rope_scaling == config({"rope_type": "default"}).rope_scaling == 0
