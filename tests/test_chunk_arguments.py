"""Arguments of the chunk step that are refused before any device is asked for (no GPU)."""

import pytest

import mla_decode_attention_02_gb300 as mla


@pytest.mark.parametrize("kw", [dict(tokens=(1 << 32) + 20), dict(tokens=-(1 << 31) - 1), dict(max_pages_per_seq=(1 << 32) + 2),
                                dict(kv_tokens=(1 << 64) + 128)], ids=["tokens", "negative", "pages", "keys"])
def test_plan_sizes_beyond_their_fields(kw):
    """ctypes keeps a field's low bits alone: 2^32 + 20 tokens would be planned as 20."""
    with pytest.raises(ValueError, match="must be below"):
        mla.chunk_plan(None, None, **{**dict(tokens=20, max_pages_per_seq=2, kv_tokens=128), **kw})


def test_scratch_of_heads_beyond_their_field():
    p = mla.ChunkPlan(1, 20, 2, 128, None)
    with pytest.raises(ValueError, match="must be below"):
        mla.chunk_scratch_size(p, (1 << 32) + 1)


def test_original_length_beyond_its_field():
    with pytest.raises(ValueError, match="must be below"):
        mla.rope_table_scaled(factor=4.0, original_positions=(1 << 32) + 4096)
