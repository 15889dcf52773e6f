"""Calls of the latent operators that the binding refuses itself, without a GPU."""
import pytest
import torch

import paged_varlen_attention_attn_gb300 as pa

BF, I32 = torch.bfloat16, torch.int32


def absorbed(**kw):
    a = dict(scale=1.0, latent_size=128, block_size=16, max_query_len=1)
    a.update(kw)
    return pa.latent_forward(torch.zeros(3, 2, 160, dtype=BF), torch.zeros(4, 16, 160, dtype=BF),
                             torch.zeros(2, 2, dtype=I32), torch.zeros(2, dtype=I32),
                             torch.zeros(3, dtype=I32), **a)


def expanded(starts=3, **kw):
    a = dict(scale=1.0)
    a.update(kw)
    return pa.latent_expanded_forward(
        torch.zeros(3, 2, 96, dtype=BF), torch.zeros(5, 2, 64, dtype=BF), torch.zeros(5, 32, dtype=BF),
        torch.zeros(5, 2, 64, dtype=BF), torch.zeros(starts, dtype=I32), torch.zeros(starts, dtype=I32),
        **a)


@pytest.mark.parametrize("latent_size", [0, -128, 160, 256])
def test_a_latent_size_without_a_part_of_the_row(latent_size):
    with pytest.raises(pa.PattnError):
        absorbed(latent_size=latent_size)


@pytest.mark.parametrize("call,name", [(absorbed, "max_query_len"), (absorbed, "max_seq_len"),
                                       (expanded, "max_query_len"), (expanded, "max_key_len")])
def test_lengths_that_no_batch_has(call, name):
    with pytest.raises(pa.PattnError):
        call(**{name: -1})


def test_starts_without_a_number():
    with pytest.raises(ValueError):
        expanded(starts=0)
    assert expanded(starts=1).shape == (3, 2, 64)  # no request: nothing to do
