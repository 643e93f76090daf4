"""CPU check of the smoke run's look at new tokens' queries and latent records: it
takes what the definition gives and nothing else."""
import pytest
import torch

import __graft_entry__ as entry
from tests import latent_reference as ref

FREQ = [10000.0 ** (-i / 32) for i in range(32)]


def make():
    g = torch.Generator().manual_seed(1)
    q = torch.randn((40, 3, 192), generator=g).to(torch.bfloat16)
    kv = torch.randn((40, 576), generator=g).to(torch.bfloat16)
    pos = torch.arange(40, dtype=torch.int32) * 7

    def outputs(q, kv, pos):
        q_out = q.clone()
        q_out[..., 128:] = ref.turned(q[..., 128:], pos, FREQ, 1.0, False)[0].to(torch.bfloat16)
        new = torch.cat((ref.normed(kv[:, :512], None, 1e-6),
                         ref.turned(kv[:, None, 512:], pos, FREQ, 1.0, False)[0][:, 0]), 1).to(torch.bfloat16)
        return q_out, ref.values(ref.pack(new, 0), 0).to(torch.bfloat16)
    return q, kv, pos, outputs


def test_the_definition_passes():
    q, kv, pos, outputs = make()
    q_out, rec = outputs(q, kv, pos)
    entry._check_latent_records(q, q_out, kv, rec, pos, FREQ)


@pytest.mark.parametrize("mistake", ["queries not turned", "positions off by one", "records of zeros", "no norm",
                                     "record not turned", "a token's record elsewhere", "one code wrong",
                                     "an untouched part touched"])
def test_mistakes_are_seen(mistake):
    q, kv, pos, outputs = make()
    q_out, rec = outputs(q, kv, pos)
    if mistake == "queries not turned":
        q_out = q.clone()
    elif mistake == "positions off by one":
        q_out, rec = outputs(q, kv, pos + 1)
    elif mistake == "records of zeros":
        rec = torch.zeros_like(rec)
    elif mistake == "no norm":
        rec = outputs(q, torch.cat((kv[:, :512] * 2, kv[:, 512:]), 1), pos)[1]
        rec[:, :512] *= 2
    elif mistake == "record not turned":
        rec[:, 512:] = kv[:, 512:]
    elif mistake == "a token's record elsewhere":
        rec = rec.roll(1, 0)
    elif mistake == "one code wrong":
        at = kv[5, :16].abs().argmax()
        rec[5, at] = 0
    else:
        q_out[3, 1, 100] += 1
    with pytest.raises(AssertionError):
        entry._check_latent_records(q, q_out, kv, rec, pos, FREQ)
