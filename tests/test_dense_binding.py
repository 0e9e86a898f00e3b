"""Arguments of the dense attentions that the binding itself has to refuse,
checked without a GPU."""

import pytest
import torch

from wavelet_guided_sparse_gb300 import binding as bd


@pytest.mark.parametrize("kw", [dict(scale=0.0), dict(scale=1e-46), dict(scale=-1e-46),
                                dict(softcap=1e-46), dict(softcap=-1e-46)])
def test_values_that_fp32_rounds_to_the_defaults_are_refused(kw):
    # 0 stands for 1/sqrt(head_dim) and for no cap: a number that becomes 0 on its way
    # must not be taken for it.
    call = dict(causal=True, prefix=None, softcap=0.0, slopes=None, scale=None, n_seqs=1, q_heads=1,
                device=torch.device("cpu"))
    with pytest.raises(ValueError):
        bd._attn_opts(**{**call, **kw})


def test_ordinary_options_are_taken():
    for scale, softcap in ((None, 0.0), (1e-30, 0.0), (0.5, 30), (1.0, 1e-30)):
        o = bd._attn_opts(True, None, softcap, None, scale, 1, 1, torch.device("cpu"))
        assert (o.scale == 0.0) == (scale is None) and (o.softcap == 0.0) == (softcap == 0.0)
