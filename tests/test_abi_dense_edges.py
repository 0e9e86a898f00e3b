"""Host-side refusals of the dense attentions at the edges of fp32's range (no
launch here)."""

import pytest

from test_abi_dense import SHAPE, lib, opts, pages, paged, prefill  # noqa: F401


@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("kw", [dict(softcap=1e38), dict(softcap=2e37), dict(scale=1e-6, softcap=1e33),
                                dict(scale=1e-38, softcap=2.0)])
def test_caps_that_leave_no_normal_quotient_are_refused(lib, kw, head_dim):  # noqa: F811
    # scale / softcap below the smallest normal float: the scores would lose their bits.
    assert paged(lib, pages(head_dim=head_dim), opts(**kw)) == SHAPE
    assert prefill(lib, opts(**kw), head_dim=head_dim) == SHAPE
