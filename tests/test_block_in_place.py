"""CPU: the gated block's dz may take z's place, row for row."""
import pytest

from quantized_moe_gb300 import build as b
from quantized_moe_gb300 import ds4moe as api

b.build()
Z, P = 1 << 20, 16


def grad(**kw):
    api.ds4moe_grouped_glu_grad(**{**dict(dh=P, x=P, w=P, offsets=P, z=Z, dz=Z, dx=P, dw=P, rows=4, n=8, k=8, n_groups=2), **kw})


@pytest.mark.parametrize("kw", [dict(ldz=24), dict(lddz=24), dict(ldz=24, lddz=32)])
def test_rows_at_other_distances_are_refused(kw):
    with pytest.raises(api.Ds4MoeError) as ei:
        grad(**kw)
    assert ei.value.code == api.DS4MOE_ERR_INVALID_ARG and "dz is z" in str(ei.value)


@pytest.mark.parametrize("kw", [dict(), dict(ldz=24, lddz=24), dict(ldz=16, lddz=0), dict(rows=1, ldz=24), dict(dz=Z + 64, ldz=24)])
def test_other_calls_are_not(kw):
    with pytest.raises(api.Ds4MoeError) as ei:  # (no device, or no memory at these addresses)
        grad(**kw)
    assert "dz is z" not in str(ei.value)
