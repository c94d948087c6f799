"""Refusals of the C ABI for updates in place: an output at an input's address needs that input's type and dense
rows (one row: any stride).  No call here reaches a launch: accepted ones end at the missing workspace."""
import pytest

from test_norm_cpu import FAKE, add_bwd, add_fwd, drop, ln_bwd, ln_fwd, lib  # noqa: F401

OTHER = [FAKE * k for k in range(2, 8)]


def test_row_strides(lib):  # noqa: F811
    assert ln_fwd(lib, x=FAKE, y=FAKE, ldx=24) == 1
    assert drop(lib, x=FAKE, y=FAKE, ldx=24) == 1
    a, b, c, e, f, _ = OTHER
    assert add_fwd(lib, x=a, res=b, y=a, z=c, ldx=24) == 1
    assert add_fwd(lib, x=a, res=b, y=b, z=c, ldres=24) == 1
    assert add_fwd(lib, x=a, res=b, y=c, z=a, ldx=24) == 1
    assert ln_bwd(lib, dy=a, x=b, dx=a, lddy=24, ws=None) == 1
    assert ln_bwd(lib, dy=a, x=b, dx=b, ldx=24, ws=None) == 1
    for over, ld in ((a, "lddy"), (b, "lddz"), (c, "ldz")):
        assert add_bwd(lib, dy=a, dz=b, z=c, dres=over, dx=e, ws=None, **{ld: 24}) == 1
        assert add_bwd(lib, dy=a, dz=b, z=c, dres=e, dx=over, ws=None, **{ld: 24}) == 1


def test_types(lib):  # noqa: F811
    """An fp32 stream with bf16 branches: an output takes the place of an input of its own type only."""
    a, b, c, e, f, _ = OTHER
    assert ln_fwd(lib, x=a, y=a, dt=0, od=1) == 1
    assert ln_bwd(lib, dy=a, x=b, dx=a, dt=0, dyt=1, ws=None) == 1
    assert add_fwd(lib, x=a, res=b, y=b, z=c, dt=1, rt=0) == 1
    assert add_fwd(lib, x=a, res=b, y=c, z=a, dt=1, rt=0) == 1
    assert add_bwd(lib, dy=a, dz=b, z=c, dres=a, dx=e, dt=1, rt=0, ws=None) == 1
    assert add_bwd(lib, dy=a, dz=b, z=c, dres=e, dx=c, dt=1, rt=0, ws=None) == 1


@pytest.mark.parametrize("rows,ld", [(4, 16), (1, 24)])
def test_dense_rows_of_the_type_are_accepted(lib, rows, ld):  # noqa: F811
    a, b, c, e, f, _ = OTHER
    for over in (a, b):
        assert ln_bwd(lib, dy=a, x=b, dx=over, lddy=ld, ldx=ld, rows=rows, ws=None) == 4
    assert ln_bwd(lib, dy=a, x=b, dx=b, ldx=ld, dt=0, dyt=1, rows=rows, ws=None) == 4
    for over in (a, b, c):
        assert add_bwd(lib, dy=a, dz=b, z=c, dres=over, dx=e, lddy=ld, lddz=ld, ldz=ld, rows=rows, ws=None) == 4
        assert add_bwd(lib, dy=a, dz=b, z=c, dres=e, dx=over, lddy=ld, lddz=ld, ldz=ld, rows=rows, ws=None) == 4
