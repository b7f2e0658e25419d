"""What the backward pass of the gated layer asks for as scratch (found on the host, on a machine without a GPU)."""
import ctypes

import pytest

from test_layers_abi import FAR, L, gated_back  # noqa: F401


def need(L, **a):  # noqa: F811
    n = ctypes.c_size_t()
    assert L.lm_gated_linear_backward_workspace_size(gated_back(**a), ctypes.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("rows", [5, 1000, 12000])
@pytest.mark.parametrize("biases", [False, True])
def test_space_for_sums_over_rows_only_where_they_are_wanted(L, rows, biases):  # noqa: F811
    k, n = 1024, 4096
    a = dict(rows=rows, k=k, n=n, xr=k, gr=k, ur=k, orow=n, grow=n)
    if biases:
        a |= dict(bg=20 * FAR, bu=21 * FAR)
    none, one, both = need(L, **a), need(L, dbg=22 * FAR, **a), need(L, dbg=22 * FAR, dbu=23 * FAR, **a)
    assert none <= 512 + 4 * rows * n  # the projections' gradients
    assert one == both >= none + 8 * n
    # The call asks for as much.
    assert L.lm_gated_linear_backward(gated_back(**a), 30 * FAR, none - 1, None) == 7
    assert L.lm_gated_linear_backward(gated_back(dbu=23 * FAR, **a), 30 * FAR, one - 1, None) == 7
