"""Arguments of the q4_G calls and of moe_groups that the binding refuses by itself (no GPU)."""
import types

import numpy as np
import pytest

mmq = pytest.importorskip("q4_q8_int8_amd")
torch = pytest.importorskip("torch")

from tests import q4g_util as qu


def test_a_group_that_the_format_cannot_hold():
    """One scale per row takes any group of K or more, up to the format's 2^31 - 1; what is above is
    refused and not cut to its low 32 bits."""
    for group in (2 ** 31 - 1, np.int64(2 ** 31 - 1), 1 << 20):
        f = mmq.q4G_format(group, torch.float16, False)
        assert f.group == group
        # a record of 16 rows x 128 values with one scale a row, as for a group of K
        assert mmq.mmq_q4G_repacked_bytes(16, 96, f) == 1024 + 32
    for group in (2 ** 31, 2 ** 32 + 64, 2 ** 63 - 1, 2 ** 64 + 32, -2 ** 32 + 32):
        with pytest.raises(mmq.MMQArgumentError):
            mmq.q4G_format(group, torch.float16, False)


def test_other_kinds_of_arguments_are_refused():
    f32 = types.SimpleNamespace(dtype=torch.float32)
    for call in (lambda: mmq.moe_groups(None, 3, 8, 2),
                 lambda: mmq.moe_groups(np.zeros(28, np.int32), 3, 8, 2),
                 lambda: mmq.mmq_q4G_repacked_bytes(16, 96, None),
                 lambda: mmq.mmq_q4G_repacked_bytes(16, 96, (32, 1, 0, 0)),
                 lambda: mmq.mmq_q4G(1, 16, 96, f32, None, None, f32),
                 lambda: mmq.repack_q4_G(None, None, None, 16, 96, None, None)):
        with pytest.raises(mmq.MMQArgumentError):
            call()


def test_the_bound_of_one_value_sees_a_lost_piece():
    """The third of x's pieces, 8 bits each, is beyond the bound wherever v is not z; so is either of its
    neighbours' in its place."""
    x = qu.full_mantissas(4000, 1)
    top = (x.view(np.uint32) & 0xFFFF0000).view(np.float32)
    mid = ((x - top).view(np.uint32) & 0xFFFF0000).view(np.float32)
    low = (x - top) - mid
    assert np.array_equal(top.astype(np.float64) + mid + low, x) and np.all(low != 0)
    v, z = np.meshgrid(np.arange(16.0), np.arange(16.0))
    v, z = v[v != z][:, None], z[v != z][:, None]
    exact = x.astype(np.float64) * (v - z)
    allowed = qu.one_value_bound(x, v, z)
    for wrong in (top.astype(np.float64) + mid, top.astype(np.float64) + mid + np.roll(low, 1),
                  top.astype(np.float64) + 2.0 * mid, 1.0 * top):
        off = np.abs(wrong * (v - z) - exact) > allowed
        assert off[:, np.abs(wrong - x) >= np.abs(low) / 2].all()
    assert np.all(np.abs((exact.astype(np.float32)).astype(np.float64) - exact) <= allowed)
