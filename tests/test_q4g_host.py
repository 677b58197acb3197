"""Arguments of the q4_G calls and of moe_groups that the binding refuses by itself (no GPU)."""
import types

import numpy as np
import pytest

mmq = pytest.importorskip("q4_q8_int8_amd")
torch = pytest.importorskip("torch")


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
