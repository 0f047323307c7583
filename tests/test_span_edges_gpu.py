"""The span attention at its edges: workspaces made for other calls, lost
pages, values that are not finite."""

import pytest
import torch

from rope_frequency_chunk_b200 import fasa as F
from tests import span_util as S

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def _clean_status():
    F.fasa_device_status(clear=True)
    yield
    assert F.fasa_device_status(clear=True) == 0


def test_one_prompt_workspace_for_every_chunk():
    """Sized once for the longest chunk, used for shorter ones and windows."""
    f = S.Filled([3000], 8, 2, BF, 16)
    ws = F.fasa_attend_prompt_workspace(f.cache, 1024, 3000)
    for n_q, window in ((1024, 0), (300, 0), (17, 0), (1, 0), (17, 900), (300, 64)):
        q = (S.randn(f.g, 1, n_q, 8, 128) * 1.5).to(BF)
        ws.fill_(255)
        out = F.fasa_attend_prompt(f.cache, f.seq_len, q, 3000, window=window, n_sink=3, workspace=ws)
        ref, _, size, z = S.attend64(f, 0, q[0], list(range(3000 - n_q, 3000)), window, 3, False)
        S.check_out(out[0], ref, size, z, 3000, p_rel=2.0 ** -8)
