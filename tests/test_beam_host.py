"""The selection's workspace where the device's clusters are small."""
import pytest
import torch

from rnn_transducer_loss_gb300 import _native as N
from rnn_transducer_loss_gb300 import build as B


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return N.load()


def select(K, workspace, nbytes):
    return N.rnnt_beam_select(1 << 20, N.RNNT_F32, 2, K, 30, 30 * K, 30, 4096, None, 4, 1, 8192,
                              8448, 8704, workspace, nbytes, None, None)


@pytest.mark.skipif(torch.cuda.is_available(), reason="for no device to ask")
@pytest.mark.parametrize("K", [9, 12, 16])
def test_workspace_without_large_clusters(K):
    """Only clusters of 8 blocks run everywhere: with more hypotheses the size has to be that of
    the two launches, and the call has to want it."""
    n = N.rnnt_beam_workspace_size(2, K, 30, 4, N.RNNT_F32)
    assert n > 0 and n % 256 == 0
    assert select(K, None, 0) == N.RNNT_INVALID_VALUE
    assert select(K, 1 << 21, n - 1) == N.RNNT_WORKSPACE_TOO_SMALL
    assert N.rnnt_beam_workspace_size(2, 8, 30, 4, N.RNNT_F32) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("K,wanted", [(8, False), (9, False), (16, False), (17, True)])
def test_workspace(K, wanted):
    """On the whole device clusters of 16 blocks run."""
    assert (N.rnnt_beam_workspace_size(2, K, 30, 4, N.RNNT_F32) > 0) == wanted


@pytest.mark.parametrize("name", ["rnnt_embed", "rnnt_embed_grad", "rnnt_beam_select",
                                  "rnnt_beam_reorder"])
def test_entry_points_are_the_library_s(name):
    """What the package calls, and the tests of refusals with it, is the library's function itself."""
    assert getattr(N, name) is getattr(N.load(), name)
    with pytest.raises(AttributeError):
        N.rnnt_no_such_name
