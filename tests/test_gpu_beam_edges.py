"""GPU: beam selection where it can go wrong: ties across the splits of a row, values beyond
float32's range."""
import numpy as np
import pytest
import torch

import beam_ref as BR
import label_ref as R
from rnn_transducer_loss_gb300 import rnnt_beam_select

pytestmark = pytest.mark.gpu
DT = R.DTYPES


def check(x, scores, want, beam, fused=True):
    """Against the first `beam` places of `want`."""
    got = rnnt_beam_select(x, scores, beam, fused_log_softmax=fused)
    want = [w[:, :beam] for w in want]
    np.testing.assert_array_equal(got[2].cpu().numpy(), want[2])
    np.testing.assert_array_equal(got[1].cpu().numpy(), want[1])
    s = R.f64(got[0])
    left = np.isinf(want[0])
    assert (s[left] == -np.inf).all()
    assert (np.abs(s - want[0])[~left] <= R.score_bound(want[0], fused)[~left]).all()


@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("B,K,V", [(1, 1, 20001), (1, 4, 50257), (2, 17, 1003), (3, 20, 4099)])
def test_ties_across_splits(B, K, V, dtype, fused):
    """Equal logits in different splits, among them the elements behind the last whole 16 bytes:
    the lowest token first, also where the tie stands at the last place; misaligned rows too."""
    x = torch.zeros(B, K, V + 9, dtype=DT[dtype], device="cuda")
    scores = torch.full((B, K), -2.0, device="cuda")
    scores[:, 0] = -1.0                             # one hypothesis ahead of equal ones
    for at in ([V // 2, V - 1], [9, V // 2, 3 * V // 4, V - 1], [0, V - 2, V - 1]):
        for skip in (0, 1, 5):
            y = x[:, :, skip:skip + V]
            y.zero_()
            y[:, :, at] = 5.0
            if skip == 0:
                want = R.select(R.f64(y), R.f64(scores), 64, None, fused)
            for beam in (1, len(at) - 1, len(at), len(at) + 3, 64):
                check(y, scores, want, beam, fused)


@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K,V", [(1, 2), (4, 9), (3, 700), (4, 20001), (18, 70), (20, 4099)])
def test_beyond_float32(K, V, dtype, fused):
    """Scores and logits whose sums leave float32's range, by one launch and by two with one split
    and several: the order is that of the values, which come back as infinite; three steps on the
    scores that came back."""
    for x, scores in BR.far_cases(DT[dtype], K, V, K):
        for _ in range(3):
            got = rnnt_beam_select(x[None].cuda(), torch.as_tensor(scores[None]).cuda(),
                                   fused_log_softmax=fused, check=not (scores == np.inf).any())
            want = BR.select(x.double().numpy(), scores, K, fused)
            s, tokens, parents = (t[0].cpu().numpy() for t in got)
            np.testing.assert_array_equal(parents, want[2])
            np.testing.assert_array_equal(tokens, want[1])
            assert BR.score_error(s, want[0], fused) <= 0
            scores = s


@pytest.mark.parametrize("V", [12, 20001])
def test_masked_two_steps(V):
    """A search whose mask leaves two outputs to four hypotheses: what is masked comes last."""
    x = torch.full((2, 4, V), torch.finfo(torch.float32).min, device="cuda")
    x[:, :, 3], x[:, :, V - 1] = 1.0, 0.5
    scores = torch.full((2, 4), float("-inf"), device="cuda")
    scores[:, 0] = 0.0
    for step in range(3):
        scores, tokens, parents = rnnt_beam_select(x, scores)
        allowed = min(4, 2 ** (step + 1))
        assert (scores[:, :allowed] > -10).all() and not scores.isnan().any()
        assert ((tokens[:, :allowed] == 3) | (tokens[:, :allowed] == V - 1)).all()
        assert (scores[:, allowed:] < -3e38).all()
