"""The selection's kernels from their source, run on the CPU, against the float64 form."""
import numpy as np
import pytest
import torch

import beam_ref as BR
import label_ref as R
import on_cpu
from rnn_transducer_loss_gb300 import _native as N

DT = R.DTYPES


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    return on_cpu.build(str(tmp_path_factory.mktemp("beam")))


def check(program, x, scores, beam, finished=None, fused=True, **how):
    got = on_cpu.select(program, x, scores, beam, finished, fused, **how)
    want = R.select(x.double().numpy()[None], np.asarray(scores, np.float32).astype(float)[None],
                    beam, None if finished is None else np.asarray(finished)[None], fused)
    np.testing.assert_array_equal(got[2], want[2][0])
    np.testing.assert_array_equal(got[1], want[1][0])
    left = np.isinf(want[0][0])
    assert (got[0][left] == -np.inf).all() and got[3] == 0
    assert (np.abs(got[0][~left] - want[0][0][~left]) <= R.score_bound(want[0][0][~left], fused)).all()


@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("K,V,beam,splits", [
    (1, 5, 8, 0), (4, 1024, 4, 0), (3, 1001, 7, 0), (2, 3001, 64, 3), (20, 70, 20, 0), (5, 515, 9, 2)])
def test_select(program, K, V, beam, splits, dtype, fused):
    """One cluster, and two launches with one split and several; every alignment of a row."""
    g = torch.Generator().manual_seed(V + K)
    x = (torch.randn(K, V, generator=g) * 3).to(DT[dtype])
    if not fused:
        x = torch.log_softmax(x.float(), -1).to(x.dtype)
    scores = -20 + 10 * np.random.default_rng(V).random(K)
    for skip in (0, 1, 3):
        check(program, x, scores, beam, None, fused, splits=splits, skip=skip)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("V,splits", [(1003, 3), (20001, 0), (517, 4), (1037, 7)])
def test_ties_across_splits(program, V, splits, dtype):
    """Equal logits in different splits, among them the elements behind the last whole 16 bytes:
    the lowest token first, also where the tie stands at the last place."""
    for skip in (0, 1, 2) if V < 20000 else (2,):
        for at in ([V // 2, V - 1], [9, V // 2, 3 * V // 4, V - 1], [0, V - 2, V - 1]):
            x = torch.zeros(1, V, dtype=DT[dtype])
            x[0, at] = 5.0
            for beam in (1, len(at) - 1, len(at), len(at) + 3):
                check(program, x, [0.0], beam, splits=splits, skip=skip)
    x = torch.zeros(3, V, dtype=DT[dtype])          # nothing but ties, of hypotheses too
    x[1:, -3:] = 1.0
    check(program, x, [-1.0, -1.0, -1.0], 16, fused=False, splits=splits or 3)


@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K,V,splits", [(4, 9, 0), (3, 700, 0), (4, 1003, 3), (18, 70, 0)])
def test_beyond_float32(program, K, V, splits, dtype, fused):
    """Scores and logits whose sums leave float32's range: the order is that of the values, which
    come back as infinite; three steps on the scores that came back."""
    for x, scores in BR.far_cases(DT[dtype], K, V, K):
        for _ in range(3):
            got = on_cpu.select(program, x, scores, K, None, fused, splits=splits)
            want = BR.select(x.double().numpy(), scores, K, fused)
            np.testing.assert_array_equal(got[2], want[2])
            np.testing.assert_array_equal(got[1], want[1])
            assert BR.score_error(got[0], want[0], fused) <= 0
            bad = (scores == np.inf).any()
            assert got[3] == (1 if bad else 0)
            scores = got[0]


@pytest.mark.parametrize("K,V,beam,splits", [(1, 5, 8, 0), (4, 40, 4, 0), (20, 70, 20, 0), (3, 515, 9, 3)])
def test_selection_without_a_winner(program, K, V, beam, splits):
    """The lists' best is always some lane's.  Were it none's, nothing may be indexed by it: the
    places are left over and the status says so."""
    x = torch.randn(K, V, generator=torch.Generator().manual_seed(V))
    scores, tokens, parents, status = on_cpu.select(program, x, np.zeros(K), beam, splits=splits,
                                                    plant=on_cpu.NO_MINIMUM)
    assert status == N.RNNT_LAUNCH_FAILED
    assert (scores == -np.inf).all() and (tokens == -1).all() and (parents == -1).all()


@pytest.mark.parametrize("K", [8, 9, 16])
def test_without_large_clusters(program, K):
    """The two launches in the place of a cluster of more than 8 blocks: the same results."""
    x = torch.randn(K, 301, generator=torch.Generator().manual_seed(K))
    x[1] = x[0]
    scores = np.repeat(-np.arange(K // 2 + 1), 2)[:K]
    check(program, x, scores, 11, splits=-1)
    for a, b in zip(on_cpu.select(program, x, scores, 11, splits=-1),
                    on_cpu.select(program, x, scores, 11)):
        np.testing.assert_array_equal(a, b)
