"""Training attention whose keys are split over workgroups, over ragged rows
that leave whole splits without keys, in sizes without 16-byte rows."""

import pytest
import torch

from gpu_util import log
from test_gpu_attention import DTYPES, IDS, _case, _check

pytestmark = pytest.mark.gpu

pytest.importorskip("gru_sequence_scan_amd")


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("Tq,Tk,B,heads,kv,D", [(1, 4100, 5, 2, 1, 33), (3, 3000, 4, 2, 2, 127), (40, 2500, 3, 2, 1, 66),
                                               (1, 2000, 6, 4, 2, 5), (70, 1500, 2, 2, 1, 101)])
def test_ragged_splits(Tq, Tk, B, heads, kv, D, dtype):
    log(f"attention splits Tq {Tq} Tk {Tk} B {B} heads {heads}/{kv} D {D} {dtype}")
    lengths = [(Tk, 0, 1, 130, Tk // 2 + 1, Tk - 1)[b] for b in range(B)]
    if B == 2:
        lengths = [3, Tk]
    q, k, v, do = _case(Tq, Tk, B, heads, kv, D, dtype, D)
    dev = torch.tensor(lengths, dtype=torch.int32, device="cuda")

    def dirty(t):
        out = t.cuda()
        if t.shape[0] == Tk:
            for b, n in enumerate(lengths):
                out[n:, b] = float("nan")
        return out

    _check(q, k, v, do, lengths, dev=dev, put=dirty, what="splits")
