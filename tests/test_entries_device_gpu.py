"""Forks and renames run on the engine's device, whichever is current, and on streams of that device alone;
an attention of an engine in the static workspace takes tensors of its device alone."""

import numpy as np
import pytest

from test_entries_gpu import Model

pytestmark = pytest.mark.gpu


class Elsewhere:
    def __init__(self):
        import torch
        self.cuda_stream, self.device = 0, torch.device("cuda", 1)


@pytest.mark.parametrize("static", [False, True])
def test_streams_of_another_device_are_refused(static):
    import torch
    m = Model(31, static_workspace=static)
    try:
        assert m.eng.device == torch.device("cuda", 0)
        m.append(np.arange(20))
        for call in (m.eng.fork, m.eng.rename):
            with pytest.raises(ValueError, match="stream"):
                call(0, 0, 100, 5, stream=Elsewhere())
        m.same("after the refusals", True)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        m.eng.fork(0, 0, 100, 5, stream=side)
        m.eng.rename(0, 100, 120, 5, stream=side.cuda_stream)
        torch.cuda.current_stream().wait_stream(side)
        m.ora.append(np.arange(100, 105), np.stack([m.rows[a] for a in range(5)]))
        m.rows.update((100 + i, m.rows[i]) for i in range(5))
        eng, m.eng = m.eng, type("Done", (), {"rename": lambda *a: None})()   # the oracle's side alone
        m.rename(100, 120, 5)
        m.eng = eng
        m.same("end", True)
        m.eng.sync()
    finally:
        m.close()
