"""lb_kv_plan refuses outputs that lie over its inputs, on the host, before anything is written."""
import numpy as np
import pytest
import torch

import bit_matvec_lb_gb300 as lb

pytestmark = pytest.mark.gpu

INPUTS = ("past", "fresh", "free_pages", "free_from")
OUTPUTS = ("block_table", "q_start", "kv_len", "position", "slot", "counts")


def buffers():
    i32 = dict(dtype=torch.int32, device="cuda")
    words = torch.arange(4096, **i32)
    at = dict(past=0, fresh=64, free_pages=128, free_from=192, block_table=256, q_start=384, kv_len=448,
              position=512, slot=576, counts=704)
    return words, {k: words.data_ptr() + 4 * v for k, v in at.items()}


def plan(a):
    """Three requests, eight free pages, four tokens, a table of eight columns."""
    lb.lb_kv_plan(a["past"], a["fresh"], 3, a["free_pages"], 8, a["free_from"], 16, a["block_table"], 8, 4,
                  a["q_start"], a["kv_len"], a["position"], a["slot"], a["counts"])


@pytest.mark.parametrize("output", OUTPUTS)
@pytest.mark.parametrize("source", INPUTS)
def test_outputs_over_inputs(source, output):
    """At the same address, and with the output's last bytes on the input's first ones."""
    size = dict(block_table=96, q_start=16, kv_len=12, position=16, slot=32, counts=8)[output]
    for shift in (0, 8 - size if output == "slot" else 4 - size):
        words, a = buffers()
        before = words.clone()
        a[output] = a[source] + shift
        with pytest.raises(lb.LBError) as e:
            plan(a)
        assert e.value.status == -3
        assert torch.equal(words, before)


def test_next_to_each_other():
    """Buffers that touch but do not overlap are taken."""
    words, a = buffers()
    words[0:3] = torch.tensor([0, 20, 5])
    words[64:67] = torch.tensor([1, 1, 2])
    words[192] = 0
    a["kv_len"] = a["past"] + 12
    plan(a)
    torch.cuda.synchronize()
    assert words[3:6].tolist() == [1, 21, 7] and np.array_equal(words[:3].cpu(), [0, 20, 5])
    assert words[384:388].tolist() == [0, 1, 2, 4]
