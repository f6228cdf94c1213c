"""skinny_verify_draft where its contract ends: rows of the draft that it does not
ask for, drafts of vanishing probability, vocabularies of many trips."""
import ctypes

import pytest
import torch

import gemv_skinny_gemm_amd as sg
from tests.gpu_util import need_gpu
from tests.test_verify_gpu import case, compare, upload

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,temps,asked", [([3, 2], [0.9, 0.7], 4), ([3, 4], [0.9, 0.0], 2),
                                              ([4], [1.0], 3), ([5, 1, 1], [0.8], 4)])
def test_rows_of_the_draft_that_are_not_asked(dtype, rows, temps, asked):
    """The last row of a sequence, greedy sequences' rows and rows of no sequence
    need no draft logits: there are none behind the last row that is asked."""
    c = case(rows, 100003, dtype, seed=40, tail=2, temps=temps)
    d = upload(c)
    T, V = c["logits"].shape
    draft = d["draft"][:asked].clone()
    d["draft"] = None
    address = ctypes.c_void_p
    v = sg.Verify(sg.LOGITS_BF16 if dtype == "bf16" else sg.LOGITS_F32, V, T, len(rows),
                  *(address(t.data_ptr()) for t in (d["q_start"], d["logits"], draft, d["tokens"],
                                                    d["temperature"], d["accept_u"], d["sample_u"],
                                                    d["out"], d["accepted"])))
    assert sg.lib().skinny_verify_draft(v, d["ws"].data_ptr(), d["ws"].numel(), None) == 0
    torch.cuda.synchronize()
    compare(c, d)
