"""Tensors that are not on the current device are refused before anything looks
at their data (stand-ins without data take the place of another GPU's)."""
import pytest
import torch

import tensor_bf16_gemm_amd as gc

pytestmark = pytest.mark.gpu


class Elsewhere(torch.Tensor):
    """A tensor of cuda:1 without data (no call reaches that device)."""
    @staticmethod
    def __new__(cls, shape, dtype):
        return torch.Tensor._make_wrapper_subclass(cls, shape, dtype=dtype, device="cuda:1")

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise AssertionError(f"{func} looks at the tensor")


BF, I32 = torch.bfloat16, torch.int32
CALLS = [
    (gc.moe_route, [("logits", (4, 8), torch.float32), 2]),
    (gc.group_rows, [("ids", (4, 2), I32), 5]),
    (gc.grouped_gemm, [("X", (4, 16), BF), ("W", (2, 16, 32), BF), ("offsets", (3,), I32), ("rows", (6,), I32),
                       ("out", (6, 32), BF)]),
    (gc.moe_combine, [("Y", (6, 16), BF), ("slots", (4, 2), I32), ("weights", (4, 2), torch.float32), None,
                      ("out", (4, 16), BF)]),
    (gc.lora_add, [("base", (4, 32), BF), ("X", (4, 16), BF), ("down", (2, 16, 8), BF), ("up", (2, 8, 32), BF),
                   ("scale", (2,), torch.float32), ("offsets", (3,), I32), ("rows", (4,), I32),
                   ("out", (4, 32), BF)])]


@pytest.mark.parametrize("call,args,which", [(c, a, x[0]) for c, a in CALLS for x in a if isinstance(x, tuple)])
def test_tensors_of_another_device_are_refused(call, args, which):
    def make(x):
        if not isinstance(x, tuple):
            return x
        if x[0] != which:
            return torch.zeros(x[1], dtype=x[2], device="cuda")
        return Elsewhere(x[1], x[2])
    with pytest.raises(ValueError, match=f"{which} is on cuda:1"):
        call(*[make(x) for x in args])


def test_workspace_of_another_device_is_refused():
    ws = Elsewhere((1 << 27,), torch.uint8)
    with pytest.raises(ValueError, match="workspace is on cuda:1"):
        gc.group_rows(torch.zeros(4, dtype=I32, device="cuda"), 2, workspace=ws)
