"""The operators' Python calls refuse tensors that are spread over two GPUs, by
their name and before anything is launched.  Shapes, types and devices without
memory stand in for the tensors, so no GPU is needed."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

R, C = 4, 64
Q4, S4, S8 = (R, 32), (512,), (R, 2)
BF, U8, F8, F32, I32 = torch.bfloat16, torch.uint8, torch.float8_e4m3fn, torch.float32, torch.int32

# name -> arguments in order: (name, shape, type) for a tensor; others as they are; a list: a pair
CALLS = {
    "fp4_quant_mx": [("x", (R, C), BF), ("q", Q4, U8), ("scales", S4, U8), ("qt", (C, 16), U8), ("scales_t", S4, U8),
                     ("skip_if", (1,), I32)],
    "fp4_dequant_mx": [("q", Q4, U8), ("scales", S4, U8), ("out", (R, C), BF)],
    "fp4_product_mx": [("a", Q4, U8), ("a_scales", S4, U8), ("b", Q4, U8), ("b_scales", S4, U8), C,
                       ("out", (R, R), BF)],
    "amp_layer_norm_forward": [("x", (R, C), BF), ("weight", (C,), F32), ("weight", (C,), F32), 1e-5,
                               ("y", (R, C), BF), ("mean", (R,), F32), ("rstd", (R,), F32),
                               [("saved", (R, C), F8), ("saved", S8, U8)]],
    "amp_layer_norm_backward": [("dy", (R, C), BF), None, ("weight", (C,), F32), ("mean", (R,), F32),
                                ("rstd", (R,), F32), ("dx", (R, C), BF), ("weight", (C,), F32),
                                ("weight", (C,), F32), ("workspace", (1 << 16,), U8),
                                [("saved", (R, C), F8), ("saved", S8, U8)]],
    "amp_act_forward_mx8": [("x", (R, C), BF), "silu", ("y", (R, C), BF), [("saved", (R, C), F8), ("saved", S8, U8)],
                            ("up", (R, C), BF), [("saved_up", (R, C), F8), ("saved_up", S8, U8)]],
    "amp_act_backward_mx8": [("dy", (R, C), BF), "silu", [("saved", (R, C), F8), ("saved", S8, U8)],
                             ("dx", (R, C), BF), [("saved_up", (R, C), F8), ("saved_up", S8, U8)],
                             ("dup", (R, C), BF)],
    "amp_ckpt8_save": [("x", (R, C), BF), ("q", (R, C), F8), ("scales", S8, U8)],
    "amp_ckpt8_restore": [("q", (R, C), F8), ("scales", S8, U8), ("out", (R, C), BF)],
}
# the tensor that gives the call its device
SHAPES = {"fp4_dequant_mx": "out", "fp4_product_mx": "out", "amp_ckpt8_restore": "out"}


def flat(args):
    return [t for a in args for t in (a if isinstance(a, list) else [a]) if isinstance(t, tuple)]


@pytest.fixture(scope="module")
def G():
    from loss_scaling_master_gb300 import build as B
    B.build()
    import loss_scaling_master_gb300 as pkg
    return pkg


@pytest.mark.parametrize("name", CALLS)
def test_a_tensor_on_another_gpu_is_refused(G, name):
    args = CALLS[name]
    tensors = flat(args)
    main = SHAPES.get(name, tensors[0][0])
    for odd in range(len(tensors)):
        place = iter(range(len(tensors)))
        with FakeTensorMode():
            def make(a):
                if isinstance(a, list):
                    return tuple(make(t) for t in a)
                if not isinstance(a, tuple):
                    return a
                dev = "cuda:1" if next(place) == odd else "cuda:0"
                return torch.empty(a[1], dtype=a[2], device=dev)
            call = [make(a) for a in args]
            # the shape's own tensor aside from the others shows as the first of those
            who = tensors[odd][0]
            match = "on cuda:0, the call is on cuda:1" if who == main else f"{who}: on cuda:1, the call is on cuda:0"
            with pytest.raises(ValueError, match=match):
                getattr(G, name)(*call)
