"""spec_process_logits with lists longer than what a CTA keeps of them: biases past
the shared list's 256, histories past the 1024 tokens in registers."""
import pytest
import torch

from test_gpu_rules import check, make, run

pytestmark = pytest.mark.gpu

CASES = {
    "biases, f32": dict(V=3000, rows=[3, 2], dtype=torch.float32, bias=900),
    "biases, bf16 odd": dict(V=2001, rows=[4, 1, 2], dtype=torch.bfloat16, bias=700, hist=100),
    "biases of two ranges": dict(V=20000, rows=[2, 3], dtype=torch.bfloat16, bias=2000),
    "biases, tree": dict(V=1024, rows=[20, 9], dtype=torch.float32, bias=600, tree=1),
    "history, f32": dict(V=1500, rows=[3, 4, 2], dtype=torch.float32, hist=6000),
    "history, bf16 odd": dict(V=30001, rows=[2, 3, 3], dtype=torch.bfloat16, hist=9000),
    "history, tree": dict(V=9000, rows=[30, 8, 1], dtype=torch.bfloat16, tree=1, hist=5000),
    "history of few tokens": dict(V=64, rows=[40, 33], dtype=torch.float32, hist=4000, repeat=True),
    "both, in segments": dict(V=4104, rows=[40, 18], dtype=torch.bfloat16, hist=3000, bias=1500),
}


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("name", CASES)
def test_long_lists(name, inplace):
    z, cu, c = make(len(name), **CASES[name])
    out = z.clone() if inplace else None
    check(z, cu, c, run(out if inplace else z, cu, c, out=out))
