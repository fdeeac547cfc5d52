"""The native calls leave alone what is not a plain call on a GPU: None, and no error set."""

import pytest
import torch

from gated_delta_rule_40_amd import binding

native = binding._native
pytestmark = pytest.mark.skipif(native is None, reason="_marshal.so is not built")

X = torch.randn(2, 256)
CODES, SCALES = torch.zeros(2, 256, dtype=torch.uint8), torch.zeros(2, 2)
POS, FREQ = torch.zeros(1, dtype=torch.int32), torch.zeros(8, dtype=torch.float64)
Q = torch.zeros(1, 2, 1, 64)


@pytest.mark.parametrize("name, args", [
    ("rms_norm", ()),
    ("rms_norm", (X, None, X.clone(), None, None, None, None, False, None, 1e-6)),
    ("rms_norm", (None,) * 10),
    ("rms_norm", (X.to_sparse(), None, X, None, None, None, None, False, None, 1e-6)),
    ("rms_norm", (X.to("meta"), None, X, None, None, None, None, False, None, "eps")),
    ("rms_norm", ("x",) * 10),
    ("quant_rows", ()),
    ("quant_rows", (X, CODES, SCALES)),
    ("quant_rows", (X, None, None)),
    ("quant_rows", (3, 4, 5)),
    ("matmul_fp8", (CODES, SCALES, CODES, SCALES, X, None)),
    ("matmul_fp8", (None,) * 6),
    ("matmul_fp8", (1,)),
    ("rope", (Q.view(1, 2, 64), FREQ, POS, Q, Q, None, False, 1.0, None)),
    ("rope", (None,) * 9),
    ("rope", (X,) * 9),
])
def test_calls_that_are_not_plain(name, args):
    assert getattr(native, name)(*args) is None


@pytest.mark.parametrize("args", [(), (1, 2, 3, 4, 5), (1.5, 2, 3, 4, None, None)])
def test_bind_refuses_what_is_no_address(args):
    with pytest.raises(TypeError):
        native.bind(*args)
