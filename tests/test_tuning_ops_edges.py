"""The fine-tuning operators' refusals where the sizes are easily taken for nothing, without a GPU.

Arguments are checked before any device work; the addresses are never dereferenced."""
import pytest

from mixed_precision_optimizer_bf16_gb300 import bf16opt as C
from mixed_precision_optimizer_bf16_gb300 import build as B
from test_tuning_ops import A, ALIGN, INVALID, has_gpu, status, tokens


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return C.load()


def test_preference_outputs_of_no_rows():
    """Pairs of empty sequences have losses and sums, which overlap neither each other nor what is read."""
    d, q = tokens(rows=0, logits=None, labels=None, row_weight=None), C.bf16opt_preference_t(2, 1, 0, A[10], A[11], 0.1, 0.0, 0.0, 0)
    for loss, logp in ((A[10] + 36, A[4]), (A[11] + 12, A[4]), (A[3], A[10]), (A[3], A[11])):
        status(C.bf16opt_preference_forward(d, q, loss, logp, None), INVALID, "overlaps an input")
    status(C.bf16opt_preference_forward(d, q, A[3], A[3] + 4, None), INVALID, "two outputs")
    status(C.bf16opt_preference_forward(d, q, A[3], A[4] + 2, None), ALIGN)
    if not has_gpu():   # what is allowed comes as far as the device
        status(C.bf16opt_preference_forward(d, q, A[3], A[4], None), C.BF16OPT_ERR_UNSUPPORTED)
        status(C.bf16opt_preference_forward(d, q, A[3], A[3] + 8, None), C.BF16OPT_ERR_UNSUPPORTED)
