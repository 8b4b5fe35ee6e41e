"""What include/qsa.h promises of the 8-bit cache calls' arguments, seen from C (no GPU needed)."""
import pytest

import sparse_attention_block_qsa_b200 as qsa
from test_kv8_refusals import A, ALIGN, INVALID, OK, S, UNSUP, WS, append, attn

REFUSALS = (INVALID, ALIGN, UNSUP, WS)


@pytest.mark.parametrize("name", ["qsa_sparse_attention_fp8", "qsa_sparse_attention_fp8_f16"])
@pytest.mark.parametrize("weights", [None, A + 11 * S])
def test_a_call_with_empty_lists_takes_the_workspace_that_its_size_says(name, weights):
    """Without lists the size is 0, and the call takes that: without a GPU it gets as far as CUDA's error."""
    assert qsa.lib().qsa_sparse_attention_fp8_workspace_size(8, 24, 2, 0, 1 if weights else 0) == 0
    st, detail = attn(name, width=0, tok=None, w=weights, ws=None, nbytes=0)
    assert st not in REFUSALS, (st, detail)
